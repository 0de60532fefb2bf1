"""The block's norms with gate and residual, forward and backward, against the 64-bit definition."""
import numpy as np
import pytest
import torch

import block_ref as ref

pytestmark = pytest.mark.gpu
EPS = 1e-6


def make(T, H, rt, gate, seed=0, y=True):
    g = torch.Generator(device="cuda").manual_seed(seed)
    n = lambda *s, std=1.0: torch.randn(*s, generator=g, device="cuda") * std
    bf = torch.bfloat16
    shape = dict(none=None, channel=(H,), token=(T,), full=(T, H))[gate]
    return dict(r=n(T, H, std=2.0).to(rt), y=n(T, H, std=0.3).to(bf) if y else None,
                w_post=(1 + n(H, std=0.2)).to(bf) if y else None, w_pre=(1 + n(H, std=0.2)).to(bf),
                g=n(*shape).to(bf) if shape else None, dr_out=n(T, H).to(rt), du=n(T, H).to(bf))


def kind_of(fe, gate, sigmoid):
    k = dict(none=fe.GATE_NONE, channel=fe.GATE_CHANNEL, token=fe.GATE_TOKEN, full=fe.GATE_FULL)[gate]
    return k | (fe.GATE_SIGMOID if sigmoid and gate != "none" else 0)


def check_forward(fe, c, gate, sigmoid, s=0.5, eps=EPS):
    r2, u = fe.block_norm(c["r"], c["y"], c["w_post"], c["w_pre"], gate=c["g"], gate_kind=kind_of(fe, gate, sigmoid), scale=s, eps=eps)
    want = ref.norm_forward(c["r"], c["y"], c["w_post"], c["w_pre"], c["g"], gate, sigmoid, s, eps)
    if r2 is not None:
        ref.close(r2, want["r_out"][0], ref.FWD * want["r_out"][1], "r_out")
    if u is not None:
        ref.close(u, want["u"][0], ref.FWD * want["u"][1], "u")


def check_backward(fe, c, gate, sigmoid, s=0.5, eps=EPS):
    got = fe.block_norm_backward(c["dr_out"], c["du"], c["r"], c["y"], c["w_post"], c["w_pre"], gate=c["g"],
                                 gate_kind=kind_of(fe, gate, sigmoid), scale=s, eps=eps)
    want = ref.norm_backward(c["dr_out"], c["du"], c["r"], c["y"], c["w_post"], c["w_pre"], c["g"], gate, sigmoid, s, eps)
    for name, t in zip(("dr", "dy", "dgate", "dw_post", "dw_pre"), got):
        assert (t is None) == (name not in want), name
        if t is not None:
            ref.close(t, want[name][0], ref.BWD * want[name][1], name)
    return got


SHAPES = [(1, 1), (1, 2048), (2, 8), (3, 64), (5, 7), (7, 1999), (33, 256), (4, 257), (130, 2048), (9, 4096), (3, 8192), (2, 8200), (2, 16384),
          (300, 40), (1, 16383)]


@pytest.mark.parametrize("gate, sigmoid", [("none", False), ("channel", False), ("token", True), ("full", True), ("full", False), ("token", False), ("channel", True)])
@pytest.mark.parametrize("rt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T, H", SHAPES)
def test_forward_and_backward(T, H, rt, gate, sigmoid):
    import fp4_expert_gemv_b200 as fe
    c = make(T, H, rt, gate, seed=T + H)
    check_forward(fe, c, gate, sigmoid)
    check_backward(fe, c, gate, sigmoid)


@pytest.mark.parametrize("drop", [("y", "w_post"), ("w_post",), ("w_pre", "du"), ("w_post", "w_pre", "du"), ("dr_out",)])
@pytest.mark.parametrize("gate", ["none", "token"])
def test_parts_left_out(drop, gate):
    import fp4_expert_gemv_b200 as fe
    if "y" in drop and gate != "none":
        return
    c = make(37, 520, torch.bfloat16, gate, seed=3)
    for name in drop:
        c[name] = None
    check_forward(fe, c, gate, True)
    check_backward(fe, c, gate, True)


def test_many_rows_walk_several_times():
    import fp4_expert_gemv_b200 as fe
    c = make(5003, 136, torch.bfloat16, "channel", seed=9)
    check_forward(fe, c, "channel", True)
    check_backward(fe, c, "channel", True)


@pytest.mark.parametrize("T, H, rt, gate", [(700, 4096, torch.bfloat16, "token"), (15001, 64, torch.float32, "full"),
                                            (2500, 512, torch.bfloat16, "full"), (1300, 2048, torch.bfloat16, "none"),
                                            (3700, 2048, torch.float32, "channel"), (320, 8192, torch.bfloat16, "channel")])
def test_streamed_rows(T, H, rt, gate):
    """Enough rows per group for the kernels that stream them, with a ragged last round."""
    import fp4_expert_gemv_b200 as fe
    c = make(T, H, rt, gate, seed=T)
    check_forward(fe, c, gate, True)
    check_backward(fe, c, gate, True)
    # the norm alone, and without its weight
    c["g"] = c["y"] = c["w_post"] = None
    check_forward(fe, c, "none", False)


@pytest.mark.parametrize("T, H", [(5, 256), (5, 255), (5003, 136), (15001, 64)])
@pytest.mark.parametrize("gate", ["none", "token", "channel", "full"])
def test_rows_where_the_residual_cancels(T, H, gate):
    """r' = r + s a v where r is -s a v but for a thousandth: the sum of squares of r' is a millionth of its
    parts, so an expansion into products of r and v alone would lose it.  The bound is the rows' own
    magnitudes' (the fp32 error of r' relative to |r| + |s a v|, through rho)."""
    import fp4_expert_gemv_b200 as fe
    c = make(T, H, torch.float32, gate, seed=31)
    zero = dict(c, r=torch.zeros_like(c["r"]))
    sav = ref.norm_forward(zero["r"], c["y"], c["w_post"], None, c["g"], gate, False, 0.5, EPS)["r_out"][0]
    c["r"] = (-sav + 1e-3 * torch.randn(T, H, device="cuda", dtype=torch.float64)).float()
    c["r"][::3] = torch.randn(T, H, device="cuda")[::3]         # other rows stay ordinary
    check_forward(fe, c, gate, False)
    check_backward(fe, c, gate, False)


def test_without_weight_gradients():
    import fp4_expert_gemv_b200 as fe
    for H in (512, 511):
        c = make(70, H, torch.bfloat16, "channel", seed=2)
        args = (c["dr_out"], c["du"], c["r"], c["y"], c["w_post"], c["w_pre"])
        kw = dict(gate=c["g"], gate_kind=fe.GATE_CHANNEL, scale=0.5)
        full, part = fe.block_norm_backward(*args, **kw), fe.block_norm_backward(*args, weight_grads=False, **kw)
        assert torch.equal(full[0], part[0]) and torch.equal(full[1], part[1]) and part[2:] == (None, None, None)


@pytest.mark.parametrize("H", [8, 136, 255, 2048, 4096, 9000])
def test_the_workspace_is_all_that_is_written(H):
    """The bytes behind the workspace and the sums over rows are watched, from one row to many per group."""
    import fp4_expert_gemv_b200 as fe
    for T in (1, 3, 147, 149, 297, 513, 1300):
        c = make(T, H, torch.bfloat16, "channel", seed=T)
        nb = fe.fe_moe_block_norm_workspace(T, H)
        ws = torch.full((nb + 4096,), 85, dtype=torch.uint8, device="cuda")
        dr, dy = torch.full((2, T * H + 64), 5.0, dtype=torch.bfloat16, device="cuda")
        sums = torch.full((3, H + 64), 5.0, device="cuda")
        st = fe.fe_moe_block_norm_backward(c["dr_out"].data_ptr(), c["du"].data_ptr(), c["r"].data_ptr(), fe.DTYPE_BF16,
                                           c["y"].data_ptr(), c["w_post"].data_ptr(), c["g"].data_ptr(), fe.GATE_CHANNEL, 0.5,
                                           c["w_pre"].data_ptr(), EPS, T, H, dr.data_ptr(), dy.data_ptr(), sums[0].data_ptr(),
                                           sums[1].data_ptr(), sums[2].data_ptr(), ws.data_ptr(), nb,
                                           torch.cuda.current_stream().cuda_stream)
        torch.cuda.synchronize()
        assert st == fe.FE_OK and (ws[nb:] == 85).all() and (sums[:, H:] == 5).all(), (T, H)
        assert (dr[T * H:] == 5).all() and (dy[T * H:] == 5).all()


def test_unaligned_rows():
    """A width of whole chunks whose rows start 2 bytes off take the narrow accesses."""
    import fp4_expert_gemv_b200 as fe
    c = make(11, 512, torch.bfloat16, "none", seed=4)
    buf = torch.empty(11 * 512 + 1, dtype=torch.bfloat16, device="cuda")
    odd = buf[1:].view(11, 512)
    odd.copy_(c["y"])
    c["y"] = odd
    check_forward(fe, c, "none", False)
    check_backward(fe, c, "none", False)


def test_extreme_rows():
    """Zero rows, huge and tiny rows, a NaN row and an infinite row stay in their rows."""
    import fp4_expert_gemv_b200 as fe
    for H in (256, 255):
        c = make(8, H, torch.float32, "token", seed=5)
        c["r"][0] = 0
        c["y"][0] = 0
        c["y"][1] = 0
        c["r"][2] *= 1e15
        c["y"][3] *= 1e-15
        c["y"][4, 3] = float("nan")
        c["r"][5, 1] = float("inf")
        r2, u = fe.block_norm(c["r"], c["y"], c["w_post"], c["w_pre"], gate=c["g"], gate_kind=fe.GATE_TOKEN, scale=0.5, eps=EPS)
        keep = [0, 1, 2, 3, 6, 7]
        want = ref.norm_forward(c["r"], c["y"], c["w_post"], c["w_pre"], c["g"], "token", False, 0.5, EPS)
        ref.close(r2[keep], want["r_out"][0][keep], ref.FWD * want["r_out"][1][keep], "r_out")
        ref.close(u[keep], want["u"][0][keep], ref.FWD * want["u"][1][keep], "u")
        assert torch.isnan(u[4]).all() and torch.isnan(r2[4]).all()
        # 1 / rms of the infinite row is 0: 0 where r' is finite, inf * 0 where it is not
        assert torch.isnan(u[5, 1]) and (u[5, 2:] == 0).all()


def test_in_place_and_untouched_rows():
    import fp4_expert_gemv_b200 as fe
    c = make(9, 192, torch.bfloat16, "none", seed=6)
    want, wu = fe.block_norm(c["r"], c["y"], c["w_post"], c["w_pre"], scale=0.5)
    buf = torch.full((12, 192), 7.0, dtype=torch.bfloat16, device="cuda")
    buf[:9] = c["r"]
    r, u = fe.block_norm(buf[:9], c["y"], c["w_post"], c["w_pre"], scale=0.5, r_out=buf[:9])
    assert torch.equal(r, want) and torch.equal(u, wu) and (buf[9:] == 7).all()


def test_no_rows():
    import fp4_expert_gemv_b200 as fe
    c = make(0, 64, torch.bfloat16, "channel")
    r2, u = fe.block_norm(c["r"], c["y"], c["w_post"], c["w_pre"], gate=c["g"], gate_kind=fe.GATE_CHANNEL)
    assert r2.shape == (0, 64) and u.shape == (0, 64)
    got = fe.block_norm_backward(c["dr_out"], c["du"], c["r"], c["y"], c["w_post"], c["w_pre"], gate=c["g"], gate_kind=fe.GATE_CHANNEL)
    assert all((t == 0).all() for t in got[2:])


def test_the_same_every_time_and_on_another_stream():
    import fp4_expert_gemv_b200 as fe
    c = make(2000, 1024, torch.bfloat16, "channel", seed=8)
    args = (c["dr_out"], c["du"], c["r"], c["y"], c["w_post"], c["w_pre"])
    kw = dict(gate=c["g"], gate_kind=fe.GATE_CHANNEL | fe.GATE_SIGMOID, scale=0.7)
    first = fe.block_norm_backward(*args, **kw)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    two = [fe.block_norm_backward(*args, stream=side, **kw), fe.block_norm_backward(*args, **kw),
           fe.block_norm_backward(*args, stream=side.cuda_stream, **kw)]
    torch.cuda.synchronize()
    for got in two:
        assert all(torch.equal(a, b) for a, b in zip(first, got))


def test_captured_and_replayed_on_new_contents():
    import fp4_expert_gemv_b200 as fe
    c = make(64, 768, torch.float32, "full", seed=1)
    kw = dict(gate=c["g"], gate_kind=fe.GATE_FULL | fe.GATE_SIGMOID, scale=0.5)

    def both():
        return (*fe.block_norm(c["r"], c["y"], c["w_post"], c["w_pre"], **kw),
                *fe.block_norm_backward(c["dr_out"], c["du"], c["r"], c["y"], c["w_post"], c["w_pre"], **kw))

    both()
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = both()
        graphs.append((g, out))
    c2 = make(64, 768, torch.float32, "full", seed=2)
    for k in ("r", "y", "w_post", "w_pre", "g", "dr_out", "du"):
        c[k].copy_(c2[k])
    for g, _ in graphs:
        g.replay()
    eager = both()
    torch.cuda.synchronize()
    for _, out in graphs:
        assert all(torch.equal(a, b) for a, b in zip(out, eager))


@pytest.mark.parametrize("gate", ["channel", "token", "full"])
def test_gradient_against_differences(gate):
    """<gradient, direction> against central differences of the 64-bit definition.  The step error is
    h^2 / 6 of the third derivative: with h = 1e-4 and terms of order one, below 1e-6 of the sums; the
    kernel's bf16 outputs dr, dy, dgate are off by 2^-8 per element, which their own magnitude bounds."""
    import fp4_expert_gemv_b200 as fe
    c = make(6, 96, torch.float32, gate, seed=12)
    s = 0.6
    got = dict(zip(("r", "y", "g", "w_post", "w_pre"),
                   fe.block_norm_backward(c["dr_out"], c["du"], c["r"], c["y"], c["w_post"], c["w_pre"], gate=c["g"],
                                          gate_kind=kind_of(fe, gate, True), scale=s)))

    def loss(v):
        o = ref.norm_forward(v["r"], v["y"], v["w_post"], v["w_pre"], v["g"], gate, True, s, 1e-6)
        return float((o["r_out"][0] * c["dr_out"].double()).sum() + (o["u"][0] * c["du"].double()).sum())

    base = {k: c[k].double() for k in ("r", "y", "g", "w_post", "w_pre")}
    gen = torch.Generator(device="cuda").manual_seed(77)
    for name in base:
        dirn = torch.randn(base[name].shape, generator=gen, device="cuda", dtype=torch.float64)
        h = 1e-4
        num = (loss({**base, name: base[name] + h * dirn}) - loss({**base, name: base[name] - h * dirn})) / (2 * h)
        grad = got[name].double()
        tol = 2.0 ** -8 * float((grad * dirn).abs().sum()) + 1e-4
        assert abs(num - float((grad * dirn).sum())) <= tol, (name, num)


def test_refuses_other_layouts():
    import fp4_expert_gemv_b200 as fe
    c = make(8, 64, torch.bfloat16, "none")
    with pytest.raises(ValueError):
        fe.block_norm(c["r"].t().contiguous().t(), c["y"], c["w_post"], c["w_pre"])
    with pytest.raises(ValueError):
        fe.block_norm(c["r"], c["y"][:4], c["w_post"], c["w_pre"])
    with pytest.raises(ValueError):
        fe.block_norm(c["r"], c["y"].float(), c["w_post"], c["w_pre"])
    with pytest.raises(fe.FeMoeError):
        fe.block_norm(c["r"], c["y"], c["w_post"], c["w_pre"], eps=0.0)
    with pytest.raises(fe.FeMoeError):
        fe.block_norm(c["r"], c["y"], c["w_post"], c["w_pre"], u=c["y"])


def extremes(T, H, rt, gate, seed, finite=False):
    """make() with extreme rows at the start, in the middle and at the end; which rows are not finite."""
    c = make(T, H, rt, gate, seed=seed)
    bad = torch.zeros(T, dtype=torch.bool, device="cuda")
    for at in (0, T // 2, T - 9):
        c["r"][at] = 0                     # nothing at all: 1 / rms is eps^-1/2
        c["y"][at] = 0
        c["y"][at + 1] = 0
        c["r"][at + 2] *= 1e15
        c["y"][at + 3] *= 1e-15
        c["y"][at + 4] *= 1e17             # s a w_post y squared is beyond fp32, the norm of y and r' are not
        c["dr_out"][at + 5] *= 1e12        # a large gradient
        c["du"][at + 5] *= 1e12
        c["y"][at + 6] *= 1e15             # the same where dr' y and du y are beyond fp32 too, but no square
        c["dr_out"][at + 6] *= 1e22
        c["du"][at + 6] *= 1e22
        if not finite:
            c["y"][at + 7, H // 3] = float("nan")
            c["r"][at + 8, 1] = float("inf")
            bad[at + 7:at + 9] = True
    return c, bad


EXTREME = [(36, 256, torch.float32), (15001, 64, torch.float32), (4000, 1024, torch.bfloat16), (37, 255, torch.float32),
           (3001, 255, torch.bfloat16), (700, 2048, torch.float32), (1501, 4096, torch.bfloat16)]


@pytest.mark.parametrize("gate", ["none", "token", "channel", "full"])
@pytest.mark.parametrize("T, H, rt", EXTREME)
def test_extreme_rows_of_every_kernel(T, H, rt, gate):
    """Zero, huge, tiny, NaN and infinite rows stay in their rows forward and backward, whichever rows share a
    ring, a reduction or a block with them, and the finite ones keep the bounds of the others.  s = 512: products of
    y without its norm reach beyond fp32 where the outputs do not."""
    import fp4_expert_gemv_b200 as fe
    s = 512.0
    c, bad = extremes(T, H, rt, gate, seed=T)
    ok = ~bad
    kw = dict(gate=c["g"], gate_kind=kind_of(fe, gate, False), scale=s, eps=EPS)
    r2, u = fe.block_norm(c["r"], c["y"], c["w_post"], c["w_pre"], **kw)
    want = ref.norm_forward(c["r"], c["y"], c["w_post"], c["w_pre"], c["g"], gate, False, s, EPS)
    ref.close(r2[ok], want["r_out"][0][ok], ref.FWD * want["r_out"][1][ok], "r_out")
    ref.close(u[ok], want["u"][0][ok], ref.FWD * want["u"][1][ok], "u")
    nan, inf = bad.nonzero()[::2, 0], bad.nonzero()[1::2, 0]
    assert torch.isnan(u[nan]).all() and torch.isnan(r2[nan]).all()
    assert torch.isnan(u[inf, 1]).all() and (u[inf, 2:] == 0).all()   # 1 / rms is 0
    got = fe.block_norm_backward(c["dr_out"], c["du"], c["r"], c["y"], c["w_post"], c["w_pre"], weight_grads=False, **kw)
    want = ref.norm_backward(c["dr_out"], c["du"], c["r"], c["y"], c["w_post"], c["w_pre"], c["g"], gate, False, s, EPS)
    for name, t in zip(("dr", "dy", "dgate"), got):
        if t is not None:
            ref.close(t[ok], want[name][0][ok], ref.BWD * want[name][1][ok], name)
    assert fe.op_status() == (fe.FE_OK, 0)


@pytest.mark.parametrize("T, H, rt", EXTREME)
def test_sums_over_extreme_rows(T, H, rt):
    import fp4_expert_gemv_b200 as fe
    c, _ = extremes(T, H, rt, "channel", seed=T + 1, finite=True)
    check_backward(fe, c, "channel", False, s=512.0)
