"""The dense product with its epilogue, forward and backward, against the 64-bit definition."""
import pytest
import torch

import block_ref as ref

pytestmark = pytest.mark.gpu
bf = torch.bfloat16
ACTS = ["none", "relu", "gelu", "silu", "swiglu"]


def act_id(fe, act):
    return dict(none=fe.ACT_NONE, relu=fe.ACT_RELU, gelu=fe.ACT_GELU, silu=fe.ACT_SILU, swiglu=fe.ACT_SWIGLU)[act]


def make(M, N, K, act, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    n = lambda *s, std=1.0: (torch.randn(*s, generator=g, device="cuda") * std).to(bf)
    cols = N // 2 if act == "swiglu" else N
    return n(M, K), n(N, K, std=K ** -0.5), n(N, std=0.2), n(M, cols), n(M, cols)


def check_forward(fe, x, w, bias, act, res, y=None, z=None):
    out = fe.linear(x, w, bias=bias, act=act_id(fe, act), residual=res.clone() if res is not None else None, y=y, z=z)
    wy, wz, ey, ez = ref.linear(x, w, bias, act, res)
    ref.close(out, wy, ey, "y")
    if z is not None:
        ref.close(z, wz, ez, "z")
    assert fe.op_status() == (fe.FE_OK, 0)
    return out


def check_backward(fe, dy, x, w, z, act):
    dx, dw, db = fe.linear_backward(dy, x, w, z=z, act=act_id(fe, act))
    dz, mag = ref.linear_dz(dy, z if z is not None else dy, act)
    # dz enters the products rounded to bf16 (half a step, 2^-8 relative), then fp32 sums as forward
    edz = 2.0 ** -8 * dz.abs() + ref.FWD * mag
    X, W = x.double(), w.double()
    adz = dz.abs() + edz
    M, N = dz.shape
    ref.close(dx, dz @ W, edz @ W.abs() + (N / 16 + 4) * 2.0 ** -22 * (adz @ W.abs()), "dx")
    ref.close(dw, dz.t() @ X, edz.t() @ X.abs() + (M / 16 + 4) * 2.0 ** -22 * (adz.t() @ X.abs()), "dw")
    # chains of at most M / 2048 + 4 rows per thread, then 8, then the chunks in a tree
    ref.close(db, dz.sum(0), (ref.FWD + (M / 512 + 32) * 2.0 ** -24) * mag.sum(0), "db")
    assert fe.op_status() == (fe.FE_OK, 0)


SHAPES = [(1, 2, 8), (1, 1536, 2048), (2, 30, 264), (3, 64, 72), (5, 130, 520), (8, 66, 1000), (9, 64, 64), (17, 34, 40), (64, 2048, 768),
          (127, 130, 200), (128, 256, 64), (129, 258, 72), (200, 1536, 2048), (1003, 1002, 1992), (700, 22, 8),
          (2000, 1300, 200), (1201, 1536, 136), (2303, 2048, 72)]   # the last: CTA pairs, 192, 128 and 256 columns wide


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("M, N, K", SHAPES)
def test_forward(M, N, K, act):
    import fp4_expert_gemv_b200 as fe
    x, w, bias, res, _ = make(M, N, K, act, seed=M + N)
    z = torch.empty(M, N, dtype=bf, device="cuda")
    a = check_forward(fe, x, w, bias, act, res, z=z)
    check_forward(fe, x, w, None, act, None)
    assert torch.equal(a, check_forward(fe, x, w, bias, act, res))   # with and without z, run to run


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("M, N, K", [(1, 2, 8), (3, 16, 64), (9, 34, 40), (64, 256, 128), (130, 258, 200), (1003, 502, 264), (2000, 96, 1032)])
def test_backward(M, N, K, act):
    import fp4_expert_gemv_b200 as fe
    x, w, bias, _, dy = make(M, N, K, act, seed=M * N)
    z = None
    if act != "none":
        z = torch.empty(M, N, dtype=bf, device="cuda")
        fe.linear(x, w, bias=bias, act=act_id(fe, act), z=z)
    check_backward(fe, dy, x, w, z, act)


@pytest.mark.parametrize("N", [1, 5, 7, 33, 1001])
@pytest.mark.parametrize("M", [1, 6, 150])
def test_odd_columns(M, N):
    import fp4_expert_gemv_b200 as fe
    x, w, bias, res, dy = make(M, N, 96, "gelu", seed=N)
    z = torch.empty(M, N, dtype=bf, device="cuda")
    check_forward(fe, x, w, bias, "gelu", res, z=z)
    check_backward(fe, dy, x, w, z, "gelu")
    check_backward(fe, dy, x, w, None, "none")


@pytest.mark.parametrize("M, N, K", [(64, 64, 64), (130, 70, 136), (5, 24, 64), (512, 264, 192), (300, 1100, 72)])
def test_small_integers_come_out_exactly(M, N, K):
    """Values in {-1, 0, 1} with at most 256 nonzero products per sum: every sum is a whole number below
    2^8, exact in bf16, so each output equals the exact product and a missing, doubled or
    misplaced term shows."""
    import fp4_expert_gemv_b200 as fe
    g = torch.Generator(device="cuda").manual_seed(M + K)
    tri = lambda *s: (torch.randint(-1, 2, s, generator=g, device="cuda")).to(bf)
    x, w, dy = tri(M, K), tri(N, K), tri(M, N)
    # thin out long sums
    if M > 256:
        dy[torch.randperm(M, generator=g, device="cuda")[256:]] = 0
    if N > 256:
        dy[:, torch.randperm(N, generator=g, device="cuda")[256:]] = 0
    assert torch.equal(fe.linear(x, w).double(), x.double() @ w.double().t())
    dx, dw, db = fe.linear_backward(dy, x, w)
    assert torch.equal(dx.double(), dy.double() @ w.double())
    assert torch.equal(dw.double(), dy.double().t() @ x.double())
    assert torch.equal(db.double(), dy.double().sum(0))


@pytest.mark.parametrize("M", [1, 4, 40, 300, 20000])
def test_strided_rows_and_the_sum_in_place(M):
    import fp4_expert_gemv_b200 as fe
    x, w, bias, res, dy = make(M, 96, 128, "none", seed=M)
    wide = torch.zeros(M, 200, dtype=bf, device="cuda")
    wide[:, 8:136] = x
    out = torch.full((M, 150), 3.0, dtype=bf, device="cuda")
    want = check_forward(fe, x, w, bias, "none", res)
    for at in (0, 8, 5):
        out.fill_(3.0)
        fe.linear(wide[:, 8:136], w, bias=bias, residual=res, y=out[:, at:at + 96])
        assert torch.equal(out[:, at:at + 96], want)
        assert (out[:, :at] == 3).all() and (out[:, at + 96:] == 3).all()
        out[:, at:at + 96] = res
        fe.linear(x, w, bias=bias, residual=out[:, at:at + 96], y=out[:, at:at + 96])
        assert torch.equal(out[:, at:at + 96], want)
    wdy = torch.zeros(M, 111, dtype=bf, device="cuda")
    wdy[:, 3:99] = dy
    a = fe.linear_backward(dy, x, w)
    b = fe.linear_backward(wdy[:, 3:99], wide[:, 8:136], w)
    assert all(torch.equal(p, q) for p, q in zip(a, b))


def test_infinities_and_nan_stay_in_their_rows():
    import fp4_expert_gemv_b200 as fe
    for M in (4, 140, 20000):
        x, w, bias, res, _ = make(M, 64, 128, "silu", seed=2)
        clean = fe.linear(x, w, act=fe.ACT_SILU)
        x[1, 5] = float("nan")
        x[2, 7] = float("inf")
        y = fe.linear(x, w, act=fe.ACT_SILU)
        assert torch.isnan(y[1]).all()
        keep = [i for i in range(M) if i not in (1, 2)]
        assert torch.equal(y[keep], clean[keep])
        relu = fe.linear(x, w, act=fe.ACT_RELU)
        assert torch.isnan(relu[1]).all()


def test_large_activations_saturate_as_the_formula_does():
    import fp4_expert_gemv_b200 as fe
    for M in (2, 64):
        for act in ("silu", "gelu", "swiglu"):
            x, w, bias, _, dy = make(M, 64, 64, act, seed=5)
            x = (x.float() * 100).to(bf)
            z = torch.empty(M, 64, dtype=bf, device="cuda")
            y = fe.linear(x, w, act=act_id(fe, act), z=z)
            assert torch.isfinite(y).all()
            for t in fe.linear_backward(dy, x, w, z=z, act=act_id(fe, act)):
                assert torch.isfinite(t).all()


def test_no_rows_and_parts_left_out():
    import fp4_expert_gemv_b200 as fe
    x, w, bias, res, dy = make(0, 32, 64, "none")
    assert fe.linear(x, w, bias=bias).shape == (0, 32)
    dx, dw, db = fe.linear_backward(dy, x, w)
    assert dx.shape == (0, 64) and (dw == 0).all() and (db == 0).all()
    x, w, bias, res, dy = make(70, 32, 64, "none")
    full = fe.linear_backward(dy, x, w)
    for i in range(3):
        part = fe.linear_backward(dy, x, w, need_dx=i == 0, need_dw=i == 1, need_db=i == 2)
        assert [t is None for t in part] == [j != i for j in range(3)]
        assert torch.equal(part[i], full[i])


def test_gradient_against_differences():
    """<gradient, direction> against central differences of the 64-bit forward at the saved z (the bf16
    rounding of z moves the point where the slope is taken: |act''| <= 1.1 times 2^-8 |z| per element;
    dz and the outputs are rounded once each: 2 * 2^-8 of the summed magnitudes)."""
    import fp4_expert_gemv_b200 as fe
    x, w, bias, _, dy = make(24, 32, 48, "gelu", seed=8)
    z = torch.empty(24, 32, dtype=bf, device="cuda")
    fe.linear(x, w, bias=bias, act=fe.ACT_GELU, z=z)
    got = dict(zip(("x", "w", "bias"), fe.linear_backward(dy, x, w, z=z, act=fe.ACT_GELU)))
    base = dict(x=x.double(), w=w.double(), bias=bias.double())
    gen = torch.Generator(device="cuda").manual_seed(1)
    for name in base:
        dirn = torch.randn(base[name].shape, generator=gen, device="cuda", dtype=torch.float64)
        f = []
        for s in (1, -1):
            v = {**base, name: base[name] + s * 1e-4 * dirn}
            f.append(float((ref.act_parts("gelu", v["x"] @ v["w"].t() + v["bias"])[0] * dy.double()).sum()))
        # slope of the loss along the direction through each element of z
        dz_dir = dict(x=lambda: dirn @ base["w"].t(), w=lambda: base["x"] @ dirn.t(), bias=lambda: dirn.expand(24, 32))[name]()
        tol = 2.0 ** -8 * float((1.1 * z.double().abs() * (dy.double() * dz_dir).abs()).sum())
        tol += 2.0 ** -8 * float((dy.double().abs() * 1.13 * dz_dir.abs()).sum())
        tol += 2.0 ** -8 * float((got[name].double() * dirn).abs().sum()) + 1e-5
        assert abs((f[0] - f[1]) / 2e-4 - float((got[name].double() * dirn).sum())) <= tol, name


@pytest.mark.parametrize("M", [384, 5000])
def test_streams_and_graphs(M):
    import fp4_expert_gemv_b200 as fe
    x, w, bias, res, dy = make(M, 512, 256, "swiglu", seed=3)
    x1 = x[:2].contiguous()

    def step(stream=None):
        z = torch.empty(M, 512, dtype=bf, device="cuda")
        y = fe.linear(x, w, bias=bias, act=fe.ACT_SWIGLU, residual=res, z=z, stream=stream)
        return (y, z, fe.linear(x1, w, act=fe.ACT_SWIGLU, stream=stream),
                *fe.linear_backward(dy, x, w, z=z, act=fe.ACT_SWIGLU, stream=stream))

    first = step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = []
    for _ in range(3):   # the two streams' products may share the SMs
        with torch.cuda.stream(side):
            got.append(step())
        got.append(step())
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = step()
        graphs.append((g, out))
    for g, out in graphs:
        g.replay()
        got.append(out)
    torch.cuda.synchronize()
    for out in got:
        assert all(torch.equal(a, b) for a, b in zip(first, out))
    assert fe.op_status() == (fe.FE_OK, 0)


@pytest.mark.parametrize("act", ["none", "gelu", "swiglu"])
@pytest.mark.parametrize("M", [1, 9, 40, 300, 1003, 5000])
def test_outputs_at_odd_addresses(M, act):
    """y, z, residual and bias two bytes off their 16-byte boundaries: the same values, nothing beside them."""
    import fp4_expert_gemv_b200 as fe
    x, w, bias, res, _ = make(M, 264, 200, act, seed=M)
    C = res.shape[1]
    z = torch.empty(M, 264, dtype=bf, device="cuda")
    want = check_forward(fe, x, w, bias, act, res, z=z)

    def odd(t):
        buf = torch.full((t.numel() + 8,), 7.0, dtype=bf, device="cuda")
        v = buf[1:1 + t.numel()].view(t.shape)
        v.copy_(t)
        return buf, v
    (yb, y), (zb, z2), (_, r2), (_, b2) = odd(want * 0), odd(z * 0), odd(res), odd(bias)
    fe.linear(x, w, bias=b2, act=act_id(fe, act), residual=r2, y=y, z=z2)
    assert torch.equal(y, want) and torch.equal(z2, z)
    for buf, n in ((yb, M * C), (zb, M * 264)):
        assert buf[0] == 7 and (buf[1 + n:] == 7).all()


@pytest.mark.parametrize("N, K", [(2, 8), (66, 72), (1002, 264), (1536, 2048)])
def test_the_workspace_is_all_that_is_written(N, K):
    import fp4_expert_gemv_b200 as fe
    for M in (1, 31, 33, 129, 1000, 8200):
        x, w, bias, res, dy = make(M, N, K, "swiglu", seed=M)
        z = torch.empty(M, N, dtype=bf, device="cuda")
        fe.linear(x, w, bias=bias, act=fe.ACT_SWIGLU, z=z)
        nb = fe.fe_moe_linear_workspace(M, N, K, fe.ACT_SWIGLU)
        ws = torch.full((nb + 4096,), 85, dtype=torch.uint8, device="cuda")
        dx, dw = (torch.full((n * K + 64,), 5.0, dtype=bf, device="cuda") for n in (M, N))
        db = torch.full((N + 64,), 5.0, device="cuda")
        st = fe.fe_moe_linear_backward(dy.data_ptr(), N // 2, x.data_ptr(), K, w.data_ptr(), z.data_ptr(), M, N, K, fe.ACT_SWIGLU,
                                       dx.data_ptr(), K, dw.data_ptr(), db.data_ptr(), ws.data_ptr(), nb,
                                       torch.cuda.current_stream().cuda_stream)
        torch.cuda.synchronize()
        assert st == fe.FE_OK and (ws[nb:] == 85).all(), (M, N, K)
        assert (dx[M * K:] == 5).all() and (dw[N * K:] == 5).all() and (db[N:] == 5).all()


def test_rows_after_the_last_stay_as_they_were():
    import fp4_expert_gemv_b200 as fe
    for M in (3, 100, 2500):
        x, w, bias, res, dy = make(M, 1536 if M > 1000 else 96, 128, "none", seed=M)
        N = w.shape[0]
        y = torch.full((M + 300, N), 5.0, dtype=bf, device="cuda")
        z = torch.full((M + 300, N), 6.0, dtype=bf, device="cuda")
        fe.linear(x, w, act=fe.ACT_SILU, y=y[:M], z=z[:M])
        assert (y[M:] == 5).all() and (z[M:] == 6).all()


def test_gelu_over_its_whole_range():
    """z = x exactly (w is the identity).  Relative to z Phi(z), down to 1e-30: half a step of bf16, and 2^-14
    for the exponential of z^2 / 2 <= 72 (its argument and the fast exponential's product each rounded to
    2^-24 of it: 72 * 3 * 2^-24) and the polynomial."""
    import fp4_expert_gemv_b200 as fe
    z = torch.linspace(-12, 12, 64 * 512, device="cuda").to(bf).view(-1, 64)
    eye = torch.eye(64, dtype=bf, device="cuda")
    for rows in (z[:16], z, z.repeat(60, 1)):
        y = fe.linear(rows.contiguous(), eye, act=fe.ACT_GELU).double()
        x = rows.double()
        want = x * 0.5 * torch.special.erfc(-x / 2 ** 0.5)
        assert ((y - want).abs() <= (2.0 ** -8 + 2.0 ** -14) * want.abs() + 1e-30).all()


def test_refusals():
    import fp4_expert_gemv_b200 as fe
    x, w, bias, res, dy = make(16, 32, 64, "none")
    with pytest.raises(ValueError):
        fe.linear(x.t().contiguous().t(), w)
    with pytest.raises(ValueError):
        fe.linear(x.float(), w)
    with pytest.raises(ValueError):
        fe.linear(x, w, residual=res[:, :16])
    with pytest.raises(ValueError):
        fe.linear(x, w, z=torch.empty(16, 30, dtype=bf, device="cuda"))
    with pytest.raises(fe.FeMoeError):
        fe.linear(x[:, :60].contiguous(), w[:, :60].contiguous())
    with pytest.raises(fe.FeMoeError):
        fe.linear(x[:, 4:60], w[:, :56].contiguous())      # rows not on 16 bytes
    with pytest.raises(fe.FeMoeError):
        fe.linear(x, w, y=x[:, :32])


def test_no_rows_and_the_gradient_of_x_alone():
    import fp4_expert_gemv_b200 as fe
    x, w, _, _, dy = make(0, 32, 64, "none")
    dx, dw, db = fe.linear_backward(dy, x, w, need_dw=False, need_db=False)
    assert dx.shape == (0, 64) and dw is None and db is None


@pytest.mark.parametrize("act, odd", [("none", False), ("none", True), ("gelu", False)])
@pytest.mark.parametrize("M", [1, 70, 1000])
def test_the_workspace_asked_for_is_enough(M, act, odd):
    """Every set of outputs with exactly the bytes of its query (no workspace at all where that says 0), the bytes behind
    watched, against the call that is given the most."""
    import fp4_expert_gemv_b200 as fe
    N, K = 264, 136
    x, w, bias, _, dy = make(M, N, K, act, seed=M)
    ld = 267 if odd else N
    rows = torch.zeros(M, ld, dtype=bf, device="cuda")
    rows[:, :N] = dy
    z = torch.empty(M, N, dtype=bf, device="cuda")
    fe.linear(x, w, bias=bias, act=act_id(fe, act), z=z)
    stream = torch.cuda.current_stream().cuda_stream

    def call(outs, ws, nb):
        dx, dw, db = (torch.full(s, 5.0, dtype=t, device="cuda") if o else None
                      for o, s, t in zip(outs, ((M, K), (N, K), (N,)), (bf, bf, torch.float32)))
        ptr = lambda t: None if t is None else t.data_ptr()
        st = fe.fe_moe_linear_backward(rows.data_ptr(), ld, x.data_ptr(), K, w.data_ptr(), z.data_ptr() if act != "none" else None,
                                       M, N, K, act_id(fe, act), ptr(dx), K, ptr(dw), ptr(db), ptr(ws), nb, stream)
        assert st == fe.FE_OK
        return dx, dw, db

    most = fe.fe_moe_linear_workspace(M, N, K, act_id(fe, act))
    want = call((1, 1, 1), torch.empty(most, dtype=torch.uint8, device="cuda"), most)
    for outs in ((1, 1, 1), (1, 1, 0), (1, 0, 0), (0, 1, 0), (0, 0, 1)):
        nb = fe.fe_moe_linear_backward_workspace(M, N, K, act_id(fe, act), not odd, *outs)
        assert nb > 0 or (act == "none" and not odd and not outs[2])
        ws = torch.full((nb + 4096,), 85, dtype=torch.uint8, device="cuda") if nb else None
        got = call(outs, ws, nb)
        for o, a, b in zip(outs, got, want):
            assert not o or torch.equal(a, b)
        assert ws is None or (ws[nb:] == 85).all()
    torch.cuda.synchronize()
    assert fe.op_status() == (fe.FE_OK, 0)


@pytest.mark.parametrize("M, N, K", [(4096, 1536, 2048), (5003, 1538, 2056), (8200, 768, 2048), (3000, 5000, 1032), (6000, 3, 8008)])
def test_many_tiles_of_both_gradients_come_out_exactly(M, N, K):
    """Both products with several tiles per CTA pair in one launch, ring and accumulators carried from dW to dX:
    values in {-1, 0, 1} with at most 256 rows and columns of dy that are not zero, so that every sum is a
    whole number of at most 256, exact in bf16, and a missing, doubled or misplaced term shows."""
    import fp4_expert_gemv_b200 as fe
    g = torch.Generator(device="cuda").manual_seed(M + N)
    tri = lambda *s: (torch.randint(-1, 2, s, generator=g, device="cuda")).to(bf)
    x, w, dy = tri(M, K), tri(N, K), tri(M, N)
    rows = torch.zeros(M, dtype=torch.bool, device="cuda")
    cols = torch.zeros(N, dtype=torch.bool, device="cuda")
    for at, n in ((rows, M), (cols, N)):
        at[torch.randperm(n, generator=g, device="cuda")[:254]] = True
        at[0] = at[n - 1] = True                              # and the ends
    dense = dy.clone()
    dy[~rows] = 0
    dense[:, ~cols] = 0                                       # for dx: every row, 256 columns
    for t, only in ((dy, "dw"), (dense, "dx")):
        dx, dw, db = fe.linear_backward(t, x, w)
        if only == "dw":
            assert torch.equal(dw.double(), t[rows].double().t() @ x[rows].double())
            assert torch.equal(db.double(), t[rows].double().sum(0))
            assert (dx[~rows] == 0).all()
        else:
            assert torch.equal(dx.double(), t[:, cols].double() @ w[cols].double())
            assert (dw[~cols] == 0).all()
    assert fe.op_status() == (fe.FE_OK, 0)


@pytest.mark.parametrize("act", ["gelu", "swiglu"])
def test_backward_of_many_tiles(act):
    import fp4_expert_gemv_b200 as fe
    M, N, K = 4100, 1546, 2056
    x, w, bias, _, dy = make(M, N, K, act, seed=1)
    z = torch.empty(M, N, dtype=bf, device="cuda")
    fe.linear(x, w, bias=bias, act=act_id(fe, act), z=z)
    check_backward(fe, dy, x, w, z, act)


@pytest.mark.parametrize("act", ["none", "gelu", "swiglu"])
@pytest.mark.parametrize("cols", [33, 34, 36, 39, 250, 1537])
@pytest.mark.parametrize("M", [5, 70, 300, 20011])
def test_nothing_is_written_behind_a_row(M, cols, act):
    """Rows of whole 16-byte pieces apart whose last piece is not all theirs, in a buffer that ends with the last row's last
    column: what lies between the rows and behind them stays."""
    import fp4_expert_gemv_b200 as fe
    N = 2 * cols if act == "swiglu" else cols
    x, w, bias, res, _ = make(M, N, 72, act, seed=cols)
    want = fe.linear(x, w, bias=bias, act=act_id(fe, act), residual=res)
    plain = fe.linear(x, w, act=act_id(fe, act))
    ld = (cols + 7) // 8 * 8 + 8
    n = (M - 1) * ld + cols
    buf = torch.empty(n + 64, dtype=bf, device="cuda")
    y = buf[:n].as_strided((M, cols), (ld, 1))
    for kw, ref_y in ((dict(bias=bias, residual=res), want), (dict(), plain), (dict(bias=bias, residual=y), want),
                      (dict(bias=bias, residual=res, z=torch.empty(M, N, dtype=bf, device="cuda")), want)):
        buf.fill_(7.0)
        if kw.get("residual") is y:
            y.copy_(res)
        fe.linear(x, w, act=act_id(fe, act), y=y, **kw)
        assert torch.equal(y, ref_y)
        y.fill_(7.0)
        assert (buf == 7).all()
    assert fe.op_status() == (fe.FE_OK, 0)


@pytest.mark.parametrize("M", [2, 12, 200, 3000])
def test_columns_of_one_buffer_as_operand_and_output(M):
    """x, the residual and y (dy, x and dx) side by side in the rows of one buffer."""
    import fp4_expert_gemv_b200 as fe
    N, K = 96, 128
    x, w, bias, res, dy = make(M, N, K, "gelu", seed=M)
    want = fe.linear(x, w, bias=bias, act=fe.ACT_GELU, residual=res)
    buf = torch.full((M, K + 2 * N + 8), 7.0, dtype=bf, device="cuda")
    bx, by, br = buf[:, :K], buf[:, K:K + N], buf[:, K + N:K + 2 * N]
    for order in ((bx, by, br), (bx, br, by)):
        bx.copy_(x), order[2].copy_(res)
        fe.linear(bx, w, bias=bias, act=fe.ACT_GELU, residual=order[2], y=order[1])
        assert torch.equal(order[1], want) and torch.equal(bx, x) and torch.equal(order[2], res) and (buf[:, K + 2 * N:] == 7).all()
    z = torch.empty(M, N, dtype=bf, device="cuda")
    fe.linear(x, w, act=fe.ACT_GELU, z=z)
    dx, dw, db = fe.linear_backward(dy, x, w, z=z, act=fe.ACT_GELU)
    wide = torch.full((M, 2 * K + N), 7.0, dtype=bf, device="cuda")
    vdy, vx, vdx = wide[:, K:K + N], wide[:, K + N:], wide[:, :K]
    vdy.copy_(dy), vx.copy_(x)
    dw2 = torch.empty_like(w)
    nb = fe.fe_moe_linear_workspace(M, N, K, fe.ACT_GELU)
    ws = torch.empty(nb, dtype=torch.uint8, device="cuda")
    st = fe.fe_moe_linear_backward(vdy.data_ptr(), wide.stride(0), vx.data_ptr(), wide.stride(0), w.data_ptr(), z.data_ptr(), M, N, K,
                                   fe.ACT_GELU, vdx.data_ptr(), wide.stride(0), dw2.data_ptr(), None, ws.data_ptr(), nb,
                                   torch.cuda.current_stream().cuda_stream)
    assert st == fe.FE_OK
    assert torch.equal(vdx, dx) and torch.equal(dw2, dw) and torch.equal(vdy, dy) and torch.equal(vx, x)
