"""The operators together: a whole block around the packed layer, two blocks in a row, and the
gradient of the balance loss through the router's product and the norm in front of it."""
import numpy as np
import pytest
import torch

import block_ref as ref
import harness
import synth

pytestmark = pytest.mark.gpu
bf = torch.bfloat16


def params(H, Is, E, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    n = lambda *s, std=1.0: (torch.randn(*s, generator=g, device="cuda") * std).to(bf)
    w = lambda: (1 + torch.randn(H, generator=g, device="cuda") * 0.2).to(bf)
    return dict(w_router=n(E, H, std=H ** -0.5), w_pre=w(), w_post=w(), w_next_pre=w(), gate=n(H),
                shared=(n(2 * Is, H, std=H ** -0.5), n(H, Is, std=Is ** -0.5)))


def by_hand(fe, layer, r, p, k, kind, scale, u=None):
    """forward_block from the single calls."""
    if u is None:
        _, u = fe.block_norm(r, w_pre=p["w_pre"])
    y, logits = layer.forward_router(u, p["w_router"], k)
    if p.get("shared"):
        a = fe.linear(u, p["shared"][0], act=fe.ACT_SWIGLU)
        fe.linear(a, p["shared"][1], residual=y, y=y)
    r2, u2 = fe.block_norm(r, y, p["w_post"], p["w_next_pre"], gate=p["gate"], gate_kind=kind, scale=scale)
    return r2, u2, logits, u


@pytest.mark.parametrize("T", [1, 3, 40])
@pytest.mark.parametrize("rt", [bf, torch.float32])
@pytest.mark.parametrize("shared", [True, False])
def test_block_is_its_parts_and_close_to_the_definition(T, rt, shared):
    import fp4_expert_gemv_b200 as fe
    E, H, I, k, seed = 8, 256, 128, 2, 0
    gl = harness.GpuLayer(E, H, I, seed, max_T=64, max_k=4)
    p = params(H, 96, E, 5 + T)
    if not shared:
        p["shared"] = None
    r = (torch.randn(T, H, generator=torch.Generator(device="cuda").manual_seed(T), device="cuda") * 2).to(rt)
    kind = fe.GATE_CHANNEL | fe.GATE_SIGMOID
    kw = dict(shared=p["shared"], w_post=p["w_post"], gate=p["gate"], gate_kind=kind, scale=0.5, w_next_pre=p["w_next_pre"])
    r2, u2, logits = gl.layer.forward_block(r, k, p["w_router"], w_pre=p["w_pre"], **kw)
    h2, hu2, hl, u = by_hand(fe, gl.layer, r, p, k, kind, 0.5)
    assert torch.equal(r2, h2) and torch.equal(u2, hu2) and torch.equal(logits, hl)
    assert gl.layer.status() == (fe.FE_OK, 0) and fe.op_status() == (fe.FE_OK, 0)
    # the oracle's layer on the same u and logits, the rest in 64 bits
    side = harness.OracleSide(E, H, I, seed)
    y64, _ = side.forward(u.view(torch.int16).cpu().numpy().view(np.uint16), logits.cpu().numpy(), k)
    y64 = torch.from_numpy(y64).cuda()
    if shared:
        a = ref.linear(u, p["shared"][0], None, "swiglu", None)[0]
        y64 = y64 + a @ p["shared"][1].double().t()
    want = ref.norm_forward(r, y64, p["w_post"], p["w_next_pre"], p["gate"], "channel", True, 0.5, 1e-6)
    # the layer's tolerance on what it adds (the norm keeps relative errors), bf16 roundings of y and of
    # the shared expert's two products (2^-8 each of their largest values) and of the output
    add = want["r_out"][0] - r.double()
    tol = (harness.MAX_REL_TOL + 3 * 2.0 ** -8) * float(add.abs().max())
    ref.close(r2, want["r_out"][0], torch.full_like(add, tol), "r_out")
    rho = float((want["r_out"][0] ** 2).mean(1).min() ** -0.5)
    ref.close(u2, want["u"][0], torch.full_like(add, 2 * tol * rho * float(p["w_next_pre"].abs().max())), "u_out")
    # in place
    buf = r.clone()
    o, uu, _ = gl.layer.forward_block(buf, k, p["w_router"], w_pre=p["w_pre"], r_out=buf, **kw)
    assert torch.equal(o, r2) and torch.equal(uu, u2)
    gl.layer.close()


def test_two_blocks_with_the_norm_between_them_fused_and_in_a_graph():
    import fp4_expert_gemv_b200 as fe
    E, H, I, k, T = 8, 256, 128, 2, 5
    layers = [harness.GpuLayer(E, H, I, s, max_T=8, max_k=2).layer for s in (0, 1)]
    ps = [params(H, 64, E, s) for s in (1, 2)]
    r = torch.randn(T, H, device="cuda", generator=torch.Generator(device="cuda").manual_seed(0))

    def chain(fused):
        x, u = r, None
        for i, (layer, p) in enumerate(zip(layers, ps)):
            nxt = ps[i + 1]["w_pre"] if i + 1 < len(ps) and fused else None
            x, u, _ = layer.forward_block(x, k, p["w_router"], w_pre=None if u is not None else p["w_pre"], u_in=u, shared=p["shared"],
                                          w_post=p["w_post"], scale=0.5, w_next_pre=nxt)
            u = u if fused else None
        return x

    # the fp32 residual is stored unrounded, so the norm inside the boundary sees what a norm of its own sees
    want = chain(False)
    assert torch.equal(chain(True), want)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = chain(True)
    r.mul_(1.5)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, chain(False)) and not torch.equal(out, want)


def test_block_refusals():
    import fp4_expert_gemv_b200 as fe
    gl = harness.GpuLayer(8, 256, 128, 0, max_T=4, max_k=2)
    p = params(256, 64, 8, 1)
    r = torch.zeros(4, 256, device="cuda")
    call = gl.layer.forward_block
    big = torch.zeros(5, 256, device="cuda")
    for bad in (lambda: call(big, 2, p["w_router"], w_pre=p["w_pre"]), lambda: call(r, 3, p["w_router"], w_pre=p["w_pre"]),
                lambda: call(r, 9, p["w_router"], w_pre=p["w_pre"]), lambda: call(r, 2, p["w_router"]),
                lambda: call(r, 2, p["w_router"], w_pre=p["w_pre"], eps=-1.0)):
        with pytest.raises(fe.FeMoeError):
            bad()
    with pytest.raises(ValueError):
        call(r, 2, p["w_router"], w_pre=p["w_pre"], gate=p["gate"])
    with pytest.raises(ValueError):
        call(r, 2, p["w_router"], w_pre=p["w_pre"], shared=(p["shared"][0], p["shared"][1][:, :32]))
    with pytest.raises(ValueError):
        call(r, 2, p["w_router"], w_pre=p["w_pre"], u_out=r.to(bf))
    # a path that cannot run the call is refused before the norm in front of it is launched
    gl.layer.set_path(fe.PATH_NVFP4)
    logits = torch.full((4, 8), 3.0, device="cuda")
    with pytest.raises(fe.FeMoeError):
        call(r, 2, p["w_router"], w_pre=p["w_pre"], logits=logits)
    torch.cuda.synchronize()
    assert (logits == 3).all()
    # outputs over operands and over each other, also of different parts of the block
    r32 = torch.ones(4, 256, device="cuda")
    kw = dict(w_pre=p["w_pre"], w_next_pre=p["w_next_pre"])
    gl.layer.set_path(fe.PATH_AUTO)
    for bad in (dict(logits=r32.view(-1)[:32].view(4, 8)), dict(u_out=r32.view(bf).view(-1)[512:1536].view(4, 256)),
                dict(u_in=r32.view(bf).view(-1)[:1024].view(4, 256), r_out=r32)):
        with pytest.raises(fe.FeMoeError):
            gl.layer.forward_block(r32, 2, p["w_router"], **{**kw, **bad})
    torch.cuda.synchronize()
    assert (r32 == 1).all()
    # in place, as said: r_out over r and u_out over u_in
    _, u0 = fe.block_norm(r32, w_pre=p["w_pre"])
    want = gl.layer.forward_block(r32, 2, p["w_router"], u_in=u0, w_next_pre=p["w_next_pre"])
    got = gl.layer.forward_block(r32, 2, p["w_router"], u_in=u0, w_next_pre=p["w_next_pre"], r_out=r32, u_out=u0)
    assert got[0] is r32 and got[1] is u0 and torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    gl.layer.close()


def test_first_calls_inside_a_capture():
    """A process whose first calls are captured: nothing in them synchronises or allocates."""
    import os
    import subprocess
    import sys
    code = """
import torch, fp4_expert_gemv_b200 as fe
bf = torch.bfloat16
x, w = torch.randn(3000, 256, device="cuda").to(bf), torch.randn(512, 256, device="cuda").to(bf)
h = torch.ones(256, device="cuda").to(bf)
l = torch.randn(3000, 16, device="cuda")
idx = torch.zeros(3000, 2, dtype=torch.int32, device="cuda")
def step():
    y = fe.linear(x, w)
    z = fe.linear(x[:70], w)
    _, u = fe.block_norm(x, w_pre=h)
    g = fe.block_norm_backward(x, u, x, x, h, h)
    loss, c, n = fe.balance_loss(l, idx)
    return y, z, u, *g[:2], loss, fe.balance_loss_backward(l, c, n, 2), *fe.linear_backward(y, x, w)
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    out = step()
g.replay()
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(out, step()))
print("same")
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, cwd=root, timeout=300)
    assert r.returncode == 0 and "same" in r.stdout, r.stderr[-2000:]


def test_training_the_router_on_the_balance_loss():
    """r -> norm -> router logits -> balance loss and back to the router's weights, the norm's weight and r,
    against differentiation of the 64-bit chain at the device's u.  dlogits enters the products
    rounded to bf16 and dx leaves them so: 2^-8 of the summed magnitudes each, then the norm's bound."""
    import fp4_expert_gemv_b200 as fe
    E, H, T, k = 16, 128, 200, 3
    gl = harness.GpuLayer(E, H, 64, 0, max_T=256, max_k=4)
    p = params(H, 64, E, 3)
    r = torch.randn(T, H, device="cuda", generator=torch.Generator(device="cuda").manual_seed(4))
    mask = (torch.arange(T, device="cuda") % 5 != 0).to(torch.uint8)
    _, u = fe.block_norm(r, w_pre=p["w_pre"])
    logits, idx, _ = gl.layer.router(u, p["w_router"], k)
    loss, counts, n = fe.balance_loss(logits, idx, mask=mask, balance_coef=1.0, z_coef=0.1)
    dl = fe.balance_loss_backward(logits, counts, n, k, mask=mask, balance_coef=1.0, z_coef=0.1, dtype=bf)
    du, dwr, _ = fe.linear_backward(dl, u, p["w_router"], need_db=False)
    dr, _, _, _, dw_pre = fe.block_norm_backward(None, du, r, w_pre=p["w_pre"])

    u64 = u.double().requires_grad_()
    w64 = p["w_router"].double().requires_grad_()
    l64 = u64 @ w64.t()
    keep = mask.bool()
    f = counts.double() / (int(n) * k)
    pr = torch.softmax(l64[keep], 1)
    want_loss = E * (f * pr.mean(0)).sum() + 0.1 * (torch.logsumexp(l64[keep], 1) ** 2).mean()
    assert abs(float(loss[0]) - float(want_loss.detach())) <= 1e-5 * float(want_loss.detach())
    gu, gw = torch.autograd.grad(want_loss, [u64, w64])
    adl = dl.double().abs()
    ref.close(dwr, gw, 2.0 ** -7 * (adl.t() @ u.double().abs()), "dW_r")
    ref.close(du, gu, 2.0 ** -7 * (adl @ p["w_router"].double().abs()), "dx")
    want = ref.norm_backward(None, du, r, None, None, p["w_pre"], None, "none", False, 1.0, 1e-6)
    ref.close(dr, want["dr"][0], ref.BWD * want["dr"][1], "dr")
    ref.close(dw_pre, want["dw_pre"][0], ref.BWD * want["dw_pre"][1], "dw_pre")
    gl.layer.close()


# from 200 to 9100 rows: through the layer's streaming and its tensor-core path (4096 pairs and more), the products by
# split tiles of several row tiles and by CTA pairs, the norms row by row and streamed
@pytest.mark.parametrize("T, H, I, Is, k, rt", [(200, 2048, 256, 768, 2, bf), (600, 1024, 128, 1000, 4, torch.float32),
                                                (2100, 2048, 256, 768, 2, bf), (5000, 512, 128, 264, 3, bf),
                                                (9100, 1024, 128, 512, 2, torch.float32)])
def test_block_of_a_prefill(T, H, I, Is, k, rt):
    """The composed call is its parts bit by bit at prefill sizes, repeats, and is close to the definition at rows from
    the start, the middle and the end (the bounds of the test of small blocks)."""
    import fp4_expert_gemv_b200 as fe
    E, seed = 8, 3
    gl = harness.GpuLayer(E, H, I, seed, max_T=T, max_k=4)
    p = params(H, Is, E, T)
    r = (torch.randn(T, H, generator=torch.Generator(device="cuda").manual_seed(T), device="cuda") * 2).to(rt)
    kind = fe.GATE_CHANNEL | fe.GATE_SIGMOID
    kw = dict(shared=p["shared"], w_post=p["w_post"], gate=p["gate"], gate_kind=kind, scale=0.5, w_next_pre=p["w_next_pre"])
    r2, u2, logits = gl.layer.forward_block(r, k, p["w_router"], w_pre=p["w_pre"], **kw)
    h2, hu2, hl, u = by_hand(fe, gl.layer, r, p, k, kind, 0.5)
    assert torch.equal(r2, h2) and torch.equal(u2, hu2) and torch.equal(logits, hl)
    again = gl.layer.forward_block(r, k, p["w_router"], u_in=u, **kw)
    assert torch.equal(again[0], r2) and torch.equal(again[1], u2) and torch.equal(again[2], logits)
    assert gl.layer.status() == (fe.FE_OK, 0) and fe.op_status() == (fe.FE_OK, 0)
    at = torch.tensor([0, 1, 2, 127, 128, 129, T // 2, T // 2 + 1, T - 3, T - 2, T - 1], device="cuda")
    side = harness.OracleSide(E, H, I, seed)
    y64, _ = side.forward(u[at].contiguous().view(torch.int16).cpu().numpy().view(np.uint16), logits[at].cpu().numpy(), k)
    a = ref.linear(u[at], p["shared"][0], None, "swiglu", None)[0]
    y64 = torch.from_numpy(y64).cuda() + a @ p["shared"][1].double().t()
    want = ref.norm_forward(r[at], y64, p["w_post"], p["w_next_pre"], p["gate"], "channel", True, 0.5, 1e-6)
    add = want["r_out"][0] - r[at].double()
    tol = (harness.MAX_REL_TOL + 3 * 2.0 ** -8) * float(add.abs().max())
    ref.close(r2[at], want["r_out"][0], torch.full_like(add, tol), "r_out")
    rho = float((want["r_out"][0] ** 2).mean(1).min() ** -0.5)
    ref.close(u2[at], want["u"][0], torch.full_like(add, 2 * tol * rho * float(p["w_next_pre"].abs().max())), "u_out")
    gl.layer.close()


def test_blocks_of_a_prefill_in_a_graph_and_on_a_stream():
    import fp4_expert_gemv_b200 as fe
    E, H, T, k = 8, 1024, 2100, 2
    gl = harness.GpuLayer(E, H, 128, 1, max_T=T, max_k=2)
    p = params(H, 512, E, 2)
    r = torch.randn(T, H, device="cuda", generator=torch.Generator(device="cuda").manual_seed(6)).to(bf)
    call = lambda **kw: gl.layer.forward_block(r, k, p["w_router"], w_pre=p["w_pre"], shared=p["shared"], w_post=p["w_post"],
                                               w_next_pre=p["w_next_pre"], **kw)
    want = call()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = call(stream=side)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = call()
    r.mul_(-0.75)
    g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(out, call())) and not torch.equal(out[0], want[0])
    assert gl.layer.status() == (fe.FE_OK, 0) and fe.op_status() == (fe.FE_OK, 0)
    gl.layer.close()


def test_tensors_of_another_device_are_refused():
    """The layer runs on the device that it was made on; its kernels must not be given another one's memory (here the
    layer is made to believe that it lies elsewhere: nothing is launched)."""
    gl = harness.GpuLayer(8, 256, 128, 0, max_T=4, max_k=2)
    p = params(256, 64, 8, 1)
    r = torch.zeros(4, 256, device="cuda")
    gl.layer.forward_block(r, 2, p["w_router"], w_pre=p["w_pre"])
    gl.layer.device += 1
    with pytest.raises(ValueError, match="layer on cuda"):
        gl.layer.forward_block(r, 2, p["w_router"], w_pre=p["w_pre"])
    gl.layer.close()
