"""The operators around the packed expert layer, as they are measured: the block's norms with
gate and residual, the router's balance loss with its gradient, and the dense product with its
epilogue (the shared expert), each forward and backward.

A case names its operator ("op") and direction ("dir"):
  norm     r' = r + s * a(g) * w_post * y / rms(y),  u = w_pre * r' / rms(r')
  balance  loss over softmax(logits) and the chosen experts, their counts; "step" also takes
           the gradient with respect to the logits
  linear   y = act(x W^T + b) + residual;  "bwd" takes dx, dW, db from the saved pre-activation
"""
import math

import torch

own = False

EPS = 1e-6
SCALE = 0.5
BALANCE, ZLOSS = 0.01, 0.001


def listed():
    return [
        # one token of a decode step, at the boundary of two blocks: the smallest call, pure latency
        dict(name="norm_t1", op="norm", dir="fwd", T=1, H=2048, r32=False, gate="none"),
        # a prefill chunk with an fp32 residual stream and one sigmoid gate per token
        dict(name="norm_t4096", op="norm", dir="fwd", T=4096, H=2048, r32=True, gate="token"),
        # training: the backward of the block boundary, a gate per channel
        dict(name="norm_bwd_t4096", op="norm", dir="bwd", T=4096, H=2048, r32=False, gate="channel"),
        # an odd width and a ragged batch with a gate per element
        dict(name="norm_bwd_odd", op="norm", dir="bwd", T=1237, H=1999, r32=False, gate="full"),
        # the decode batch's expert counts and loss
        dict(name="balance_t64", op="balance", dir="fwd", T=64, E=128, k=8, pad=False),
        # a training microbatch with padded tokens
        dict(name="balance_t4096", op="balance", dir="step", T=4096, E=128, k=8, pad=True),
        # a long batch of the 512-expert layer: the largest
        dict(name="balance_t65536", op="balance", dir="step", T=65536, E=512, k=10, pad=True),
        # shared expert, one token: gate and up rows streamed once
        dict(name="linear_t1", op="linear", dir="fwd", M=1, N=1536, K=2048, act="swiglu", bias=False, res=False),
        # shared expert's second product for a decode batch, added onto the routed experts' output
        dict(name="linear_t64", op="linear", dir="fwd", M=64, N=2048, K=768, act="none", bias=True, res=True),
        # ragged rows and an odd number of columns
        dict(name="linear_odd", op="linear", dir="fwd", M=1003, N=1001, K=1992, act="gelu", bias=True, res=True),
        # shared expert over a long prefill: the largest product
        dict(name="linear_t16384", op="linear", dir="fwd", M=16384, N=1536, K=2048, act="swiglu", bias=False, res=False),
        # training the shared expert's first product
        dict(name="linear_bwd_t4096", op="linear", dir="bwd", M=4096, N=1536, K=2048, act="swiglu", bias=True, res=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "balance", "linear"])
    if op == "norm":
        T = _log(rng, 1, 8192)
        H = _log(rng, 64, min(8192, (4096 * 2048) // T))
        if rng.random() < 0.6:
            H = max(64, H // 64 * 64)
        return dict(op=op, dir=rng.choice(["fwd", "bwd"]), T=T, H=H, r32=rng.random() < 0.5,
                    gate=rng.choice(["none", "channel", "token", "full"]))
    if op == "balance":
        E = _log(rng, 4, 512)
        T = _log(rng, 1, 65536)
        return dict(op=op, dir=rng.choice(["fwd", "step"]), T=T, E=E, k=rng.randint(1, min(E, 10)), pad=rng.random() < 0.5)
    d = rng.choice(["fwd", "fwd", "bwd"])
    K = 8 * _log(rng, 8, 512)
    N = 2 * _log(rng, 8, 2048) - (rng.random() < 0.2)
    M = _log(rng, 1, max(1, min(16384, int(1e11 / (2.0 * N * K * (2 if d == "bwd" else 1))))))
    act = rng.choice(["none", "relu", "gelu", "silu", "swiglu"])
    if act == "swiglu":
        N += N % 2
    return dict(op=op, dir=d, M=M, N=N, K=K, act=act, bias=rng.random() < 0.5, res=d == "fwd" and rng.random() < 0.5)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, std=1.0, dtype=torch.bfloat16):
        return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)

    def empty(*shape, dtype=torch.bfloat16):
        return torch.empty(*shape, device="cuda", dtype=dtype)

    s = dict(case)
    if case["op"] == "norm":
        T, H = case["T"], case["H"]
        rt = torch.float32 if case["r32"] else torch.bfloat16
        s["r"], s["y"] = normal(T, H, std=2.0, dtype=rt), normal(T, H, std=0.3)
        s["w_post"], s["w_pre"] = (1 + normal(H, std=0.2, dtype=torch.float32)).bfloat16(), (1 + normal(H, std=0.2, dtype=torch.float32)).bfloat16()
        shape = dict(none=None, channel=(H,), token=(T,), full=(T, H))[case["gate"]]
        s["g"] = normal(*shape) if shape else None
        if case["dir"] == "bwd":
            s["dr_out"], s["du"] = normal(T, H, dtype=rt), normal(T, H)
        else:
            s["r_out"], s["u"] = empty(T, H, dtype=rt), empty(T, H)
    elif case["op"] == "balance":
        T, E, k = case["T"], case["E"], case["k"]
        # some experts are liked more than others
        s["logits"] = normal(T, E, dtype=torch.float32) + normal(E, std=0.7, dtype=torch.float32)
        s["idx"] = torch.topk(s["logits"], k, dim=1).indices.to(torch.int32)
        s["mask"] = (torch.rand(T, generator=g, device="cuda") < 0.8).to(torch.uint8) if case["pad"] else None
        s["dloss"] = normal(1, dtype=torch.float32).abs() + 0.5
    else:
        M, N, K = case["M"], case["N"], case["K"]
        cols = N // 2 if case["act"] == "swiglu" else N
        s["x"], s["w"] = normal(M, K), normal(N, K, std=K ** -0.5)
        s["b"] = normal(N, std=0.1) if case["bias"] else None
        if case["dir"] == "bwd":
            z = s["x"].float() @ s["w"].float().t()
            s["z"] = (z + s["b"].float() if case["bias"] else z).bfloat16()
            s["dy"] = normal(M, cols)
        else:
            s["res"] = normal(M, cols) if case["res"] else None
            s["y"] = empty(M, cols)
    return s


# ---- the framework's operators ---------------------------------------------------------


def _own(s):
    import fp4_expert_gemv_b200 as fe
    if s["op"] == "norm":
        kind = fe.GATE_NONE if s["g"] is None else dict(channel=fe.GATE_CHANNEL, token=fe.GATE_TOKEN, full=fe.GATE_FULL)[s["gate"]] | fe.GATE_SIGMOID
        if s["dir"] == "fwd":
            return fe.block_norm(s["r"], s["y"], s["w_post"], s["w_pre"], gate=s["g"], gate_kind=kind, scale=SCALE, eps=EPS,
                                 r_out=s["r_out"], u=s["u"])
        return fe.block_norm_backward(s["dr_out"], s["du"], s["r"], s["y"], s["w_post"], s["w_pre"], gate=s["g"], gate_kind=kind,
                                      scale=SCALE, eps=EPS)
    if s["op"] == "balance":
        loss, counts, n = fe.balance_loss(s["logits"], s["idx"], mask=s["mask"], balance_coef=BALANCE, z_coef=ZLOSS)
        if s["dir"] == "fwd":
            return loss, counts, n
        d = fe.balance_loss_backward(s["logits"], counts, n, s["k"], mask=s["mask"], dloss=s["dloss"], balance_coef=BALANCE, z_coef=ZLOSS)
        return loss, counts, n, d
    act = dict(none=fe.ACT_NONE, relu=fe.ACT_RELU, gelu=fe.ACT_GELU, silu=fe.ACT_SILU, swiglu=fe.ACT_SWIGLU)[s["act"]]
    if s["dir"] == "fwd":
        return fe.linear(s["x"], s["w"], bias=s["b"], act=act, residual=s["res"], y=s["y"])
    return fe.linear_backward(s["dy"], s["x"], s["w"], z=s["z"], act=act)


# ---- the plain form ---------------------------------------------------------------------


def _norm(s):
    r, y, w_post, w_pre = s["r"].float(), s["y"].float(), s["w_post"].float(), s["w_pre"].float()
    m = y * torch.rsqrt((y * y).mean(1, keepdim=True) + EPS)
    v = m * w_post
    if s["g"] is None:
        a = torch.ones((), device=r.device)
    else:
        g = s["g"].float()
        a = 1 / (1 + torch.exp(-(g[:, None] if s["gate"] == "token" else g)))
    r2 = r + SCALE * a * v
    rho = torch.rsqrt((r2 * r2).mean(1, keepdim=True) + EPS)
    n = r2 * rho
    if s["dir"] == "fwd":
        return r2.to(s["r"].dtype), (n * w_pre).bfloat16()
    rho_y = torch.rsqrt((y * y).mean(1, keepdim=True) + EPS)
    du = s["du"].float()
    dn = du * w_pre
    D = s["dr_out"].float() + rho * (dn - n * (dn * n).mean(1, keepdim=True))
    dv = SCALE * a * D
    dm = dv * w_post
    dy = rho_y * (dm - m * (dm * m).mean(1, keepdim=True))
    dg = None
    if s["g"] is not None:
        dg = SCALE * v * D * a * (1 - a)
        dg = dg.sum(0) if s["gate"] == "channel" else dg.sum(1) if s["gate"] == "token" else dg.bfloat16()
    return D.to(s["r"].dtype), dy.bfloat16(), dg, (dv * m).sum(0), (du * n).sum(0)


def _balance(s):
    l, T, E, k = s["logits"], s["T"], s["E"], s["k"]
    keep = torch.ones(T, device=l.device) if s["mask"] is None else (s["mask"] != 0).float()
    top = l.max(1, keepdim=True).values
    ex = torch.exp(l - top)
    tot = ex.sum(1, keepdim=True)
    p = ex / tot * keep[:, None]
    lse = (top + torch.log(tot))[:, 0]
    n = keep.sum()
    counts = torch.zeros(E, device=l.device).index_add_(0, s["idx"].reshape(-1), keep[:, None].expand(T, k).reshape(-1))
    f = counts / (n.clamp(min=1) * k)
    bal = E * (f * p.sum(0)).sum() / n.clamp(min=1)
    z = (lse * lse * keep).sum() / n.clamp(min=1)
    loss = torch.stack([BALANCE * bal + ZLOSS * z, bal, z])
    out = loss, counts.to(torch.int32), n.to(torch.int32).reshape(1)
    if s["dir"] == "fwd":
        return out
    up = s["dloss"] / n.clamp(min=1)
    return *out, up * p * (BALANCE * E * (f - (p * f).sum(1, keepdim=True)) + 2 * ZLOSS * lse[:, None])


def _phi(z):
    return 0.5 * (1 + torch.erf(z * math.sqrt(0.5)))


def _linear(s):
    x, w = s["x"].float(), s["w"].float()
    act, half = s["act"], s["N"] // 2
    if s["dir"] == "fwd":
        z = x @ w.t()
        if s["b"] is not None:
            z = z + s["b"].float()
        if act == "relu":
            z = torch.where(z > 0, z, torch.zeros_like(z))
        elif act == "gelu":
            z = z * _phi(z)
        elif act == "silu":
            z = z / (1 + torch.exp(-z))
        elif act == "swiglu":
            z = z[:, :half] / (1 + torch.exp(-z[:, :half])) * z[:, half:]
        return (z if s["res"] is None else z + s["res"].float()).bfloat16()
    z, dy = s["z"].float(), s["dy"].float()
    if act == "relu":
        dz = dy * (z > 0)
    elif act == "gelu":
        dz = dy * (_phi(z) + z * torch.exp(-0.5 * z * z) * (2 * math.pi) ** -0.5)
    elif act == "silu":
        q = 1 / (1 + torch.exp(-z))
        dz = dy * q * (1 + z * (1 - q))
    elif act == "swiglu":
        zg, zu = z[:, :half], z[:, half:]
        q = 1 / (1 + torch.exp(-zg))
        dz = torch.cat([dy * zu * q * (1 + zg * (1 - q)), dy * zg * q], 1)
    else:
        dz = dy
    return (dz @ w).bfloat16(), (dz.t() @ x).bfloat16(), dz.sum(0)


def run(state):
    if own:
        return _own(state)
    return dict(norm=_norm, balance=_balance, linear=_linear)[state["op"]](state)


# ---- what a pass cannot do without --------------------------------------------------------


def work(case):
    if case["op"] == "norm":
        T, H = case["T"], case["H"]
        rb = 4 if case["r32"] else 2
        gate = dict(none=0, channel=2 * H, token=2 * T, full=2 * T * H)[case["gate"]]
        if case["dir"] == "fwd":
            return dict(bytes=T * H * (2 * rb + 4) + gate + 4 * H, flops=10 * T * H)
        dgate = dict(none=0, channel=4 * H, token=4 * T, full=2 * T * H)[case["gate"]]
        return dict(bytes=T * H * (3 * rb + 6) + gate + dgate + 12 * H, flops=30 * T * H)
    if case["op"] == "balance":
        T, E, k = case["T"], case["E"], case["k"]
        fwd = 4 * T * E + 4 * T * k + (T if case["pad"] else 0) + 4 * E + 16
        return dict(bytes=fwd + (4 * T * E if case["dir"] == "step" else 0), flops=(6 if case["dir"] == "fwd" else 14) * T * E)
    M, N, K = case["M"], case["N"], case["K"]
    cols = N // 2 if case["act"] == "swiglu" else N
    if case["dir"] == "fwd":
        return dict(bytes=2 * (M * K + N * K + M * cols * (2 if case["res"] else 1) + (N if case["bias"] else 0)), flops=2.0 * M * N * K)
    return dict(bytes=2 * (M * cols + 2 * M * K + 2 * N * K + (M * N if case["act"] != "none" else 0)) + 4 * N, flops=4.0 * M * N * K)


# ---- the definitions in 64 bits -----------------------------------------------------------


def exact(case, seed):
    s = prepare(case, seed)
    v = {k: t.double() if isinstance(t, torch.Tensor) and t.is_floating_point() else t for k, t in s.items()}
    if case["op"] == "norm":
        H = case["H"]
        leaves = {k: v[k].clone().requires_grad_(case["dir"] == "bwd") for k in ("r", "y", "w_post", "w_pre")}
        g = None if v["g"] is None else v["g"].clone().requires_grad_(case["dir"] == "bwd")
        a = 1.0 if g is None else torch.sigmoid(g.view(-1, 1) if case["gate"] == "token" else g)
        y, r = leaves["y"], leaves["r"]
        branch = y / torch.sqrt(torch.linalg.vecdot(y, y)[:, None] / H + EPS) * leaves["w_post"]
        r2 = r + SCALE * (a * branch)
        u = r2 / torch.sqrt(torch.linalg.vecdot(r2, r2)[:, None] / H + EPS) * leaves["w_pre"]
        if case["dir"] == "fwd":
            return r2, u
        # the gradients by differentiation of the definition
        asked = [r, y] + ([] if g is None else [g]) + [leaves["w_post"], leaves["w_pre"]]
        got = list(torch.autograd.grad([r2, u], asked, [v["dr_out"], v["du"]]))
        if g is None:
            got.insert(2, None)
        return tuple(got)
    if case["op"] == "balance":
        E, k = case["E"], case["k"]
        keep = slice(None) if v["mask"] is None else v["mask"].bool()
        l = v["logits"].clone().requires_grad_(True)
        kept, idx = l[keep], v["idx"][keep].long()
        n = max(1, kept.shape[0])
        f = torch.nn.functional.one_hot(idx.flatten(), E).sum(0).double() / (n * k)
        bal = E * torch.dot(f, torch.softmax(kept, 1).sum(0) / n)
        z = torch.logsumexp(kept, 1).square().sum() / n
        loss = BALANCE * bal + ZLOSS * z
        out = torch.stack([loss, bal, z]).detach(), None, None
        if case["dir"] == "fwd":
            return out
        return *out, torch.autograd.grad(loss * v["dloss"][0], l)[0]
    half = case["N"] // 2
    acts = dict(none=lambda t: t, relu=torch.relu, gelu=torch.nn.functional.gelu, silu=torch.nn.functional.silu,
                swiglu=lambda t: torch.nn.functional.silu(t[:, :half]) * t[:, half:])
    if case["dir"] == "fwd":
        z = torch.einsum("mk,nk->mn", v["x"], v["w"])
        y = acts[case["act"]](z if v["b"] is None else z + v["b"])
        return y if v["res"] is None else y + v["res"]
    z = v["z"].clone().requires_grad_(True)
    dz = torch.autograd.grad(acts[case["act"]](z), z, v["dy"])[0]
    return torch.einsum("mn,nk->mk", dz, v["w"]), torch.einsum("mn,mk->nk", dz, v["x"]), dz.sum(0)
