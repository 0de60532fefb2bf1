"""The operators around the experts without a GPU: every call here is refused on the host before
anything is enqueued, or has nothing to do."""
import pytest
import torch

import fp4_expert_gemv_b200 as fe

A, B, C, D, F, G, W = (i << 30 for i in range(1, 8))   # aligned, far apart; never dereferenced
INV, UNS, CAP, OK = fe.FE_ERR_INVALID_ARG, fe.FE_ERR_UNSUPPORTED, fe.FE_ERR_CAPACITY, fe.FE_OK


def norm(**kw):
    a = dict(r=A, dt=0, y=B, w_post=C, gate=None, kind=0, scale=1.0, w_pre=D, eps=1e-6, T=4, H=64, r_out=F, u=G)
    a.update(kw)
    return fe.fe_moe_block_norm(*a.values(), None)


@pytest.mark.parametrize("kw, want", [
    (dict(T=-1), INV), (dict(H=0), INV), (dict(dt=2), INV), (dict(eps=0.0), INV), (dict(eps=float("nan")), INV),
    (dict(eps=float("inf")), INV), (dict(r=None), INV), (dict(kind=1), INV), (dict(gate=W), INV),
    (dict(gate=W, kind=4), INV), (dict(kind=16), INV), (dict(gate=W, kind=16), INV), (dict(u=None), INV),
    (dict(w_pre=None), INV), (dict(y=None), INV), (dict(y=None, w_post=None), INV), (dict(r_out=None, u=None, w_pre=None), INV),
    (dict(r=A + 1), INV), (dict(dt=1, r=A + 2), INV), (dict(u=G + 1), INV), (dict(H=16385), UNS), (dict(T=1 << 31), UNS),
    (dict(r_out=A + 2), INV), (dict(u=A), INV), (dict(u=B + 16), INV), (dict(r_out=B), INV), (dict(u=F + 8), INV),
    (dict(r_out=C - 16), INV), (dict(gate=W, kind=3, u=W + 500), INV), (dict(T=0), OK), (dict(T=0, r=None, y=None), OK),
])
def test_norm_refusals(kw, want):
    assert norm(**kw) == want


def norm_bwd(**kw):
    X = 100 << 30
    a = dict(dr_out=A, du=B, r=C, dt=0, y=D, w_post=F, gate=None, kind=0, scale=1.0, w_pre=G, eps=1e-6, T=4, H=64, dr=X,
             dy=X + (1 << 20), dgate=None, dw_post=X + (2 << 20), dw_pre=X + (3 << 20), ws=X + (4 << 20),
             nb=fe.fe_moe_block_norm_workspace(4, 64))
    a.update(kw)
    return fe.fe_moe_block_norm_backward(*a.values(), None)


@pytest.mark.parametrize("kw, want", [
    (dict(du=None), INV), (dict(w_pre=None), INV), (dict(dr_out=None, du=None, w_pre=None, dw_pre=None), INV),
    (dict(y=None), INV), (dict(dgate=W), INV), (dict(dw_post=W + 2), INV), (dict(ws=None), INV), (dict(nb=8), CAP),
    (dict(dr=A + 4), INV), (dict(dr=C), INV), (dict(dy=B), INV), (dict(dw_pre=A), INV), (dict(ws=100 << 30), INV),
    (dict(dr=None, dy=None, dw_post=None, dw_pre=None), INV), (dict(w_post=None), INV), (dict(T=-4), INV),
    (dict(gate=W, kind=3, dgate=W), INV), (dict(gate=W, kind=2, dgate=W + 4), INV), (dict(H=20000), UNS),
])
def test_norm_backward_refusals(kw, want):
    assert norm_bwd(**kw) == want


def balance(**kw):
    a = dict(logits=A, idx=B, mask=None, T=50000, E=8, k=2, a=1.0, b=0.0, loss=C, counts=D, n=F, ws=G,
             nb=fe.fe_moe_balance_workspace(50000, 8))
    a.update(kw)
    return fe.fe_moe_balance_loss(*a.values(), None)


@pytest.mark.parametrize("kw, want", [
    (dict(T=-1), INV), (dict(E=0), INV), (dict(k=0), INV), (dict(k=9), INV), (dict(logits=None), INV), (dict(idx=None), INV),
    (dict(loss=None), INV), (dict(counts=None), INV), (dict(n=None), INV), (dict(ws=None), INV), (dict(nb=8), CAP),
    (dict(logits=A + 2), INV), (dict(idx=B + 1), INV), (dict(counts=C + 8), INV), (dict(loss=A + 4), INV), (dict(ws=B), INV),
    (dict(E=1025, k=2), UNS), (dict(T=1 << 30, k=2, E=8), UNS), (dict(mask=G + 4), INV),
])
def test_balance_refusals(kw, want):
    assert balance(**kw) == want


def balance_bwd(**kw):
    a = dict(logits=A, counts=B, n=C, mask=None, dloss=None, T=16, E=8, k=2, a=1.0, b=0.0, dl=D, dt=1)
    a.update(kw)
    return fe.fe_moe_balance_loss_backward(*a.values(), None)


@pytest.mark.parametrize("kw, want", [
    (dict(dt=2), INV), (dict(counts=None), INV), (dict(n=None), INV), (dict(dl=None), INV), (dict(dl=D + 2), INV),
    (dict(dl=A, dt=0), INV), (dict(dl=A + 4), INV), (dict(dl=B), INV), (dict(E=2000), UNS), (dict(dloss=D + 4), INV),
    (dict(T=0, dl=None, counts=None), OK), (dict(k=9), INV), (dict(logits=None), INV),
])
def test_balance_backward_refusals(kw, want):
    assert balance_bwd(**kw) == want


def linear(**kw):
    a = dict(x=A, ldx=64, w=B, bias=None, res=None, ldr=0, M=16, N=32, K=64, act=0, y=C, ldy=32, z=None)
    a.update(kw)
    return fe.fe_moe_linear(*a.values(), None)


@pytest.mark.parametrize("kw, want", [
    (dict(M=-1), INV), (dict(N=0), INV), (dict(K=0), INV), (dict(act=5), INV), (dict(act=-1), INV), (dict(act=4, N=31), INV),
    (dict(K=60, ldx=64), UNS), (dict(ldx=68), UNS), (dict(ldx=56), INV), (dict(ldy=31), INV), (dict(res=D, ldr=31), INV),
    (dict(x=None), INV), (dict(w=None), INV), (dict(y=None), INV), (dict(x=A + 8), INV), (dict(w=B + 2), INV),
    (dict(y=C + 1), INV), (dict(y=A), INV), (dict(y=B + 64), INV), (dict(z=C), INV), (dict(z=A + 16), INV),
    (dict(res=C, ldr=64), INV), (dict(res=C + 2, ldr=32), INV), (dict(bias=C + 4), INV), (dict(M=0, x=None, y=None), OK),
    (dict(M=(1 << 31) - 1, y=1 << 45, ldy=1 << 10), UNS),
])
def test_linear_refusals(kw, want):
    assert linear(**kw) == want


def linear_bwd(**kw):
    a = dict(dy=A, lddy=16, x=B, ldx=64, w=C, z=D, M=16, N=32, K=64, act=4, dx=F, lddx=64, dw=G, db=W, ws=100 << 30,
             nb=fe.fe_moe_linear_workspace(16, 32, 64, 4))
    a.update(kw)
    return fe.fe_moe_linear_backward(*a.values(), None)


@pytest.mark.parametrize("kw, want", [
    (dict(dy=None), INV), (dict(z=None), INV), (dict(x=None), INV), (dict(w=None), INV), (dict(ws=None), INV), (dict(nb=64), CAP),
    (dict(lddy=15), INV), (dict(ldx=68), UNS), (dict(ldx=56), INV), (dict(lddx=63), INV), (dict(dx=None, dw=None, db=None), INV),
    (dict(dx=A), INV), (dict(dw=C), INV), (dict(db=G + 8), INV), (dict(db=W + 2), INV), (dict(ws=(100 << 30) + 8), INV),
    (dict(K=60), UNS), (dict(N=31), INV), (dict(ws=B), INV), (dict(dx=D + 2), INV),
])
def test_linear_backward_refusals(kw, want):
    assert linear_bwd(**kw) == want


def test_workspace_queries_answer_zero_for_refused_sizes():
    assert fe.fe_moe_block_norm_workspace(4, 0) == 0 and fe.fe_moe_block_norm_workspace(4, 16385) == 0
    assert fe.fe_moe_balance_workspace(4, 1025) == 0 and fe.fe_moe_balance_workspace(-1, 8) == 0
    assert fe.fe_moe_balance_workspace(64, 128) == 0 and fe.fe_moe_balance_workspace(50000, 128) > 8 * 128
    assert fe.fe_moe_linear_workspace(4, 8, 12, 0) == 0 and fe.fe_moe_linear_workspace(4, 7, 16, 4) == 0
    assert fe.fe_moe_forward_block_workspace(None, 4, 8) == 0
    # at least dz [M][N rounded up to 8] in bf16 and one partial row of column sums
    assert fe.fe_moe_linear_workspace(100, 33, 64, 0) >= 100 * 40 * 2 + 33 * 4


def test_forward_block_needs_a_handle():
    assert fe.fe_moe_forward_block(None, None, A, 0, None, 1, 1, B, None, C, D, 1 << 20, None) == INV


def test_the_binding_refuses_before_the_library():
    """CPU tensors, wrong types, shapes and orders never reach the C entry points."""
    bf = torch.bfloat16
    r, w = torch.zeros(4, 64, dtype=bf), torch.ones(64, dtype=bf)
    with pytest.raises(ValueError):
        fe.block_norm(r, w_pre=w)                                # not on a GPU
    with pytest.raises(ValueError):
        fe.block_norm(torch.zeros(4, 64, dtype=torch.float16), w_pre=w)
    with pytest.raises(ValueError):
        fe.balance_loss(torch.zeros(4, 8), torch.zeros(4, 2, dtype=torch.int64))
    with pytest.raises(ValueError):
        fe.linear(r, torch.zeros(8, 32, dtype=bf))
    with pytest.raises(ValueError):
        fe.linear_backward(r, r, torch.zeros(64, 64, dtype=bf), act=fe.ACT_SILU)


def test_the_binding_refuses_to_lose_a_gradient():
    """No call records a graph: an operand or a given output that requires grad is refused while grad mode is on, and
    taken without it (here up to the next check, which wants a GPU)."""
    bf = torch.bfloat16
    f = lambda *s, dtype=bf: torch.zeros(*s, dtype=dtype)
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)
    r, w, lg = f(4, 64), f(64), f(4, 8, dtype=torch.float32)
    kw = dict(y=f(4, 64), w_post=w, w_pre=f(64), gate=f(64), gate_kind=fe.GATE_CHANNEL)
    calls = [
        (fe.block_norm, dict(r=r, r_out=f(4, 64), u=f(4, 64), **kw)),
        (fe.block_norm_backward, dict(dr_out=f(4, 64), du=f(4, 64), r=r, **kw)),
        (fe.balance_loss, dict(logits=lg, loss=f(3, dtype=torch.float32))),
        (fe.balance_loss_backward, dict(logits=lg, dloss=f(1, dtype=torch.float32), dlogits=f(4, 8))),
        (fe.linear, dict(x=r, w=f(32, 64), bias=f(32), residual=f(4, 32), y=f(4, 32), z=f(4, 32))),
        (fe.linear_backward, dict(dy=f(4, 32), x=r, w=f(32, 64), z=f(4, 32))),
    ]
    whole = {fe.balance_loss: dict(idx=i32(4, 2)), fe.balance_loss_backward: dict(counts=i32(8), n_tokens=i32(1), top_k=2)}
    for fn, args in calls:
        rest = whole.get(fn, {})
        with pytest.raises(ValueError, match="CUDA tensors"):
            fn(**args, **rest)
        for name, t in args.items():
            if not isinstance(t, torch.Tensor):
                continue
            with_grad = {**args, name: t.clone().requires_grad_()}
            with pytest.raises(ValueError, match=f"{name} requires grad"):
                fn(**with_grad, **rest)
            with torch.no_grad(), pytest.raises(ValueError, match="CUDA tensors"):
                fn(**with_grad, **rest)


def test_linear_backward_of_no_rows_may_have_no_dx():
    """The gradient of an empty x has no address (torch gives an empty tensor none)."""
    none = dict(M=0, dy=None, x=None, z=None, dx=None, dw=None, db=None, ws=None, nb=0)
    assert linear_bwd(**none) == OK and linear_bwd(**none, act=0) == OK
    assert linear_bwd(**{**none, "M": 1}) == INV


def test_linear_backward_asks_for_what_it_writes():
    """dz [M][N rounded up to 8] in bf16 unless dy itself serves, rounded up to 256 bytes, and partial sums of db."""
    q = fe.fe_moe_linear_backward_workspace
    for M, N, K, act in ((16, 32, 64, 0), (100, 33, 64, 0), (100, 32, 64, 4), (2_200_000, 1024, 64, 0)):
        dz = (2 * M * ((N + 7) // 8 * 8) + 255) // 256 * 256
        db = 4 * N * max(1, min(256, (M + 31) // 32))
        for rows16 in (0, 1):
            for dx, dw, b in ((1, 1, 1), (1, 0, 0), (0, 1, 0), (0, 0, 1), (1, 0, 1)):
                want = (dz if (dx or dw) and not (act == 0 and rows16) else 0) + (db if b else 0)
                assert q(M, N, K, act, rows16, dx, dw, b) == want, (M, N, act, rows16, dx, dw, b)
        assert fe.fe_moe_linear_workspace(M, N, K, act) == dz + db
    assert q(4, 8, 12, 0, 0, 1, 1, 1) == 0
    # a byte less, or none where some is needed, is refused
    for kw in (dict(), dict(act=0, z=None, lddy=33, N=32), dict(dx=None, dw=None)):
        a = dict(dict(M=16, N=32, K=64, act=4, lddy=16, dx=F, dw=G), **kw)
        nb = q(a["M"], a["N"], a["K"], a["act"], a["lddy"] % 8 == 0, a["dx"] is not None, a["dw"] is not None, 1)
        assert nb > 0 and linear_bwd(**kw, nb=nb - 1) == CAP and linear_bwd(**kw, nb=nb, ws=None) == INV


def test_the_norms_workspace_is_what_the_partials_take():
    """Three sums of H floats from each of up to two CTAs on 148 SMs, a row each at least."""
    for T, H in ((1, 8), (100, 2048), (296, 64), (4096, 2048), (1 << 30, 16384)):
        assert fe.fe_moe_block_norm_workspace(T, H) == 12 * H * min(T, 2 * 148)


def test_rows_beside_each_other_do_not_overlap():
    """Columns of one buffer serve as operand and output where they are apart; a column in common is refused.  (What is
    not refused here is refused afterwards for z, so that nothing is enqueued.)"""
    # x in columns 0..63, y in 64..95, the residual in 96..127 of rows of 128, z over the weights
    ok = dict(x=A, ldx=128, y=A + 128, ldy=128, res=A + 192, ldr=128, w=B, z=B)
    assert linear(**ok) == INV                                      # z alone
    assert linear(**{**ok, "z": None, "y": A + 126}) == INV         # y over x's last column
    assert linear(**{**ok, "z": None, "y": A + 130}) == INV         # y over the residual's first
    assert linear(**{**ok, "z": None, "y": A + 2 * 100, "res": None}) == INV   # y runs into the next row's x
    assert linear(**{**ok, "z": None, "ldy": 130}) == INV           # strides that drift apart
