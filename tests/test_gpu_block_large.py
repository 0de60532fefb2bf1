"""Operands of more than 2^31 elements (and 2^32 bytes).  Rows repeat with a period, and every row's outputs depend on
that row alone (and on sums over all rows), so the last period has to come out as the first, bit by bit."""
import pytest
import torch

pytestmark = pytest.mark.gpu
bf = torch.bfloat16
PERIOD = 1000


def rows(n, width, dtype, seed, std=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    base = (torch.randn(PERIOD, width, generator=g, device="cuda") * std).to(dtype)
    return base, base.repeat(n // PERIOD, 1)


def same_ends(t):
    assert torch.equal(t[:PERIOD], t[-PERIOD:])


def test_norm():
    import fp4_expert_gemv_b200 as fe
    T, H = 1_100_000, 2048
    assert T * H > 2 ** 31
    (_, r), (_, y) = rows(T, H, bf, 1), rows(T, H, bf, 2)
    w = torch.linspace(0.5, 1.5, H, device="cuda").to(bf)
    r1, u = fe.block_norm(r, y, w, w)
    same_ends(r1)
    same_ends(u)
    small = fe.block_norm(r[-PERIOD:].contiguous(), y[-PERIOD:].contiguous(), w, w)
    # another kernel may take the short call: both are within half a step of bf16 and 2^-14 of the value
    for a, b in ((r1[-PERIOD:], small[0]), (u[-PERIOD:], small[1])):
        assert ((a.double() - b.double()).abs() <= 2 * (2.0 ** -8 + 2.0 ** -14) * b.double().abs() + 2.0 ** -20).all()
    dr, dy, _, _, _ = fe.block_norm_backward(r1, u, r, y, w, w, weight_grads=False)
    same_ends(dr)
    same_ends(dy)
    assert fe.op_status() == (fe.FE_OK, 0)


def test_balance_loss():
    import fp4_expert_gemv_b200 as fe
    T, E, k = 4_400_000, 512, 4
    assert T * E > 2 ** 31
    base, l = rows(T, E, torch.float32, 3, std=2.0)
    ids = torch.stack([torch.randperm(E, device="cuda")[:k] for _ in range(PERIOD)]).int()
    loss, counts, n = fe.balance_loss(l, ids.repeat(T // PERIOD, 1), z_coef=0.1)
    want = fe.balance_loss(base, ids, z_coef=0.1)
    # a lane adds up one row in 148 * 24, then the partials join: a rounding each
    assert ((loss - want[0]).abs() <= (T / (148 * 24) + 300) * 2.0 ** -24 * want[0].abs()).all()
    assert torch.equal(counts, want[1] * (T // PERIOD)) and int(n) == T
    dl = fe.balance_loss_backward(l, counts, n, k, z_coef=0.1)
    same_ends(dl)
    assert torch.isfinite(dl[-1]).all() and (dl[-1] != 0).any()
    assert fe.op_status() == (fe.FE_OK, 0)


@pytest.mark.parametrize("M, N, K", [(2_200_000, 1024, 64), (2_200_000, 64, 1024), (2_200_000, 1023, 64)])
def test_linear(M, N, K):
    import fp4_expert_gemv_b200 as fe
    assert M * max(N, K) > 2 ** 31
    _, x = rows(M, K, bf, 4)
    _, res = rows(M, N, bf, 5)
    w = (torch.randn(N, K, generator=torch.Generator(device="cuda").manual_seed(6), device="cuda") * K ** -0.5).to(bf)
    z = torch.empty(M, N, dtype=bf, device="cuda")
    y = fe.linear(x, w, act=fe.ACT_SILU, residual=res, z=z)
    same_ends(y)
    same_ends(z)
    want = x[-PERIOD:].double() @ w.double().t()
    mag = x[-PERIOD:].double().abs() @ w.double().abs().t()
    # half a step of bf16, and fp32 sums of K products with a rounding of 2^-22 per 16
    assert ((z[-PERIOD:].double() - want).abs() <= 2.0 ** -8 * want.abs() + (K / 16 + 4) * 2.0 ** -22 * mag).all()
    if N % 8 == 0:
        dx, _, db = fe.linear_backward(res, x, w, z=z, act=fe.ACT_SILU, need_dw=False)
        same_ends(dx)
        assert torch.isfinite(db).all()
    assert fe.op_status() == (fe.FE_OK, 0)
