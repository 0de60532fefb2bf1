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


def near(got, want, err):
    """Within half a step of bf16 and err, element by element, and not all zero."""
    want = want.double()
    assert ((got.double() - want).abs() <= 2.0 ** -8 * want.abs() + err).all() and (want != 0).any()


def test_the_last_rows_gradients():
    """The last period's gradients against the 64-bit definition (the other tests compare it with the first)."""
    import block_ref as ref
    import fp4_expert_gemv_b200 as fe
    T, H = 1_100_000, 2048
    (r, big_r), (y, big_y) = rows(T, H, bf, 1), rows(T, H, bf, 2)
    (dr, big_dr), (du, big_du) = rows(T, H, bf, 3), rows(T, H, bf, 4)
    w = torch.linspace(0.5, 1.5, H, device="cuda").to(bf)
    got = fe.block_norm_backward(big_dr, big_du, big_r, big_y, w, w, weight_grads=False)
    want = ref.norm_backward(dr, du, r, y, w, w, None, "none", False, 1.0, 1e-6)
    for name, t in zip(("dr", "dy"), got):
        for part in (t[:PERIOD], t[-PERIOD:]):
            near(part, want[name][0], ref.BWD * want[name][1])
    del got, big_r, big_y, big_dr, big_du
    M, N, K = 2_200_000, 1024, 64
    (x, big_x), (dy, big_dy) = rows(M, K, bf, 4), rows(M, N, bf, 5)
    w = (torch.randn(N, K, generator=torch.Generator(device="cuda").manual_seed(6), device="cuda") * K ** -0.5).to(bf)
    z = torch.empty(M, N, dtype=bf, device="cuda")
    fe.linear(big_x, w, act=fe.ACT_SILU, z=z)
    dx, _, _ = fe.linear_backward(big_dy, big_x, w, z=z, act=fe.ACT_SILU, need_dw=False)
    dz, mag = ref.linear_dz(dy, z[-PERIOD:], "silu")
    edz = 2.0 ** -8 * dz.abs() + ref.FWD * mag
    W = w.double()
    err = edz @ W.abs() + (N / 16 + 4) * 2.0 ** -22 * ((dz.abs() + edz) @ W.abs())
    near(dx[-PERIOD:], dz @ W, err)
    assert fe.op_status() == (fe.FE_OK, 0)


@pytest.mark.parametrize("M, N, K", [(2_200_000, 64, 1024), (2_200_000, 1024, 64)])
def test_the_weights_gradient_over_more_rows(M, N, K):
    """Values in {-1, 0, 1}: every sum is a whole number below 2^24 and exact in fp32 whatever the order, so dw and dx are the
    exact sums rounded once, and db is exact."""
    import fp4_expert_gemv_b200 as fe
    g = torch.Generator(device="cuda").manual_seed(8)
    tri = lambda *s: (torch.randint(-1, 2, s, generator=g, device="cuda")).to(bf)
    x, dy, w = tri(PERIOD, K), tri(PERIOD, N), tri(N, K)
    dx, dw, db = fe.linear_backward(dy.repeat(M // PERIOD, 1), x.repeat(M // PERIOD, 1), w)
    n = M // PERIOD
    assert torch.equal(dw, (n * (dy.double().t() @ x.double())).to(bf))
    assert torch.equal(db.double(), n * dy.double().sum(0))
    want = (dy.double() @ w.double()).to(bf)
    assert torch.equal(dx[:PERIOD], want) and torch.equal(dx[-PERIOD:], want) and (want != 0).any()
    assert fe.op_status() == (fe.FE_OK, 0)


def test_one_tile_over_a_billion_rows():
    """dW of one tile whose k steps take a single pair of CTAs seconds: the epilogue's wait lasts as long.  All rows are
    zero but a few, so that every sum is exact."""
    import fp4_expert_gemv_b200 as fe
    M, N, K = 1_200_000_000, 8, 8
    x = torch.zeros(M, K, dtype=bf, device="cuda")
    dy = torch.zeros(M, N, dtype=bf, device="cuda")
    w = torch.ones(N, K, dtype=bf, device="cuda")
    at = torch.tensor([0, 1, 63, 64, 12345, M // 2, M - 2, M - 1], device="cuda")
    g = torch.Generator(device="cuda").manual_seed(3)
    x[at] = torch.randint(-3, 4, (8, K), generator=g, device="cuda").to(bf)
    dy[at] = torch.randint(-3, 4, (8, N), generator=g, device="cuda").to(bf)
    _, dw, db = fe.linear_backward(dy, x, w, need_dx=False)
    assert torch.equal(dw.double(), dy[at].double().t() @ x[at].double())
    assert torch.equal(db.double(), dy[at].double().sum(0))
    assert fe.op_status() == (fe.FE_OK, 0)
