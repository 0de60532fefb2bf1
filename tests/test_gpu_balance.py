"""The router's balance loss, its counts and its gradient against the 64-bit definition."""
import math

import pytest
import torch

import block_ref as ref

pytestmark = pytest.mark.gpu
A, B = 0.01, 0.001


def make(T, E, k, pad, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    l = torch.randn(T, E, generator=g, device="cuda") + torch.randn(E, generator=g, device="cuda") * 0.7
    idx = torch.topk(l, k, dim=1).indices.int()
    mask = (torch.rand(T, generator=g, device="cuda") < 0.7).to(torch.uint8) if pad else None
    return l, idx, mask


def check(fe, l, idx, mask, a=A, b=B, up=None):
    loss, counts, n = fe.balance_loss(l, idx, mask=mask, balance_coef=a, z_coef=b)
    dup = None if up is None else torch.tensor([up], device="cuda")
    dl = fe.balance_loss_backward(l, counts, n, idx.shape[1], mask=mask, dloss=dup, balance_coef=a, z_coef=b)
    wl, wc, wn, wd, ml, md = ref.balance(l, idx, mask, a, b, 1.0 if up is None else up)
    assert torch.equal(counts.long(), wc) and int(n) == wn
    # sums of T positive terms: chains of at most T / 4096 + 8 per warp and a tree
    depth = l.shape[0] / 4096 + 64
    ref.close(loss, wl, (ref.FWD + depth * 2.0 ** -24) * ml, "loss")
    ref.close(dl, wd, ref.FWD * md, "dlogits")
    return loss, counts, n, dl


@pytest.mark.parametrize("pad", [False, True])
@pytest.mark.parametrize("T, E, k", [(1, 1, 1), (1, 128, 8), (2, 3, 2), (7, 33, 33), (64, 128, 8), (65, 96, 4), (33, 250, 6), (100, 256, 1),
                                     (9, 511, 10), (20, 512, 10), (13, 1024, 8), (11, 1021, 40), (4099, 128, 8), (20011, 60, 3), (50000, 8, 2)])
def test_loss_counts_and_gradient(T, E, k, pad):
    import fp4_expert_gemv_b200 as fe
    check(fe, *make(T, E, k, pad, seed=T + E), up=None if pad else -1.75)


@pytest.mark.parametrize("T, E, k", [(15003, 512, 10), (60001, 128, 8), (8001, 1024, 40), (30000, 200, 3),
                                     (700, 128, 8), (1536, 128, 8), (1537, 128, 8), (300, 512, 10), (150, 1024, 4),
                                     (9000, 16, 2), (1000, 129, 4), (1100, 129, 4), (4097, 512, 10), (200, 1024, 4),
                                     (900, 1024, 4), (193, 516, 3)])
def test_streamed_batches(T, E, k):
    """Rows for one cluster's rings, for the pass over all SMs and around the sizes between, padded rows holding anything, rows of -inf."""
    import fp4_expert_gemv_b200 as fe
    l, idx, mask = make(T, E, k, True, seed=T)
    l[mask == 0] = float("nan")
    idx[::7, 0] = -1
    l[::11] = -math.inf
    l[5::11, 1:] = -math.inf
    mask[5::11] = 0
    check(fe, l, idx, mask)
    a = fe.balance_loss(l, idx, mask=mask)
    b = fe.balance_loss(l, idx, mask=mask)
    assert all(torch.equal(p, q) for p, q in zip(a, b))


def test_large_logits_keep_their_differences():
    """Softmax depends on differences alone, however large the logits (exact multiples of 2 here)."""
    import fp4_expert_gemv_b200 as fe
    l, idx, _ = make(300, 64, 4, False, seed=8)
    l = torch.round(l * 4) * 2
    base = fe.balance_loss(l, idx)
    for off in (1e4, -1e6, 2.0 ** 23):
        got = fe.balance_loss(l + off, idx)
        assert torch.equal(got[0][1], base[0][1]) and torch.isfinite(got[0]).all()


def test_chosen_ids_given_twice_or_out_of_range():
    import fp4_expert_gemv_b200 as fe
    l, idx, mask = make(50, 40, 4, False, seed=3)
    idx[3] = 7
    idx[5, 1] = -1
    idx[6, 2] = 40
    idx[7] = -(1 << 31)
    check(fe, l, idx, mask)


def test_masked_and_empty_rows():
    import fp4_expert_gemv_b200 as fe
    inf = math.inf
    for E in (40, 41):
        l, idx, _ = make(60, E, 4, False, seed=4)
        l[0] = -inf                       # nothing left
        l[1, 1:] = -inf                   # one expert left
        l[2, ::2] = -inf
        l[3] = -3e38                      # all at the lowest: a uniform row
        l[3] += torch.arange(E, device="cuda") * 0
        l[4, :5] = torch.finfo(torch.float32).min
        mask = torch.ones(60, dtype=torch.uint8, device="cuda")
        mask[5:9] = 0
        l[5] = float("nan")               # padding may hold anything
        l[6] = inf
        idx[7] = 1 << 30
        mask[10] = 255                    # anything but 0 keeps
        loss, _, _, dl = check(fe, l, idx, mask, b=0.0)
        assert (dl[0] == 0).all() and (dl[5:9] == 0).all() and torch.isfinite(dl).all()
        l[3] = 1.0
        check(fe, l, idx, mask)


def test_no_tokens_kept():
    import fp4_expert_gemv_b200 as fe
    l, idx, _ = make(30, 16, 2, False)
    loss, counts, n, dl = check(fe, l, idx, torch.zeros(30, dtype=torch.uint8, device="cuda"))
    assert (loss == 0).all() and (counts == 0).all() and int(n) == 0 and (dl == 0).all()
    loss, counts, n = fe.balance_loss(l[:0], idx[:0])
    assert (loss == 0).all() and (counts == 0).all() and int(n) == 0
    assert fe.balance_loss_backward(l[:0], counts, n, 2).shape == (0, 16)


def test_nan_and_infinite_logits_show():
    import fp4_expert_gemv_b200 as fe
    for bad in (float("nan"), math.inf):
        l, idx, _ = make(30, 64, 2, False)
        l[4, 9] = bad
        loss, counts, n = fe.balance_loss(l, idx, balance_coef=A, z_coef=B)
        assert torch.isnan(loss[:2]).all() and int(counts.sum()) == 60
        dl = fe.balance_loss_backward(l, counts, n, 2, balance_coef=A, z_coef=B)
        assert torch.isnan(dl[4]).any() and torch.isfinite(dl[:4]).all() and torch.isfinite(dl[5:]).all()


def test_unaligned_logits_bf16_gradient_and_in_place():
    import fp4_expert_gemv_b200 as fe
    l, idx, _ = make(70, 128, 8, False, seed=6)
    buf = torch.empty(70 * 128 + 1, device="cuda")
    odd = buf[1:].view(70, 128)
    odd.copy_(l)
    _, counts, n, dl = check(fe, odd, idx, None)
    for src in (l, odd):
        b16 = fe.balance_loss_backward(src, counts, n, 8, balance_coef=A, z_coef=B, dtype=torch.bfloat16)
        assert b16.dtype == torch.bfloat16
        want = ref.balance(l, idx, None, A, B)
        ref.close(b16, want[3], ref.FWD * want[5], "bf16 dlogits")
    again = fe.balance_loss_backward(l, counts, n, 8, balance_coef=A, z_coef=B)
    same = fe.balance_loss_backward(l, counts, n, 8, balance_coef=A, z_coef=B, dlogits=l)
    assert same is l and torch.equal(l, again)


@pytest.mark.parametrize("T, E, k", [(600, 128, 8), (1500, 128, 8), (300, 512, 4), (5000, 128, 8), (3, 1024, 1024)])
def test_unaligned_logits_of_every_size(T, E, k):
    import fp4_expert_gemv_b200 as fe
    l, idx, mask = make(T, E, k, True, seed=T)
    buf = torch.empty(T * E + 1, device="cuda")
    odd = buf[1:].view(T, E)
    odd.copy_(l)
    check(fe, odd, idx, mask)


@pytest.mark.parametrize("E", [16, 128, 512, 516, 1024, 1023])
def test_the_workspace_is_all_that_is_written(E):
    """Every size at which the launches change, with the bytes behind the workspace and the outputs watched."""
    import fp4_expert_gemv_b200 as fe
    R = max(1, 512 // E) if E <= 512 else 1
    for T in sorted({1, 5, 128 * R, 128 * R + 1, 193, 200, 256 * R + 1, 384 * R + 1, 600, 1000, 1185, 3553 * R, 5000}):
        l, idx, _ = make(T, E, 4, False, seed=T)
        nb = fe.fe_moe_balance_workspace(T, E)
        ws = torch.full((nb + 4096,), 85, dtype=torch.uint8, device="cuda")
        out = torch.full((3 + 64,), 5.0, device="cuda")
        ints = torch.full((E + 1 + 64,), 5, dtype=torch.int32, device="cuda")
        st = fe.fe_moe_balance_loss(l.data_ptr(), idx.data_ptr(), None, T, E, 4, 1.0, 0.1, out.data_ptr(), ints.data_ptr(),
                                    ints.data_ptr() + 4 * E, ws.data_ptr(), nb, torch.cuda.current_stream().cuda_stream)
        torch.cuda.synchronize()
        assert st == fe.FE_OK and (ws[nb:] == 85).all() and (out[3:] == 5).all() and (ints[E + 1:] == 5).all(), (T, E)
        want = fe.balance_loss(l, idx, balance_coef=1.0, z_coef=0.1)
        assert torch.equal(out[:3], want[0]) and torch.equal(ints[:E], want[1]) and int(ints[E]) == T


def test_gradient_against_differences():
    """Central differences of the 64-bit loss with the counts held (step error h^2: below 1e-7 here)."""
    import fp4_expert_gemv_b200 as fe
    l, idx, mask = make(40, 24, 3, True, seed=2)
    loss, counts, n, dl = check(fe, l, idx, mask, a=1.0, b=0.3)
    gen = torch.Generator(device="cuda").manual_seed(5)
    for _ in range(4):
        dirn = torch.randn(40, 24, generator=gen, device="cuda", dtype=torch.float64)
        h = 1e-4
        f = [float(ref.balance(l.double() + s * h * dirn, idx, mask, 1.0, 0.3)[0][0]) for s in (1, -1)]
        got = float((dl.double() * dirn).sum())
        assert abs((f[0] - f[1]) / (2 * h) - got) <= 1e-6 + 2.0 ** -18 * float((dl.double() * dirn).abs().sum())


def test_the_same_every_time_on_streams_and_in_graphs():
    import fp4_expert_gemv_b200 as fe
    l, idx, mask = make(9000, 128, 8, True, seed=1)

    def step(stream=None):
        loss, c, n = fe.balance_loss(l, idx, mask=mask, balance_coef=A, z_coef=B, stream=stream)
        return loss, c, n, fe.balance_loss_backward(l, c, n, 8, mask=mask, balance_coef=A, z_coef=B, stream=stream)

    first = step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = [step(side), step()]
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
    l2, idx2, mask2 = make(9000, 128, 8, True, seed=2)
    l.copy_(l2), idx.copy_(idx2), mask.copy_(mask2)
    for g, _ in graphs:
        g.replay()
    want = step()
    torch.cuda.synchronize()
    for _, out in graphs:
        assert all(torch.equal(a, b) for a, b in zip(want, out))


def test_refusals():
    import fp4_expert_gemv_b200 as fe
    l, idx, mask = make(8, 16, 2, True)
    with pytest.raises(ValueError):
        fe.balance_loss(l.bfloat16(), idx)
    with pytest.raises(ValueError):
        fe.balance_loss(l, idx.long())
    with pytest.raises(ValueError):
        fe.balance_loss(l, idx, mask=mask.bool())
    with pytest.raises(ValueError):
        fe.balance_loss(l[:, ::2], idx)
    with pytest.raises(fe.FeMoeError):
        fe.balance_loss(torch.zeros(2, 1025, device="cuda"), idx[:2].contiguous())


@pytest.mark.parametrize("T, E, k", [(50, 64, 4), (700, 128, 8), (3000, 128, 8), (9000, 512, 10), (33, 250, 6), (5000, 1024, 8)])
def test_logits_spread_to_underflow(T, E, k):
    """Every p from 1 down to below the smallest normal number: the exponential's argument d log2 e is rounded three times
    (the difference, the constant and the product), 2^-24 of itself each, so p is off by 3 |d| 2^-24 of
    itself besides what the other tests allow; below 2^-126 it is 0."""
    import fp4_expert_gemv_b200 as fe
    l, idx, mask = make(T, E, k, True, seed=E)
    l = l * 0.1 - torch.rand(T, E, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda") * 100
    a, b = 1.0, 0.1
    loss, counts, n = fe.balance_loss(l, idx, mask=mask, balance_coef=a, z_coef=b)
    dl = fe.balance_loss_backward(l, counts, n, k, mask=mask, balance_coef=a, z_coef=b)
    wl, wc, wn, wd, ml, md = ref.balance(l, idx, mask, a, b)
    assert torch.equal(counts.long(), wc) and int(n) == wn
    depth = T / 4096 + 64
    # the loss holds sums of p: a small p's own error is small beside them
    ref.close(loss, wl, (ref.FWD + depth * 2.0 ** -24) * ml, "loss")
    d = (l.double().max(1, keepdim=True).values - l.double()).clamp(max=100)
    lse = torch.logsumexp(l.double(), 1).abs()[:, None]
    flushed = 2.0 ** -126 * (a * E * 2 + 2 * b * (lse + 1)) / max(wn, 1)
    ref.close(dl, wd, (ref.FWD + 3 * d * 2.0 ** -24) * md + flushed, "dlogits")
    assert (wd.abs() > 0).float().mean() > 0.3
