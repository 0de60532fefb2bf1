"""64-bit definitions of the operators around the experts, with the magnitudes their error bounds
scale with.  Test infrastructure: plain torch on float64, nothing of the library.

Every bound counts, for each output, half a step of its type relative to the value
(torch.finfo(t).eps / 2) plus an fp32 evaluation error relative to the sum of the absolute
values of what is added up (cancellation makes the result smaller than its error's scale)."""
import math

import torch

HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
# fp32 evaluation of one element: about 30 roundings of 2^-24, the fast exponential (2 ulp plus half an
# ulp of its argument, |x| < 16: 2^-20 relative) and a row sum of at most 2^14 squares added by 8
# per thread and a tree (25 roundings): below 2^-18 of the summed magnitudes forward; the backward
# pass chains two such row sums and forward values: 2^-16
FWD, BWD = 2.0 ** -18, 2.0 ** -16


def d(t):
    return None if t is None else t.double()


def gate_of(g, kind, sigmoid):
    """a(g) and a'(g), broadcast to rows of H."""
    if g is None:
        return 1.0, 0.0
    g = g.double()
    g = g[:, None] if kind == "token" else g
    if not sigmoid:
        return g, torch.ones_like(g)
    a = 1 / (1 + torch.exp(-g))
    return a, a * (1 - a)


def norm_forward(r, y, w_post, w_pre, g, kind, sigmoid, s, eps):
    """{name: (value, magnitude)}"""
    r, y, w_post, w_pre = d(r), d(y), d(w_post), d(w_pre)
    a, _ = gate_of(g, kind, sigmoid)
    out, mag = r, r.abs()
    if y is not None:
        v = y if w_post is None else w_post * y / ((y * y).mean(1, keepdim=True) + eps).sqrt()
        out = r + s * a * v
        mag = r.abs() + (s * a * v).abs()
    res = dict(r_out=(out, mag))
    if w_pre is not None:
        rho = 1 / ((out * out).mean(1, keepdim=True) + eps).sqrt()
        # an error of r' relative to its magnitudes passes through rho, and through the mean once more
        n_mag = mag * rho
        res["u"] = (w_pre * out * rho, w_pre.abs() * (n_mag + (out * rho).abs() * (n_mag * (out * rho).abs()).mean(1, keepdim=True)))
    return res


def norm_backward(dr_out, du, r, y, w_post, w_pre, g, kind, sigmoid, s, eps):
    """The gradient formulas; {name: (value, magnitude)}."""
    r, y, w_post, w_pre, du = d(r), d(y), d(w_post), d(w_pre), d(du)
    a, da = gate_of(g, kind, sigmoid)
    one = torch.ones((), dtype=torch.float64, device=r.device)
    res = {}
    out, mag = r, r.abs()
    if y is not None:
        rho_y = 1 / ((y * y).mean(1, keepdim=True) + eps).sqrt() if w_post is not None else one
        m = y * rho_y
        wp = w_post if w_post is not None else one
        v = wp * m
        out, mag = r + s * a * v, r.abs() + (s * a * v).abs()
    D = d(dr_out) if dr_out is not None else torch.zeros_like(r)
    Dm = D.abs()
    if du is not None:
        rho = 1 / ((out * out).mean(1, keepdim=True) + eps).sqrt()
        n, dn = out * rho, du * w_pre
        # magnitudes of n: r' can cancel, and its relative error grows by mag / |r'|
        nm = mag * rho * (1 + (mag * mag).mean(1, keepdim=True) * rho * rho)
        D = D + rho * (dn - n * (dn * n).mean(1, keepdim=True))
        Dm = Dm + rho * (1 + (mag * mag).mean(1, keepdim=True) * rho * rho) * (dn.abs() + nm * (dn.abs() * nm).mean(1, keepdim=True))
        res["dw_pre"] = ((du * n).sum(0), (du.abs() * nm).sum(0))
    res["dr"] = (D, Dm)
    if y is not None:
        dv, dvm = s * a * D, (abs(s) * (a.abs() if g is not None else 1.0)) * Dm
        dm, dmm = dv * wp, dvm * wp.abs()
        if w_post is not None:
            res["dw_post"] = ((dv * m).sum(0), (dvm * m.abs()).sum(0))
            res["dy"] = (rho_y * (dm - m * (dm * m).mean(1, keepdim=True)),
                         rho_y * (dmm + m.abs() * (dmm * m.abs()).mean(1, keepdim=True)))
        else:
            res["dy"] = (dm, dmm)
        if g is not None:
            dg, dgm = s * v * D * da, (s * v * da).abs() * Dm
            dim = {"channel": 0, "token": 1}.get(kind)
            res["dgate"] = (dg, dgm) if dim is None else (dg.sum(dim), dgm.sum(dim))
    return res


def balance(logits, idx, mask, a, b, up=1.0):
    """(loss [3], counts [E], n, dlogits, their magnitudes)"""
    l = logits.double()
    T, E = l.shape
    k = idx.shape[1]
    keep = torch.ones(T, dtype=torch.bool, device=l.device) if mask is None else mask != 0
    l = torch.where(keep[:, None], l, torch.zeros_like(l))
    top = l.max(1, keepdim=True).values
    dead = top[:, 0] == -math.inf
    ex = torch.where(dead[:, None], torch.zeros_like(l), torch.exp(l - top))
    tot = ex.sum(1, keepdim=True)
    p = torch.where(dead[:, None] | ~keep[:, None], torch.zeros_like(l), ex / tot)
    lse = torch.where(dead | ~keep, torch.zeros_like(tot[:, 0]), (top + torch.log(tot))[:, 0])
    n = int(keep.sum())
    ids = idx[keep].reshape(-1).long()
    ids = ids[(ids >= 0) & (ids < E)]
    counts = torch.bincount(ids, minlength=E)
    nn = max(n, 1)
    f = counts.double() / (nn * k)
    bal = E * (f * p.sum(0)).sum() / nn
    z = (lse * lse).sum() / nn
    loss = torch.stack([a * bal + b * z, bal, z])
    zmag = ((lse.abs() + 1) ** 2 * (keep & ~dead)).sum() / nn
    mag = torch.stack([abs(a) * bal + abs(b) * zmag, bal, zmag])
    pf = (p * f).sum(1, keepdim=True)
    dl = up / nn * p * (a * E * (f - pf) + 2 * b * lse[:, None])
    dmag = abs(up) / nn * p * (abs(a) * E * (f + pf) + 2 * abs(b) * (lse.abs() + 1)[:, None])
    return loss, counts, n, dl, mag, dmag


def act_parts(act, z):
    """act(z) and its derivative(s) for "none", "relu", "gelu", "silu"."""
    if act == "relu":
        return z.clamp(min=0), (z > 0).double()
    if act == "gelu":
        phi = 0.5 * (1 + torch.erf(z / math.sqrt(2)))
        return z * phi, phi + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    if act == "silu":
        q = 1 / (1 + torch.exp(-z))
        return z * q, q * (1 + z * (1 - q))
    return z, torch.ones_like(z)


def linear(x, w, bias, act, res):
    """(y, z, error scale of y, error scale of z): the scales are the fp32 evaluation errors."""
    x, w, bias, res = d(x), d(w), d(bias), d(res)
    K = x.shape[1]
    z, mag = x @ w.t(), x.abs() @ w.abs().t()
    if bias is not None:
        z, mag = z + bias, mag + bias.abs()
    # the products are exact; every 16 of k are added to the accumulator with an error of at most
    # 2^-22 of the magnitudes so far (the adders may truncate), plus a few final roundings
    ez = (K / 16 + 4) * 2.0 ** -22 * mag
    if act == "swiglu":
        h = z.shape[1] // 2
        q, dq = act_parts("silu", z[:, :h])
        y = q * z[:, h:]
        ey = 1.1 * ez[:, :h] * (z[:, h:].abs() + ez[:, h:]) + (q.abs() + 1.1 * ez[:, :h]) * ez[:, h:] + FWD * y.abs()
    else:
        y, _ = act_parts(act, z)
        ey = 1.13 * ez + FWD * z.abs() * (act != "none")
    if res is not None:
        y, ey = y + res, ey + 2.0 ** -23 * (y.abs() + res.abs())
    return y, z, ey, ez


def linear_dz(dy, z, act):
    dy, z = d(dy), d(z)
    if act == "swiglu":
        h = z.shape[1] // 2
        q, dq = act_parts("silu", z[:, :h])
        dz = torch.cat([dy * z[:, h:] * dq, dy * q], 1)
        mag = torch.cat([(dy * z[:, h:]).abs() * (1 + z[:, :h].abs()), (dy * z[:, :h]).abs()], 1)
        return dz, mag
    if act == "none":
        return dy, dy.abs()
    _, da = act_parts(act, z)
    return dy * da, dy.abs() * (1 + z.abs())


def close(got, want, err, what):
    """|got - want| <= err + half a step of got's type, element by element; same non-finite values."""
    got64, want = got.double(), want.double()
    # a value of 64 bits beyond the type's largest rounds to the type's infinity
    want = torch.where(want.abs() > 1.01 * torch.finfo(got.dtype).max, want.to(got.dtype).double(), want)
    fin = torch.isfinite(want)
    assert torch.equal(torch.isnan(got64), torch.isnan(want)), what
    assert torch.equal(got64[~fin & ~torch.isnan(want)], want[~fin & ~torch.isnan(want)]), what
    tol = HALF[got.dtype] * (want.abs() + err) + err + 2.0 ** -126
    bad = ((got64 - want).abs() > tol) & fin
    assert not bad.any(), (what, int(bad.sum()), got64[bad][:3].tolist(), want[bad][:3].tolist(), tol.expand_as(want)[bad][:3].tolist())
