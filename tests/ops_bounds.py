"""Float64 references of cross attention, layer norm and gradient clipping, each with an elementwise
bound on how far a correct kernel's result may be from it.

The bounds are sums of the roundings a kernel makes: u = 2^-24 for each fp32 operation (a sum of n
terms: n u times the sum of magnitudes), and r = half a step of the I/O type (2^-8 for bfloat16, u
for float32) for each value that is rounded to it: the results themselves and, on the bfloat16 path
of attention, the probabilities and dS that feed the second products.
"""
import math

import torch

U = 2.0 ** -24


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def cross(q, k, v, mask, scale=None, dO=None):
    """name -> (reference, bound) for o, lse and, with dO, dq, dk, dv."""
    dt = q.dtype
    r = half_step(dt)
    rp = r if dt == torch.bfloat16 else 0.0  # rounding of P and dS
    q, k, v = q.double(), k.double(), v.double()
    B, H, N, d = q.shape
    HK, L = k.shape[1], k.shape[2]
    G = H // HK
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    if mask is None:
        mask = torch.ones(B, L, dtype=torch.bool, device=q.device)
    on = mask.bool()[:, None, :, None]
    # what a masked state holds takes no part
    k = torch.where(on, k, torch.zeros_like(k))
    v = torch.where(on, v, torch.zeros_like(v))
    ke, ve = k.repeat_interleave(G, 1), v.repeat_interleave(G, 1)
    s = scale * q @ ke.transpose(2, 3)
    s = s.masked_fill(~mask.bool()[:, None, None, :], -math.inf)
    some = mask.bool().any(1)[:, None, None].expand(B, H, N)
    lse = torch.where(some, torch.logsumexp(s, 3), torch.full_like(s[..., 0], -math.inf)) if L else \
        torch.full((B, H, N), -math.inf, dtype=q.dtype, device=q.device)
    p = torch.exp(s - torch.where(some, lse, torch.zeros_like(lse))[..., None])
    o = p @ ve
    # a logit: a product of d terms, its scaling, and the subtraction of the row's reference
    es = (d + 4) * U * scale * (q.abs() @ ke.abs().transpose(2, 3))
    fin = torch.where(torch.isfinite(s), s.abs(), torch.zeros_like(s))
    row = (es + 4 * U * fin).amax(3) if L else torch.zeros_like(lse)
    # p relative to the row's sum: numerator and denominator (L terms), the exponential (2^-21)
    ep = (2 * row + (L + 8) * U + 2.0 ** -21)[..., None]
    out = {}
    a = p @ ve.abs()
    bo = a * (rp + ep + L * U) + r * o.abs() + 1e-30
    out["o"] = (o, bo)
    out["lse"] = (lse, row + 2.0 ** -20 + 2 * U * torch.where(some, lse, torch.zeros_like(lse)).abs())
    if dO is None:
        return out
    g = dO.double()
    dp = g @ ve.transpose(2, 3)
    D = (g * o).sum(3, keepdim=True)
    ds = p * (dp - D) * scale
    # D is taken from the rounded o; dP is a product of d terms
    eD = (g.abs() * bo).sum(3, keepdim=True) + d * U * (g * o).abs().sum(3, keepdim=True)
    edp = (d + 4) * U * (g.abs() @ ve.abs().transpose(2, 3))
    eds = (rp + ep) * ds.abs() + scale * p * (eD + edp + 4 * U * (dp.abs() + D.abs()))
    fold = lambda x: x.reshape(B, HK, G, L, d).sum(2)  # noqa: E731  a KV head's query heads

    def product(m, em, x, n):
        """m @ x with errors em in m, n terms a sum."""
        return m @ x, em @ x.abs() + n * U * (m.abs() @ x.abs())

    dq, bq = product(ds, eds, ke, L + 2)
    out["dq"] = (dq, bq + r * dq.abs() + 1e-30)
    t = lambda x: x.transpose(2, 3)  # noqa: E731
    dk, bk = product(t(ds), t(eds), q, G * N + 64)
    dv, bv = product(t(p), t((rp + ep) * p), g, G * N + 64)
    dk, bk, dv, bv = fold(dk), fold(bk), fold(dv), fold(bv)
    out["dk"] = (dk, bk + r * dk.abs() + 1e-30)
    out["dv"] = (dv, bv + r * dv.abs() + 1e-30)
    return out


def layer_norm(x, w, b, eps, dy=None, wdtype=torch.float32):
    """name -> (reference, bound) for y, mean, rstd and, with dy, dx, dweight, dbias."""
    r, rw = half_step(x.dtype), half_step(wdtype)
    x = x.double().reshape(-1, x.shape[-1])
    R, C = x.shape
    one = torch.ones(C, dtype=torch.float64, device=x.device)
    w = one if w is None else w.double()
    b = 0 * one if b is None else b.double()
    mu = x.mean(1, keepdim=True)
    xc = x - mu
    var = (xc * xc).mean(1, keepdim=True)
    rs = 1 / torch.sqrt(var + eps)
    xh = xc * rs
    y = xh * w + b
    emu = (C + 2) * U * x.abs().mean(1, keepdim=True)
    exc = emu + U * (x.abs() + mu.abs())             # of x - mu
    evar = 2 * (xc.abs() * exc).mean(1, keepdim=True) + (exc * exc).mean(1, keepdim=True) + (C + 4) * U * var
    ers = 0.5 * evar / (var + eps) * 1.01 + 4 * U     # relative error of rstd
    exh = exc * rs * (1 + ers) + xh.abs() * (ers + 2 * U)
    out = {"y": (y, w.abs() * exh + 2 * U * (y.abs() + b.abs()) + r * y.abs()),
           "mean": (mu[:, 0], emu[:, 0]), "rstd": (rs[:, 0], (rs * ers)[:, 0])}
    if dy is None:
        return out
    dy = dy.double().reshape(R, C)
    g = dy * w
    mg, mgx = g.mean(1, keepdim=True), (g * xh).mean(1, keepdim=True)
    emg = (C + 4) * U * g.abs().mean(1, keepdim=True)
    emgx = (C + 4) * U * (g * xh).abs().mean(1, keepdim=True) + (g.abs() * exh).mean(1, keepdim=True)
    dx = rs * (g - mg - xh * mgx)
    edx = rs * (emg + xh.abs() * emgx + exh * (mgx.abs() + emgx)
                + 8 * U * (g.abs() + mg.abs() + (xh * mgx).abs())) + dx.abs() * (ers + 2 * U)
    out["dx"] = (dx, edx + r * dx.abs())
    dw, db = (dy * xh).sum(0), dy.sum(0)
    out["dweight"] = (dw, (dy.abs() * exh).sum(0) + (R + 16) * U * (dy * xh).abs().sum(0) + rw * dw.abs())
    out["dbias"] = (db, (R + 16) * U * dy.abs().sum(0) + rw * db.abs())
    return out


def clip(grads, max_norm):
    """(norm, its bound), [(out, bound)]: fp32 squares in sums of up to 64, then float64."""
    norm = math.sqrt(sum(float((g.double() ** 2).sum()) for g in grads))
    coef = min(1.0, max_norm / (norm + 1e-6)) if math.isfinite(norm) else max_norm / (norm + 1e-6)
    outs = [(g.double() * coef, (g.double() * coef).abs() * (80 * U + half_step(g.dtype)) + 2.0 ** -133)
            for g in grads]
    return norm, norm * 70 * U, outs


def check(got, want, what):
    ref, bound = want
    got = got.double().reshape(ref.shape)
    same = torch.isfinite(ref) == torch.isfinite(got)
    assert bool(same.all()), f"{what}: non-finite values differ at {int((~same).sum())} places"
    inf = ~torch.isfinite(ref)
    assert bool((got[inf] == ref[inf]).all()), f"{what}: infinities differ"
    err = (got - ref).abs()
    err[inf] = 0
    over = err > bound * 1.0 + 0.0
    over &= ~inf
    if bool(over.any()):
        i = int((err / bound.clamp_min(1e-300)).masked_fill(inf, 0).argmax())
        raise AssertionError(
            f"{what}: {int(over.sum())} of {over.numel()} beyond the bound; worst {i}: "
            f"{float(got.flatten()[i])} vs {float(ref.flatten()[i])}, bound {float(bound.flatten()[i])}")
