"""Plain 64-bit forms of the row operators, with bounds on what float32 arithmetic
and one rounding may be off from them.

u = 2^-24 is float32's unit roundoff: one operation is off by at most u relative to
its result.  A sum of n terms, however it is associated over d additions in a row, is
off by at most d u times the sum of the terms' magnitudes.  An output rounded to type
t is off by finfo(t).eps / 2 relative, and by half the smallest subnormal.
"""

import math

import torch

U = 2.0 ** -24
F64 = torch.float64


def rounded(value, err, dtype):
    """Bound of |round(computed) - value| for a computed value within `err` of `value`."""
    fi = torch.finfo(dtype)
    return (value.abs() + err) * (fi.eps / 2) + err + fi.smallest_normal * fi.eps / 2


def check(got, want, tol, what):
    got = got.to(F64)
    assert got.shape == want.shape, (what, got.shape, want.shape)
    off = (got - want).abs()
    bad = ~(off <= tol)
    bad &= ~((got == want) | (got.isnan() & want.isnan()))
    if bad.any():
        at = tuple(int(i) for i in bad.nonzero()[0])
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} off, first at {at}: "
                             f"{got[at].item()!r} for {want[at].item()!r}, tolerance {tol[at].item():.3g}")


# ---------------------------------------------------------------- norm

def norm(bufs, residual, weight, eps):
    """(h, rstd, y) and their float32 error bounds (eh, er, ey)."""
    p = len(bufs)
    h = torch.zeros(bufs[0].shape, dtype=F64, device=bufs[0].device)
    a = torch.zeros_like(h)
    for b in bufs:
        h += b.to(F64)
        a += b.to(F64).abs()
    if residual is not None:
        h += residual.to(F64)
        a += residual.to(F64).abs()
    n = h.shape[1]
    # p + 1 additions in a row
    eh = (p + 1) * U * a
    ms = (h * h).mean(1, keepdim=True) + eps
    r = ms.rsqrt()
    # the squares: at most 32 in a row in a lane, 6 + 16 additions over lanes and waves;
    # half of it in the root, then the product with 1 / n, eps, root and quotient: 27 + 5.
    # h's own error moves the mean by 2 sum |h| eh / n, half of that relative to ms in r.
    er = r * (32 * U + (h.abs() * eh).mean(1, keepdim=True) / ms)
    w = weight.to(F64)
    y = h * r * w
    ey = (r * w).abs() * eh + (h * w).abs() * er + 3 * U * y.abs()
    return h, r.squeeze(1), y, eh, er.squeeze(1), ey


def norm_backward(dys, h, rstd, weight, dh_in):
    p = len(dys)
    h, w, r = h.to(F64), weight.to(F64), rstd.to(F64).unsqueeze(1)
    g = torch.zeros_like(h)
    a = torch.zeros_like(h)
    for d in dys:
        g += d.to(F64)
        a += d.to(F64).abs()
    x = h * r
    n = h.shape[1]
    dot = (w * g * x).mean(1, keepdim=True)
    # terms: p additions, three products; the sum: 32 + 22 additions, 1 / n
    edot = (w * a * x).abs().mean(1, keepdim=True) * (p + 60) * U
    d0 = torch.zeros_like(h) if dh_in is None else dh_in.to(F64)
    dh = d0 + r * (w * g - x * dot)
    edh = r * (w.abs() * a * (p + 3) * U + x.abs() * edot) + 5 * U * (d0.abs() + r * ((w * g).abs() + (x * dot).abs()))
    dw = (g * x).sum(0)
    # a workgroup takes at most t / 512 + 1 rows; their sums go 32 + 16 in a row
    t = h.shape[0]
    edw = (a * x.abs()).sum(0) * (t / 512 + 1 + 32 + 16 + p + 3) * U
    return dh, dw, edh, edw


# ---------------------------------------------------------------- cross entropy

def xent(x, targets, valid, dloss, grad_scale):
    """(loss, lse, grad) for logits x [tokens, vocab] and their bounds.

    exp(x - m) as 2^((x - m) log2 e): the argument is off by 2 u relative (product,
    constant), which is 2 u |x - m| in the result, and the exponential by 2 u; a term
    passes at most 13 joins over lanes, waves and parts, each a product with another
    such exponential, whose arguments add up to no more than m - x."""
    x = x.to(F64).clone()
    t, v = x.shape
    x[:, valid:] = -math.inf
    m = x.amax(1, keepdim=True)
    at = torch.where(m.isinf(), torch.zeros_like(m), m)
    e = torch.exp(x - at)
    z = e.sum(1, keepdim=True)
    lse = (m + torch.log(z)).squeeze(1)
    # where there is nothing, (x - at) is -inf and its share 0
    far = torch.where(x.isinf(), torch.zeros_like(x), (at - x))
    share = torch.where(z > 0, e / z, torch.zeros_like(e))
    depth = 32 + v / 256 + 6 + 16 + 64      # additions in a row: a lane, the wave, the waves, the parts
    ez = ((60 + depth) + 4 * (share * far).sum(1, keepdim=True)) * U
    live = (targets >= 0) & (targets < valid)
    y = torch.where(live, targets, torch.zeros_like(targets)).long().unsqueeze(1)
    xy = x.gather(1, y)
    loss = (torch.log(z) + (m - xy)).squeeze(1)
    logz = torch.log(z).abs()
    eloss = (ez + 2.0 ** -22 + 4 * U * logz + 2 * U * (logz + (at - xy).abs())).squeeze(1)
    elses = (ez + 2.0 ** -22 + 4 * U * logz).squeeze(1) + U * (lse.abs() + m.squeeze(1).abs())
    empty = (z == 0).squeeze(1)
    loss = torch.where(empty, math.inf, loss)
    lse = torch.where(empty, -math.inf, lse)
    loss = torch.where(targets < 0, 0.0, loss)
    loss = torch.where(targets >= valid, math.nan, loss)
    c = grad_scale * (torch.ones(t, dtype=F64, device=x.device) if dloss is None else dloss.to(F64))
    one = torch.zeros_like(x).scatter_(1, y, 1.0) * live.unsqueeze(1)
    grad = c.unsqueeze(1) * (share - one)
    grad = torch.where(((targets < 0) | (live & empty)).unsqueeze(1), 0.0, grad)
    grad[targets >= valid] = math.nan
    grad[:, valid:] = 0.0
    cc = c.abs().unsqueeze(1)
    # the exponential gives 0 below float32's smallest normal number, 2^-126, relative to a z that
    # is at least 2 to the minus rounding of m log2 e (u of itself), and never below 2^-100
    flushed = 2.0 ** -126 * torch.exp2((at.abs() * 1.45 * U).clamp_max(100.0))
    egrad = cc * (share * ((6 + 2 * far) * U + ez) + 3 * U * one + flushed) + U * grad.abs()
    zero = torch.zeros_like
    return (loss, lse, grad, torch.where(eloss.isfinite(), eloss, zero(eloss)),
            torch.where(elses.isfinite(), elses, zero(elses)), torch.where(egrad.isfinite(), egrad, zero(egrad)))


# ---------------------------------------------------------------- embedding

def embedding(table, ids, scale):
    v = table.shape[0]
    at = ids.long().clamp(0, v - 1)
    y = table.to(F64)[at] * scale
    y[ids < 0] = 0.0
    y[ids >= v] = math.nan
    return y, 3 * U * y.abs()      # the factor in float32, the product


def embedding_backward(dy, ids, vocab, scale, old):
    h = dy.shape[1]
    k = ((ids >= 0) & (ids < vocab)).nonzero().squeeze(1)
    at = ids[k].long()
    d = torch.zeros((vocab, h), dtype=F64, device=dy.device).index_add_(0, at, dy[k].to(F64))
    a = torch.zeros_like(d).index_add_(0, at, dy[k].to(F64).abs())
    n = torch.bincount(at, minlength=vocab).to(F64).unsqueeze(1)
    err = (n + 3) * U * a * abs(scale)
    d *= scale
    if old is not None:
        d += old.to(F64)
        err += U * d.abs() + U * old.to(F64).abs()
    return d, err, n.squeeze(1) > 0
