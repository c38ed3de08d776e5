"""Plain 64-bit forms of the log probabilities, of their gradient, and of the gradients' norm
and clipping, with bounds on what float32 arithmetic and the outputs' rounding may be off
from them (u = 2^-24, as in tests/rows_ref.py)."""

import math

import torch

from tests.rows_ref import F64, U, rounded


def best(x, k):
    """Columns of the k largest values of each row, NaN the largest, of equal ones the lowest first."""
    key = torch.where(x.isnan(), math.inf, x.to(F64))
    key, nan = torch.where(key == 0, 0.0, key), x.isnan()
    # two stable sorts: by value, then NaN in front
    at = torch.sort(key, dim=1, descending=True, stable=True).indices
    again = torch.sort(nan.gather(1, at).int(), dim=1, descending=True, stable=True).indices
    return at.gather(1, again)[:, :k]


def in_float32(w):
    """Values beyond float32's range (from (2 - 2^-24) 2^127 on) are rounded to infinity."""
    return torch.where(w.abs() < (2 - U) * 2.0 ** 127, w, torch.where(w.isnan(), w, w.sign() * math.inf))


def logprobs(x, ids, scale, valid, top):
    """(logprob, entropy, lse, top ids, top log probabilities) of x[:, :valid], and the float32
    bounds of the four that are no ids.

    far_j = scale (m - x_j).  An exponential is off by the roundings of scale log2 e (2 u, relative to
    far_j), of the multiply-add (u far_j), and of itself (2 u).  A lane adds up at most 256 + v / 512
    of them, then come 6 + 16 + 64 additions over lanes, waves and parts, each with a factor
    2^(c - c') that is off by 4 u where it is not one."""
    x = x[:, :valid].to(F64)
    t, v = x.shape
    s = float(torch.tensor(scale, dtype=torch.float32))
    m = x.max(1, keepdim=True).values
    bad = x.isnan().any(1, keepdim=True) | (m == math.inf)
    empty = ((m == -math.inf) & ~bad).squeeze(1)
    at = torch.where(m.isinf(), 0.0, m)
    far = (at - x) * s
    e = torch.exp(-far)
    z = e.sum(1, keepdim=True)
    ln_z = torch.log(z)
    p = torch.where(e > 0, e / z, 0.0)
    near = torch.where(e > 0, far, 0.0)                     # where there is nothing, far is inf and its share 0
    mean = (p * near).sum(1, keepdim=True)
    lse = (s * at + ln_z).squeeze(1)
    ent = (ln_z + mean).squeeze(1)
    depth = 4 * (256 + v / 512 + 6 + 16 + 64)
    ez = (depth + 20 + 4 * mean) * U
    eln = ez + 2.0 ** -22 + 4 * U * ln_z.abs()
    elp = eln + 3 * U * far.abs() + U * (far + ln_z).abs()
    else_ = eln.squeeze(1) + 2 * U * lse.abs()
    eent = (eln + mean * (ez + depth * U + 10 * U) + 4 * U * (p * near * near).sum(1, keepdim=True)
            + U * (ln_z.abs() + 2 * mean)).squeeze(1)
    lp = -far - ln_z
    lp[empty], lse[empty], ent[empty] = -math.inf, -math.inf, 0.0
    for r in (lp, lse, ent):
        r[bad.squeeze(1)] = math.nan
    there = ids.clamp(0, valid - 1).long().unsqueeze(1)
    logprob = torch.where(ids < 0, 0.0, torch.where(ids >= valid, math.nan, lp.gather(1, there).squeeze(1)))
    elogprob = elp.gather(1, there).squeeze(1)
    cols = best(x, top)

    def finite(e):
        return torch.where(e.isfinite(), e, 0.0)
    return ((in_float32(logprob), ent, in_float32(lse), cols, in_float32(lp.gather(1, cols))),
            (finite(elogprob), finite(eent), finite(else_), None, finite(elp.gather(1, cols))))


def logprobs_backward(x, ids, lse, ent, da, db, scale, valid):
    """The gradient, and its float32 bound.  ln p is off by u of itself, its exponential by the rounding of
    the product with log2 e (u, and u of the constant) and by 2 u, and is 0 below 2^-126."""
    full = x.shape
    x = x[:, :valid].to(F64)
    t = x.shape[0]
    s = float(torch.tensor(scale, dtype=torch.float32))
    lse = lse.to(F64).unsqueeze(1)
    ln_p = s * x - lse
    p = torch.exp(ln_p)
    ln0 = torch.where(p > 0, ln_p, 0.0)
    a = torch.zeros(t, 1, dtype=F64, device=x.device) if da is None else da.to(F64).unsqueeze(1)
    a = torch.where(ids.unsqueeze(1) < 0, 0.0, a) if ids is not None else a
    b = torch.zeros_like(a) if db is None else db.to(F64).unsqueeze(1)
    h = torch.zeros_like(a) if db is None else ent.to(F64).unsqueeze(1)
    one = torch.zeros_like(x)
    if ids is not None:
        live = (ids >= 0) & (ids < valid)
        one.scatter_(1, ids.clamp(0, valid - 1).long().unsqueeze(1), 1.0)
        one *= live.unsqueeze(1)
    d = s * (a * one - p * (a + b * (ln0 + h)))
    reach = a.abs() + b.abs() * (ln0.abs() + h.abs())
    err = s * (p * ((10 + 4 * ln0.abs()) * U) * reach + 4 * U * a.abs() * one + 2.0 ** -126 * reach) + U * d.abs()
    zero = (a == 0) & (b == 0) | (lse == -math.inf)
    nan = lse.isnan() | (lse == math.inf)
    if ids is not None:
        zero &= ids.unsqueeze(1) < valid
        nan |= ids.unsqueeze(1) >= valid
    d = torch.where(zero, 0.0, torch.where(nan, math.nan, d))
    grad, bound = torch.zeros(full, dtype=F64, device=x.device), torch.zeros(full, dtype=F64, device=x.device)
    grad[:, :valid], bound[:, :valid] = d, torch.where(err.isfinite(), err, 0.0)
    return grad, bound


def norm(tensors, scale):
    """The norm, as a 64-bit number, and the bound of its float32 output: u, and some 2^-53 for each of the
    additions in a row, fewer than 2^13."""
    total = 0.0
    for t in tensors:
        total += float(torch.linalg.vector_norm(t.to(F64)) ** 2) if t.numel() else 0.0
    n = float(torch.tensor(scale, dtype=torch.float32)) * math.sqrt(total)
    return n, n * (U + 2.0 ** -40)


def factor(n, max_norm, scale):
    """c, rounded to float32 where it is off by 2^-40 at most before: a bound of its error."""
    s = float(torch.tensor(scale, dtype=torch.float32))
    m = float(torch.tensor(max_norm, dtype=torch.float32))
    c = s * min(1.0, m / (n + 1e-6))
    return c, c * (U + 2.0 ** -39)


def scaled(g, c, ec, dtype):
    """g c and the bound of what is rounded to dtype: the factor, and a product in float32."""
    want = g.to(F64) * c
    err = g.to(F64).abs() * ec + U * want.abs() + 2.0 ** -150
    return want, rounded(want, err, dtype)
