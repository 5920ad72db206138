"""Plain 64-bit forms of the mixture-of-experts operators, on the host, with bounds
on how far fp32 kernels may be from them (roundings counted as in token_ref: U =
2^-24 a rounding, an exponential of d: (3 |d| + 2) U)."""

import math

import torch

from token_ref import U

TINY = 2.0 ** -126  # exponentials below it may be flushed


def top_ids(x, k):
    """The k largest of each row, NaN above all, equal ones by lower id; -1 for -inf."""
    x = x.detach().cpu().double()
    v = torch.where(torch.isnan(x), torch.full_like(x, math.inf), x)
    order = torch.argsort(-v, dim=1, stable=True)
    # NaN before +inf
    nan = torch.gather(torch.isnan(x), 1, order).to(torch.int8)
    order = torch.gather(order, 1, torch.argsort(-nan, dim=1, stable=True))[:, :k]
    shut = torch.gather(x, 1, order) == -math.inf
    return torch.where(shut, torch.full_like(order, -1), order)


class Route:
    """Weights of listed experts (``w``, bound ``tol``) and their gradient."""

    def __init__(self, x, ids, normalize):
        x = x.detach().cpu().double()
        self.x, self.normalize = x, normalize
        ids = ids.cpu().long()
        n, e = x.shape
        self.ok = (ids >= 0) & (ids < e)
        self.at = torch.where(self.ok, ids, torch.zeros_like(ids))
        listed = torch.where(self.ok, x.gather(1, self.at), torch.full_like(self.at, -math.inf,
                                                                            dtype=x.dtype))
        pool = listed if normalize else x
        m = pool.max(1, keepdim=True).values
        shut = m == -math.inf
        m = torch.where(shut, torch.zeros_like(m), m)
        ep = torch.where(pool == -math.inf, torch.zeros_like(pool), torch.exp(pool - m))
        s = ep.sum(1, keepdim=True)
        self.s = torch.where(shut, torch.ones_like(s), s)
        d = lambda v: torch.where(v == -math.inf, torch.zeros_like(v), (v - m).abs())
        # relative error of the sum: each term's, and the additions one takes part in
        depth = 16 + 6 + 2 if not normalize else ids.shape[1]
        tol_s = ((ep * (3 * d(pool) + 2)).sum(1, keepdim=True) / self.s + depth) * U
        # a slot without an expert weighs 0, in a row without a softmax too
        self.w = torch.where(self.ok, torch.where(listed == -math.inf, torch.zeros_like(listed),
                                                  torch.exp(listed - m)) / self.s,
                             torch.zeros_like(listed))
        self.rel = (3 * d(listed) + 2) * U + tol_s + U
        self.tol = self.w * self.rel * 1.01 + TINY
        if not normalize:
            self.p = ep / self.s
            self.p_tol = self.p * ((3 * d(x) + 2) * U + tol_s + U) * 1.01 + TINY

    def grad(self, dw):
        dw = dw.cpu().double()
        k = dw.shape[1]
        g = torch.where(self.ok, dw, torch.zeros_like(dw))
        some = (g != 0).any(1, keepdim=True)
        gw = g * self.w
        both = gw.sum(1, keepdim=True)
        mag = gw.abs().sum(1, keepdim=True)
        both_tol = (g.abs() * self.tol).sum(1, keepdim=True) + (k + 6) * U * mag
        if self.normalize:
            share = self.w * (g - both)
            tol = (self.tol * (g - both).abs() + self.w * both_tol
                   + 3 * U * self.w * (g.abs() + both.abs()))
        else:
            share, tol = gw, g.abs() * self.tol + 2 * U * gw.abs()
        out = torch.zeros_like(self.x)
        lim = torch.zeros_like(self.x)
        share = torch.where(self.ok, share, torch.zeros_like(share))
        tol = torch.where(self.ok, tol + k * U * share.abs().sum(1, keepdim=True),
                          torch.zeros_like(tol))
        out.scatter_add_(1, self.at, share)
        lim.scatter_add_(1, self.at, tol)
        if not self.normalize:
            out = out - both * self.p
            lim = lim + (both.abs() * self.p_tol + self.p * both_tol
                         + 3 * U * (mag * self.p + out.abs()))
        zero = torch.zeros_like(out)
        return torch.where(some, out, zero), torch.where(some, lim, zero) + TINY * (
            1 + mag + g.abs().sum(1, keepdim=True))


def sort(ids, experts):
    """(offsets, places), by counting in order."""
    flat = ids.reshape(-1).cpu().long()
    ok = (flat >= 0) & (flat < experts)
    key = torch.where(ok, flat, torch.full_like(flat, experts))
    order = torch.sort(key, stable=True).indices
    places = torch.empty_like(flat)
    places[order] = torch.arange(flat.numel())
    places[~ok] = -1
    counts = torch.bincount(key, minlength=experts + 1)[:experts]
    offsets = torch.cat([torch.zeros(1, dtype=torch.long), torch.cumsum(counts, 0)])
    return offsets.int(), places.view(ids.shape).int()


def live(places, rows):
    p = places.cpu().long()
    return (p >= 0) & (p < rows), p.clamp(0, max(rows - 1, 0))


def dispatch(x, places, weights, out):
    """What ``out`` holds after it (its type's rounding included): one product."""
    out = out.cpu().clone()
    ok, at = live(places, out.shape[0])
    x = x.cpu().float()
    for i, j in ok.nonzero().tolist():
        row = x[i] * weights.cpu()[i, j] if weights is not None else x[i]
        out[at[i, j]] = row.to(out.dtype)
    return out


def combine(y, places, weights, old=None):
    """(out, bound) in 64 bits."""
    y = y.detach().cpu().double()
    n, k = places.shape
    ok, at = live(places, y.shape[0])
    w = torch.ones(n, k, dtype=torch.float64) if weights is None else weights.cpu().double()
    out = torch.zeros(n, y.shape[1], dtype=torch.float64)
    if old is not None:
        out = out + old.cpu().double()
    mag = out.abs()
    for j in range(k):
        some = ok[:, j]
        term = w[some, j:j + 1] * y[at[some, j]]
        out[some] += term
        mag[some] += term.abs()
    return out, (k + 1) * U * mag


def combine_grad(dout, y, places, weights, dy):
    """(dy with its rounding, dweights in 64 bits, bound of the latter)."""
    want = dispatch(dout, places, weights, dy)
    n, k = places.shape
    ok, at = live(places, y.shape[0])
    d, y = dout.detach().cpu().double(), y.detach().cpu().double()
    dw = torch.zeros(n, k, dtype=torch.float64)
    mag = torch.zeros(n, k, dtype=torch.float64)
    for j in range(k):
        some = ok[:, j]
        term = d[some] * y[at[some, j]]
        dw[some, j] = term.sum(1)
        mag[some, j] = term.abs().sum(1)
    # a lane's own terms (runs of up to 16 columns), six steps in a wave, two more
    return want, dw, (d.shape[1] / 64 + 16 + 1 + 6 + 2) * U * mag
