"""Plain 64-bit forms of the token operators, on the host, with bounds on how
far fp32 kernels may be from them.

u = 2^-24 is the largest relative rounding error of an fp32 operation.  The
bounds below count roundings of the operators' definitions, not of a
particular kernel:

* d = x - m: one rounding, u |d|.
* e = exp(d), computed as 2^(d log2 e): the constant and the product are off by
  2 u |d log2 e| in the exponent, i.e. 2 u |d| relative in e, the subtraction by
  u |d|, the exponential itself by at most 1 ulp = 2 u: (3 |d| + 2) u.
* a sum of V terms in any order: at most (V - 1) u times the sum of |terms|;
  the kernels add in trees, so ``depth`` (an upper bound on the additions any
  one term takes part in) replaces V - 1.
* log S: the relative error of S, plus 2 ulp = 4 u of |log S| (and of 1 near
  S = 1, where the logarithm itself vanishes).
"""

import math

import torch

U = 2.0 ** -24


def half_step(dtype):
    return {torch.float32: U, torch.bfloat16: 2.0 ** -8}[dtype]


def depth(v):
    """Additions a term of a row of ``v`` values takes part in: at most a thread's
    own elements (64 threads at least, 16 elements over per thread for vector
    and edge granularity), six steps in its wave and sixteen waves."""
    return v / 64 + 16 + 6 + 16


class Softmax:
    """log-softmax of the rows of ``x`` (times ``inv_tau``) in 64 bits; ``tol`` bounds
    an fp32 log q, ``tol_s`` the relative error of an fp32 sum of exponentials."""

    def __init__(self, x, inv_tau=1.0):
        x = x.detach().cpu().double()
        self.m = x.max(1, keepdim=True).values
        d = (x - self.m) * inv_tau
        self.d = d
        e = torch.exp(d)
        s = e.sum(1, keepdim=True)
        self.logs = torch.log(s)
        self.lq = d - self.logs
        self.q = e / s
        ad = torch.where(e > 0, d.abs(), torch.zeros_like(d))
        # one more rounding of d for the product with 1 / T (and of 1 / T itself)
        self.tol_s = U * ((self.q * (5 * ad + 2)).sum(1, keepdim=True) + depth(x.shape[1]))
        self.tol_lse = self.tol_s + 4 * U * (self.logs.abs() + 1)
        self.tol = self.tol_lse + U * (3 * ad + 2 * self.lq.abs().clamp(max=1e30))
        self.ad = ad

    def entropy(self):
        """(H, bound): H = log S - A / S with A = sum e d."""
        t = torch.where(self.q > 0, self.q * self.lq, torch.zeros_like(self.q))
        h = -t.sum(1)
        qd = self.q * self.ad
        a = qd.sum(1, keepdim=True)
        tol = ((qd * U * (5 * self.ad + 3)).sum(1, keepdim=True) + a * depth(self.q.shape[1]) * U
               + a * (self.tol_s + 2 * U) + self.tol_lse + U * h.abs()[:, None])
        return h, tol[:, 0]

    def tol_q(self):
        """Bound of an fp32 q = exp(log q): relative error of the exponent's
        argument, its two roundings and the exponential's ulp."""
        alq = torch.where(self.q > 0, self.lq.abs(), torch.zeros_like(self.lq))
        return self.q * (self.tol_lse + U * (5 * self.ad + 4 * alq + 4)) + 2.0 ** -126


def logprob_grad(x, targets, glp, gent):
    """(dx, bound) of glp log q_t + gent H."""
    sm = Softmax(x)
    n, v = sm.q.shape
    t = targets.cpu().long()
    ok = (t >= 0) & (t < v)
    glp = torch.zeros(n, dtype=torch.float64) if glp is None else glp.cpu().double()
    glp = torch.where(ok, glp, torch.zeros_like(glp))[:, None]
    gent = (torch.zeros(n, dtype=torch.float64) if gent is None else gent.cpu().double())[:, None]
    h, tol_h = sm.entropy()
    h, tol_h = h[:, None], tol_h[:, None]
    lq = torch.where(sm.q > 0, sm.lq, torch.zeros_like(sm.lq))
    inner = glp + gent * (lq + h)
    dx = -sm.q * inner
    hot = torch.zeros_like(dx)
    hot[torch.arange(n)[ok], t[ok]] = 1.0
    dx = dx + glp * hot
    tol_lq = torch.where(sm.q > 0, sm.tol, torch.zeros_like(sm.q))
    tol_inner = (gent.abs() * (tol_lq + tol_h) +
                 4 * U * (glp.abs() + gent.abs() * (lq.abs() + h.abs())))
    tol = (sm.tol_q() * inner.abs() + sm.q * tol_inner + 2 * U * (sm.q * inner.abs())
           + 2 * U * glp.abs() * hot)
    return dx, tol


class Distill:
    """Loss and gradient, with bounds, of distillation from listed teacher logits."""

    def __init__(self, x, ids, teacher, tau, weights=None, grad_scale=1.0):
        inv_tau = 1.0 / tau
        sm = Softmax(x, inv_tau)
        n, v = sm.q.shape
        k = ids.shape[1]
        ids = ids.cpu().long()
        z = teacher.detach().cpu().double() * inv_tau
        ok = (ids >= 0) & (ids < v)
        z = torch.where(ok, z, torch.full_like(z, -math.inf))
        zm = z.max(1, keepdim=True).values
        listed = torch.isfinite(zm)
        z = torch.where(listed, z - zm, torch.full_like(z, -math.inf))
        e = torch.exp(z)
        s = e.sum(1, keepdim=True).clamp(min=1e-300)
        logs = torch.log(s)
        p, lp = e / s, z - logs
        az = torch.where(p > 0, z.abs(), torch.zeros_like(z))
        tol_s = U * ((p * (5 * az + 2)).sum(1, keepdim=True) + k)
        tol_lp = tol_s + 4 * U * (logs.abs() + 1) + U * (5 * az + 2 * logs.abs())
        tol_p = p * (tol_s + U * (5 * az + 5))
        w = torch.ones(n, dtype=torch.float64) if weights is None else weights.cpu().double()
        live = (listed[:, 0] & (w != 0))
        at = ids.clamp(0, v - 1)
        lq, tol_lq = sm.lq.gather(1, at), sm.tol.gather(1, at)
        use = p > 0
        zero = torch.zeros_like(p)
        term = torch.where(use, p * (lp - lq), zero)
        t_tol = torch.where(use, tol_p * (lp - lq).abs() + p * (tol_lp + tol_lq), zero)
        scale = w * tau * tau
        self.loss = torch.where(live, scale * term.sum(1), torch.zeros_like(w))
        # a share of the weight's and temperature's products, and of the k additions
        self.loss_tol = torch.where(live, scale.abs() * (
            t_tol.sum(1) + U * (k + 8) * torch.where(use, p * (lp.abs() + lq.abs()),
                                                     zero).sum(1)), torch.zeros_like(w))
        c = (w * grad_scale * tau)[:, None]
        tp = torch.zeros_like(sm.q).scatter_add(1, at, torch.where(ok, p, zero))
        tt = torch.zeros_like(sm.q).scatter_add(1, at, torch.where(ok, tol_p + k * U * p, zero))
        dead = ~live[:, None]
        self.dx = (c * (sm.q - tp)).masked_fill(dead, 0.0)
        self.dx_tol = (c.abs() * (sm.tol_q() + tt + 4 * U * (sm.q + tp))).masked_fill(dead, 0.0)


def embed_grad(dout, ids, vocab, scale, old=None):
    """(dtable, bound): sums in any order, at most one rounding per addition."""
    x = dout.detach().cpu().double()
    ids = ids.cpu().long()
    ok = (ids >= 0) & (ids < vocab)
    out = torch.zeros(vocab, x.shape[1], dtype=torch.float64)
    mag, cnt = torch.zeros_like(out), torch.zeros(vocab, dtype=torch.float64)
    out.index_add_(0, ids[ok], x[ok])
    mag.index_add_(0, ids[ok], x[ok].abs())
    cnt.index_add_(0, ids[ok], torch.ones(int(ok.sum()), dtype=torch.float64))
    out, mag = out * scale, mag * abs(scale)
    if old is not None:
        out, mag = out + old.cpu().double(), mag + old.cpu().double().abs()
    return out, (cnt[:, None] + 3) * U * mag


def assert_close(got, want, tol, what, dtype=None):
    """|got - want| <= tol plus the rounding to ``dtype`` of a value up to tol off;
    non-finite values agree in kind.  A wanted value beyond the largest fp32 number,
    (2 - 2^-23) 2^127, by more than half a step, i.e. from (2 - 2^-24) 2^127 on, is an
    infinity in fp32: -3e38 less 3e38 cannot be anything else."""
    want = torch.where(want.abs() >= (2 - U) * 2.0 ** 127, torch.sign(want) * math.inf, want)
    got = got.detach().cpu()
    dtype = dtype or got.dtype
    got = got.double()
    tiny = 2.0 ** -149 if dtype == torch.float32 else 2.0 ** -133
    lim = tol + half_step(dtype) * (want.abs() + tol) * (1 + U) + tiny
    fin = torch.isfinite(want)
    assert torch.equal(torch.isnan(got), torch.isnan(want)), f"{what}: NaNs differ"
    assert torch.equal(got[~fin & ~torch.isnan(want)], want[~fin & ~torch.isnan(want)]), what
    off = (got - want).abs()[fin]
    bad = off > lim[fin]
    if bad.any():
        i = int(torch.argmax(off - lim[fin]))
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} off; worst "
                             f"{got[fin][i].item()!r} for {want[fin][i].item()!r}, allowed "
                             f"{lim[fin][i].item():.3g}")
