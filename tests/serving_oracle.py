"""Plain 64-bit forms of the operators around the decode step (page tables, per-head norm with rotation, dense
one-token attention) and the bounds their kernels have to keep, for the GPU tests.

Bounds.  u = eps / 2 is the relative error of one rounding to the tensor's type, f = 2^-24 that of fp32.

* norm + rotation: the sum of squares runs over at most 16 + 3 sequential additions (relative 20 f, halved by the
  square root), rsqrtf is good to 2^-22 and three products follow: y is within 32 f of its value, 2^-19.  An angle
  reduced in 64 bits and rounded to fp32 (|r| <= pi: 2^-23) plus sincosf's own error (2^-23) leaves 2^-22 on cos and sin;
  with the two products and the sum of z = a c - b s: |dz| <= (|a| + |b|) (2^-19 + 2^-22 + 3 f) < 2^-18 (|a| + |b|).  The
  output rounding adds u |z|, or half of the type's smallest step.
* its gradient: the same for dy; dx = r (w dy - x k) adds one more mean (20 f) and four products, so 2^-17 of the
  terms' magnitudes r |w| |dy| + r^3 |x| mean |w dy x|, with |dy| the sum of the rotated pair's magnitudes.  dw adds fp32
  additions: at least 32 rows are summed side by side, so a chain is at most N / 32 long, plus 64 for the joins.
* dense attention: a score is an fp32 sum of d products: |ds| <= (d + 4) f scale sum |q k|, which is the relative error
  of its weight (exp2f and the running rescale add 2^-20); weights are rounded to the cache's type
  (u, or half of its smallest step against a maximum of 1), so |dout| <= (u + max |ds| + 2^-20 + T f) sum p |V| + tiny sum |V| / l
  + u |out|, where T f bounds the additions over T tokens, twice (sum and product): doubled below.
"""

import math

import torch

F = 2.0 ** -24


def half_step(dt):
    return torch.finfo(dt).eps / 2


def tiny(dt):
    """Half of the smallest step near zero."""
    return torch.finfo(dt).tiny * torch.finfo(dt).eps / 2


# ---------------------------------------------------------------- norm + rotation
def rotate(x, pos, base, rope, sign=1):
    h = rope // 2
    if h == 0:
        return x
    theta = float(base) ** (-2.0 * torch.arange(h, dtype=torch.float64, device=x.device) / rope)
    ang = pos.double()[:, None, None] * theta
    c, s = ang.cos(), sign * ang.sin()
    a, b = x[..., :h], x[..., h:rope]
    return torch.cat([a * c - b * s, b * c + a * s, x[..., rope:]], -1)


def pair_size(x, rope):
    """|a| + |b| of each channel's pair."""
    h = rope // 2
    s = x[..., :h].abs() + x[..., h:rope].abs()
    return torch.cat([s, s, x[..., rope:].abs()], -1)


def norm(x, w, eps):
    x = x.double()
    return x if w is None else x / (x.square().mean(-1, keepdim=True) + eps).sqrt() * w.double()


def norm_grad(x, w, eps, pos, base, rope, dz, dy_plain):
    """(dx, dw, bound of dx before rounding, sum of |terms| of dw) in 64 bits."""
    x = x.double()
    zero = torch.zeros_like(x)
    dz = zero if dz is None else dz.double()
    dyp = zero if dy_plain is None else dy_plain.double()
    dy = rotate(dz, pos, base, rope, -1) + dyp
    size = pair_size(dz, rope) + dyp.abs()
    if w is None:
        return dy, None, 2.0 ** -18 * size, None
    w = w.double()
    r = (x.square().mean(-1, keepdim=True) + eps).rsqrt()
    dx = r * (w * dy) - x * r ** 3 * (w * dy * x).mean(-1, keepdim=True)
    mag = r * w.abs() * size + x.abs() * r ** 3 * (w * size * x).abs().mean(-1, keepdim=True)
    return dx, (dy * x * r).sum((0, 1)), 2.0 ** -17 * mag, (size * x.abs() * r).sum((0, 1))


def close(got, ref, bound, what=""):
    """|got - ref| <= bound + one rounding to got's type, everywhere."""
    dt = got.dtype
    tol = bound + half_step(dt) * ref.abs() * (1 + 2.0 ** -8) + tiny(dt)
    err = (got.double() - ref).abs()
    bad = ~(err <= tol)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} off, worst {float((err / tol).max()):.2f} x bound"


# ---------------------------------------------------------------- dense attention
def dense(q, rows, lens, window, scale, dt):
    """rows(b, h) -> (K, V, valid) of the sequence's cache rows; returns out, lse and their bounds."""
    B, Hq, d = q.shape
    out = torch.zeros(B, Hq, d, dtype=torch.float64, device=q.device)
    lse = torch.full((B, Hq), -math.inf, dtype=torch.float64, device=q.device)
    bo, bl = torch.zeros_like(out), torch.zeros_like(lse)
    H = rows.heads
    g = Hq // H
    for b, n in enumerate(lens):
        lo = max(0, n - window) if window else 0
        if n - lo <= 0:
            continue
        for h in range(H):
            K, V, ok = (x[lo:n] for x in rows(b, h))
            K, V = K[ok].double(), V[ok].double()
            if not len(K):
                continue
            T = len(K)
            qq = q[b, h * g:(h + 1) * g].double()
            s = qq @ K.T * scale
            ds = (d + 4) * F * scale * (qq.abs() @ K.abs().T).amax(1, keepdim=True)
            p = torch.softmax(s, 1)
            at = slice(h * g, (h + 1) * g)
            out[b, at] = p @ V
            lse[b, at] = torch.logsumexp(s, 1)
            l = torch.exp(lse[b, at] - s.amax(1))[:, None]
            pv = p @ V.abs()
            bo[b, at] = (half_step(dt) + 2 * (ds + 2.0 ** -20 + T * F)) * pv + tiny(dt) * V.abs().sum(0) / l
            bl[b, at] = ds[:, 0] + 2.0 ** -20 + T * F + 2.0 ** -22 * lse[b, at].abs() + 2.0 ** -22 * s.abs().amax(1)
    return out, lse, bo, bl


# ---------------------------------------------------------------- page tables
def plan(page, lens, new, table, free, count, room):
    """The definition, request by request (lists of whole numbers in, lists out)."""
    table = [list(r) for r in table]
    cu, slots, pos = [0], [], []
    for b, (n, m) in enumerate(zip(lens, new)):
        for i in range(-(-n // page), -(-(n + m) // page)):
            count -= 1
            table[b][i] = free[count]
        for at in range(n, n + m):
            slots.append(table[b][at // page] * page + at % page)
            pos.append(at)
        cu.append(len(slots))
    return dict(table=table, lens=[n + m for n, m in zip(lens, new)], count=count, cu=cu,
                slots=slots + [-1] * (room - len(slots)), pos=pos + [0] * (room - len(pos)))


def release(page, lens, done, table, free, count):
    free, lens = list(free), list(lens)
    for b, n in enumerate(lens):
        if done[b]:
            for i in range(-(-n // page)):
                free[count] = table[b][i]
                count += 1
            lens[b] = 0
    return dict(free=free, lens=lens, count=count)
