"""GPU tests of the operators around the decode step at their edges: how many bits the weights of the dense attention
keep, page tables whose results go to other buffers, few long rows among very many."""

import math
import random

import pytest
import torch

import serving_oracle as R
from test_gpu_serving_ops import BF16, FP16, S, gen, i32, rnd

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------- weights of the dense attention
# What a weight loses on its way to V: carried as two numbers of the cache's type, the leading bits cut (2 u of it remain)
# and the rest rounded (u of that), 2 u^2; u = 2^-8 for bf16, 2^-11 for fp16.  fp16's, held as 2^14 times the
# weight, end at steps of 2^-24 (the rest is raised to one such step, or rounded to half of one): 1.5 x 2^-38 < 2^-37.  bf16
# has fp32's exponents; its floor is 1e-36.
FLOOR = {BF16: 1e-36, FP16: 2.0 ** -37}


def tight(q, K, V, scale, dt):
    """softmax(scale q K^T) V of one group in 64 bits, log-sum-exp, and the output's bound but for its own rounding: scores
    (d + 4 additions of fp32), exp2f and rescaling (2^-20), T additions to the sum and to the product, and the above."""
    q, K, V = q.double(), K.double(), V.double()
    T, d = K.shape
    s = q @ K.T * scale
    ds = (d + 4) * R.F * scale * (q.abs() @ K.abs().T).amax(1, keepdim=True)
    p = torch.softmax(s, 1)
    l = torch.exp(torch.logsumexp(s, 1) - s.amax(1))[:, None]
    bound = (2 * R.half_step(dt) ** 2 + 2 * (ds + 2.0 ** -20 + T * R.F)) * (p @ V.abs()) + FLOOR[dt] * V.abs().sum(0) / l
    return p @ V, bound


def run_dense(q, k, v, lens, **kw):
    B, Hq, d = q.shape
    out, lse = torch.empty_like(q), torch.empty(B, Hq, device="cuda")
    ws = S().alloc_dense_workspace(B, Hq, k.shape[1], d)
    S().dense_decode(q, S().KVCache.contiguous(k), S().KVCache.contiguous(v), i32(lens), out, ws, lse=lse, **kw)
    return out, lse


@pytest.mark.parametrize("dt", [BF16, FP16])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("g", [4, 16])
def test_dense_weights_keep_their_bits(dt, d, g):
    """Values of both signs, so that many channels come out far below their terms: there the output's own rounding is small
    and what the weights have lost shows."""
    B, H, cap = 6, 2, 3000
    lens = [2, 7, 16, 40, 333, 3000]
    gn = gen(d + g)
    q, k = rnd(gn, B, g * H, d, dt=dt), rnd(gn, B, H, cap, d, dt=dt)
    v = torch.where(torch.rand(B, H, cap, d, generator=gn, device="cuda") < 0.5, -1.0, 1.0).to(dt)
    out, _ = run_dense(q, k, v, lens)
    for b, n in enumerate(lens):
        for h in range(H):
            at = slice(h * g, (h + 1) * g)
            o, bound = tight(q[b, at], k[b, h, :n], v[b, h, :n], d ** -0.5, dt)
            R.close(out[b, at], o, bound, f"{n} tokens")


@pytest.mark.parametrize("dt", [BF16, FP16])
@pytest.mark.parametrize("low", [12.25, 17.5, 21.0])
def test_dense_many_small_weights(dt, low):
    """Twelve keys stand out by e^low over 1988 equal ones, whose values alone are not zero: one in every twelfth step of 32
    tokens from the front, so that each of a CTA's warps meets one.  296 rows: a whole number of them is a CTA's share."""
    B, H, T, d, top = 2, 148, 2000, 64, 12
    k, v = torch.zeros(B, H, T, d, dtype=dt, device="cuda"), torch.ones(B, H, T, d, dtype=dt, device="cuda")
    k[..., 0] = -low / 3.5
    k[:, :, :32 * top:32], v[:, :, :32 * top:32] = 0, 0
    q = torch.zeros(B, H, d, dtype=dt, device="cuda")
    q[..., 0] = 3.5
    out, lse = run_dense(q, k, v, [T] * B, softmax_scale=1.0)
    o, bound = tight(q[0, :1], k[0, 0], v[0, 0], 1.0, dt)
    R.close(out.view(-1, d), o.expand(B * H, d), bound.expand(B * H, d), "out")
    want = math.log(top + (T - top) * math.exp(-low))
    assert ((lse.double() - want).abs() <= 68 * R.F * low + 2.0 ** -20 + T * R.F + 2.0 ** -22 * low).all()


@pytest.mark.parametrize("dt", [BF16, FP16])
@pytest.mark.parametrize("n", [5, 2500])
def test_dense_infinite_values(dt, n):
    """A value that is seen and infinite shows as what it is in its channel, whatever its weight's bits."""
    g, d = 4, 64
    gn = gen(n)
    q, k, v = rnd(gn, 1, g, d, dt=dt), rnd(gn, 1, 1, n, d, dt=dt), rnd(gn, 1, 1, n, d, dt=dt)
    k[0, 0, n // 2] = 0
    v[0, 0, n // 2, 3], v[0, 0, n // 2, 40] = math.inf, -math.inf
    one = torch.zeros_like(k)        # equal weights: powers of two where n is, and no bits behind the leading ones
    for keys in (k, one):
        out, _ = run_dense(q, keys, v, [n])
        assert (out[..., 3] == math.inf).all() and (out[..., 40] == -math.inf).all()
        rest = [c for c in range(d) if c not in (3, 40)]
        assert out[..., rest].isfinite().all()


# ---------------------------------------------------------------- page tables: lengths and count to other buffers
def release_problem(seed, B, page, high, spare):
    r = random.Random(seed)
    lens = [r.choice([0, 1, page, r.randint(0, high)]) for _ in range(B)]
    held = [-(-n // page) for n in lens]
    width = -(-high // page) + 1
    ids = list(range(sum(held) + spare))
    r.shuffle(ids)
    table, at = [[-7] * width for _ in range(B)], 0
    for b in range(B):
        table[b][:held[b]] = ids[at:at + held[b]]
        at += held[b]
    return lens, table, ids[at:] + [-9] * at, spare


@pytest.mark.parametrize("B,page,high,spare", [(1, 16, 40, 0), (7, 16, 300, 5), (200, 7, 900, 3), (512, 16, 2000, 100),
                                               (513, 1, 60, 1), (4096, 16, 400, 9)])
@pytest.mark.parametrize("own", ["both", "lengths", "count", "neither"])
@pytest.mark.parametrize("share", [0.3, 1.0])
def test_page_release_buffers(B, page, high, spare, own, share):
    """In place, to buffers of its own, and one of each: up to 64 CTAs without a cluster, or a cluster of eight."""
    lens, table, free, count = release_problem(B + page, B, page, high, spare)
    r = random.Random(B)
    done = [r.choice([1, 9, -1]) if r.random() < share else 0 for _ in range(B)]
    ref = R.release(page, lens, done, table, free, count)
    L, F, C, T, err = i32(lens), i32(free), i32([count]), i32(table), i32([0])
    Lo = torch.full_like(L, -5) if own in ("both", "lengths") else None
    Co = torch.full_like(C, -5) if own in ("both", "count") else None
    S().page_release(page, L, i32(done), T, F, C, seqlens_out=Lo, free_count_out=Co, err=err)
    assert int(err) == 0 and F.tolist() == ref["free"] and T.tolist() == table
    assert (L if Lo is None else Lo).tolist() == ref["lens"] and int(C if Co is None else Co) == ref["count"]
    assert (Lo is None or L.tolist() == lens) and (Co is None or int(C) == count)


@pytest.mark.parametrize("what", ["negative length", "too many pages"])
def test_page_release_buffers_all_or_nothing(what):
    pkg, page, B = S(), 16, 400
    lens, table, free, count = release_problem(3, B, page, 2000, 50)
    if what == "negative length":
        lens[9] = -4
    else:
        count = len(free) - sum(-(-n // page) for n in lens) + 1
    L, F, C, Lo, Co, err = i32(lens), i32(free), i32([count]), i32([-5] * B), i32([-5]), i32([0])
    pkg.page_release(page, L, i32([1] * B), i32(table), F, C, seqlens_out=Lo, free_count_out=Co, err=err)
    assert int(err) == pkg.DEVERR_COUNT and F.tolist() == free
    assert Lo.tolist() == lens == L.tolist() and int(Co) == count == int(C)


# ---------------------------------------------------------------- dense attention: many rows, a few of them long
class Packed:
    """A paged cache in which a sequence has as many pages as its length takes (its table is -7 beyond)."""

    def __init__(self, g, lens, H, d, page, dt):
        self.heads, self.page = H, page
        need = [-(-n // page) for n in lens]
        ids, at = torch.randperm(sum(need) + 1, generator=g, device="cuda").tolist(), 0
        table = [[-7] * max(need) for _ in lens]
        for b, n in enumerate(need):
            table[b][:n] = ids[at:at + n]
            at += n
        self.table = i32(table)
        self.k, self.v = rnd(g, at + 1, H, page, d, dt=dt), rnd(g, at + 1, H, page, d, dt=dt)
        for b, n in enumerate(lens):   # behind a sequence's end, in its last page
            if n % page:
                self.k[table[b][n // page], :, n % page:] = math.nan
                self.v[table[b][n // page], :, n % page:] = math.inf
        self.kc, self.vc = S().KVCache.paged(self.k, self.table), S().KVCache.paged(self.v, self.table)
        self.need = need

    def __call__(self, b, h):
        t = self.table[b, :self.need[b]].long()
        k, v = self.k[t, h].flatten(0, 1), self.v[t, h].flatten(0, 1)
        return k, v, torch.ones(len(k), dtype=torch.bool, device="cuda")


@pytest.mark.parametrize("B,H,g,d,dt", [(128, 8, 4, 128, BF16), (230, 8, 2, 64, FP16), (256, 8, 9, 64, BF16), (2100, 1, 4, 128, FP16)])
@pytest.mark.parametrize("window", [0, 9000])
def test_dense_long_rows_among_many(B, H, g, d, dt, window):
    """Rows enough for teams of single warps whatever the lengths (six an SM; by row, or, above twelve an SM, by range): a long
    row then lies in hundreds of ranges and is joined piece after piece."""
    r = random.Random(B)
    lens = [r.randint(0, 40) for _ in range(B)]
    lens[0], lens[B // 2], lens[-1] = 20003, 5000, 20480
    gn = gen(B + g)
    rows = Packed(gn, lens, H, d, 16, dt)
    q = rnd(gn, B, g * H, d, dt=dt)
    out, lse, err = torch.full_like(q, math.nan), torch.full((B, g * H), math.nan, device="cuda"), i32([0])
    ws = S().alloc_dense_workspace(B, g * H, H, d)
    ws.fill_(255)
    S().dense_decode(q, rows.kc, rows.vc, i32(lens), out, ws, window=window, lse=lse, err=err)
    assert int(err) == 0
    o, l, bo, bl = R.dense(q, rows, lens, window, d ** -0.5, dt)
    R.close(out, o, bo, "out")
    dead = torch.isinf(l)
    assert (lse[dead] == -math.inf).all() and (out[dead] == 0).all()
    assert ((lse.double() - l).abs()[~dead] <= bl[~dead]).all()
