"""GPU tests of the operators around the decode step: page tables, per-head norm + rotation + cache write with its
gradients, dense one-token attention, and a run of them together with the gated decode."""

import math
import random

import pytest
import torch

import serving_oracle as R

pytestmark = pytest.mark.gpu

BF16, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32


def S():
    import block_sparse_attention_attngate_b200 as pkg
    return pkg


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def rnd(g, *shape, dt=FP32, scale=1.0):
    return (scale * torch.randn(*shape, generator=g, device="cuda")).to(dt)


# ---------------------------------------------------------------- page tables
def pages_problem(seed, B, page, high, new_high, spare, width=None):
    r = random.Random(seed)
    lens = [r.choice([0, 1, page - 1, page, page + 1, r.randint(0, high)]) for _ in range(B)]
    lens = [min(n, high) for n in lens]
    new = [r.choice([0, 1, r.randint(0, new_high)]) for _ in range(B)]
    width = width or -(-(high + new_high) // page) + 1
    held = [-(-n // page) for n in lens]
    pages = sum(held) + sum(-(-(n + m) // page) - h for n, m, h in zip(lens, new, held)) + spare
    ids = list(range(max(pages, 1)))
    r.shuffle(ids)
    table = [[-7] * width for _ in range(B)]
    at = 0
    for b in range(B):
        table[b][:held[b]] = ids[at:at + held[b]]
        at += held[b]
    free = ids[at:] + [-9] * at
    return lens, new, table, free, len(ids) - at, width


PLANS = [(200, 16, 400, 300, 7), (1, 64, 200, 3, 0), (1, 1, 5, 4, 2), (3, 16, 100, 40, 1), (33, 7, 50, 9, 5), (500, 16, 300, 20, 3),
         (1025, 48, 100, 2, 0), (4096, 16, 40, 3, 11), (64, 128, 4000, 400, 9)]


@pytest.mark.parametrize("B,page,high,new_high,spare", PLANS)
@pytest.mark.parametrize("in_place", [False, True])
def test_page_plan(B, page, high, new_high, spare, in_place):
    lens, new, table, free, count, width = pages_problem(B + page, B, page, high, new_high, spare)
    room = sum(new) + (0 if in_place else 37)
    room = max(room, 1)
    ref = R.plan(page, lens, new, table, free, count, room)
    L, T, C = i32(lens), i32(table), i32([count])
    Lo, Co = (None, None) if in_place else (torch.full_like(L, -5), torch.full_like(C, -5))
    cu, slots, pos = torch.full((B + 1,), -3, dtype=torch.int32, device="cuda"), i32([-3] * room), i32([-3] * room)
    err = i32([0])
    S().page_plan(page, L, i32(new), T, i32(free), C, cu, slots, pos, seqlens_out=Lo, free_count_out=Co, err=err)
    assert int(err) == 0
    assert T.tolist() == ref["table"] and cu.tolist() == ref["cu"]
    assert slots.tolist() == ref["slots"] and pos.tolist() == ref["pos"]
    assert (L if in_place else Lo).tolist() == ref["lens"] and int(C if in_place else Co) == ref["count"]
    if not in_place:
        assert L.tolist() == lens and int(C) == count


@pytest.mark.parametrize("B,page,high,new_high,spare", PLANS)
@pytest.mark.parametrize("share", [0.0, 0.3, 1.0])
def test_page_release(B, page, high, new_high, spare, share):
    lens, _, table, free, count, width = pages_problem(7 * B + page, B, page, high, new_high, spare)
    r = random.Random(B)
    done = [r.choice([1, 5, -1]) if r.random() < share else 0 for _ in range(B)]
    ref = R.release(page, lens, done, table, free, count)
    L, F, C, T = i32(lens), i32(free), i32([count]), i32(table)
    err = i32([0])
    S().page_release(page, L, i32(done), T, F, C, err=err)
    assert int(err) == 0
    assert F.tolist() == ref["free"] and L.tolist() == ref["lens"] and int(C) == ref["count"]
    assert T.tolist() == table
    S().page_release(page, L, i32(done), T, F, C, err=err)   # a second time gives nothing back
    assert int(err) == 0 and F.tolist() == ref["free"] and int(C) == ref["count"]


@pytest.mark.parametrize("what", ["negative length", "negative new", "too wide", "room", "free", "count high", "count low"])
def test_page_plan_all_or_nothing(what):
    pkg, page, B = S(), 16, 40
    lens, new, table, free, count, width = pages_problem(3, B, page, 90, 30, 0)
    new[5], lens[7], new[7] = 20, 16, 1
    count = len(free)
    free = list(range(len(free)))
    room = sum(new)
    if what == "negative length":
        lens[11] = -1
    elif what == "negative new":
        new[11] = -2
    elif what == "too wide":
        new[11] = width * page + 1 - lens[11]
        room = 10 ** 4
    elif what == "room":
        room -= 1
    elif what == "free":
        count = 2
    elif what == "count high":
        count = len(free) + 1
    else:
        count = -1
    L, T, C, err = i32(lens), i32(table), i32([count]), i32([0])
    cu, slots, pos = i32([-3] * (B + 1)), i32([-3] * room), i32([-3] * room)
    pkg.page_plan(page, L, i32(new), T, i32(free), C, cu, slots, pos, err=err)
    assert int(err) == pkg.DEVERR_COUNT
    assert L.tolist() == lens and T.tolist() == table and int(C) == count
    assert cu.tolist() == [0] * (B + 1) and slots.tolist() == [-1] * room and pos.tolist() == [0] * room


@pytest.mark.parametrize("what", ["negative length", "too wide", "overflow", "count"])
def test_page_release_all_or_nothing(what):
    pkg, page, B = S(), 16, 40
    lens, _, table, free, count, width = pages_problem(3, B, page, 90, 30, 0)
    done = [1] * B
    if what == "negative length":
        lens[9] = -4
    elif what == "too wide":
        lens[9] = width * page + 1
    elif what == "overflow":
        count = len(free) - sum(-(-n // page) for n in lens) + 1
    else:
        count = -2
    L, F, C, err = i32(lens), i32(free), i32([count]), i32([0])
    pkg.page_release(page, L, i32(done), i32(table), F, C, err=err)
    assert int(err) == pkg.DEVERR_COUNT
    assert L.tolist() == lens and F.tolist() == free and int(C) == count


def test_page_plan_lengths_past_31_bits():
    """A table wide enough for more than 2^31 tokens: a length that would pass them is refused as a whole."""
    pkg, page, T = S(), 1 << 29, i32([[0, 1, 2, 3, 4, 5, 6, 7], [-1] * 8])
    for lens, new, ok in (([2 ** 31 - 6, 0], [5, 3], True), ([2 ** 31 - 6, 0], [6, 3], False)):
        L, C, err, table = i32(lens), i32([1]), i32([0]), T.clone()
        cu, slots, pos = i32([0] * 3), i32([7] * 12), i32([7] * 12)
        pkg.page_plan(page, L, i32(new), table, i32([2, 1, 0]), C, cu, slots, pos, err=err)
        if not ok:
            assert int(err) == pkg.DEVERR_COUNT and L.tolist() == lens and table.tolist() == T.tolist()
            assert slots.tolist() == [-1] * 12
            continue
        # the first row's tokens lie in its page 3, which is outside the pool of 3
        assert int(err) == pkg.DEVERR_PAGE_INDEX and L.tolist() == [2 ** 31 - 1, 3] and table[1, 0] == 2
        assert slots.tolist() == [-1] * 5 + [2 * page, 2 * page + 1, 2 * page + 2] + [-1] * 4


def test_page_ids_outside_the_pool():
    """A bad id from the stack or in the table: reported, its slots -1, every other result as it should be."""
    pkg, page = S(), 4
    table = [[0, -1, -1], [99, -1, -1]]           # row 1's part-filled page is bad
    free, count = [5, -8, 3, 2], 4                # pops 2, 3, then -8
    L, T, C, err = i32([3, 2]), i32(table), i32([count]), i32([0])
    cu, slots, pos = i32([0] * 3), i32([0] * 14), i32([0] * 14)
    pkg.page_plan(page, L, i32([6, 4]), T, i32(free + [0] * 8), C, cu, slots, pos, err=err)
    assert int(err) == pkg.DEVERR_PAGE_INDEX
    assert T.tolist() == [[0, 2, 3], [99, -1, -1]] and int(C) == 1
    assert slots.tolist() == [3, 8, 9, 10, 11, 12, -1, -1, -1, -1] + [-1] * 4
    assert pos.tolist() == [3, 4, 5, 6, 7, 8, 2, 3, 4, 5] + [0] * 4
    F, err = i32([7, 7, 7, 7]), i32([0])
    pkg.page_release(page, i32([8]), i32([1]), i32([[3, 44]]), F, i32([1]), err=err)
    assert int(err) == pkg.DEVERR_PAGE_INDEX and F.tolist() == [7, 3, -1, 7]


def test_pages_conserved_over_many_steps():
    """Plan and release in turn, lengths and count in place: no page is lost or given twice."""
    pkg, page, B, pages, width = S(), 8, 24, 400, 32
    r = random.Random(0)
    L, T, F, C = i32([0] * B), i32([[-1] * width] * B), i32(r.sample(range(pages), pages)), i32([pages])
    cu, slots, pos, err = i32([0] * (B + 1)), i32([0] * 512), i32([0] * 512), i32([0])
    for step in range(60):
        lens = L.tolist()
        S().page_plan(page, L, i32([min(r.randint(0, 9), width * page - n) for n in lens]), T, F, C, cu, slots, pos, err=err)
        pkg.page_release(page, L, i32([int(r.random() < 0.15) for _ in range(B)]), T, F, C, err=err)
        assert int(err) == 0
        held = [p for row, n in zip(T.tolist(), L.tolist()) for p in row[:-(-n // page)]]
        assert sorted(held + F.tolist()[:int(C)]) == list(range(pages))


# ---------------------------------------------------------------- norm + rotation
def rope_problem(seed, T, Hq, Hkv, d, dt, far=131072, packed=True):
    g = gen(seed)
    if packed:
        x = rnd(g, T, Hq + 2 * Hkv, d, dt=dt, scale=2.0)
        q, k, v = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
    else:   # head-major
        q, k, v = (rnd(g, h, T, d, dt=dt, scale=2.0).transpose(0, 1) for h in (Hq, Hkv, Hkv))
    wq, wk = (1 + 0.3 * rnd(g, d)).to(dt), (1 + 0.3 * rnd(g, d)).to(dt)
    pos = torch.randint(0, far, (T,), generator=g, device="cuda", dtype=torch.int32)
    return g, q, k, v, wq, wk, pos


ROPES = [
    # T, Hq, Hkv, d, rope, dtype, norm, packed
    (1, 1, 1, 64, 64, BF16, True, True),
    (1, 32, 8, 128, 128, BF16, True, True),
    (5, 8, 2, 128, 64, FP16, True, True),
    (17, 5, 5, 64, 16, BF16, False, True),
    (33, 7, 1, 128, 48, FP32, True, False),
    (130, 40, 8, 128, 128, FP16, False, False),
    (257, 3, 3, 64, 0, BF16, True, True),
    (1001, 16, 2, 64, 64, FP32, True, True),
    (2050, 32, 8, 128, 128, BF16, True, True),
]


@pytest.mark.parametrize("T,Hq,Hkv,d,rope,dt,norm,packed", ROPES)
def test_norm_rope_forward(T, Hq, Hkv, d, rope, dt, norm, packed):
    g, q, k, v, wq, wk, pos = rope_problem(T + d, T, Hq, Hkv, d, dt, packed=packed)
    if not norm:
        wq = wk = None
    live = max(1, T - 3)
    mark = 7.0
    outs = {n: torch.full((T, h, d), mark, dtype=dt, device="cuda") for n, h in
            (("q_out", Hq), ("k_out", Hkv), ("q_nope", Hq), ("k_nope", Hkv))}
    S().qk_norm_rope(q, k, pos if rope else None, q_weight=wq, k_weight=wk, rope_base=1e6, rope_dim=rope, eps=1e-5,
                     num_tokens=i32([live]), **outs)
    for x, w, o, n in ((q, wq, "q_out", "q_nope"), (k, wk, "k_out", "k_nope")):
        y = R.norm(x, w, 1e-5)
        bound = 2.0 ** -18 * R.pair_size(y, rope)
        R.close(outs[n][:live], y[:live], 2.0 ** -19 * y[:live].abs(), n)
        R.close(outs[o][:live], R.rotate(y, pos, 1e6, rope)[:live], bound[:live], o)
        assert (outs[o][live:] == mark).all() and (outs[n][live:] == mark).all()


@pytest.mark.parametrize("dt", [BF16, FP16, FP32])
def test_norm_rope_in_place_and_alone(dt):
    """Outputs on their inputs' rows, query or key rows alone, no un-rotated output: the same bits."""
    T, Hq, Hkv, d = 77, 6, 2, 128
    g, q, k, v, wq, wk, pos = rope_problem(3, T, Hq, Hkv, d, dt)
    qo, ko = torch.empty(T, Hq, d, dtype=dt, device="cuda"), torch.empty(T, Hkv, d, dtype=dt, device="cuda")
    S().qk_norm_rope(q, k, pos, qo, ko, wq, wk, rope_dim=64)
    q1, k1 = torch.empty_like(qo), torch.empty_like(ko)
    S().qk_norm_rope(q, None, pos, q1, None, wq, rope_dim=64)
    S().qk_norm_rope(None, k, pos, None, k1, None, wk, rope_dim=64)
    assert torch.equal(q1, qo) and torch.equal(k1, ko)
    v0 = v.clone()
    S().qk_norm_rope(q, k, pos, q, k, wq, wk, rope_dim=64)   # views into the packed projection
    assert torch.equal(q, qo) and torch.equal(k, ko) and torch.equal(v, v0)


@pytest.mark.parametrize("dt,page,order", [(BF16, 64, "head"), (FP16, 16, "token"), (BF16, 5, "flat")])
def test_norm_rope_cache_write(dt, page, order):
    pkg, T, Hq, Hkv, d, pages = S(), 101, 8, 2, 64, 40
    g, q, k, v, wq, wk, pos = rope_problem(9, T, Hq, Hkv, d, dt)
    mark = -3.0
    if order == "token":
        kc, vc = (torch.full((pages, page, Hkv, d), mark, dtype=dt, device="cuda").transpose(1, 2) for _ in range(2))
    else:
        kc, vc = (torch.full((pages, Hkv, page, d), mark, dtype=dt, device="cuda") for _ in range(2))
    slots = torch.randperm(pages * page, generator=g, device="cuda")[:T].to(torch.int32)
    slots[4], slots[9], slots[11] = -1, pages * page, -2       # nowhere; two bad ones
    live, err = 97, i32([0])
    ko = torch.empty(T, Hkv, d, dtype=dt, device="cuda")
    pkg.qk_norm_rope(q, k, pos, torch.empty(T, Hq, d, dtype=dt, device="cuda"), ko, wq, wk, v=v, k_cache=kc, v_cache=vc,
                     slot_map=slots, num_tokens=i32([live]), err=err)
    assert int(err) == pkg.DEVERR_PAGE_INDEX
    kr, vr = torch.full_like(kc, mark), torch.full_like(vc, mark)
    for t, s in enumerate(slots.tolist()[:live]):
        if 0 <= s < pages * page:
            kr[s // page, :, s % page], vr[s // page, :, s % page] = ko[t], v[t]
    assert torch.equal(kc, kr) and torch.equal(vc, vr)
    vc2 = torch.full_like(vc, mark)     # keys without values and values without keys
    pkg.qk_norm_rope(None, k, None, k_nope=torch.empty(T, Hkv, d, dtype=dt, device="cuda"), v=v, v_cache=vc2,
                     slot_map=slots, num_tokens=i32([live]), rope_dim=0)
    assert torch.equal(vc2, vr)


def test_norm_rope_extremes():
    """Rows of zeros (the norm's eps), large rows, negative and far positions, a zero live count."""
    T, H, d = 6, 2, 128
    g, q, k, v, wq, wk, _ = rope_problem(5, T, H, H, d, FP32)
    q[0], q[1] = 0, q[1] * 1e15
    pos = i32([0, -1, 2 ** 31 - 1, -2 ** 31, 1 << 20, 131071])
    qo = torch.empty(T, H, d, device="cuda")
    S().qk_norm_rope(q, None, pos, qo, q_weight=wq, rope_base=1e4)
    y = R.norm(q, wq, 1e-6)
    assert (qo[0] == 0).all()
    # positions of 31 bits: the angle's product carries 2^31 2^-53, the reduction the same again
    R.close(qo, R.rotate(y, pos, 1e4, d), (2.0 ** -18 + 2.0 ** -20) * R.pair_size(y, d))
    keep = qo.clone()
    S().qk_norm_rope(q, None, pos, qo, q_weight=wq, num_tokens=i32([0]))
    S().qk_norm_rope(q, None, pos, qo, q_weight=wq, num_tokens=i32([-3]))
    assert torch.equal(qo, keep)
    e = torch.empty(0, H, d, device="cuda")
    S().qk_norm_rope(e, None, i32([]), e, q_weight=wq)


@pytest.mark.parametrize("T,Hq,Hkv,d,rope,dt,norm,packed", ROPES)
@pytest.mark.parametrize("plain", [False, True])
def test_norm_rope_backward(T, Hq, Hkv, d, rope, dt, norm, packed, plain):
    g, q, k, v, wq, wk, pos = rope_problem(T + d, T, Hq, Hkv, d, dt, packed=packed)
    if not norm:
        wq = wk = None
    live, mark = max(1, T - 3), 7.0
    gq, gk = rnd(g, T, Hq, d, dt=dt), rnd(g, T, Hkv, d, dt=dt)
    gqn, gkn = (rnd(g, T, Hq, d, dt=dt), rnd(g, T, Hkv, d, dt=dt)) if plain else (None, None)
    ws = S().alloc_norm_workspace(d)
    ws.fill_(255)
    res = []
    for _ in range(2):
        dq, dk = torch.full_like(gq, mark), torch.full_like(gk, mark)
        dwq, dwk = (torch.full((d,), mark, device="cuda") for _ in range(2)) if norm else (None, None)
        S().qk_norm_rope_backward(gq, gk, q, k, pos, dq, dk, ws if norm else None, wq, wk, dwq, dwk, rope_base=5e5,
                                  rope_dim=rope, eps=1e-5, dq_nope=gqn, dk_nope=gkn, num_tokens=i32([live]))
        res.append((dq, dk, dwq, dwk))
    for a, b in zip(*res):
        assert a is None or torch.equal(a, b)
    for x, w, z, y, dx, dw in ((q, wq, gq, gqn, dq, dwq), (k, wk, gk, gkn, dk, dwk)):
        c = lambda t: None if t is None else t[:live]
        rx, rw, bx, mw = R.norm_grad(c(x), w, 1e-5, c(pos), 5e5, rope, c(z), c(y))
        R.close(dx[:live], rx, bx, "dx")
        assert (dx[live:] == mark).all()
        if norm:
            chain = live * x.shape[1] / 32 + 64
            R.close(dw, rw, (2.0 ** -17 + chain * R.F) * mw, "dw")


def test_norm_rope_backward_against_differences():
    """Directional differences of the 64-bit forward pass."""
    T, H, d, rope = 9, 3, 64, 32
    g, q, k, v, wq, wk, pos = rope_problem(2, T, H, H, d, FP32)
    gz, gy = rnd(g, T, H, d), rnd(g, T, H, d)
    dq, dw = torch.empty(T, H, d, device="cuda"), torch.empty(d, device="cuda")
    S().qk_norm_rope_backward(gz, None, q, None, pos, dq, None, S().alloc_norm_workspace(d), wq, None, dw, None,
                              rope_dim=rope, dq_nope=gy)

    def loss(x, w):
        y = R.norm(x, w, 1e-6)
        return float((R.rotate(y, pos, 1e6, rope) * gz.double() + y * gy.double()).sum())

    h = 1e-5
    for i in range(4):
        vx, vw = rnd(g, T, H, d).double(), rnd(g, d).double()
        diff = (loss(q.double() + h * vx, wq.double() + h * vw) - loss(q.double() - h * vx, wq.double() - h * vw)) / (2 * h)
        got = float((dq.double() * vx).sum() + (dw.double() * vw).sum())
        # fp32 gradients (2^-17 of about 2000 terms of order one, added with random signs but bounded as if not),
        # the differences' own error (h^2 and 1e-16 / h) far below
        size = float((dq.double() * vx).abs().sum() + (dw.double() * vw).abs().sum())
        assert abs(diff - got) <= 2.0 ** -15 * size, (diff, got)


def test_norm_rope_backward_in_place_and_alone():
    T, Hq, Hkv, d = 50, 4, 2, 128
    g, q, k, v, wq, wk, pos = rope_problem(8, T, Hq, Hkv, d, BF16)
    gq, gk = rnd(g, T, Hq, d, dt=BF16), rnd(g, T, Hkv, d, dt=BF16)
    ws = S().alloc_norm_workspace(d)
    new = lambda h: torch.empty(T, h, d, dtype=BF16, device="cuda")
    dq, dk, dwq, dwk = new(Hq), new(Hkv), torch.empty(d, device="cuda"), torch.empty(d, device="cuda")
    S().qk_norm_rope_backward(gq, gk, q, k, pos, dq, dk, ws, wq, wk, dwq, dwk)
    a, b = gq.clone(), gk.clone()
    S().qk_norm_rope_backward(a, b, q, k, pos, a, b, ws, wq, wk, torch.empty_like(dwq), torch.empty_like(dwk))
    assert torch.equal(a, dq) and torch.equal(b, dk)
    only = new(Hkv)
    w2 = torch.empty_like(dwk)
    S().qk_norm_rope_backward(None, gk, None, k, pos, None, only, ws, None, wk, None, w2)
    assert torch.equal(only, dk)
    R.close(w2, dwk.double(), (T * Hkv / 32 + 64) * R.F * 2 * R.norm_grad(k, wk, 1e-6, pos, 1e6, d, gk, None)[3])
    z = torch.empty(0, Hq, d, dtype=BF16, device="cuda")
    dwq.fill_(5)
    S().qk_norm_rope_backward(z, None, z, None, i32([]), z, None, ws, wq, None, dwq, None)
    assert (dwq == 0).all()


# ---------------------------------------------------------------- dense attention
class Rows:
    """A cache of one of three layouts and the rows of a sequence in it."""

    def __init__(self, g, B, H, cap, d, page, dt, order, bad=()):
        self.heads, self.page, self.order = H, page, order
        width = -(-cap // page)
        self.bad = bad
        if order == "flat":
            self.k, self.v = rnd(g, B, H, cap, d, dt=dt), rnd(g, B, H, cap, d, dt=dt)
            self.kc, self.vc = S().KVCache.contiguous(self.k), S().KVCache.contiguous(self.v)
            return
        n = B * width + 3
        shape = (n, H, page, d) if order == "head" else (n, page, H, d)
        self.k, self.v = rnd(g, *shape, dt=dt), rnd(g, *shape, dt=dt)
        if order == "token":
            self.k, self.v = self.k.transpose(1, 2), self.v.transpose(1, 2)
        self.table = torch.randperm(n, generator=g, device="cuda")[:B * width].to(torch.int32).view(B, width)
        for b, i, what in bad:
            self.table[b, i] = what
        self.kc, self.vc = S().KVCache.paged(self.k, self.table), S().KVCache.paged(self.v, self.table)

    def __call__(self, b, h):
        if self.order == "flat":
            return self.k[b, h], self.v[b, h], torch.ones(self.k.shape[2], dtype=torch.bool, device="cuda")
        t = self.table[b].long()
        ok = (t >= 0) & (t < self.k.shape[0])
        t = torch.where(ok, t, 0)
        return (self.k[t, h].flatten(0, 1), self.v[t, h].flatten(0, 1), ok.repeat_interleave(self.page))


def spoil(rows, lens, window):
    """NaN and infinities in every row that must not be used."""
    for b, n in enumerate(lens):
        lo = max(0, n - window) if window else 0
        for x in (rows.k, rows.v):
            if rows.order == "flat":
                x[b, :, max(n, 0):] = math.nan
                x[b, :, :lo] = math.inf
                continue
            t = rows.table[b].long()
            at = torch.cat([torch.arange(0, lo), torch.arange(max(n, 0), len(t) * rows.page)]).cuda()
            page = t[at // rows.page]
            ok = (page >= 0) & (page < x.shape[0])
            for odd, what in ((0, -math.inf), (1, math.nan)):
                pick = ok & (at % 2 == odd)
                x[page[pick], :, (at % rows.page)[pick]] = what


def check_dense(B, g, H, d, lens, cap, page, dt, order, window=0, scale=0.0, bad=(), err_bits=0, seed=0, q_scale=1.0):
    pkg = S()
    gn = gen(seed + 17)
    rows = Rows(gn, B, H, cap, d, page, dt, order, bad)
    spoil(rows, [min(n, cap) for n in lens], window)
    q = rnd(gn, B, g * H, d, dt=dt, scale=q_scale)
    out = torch.full_like(q, math.nan)
    lse, err = torch.full((B, g * H), math.nan, device="cuda"), i32([0])
    ws = pkg.alloc_dense_workspace(B, g * H, H, d)
    ws.fill_(255)
    pkg.dense_decode(q, rows.kc, rows.vc, i32(lens), out, ws, window=window, softmax_scale=scale, lse=lse, err=err)
    assert int(err) == err_bits
    o, l, bo, bl = R.dense(q, rows, [min(max(n, 0), cap) for n in lens], window, scale or d ** -0.5, dt)
    R.close(out, o, bo, "out")
    dead = torch.isinf(l)
    assert (lse[dead] == -math.inf).all() and (out[dead] == 0).all()
    assert ((lse.double() - l).abs()[~dead] <= bl[~dead]).all()
    again, l2 = torch.empty_like(out), torch.empty_like(lse)
    pkg.dense_decode(q, rows.kc, rows.vc, i32(lens), again, ws, window=window, softmax_scale=scale, lse=l2)
    assert torch.equal(out, again) and torch.equal(lse, l2)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dt", [BF16, FP16])
@pytest.mark.parametrize("n", [0, 1, 15, 16, 17, 31, 32, 33, 63, 64, 65, 511, 4097])
def test_dense_lengths(d, dt, n):
    check_dense(1, 4, 1, d, [n], max(n, 1), 64, dt, "flat", seed=n)
    check_dense(2, 3, 2, d, [n, max(0, n - 1)], n + 5, 16, dt, "head", seed=n)


@pytest.mark.parametrize("g", [1, 2, 5, 7, 8, 9, 13, 16])
@pytest.mark.parametrize("order", ["head", "token", "flat"])
def test_dense_groups_and_layouts(g, order):
    check_dense(3, g, 3, 128, [300, 1, 77], 320, 16, BF16, order, seed=g)
    check_dense(3, g, 2, 64, [0, 259, 130], 259, 16, FP16, order, seed=g)


@pytest.mark.parametrize("page", [1, 3, 8, 16, 48, 100, 256])
def test_dense_pages(page):
    check_dense(2, 4, 2, 128, [701, 95], 701, page, BF16, "head", seed=page)
    check_dense(2, 4, 2, 64, [333, 601], 601, page, FP16, "token", seed=page)


@pytest.mark.parametrize("window", [1, 2, 16, 33, 100, 5000])
def test_dense_window(window):
    check_dense(3, 4, 2, 128, [701, 33, 0], 704, 48, BF16, "head", window=window)
    check_dense(2, 9, 1, 64, [16, 1500], 1500, 7, BF16, "token", window=window)


def test_dense_many_rows_and_batches():
    r = random.Random(4)
    lens = [r.choice([0, 1, 5, r.randint(0, 200)]) for _ in range(300)]
    check_dense(300, 2, 8, 64, lens, 200, 16, BF16, "head")             # more rows than warps
    check_dense(64, 4, 1, 128, [0] * 31 + [900] + [0] * 32, 900, 64, BF16, "head")
    check_dense(1, 1, 1300, 64, [70], 70, 64, BF16, "flat")             # more heads than warps
    check_dense(4096, 1, 1, 64, [i % 3 for i in range(4096)], 4, 4, BF16, "head")
    check_dense(5, 2, 2, 64, [0] * 5, 8, 8, BF16, "head")


@pytest.mark.parametrize("g", [1, 5, 8, 9, 16])
@pytest.mark.parametrize("d", [64, 128])
def test_dense_long_rows(g, d):
    """Rows long enough to be split over CTAs whose warps merge."""
    check_dense(3, g, 2, d, [3000, 1, 2111], 3000, 48, BF16, "head", seed=g)
    check_dense(2, g, 1, d, [20001, 0], 20001, 16, FP16, "token", seed=g)
    check_dense(1, g, 3, d, [6007], 6100, 64, BF16, "flat", window=4999, seed=g)


def test_dense_mixed_lengths():
    """Few long rows beside many short ones, in both orders, and rows that leave many pieces."""
    r = random.Random(8)
    short = [r.randint(0, 40) for _ in range(45)]
    check_dense(47, 4, 2, 128, [9000] + short + [7000], 9000, 64, BF16, "head")
    check_dense(47, 4, 2, 64, short + [30000, 1], 30000, 256, BF16, "flat")
    check_dense(90, 2, 4, 64, short * 2, 40, 8, FP16, "token")
    check_dense(12, 8, 1, 128, [5000 + 37 * i for i in range(12)], 6000, 16, BF16, "token")


def test_dense_scales_and_peaks():
    check_dense(2, 4, 2, 128, [700, 300], 700, 64, BF16, "head", scale=0.5)
    check_dense(2, 4, 2, 128, [700, 300], 700, 64, FP16, "head", q_scale=12.0)    # near one-hot weights
    check_dense(2, 4, 2, 128, [700, 300], 700, 64, BF16, "head", q_scale=0.0)     # equal weights


def test_dense_bad_pages_and_lengths():
    pkg = S()
    check_dense(2, 4, 2, 128, [200, 90], 200, 16, BF16, "head", bad=[(0, 3, -1), (1, 0, 10 ** 6)],
                err_bits=pkg.DEVERR_PAGE_INDEX)
    check_dense(1, 4, 2, 64, [40], 48, 16, BF16, "head", bad=[(0, 0, -1), (0, 1, -5), (0, 2, 99)],
                err_bits=pkg.DEVERR_PAGE_INDEX)                       # nothing left: zeros, -inf
    check_dense(1, 4, 2, 64, [40], 48, 16, BF16, "head", bad=[(0, 0, -1)], window=20)   # before the window: not looked at
    check_dense(3, 4, 2, 64, [49, -7, 2 ** 31 - 1], 48, 16, BF16, "head", err_bits=pkg.DEVERR_COUNT)


def test_dense_keys_and_values_of_different_layouts():
    """Keys paged and values contiguous, and the two paged by different tables; the output on the query's memory."""
    pkg, B, g, H, d, page, cap = S(), 3, 4, 2, 128, 24, 900
    gn = gen(21)
    a, b, c = (Rows(gn, B, H, cap, d, page, BF16, o) for o in ("head", "token", "flat"))
    lens = [900, 31, 470]
    for k, v in ((a, c), (c, b), (a, b)):
        q = rnd(gn, B, g * H, d, dt=BF16)
        out, lse = torch.empty_like(q), torch.empty(B, g * H, device="cuda")
        ws = pkg.alloc_dense_workspace(B, g * H, H, d)
        pkg.dense_decode(q, k.kc, v.vc, i32(lens), out, ws, lse=lse)

        def rows(i, h):
            K, V = k(i, h)[0][:cap], v(i, h)[1][:cap]
            return K, V, torch.ones(cap, dtype=torch.bool, device="cuda")

        rows.heads = H
        o, l, bo, bl = R.dense(q, rows, lens, 0, d ** -0.5, BF16)
        R.close(out, o, bo)
        assert ((lse.double() - l).abs() <= bl).all()
        pkg.dense_decode(q, k.kc, v.vc, i32(lens), q, ws)
        assert torch.equal(q, out)


def test_dense_nan_stays_in_its_row():
    """A NaN key or value that is seen shows in its sequence's rows of that head alone."""
    pkg, B, g, H, d = S(), 2, 4, 2, 64
    for T in (60, 2500):
        gn = gen(T)
        rows = Rows(gn, B, H, T, d, 64, BF16, "flat")
        rows.k[0, 1, T // 2] = math.nan
        q = rnd(gn, B, g * H, d, dt=BF16)
        out, lse = torch.empty_like(q), torch.empty(B, g * H, device="cuda")
        pkg.dense_decode(q, rows.kc, rows.vc, i32([T, T]), out, pkg.alloc_dense_workspace(B, g * H, H, d), lse=lse)
        bad = torch.zeros(B, g * H, dtype=torch.bool, device="cuda")
        bad[0, g:] = True
        assert torch.equal(out.isnan().all(-1), bad) and torch.equal(out.isnan().any(-1), bad) and torch.equal(lse.isnan(), bad)


def test_dense_offsets_past_32_bits():
    """A contiguous cache whose second sequence starts beyond 2^32 bytes and 2^31 elements."""
    pkg, d, T = S(), 128, 130
    base = torch.zeros((1 << 31) + (1 << 20), dtype=BF16, device="cuda")
    kv = base.as_strided((2, 1, T, d), ((1 << 31) + 4096, T * d, d, 1))
    gn = gen(1)
    kv.copy_(rnd(gn, 2, 1, T, d, dt=BF16))
    q = rnd(gn, 2, 4, d, dt=BF16)
    out, lse = torch.empty_like(q), torch.empty(2, 4, device="cuda")
    c = pkg.KVCache.contiguous(kv)
    pkg.dense_decode(q, c, c, i32([T, T]), out, pkg.alloc_dense_workspace(2, 4, 1, d), lse=lse)

    def rows(b, h):
        return kv[b, h], kv[b, h], torch.ones(T, dtype=torch.bool, device="cuda")

    rows.heads = 1
    o, l, bo, bl = R.dense(q, rows, [T, T], 0, d ** -0.5, BF16)
    R.close(out, o, bo)
    assert ((lse.double() - l).abs() <= bl).all()


def test_dense_other_stream_and_graph():
    """On a side stream, and captured and replayed with new inputs and lengths; two graphs on one workspace in turn."""
    pkg, B, Hq, H, d, page = S(), 3, 8, 2, 64, 16
    gn = gen(6)
    rows = Rows(gn, B, H, 400, d, page, BF16, "head")
    q, lens = rnd(gn, B, Hq, d, dt=BF16), i32([400, 7, 120])
    ws = pkg.alloc_dense_workspace(B, Hq, H, d)
    out, side = torch.empty_like(q), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    pkg.dense_decode(q, rows.kc, rows.vc, lens, out, ws, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    want = torch.empty_like(q)
    pkg.dense_decode(q, rows.kc, rows.vc, lens, want, ws)
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    outs, graphs = [torch.empty_like(q), torch.empty_like(q)], []
    for i in range(2):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            pkg.dense_decode(q, rows.kc, rows.vc, lens, outs[i], ws, window=50 * i)
        graphs.append(gr)
    q.copy_(rnd(gn, B, Hq, d, dt=BF16))
    lens.copy_(i32([33, 400, 0]))
    for gr in graphs:
        gr.replay()
    torch.cuda.synchronize()
    for i in range(2):
        pkg.dense_decode(q, rows.kc, rows.vc, lens, want, ws, window=50 * i)
        assert torch.equal(outs[i], want)


# ---------------------------------------------------------------- together
def test_serving_steps_together():
    """Requests admitted, prefilled and decoded over a paged cache as a serving loop does it: pages and slots from
    lengths, norm + rotation + cache write, then the new token's attention -- dense, and gated with every block selected --
    against attention over the whole history in 64 bits."""
    pkg, B, Hq, H, d, page, width, dt = S(), 3, 8, 2, 128, 64, 6, BF16
    gn = gen(12)
    pages = B * width
    L, T, F, C = i32([0] * B), i32([[-1] * width] * B), torch.randperm(pages, generator=gn, device="cuda").int(), i32([pages])
    room, err = 320, i32([0])
    cu, slots, pos = i32([0] * (B + 1)), i32([0] * room), i32([0] * room)
    kc, vc = (torch.zeros(pages, H, page, d, dtype=dt, device="cuda") for _ in range(2))
    K, V = pkg.KVCache.paged(kc, T), pkg.KVCache.paged(vc, T)
    wq, wk = (1 + 0.2 * rnd(gn, d)).to(dt), (1 + 0.2 * rnd(gn, d)).to(dt)
    ws = pkg.alloc_dense_workspace(B, Hq, H, d)
    sh = pkg.Shape(B, Hq, H, d, 128, page, width)
    sws = pkg.alloc_workspace(sh, width, 0)
    hist = [[[], []] for _ in range(B)]      # rotated keys and values in 64 bits, rounded to the cache's type

    def forward(new):
        n = sum(new)
        pkg.page_plan(page, L, i32(new), T, F, C, cu, slots, pos, err=err)
        x = torch.zeros(room, Hq + 2 * H, d, dtype=dt, device="cuda")
        x[:n] = rnd(gn, n, Hq + 2 * H, d, dt=dt, scale=1.5)
        q, k, v = x[:, :Hq], x[:, Hq:Hq + H], x[:, Hq + H:]
        qo = torch.zeros(room, Hq, d, dtype=dt, device="cuda")
        pkg.qk_norm_rope(q, k, pos, qo, q_weight=wq, k_weight=wk, v=v, k_cache=kc, v_cache=vc, slot_map=slots,
                         num_tokens=cu[B:], err=err)
        kr = R.rotate(R.norm(k, wk, 1e-6), pos, 1e6, d).to(dt)
        at = 0
        for b, m in enumerate(new):
            hist[b][0].append(kr[at:at + m])
            hist[b][1].append(v[at:at + m])
            at += m
        return qo

    forward([130, 64, 1])
    for step in range(3):
        if step == 2:      # sequence 1 ends; its pages go back and another takes its row
            pkg.page_release(page, L, i32([0, 1, 0]), T, F, C, err=err)
            hist[1] = [[], []]
            forward([0, 70, 0])
        qo = forward([1, 1, 1])[:B].contiguous()
        lens = L.tolist()
        out, lse = torch.empty_like(qo), torch.empty(B, Hq, device="cuda")
        pkg.dense_decode(qo, K, V, L, out, ws, lse=lse, err=err)
        assert int(err) == 0 and lens == [sum(len(x) for x in hist[b][0]) for b in range(B)]

        def rows(b, h):
            k, v = (torch.cat(x)[:, h] for x in hist[b])
            return k, v, torch.ones(len(k), dtype=torch.bool, device="cuda")

        rows.heads = H
        o, l, bo, bl = R.dense(qo, rows, lens, 0, d ** -0.5, dt)
        # the history's keys were rounded from 64 bits, the cache's from fp32: a rounding may fall the other way (one
        # step, 2u, of a key now and then), so a score may move by 2u scale sum |q k| on top
        move = torch.stack([torch.stack([(qo[b, i].double().abs() @ rows(b, i // (Hq // H))[0].double().abs().T).amax()
                                         for i in range(Hq)]) for b in range(B)]) * 2 * R.half_step(dt) * d ** -0.5
        pv = torch.stack([torch.stack([rows(b, i // (Hq // H))[1].double().abs().amax(0) for i in range(Hq)]) for b in range(B)])
        R.close(out, o, bo + 2 * move[..., None] * pv, "out")
        assert ((lse.double() - l).abs() <= bl + move).all()
        nb = [-(-n // page) for n in lens]
        idx = i32([[list(range(n)) + [-1] * (width - n)] * H for n in nb])
        sparse, slse = torch.empty_like(out), torch.empty_like(lse)
        pkg.sparse_decode(sh, qo, K, V, idx, i32([[n] * H for n in nb]), L, sparse, sws, lse=slse)
        R.close(sparse, out.double(), 2 * bo + 2 * R.half_step(dt) * out.double().abs(), "gated, all blocks")
        assert ((slse - lse).abs() <= 2e-3).all()


def test_call_layer_and_named_checks_agree(monkeypatch):
    """Every operator through the compiled call layer, then through the binding's own checks: the same results; and the
    call layer takes the well-formed calls itself."""
    pkg = S()
    from block_sparse_attention_attngate_b200 import seer
    gn = gen(3)
    T, Hq, H, d, page = 9, 4, 2, 64, 16
    x = rnd(gn, T, Hq + 2 * H, d, dt=BF16)
    w, pos = rnd(gn, d, dt=BF16), i32(list(range(T)))
    taken = []

    class Layer:
        def __init__(self, use):
            self.use = use

        def __getattr__(self, name):
            def call(*a):
                if not self.use:
                    return -1
                taken.append(getattr(real, name)(*a))
                return taken[-1]
            return call

    real, results = seer._call, []
    for use in (True, False):
        monkeypatch.setattr(seer, "_call", Layer(use))
        L, T2, F, C = i32([3, 0]), i32([[5, -1], [-1, -1]]), i32([2, 4, 1, 0, 3, -1]), i32([5])
        cu, slots, ps, err = i32([0] * 3), i32([0] * 40), i32([0] * 40), i32([0])
        pkg.page_plan(page, L, i32([20, 5]), T2, F, C, cu, slots, ps, err=err)
        qo, ko = torch.empty(T, Hq, d, dtype=BF16, device="cuda"), torch.empty(T, H, d, dtype=BF16, device="cuda")
        kc, vc = (torch.zeros(6, H, page, d, dtype=BF16, device="cuda") for _ in range(2))
        pkg.qk_norm_rope(x[:, :Hq], x[:, Hq:Hq + H], pos, qo, ko, w, w, rope_dim=32, v=x[:, Hq + H:], k_cache=kc,
                         v_cache=vc, slot_map=slots[:T], num_tokens=i32([T]), err=err)
        dq, dk, gq, gk = torch.empty_like(qo), torch.empty_like(ko), torch.empty(d, device="cuda"), torch.empty(d, device="cuda")
        pkg.qk_norm_rope_backward(qo, ko, x[:, :Hq], x[:, Hq:Hq + H], pos, dq, dk, pkg.alloc_norm_workspace(d), w, w, gq, gk)
        out, lse = torch.empty(2, Hq, d, dtype=BF16, device="cuda"), torch.empty(2, Hq, device="cuda")
        pkg.dense_decode(qo[:2], pkg.KVCache.paged(kc, T2), pkg.KVCache.paged(vc, T2), L, out,
                         pkg.alloc_dense_workspace(2, Hq, H, d), lse=lse, err=err, stream=torch.cuda.current_stream())
        pkg.page_release(page, L, i32([1, 0]), T2, F, C, err=err)
        results.append([L, T2, F, C, cu, slots, ps, err, qo, ko, kc, vc, dq, dk, gq, gk, out, lse])
    assert taken == [0] * 5
    for a, b in zip(*results):
        assert torch.equal(a, b)


def test_refusals_on_the_device():
    """What the call layer does not take is refused by name."""
    pkg, T, H, d = S(), 4, 2, 64
    q = torch.zeros(T, H, d, dtype=BF16, device="cuda")
    pos = i32([0] * T)
    for bad, exc in ((q.transpose(0, 1).transpose(0, 1)[..., ::2], ValueError), (q.half(), TypeError), (q.cpu(), TypeError),
                     (q[:3], ValueError)):
        with pytest.raises(exc):
            pkg.qk_norm_rope(q, None, pos, bad)
    with pytest.raises(TypeError):
        pkg.qk_norm_rope(q, None, pos.long(), torch.empty_like(q))
    with pytest.raises(pkg.SeerError, match="rope_dim"):
        pkg.qk_norm_rope(q, None, pos, torch.empty_like(q), rope_dim=24)
    with pytest.raises(pkg.SeerError, match="share"):
        pkg.qk_norm_rope(q, None, pos, q, q_nope=q)
    kv = pkg.KVCache.contiguous(torch.zeros(T, H, 8, d, dtype=BF16, device="cuda"))
    ws, lens = pkg.alloc_dense_workspace(T, H, H, d), i32([1] * T)
    with pytest.raises(pkg.SeerError, match="workspace"):
        pkg.dense_decode(q, kv, kv, lens, torch.empty_like(q), ws[:64])
    with pytest.raises(pkg.SeerError, match="window"):
        pkg.dense_decode(q, kv, kv, lens, torch.empty_like(q), ws, window=-1)
    with pytest.raises(TypeError):
        pkg.dense_decode(q, kv, kv, lens.float(), torch.empty_like(q), ws)
    with pytest.raises(TypeError):
        pkg.dense_decode(q.half(), kv, kv, lens, q.half(), ws)


def test_norm_rope_offsets_past_32_bits():
    """Rows 2^31 elements apart, read and written."""
    T, d = 2, 64
    gn = gen(4)
    base = torch.zeros((1 << 31) + 4096, dtype=BF16, device="cuda")
    far = base.as_strided((T, 1, d), (1 << 31, d, 1))
    x, w, pos = rnd(gn, T, 1, d, dt=BF16), rnd(gn, d, dt=BF16), i32([3, 70000])
    want, dwant, gw, gw2 = torch.empty_like(x), torch.empty_like(x), torch.empty(d, device="cuda"), torch.empty(d, device="cuda")
    S().qk_norm_rope(x, None, pos, want, q_weight=w)
    far.copy_(x)
    S().qk_norm_rope(far, None, pos, far, q_weight=w)
    assert torch.equal(far, want)
    ws = S().alloc_norm_workspace(d)
    S().qk_norm_rope_backward(want, None, x, None, pos, dwant, None, ws, w, None, gw, None)
    S().qk_norm_rope_backward(far, None, x, None, pos, far, None, ws, w, None, gw2, None)
    assert torch.equal(far, dwant) and torch.equal(gw, gw2)


def test_norm_rope_backward_of_many_rows():
    """More passes than the workspace has rows for at the usual run (every warp then takes more of them)."""
    T, Hq, Hkv, d, rope = 20011, 64, 8, 64, 64
    g, q, k, v, wq, wk, pos = rope_problem(1, T, Hq, Hkv, d, BF16)
    gq, gk = rnd(g, T, Hq, d, dt=BF16), rnd(g, T, Hkv, d, dt=BF16)
    dq, dk, dwq, dwk = torch.empty_like(gq), torch.empty_like(gk), torch.empty(d, device="cuda"), torch.empty(d, device="cuda")
    S().qk_norm_rope_backward(gq, gk, q, k, pos, dq, dk, S().alloc_norm_workspace(d), wq, wk, dwq, dwk)
    for x, w, z, dx, dw in ((q, wq, gq, dq, dwq), (k, wk, gk, dk, dwk)):
        sums, sizes = 0, 0
        for a in range(0, T, 5000):
            c = slice(a, a + 5000)
            rx, rw, bx, mw = R.norm_grad(x[c], w, 1e-6, pos[c], 1e6, rope, z[c], None)
            R.close(dx[c], rx, bx, "dx")
            sums, sizes = sums + rw, sizes + mw
        # a lane adds at most 8 x 11 rows, the CTA's 32 lanes of a channel and the CTAs (at most 4096) follow
        R.close(dw, sums, (2.0 ** -17 + (88 + 32 + 4096 / 128 + 40) * R.F) * sizes, "dw")


def test_serving_step_in_a_graph():
    """A decode step -- pages, norm + rotation + cache write, dense attention -- captured once, replayed with lengths and the
    free count carried on in place, against the same calls made one by one on a side stream."""
    pkg, B, Hq, H, d, page, width, dt = S(), 5, 8, 2, 64, 16, 8, FP16
    gn = gen(31)
    pages, steps, wq, wk = B * width, 6, rnd(gn, d, dt=dt), rnd(gn, d, dt=dt)
    xs = [rnd(gn, B, Hq + 2 * H, d, dt=dt) for _ in range(steps)]
    order, lens0 = torch.randperm(pages, generator=gn, device="cuda").int(), [0, 15, 16, 31, 40]

    class State:
        def __init__(self):
            held = [-(-n // page) for n in lens0]
            ids, at, table = order.tolist(), 0, [[-1] * width for _ in range(B)]
            for b, n in enumerate(held):
                table[b][:n] = ids[at:at + n]
                at += n
            self.L, self.T, self.F, self.C = i32(lens0), i32(table), i32(ids[at:] + [-1] * at), i32([pages - at])
            self.cu, self.slots, self.pos, self.err, self.one = i32([0] * (B + 1)), i32([0] * B), i32([0] * B), i32([0]), i32([1] * B)
            g2 = gen(32)
            self.kc, self.vc = rnd(g2, pages, H, page, d, dt=dt), rnd(g2, pages, H, page, d, dt=dt)
            self.K, self.V = pkg.KVCache.paged(self.kc, self.T), pkg.KVCache.paged(self.vc, self.T)
            self.x, self.q = torch.zeros(B, Hq + 2 * H, d, dtype=dt, device="cuda"), torch.zeros(B, Hq, d, dtype=dt, device="cuda")
            self.out, self.lse = torch.zeros_like(self.q), torch.zeros(B, Hq, device="cuda")
            self.ws = pkg.alloc_dense_workspace(B, Hq, H, d)

        def step(self, stream=None):
            x = self.x
            pkg.page_plan(page, self.L, self.one, self.T, self.F, self.C, self.cu, self.slots, self.pos, err=self.err,
                          stream=stream)
            pkg.qk_norm_rope(x[:, :Hq], x[:, Hq:Hq + H], self.pos, self.q, q_weight=wq, k_weight=wk, v=x[:, Hq + H:],
                             k_cache=self.kc, v_cache=self.vc, slot_map=self.slots, num_tokens=self.cu[B:], err=self.err,
                             stream=stream)
            pkg.dense_decode(self.q, self.K, self.V, self.L, self.out, self.ws, lse=self.lse, err=self.err, stream=stream)

    a, b = State(), State()
    side = torch.cuda.Stream()
    warm = State()
    warm.step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a.step()
    for x in xs:
        a.x.copy_(x)
        b.x.copy_(x)
        graph.replay()
        side.wait_stream(torch.cuda.current_stream())
        b.step(side)
        torch.cuda.current_stream().wait_stream(side)
        for n in ("L", "T", "C", "cu", "slots", "pos", "q", "kc", "vc", "out", "lse"):
            assert torch.equal(getattr(a, n), getattr(b, n)), n
    torch.cuda.synchronize()
    assert int(a.err) == 0 and a.L.tolist() == [n + steps for n in lens0]


def test_two_streams_at_once():
    """Two dense decodes and two gradient passes with workspaces of their own, overlapping on two streams."""
    pkg, B, Hq, H, d, T = S(), 4, 8, 2, 128, 300
    gn = gen(41)
    rows = Rows(gn, B, H, 5000, d, 64, BF16, "head")
    lens = i32([5000, 17, 3333, 1024])
    x, w, pos = rnd(gn, T, Hq, d, dt=BF16), rnd(gn, d, dt=BF16), torch.arange(T, dtype=torch.int32, device="cuda")
    qs, gs = [rnd(gn, B, Hq, d, dt=BF16) for _ in range(2)], [rnd(gn, T, Hq, d, dt=BF16) for _ in range(2)]

    def work(i, stream=None):
        out, dq, dw = torch.empty_like(qs[i]), torch.empty_like(gs[i]), torch.empty(d, device="cuda")
        ws, wn = pkg.alloc_dense_workspace(B, Hq, H, d), pkg.alloc_norm_workspace(d)
        torch.cuda.synchronize()

        def go():
            for _ in range(10):
                pkg.dense_decode(qs[i], rows.kc, rows.vc, lens, out, ws, stream=stream)
                pkg.qk_norm_rope_backward(gs[i], None, x, None, pos, dq, None, wn, w, None, dw, None, stream=stream)
        return go, (out, dq, dw)

    want = []
    for i in range(2):
        go, res = work(i)
        go()
        want.append(res)
    torch.cuda.synchronize()
    runs = [work(i, torch.cuda.Stream()) for i in range(2)]
    for go, _ in runs:
        go()
    torch.cuda.synchronize()
    for (_, got), ref in zip(runs, want):
        for a, b in zip(got, ref):
            assert torch.equal(a, b)
