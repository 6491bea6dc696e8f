"""Cases for the serving-step operators around the gated decode, with their plain torch forms.

Four operators: the page tables of a paged cache (plan and release), the per-head norm and rotation of queries and keys
with the cache write (forward and backward), and dense attention of one new token over a paged or contiguous cache.
"""

import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZES = {"bf16": 2, "fp16": 2, "fp32": 4}


# ---------------------------------------------------------------------------------------------------- cases
def listed():
    return [
        # one decode step of the 32-sequence loop: one new token each, 64-token pages, the latency-bound call
        dict(name="pages-step-32", op="plan", batch=32, page=64, pages=16384, width=264, low=16000, high=16640, new_low=1,
             new_high=1, room=32),
        # a large mixed batch: running sequences with one token each beside admitted prompts, 16-token pages
        dict(name="pages-mixed-1024", op="plan", batch=1024, page=16, pages=524288, width=1024, low=0, high=8000,
             new_low=0, new_high=127, room=131072),
        # sequences that ended give their pages back: a fifth of a large batch
        dict(name="pages-release-512", op="release", batch=512, page=16, pages=524288, width=1024, low=0, high=16000,
             share=0.2),
        # the same for a small batch of long sequences with block-sized pages
        dict(name="pages-release-16", op="release", batch=16, page=128, pages=8192, width=256, low=8000, high=32000,
             share=0.25),
        # one decode step of the 8-sequence 32k workload: rotated and plain outputs, the new tokens' keys and values
        # scattered into the paged cache
        dict(name="rope-step-8", op="rope", tokens=8, hq=32, hkv=8, d=128, rope=128, dtype="bf16", norm=True, plain=True,
             cache=True, page=64, slots=2048, base=1e6, far=32768, pad=0),
        # a prefill chunk of 8192 tokens of the same layer, written to the cache
        dict(name="rope-prefill-8192", op="rope", tokens=8192, hq=32, hkv=8, d=128, rope=128, dtype="bf16", norm=True,
             plain=True, cache=True, page=64, slots=8192, base=1e6, far=32768, pad=0),
        # odd sizes: 40 query heads, half precision, half of the channels rotated, some padding rows, no cache
        dict(name="rope-odd-2049", op="rope", tokens=2049, hq=40, hkv=8, d=128, rope=64, dtype="fp16", norm=True,
             plain=False, cache=False, page=64, slots=0, base=1e4, far=131072, pad=5),
        # the training direction of a packed 8192-token sequence
        dict(name="rope-grad-8192", op="grad", tokens=8192, hq=32, hkv=8, d=128, rope=128, dtype="bf16", norm=True,
             plain=False, base=1e6, far=8192, pad=0),
        # a short one in 32 bits, with gradients of the un-rotated outputs (the gate's inputs) as well
        dict(name="rope-grad-501", op="grad", tokens=501, hq=8, hkv=2, d=64, rope=64, dtype="fp32", norm=True, plain=True,
             base=1e6, far=65536, pad=0),
        # the tiny decode configuration: one sequence of 2048 tokens, where latency counts
        dict(name="dense-tiny", op="dense", batch=1, hq=4, hkv=1, d=64, low=2048, high=2048, page=64, dtype="bf16",
             order="head", window=0),
        # the ragged 16-sequence workload with five query heads a group, small pages, token-major pool, half precision
        dict(name="dense-ragged-16", op="dense", batch=16, hq=40, hkv=8, d=128, low=8000, high=32000, page=16,
             dtype="fp16", order="token", window=0),
        # the long sweep: four sequences of 65536 tokens
        dict(name="dense-long-4", op="dense", batch=4, hq=32, hkv=8, d=128, low=65000, high=65536, page=64, dtype="bf16",
             order="head", window=0),
    ]


def _between(rng, low, high):
    """A whole number in [low, high], spread over its logarithm where the range is wide."""
    if high <= 10 * max(low, 1):
        return rng.randint(low, high)
    x = math.exp(rng.uniform(math.log(max(low, 1)), math.log(high)))
    return min(high, max(low, int(round(x))))


def draw(rng):
    op = rng.choice(["plan", "release", "rope", "rope", "grad", "dense", "dense", "dense"])
    if op in ("plan", "release"):
        batch, page = _between(rng, 1, 1024), rng.choice([16, 32, 48, 64, 128])
        high = min(16000, 524288 * page // (batch * 2))
        high = max(page, _between(rng, min(64, high), high))
        low = rng.randint(0, high)
        new_high = max(1, min(131072 // batch, _between(rng, 1, 4096)))
        new_low = rng.choice([0, 1, new_high // 2])
        width = (high + new_high + page - 1) // page + rng.randint(0, 8)
        pages = batch * width + rng.randint(1, 64)
        if op == "plan":
            return dict(op=op, batch=batch, page=page, pages=pages, width=width, low=low, high=high,
                        new_low=min(new_low, new_high), new_high=new_high,
                        room=batch * new_high + rng.choice([0, 0, 13, 100]))
        return dict(op=op, batch=batch, page=page, pages=pages, width=width, low=low, high=high,
                    share=rng.choice([0.0, 0.1, 0.5, 1.0]))
    if op in ("rope", "grad"):
        d = rng.choice([64, 128])
        hkv = rng.choice([1, 2, 4, 8])
        hq = hkv * rng.randint(1, 8)
        tokens = _between(rng, 1, min(8192, 8192 * 48 * 128 // ((hq + 2 * hkv) * d)))
        dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
        if dtype == "fp32":
            tokens = max(1, tokens // 2)
        case = dict(op=op, tokens=tokens, hq=hq, hkv=hkv, d=d, rope=rng.choice([d, d, d // 2, 16]), dtype=dtype,
                    norm=rng.random() < 0.8, plain=rng.random() < 0.5, base=rng.choice([1e4, 5e5, 1e6]),
                    far=_between(rng, 1024, 131072), pad=min(tokens - 1, rng.choice([0, 0, 1, 7])))
        if op == "rope":
            page = rng.choice([16, 48, 64, 128])
            cache = dtype != "fp32" and rng.random() < 0.6
            case.update(cache=cache, page=page, slots=(tokens + page - 1) // page * page + page * rng.randint(0, 4))
        return case
    d = rng.choice([64, 128])
    hkv = rng.choice([1, 2, 4, 8])
    group = rng.choice([1, 2, 4, 5, 8, 16])
    batch = _between(rng, 1, 64)
    most = min(65536, 4 * 65536 * 8 * 128 // (batch * hkv * d))
    high = _between(rng, 1, most)
    return dict(op="dense", batch=batch, hq=hkv * group, hkv=hkv, d=d, low=rng.choice([0, high // 2, high]), high=high,
                page=rng.choice([8, 16, 48, 64, 128, 256]), dtype=rng.choice(["bf16", "bf16", "fp16"]),
                order=rng.choice(["head", "token", "flat"]),
                window=rng.choice([0, 0, 0, max(1, high // 3)]))


# ---------------------------------------------------------------------------------------------------- inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _ints(g, low, high, n):
    return torch.randint(low, high + 1, (n,), generator=g, device="cuda", dtype=torch.int32)


def _owned(g, lens, page, pages, width):
    """A block table whose first ceil(len / page) entries of each row are distinct pages of the pool (-1 beyond), and the
    stack of the pages that are left with their count."""
    perm = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    held = (lens.long() + page - 1) // page
    ends = held.cumsum(0)
    col = torch.arange(width, device="cuda")
    at = (ends - held)[:, None] + col[None]
    table = torch.where(col[None] < held[:, None], perm[at.clamp(max=pages - 1)], torch.full_like(perm[:1], -1))
    free = perm.roll(-int(ends[-1]))
    left = torch.tensor([pages - int(ends[-1])], dtype=torch.int32, device="cuda")
    return table.contiguous(), free.contiguous(), left


def prepare(case, seed):
    g = _gen(seed)
    if case["op"] in ("plan", "release"):
        s = _pages_inputs(case, g)
    elif case["op"] in ("rope", "grad"):
        s = _rope_inputs(case, g)
    else:
        s = _dense_inputs(case, g)
    if own:
        import block_sparse_attention_attngate_b200 as S
        s["S"] = S
        if case["op"] == "grad":
            s["work"] = S.alloc_norm_workspace(case["d"])
        if case["op"] == "dense":
            s["k"], s["v"] = ((S.KVCache.contiguous(s["kc"]), S.KVCache.contiguous(s["vc"])) if case["order"] == "flat"
                              else (S.KVCache.paged(s["kc"], s["table"]), S.KVCache.paged(s["vc"], s["table"])))
            s["work"] = S.alloc_dense_workspace(case["batch"], case["hq"], case["hkv"], case["d"])
    s["case"] = case
    return s


def _pages_inputs(case, g):
    b, page = case["batch"], case["page"]
    lens = _ints(g, case["low"], case["high"], b)
    new = _ints(g, case["new_low"], case["new_high"], b) if case["op"] == "plan" else None
    table, free, left = _owned(g, lens, page, case["pages"], case["width"])
    s = dict(lens=lens, table=table, free=free, left=left, lens_out=torch.empty_like(lens), left_out=torch.empty_like(left))
    if case["op"] == "plan":
        i32 = dict(dtype=torch.int32, device="cuda")
        s.update(new=new, cu=torch.empty(b + 1, **i32), slots=torch.empty(case["room"], **i32),
                 pos=torch.empty(case["room"], **i32))
    else:
        s["done"] = (torch.rand(b, generator=g, device="cuda") < case["share"]).to(torch.int32)
    return s


def _rope_inputs(case, g):
    """Rows of one packed projection (queries, keys and values of a token side by side), a few times the size of their
    norm, norm weights around one, positions of several sequences one after another."""
    t, hq, hkv, d, dt = case["tokens"], case["hq"], case["hkv"], case["d"], DTYPES[case["dtype"]]

    def rand(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    packed = (2.0 * rand(t, hq + 2 * hkv, d)).to(dt)
    s = dict(packed=packed, q=packed[:, :hq], k=packed[:, hq:hq + hkv], v=packed[:, hq + hkv:])
    s["wq"], s["wk"] = ((1 + 0.2 * rand(d)).to(dt), (1 + 0.2 * rand(d)).to(dt)) if case["norm"] else (None, None)
    start = _ints(g, 0, max(0, case["far"] - 1), 8)
    run = (t + 7) // 8
    i = torch.arange(t, device="cuda")
    s["pos"] = ((start[i // run].long() + i % run) % case["far"]).to(torch.int32)
    s["live"] = torch.tensor([t - case["pad"]], dtype=torch.int32, device="cuda")

    def empty(h):
        return torch.zeros(t, h, d, dtype=dt, device="cuda")

    if case["op"] == "grad":
        s["gq"], s["gk"] = rand(t, hq, d).to(dt), rand(t, hkv, d).to(dt)
        s["gqn"], s["gkn"] = (rand(t, hq, d).to(dt), rand(t, hkv, d).to(dt)) if case["plain"] else (None, None)
        s["dq"], s["dk"] = empty(hq), empty(hkv)
        s["dwq"], s["dwk"] = ((torch.empty(d, device="cuda"), torch.empty(d, device="cuda")) if case["norm"]
                              else (None, None))
        return s
    s["qo"], s["ko"] = empty(hq), None if case["cache"] else empty(hkv)
    s["qn"], s["kn"] = (empty(hq), empty(hkv)) if case["plain"] else (None, None)
    if case["cache"]:
        pool = (case["slots"] // case["page"], hkv, case["page"], d)
        s["kc"], s["vc"] = torch.zeros(pool, dtype=dt, device="cuda"), torch.zeros(pool, dtype=dt, device="cuda")
        s["slots"] = torch.randperm(case["slots"], generator=g, device="cuda")[:t].to(torch.int32)
    else:
        s["kc"] = s["vc"] = s["slots"] = None
    return s


def _dense_inputs(case, g):
    b, hq, hkv, d, page, dt = case["batch"], case["hq"], case["hkv"], case["d"], case["page"], DTYPES[case["dtype"]]
    lens = _ints(g, case["low"], case["high"], b)
    width = max(1, (case["high"] + page - 1) // page)

    def rand(*shape):
        return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32 if math.prod(shape) < 1 << 20 else dt
                           ).to(dt)

    s = dict(lens=lens, q=rand(b, hq, d))
    if case["order"] == "flat":
        s["kc"], s["vc"], s["table"] = rand(b, hkv, width * page, d), rand(b, hkv, width * page, d), None
    else:
        pages = b * width
        s["table"] = torch.randperm(pages, generator=g, device="cuda").to(torch.int32).view(b, width)
        if case["order"] == "head":
            s["kc"], s["vc"] = rand(pages, hkv, page, d), rand(pages, hkv, page, d)
        else:
            s["kc"], s["vc"] = rand(pages, page, hkv, d).transpose(1, 2), rand(pages, page, hkv, d).transpose(1, 2)
    s["out"] = torch.empty_like(s["q"])
    s["lse"] = torch.empty(b, hq, device="cuda")
    return s


# ---------------------------------------------------------------------------------------------------- passes
def run(s):
    op = s["case"]["op"]
    if own:
        return _own(s)
    return {"plan": _plan, "release": _release, "rope": _rope, "grad": _grad, "dense": _dense}[op](s)


def _own(s):
    S, case = s["S"], s["case"]
    op = case["op"]
    if op == "plan":
        S.page_plan(case["page"], s["lens"], s["new"], s["table"], s["free"], s["left"], s["cu"], s["slots"], s["pos"],
                    seqlens_out=s["lens_out"], free_count_out=s["left_out"])
        return [s["table"], s["lens_out"], s["left_out"], s["cu"], s["slots"], s["pos"]]
    if op == "release":
        S.page_release(case["page"], s["lens"], s["done"], s["table"], s["free"], s["left"], seqlens_out=s["lens_out"],
                       free_count_out=s["left_out"])
        return [s["free"], s["lens_out"], s["left_out"]]
    if op == "rope":
        S.qk_norm_rope(s["q"], s["k"], s["pos"], s["qo"], s["ko"], q_weight=s["wq"], k_weight=s["wk"],
                       rope_base=case["base"], rope_dim=case["rope"], q_nope=s["qn"], k_nope=s["kn"],
                       v=s["v"] if case["cache"] else None, k_cache=s["kc"], v_cache=s["vc"], slot_map=s["slots"],
                       num_tokens=s["live"])
        return [x for x in (s["qo"], s["ko"], s["qn"], s["kn"], s["kc"], s["vc"]) if x is not None]
    if op == "grad":
        S.qk_norm_rope_backward(s["gq"], s["gk"], s["q"], s["k"], s["pos"], s["dq"], s["dk"], s["work"], q_weight=s["wq"],
                                k_weight=s["wk"], dq_weight=s["dwq"], dk_weight=s["dwk"], rope_base=case["base"],
                                rope_dim=case["rope"], dq_nope=s["gqn"], dk_nope=s["gkn"], num_tokens=s["live"])
        return [x for x in (s["dq"], s["dk"], s["dwq"], s["dwk"]) if x is not None]
    S.dense_decode(s["q"], s["k"], s["v"], s["lens"], s["out"], s["work"], window=case["window"], lse=s["lse"])
    return [s["out"], s["lse"]]


def _plan(s):
    page, width = s["case"]["page"], s["case"]["width"]
    lens, new = s["lens"].long(), s["new"].long()
    held, need = (lens + page - 1) // page, (lens + new + page - 1) // page
    more = need - held
    first = more.cumsum(0) - more
    col = torch.arange(width, device="cuda")
    fresh = (col[None] >= held[:, None]) & (col[None] < need[:, None])
    at = (s["left"].long() - 1 - first)[:, None] - (col[None] - held[:, None])
    table = torch.where(fresh, s["free"][at.clamp(0, s["free"].numel() - 1)], s["table"])
    s["table"].copy_(table)
    cu = torch.cat([new.new_zeros(1), new.cumsum(0)])
    t = torch.arange(s["slots"].numel(), device="cuda")
    row = torch.searchsorted(cu[1:], t, right=True)
    live = row < lens.numel()
    row = row.clamp(max=lens.numel() - 1)
    pos = torch.where(live, lens[row] + t - cu[row], 0)
    slot = table[row, (pos // page).clamp(max=width - 1)].long() * page + pos % page
    slots = torch.where(live, slot, -1)
    return [s["table"], (lens + new).int(), (s["left"] - more.sum()).int(), cu.int(), slots.int(), pos.int()]


def _release(s):
    page = s["case"]["page"]
    lens, done = s["lens"].long(), s["done"] != 0
    held = torch.where(done, (lens + page - 1) // page, 0)
    first = held.cumsum(0) - held
    col = torch.arange(s["table"].shape[1], device="cuda")
    back = col[None] < held[:, None]
    at = torch.where(back, s["left"].long() + first[:, None] + col[None], s["free"].numel())
    free = torch.cat([s["free"], s["free"][:1]])
    free.scatter_(0, at.view(-1), s["table"].view(-1))
    s["free"].copy_(free[:-1])
    return [s["free"], torch.where(done, 0, s["lens"]).int(), (s["left"] + held.sum()).int()]


def _angles(s):
    """cos and sin of position * theta for each pair, [tokens, 1, rope / 2], angles in 64 bits."""
    r = s["case"]["rope"]
    theta = float(s["case"]["base"]) ** (-torch.arange(0, r, 2, dtype=torch.float64, device="cuda") / r)
    a = s["pos"].double()[:, None] * theta[None]
    return a.cos().float()[:, None], a.sin().float()[:, None]


def _turn(x, cos, sin):
    h = cos.shape[-1]
    a, b = x[..., :h], x[..., h:2 * h]
    return torch.cat([a * cos - b * sin, b * cos + a * sin, x[..., 2 * h:]], -1)


def _live(s, x):
    """x with the padding rows behind the last token zero (the outputs' rows there stay as they were: zero)."""
    return torch.where((torch.arange(x.shape[0], device="cuda") < s["live"])[:, None, None], x, 0.0)


def _rope(s):
    case, dt = s["case"], s["packed"].dtype
    cos, sin = _angles(s)

    def norm(x, w):
        x = x.float()
        return x if w is None else x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6) * w.float()

    qn, kn = norm(s["q"], s["wq"]), norm(s["k"], s["wk"])
    out = [_live(s, _turn(qn, cos, sin)).to(dt)]
    kr = _turn(kn, cos, sin)
    if not case["cache"]:
        out.append(_live(s, kr).to(dt))
    if case["plain"]:
        out += [_live(s, qn).to(dt), _live(s, kn).to(dt)]
    if case["cache"]:
        t = torch.arange(case["tokens"], device="cuda")
        # padding rows go to a spare slot behind the pool
        to = torch.where(t < s["live"], s["slots"].long(), case["slots"])
        out += [_put(s["kc"], kr.to(dt), to), _put(s["vc"], s["v"], to)]
    return out


def _put(cache, rows, to):
    p, h, page, d = cache.shape
    flat = torch.cat([cache.transpose(1, 2).reshape(p * page, h, d), cache.new_zeros(1, h, d)])
    flat[to] = rows
    cache.copy_(flat[:-1].view(p, page, h, d).transpose(1, 2))
    return cache


def _grad(s):
    dt = s["packed"].dtype
    cos, sin = _angles(s)

    def one(x, w, g, gn):
        x, gy = _live(s, x.float()), _live(s, _turn(g.float(), cos, -sin) + (0 if gn is None else gn.float()))
        if w is None:
            return gy.to(dt), None
        r = torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6)
        wg = gy * w.float()
        dx = r * wg - x * r ** 3 * (wg * x).mean(-1, keepdim=True)
        return dx.to(dt), (gy * x * r).sum((0, 1), dtype=torch.float64).float()

    dq, dwq = one(s["q"], s["wq"], s["gq"], s["gqn"])
    dk, dwk = one(s["k"], s["wk"], s["gk"], s["gkn"])
    return [x for x in (dq, dk, dwq, dwk) if x is not None]


def _dense(s):
    case = s["case"]
    b, hq, hkv, d = case["batch"], case["hq"], case["hkv"], case["d"]
    lens = s["lens"].long()

    def rows(cache):
        if s["table"] is None:
            return cache.float()
        return cache[s["table"].long()].transpose(1, 2).reshape(b, hkv, -1, d).float()

    q = s["q"].float().view(b, hkv, hq // hkv, d)
    score = torch.matmul(q, rows(s["kc"]).transpose(2, 3)) / math.sqrt(d)
    t = torch.arange(score.shape[-1], device="cuda")
    low = (lens - case["window"]).clamp(min=0) if case["window"] else torch.zeros_like(lens)
    seen = ((t[None] < lens[:, None]) & (t[None] >= low[:, None]))[:, None, None]
    score = torch.where(seen, score, -math.inf)
    top = score.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    p = torch.exp(score - top)
    total = p.sum(-1, keepdim=True)
    # rows behind a sequence's end take no part, whatever they hold
    out = torch.matmul(p, rows(s["vc"])) / torch.where(total == 0, 1.0, total)
    return [out.view(b, hq, d).to(s["q"].dtype), (top + torch.log(total)).view(b, hq)]


# ---------------------------------------------------------------------------------------------------- what it cannot do without
def work(case):
    op = case["op"]
    if op == "plan":
        b, mean = case["batch"], (case["new_low"] + case["new_high"]) / 2
        fresh = b * mean / case["page"]
        return {"bytes": 16 * b + 8 * case["room"] + 8 * fresh, "flops": 2 * case["room"]}
    if op == "release":
        held = case["batch"] * case["share"] * (case["low"] + case["high"]) / 2 / case["page"]
        return {"bytes": 12 * case["batch"] + 8 * held, "flops": 2 * case["batch"]}
    if op in ("rope", "grad"):
        n, es = case["tokens"] * case["d"], SIZES[case["dtype"]]
        heads = case["hq"] + case["hkv"]
        if op == "grad":
            moved = n * es * heads * (3 + (1 if case["plain"] else 0))
        else:
            moved = n * es * (heads * (2 + (1 if case["plain"] else 0)) + (2 * case["hkv"] if case["cache"] else 0))
        return {"bytes": moved + 4 * case["tokens"], "flops": n * heads * (16 if op == "grad" else 8)}
    mean = (case["low"] + case["high"]) / 2
    if case["window"]:
        mean = min(mean, case["window"])
    keys = case["batch"] * mean
    return {"bytes": keys * case["hkv"] * case["d"] * 4 + 4 * case["batch"] * case["hq"] * case["d"],
            "flops": 4 * keys * case["hq"] * case["d"]}


# ---------------------------------------------------------------------------------------------------- 64 bits
def exact(case, seed):
    g = _gen(seed)
    if case["op"] == "plan":
        return _exact_plan(case, _pages_inputs(case, g))
    if case["op"] == "release":
        return _exact_release(case, _pages_inputs(case, g))
    if case["op"] == "dense":
        return _exact_dense(case, _dense_inputs(case, g))
    return _exact_rope(case, _rope_inputs(case, g))


def _exact_plan(case, s):
    """The definition, request by request, on the host."""
    page = case["page"]
    lens, new, table = s["lens"].tolist(), s["new"].tolist(), s["table"].tolist()
    free, left = s["free"].tolist(), int(s["left"])
    cu, slots, pos = [0], [], []
    for b, (n, m) in enumerate(zip(lens, new)):
        for i in range((n + page - 1) // page, (n + m + page - 1) // page):
            left -= 1
            table[b][i] = free[left]
        for at in range(n, n + m):
            slots.append(table[b][at // page] * page + at % page)
            pos.append(at)
        cu.append(len(slots))
    slots += [-1] * (case["room"] - len(slots))
    pos += [0] * (case["room"] - len(pos))
    back = [table, [n + m for n, m in zip(lens, new)], [left], cu, slots, pos]
    return [torch.tensor(x, dtype=torch.int32, device="cuda") for x in back]


def _exact_release(case, s):
    page = case["page"]
    lens, done, table = s["lens"].tolist(), s["done"].tolist(), s["table"].tolist()
    free, left = s["free"].tolist(), int(s["left"])
    for b, n in enumerate(lens):
        if done[b]:
            for i in range((n + page - 1) // page):
                free[left] = table[b][i]
                left += 1
            lens[b] = 0
    return [torch.tensor(x, dtype=torch.int32, device="cuda") for x in (free, lens, [left])]


def _exact_rope(case, s):
    """Norm and rotation as products of complex numbers, and the gradients as the products of their Jacobians, in blocks
    of tokens."""
    r, d, n = case["rope"], case["d"], case["tokens"]
    live = n - case["pad"]
    i = torch.arange(r // 2, dtype=torch.float64, device="cuda")
    angle = s["pos"].double()[:, None, None] * torch.exp(-2 * i / r * math.log(case["base"]))
    unit = torch.polar(torch.ones_like(angle), angle)

    def spin(x, u):
        z = torch.complex(x[..., :r // 2].contiguous(), x[..., r // 2:r].contiguous()) * u
        return torch.cat([z.real, z.imag, x[..., r:]], -1)

    def shut(x):
        x[live:] = 0
        return x

    def blocks(f, *xs):
        parts = [f(*[None if x is None else x[a:a + 1024].double() if x.dtype.is_floating_point else x[a:a + 1024]
                     for x in xs]) for a in range(0, n, 1024)]
        return [torch.cat(p) for p in zip(*parts)]

    if case["op"] == "rope":
        def forward(x, u, w):
            y = x if w is None else x / (x.pow(2).sum(-1, keepdim=True) / d + 1e-6).sqrt() * w.double()
            return y, spin(y, u)

        qn, qr = blocks(lambda x, u: forward(x, u, s["wq"]), s["q"], unit)
        kn, kr = blocks(lambda x, u: forward(x, u, s["wk"]), s["k"], unit)
        out = [shut(qr)] + ([] if case["cache"] else [shut(kr)])
        if case["plain"]:
            out += [shut(qn), shut(kn)]
        if case["cache"]:
            to = s["slots"][:live].long()
            for rows in (kr, s["v"].double()):
                cache = torch.zeros(s["kc"].shape, dtype=torch.float64, device="cuda")
                cache[to // case["page"], :, to % case["page"]] = rows[:live]
                out.append(cache)
        return out

    def backward(x, u, g, gn, w):
        y = spin(g, u.conj()) + (0 if gn is None else gn)
        if w is None:
            return y, y
        size = (x.pow(2).sum(-1, keepdim=True) / d + 1e-6).sqrt()
        hat = x / size
        gh = y * w.double()
        return (gh - hat * (gh * hat).sum(-1, keepdim=True) / d) / size, y * hat

    dq, hq = blocks(lambda x, u, g, gn: backward(x, u, g, gn, s["wq"]), s["q"], unit, s["gq"],
                    s["gqn"] if case["plain"] else torch.zeros_like(s["gq"]))
    dk, hk = blocks(lambda x, u, g, gn: backward(x, u, g, gn, s["wk"]), s["k"], unit, s["gk"],
                    s["gkn"] if case["plain"] else torch.zeros_like(s["gk"]))
    out = [shut(dq), shut(dk)]
    if case["norm"]:
        out += [hq[:live].sum((0, 1)), hk[:live].sum((0, 1))]
    return out


def _exact_dense(case, s):
    """Sequence by sequence and head by head over the tokens that are seen."""
    b, hq, hkv, d, page = case["batch"], case["hq"], case["hkv"], case["d"], case["page"]
    group = hq // hkv
    out = torch.zeros(b, hq, d, dtype=torch.float64, device="cuda")
    lse = torch.full((b, hq), -math.inf, dtype=torch.float64, device="cuda")
    for i, n in enumerate(s["lens"].tolist()):
        low = max(0, n - case["window"]) if case["window"] else 0
        t = torch.arange(low, n, device="cuda")
        if not len(t):
            continue
        for h in range(hkv):
            if s["table"] is None:
                k, v = s["kc"][i, h, low:n].double(), s["vc"][i, h, low:n].double()
            else:
                at = s["table"][i].long()[t // page], t % page
                k, v = s["kc"][at[0], h, at[1]].double(), s["vc"][at[0], h, at[1]].double()
            e = k @ s["q"][i, h * group:(h + 1) * group].double().T / d ** 0.5
            lse[i, h * group:(h + 1) * group] = torch.logsumexp(e, 0)
            out[i, h * group:(h + 1) * group] = torch.softmax(e, 0).T @ v
    return [out, lse]
