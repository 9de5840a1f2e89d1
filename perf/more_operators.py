"""Operators of a serving step around the 8-bit key/value cache, as measured cases: page tables
and slot maps built from request lengths (KV8Pages.step), norms of the query and key heads with
the rotary positions in the same pass (NormRope), attention with a sliding window and first
positions that stay visible (KV8Cache.attention, `window` and `sinks`), and attention for
sequences that share a long prefix, computed once for all of them (`prefix`).

`run` computes a case either in its plain form (elementary torch operations, in 32 bits) or,
with `own` set, by the calls that a user of the library makes (bit_expert_layer_gb300.kv8).

The cache is the one of perf/operators.py: pages of `page` positions, one byte per number, and
for every 16 positions of a head one power-of-two scale; value = code * scale.
"""
import math

import numpy as np
import torch

own = False

BLOCK = 16
TOP = {"e4m3": 448.0, "int8": 127.0}
THETA, EPS = 1e7, 1e-6


# ----------------------------------------------------------------------------- the cases
def listed():
    gqa = dict(hq=16, hkv=2, d=128, page=64)     # the model's full-attention layers
    norm = dict(op="norm_rope", hq=16, hkv=2, d=128)
    return [
        # one user, one new token: the window's few pages, the first ones (latency)
        dict(name="window-1", op="window", b=1, lo=5003, hi=5003, new=1, window=1024, sinks=4, fmt="e4m3", **gqa),
        # a step of a busy server, 64 conversations of very different lengths, int8 cache
        dict(name="window-64-mixed-int8", op="window", b=64, lo=64, hi=16384, new=1, window=4096, sinks=4, fmt="int8", **gqa),
        # one 2048-token piece of a long document, 14 thousand positions before it
        dict(name="window-piece-16k", op="window", b=1, lo=16301, hi=16301, new=2048, window=1024, sinks=16, fmt="e4m3", **gqa),
        # 8 short answers under one system prompt
        dict(name="prefix-8-5k", op="prefix", b=8, groups=1, shared=5003, lo=20, hi=900, new=1, fmt="e4m3", **gqa),
        # 24 sequences of two assistants, each with 4 drafted tokens, int8 cache
        dict(name="prefix-24-drafts-int8", op="prefix", b=24, groups=2, shared=12001, lo=40, hi=500, new=4, fmt="int8", **gqa),
        # 128 questions about the same long document
        dict(name="prefix-128-32k", op="prefix", b=128, groups=1, shared=32768, lo=64, hi=2000, new=1, fmt="e4m3", **gqa),
        # queries and keys of a decode step, three axes, a quarter of the head rotated
        dict(name="norm-rope-64", t=64, rot=32, axes=3, cyclic=True, far=200000, offset=1.0, **norm),
        # queries and keys of a prompt with images, the whole head rotated
        dict(name="norm-rope-16k-images", t=16384, rot=128, axes=3, cyclic=False, far=20000, offset=0.0, **norm),
        # a decode step of 64 sequences: some need a page, one in nine is done and gives its pages back
        dict(name="pages-64", op="pages", b=64, lo=64, hi=16384, new=1, drop=0, done=9, spare=40, page=64),
        # 200 prompts of odd lengths admitted at once, 184 thousand tokens
        dict(name="pages-200-prompts", op="pages", b=200, lo=0, hi=0, new=1500, drop=0, done=0, spare=500, page=64),
    ]


def _between(rng, lo, hi):
    """A whole number of [lo, hi], spread evenly over the logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["window", "window", "window", "prefix", "prefix", "prefix", "norm_rope", "pages"])
    # the model's own head layout and others: 1 to 16 query heads to a key/value head
    hq, hkv, d = rng.choice([(16, 2, 128), (16, 2, 128), (32, 4, 128), (10, 2, 128), (7, 7, 64), (32, 2, 64), (8, 1, 128)])
    fmt, page = rng.choice(["e4m3", "int8"]), rng.choice([16, 32, 64, 128])
    if op == "norm_rope":
        return dict(op=op, t=_between(rng, 1, 16384 * 18 * 128 // max(18 * 128, (hq + hkv) * d)), hq=hq, hkv=hkv, d=d, rot=rng.choice([d // 4, d // 2, d]),
                    axes=rng.choice([1, 3, 3]), cyclic=rng.random() < 0.5, far=_between(rng, 100, 1000000),
                    offset=rng.choice([0.0, 1.0]))
    if op == "pages":
        b = _between(rng, 1, 512)
        new = _between(rng, 1, min(4096, 262144 // b))
        hi = rng.choice([0, _between(rng, 10, 20000)])
        return dict(op=op, b=b, lo=hi // rng.choice([1, 3, 50]), hi=hi, new=new, drop=rng.choice([0, 0, 3, 40]),
                    done=rng.choice([0, 2, 9]), spare=_between(rng, 3, 2000), page=page)
    gqa = dict(hq=hq, hkv=hkv, d=d, page=page, fmt=fmt)
    if op == "window":
        window, sinks = _between(rng, 16, 4096), rng.choice([0, 1, 4, 4, 33, 130])
        if rng.random() < 0.35:                              # a prompt, whole or a piece of one
            b, new = rng.choice([1, 1, 2, 3]), _between(rng, 40, 2048)
            lo = new + _between(rng, 1, 12000) - 1
            b = max(1, min(b, 2048 // new))
            return dict(op=op, b=b, lo=lo, hi=lo + rng.randrange(0, 200), new=new, window=window, sinks=sinks, **gqa)
        b, new = _between(rng, 1, 64), rng.choice([1, 1, 1, 2, 3, 5, 8])
        hi = _between(rng, 20, min(32768, 262144 // b))
        return dict(op=op, b=b, lo=max(new, hi // rng.choice([1, 2, 50])), hi=hi, new=new, window=window, sinks=sinks, **gqa)
    b, new = _between(rng, 2, 128), rng.choice([1, 1, 1, 2, 3, 5, 20])
    b = max(2, min(b, 512 // new))
    # as many positions as keep the scores under those of the largest listed case
    shared = _between(rng, 100, min(32768, 4000000 // b, 90 * 32768 * 16 * 128 // (b * new * hq * d)))
    hi = new + _between(rng, 1, 2000)
    return dict(op=op, b=b, groups=min(b, rng.choice([1, 1, 2, 5])), shared=shared, lo=max(new, hi // rng.choice([1, 3, 30])),
                hi=hi, new=new, **gqa)


def _spread(b, lo, hi):
    """b lengths from `hi` down to `lo`, evenly spread over the logarithm."""
    if b == 1 or lo == hi:
        return [hi] * b
    return [int(round(hi * (max(lo, 1) / hi) ** (i / (b - 1)))) for i in range(b)]


def _new(case):
    """New tokens per sequence: `new`, a little fewer in every second sequence where there are several tokens."""
    return [max(1, case["new"] - (i % 2) * (case["new"] // 7)) for i in range(case["b"])]


def _groups(case):
    """The first sequence of each group, the end, and the positions that each group shares (whole pages)."""
    n = case["groups"]
    first = [i * case["b"] // n for i in range(n + 1)]
    return first, [case["shared"] // (i + 1) // case["page"] * case["page"] for i in range(n)]


def _lens(case):
    """The sequences' lengths, the new tokens (and what they share) among them."""
    lens = _spread(case["b"], case["lo"], case["hi"])
    if case["op"] == "prefix":
        first, shared = _groups(case)
        for g, s in enumerate(shared):
            for i in range(first[g], first[g + 1]):
                lens[i] += s
    return lens


def _requests(case):
    """Of a pages case, per sequence: cached positions, positions that stay, new tokens."""
    b, new = case["b"], case["new"]
    cached = _spread(b, case["lo"], case["hi"])
    done = [case["done"] > 0 and i % case["done"] == case["done"] - 1 for i in range(b)]
    keep = [0 if f else max(0, n - case["drop"] * (i % 3)) for i, (n, f) in enumerate(zip(cached, done))]
    fresh = [0 if f else max(1, new - (i * 37 % 100) * new // 128) for i, f in enumerate(done)]
    return cached, keep, fresh


# ----------------------------------------------------------------------------- inputs
def _quantise(x, fmt):
    """Blocks x (float32 [..., 16, d]) -> codes (uint8), scales (float32 [...])."""
    mant, ex = torch.frexp(x.abs().amax(dim=(-2, -1)) / TOP[fmt])
    ex = torch.where(mant == 0.5, ex - 1, ex).clamp_min(-100)
    scale = torch.ldexp(torch.ones_like(mant), ex)
    y = x / scale[..., None, None]
    codes = y.to(torch.float8_e4m3fn) if fmt == "e4m3" else y.round().to(torch.int8)
    return codes.view(torch.uint8), scale


def _values(codes, scales, fmt):
    """Codes [..., page, d] and scales [..., page / 16] -> float32 values."""
    c = codes.view(torch.float8_e4m3fn if fmt == "e4m3" else torch.int8).to(torch.float32)
    return c * scales.repeat_interleave(BLOCK, dim=-1)[..., None]


def _ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    state = dict(case=case)
    fill = {"norm_rope": _prepare_norm_rope, "pages": _prepare_pages}.get(case["op"], _prepare_attention)
    fill(case, state, g)
    return state


def _prepare_norm_rope(case, state, g):
    t, axes, far, hq, hkv, d = (case[n] for n in ("t", "axes", "far", "hq", "hkv", "d"))
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    state["qkv"] = (rnd(t, hq + 2 * hkv, d) * torch.exp(rnd(t, 1, 1))).to(torch.bfloat16)   # the fused projection's output
    for name in ("q_weight", "k_weight"):
        state[name] = (rnd(d) * 0.2 + 1.0 - case["offset"]).to(torch.bfloat16)
    # text runs along all axes; images hold time still and move height and width
    start = torch.randint(0, far, (1,), generator=g, device="cuda")
    i = torch.arange(t, device="cuda")
    image = (i // 256) % 2 == 1
    rows = [torch.where(image, i // 256 * 256, i), torch.where(image, i // 256 * 256 + i % 256 // 16, i),
            torch.where(image, i // 256 * 256 + i % 16, i)]
    state["pos"] = (torch.stack(rows[:axes]) + start).to(torch.int32)
    pairs = case["rot"] // 2
    sections = [pairs - (axes - 1) * (pairs // axes)] + [pairs // axes] * (axes - 1)
    # the axis of each rotated pair: runs of `sections` pairs, or the axes in turn while each has pairs left
    runs = [a for a, n in enumerate(sections) for _ in range(n)]
    if case["cyclic"]:
        runs = [a for _, a in sorted((runs[:j].count(a), a) for j, a in enumerate(runs))]
    state["axis_of"] = runs
    state["inv_freq"] = torch.tensor(THETA ** (-np.arange(pairs, dtype=np.float64) * 2 / case["rot"]), device="cuda")
    state["axis_index"] = torch.tensor(runs, device="cuda")
    if own:
        from bit_expert_layer_gb300 import kv8
        rope = kv8.Rope(head_size=d, rotary=case["rot"], theta=THETA, sections=sections, cyclic=case["cyclic"])
        state["norm_rope"] = kv8.NormRope(rope, state["q_weight"], state["k_weight"], eps=EPS, offset=case["offset"])


def _prepare_pages(case, state, g):
    b, page = case["b"], case["page"]
    cached, keep, new = _requests(case)
    held = [-(-n // page) for n in cached]
    after = [-(-(k + n) // page) for k, n in zip(keep, new)]
    need = sum(max(0, a - h) for a, h in zip(after, held))
    n_pages = sum(held) + need + case["spare"]
    width = max(1, max(held + after)) + 2
    order = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32).cpu().numpy()
    table, at = np.zeros((b, width), np.int32), 0
    for i, n in enumerate(held):
        table[i, :n] = order[at:at + n]
        at += n
    free = np.zeros(n_pages, np.int32)
    free[:n_pages - at] = order[at:]
    state.update(table=_ints(table), held=_ints(held), cached=_ints(cached), keep=_ints(keep), new=_ints(new), free=_ints(free),
                 n_free=_ints([n_pages - at]), t=sum(new))
    if own:
        from bit_expert_layer_gb300 import kv8
        state["pages"] = kv8.KV8Pages(state["table"], state["free"], page, lens=state["cached"], held=state["held"],
                                      n_free=state["n_free"])
        state["next"] = state["pages"].fork()


def _prepare_attention(case, state, g):
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    b, page, fmt, hq, hkv, d = (case[n] for n in ("b", "page", "fmt", "hq", "hkv", "d"))
    lens, new = _lens(case), _new(case)
    width = -(-max(lens) // page)
    need = [-(-n // page) for n in lens]
    n_pages = sum(need) + 3
    order = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32).cpu().numpy()
    table, at = np.zeros((b, width), np.int32), 0
    for i, n in enumerate(need):
        table[i, :n] = order[at:at + n]
        at += n
    if case["op"] == "prefix":               # the shared pages stand in every sequence's row
        first, shared = _groups(case)
        for j, s in enumerate(shared):
            table[first[j]:first[j + 1], :s // page] = table[first[j], :s // page]
        state["groups"], state["shared"] = _ints(first), _ints(shared)
    offsets = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    t = int(offsets[-1])
    blocks = (n_pages, hkv, page // BLOCK, BLOCK, d)
    loud = 1 + 3 * (torch.rand(hkv, 1, 1, d, generator=g, device="cuda") > 0.97)   # a few channels of the keys are large
    cache = {}
    for name, scale in (("k", loud), ("v", 0.5)):
        codes, scales = _quantise((rnd(*blocks) * scale).to(torch.bfloat16).float(), fmt)
        cache[name] = codes.reshape(n_pages, hkv, page, d)
        cache[name + "_scale"] = scales
    qkv = rnd(t, hq + 2 * hkv, d)                        # the fused projection's output
    qkv[:, :hq] *= 2
    state.update(cache=cache, qkv=qkv.to(torch.bfloat16), lens_host=lens, new_host=new, t=t, table=_ints(table),
                 lens=_ints(lens), offsets=_ints(offsets))
    if own:
        from bit_expert_layer_gb300 import kv8
        state["kv"] = kv8.KV8Cache(cache["k"], cache["v"], cache["k_scale"], cache["v_scale"], fmt=fmt)
        state["batch"] = kv8.KV8Batch(state["table"], state["lens"], state["offsets"], max_new=max(new))
        if case["op"] == "prefix":
            state["prefix"] = kv8.KV8Prefix(state["groups"], state["shared"])
            state["workspace"] = state["kv"].new_workspace(hq, max(new), prefix_tokens=t)
        else:
            state["workspace"] = state["kv"].new_workspace(hq, max(new))


# ----------------------------------------------------------------------------- one pass
def run(state):
    case = state["case"]
    op = case["op"]
    if op == "pages":
        if not own:
            return _pages(state)
        pages, after = state["pages"], state["next"]
        offsets, positions, slots = pages.step(state["new"], state["t"], keep=state["keep"], into=after)
        return dict(table=pages.table, free=pages.free, lens=after.lens, held=after.held, n_free=after.n_free, offsets=offsets,
                    positions=positions, slots=slots)
    hq, hkv = case["hq"], case["hkv"]
    q = state["qkv"][:, :hq]
    if op == "norm_rope":
        k = state["qkv"][:, hq:hq + hkv]
        if own:
            return state["norm_rope"](q, k, state["pos"])
        return _norm_rope(q, state["q_weight"], state), _norm_rope(k, state["k_weight"], state)
    if not own:
        return _attention(q, state)
    if op == "window":
        return state["kv"].attention(state["batch"], q, workspace=state["workspace"], window=case["window"], sinks=case["sinks"])
    return state["kv"].attention(state["batch"], q, workspace=state["workspace"], prefix=state["prefix"])


def _norm_rope(x, weight, state):
    half = state["case"]["rot"] // 2
    y = x.float()
    y = y / torch.sqrt((y * y).mean(-1, keepdim=True) + EPS) * (weight.float() + state["case"]["offset"])
    pos = state["pos"].double()[state["axis_index"]]                        # [half, t]
    angle = (pos * state["inv_freq"][:, None]).T[:, None, :]                # [t, 1, half]
    c, s = angle.cos().float(), angle.sin().float()
    a, b = y[..., :half], y[..., half:2 * half]
    return torch.cat([a * c - b * s, b * c + a * s, y[..., 2 * half:]], dim=-1).to(torch.bfloat16)


def _pages(state):
    """Pages that a sequence no longer needs are put on the free list, in order of sequence and
    page; then every sequence that needs more takes them from the list's end, in the same order."""
    page, table, free, held = state["case"]["page"], state["table"], state["free"], state["held"].long()
    lens = state["keep"].long() + state["new"].long()
    n_free, n_pages = state["n_free"].long(), free.shape[0]
    offsets = torch.cat([torch.zeros(1, dtype=torch.int64, device="cuda"), state["new"].long().cumsum(0)])
    after = (lens + page - 1) // page
    give, take = (held - after).clamp_min(0), (after - held).clamp_min(0)
    j = torch.arange(table.shape[1], device="cuda")
    given = (j >= after[:, None]) & (j < held[:, None])
    wanted = (j >= held[:, None]) & (j < after[:, None])
    rank = (give.cumsum(0) - give)[:, None] + j - after[:, None]
    stack = torch.cat([free, torch.zeros(table.numel() + 1, dtype=torch.int32, device="cuda")])
    stack.scatter_(0, torch.where(given, n_free + rank, stack.shape[0] - 1).flatten(), table.flatten())
    top = n_free + give.sum()
    k = (take.cumsum(0) - take)[:, None] + j - held[:, None]
    table = torch.where(wanted, stack[(top - 1 - k).clamp(0, stack.shape[0] - 1)], table)
    left = top - take.sum()
    free = torch.where(torch.arange(n_pages, device="cuda") < left, stack[:n_pages], free)
    i = torch.arange(state["t"], device="cuda")
    seq = torch.bucketize(i, offsets[1:], right=True)
    pos = state["keep"].long()[seq] + i - offsets[seq]
    slots = table[seq, pos // page].long() * page + pos % page
    to = lambda x: x.to(torch.int32)  # noqa: E731
    return dict(table=table, free=free, lens=to(lens), held=to(after), n_free=to(left), offsets=to(offsets), positions=to(pos),
                slots=to(slots))


def _attention(q, state):
    case, c = state["case"], state["cache"]
    b, hq, hkv, d, page, fmt = (case[n] for n in ("b", "hq", "hkv", "d", "page", "fmt"))
    lens, off, new = state["lens"].long(), state["offsets"].long(), max(state["new_host"])
    table = state["table"].long()
    width = table.shape[1] * page
    # the cache as [b, hkv, positions, d], the queries as [b, hkv, group, new, d]
    k = _values(c["k"][table], c["k_scale"][table], fmt).transpose(1, 2).reshape(b, hkv, width, d)
    v = _values(c["v"][table], c["v_scale"][table], fmt).transpose(1, 2).reshape(b, hkv, width, d)
    i = torch.arange(new, device="cuda")
    row = (off[:-1, None] + i).clamp_max(state["t"] - 1)
    qs = q[row].float().view(b, new, hkv, hq // hkv, d).permute(0, 2, 3, 1, 4).reshape(b, hkv, -1, d)
    s = torch.matmul(qs, k.transpose(-1, -2)).view(b, hkv, hq // hkv, new, width) / math.sqrt(d)
    at = ((lens - off[1:] + off[:-1])[:, None] + i)[..., None]              # the new tokens' positions
    there = torch.arange(width, device="cuda")
    ok = there <= at                                                        # [b, new, positions]
    if case["op"] == "window":
        ok = ok & ((there > at - case["window"]) | (there < case["sinks"]))
    s = s.masked_fill_(~ok[:, None, None], -math.inf)
    s = s.sub_(s.amax(-1, keepdim=True)).exp_()
    o = torch.matmul(s.view(b, hkv, -1, width), v).view(b, hkv, hq // hkv, new, d) / s.sum(-1, keepdim=True)
    o = o.permute(0, 3, 1, 2, 4).reshape(b, new, hq, d)
    seq = torch.bucketize(torch.arange(state["t"], device="cuda"), off[1:], right=True)
    return o[seq, torch.arange(state["t"], device="cuda") - off[seq]].to(torch.bfloat16)


# ----------------------------------------------------------------------------- what a pass cannot do without
def work(case):
    op = case["op"]
    if op == "pages":
        cached, keep, new = _requests(case)
        page, t = case["page"], sum(new)
        moved = sum(abs(-(-(k + n) // page) - -(-c // page)) for c, k, n in zip(cached, keep, new))
        # per token its position and slot, per page that changes hands its entry read and written
        return dict(bytes=8 * t + 8 * moved + 28 * case["b"], flops=4 * t)
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    if op == "norm_rope":
        x = case["t"] * (hq + hkv)
        return dict(bytes=4 * x * d + 4 * case["axes"] * case["t"] + 4 * d, flops=x * (4 * d + 3 * case["rot"]))
    lens, new = _lens(case), _new(case)
    row = 2 * hkv * (d + 4 / BLOCK)                        # one position's codes and its share of the scales
    t, rows, seen = sum(new), 0, 0                         # rows of the cache; (query, position) pairs
    if op == "window":
        w, s = case["window"], case["sinks"]
        for n, m in zip(lens, new):
            low = max(0, n - m + 1 - w)                    # the lowest position in a window
            rows += n - low + min(s, low)
            seen += sum(p + 1 - max(0, p + 1 - w) + min(s, max(0, p + 1 - w)) for p in range(n - m, n))
    else:
        first, shared = _groups(case)
        rows = sum(lens) - sum((first[g + 1] - first[g] - 1) * s for g, s in enumerate(shared))
        seen = sum(m * n - m * (m - 1) // 2 for n, m in zip(lens, new))
    return dict(bytes=rows * row + 4 * t * hq * d + 4 * rows // case["page"], flops=4 * seen * hq * d)


# ----------------------------------------------------------------------------- the definition, in 64 bits
def _code_values(fmt):
    """The value of each code."""
    u = np.arange(256)
    if fmt == "int8":
        return np.where(u < 128, u, u - 256).astype(np.float64)
    e, m = (u >> 3) & 15, u & 7
    mag = np.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (e - 10.0))
    mag[127] = mag[255] = np.nan
    return np.where(u < 128, mag, -mag)


def exact(case, seed):
    state = prepare(case, seed)
    if case["op"] == "pages":
        return None                                        # whole numbers only
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    qkv = state["qkv"].double()
    if case["op"] == "norm_rope":
        outs, half = [], case["rot"] // 2
        for x, w in ((qkv[:, :hq], state["q_weight"]), (qkv[:, hq:hq + hkv], state["k_weight"])):
            x = x * (case["offset"] + w.double()) * (torch.linalg.vector_norm(x, dim=-1, keepdim=True) ** 2 / d + EPS) ** -0.5
            out = x.clone()
            for j, a in enumerate(state["axis_of"]):
                turn = state["pos"][a].double() * float(THETA ** (-2.0 * j / case["rot"]))
                c, s = turn.cos()[:, None], turn.sin()[:, None]
                out[:, :, j] = x[:, :, j] * c - x[:, :, j + half] * s
                out[:, :, j + half] = x[:, :, j + half] * c + x[:, :, j] * s
            outs.append(out)
        return tuple(outs)
    page, cache = case["page"], state["cache"]
    of_code = torch.tensor(_code_values(case["fmt"]), device="cuda")
    table, off, outs = state["table"].long(), state["offsets"].tolist(), []
    for i, (n, w) in enumerate(zip(state["lens_host"], state["new_host"])):
        at = torch.arange(n, device="cuda")
        if case["op"] == "window":                         # what no token of the sequence sees is left out
            at = at[(at < case["sinks"]) | (at > n - w - case["window"])]
        pg = table[i, at // page]
        k, v = [of_code[cache[m][pg, :, at % page].long()] * cache[m + "_scale"][pg, :, at % page // BLOCK].double()[..., None]
                for m in ("k", "v")]                       # [positions, hkv, d]
        p = n - w + torch.arange(w, device="cuda")[:, None]
        hide = at > p
        if case["op"] == "window":
            hide |= (p - at >= case["window"]) & (at >= case["sinks"])
        q = qkv[off[i]:off[i + 1], :hq].unflatten(1, (hkv, hq // hkv))       # [w, hkv, group, d]
        o = torch.empty(w, hkv, hq // hkv, d, device="cuda", dtype=torch.float64)
        for h in range(hkv):
            for r in range(hq // hkv if w > 64 else 1):    # a head at a time, or all of a group
                part = slice(r, r + 1) if w > 64 else slice(None)
                s = torch.einsum("wgd,nd->gwn", q[:, h, part], k[:, h]) * d ** -0.5
                o[:, h, part] = torch.einsum("gwn,nd->wgd", torch.softmax(s.masked_fill(hide, -math.inf), dim=-1), v[:, h])
        outs.append(o.flatten(1, 2))
    return torch.cat(outs)
