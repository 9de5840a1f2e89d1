"""Window and prefix attention, head norms with rotary positions and page tables on the GPU, against
tests/serving_ref.py: whole numbers for equality, the others within bounds derived there."""
from __future__ import annotations

import copy
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")
import kv8_ref  # noqa: E402
import serving_ref  # noqa: E402
from test_gpu_kv8 import EDGE, LAYOUTS, Setup, gen, ints, kv8  # noqa: E402, F401

pytestmark = pytest.mark.gpu


def check(s, out, lens=None, table=None, **kw):
    n = int(s.offsets[-1])
    want, bound = serving_ref.attention(s.ref(), s.table if table is None else table, s.lens if lens is None else lens, s.offsets,
                                        s.q[:n].double(), **kw)
    err = (out[:n].double() - want).abs()
    assert torch.isfinite(out[:n]).all()
    worst = torch.argmax((err / bound).flatten())
    assert torch.all(err <= bound), (np.unravel_index(int(worst), err.shape), float(err.flatten()[worst]),
                                     float(bound.flatten()[worst]))


# ----------------------------------------------------------------------------- sliding windows and sinks
@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("page", [16, 64])
@pytest.mark.parametrize("layout", LAYOUTS, ids=str)
@pytest.mark.parametrize("window,sinks", [(1, 0), (16, 4), (33, 17), (100, 0)])
def test_window_one_token(kv8, layout, page, fmt, window, sinks):
    s = Setup(kv8, EDGE, [1] * len(EDGE), layout, page, fmt, seed=layout[0] + page)
    check(s, s.cache.attention(s.batch, s.q, window=window, sinks=sinks), window=window, sinks=sinks)
    assert s.cache.get_error() == 0


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("layout", LAYOUTS, ids=str)
@pytest.mark.parametrize("lens,new", [([5, 40, 100], [2, 2, 2]), ([70, 9, 333], [5, 4, 8]), ([20, 300], [20, 17]),
                                      ([131, 513, 64], [131, 130, 33])], ids=["two", "eight", "twenty", "prompt"])
@pytest.mark.parametrize("window,sinks", [(1, 2), (30, 0), (128, 130)])
def test_window_several_tokens(kv8, layout, fmt, lens, new, window, sinks):
    s = Setup(kv8, lens, new, layout, 32, fmt, seed=layout[0] + len(new), pad=2)
    out = torch.full(s.q.shape, 5.0, dtype=torch.bfloat16, device="cuda")
    s.cache.attention(s.batch, s.q, out=out, window=window, sinks=sinks)
    check(s, out, window=window, sinks=sinks)
    assert (out[int(s.offsets[-1]):] == 5).all() and s.cache.get_error() == 0


@pytest.mark.parametrize("fmt,lens,new,window,sinks", [("e4m3", [32768, 4097], [1, 1], 4096, 4), ("int8", [20001], [1], 700, 0),
                                                       ("e4m3", [9000, 8192], [4, 4], 1024, 33), ("int8", [5000], [700], 512, 4),
                                                       ("e4m3", [2048], [2048], 300, 1), ("e4m3", [6000], [1500], 64, 200)],
                         ids=["decode-32k", "decode-20k", "draft", "piece", "prompt", "far-sinks"])
def test_window_long(kv8, fmt, lens, new, window, sinks):
    s = Setup(kv8, lens, new, fmt=fmt, seed=lens[0])
    check(s, s.cache.attention(s.batch, s.q, window=window, sinks=sinks), window=window, sinks=sinks)


@pytest.mark.parametrize("new", [1, 3, 70])
@pytest.mark.parametrize("window,sinks", [(1 << 24, 0), (600, 0), (1, 1 << 24), (100, 600)])
def test_a_window_over_everything_is_causal_attention(kv8, new, window, sinks):
    """Also where sinks and window meet or overlap.  Units are divided differently, so not bit for bit."""
    s = Setup(kv8, [500, 77, 70], [new] * 3, seed=41)
    check(s, s.cache.attention(s.batch, s.q, window=window, sinks=sinks))


@pytest.mark.parametrize("new", [1, 3, 130])
@pytest.mark.parametrize("page", [16, 64, 256])
@pytest.mark.parametrize("window,sinks", [(50, 4), (17, 0), (200, 20)])
def test_pages_that_no_token_sees_may_be_gone(kv8, new, page, window, sinks):
    """Their page-table entries are out of range, their codes NaN: nothing is read or recorded."""
    lens = [900, 411, new]
    s = Setup(kv8, lens, [new] * 3, page=page, seed=42)
    a = s.cache.attention(s.batch, s.q, window=window, sinks=sinks)
    check(s, a, window=window, sinks=sinks)
    t, gone = s.table.copy(), []
    for b, n in enumerate(lens):
        for j in range(-(-n // page)):
            if j * page >= sinks and (j + 1) * page <= n - new + 1 - window:
                gone.append(t[b, j])
                t[b, j] = (-1, 2 ** 31 - 1, s.n_pages)[j % 3]
    for x in gone:
        s.cache.k[int(x)] = 0x7F
        s.cache.v[int(x)] = 0x7F
        s.cache.k_scale[int(x)] = math.nan
        s.cache.v_scale[int(x)] = math.inf
    b = kv8.KV8Batch(ints(t), s.batch.lens, s.batch.offsets, s.batch.max_new)
    assert torch.equal(s.cache.attention(b, s.q, window=window, sinks=sinks), a) and s.cache.get_error() == 0


@pytest.mark.parametrize("new", [1, 3])
def test_window_many_sequences(kv8, new):
    rng = np.random.RandomState(3)
    lens = [int(x) for x in rng.choice([3, 5, 16, 40, 100, 257], 1024)]
    s = Setup(kv8, lens, [0 if i % 17 == 5 else new for i in range(1024)], (4, 2, 64), 16, seed=8)
    check(s, s.cache.attention(s.batch, s.q, window=37, sinks=3), window=37, sinks=3)


@pytest.mark.parametrize("layout", [(16, 2, 128), (16, 1, 128), (7, 7, 64)], ids=str)
@pytest.mark.parametrize("n,new", [(100, 400), (0, 300), (126, 129), (3, 4), (0, 1)])
def test_window_with_fewer_positions_than_new_tokens(kv8, n, new, layout):
    from bit_expert_layer_gb300 import _abi
    s = Setup(kv8, [300, n, 200], [2, new, 3], layout, seed=43)
    out = s.cache.attention(s.batch, s.q, window=40, sinks=5)
    check(s, out, window=40, sinks=5)
    assert (out[2:2 + new - n] == 0).all() and s.cache.get_error() == _abi.MOE_ERR_DEVICE_BOUNDS


@pytest.mark.parametrize("new", [1, 4, 90])
def test_window_extremes(kv8, new):
    """Scores of any size, value scales far apart, rows that are not finite: as without a window."""
    s = Setup(kv8, [400, 300], [new, new], seed=44, q_gain=1.0)
    c = s.cache
    c.v_scale[:] = torch.exp2(torch.randint(-30, 10, c.v_scale.shape, generator=s.g, device="cuda").float())
    s.q[0] = 0
    s.q[new] *= 2.0 ** 60
    c.k_scale[int(s.table[1, 0]):] *= 2.0 ** -58
    a = c.attention(s.batch, s.q, window=100, sinks=20)
    check(s, a, window=100, sinks=20)
    s.q[new - 1, 3, 5] = math.nan
    b = c.attention(s.batch, s.q, window=100, sinks=20)
    keep = torch.ones(2 * new, 16, dtype=torch.bool, device="cuda")
    keep[new - 1, 3] = False
    assert torch.equal(a[keep], b[keep]) and torch.isnan(b[~keep]).all()


def test_window_three_million_positions(kv8):
    """A far window: positions of a long sequence that reads the same pages over and over."""
    s = Setup(kv8, [256], [1], seed=45)
    n = 700 * 256 * 16
    t = np.tile(s.table[0], n // 256)[None]
    for new in (1, 40):
        q = s.q[:1].expand(new, -1, -1).contiguous()
        b = kv8.KV8Batch(ints(t), ints([n]), ints([0, new]), new)
        out = s.cache.attention(b, q, window=256, sinks=0)
        # the last token sees every position of the 256 once; the others too, in another order
        want = serving_ref.attention(s.ref(), s.table, [256], [0, 1], s.q[:1].double())
        err = (out.double() - want[0]).abs()
        assert torch.all(err <= want[1])
    assert s.cache.get_error() == 0


# ----------------------------------------------------------------------------- shared prefixes
ALWAYS = 1 << 24         # a bound under which sharing pays from few sequences on


class Shared(Setup):
    """Groups of sequences: groups[i] sequences that share[i] positions; own[b] positions after them."""

    def __init__(self, kv8, groups, share, own, new, layout=(16, 2, 128), page=64, fmt="e4m3", seed=0, pad=0, **kw):
        lens, first = [], [0]
        for g, n in zip(groups, share):
            lens += [n + x for x in own[first[-1]:first[-1] + g]]
            first.append(first[-1] + g)
        super().__init__(kv8, lens, new, layout, page, fmt, seed, pad, **kw)
        for i, n in enumerate(share):
            rows = self.table[first[i]:first[i + 1]]
            if len(rows):
                rows[:, :n // page] = rows[0, :n // page]
                if n % page:                           # the partly shared page is copied
                    for r in rows[1:]:
                        src, dst, m = int(rows[0, n // page]), int(r[n // page]), n % page
                        for x in (self.cache.k, self.cache.v):
                            x[dst, :, :m] = x[src, :, :m]
                        for x in (self.cache.k_scale, self.cache.v_scale):
                            x[dst, :, :-(-m // 16)] = x[src, :, :-(-m // 16)]
        self.batch = kv8.KV8Batch(ints(self.table), ints(self.lens), ints(self.offsets), max_new=max(1, max(new)))
        self.prefix = kv8.KV8Prefix(ints(first), ints(share), ALWAYS)


PREFIX = [([8], [256], [20] * 8, [1] * 8), ([5], [1000], [3, 1, 130, 40, 7], [3, 1, 2, 3, 3]),
          ([9, 1, 7], [300, 128, 129], list(range(1, 18)), [1] * 17),
          ([4, 3], [128, 700], [50, 60, 70, 300, 64, 64, 33], [17, 40, 1, 200, 33, 2, 5])]


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("page", [16, 64])
@pytest.mark.parametrize("layout", LAYOUTS, ids=str)
@pytest.mark.parametrize("case", PREFIX, ids=["decode", "draft", "groups", "prompt"])
def test_prefix(kv8, case, layout, page, fmt):
    s = Shared(kv8, *case, layout, page, fmt, seed=layout[0] + page, pad=3)
    out = torch.full(s.q.shape, 5.0, dtype=torch.bfloat16, device="cuda")
    s.cache.attention(s.batch, s.q, out=out, prefix=s.prefix)
    check(s, out)
    assert (out[int(s.offsets[-1]):] == 5).all() and s.cache.get_error() == 0


@pytest.mark.parametrize("fmt,groups,share,own,new", [("e4m3", [64], [8192], [100] * 64, [1] * 64),
                                                      ("int8", [13, 11], [5001, 3003], [40] * 24, [4] * 24),
                                                      ("e4m3", [3], [6000], [500, 100, 900], [400, 100, 20])],
                         ids=["decode", "draft", "prompt"])
def test_prefix_long(kv8, fmt, groups, share, own, new):
    s = Shared(kv8, groups, share, own, new, fmt=fmt, seed=51)
    check(s, s.cache.attention(s.batch, s.q, prefix=s.prefix))
    assert s.cache.get_error() == 0


def test_prefix_of_the_largest_batch(kv8):
    """1024 sequences in 300 groups, empty groups and empty sequences among them."""
    rng = np.random.RandomState(4)
    cut = np.sort(rng.randint(0, 1025, 299))
    groups = np.diff(np.concatenate([[0], cut, [1024]])).tolist()
    share = [int(x) for x in rng.choice([0, 100, 128, 260], 300)]
    new = [0 if i % 13 == 5 else 3 for i in range(1024)]
    s = Shared(kv8, groups, share, [3 + i % 40 for i in range(1024)], new, (16, 1, 64), 16, seed=52)
    out = torch.zeros_like(s.q)
    s.cache.attention(s.batch, s.q, out=out, prefix=s.prefix)
    check(s, out)
    assert s.cache.get_error() == 0


@pytest.mark.parametrize("new", [1, 3, 20])
@pytest.mark.parametrize("page", [256, 1024])
def test_prefix_and_window_with_large_pages(kv8, page, new):
    """The shared positions end inside a page; the first rows of the call belong to no sequence."""
    s = Shared(kv8, [7, 5], [1000, 640], [new + 30 * i for i in range(12)], [new] * 12, page=page, seed=65)
    s.offsets = s.offsets + 3
    qkv = torch.cat([s.qkv[:3], s.qkv])
    s.q = qkv[:, :s.hq]
    b = kv8.KV8Batch(s.batch.page_table, s.batch.lens, ints(s.offsets), new)
    for kw in (dict(prefix=s.prefix), dict(window=100, sinks=20)):
        out = torch.full(s.q.shape, 5.0, dtype=torch.bfloat16, device="cuda")
        s.cache.attention(b, s.q, out=out, **kw)
        want, bound = serving_ref.attention(s.ref(), s.table, s.lens, s.offsets, s.q.double(), **{k: v for k, v in kw.items() if k != "prefix"})
        assert torch.all((out[3:].double() - want[3:]).abs() <= bound[3:]) and (out[:3] == 5).all()
    assert s.cache.get_error() == 0


def test_many_groups(kv8):
    """100 groups of 10 sequences; as many groups as there can be, most of them of one sequence (which
    share nothing); more groups than sequences."""
    g = Shared(kv8, [10] * 100, [128 * (i % 4) + 5 for i in range(100)], [1 + i % 70 for i in range(1000)], [1] * 1000, (16, 1, 64), 16,
               seed=68)
    check(g, g.cache.attention(g.batch, g.q, prefix=g.prefix))
    assert g.cache.get_error() == 0
    n = 1023
    s = Shared(kv8, [1] * 20 + [2] * 2 + [1] * (n - 24), [128 * (i % 3) for i in range(n - 2)], [1 + i % 50 for i in range(n)], [1] * n,
               (16, 1, 64), 16, seed=66)
    check(s, s.cache.attention(s.batch, s.q, prefix=s.prefix))
    few = Shared(kv8, [12], [300], [20 + i for i in range(12)], [4] * 12, seed=67)
    many = kv8.KV8Prefix(ints([0] * 500 + [12] * 525), ints([300] * 1024), ALWAYS)
    check(few, few.cache.attention(few.batch, few.q, prefix=many))
    assert s.cache.get_error() == 0 and few.cache.get_error() == 0


@pytest.mark.parametrize("new", [1, 3, 40])
def test_sequences_that_share_nothing(kv8, new):
    """Outside every group; new tokens that begin before the shared positions end; a group that shares
    less than 128; and few query rows, where nothing is shared at all."""
    from bit_expert_layer_gb300 import _abi
    s = Shared(kv8, [12], [512], [40 + i for i in range(12)], [new] * 12, seed=53)
    c = s.cache
    for first, share in [([3, 7], [512]), ([0, 4, 4, 12], [512, 0, 512]), ([0, 12], [127]), ([0, 0], [512]), ([12, 12], [512])]:
        check(s, c.attention(s.batch, s.q, prefix=kv8.KV8Prefix(ints(first), ints(share), ALWAYS)))
    assert c.get_error() == 0
    lens = list(s.lens)
    lens[4], lens[9] = 512 + new - 1, 300           # the first has a new token among the shared ones
    b = kv8.KV8Batch(s.batch.page_table, ints(lens), s.batch.offsets, new)
    check(s, c.attention(b, s.q, prefix=s.prefix), lens=lens)
    assert c.get_error() == 0
    # groups and lengths out of order or range: recorded, and the result is still theirs
    for first, share in [([4, 2], [512]), ([-1, 12], [512]), ([0, 13], [512]), ([0, 2 ** 31 - 1], [512]), ([0, 12], [-5])]:
        check(s, c.attention(s.batch, s.q, prefix=kv8.KV8Prefix(ints(first), ints(share), ALWAYS)))
        assert c.get_error() == _abi.MOE_ERR_DEVICE_BOUNDS
    check(s, c.attention(s.batch, s.q, prefix=kv8.KV8Prefix(ints([0, 12]), ints([2 ** 31 - 1]), ALWAYS)))
    assert c.get_error() == _abi.MOE_ERR_DEVICE_BOUNDS
    # too little to share for it to pay: the ordinary kernels
    plain = c.attention(s.batch, s.q)
    for few in (kv8.KV8Prefix(ints([0, 12]), ints([512])), kv8.KV8Prefix(ints([0, 12]), ints([512]), 100)):
        assert torch.equal(c.attention(s.batch, s.q, prefix=few), plain)


@pytest.mark.parametrize("bound", [127, 128, 300, 511, 513])
def test_shared_positions_past_the_bound_are_the_sequences_own(kv8, bound):
    """120 sequences, so that sharing pays from few positions on (or not at all); never a position twice."""
    s = Shared(kv8, [120], [512], [20 + i for i in range(120)], [4] * 120, (16, 1, 64), seed=63)
    check(s, s.cache.attention(s.batch, s.q, prefix=kv8.KV8Prefix(ints([0, 120]), ints([512]), bound)))
    big = Shared(kv8, [60], [9000], [20 + i for i in range(60)], [1] * 60, seed=64)
    check(big, big.cache.attention(big.batch, big.q, prefix=kv8.KV8Prefix(ints([0, 60]), ints([9000]), 16 * bound)))
    assert s.cache.get_error() == 0 and big.cache.get_error() == 0


@pytest.mark.parametrize("new", [1, 4, 90])
def test_prefix_extremes(kv8, new):
    """All the weight before or behind the border, zero blocks, rows that are not finite."""
    s = Shared(kv8, [6], [384], [100] * 6, [new] * 6, seed=55, q_gain=1.0)
    c = s.cache
    c.v_scale[:] = torch.exp2(torch.randint(-30, 10, c.v_scale.shape, generator=s.g, device="cuda").float())
    c.v[int(s.table[0, 1])] = 0
    c.v_scale[int(s.table[0, 1])] = 2.0 ** -100
    for b, at in ((0, 5), (1, 400), (2, 383), (3, 384)):           # one key that the sequence's queries point to
        page, i = int(s.table[b, at // 64]), at % 64
        c.k[page, :, i] = 0x7E                                     # 448 in all dims
        s.q[s.offsets[b]:s.offsets[b + 1]] = 1.0
    s.q[s.offsets[4]] = 0
    s.q[s.offsets[5]] *= 2.0 ** -60
    a = c.attention(s.batch, s.q, prefix=s.prefix)
    check(s, a)
    s.q[new - 1, 3, 5] = math.nan
    s.q[new, 8] = math.inf
    b = c.attention(s.batch, s.q, prefix=s.prefix)
    keep = torch.ones(6 * new, 16, dtype=torch.bool, device="cuda")
    keep[new - 1, 3] = keep[new, 8] = False
    assert torch.equal(a[keep], b[keep]) and torch.isnan(b[~keep]).all()


@pytest.mark.parametrize("new", [1, 40])
def test_prefix_bad_pages(kv8, new):
    """A shared page out of range is left out for the whole group, an own one for its sequence."""
    from bit_expert_layer_gb300 import _abi
    s = Shared(kv8, [6], [512], [100] * 6, [new] * 6, page=16, seed=56)
    good = s.cache.attention(s.batch, s.q, prefix=s.prefix)
    for at in (3, 34):
        t = s.table.copy()
        t[0, at] = s.n_pages
        b = kv8.KV8Batch(ints(t), s.batch.lens, s.batch.offsets, new)
        out = s.cache.attention(b, s.q, prefix=s.prefix)
        assert s.cache.get_error() == _abi.MOE_ERR_DEVICE_BOUNDS and torch.isfinite(out).all()
        if at == 34:
            assert torch.equal(out[new:], good[new:])
    assert torch.equal(s.cache.attention(s.batch, s.q, prefix=s.prefix), good) and s.cache.get_error() == 0


@pytest.mark.parametrize("kind", ["window", "prefix"])
@pytest.mark.parametrize("new", [1, 4, 50])
def test_same_bits_streams_graphs_and_workspaces(kv8, kind, new):
    """The same call gives the same bits: again, on another stream, two at once with a workspace each,
    captured and replayed with other inputs, and on a workspace that served other shapes."""
    s = Shared(kv8, [9], [700], [90 + 9 * i for i in range(9)], [new] * 9, seed=57)
    o = Shared(kv8, [20, 3], [300, 2000], [33] * 23, [1] * 23, (10, 2, 128), seed=58)
    kw = lambda x: dict(window=200, sinks=9) if kind == "window" else dict(prefix=x.prefix)  # noqa: E731
    ws = [max((x.cache.new_workspace(x.hq, x.batch.max_new, x.t if kind == "prefix" else 0) for x in (s, o)),
              key=lambda w: w.numel()) for _ in range(2)]
    a, b = (x.cache.attention(x.batch, x.q, **kw(x)) for x in (s, o))
    check(s, a, **(kw(s) if kind == "window" else {}))
    for _ in range(3):
        for x, want in ((s, a), (o, b)):
            assert torch.equal(x.cache.attention(x.batch, x.q, workspace=ws[0], **kw(x)), want)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [s.cache.attention(s.batch, s.q, workspace=w, stream=st, **kw(s)) for _ in range(5) for w, st in zip(ws, streams)]
    torch.cuda.synchronize()
    assert all(torch.equal(x, a) for x in outs)
    out, q = torch.zeros_like(s.q).contiguous(), s.q.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s.cache.attention(s.batch, q, out=out, workspace=ws[0], **kw(s))
    graph.replay()
    assert torch.equal(out, a)
    q.mul_(0.5)
    s.batch.lens.sub_(50)                      # the graph follows its inputs
    s.prefix.shared.fill_(130)
    graph.replay()
    o.cache.attention(o.batch, o.q, workspace=ws[0], **kw(o))
    s.q[:] = q
    check(s, out, lens=[n - 50 for n in s.lens], **(kw(s) if kind == "window" else {}))
    assert torch.equal(out, s.cache.attention(s.batch, s.q, workspace=ws[1], **kw(s))) and s.cache.get_error() == 0


@pytest.mark.parametrize("kind", ["window", "prefix"])
def test_attention_short_wait_limit(kv8, kind):
    """A wait that gives up is recorded (one whose data is there at its first look does not give up),
    and the next call on the same workspace is whole again."""
    from bit_expert_layer_gb300 import _abi
    s = Shared(kv8, [24], [6000], [500] * 24, [1] * 24, seed=59)
    kw = dict(window=4000, sinks=4) if kind == "window" else dict(prefix=s.prefix)
    ws = s.cache.new_workspace(16, 1, 24)
    a = s.cache.attention(s.batch, s.q, workspace=ws, **kw)
    _abi.moe_set_wait_limit_ns(1)
    try:
        b = s.cache.attention(s.batch, s.q, workspace=ws, **kw)
        torch.cuda.synchronize()
    finally:
        _abi.moe_set_wait_limit_ns(0)
    assert s.cache.get_error() == _abi.MOE_ERR_TIMEOUT or torch.equal(a, b)
    assert torch.equal(s.cache.attention(s.batch, s.q, workspace=ws, **kw), a) and s.cache.get_error() == 0


def test_attention_refusals(kv8):
    s = Shared(kv8, [3], [200], [20, 30, 40], [1] * 3, seed=60)
    c = s.cache
    with pytest.raises(ValueError):
        c.attention(s.batch, s.q, sinks=4)
    with pytest.raises(ValueError):
        c.attention(s.batch, s.q, window=4, prefix=s.prefix)
    for w in (0, -3, 1 << 25):
        with pytest.raises(RuntimeError):
            c.attention(s.batch, s.q, window=w)
    with pytest.raises(RuntimeError):          # the workspace of a call without a prefix
        c.attention(s.batch, s.q, workspace=c.new_workspace(16, 1), prefix=s.prefix)
    with pytest.raises(ValueError):
        kv8.KV8Prefix(ints([0, 3]), ints([5, 5]))
    with pytest.raises(ValueError):
        kv8.KV8Prefix(ints([0]), ints([]))
    for bound in (-1, (1 << 24) + 1):
        with pytest.raises(ValueError):
            kv8.KV8Prefix(ints([0, 3]), ints([5]), bound)
    with pytest.raises(ValueError):
        kv8.KV8Prefix(ints([0, 3]).cpu(), ints([5]))
    with pytest.raises(ValueError):
        kv8.KV8Prefix(ints([0, 3]).long(), ints([5]))
    e = c.attention(s.batch, s.q[:0], window=5)
    assert e.shape == (0, 16, 128) and c.attention(s.batch, s.q[:0], prefix=s.prefix).shape == (0, 16, 128)


# ----------------------------------------------------------------------------- norms with rotary positions
@pytest.mark.parametrize("t", [1, 2, 7, 64, 2049])
@pytest.mark.parametrize("d,rotary,axes,cyclic", [(128, 128, 1, False), (128, 32, 3, True), (64, 64, 3, False),
                                                  (64, 16, 2, True), (128, 96, 4, True)])
@pytest.mark.parametrize("dtype,offset", [(torch.bfloat16, 0.0), (torch.float32, 1.0), (None, 0.0)], ids=["bf16", "fp32", "ones"])
def test_norm_rope(kv8, t, d, rotary, axes, cyclic, dtype, offset):
    g = gen(t * 7 + d + rotary)
    half = rotary // 2
    sections = [half - (axes - 1) * (half // axes)] + [half // axes] * (axes - 1)
    rope = kv8.Rope(d, rotary, theta=1e6, sections=sections, cyclic=cyclic)
    x = (torch.randn(t, 7, d, generator=g, device="cuda") * torch.exp2(torch.randint(-20, 20, (t, 7, 1), generator=g, device="cuda"))).to(torch.bfloat16)
    wq, wk = (None if dtype is None else (torch.randn(d, generator=g, device="cuda") + 1 - offset).to(dtype) for _ in range(2))
    pos = torch.randint(-1000000, 1000000, (axes, t), generator=g, device="cuda", dtype=torch.int32)
    inv, axis_of = [1e6 ** (-2 * j / rotary) for j in range(half)], list(rope.plan.axis)[:half]
    op = kv8.NormRope(rope, wq, wk, eps=1e-6, offset=offset)
    q, k = op(x[:, :5], x[:, 5:], pos)
    for got, part, w in ((q, x[:, :5], wq), (k, x[:, 5:], wk)):
        want, bound = serving_ref.norm_rope(part.double(), w, 1e-6, offset, pos, inv, axis_of, rotary)
        assert torch.all((got.double() - want).abs() <= bound)
    # in place, in a wider tensor: the other heads stay; q alone
    y = x.clone()
    op(y[:, 1:5], y[:, 5:], pos, out=(y[:, 1:5], y[:, 5:]))
    assert torch.equal(y[:, 1:5], q[:, 1:]) and torch.equal(y[:, 5:], k) and torch.equal(y[:, 0], x[:, 0])
    q2, none = op(x[:, :5], None, pos)
    assert none is None and torch.equal(q2, q)


@pytest.mark.parametrize("eps", [0.0, 1e-30, 1e-6, 1.0])
def test_norm_rope_magnitudes(kv8, eps):
    """Heads whose squares leave fp32 at either end, zeros, subnormals, one large number among small
    ones; infinities and NaN stay in their heads."""
    g = gen(61)
    x = torch.randn(40, 3, 128, generator=g, device="cuda").double()
    x[0] = 0
    x[1, 0] = 2.0 ** -133
    for i, e in enumerate((-130, -120, -75, -64, -50, -40, 30, 59, 60, 61, 64, 100, 120)):
        x[2 + i] *= 2.0 ** e
    x[20, :, 1:] = 0
    x[21, :, 5] = 3e38
    x = x.to(torch.bfloat16)
    pos = torch.arange(40, dtype=torch.int32, device="cuda")
    rope = kv8.Rope(128, 128, theta=1e4)
    inv = [1e4 ** (-2 * j / 128) for j in range(64)]
    op = kv8.NormRope(rope, eps=eps)
    q, _ = op(x, None, pos)
    want, bound = serving_ref.norm_rope(x.double(), None, eps, 0.0, pos[None], inv, [0] * 64, 128)
    assert torch.all((q.double() - want).abs() <= bound)
    z = x.clone()
    z[30, 1, 3], z[31, 2, 7], z[32, 0, 100] = math.inf, math.nan, -math.inf
    q2, _ = op(z, None, pos)
    keep = torch.ones(40, 3, dtype=torch.bool, device="cuda")
    keep[30, 1] = keep[31, 2] = keep[32, 0] = False
    assert torch.equal(q2[keep], q[keep])
    assert torch.isnan(q2[31, 2]).all()
    # an infinity: zeros beside it, and NaN in its pair
    for r, h, j in ((30, 1, 3), (32, 0, 100)):
        pair = torch.zeros(128, dtype=torch.bool, device="cuda")
        pair[j % 64] = pair[j % 64 + 64] = True
        assert torch.isnan(q2[r, h][pair]).all() and (q2[r, h][~pair] == 0).all()


def test_norm_rope_streams_graphs_and_refusals(kv8):
    g = gen(62)
    rope = kv8.Rope(64, 32)
    w = torch.randn(64, generator=g, device="cuda")
    op = kv8.NormRope(rope, w, w.clone(), eps=1e-5)
    x = torch.randn(100, 6, 64, generator=g, device="cuda").to(torch.bfloat16)
    pos = torch.arange(100, dtype=torch.int32, device="cuda")
    a = op(x[:, :4], x[:, 4:], pos)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    b = op(x[:, :4], x[:, 4:], pos, stream=st)
    st.synchronize()
    assert all(torch.equal(m, n) for m, n in zip(a, b))
    out = tuple(torch.zeros_like(m) for m in a)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        op(x[:, :4], x[:, 4:], pos, out=out)
    w.mul_(2)                                   # the weights are read when the kernel runs
    graph.replay()
    assert torch.equal(out[0].float(), 2 * a[0].float()) and torch.equal(out[1], a[1])
    for bad in (w[:32], w.double(), w.cpu(), w[:, None], torch.randn(128, device="cuda")[::2]):
        with pytest.raises(ValueError):
            kv8.NormRope(rope, bad)
    with pytest.raises(ValueError):
        kv8.NormRope(rope, w, w.to(torch.bfloat16))
    for eps in (-1e-6, math.nan, math.inf):
        with pytest.raises(ValueError):
            kv8.NormRope(rope, w, w, eps=eps)
    with pytest.raises(ValueError):
        op(x[:, :4].float(), None, pos)
    e, _ = op(x[:0], None, pos[:0])
    assert e.shape == (0, 6, 64)


# ----------------------------------------------------------------------------- page tables
class Pool:
    """A KV8Pages with some sequences in it and the same in lists."""

    def __init__(self, kv8, lens, page=64, spare=10, width=None, n_pages=None, seed=0, borrowed=None):
        rng = np.random.RandomState(seed)
        held = [-(-n // page) for n in lens]
        self.n_pages = n_pages or sum(held) + spare
        order = rng.permutation(self.n_pages).tolist()
        width = width or max(held) + 8
        table, at = rng.randint(0, 99, (len(lens), width)).tolist(), 0
        for i, n in enumerate(held):
            table[i][:n] = order[at:at + n]
            at += n
        free = order[at:] + [-3] * at
        self.ref = serving_ref.Pages(table, free, self.n_pages - at, lens, held, page)
        self.pages = kv8.KV8Pages(ints(table), ints(free), page, ints(lens), ints(held), ints([self.n_pages - at]),
                                  None if borrowed is None else ints(borrowed))
        self.borrowed = borrowed

    def step(self, new, keep=None, into=None, pad=5, check_error=True):
        t = sum(new)
        out = tuple(torch.full((n,), -9, dtype=torch.int32, device="cuda") for n in (len(new) + 1, t + pad, t + pad))
        self.pages.step(ints(new), t + pad, None if keep is None else ints(keep), out=out, into=into)
        *want, missing = self.ref.step(new, keep, self.borrowed)
        for x, w in zip(out, want):
            assert x.tolist() == w + [-9] * (x.numel() - len(w))
        self.check(into or self.pages)
        if check_error:
            assert (self.pages.get_error() != 0) == missing
        return out

    def check(self, pages):
        assert pages.table.tolist() == self.ref.table and pages.free.tolist() == self.ref.free
        assert pages.lens.tolist() == self.ref.lens and pages.held.tolist() == self.ref.held
        assert pages.n_free.tolist() == [self.ref.n_free] and pages.control.tolist()[1] == 0


@pytest.mark.parametrize("page", [16, 64, 1024])
@pytest.mark.parametrize("n", [1, 7, 300, 1024])
def test_pages_steps(kv8, page, n):
    """Many steps of every kind: admissions, single tokens, drafts that fall back, requests that are done."""
    rng = np.random.RandomState(n + page)
    pool = Pool(kv8, [0] * n, page, n_pages=n * 5 + 7, width=12)
    for i in range(8):
        lens = pool.ref.lens
        keep = [int(rng.choice([0, x, x, x, max(0, x - int(rng.randint(0, 90)))])) for x in lens]
        new = [int(rng.choice([0, 1, 1, 4, rng.randint(0, 2 * page)])) for _ in range(n)]
        new = [min(m, 12 * page - k) for m, k in zip(new, keep)]
        pool.step(new, None if i % 3 == 2 and max(a + b for a, b in zip(lens, new)) <= 12 * page else keep)


@pytest.mark.parametrize("lens,new,keep", [([0], [0], None), ([5], [0], [0]), ([0], [100000], None), ([64, 128, 1], [0, 1, 63], None),
                                           ([1000, 900, 800], [0, 0, 700], [0, 0, 800]), ([300] * 4, [1, 900, 0, 2], [300, 0, 10, 299])])
def test_pages_edges(kv8, lens, new, keep):
    pool = Pool(kv8, lens, spare=2000, width=1700)
    pool.step(new, keep)
    pool.step([1] * len(lens))


def test_pages_large_prompts(kv8):
    """A million tokens; rows that are not 16-byte aligned."""
    rng = np.random.RandomState(9)
    new = rng.randint(0, 2040, 1024).tolist()
    pool = Pool(kv8, [0] * 1024, 16, n_pages=70000, width=130)
    pool.step(new)
    t = sum(new)
    assert t > 1000000
    big = torch.full((2, t + 9), -9, dtype=torch.int32, device="cuda")
    other = Pool(kv8, [0] * 1024, 16, n_pages=70000, width=130)
    out = (torch.zeros(1025, dtype=torch.int32, device="cuda"), big[0, 1:t + 1], big[1, 3:t + 3])
    other.pages.step(ints(new), t, out=out)
    *want, _ = other.ref.step(new)
    assert out[1].tolist() == want[1] and out[2].tolist() == want[2]
    assert big[0, 0] == -9 and (big[0, t + 1:] == -9).all() and (big[1, :3] == -9).all() and (big[1, t + 3:] == -9).all()


def test_pages_the_list_runs_out(kv8):
    """Some entries become -1 and are asked for again when pages come back."""
    pool = Pool(kv8, [100, 200, 300], 64, spare=3)
    pool.step([200, 200, 200])
    pool.step([1, 1, 1])
    pool.step([0, 1, 0], [301, 401, 0])
    pool.step([1, 1, 1])
    assert -1 not in sum((r[:h] for r, h in zip(pool.ref.table, pool.ref.held)), [])


def test_pages_borrowed(kv8):
    """The first pages of a row that belong to a shared prefix are not given back."""
    pool = Pool(kv8, [640, 200, 300], 64, spare=9, borrowed=[4, 0, 2])
    pool.step([0, 10, 0], [0, 200, 100])
    pool.borrowed[:] = [0, 0, 1]
    pool.pages.borrowed.copy_(ints(pool.borrowed))
    pool.step([70, 0, 1])
    pool.step([0, 0, 0], [0, 0, 0])


def test_pages_fork_and_graph(kv8):
    """A step into another state leaves the first one good; a captured step goes on from replay to replay."""
    pool = Pool(kv8, [100, 200, 300], 64, spare=40)
    before = (list(pool.ref.lens), list(pool.ref.held), pool.ref.n_free)
    draft = pool.pages.fork()
    out = tuple(torch.zeros(n, dtype=torch.int32, device="cuda") for n in (4, 300, 300))
    pool.pages.step(ints([100, 100, 100]), 300, out=out, into=draft)
    assert (pool.pages.lens.tolist(), pool.pages.held.tolist(), pool.pages.n_free.item()) == before
    assert draft.lens.tolist() == [200, 300, 400]
    taken = copy.deepcopy(pool.ref)             # the table is one: the draft's entries stand behind those that are held
    taken.step([100, 100, 100])
    pool.ref.table = taken.table
    pool.step([10, 0, 70])                      # the draft was not taken
    new = ints([1, 3, 0])
    offsets, positions, slots = (torch.zeros(n, dtype=torch.int32, device="cuda") for n in (4, 64, 64))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pool.pages.step(new, 64, out=(offsets, positions, slots))
    for i in range(60):
        new.copy_(ints([1, i % 4, 2 if i == 30 else 0]))
        graph.replay()
        *want, missing = pool.ref.step(new.tolist())
        n = want[0][-1]
        assert not missing and offsets.tolist() == want[0]
        assert positions[:n].tolist() == want[1] and slots[:n].tolist() == want[2]
    pool.check(pool.pages)
    assert pool.pages.get_error() == 0


def test_pages_out_of_range(kv8):
    """Counts, lengths and pages that cannot be: cut to range and recorded; nothing out of place is written."""
    from bit_expert_layer_gb300 import _abi

    def run(lens, new, keep, n_tokens, held=None, n_free=None, table=None, borrowed=None):
        p = Pool(kv8, [100, 200, 64], 16, spare=30, width=20, borrowed=borrowed).pages
        for x, v in ((p.lens, lens), (p.held, held), (p.n_free, n_free), (p.table, table)):
            if v is not None:
                x.copy_(ints(v))
        guard = torch.full((3, 400), -9, dtype=torch.int32, device="cuda")
        out = (guard[0, :4], guard[1, :n_tokens], guard[2, :n_tokens])
        p.step(ints(new), n_tokens, None if keep is None else ints(keep), out=out)
        assert p.get_error() == _abi.MOE_ERR_DEVICE_BOUNDS
        assert (guard[0, 4:] == -9).all() and (guard[1:, n_tokens:] == -9).all()
        assert 0 <= p.n_free.item() <= p.free.numel() and (p.lens >= 0).all() and (p.held >= 0).all() and (p.held <= 20).all()
        return p, guard
    big = 2 ** 31 - 1
    run(None, [1, 1, 1], [100, 201, 64], 50)             # keeps more than there is
    run(None, [1, -1, 1], None, 50)
    run(None, [big, big, 1], None, 50)
    run(None, [1, 1, 1], [100, -1, -big - 1], 50)
    run([100, big, 64], [1, 1, 1], None, 50)
    run([-4, 100, 64], [1, 1, 1], None, 50)
    run(None, [1, 1, 1], None, 50, held=[7, big, -2])
    run(None, [1, 1, 1], None, 50, n_free=[big])
    run(None, [300, 1, 1], None, 302)                    # past its row of the table
    p, guard = run(None, [30, 30, 30], None, 50)         # more tokens than rows
    assert guard[0, :4].tolist() == [0, 30, 60, 90]
    t = [[-1] * 20] * 3
    _, guard = run(None, [1, 1, 1], None, 50, table=t)
    assert guard[2, 1].item() == -1
    p = Pool(kv8, [10], 16).pages
    for bad in (dict(new=ints([1, 1])), dict(new=ints([1]), keep=ints([1, 1])), dict(new=ints([1]).long()),
                dict(new=ints([1]), into=Pool(kv8, [10], 16).pages)):
        with pytest.raises(ValueError):
            p.step(n_tokens=1, **bad)
    with pytest.raises(RuntimeError):
        kv8.KV8Pages(p.table, p.free, 48, p.lens, p.held, p.n_free).step(ints([1]), 1)
    with pytest.raises(ValueError):
        kv8.KV8Pages(p.table, p.free, 16, p.lens, ints([1, 2]), p.n_free)
    with pytest.raises(AttributeError):
        p.lens = ints([4])


# ----------------------------------------------------------------------------- all together
@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("layer", ["prefix", "window"])
def test_a_server(kv8, fmt, layer):
    """Two prompts, then answers that share the first one's beginning: page tables, norms with rotary
    positions, cache write and attention, as a server calls them, against the same steps in 64 bits."""
    hq, hkv, d, page, n = 8, 2, 128, 64, 6
    g = gen(70)
    pages = kv8.KV8Pages.all_free(90, page, n, 12)
    cache = kv8.KV8Cache.empty(90, hkv, page, d, fmt)
    wq, wk = ((torch.randn(d, generator=g, device="cuda") * 0.2).to(torch.bfloat16) for _ in range(2))
    rope = kv8.Rope(d, 64, theta=1e4)
    norm = kv8.NormRope(rope, wq, wk, offset=1.0)
    inv = [1e4 ** (-2 * j / 64) for j in range(32)]
    borrowed = torch.zeros(n, dtype=torch.int32, device="cuda")
    pages = kv8.KV8Pages(pages.table, pages.free, page, pages.lens, pages.held, pages.n_free, borrowed)
    ref = kv8_ref.RefCache(cache.k, cache.v, cache.k_scale, cache.v_scale, fmt)
    prefix = None
    for i, new in enumerate([[300, 0, 0, 0, 0, 0], [0, 0, 0, 0, 0, 41]] + [[1] * 6, [3] * 6, [1, 0, 1, 1, 1, 1], [1] * 6]):
        if i == 2:                              # four more sequences begin with the first 4 pages of the first one
            pages.table[1:5, :4] = pages.table[0, :4]
            pages.lens[1:5] = 256
            pages.held[1:5] = 4
            borrowed[1:5] = 4
            prefix = kv8.KV8Prefix(ints([0, 5]), ints([256]), ALWAYS)
        t = sum(new)
        offsets, positions, slots = pages.step(ints(new), t)
        batch = kv8.KV8Batch(pages.table, pages.lens, offsets, max(new))
        qkv = (torch.randn(t, hq + 2 * hkv, d, generator=g, device="cuda") * 3).to(torch.bfloat16)
        q0, k0, v = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
        q, k = norm(q0, k0, positions)
        for got, x, w in ((q, q0, wq), (k, k0, wk)):
            want, bound = serving_ref.norm_rope(x.double(), w, 1e-6, 1.0, positions[None], inv, [0] * 32, 64)
            assert torch.all((got.double() - want).abs() <= bound)
        cache.append(batch, k, v)
        table, lens = pages.table.cpu().numpy(), pages.lens.tolist()
        ref.append(table, lens, offsets.tolist(), k.double(), v.double())
        kw = dict(window=100, sinks=4) if layer == "window" else {}
        out = cache.attention(batch, q, **(kw or dict(prefix=prefix)))
        want, bound = serving_ref.attention(ref, table, lens, offsets.tolist(), q.double(), **kw)
        assert torch.all((out.double() - want).abs() <= bound)
        # a slot is where append has put the token
        at = slots.long()
        kk = cache.k[at // page, :, at % page]
        back, _ = cache.gather(batch, t)
        of = kv8_ref.code_values(fmt).cuda()
        scale = cache.k_scale[at // page, :, at % page // 16].double()
        assert torch.equal(of[kk.long()] * scale[..., None], back.double())
    pages.step(torch.zeros(n, dtype=torch.int32, device="cuda"), 0, keep=torch.zeros(n, dtype=torch.int32, device="cuda"))
    assert pages.n_free.item() == 90 and sorted(pages.free.tolist()) == list(range(90))
    assert cache.get_error() == 0 and pages.get_error() == 0
