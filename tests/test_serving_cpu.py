"""Window and prefix attention, head norms with rotary positions and page tables without a GPU:
every refusal of their entry points (host checks return before anything reaches the device), and
the index arithmetic that the kernels use, restated and compared with brute force."""
import math
import random

import pytest

from bit_expert_layer_gb300 import _abi
from bit_expert_layer_gb300.build import build

pytest.importorskip("torch")
import serving_ref  # noqa: E402
from test_kv8_cpu import BAD_BATCH, BAD_CACHE, FAKE, _before, batch, cache  # noqa: E402

A, I, U, W = 3, 1, 2, 7
FAR, BIG = FAKE << 4, 1 << 40


@pytest.fixture(scope="module")
def lib():
    build()
    return _abi.lib()


def prefix(**kw):
    a = dict(groups=FAKE, shared=FAKE, n_groups=1, max_shared=0)
    a.update(kw)
    return _abi.GqaKv8Prefix(*a.values())


# ----------------------------------------------------------------------------- refusals
@pytest.mark.parametrize("which", ["window", "prefix"])
def test_refused_caches_batches_and_rows(lib, which):
    def call(c, b, q=FAKE, qs=2048, hq=16, scale=0.0, out=FAR, ws=FAKE, n=BIG):
        if which == "window":
            return lib.gqa_kv8_window_attention(c, b, q, qs, hq, scale, 64, 4, out, ws, n, None)
        return lib.gqa_kv8_prefix_attention(c, b, prefix(), q, qs, hq, scale, out, ws, n, None)
    assert call(None, batch()) == I and call(cache(), None) == I
    for kw, st in BAD_CACHE:
        assert call(cache(**kw), batch()) == st, kw
    for kw, st in BAD_BATCH:
        assert call(cache(), batch(**kw)) == st, kw
    assert call(cache(), batch(n_tokens=0)) == 0
    ws = lib.gqa_kv8_workspace_bytes(cache(), 16, 1) if which == "window" else \
        lib.gqa_kv8_prefix_workspace_bytes(cache(), 16, 1, 2)
    for kw, st in [(dict(q=None), I), (dict(out=None), I), (dict(ws=None), I), (dict(hq=0), I), (dict(hq=15), U),
                   (dict(hq=34, qs=4352), U), (dict(qs=2040), I), (dict(qs=2052), A), (dict(q=FAKE + 8), A),
                   (dict(out=FAR + 2), A), (dict(ws=FAKE + 128), A), (dict(scale=-1.0), I), (dict(scale=math.nan), I),
                   (dict(out=FAKE), I), (dict(out=FAKE + 4096), I), (dict(n=ws - 1), W)]:
        assert call(cache(), batch(), **kw) == st, kw


def test_refused_windows(lib):
    for window, sinks in [(0, 4), (-1, 4), ((1 << 24) + 1, 0), (64, -1), (64, (1 << 24) + 1)]:
        assert lib.gqa_kv8_window_attention(cache(), batch(), FAKE, 2048, 16, 0.0, window, sinks, FAR, FAKE, BIG, None) == I


def test_refused_prefixes(lib):
    for kw, st in [(dict(groups=None), I), (dict(shared=None), I), (dict(n_groups=0), I), (dict(n_groups=1025), I),
                   (dict(max_shared=-1), I), (dict(max_shared=(1 << 24) + 1), I), (dict(groups=FAKE + 2), A), (dict(shared=FAKE + 1), A)]:
        assert lib.gqa_kv8_prefix_attention(cache(), batch(), prefix(**kw), FAKE, 2048, 16, 0.0, FAR, FAKE, BIG, None) == st
    assert lib.gqa_kv8_prefix_attention(cache(), batch(), None, FAKE, 2048, 16, 0.0, FAR, FAKE, BIG, None) == I


def test_prefix_workspace_bytes(lib):
    w = lib.gqa_kv8_prefix_workspace_bytes
    assert w(None, 16, 1, 4) == 0 and w(cache(), 15, 1, 4) == 0 and w(cache(), 16, 0, 4) == 0 and w(cache(), 16, 1, 0) == 0
    assert w(cache(), 16, 1, (1 << 20) + 1) == 0
    # a row of sums (for few new tokens two) per token and query head, past the 2^32 bytes of an ordinary size
    for m in (1, 4, 5, 4096):
        assert w(cache(), 16, m, 1) >= lib.gqa_kv8_workspace_bytes(cache(), 16, m) + 16 * 136 * 4
    assert w(cache(), 16, 1, 1 << 20) - w(cache(), 16, 1, 1) == ((1 << 20) - 1) * 16 * 136 * 4 * 2
    # what is enough for many new tokens is enough for few, and for fewer rows
    for t in (1, 100, 5000, 1 << 20):
        sizes = [w(cache(), 16, m, t) for m in (1, 2, 4, 5, 4096)]
        assert sizes == sorted(sizes) and sizes[0] > w(cache(), 16, 1, t - 1)


def test_refused_norms(lib):
    plan = _abi.gqa_rope_plan_init(128, 128, 1e4)
    rows = (FAKE, 256, 2, FAKE, 128, 1, FAKE, 4, FAKE << 4, 256, FAKE << 5, 128, None)
    for a, st in [((FAKE, FAKE, 0, -1e-6, 0.0), I), ((FAKE, FAKE, 0, math.nan, 0.0), I), ((FAKE, FAKE, 0, math.inf, 0.0), I),
                  ((FAKE, FAKE, 0, 0.0, math.nan), I), ((FAKE, FAKE, 0, 0.0, math.inf), I), ((FAKE + 1, FAKE, 0, 0.0, 0.0), A),
                  ((FAKE, FAKE + 2, 1, 0.0, 0.0), A)]:
        assert lib.gqa_norm_rope(plan, _abi.GqaNorm(*a), *rows) == st, a
    good = _abi.GqaNorm(FAKE, None, 0, 1e-6, 1.0)
    assert lib.gqa_norm_rope(plan, None, *rows) == I and lib.gqa_norm_rope(None, good, *rows) == I
    assert lib.gqa_norm_rope(plan, good, None, *rows[1:]) == I
    assert lib.gqa_norm_rope(plan, good, FAKE + 8, *rows[1:]) == A
    assert lib.gqa_norm_rope(plan, good, *rows[:7], 0, *rows[8:]) == 0


def test_refused_pages(lib):
    def call(pages=None, state=None, to=None, keep=FAKE, new=FAKE, borrowed=None, offsets=FAKE, positions=FAKE, slots=FAKE,
             n_tokens=8):
        p = dict(page_table=FAKE, free_pages=FAKE, control=FAKE, n_seqs=2, max_pages=4, n_pages=8, page_size=64)
        p.update(pages or {})
        s, t = (dict(dict(lens=FAKE, held=FAKE, n_free=FAKE), **(x or {})) for x in (state, to))
        return lib.gqa_kv8_pages_step(_abi.GqaKv8Pages(*p.values()), _abi.GqaKv8PagesState(*s.values()),
                                      _abi.GqaKv8PagesState(*t.values()), keep, new, borrowed, offsets, positions, slots,
                                      n_tokens, None)
    for kw in ([dict(pages={n: None}) for n in ("page_table", "free_pages", "control")] +
               [dict(**{w: {n: None}}) for w in ("state", "to") for n in ("lens", "held", "n_free")] +
               [dict(new=None), dict(offsets=None), dict(n_tokens=-1), dict(n_tokens=(1 << 20) + 1)] +
               [dict(pages=x) for x in (dict(n_seqs=0), dict(n_seqs=1025), dict(max_pages=0), dict(n_pages=0), dict(page_size=8),
                                        dict(page_size=48), dict(page_size=2048), dict(max_pages=(1 << 18) + 1),
                                        dict(n_pages=1 << 25))]):
        assert call(**kw) == I, kw
    for kw in ([dict(pages={n: FAKE + 2}) for n in ("page_table", "free_pages", "control")] +
               [dict(**{w: {n: FAKE + 1}}) for w in ("state", "to") for n in ("lens", "held", "n_free")] +
               [{n: FAKE + 2} for n in ("keep", "new", "borrowed", "offsets", "positions", "slots")]):
        assert call(**kw) == A, kw
    assert lib.gqa_kv8_pages_step(None, None, None, None, FAKE, None, FAKE, None, None, 0, None) == I
    assert lib.gqa_kv8_pages_get_error(None) == I and lib.gqa_kv8_pages_get_error(_abi.GqaKv8Pages()) == I


# ----------------------------------------------------------------------------- the reference itself
def test_reference_of_page_tables():
    p = serving_ref.Pages([[5, 6, 9], [7, 9, 9]], [0, 1, 2, 9, 9], 3, [20, 10], [2, 1], 16)
    # sequence 0 falls back to 3 positions and gives page 6 back; sequence 1 takes it, then page 2
    assert p.step([1, 30], [3, 10]) == ([0, 1, 31], [3] + list(range(10, 40)),
                                        [5 * 16 + 3] + [7 * 16 + i for i in range(10, 16)] +
                                        [6 * 16 + i for i in range(16)] + [2 * 16 + i for i in range(8)], False)
    assert p.table == [[5, 6, 9], [7, 6, 2]] and p.held == [1, 3] and p.lens == [4, 40] and p.n_free == 2
    assert p.step([0, 0], [0, 40])[0] == [0, 0, 0] and p.free[:3] == [0, 1, 5] and p.n_free == 3 and p.held == [0, 3]


# ----------------------------------------------------------------------------- the window's line of units
def window_tile(first, n, tq, t, U, window, sinks):
    """(units of the line but C, positions of each unit's places or None) of a tile, as the kernels count them."""
    g = 16 if U == 128 else U
    K = -(-((window + tq - 1 + 2 * g - 2) // g + -(-sinks // g)) * g // U)
    end = max(first + min((t + 1) * tq, n), 0)
    line = min(-(-(max(first, 0) + min((t + 1) * tq, n)) // U), K)
    low = max(first + t * tq + 1 - window, 0)
    sunk = min(-(-sinks // g), low // g) * g
    skip = low // g * g - sunk
    units = max(-(-(end - skip) // U), 1)
    at = [i + (0 if i < sunk else skip) for i in range(units * U)]
    return line, [[p if p < end else None for p in at[u * U:(u + 1) * U]] for u in range(units)]


def test_window_units():
    """A tile's units hold the positions that its tokens see, each once and in order, in whole granules that
    each hold one; the masks, which are made from a unit's place in the row, are the definition's; and
    the line's closed form for the tiles before one is the sum over them."""
    rng = random.Random(5)
    for _ in range(1200):
        U = rng.choice([32, 128])
        g = 16 if U == 128 else U
        tq = rng.choice([1, 2, 4, 8, 16, 32] + ([64, 128, 256] if U == 128 else []))
        first = rng.choice([0, rng.randint(0, 1500), -rng.randint(0, 40)])
        n = rng.choice([1, rng.randint(1, 90), rng.randint(100, 400)])
        window = rng.choice([1, 2, 16, 31, 32, 33, 128, rng.randint(1, 2000), 1 << 24])
        sinks = rng.choice([0, 0, 1, 4, 16, 17, 128, rng.randint(0, 400), 1 << 24])
        K = -(-((window + tq - 1 + 2 * g - 2) // g + -(-sinks // g)) * g // U)
        C, total = 2, 0
        for t in range(-(-n // tq)):
            full = max(((K - 1) * U - max(first, 0)) // tq, 0)
            done = min(t, full)
            assert _before(first, U, C, tq, done) + (t - done) * (K + C) == total
            line, units = window_tile(first, n, tq, t, U, window, sinks)
            total += line + C
            assert len(units) <= line
            held = [p for u in units for p in u if p is not None]
            assert held == sorted(set(held))
            last = max(first + min((t + 1) * tq, n), 0)
            low = max(first + t * tq + 1 - window, 0)
            skip = low // g * g - min(-(-sinks // g), low // g) * g
            tokens = [p for p in (first + t * tq, first + min((t + 1) * tq, n) - 1) if p >= 0]
            seen = set()
            for p in tokens:
                mine = set(range(max(0, p + 1 - window), p + 1)) | set(range(min(sinks, p + 1)))
                seen |= mine
                assert mine <= set(held)
                if U == 128:                 # the prompt kernel's masks
                    for u, places in enumerate(units):
                        left = p + 1 - skip - u * U
                        before, under = left - window, sinks - u * U
                        got = {x for i, x in enumerate(places) if i < left and (i >= before or i < under)}
                        assert got == mine & {x for x in places if x is not None}
            if len(tokens) == 2 and tokens[0] >= 0:
                seen |= set(range(max(0, low), last))
                assert {x // g for x in held} == {x // g for x in seen}


def test_a_run_that_holds_none_of_a_windows_units():
    """The line counts a tile's units by a bound; a run in what the tile has less than that works on
    nothing and owns no part, and the others cover the tile."""
    rng = random.Random(6)
    for _ in range(2000):
        U, C, tq = 32, 2, rng.choice([1, 2])
        tiles = []
        for b in range(rng.randint(1, 5)):
            first, n = rng.randint(0, 900), rng.choice([1, 1, 2, 8])
            window, sinks = rng.randint(1, 500), rng.choice([0, 4, 40])
            tiles += [window_tile(first, n, tq, t, U, window, sinks) for t in range(-(-n // tq))]
        total = sum(line + C for line, _ in tiles)
        runs = min(total, rng.choice([1, 7, 40, 152 * 8]))
        begin = [i * total // runs for i in range(runs + 1)]
        run_of = lambda w: ((w + 1) * runs - 1) // total  # noqa: E731
        start = 0
        for line, units in tiles:
            n, done = len(units), 0
            first, last = run_of(start + C), run_of(start + C + n - 1)
            for i in range(run_of(start), run_of(start + line + C - 1) + 1):
                x = max(begin[i] - start, 0)
                end = min(begin[i + 1] - start, line + C)
                u0, u1 = max(x - C, 0), min(end - C, n)
                if u1 > u0:
                    assert u0 == done and first <= i <= last
                    done = u1
                else:
                    assert i < first or i > last
            assert done == n
            start += line + C


@pytest.mark.parametrize("U,per_cta", [(32, 8), (128, 1)])
def test_runs_that_hold_whole_tiles(U, per_cta):
    """A line whose tiles all count as long as the longest, cut so that a CTA has whole tiles: the runs
    cover the line, none is empty, every tile's units lie in one CTA, each once and in order, and the
    runs between its first and its last one hold some of it."""
    rng = random.Random(7)
    C = 2
    for _ in range(3000):
        tiles = [rng.choice([1, 1, 2, 5, rng.randint(1, 60)]) for _ in range(rng.choice([1, 3, 20, 400]))]
        grid = rng.choice([1, 7, 152])
        waves = -(-len(tiles) // grid)
        longest = max(max(tiles) + C, per_cta)
        ctas = -(-len(tiles) // waves)
        n, span, total = ctas * per_cta, ctas * waves * longest, len(tiles) * longest
        assert ctas <= grid
        begin = [min(i * span // n, total) for i in range(n + 1)]
        assert begin[0] == 0 and begin[n] == total
        run_of = lambda w: ((w + 1) * n - 1) // span  # noqa: E731
        assert all(begin[i] < begin[i + 1] or begin[i] == total for i in range(n))
        for t, units in enumerate(tiles):
            start, done = t * longest, 0
            first, last = run_of(start + C), run_of(start + C + units - 1)
            assert first // per_cta == last // per_cta == t // waves
            for i in range(first, last + 1):
                u0, u1 = max(begin[i] - start - C, 0), min(begin[i + 1] - start - C, units)
                assert u0 == done and u1 > u0
                done = u1
            assert done == units


def test_step_numbers():
    """The norm kernel's division of a step's number by a token's steps, by a multiplication: up to 32
    tokens of up to 128 steps."""
    for per in range(1, 129):
        inv = ((1 << 21) + per - 1) // per
        assert 32 * per * inv < 1 << 32
        assert all(i * inv >> 21 == i // per for i in range(32 * per))
