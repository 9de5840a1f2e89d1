"""The 8-bit key/value cache without a GPU: every refusal of its entry points (host checks
return before anything reaches the device), rotary plans, the 64-bit reference's own
rounding, and the index arithmetic that the kernels use, restated and compared with brute
force: the map of 16-position blocks to work units and the line of attention units."""
import ctypes as C
import math
import random

import pytest

from bit_expert_layer_gb300 import _abi
from bit_expert_layer_gb300.build import build

torch = pytest.importorskip("torch")
import kv8_ref  # noqa: E402

FAKE = 1 << 20       # never dereferenced: every call below fails a host check first


@pytest.fixture(scope="module")
def lib():
    build()
    return _abi.lib()


def cache(**kw):
    a = dict(k_codes=FAKE, v_codes=FAKE, k_scales=FAKE, v_scales=FAKE, error=FAKE, n_pages=8, page_size=64,
             n_kv_heads=2, head_size=128, format=0)
    a.update(kw)
    return _abi.GqaKv8Cache(*a.values())


def batch(**kw):
    a = dict(page_table=FAKE, lens=FAKE, offsets=FAKE, n_seqs=2, max_pages=4, n_tokens=2, max_new=1)
    a.update(kw)
    return _abi.GqaKv8Batch(*a.values())


BAD_CACHE = [(dict(k_codes=None), 1), (dict(v_codes=None), 1), (dict(k_scales=None), 1), (dict(v_scales=None), 1),
             (dict(error=None), 1), (dict(n_pages=0), 1), (dict(page_size=8), 1), (dict(page_size=48), 1),
             (dict(page_size=2048), 1), (dict(n_kv_heads=0), 1), (dict(n_kv_heads=65), 1), (dict(head_size=96), 1),
             (dict(head_size=256), 1), (dict(format=2), 1), (dict(format=-1), 1),
             (dict(n_pages=1 << 24, n_kv_heads=2, page_size=64), 1),       # 2^31 rows
             (dict(k_codes=FAKE + 8), 3), (dict(v_codes=FAKE + 4), 3), (dict(k_scales=FAKE + 2), 3),
             (dict(error=FAKE + 1), 3)]
BAD_BATCH = [(dict(page_table=None), 1), (dict(lens=None), 1), (dict(offsets=None), 1), (dict(n_seqs=0), 1),
             (dict(n_seqs=1025), 1), (dict(max_pages=0), 1), (dict(max_pages=1 << 19), 1), (dict(n_tokens=-1), 1),
             (dict(n_tokens=(1 << 20) + 1), 1), (dict(max_new=0), 1), (dict(max_new=(1 << 20) + 1), 1),
             (dict(lens=FAKE + 2), 3)]


def calls(lib):
    return [lambda c, b: lib.gqa_kv8_append(c, b, FAKE, 256, FAKE, 256, None),
            lambda c, b: lib.gqa_kv8_gather(c, b, FAKE, FAKE, None),
            lambda c, b: lib.gqa_kv8_attention(c, b, FAKE, 2048, 16, 0.0, FAKE << 4, FAKE, 1 << 40, None)]


@pytest.mark.parametrize("which", range(3), ids=["append", "gather", "attention"])
def test_refused_caches_and_batches(lib, which):
    call = calls(lib)[which]
    assert call(None, batch()) == _abi.MOE_ERR_INVALID_ARG
    assert call(cache(), None) == _abi.MOE_ERR_INVALID_ARG
    for kw, st in BAD_CACHE:
        assert call(cache(**kw), batch()) == st, kw
    for kw, st in BAD_BATCH:
        assert call(cache(), batch(**kw)) == st, kw
    assert call(cache(), batch(n_tokens=0)) == _abi.MOE_OK      # nothing to do, nothing launched


def test_refused_rows(lib):
    c, b = cache(), batch()
    A, I = _abi.MOE_ERR_ALIGNMENT, _abi.MOE_ERR_INVALID_ARG
    for args, st in [((None, 256, FAKE, 256), I), ((FAKE, 256, None, 256), I), ((FAKE, 248, FAKE, 256), I),
                     ((FAKE, 256, FAKE, 0), I), ((FAKE, -256, FAKE, 256), I), ((FAKE, 260, FAKE, 256), A),
                     ((FAKE + 8, 256, FAKE, 256), A), ((FAKE, 256, FAKE + 2, 256), A), ((FAKE, 1 << 41, FAKE, 256), I)]:
        assert lib.gqa_kv8_append(c, b, *args, None) == st, args
    for args, st in [((None, FAKE), I), ((FAKE, None), I), ((FAKE + 8, FAKE), A), ((FAKE, FAKE + 2), A)]:
        assert lib.gqa_kv8_gather(c, b, *args, None) == st, args


def test_refused_attention(lib):
    c, b = cache(), batch()
    far, big = FAKE << 4, 1 << 40
    A, I, U, W = 3, 1, 2, 7
    ws = lib.gqa_kv8_workspace_bytes(c, 16, 1)
    assert ws > 0
    for args, st in [((None, 2048, 16, 0.0, far, FAKE, big), I), ((FAKE, 2048, 16, 0.0, None, FAKE, big), I),
                     ((FAKE, 2048, 16, 0.0, far, None, big), I), ((FAKE, 2048, 0, 0.0, far, FAKE, big), I),
                     ((FAKE, 2048, 15, 0.0, far, FAKE, big), U), ((FAKE, 4352, 34, 0.0, far, FAKE, big), U),
                     ((FAKE, 2040, 16, 0.0, far, FAKE, big), I), ((FAKE, 2052, 16, 0.0, far, FAKE, big), A),
                     ((FAKE + 8, 2048, 16, 0.0, far, FAKE, big), A), ((FAKE, 2048, 16, 0.0, far + 2, FAKE, big), A),
                     ((FAKE, 2048, 16, 0.0, far, FAKE + 128, big), A), ((FAKE, 2048, 16, -1.0, far, FAKE, big), I),
                     ((FAKE, 2048, 16, math.nan, far, FAKE, big), I), ((FAKE, 2048, 16, math.inf, far, FAKE, big), I),
                     ((FAKE, 2048, 16, 0.0, FAKE, FAKE, big), I),             # out on q
                     ((FAKE, 2048, 16, 0.0, FAKE + 4096, FAKE, big), I),      # out on q's second row
                     ((FAKE, 2048, 16, 0.0, far, FAKE, ws - 1), W)]:
        assert lib.gqa_kv8_attention(c, b, *args, None) == st, args


def test_workspace_bytes(lib):
    w = lib.gqa_kv8_workspace_bytes
    assert w(None, 16, 1) == 0 and w(cache(), 0, 1) == 0 and w(cache(), 15, 1) == 0 and w(cache(), 34, 1) == 0
    assert w(cache(), 16, 0) == 0 and w(cache(), 16, 1 << 21) == 0 and w(cache(head_size=96), 16, 1) == 0
    assert 0 < w(cache(), 16, 1) <= w(cache(), 16, 2) <= w(cache(), 16, 4096)


def test_get_error_refuses(lib):
    assert lib.gqa_kv8_get_error(None) == _abi.MOE_ERR_INVALID_ARG
    assert lib.gqa_kv8_get_error(cache(error=None)) == _abi.MOE_ERR_INVALID_ARG
    assert _abi.moe_status_string(_abi.MOE_ERR_NONFINITE) == "value that is not finite"


# ----------------------------------------------------------------------------- rotary plans
def test_rope_plan(lib):
    for bad, st in [(dict(head_size=96), 2), (dict(rotary=8), 1), (dict(rotary=24), 1), (dict(rotary=144), 1),
                    (dict(theta=0.0), 1), (dict(theta=math.nan), 1), (dict(sections=[30, 30]), 1),
                    (dict(sections=[65, -1]), 1), (dict(sections=[16] * 5), 1), (dict(inv_freq=[math.inf] * 64), 1)]:
        a = dict(head_size=128, rotary=128, theta=1e4)
        a.update(bad)
        with pytest.raises(_abi.MoEError) as e:
            _abi.gqa_rope_plan_init(**a)
        assert e.value.status == st, bad
    with pytest.raises(ValueError):
        _abi.gqa_rope_plan_init(128, 128, 1e4, inv_freq=[1.0] * 63)
    # two axes without their sections
    assert lib.gqa_rope_plan_init(_abi.GqaRopePlan(), 128, 128, 1e4, None, None, 2, 0) == 1
    assert lib.gqa_rope_plan_init(None, 128, 128, 1e4, None, None, 1, 0) == 1
    p = _abi.gqa_rope_plan_init(128, 64, 1e7, sections=[12, 10, 10], cyclic=True)
    assert list(p.axis)[:32] == [0, 1, 2] * 10 + [0, 0]
    p = _abi.gqa_rope_plan_init(128, 64, 1e7, sections=[12, 0, 20])
    assert list(p.axis)[:32] == [0] * 12 + [2] * 20
    for j in range(32):
        want = (1e7 ** (-2 * j / 64)) / (2 * math.pi)
        assert abs(p.turn[j] / 2.0 ** 64 - want) <= 2.0 ** -52 * want + 2.0 ** -63
    p = _abi.gqa_rope_plan_init(128, 16, 0.0, inv_freq=[2 * math.pi * x for x in (0, 0.25, 1.25, -0.25, 7, 0.5, 1, 3)])
    for got, want in zip(list(p.turn)[:8], (0, 0.25, 0.25, 0.75, 0, 0.5, 0, 0)):
        d = abs(got / 2.0 ** 64 - want)
        assert min(d, 1 - d) < 1e-14


def test_refused_rope(lib):
    plan = _abi.gqa_rope_plan_init(128, 128, 1e4)
    ok = dict(q=FAKE, qs=256, nq=2, k=FAKE, ks=128, nk=1, pos=FAKE, T=4, qo=FAKE << 4, qos=256, ko=FAKE << 5, kos=128)
    A, I = 3, 1
    for bad, st in [(dict(q=None), I), (dict(qo=None), I), (dict(k=None), I), (dict(ko=None), I), (dict(pos=None), I),
                    (dict(nq=0), I), (dict(nq=257), I), (dict(nk=-1), I), (dict(T=-1), I), (dict(T=(1 << 20) + 1), I),
                    (dict(qs=248), I), (dict(qs=260), A), (dict(ks=120), I), (dict(qos=8), I), (dict(kos=132), A),
                    (dict(q=FAKE + 8), A), (dict(ko=FAKE + 2), A), (dict(pos=FAKE + 2), A),
                    (dict(qo=FAKE, qos=512), I), (dict(T=0), 0)]:
        a = dict(ok)
        a.update(bad)
        assert lib.gqa_rope(plan, *a.values(), None) == st, bad
    assert lib.gqa_rope(None, *ok.values(), None) == I
    assert lib.gqa_rope(_abi.GqaRopePlan(), *ok.values(), None) == I          # never filled
    plan.axis[3] = 1
    assert lib.gqa_rope(plan, *ok.values(), None) == I                        # an axis that it does not have


# ----------------------------------------------------------------------------- the reference itself
@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_reference_rounding(fmt):
    """Every representable number is its own code; a midpoint goes to the even code."""
    val = kv8_ref.code_values(fmt)
    fine = torch.isfinite(val) & ~((torch.arange(256) == 128) if fmt == "int8" else torch.zeros(256, dtype=torch.bool))
    codes = torch.arange(256)[fine]
    assert torch.equal(kv8_ref.nearest_code(val[fine], fmt), codes)
    if fmt == "e4m3":
        assert torch.equal(val[fine].float(), codes.to(torch.uint8).view(torch.float8_e4m3fn).float())
        y = torch.linspace(-448, 448, 100003, dtype=torch.float64)
        want = y.to(torch.float32).to(torch.float8_e4m3fn).view(torch.uint8).long()
        same = y.to(torch.float32).double() == y
        assert torch.equal(kv8_ref.nearest_code(y[same], fmt), want[same])
    mid = (val[:126] + val[1:127]) / 2
    got = kv8_ref.nearest_code(mid, fmt)
    assert torch.all(got % 2 == 0)
    for amax, e in [(448.0, 0), (448.0 * 2 ** 9, 9), (450.0, 1), (1.0, -8), (0.0, -100), (1e-38, -100)] \
            if fmt == "e4m3" else [(127.0, 0), (127.5, 1), (64.0, 0), (63.5, -1), (63.75, 0), (0.0, -100)]:
        assert kv8_ref.scale_exp(amax, fmt) == e, amax


# ----------------------------------------------------------------------------- the kernels' index arithmetic
def test_block_units_do_not_meet():
    """Sequence b owns units offsets[b] / 16 + 2 b and up; whatever the lengths are, its
    blocks fit before the next sequence's and n_tokens / 16 + 2 n_seqs units cover all."""
    rng = random.Random(1)
    for _ in range(3000):
        B = rng.randint(1, 12)
        new = [rng.choice([0, 1, 1, 2, 15, 16, 17, 31, 33, rng.randint(0, 200)]) for _ in range(B)]
        off = [0]
        for n in new:
            off.append(off[-1] + n)
        units = off[-1] // 16 + 2 * B
        taken = set()
        for b, n in enumerate(new):
            first = rng.randint(0, 100)
            blocks = (first + n - 1) // 16 - first // 16 + 1 if n else 0
            for j in range(blocks):
                u = off[b] // 16 + 2 * b + j
                assert u < units and u not in taken
                taken.add(u)
                # the kernel's search: the last sequence whose first unit is at or before u
                assert max(s for s in range(B) if off[s] // 16 + 2 * s <= u) == b


def _before(first, U, C, tq, t):
    """Units of a sequence's tiles 0 .. t - 1, in closed form."""
    if tq > U:
        return t * (-(-max(first, 0) // U) + C) + tq // U * t * (t + 1) // 2
    r = U // tq
    F = lambda X: r * (X // r) * (X // r - 1) // 2 + (X // r) * (X % r + 1)  # noqa: E731
    A = (max(first, 0) + U - 1) // tq
    return F(A + t) - F(A) + C * t


@pytest.mark.parametrize("U,C,per_cta", [(32, 2, 8), (128, 2, 1), (32, 0, 8)])
def test_line_of_units(U, C, per_cta):
    """The closed form of a sequence's units against a sum over its tiles.  And a line cut into
    runs: every run's segments cover each tile's units of positions once, in order; a run
    holds at most one tile that began before it and one that goes on after it; a CTA's runs
    share a ticket and two workspace slots with other CTAs without conflict."""
    rng = random.Random(2)
    for _ in range(1500):
        tq = rng.choice([1, 2, 4, 8, 16, 32] + ([64, 128, 256] if U == 128 else []))
        hkv = rng.randint(1, 3)
        seqs = [(rng.choice([0, rng.randint(0, 700)]), rng.choice([1, 1, rng.randint(1, 90), rng.randint(200, 900)]))
                for _ in range(rng.randint(1, 6))]
        tiles = []                                   # (name, units of positions)
        for b, (first, n) in enumerate(seqs):
            nt = -(-n // tq)
            per = [-(-(first + min((t + 1) * tq, n)) // U) for t in range(nt)]
            for t in range(nt):
                assert _before(first, U, C, tq, t) == sum(per[:t]) + C * t
            for g in range(hkv):
                tiles += [((b, g, t), per[t]) for t in range(nt)]
        total = sum(n + C for _, n in tiles)
        ctas = rng.choice([1, 3, 16, 152])
        runs = min(total, ctas * per_cta)
        run_of = lambda w: ((w + 1) * runs - 1) // total  # noqa: E731
        begin = [i * total // runs for i in range(runs + 1)]
        assert all(run_of(w) == i for i in range(runs) for w in (begin[i], begin[i + 1] - 1))
        start, seen, slots, tickets = 0, {}, set(), {}
        for name, n in tiles:
            first, last = run_of(start + C), run_of(start + C + n - 1)
            done = 0
            for i in range(first, last + 1):
                u0 = max(begin[i] - start - C, 0)
                u1 = min(begin[i + 1] - start - C, n)
                assert u0 == done and u1 > u0            # a run between holds some of the tile
                done = u1
                if u0 > 0:
                    assert seen.setdefault((i, "began before"), name) == name
                elif u1 < n:
                    assert seen.setdefault((i, "goes on"), name) == name
            assert done == n
            c0, c1 = first // per_cta, last // per_cta
            if c0 != c1:
                assert tickets.setdefault(c0, name) == name       # a ticket serves one tile
                for c in range(c0, c1 + 1):
                    slot = (c, 1 if c == c0 else 0)
                    assert slot not in slots
                    slots.add(slot)
            start += n + C
