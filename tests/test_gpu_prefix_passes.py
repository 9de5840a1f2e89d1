"""The two passes of attention with shared prefixes: that they are taken where a test says so, how they
divide the SMs, and what they leave out.  (Results in general: test_gpu_serving.py.)"""
from __future__ import annotations

import random

import pytest

torch = pytest.importorskip("torch")
import serving_ref  # noqa: E402
from test_gpu_kv8 import ints, kv8  # noqa: E402, F401
from test_gpu_serving import ALWAYS, Shared, check  # noqa: E402

pytestmark = pytest.mark.gpu

MAX_CTAS, TICKET_BYTES = 160, 1024


def workspace(s):
    return s.cache.new_workspace(s.hq, s.batch.max_new, s.t)


def shared(ws):
    """Whether the last call on the workspace shared anything: the last word of the tickets'."""
    return ws[:TICKET_BYTES].view(torch.int32)[-1].item() == 1


def rows_of(g, max_new):
    return 8 if g * max_new <= 8 else 16 if g * max_new <= 32 else 0


def prefix_ctas(s, ws):
    """CTAs that the prefix pass worked with beside a decode pass, from the list of tiles that it leaves: entry c
    {CTAs of the tile that begins in CTA c and goes on, ..., whether c has whole tiles, 0}."""
    rows = rows_of(s.hq // s.hkv, s.batch.max_new)
    at = TICKET_BYTES + MAX_CTAS * 2 * rows * (s.d + 4) * 4
    at = (at + 255) // 256 * 256 + TICKET_BYTES
    tiles = ws[at:at + MAX_CTAS * 32].view(torch.int32).view(MAX_CTAS, 8).tolist()
    return max([c + max(t[0], 1) for c, t in enumerate(tiles) if t[0] or t[6]], default=0)


def best_split(s, groups, share, sms):
    """CTAs of the prefix pass by the definition: those that make the longer of the two passes shortest, by
    the sums over the sequences as they are."""
    g = s.hq // s.hkv
    block = 0
    while (2 << block) * g <= 128:
        block += 1
    mean = (s.batch_tokens - 1) // len(groups) + 1
    shift = block + (mean > 1 << block)
    rows = rows_of(g, s.batch.max_new)
    own = (rows // g).bit_length() - 1
    units = pieces = b = 0
    for n, share_n in zip(groups, share):
        base = share_n // 128 * 128
        tokens = sum(s.new[b:b + n])
        if tokens and base:
            units += -(-tokens // (1 << shift)) * (base // 128 + 4) * s.hkv
        for new, length in list(zip(s.new, s.lens))[b:b + n]:
            if new:
                first = length - new
                rest = first - base if first >= base else first
                pieces += (-(-new // (1 << own))) * ((rest + new + 31) // 32 + 8) * s.hkv
        b += n
    per_unit = 1.3 if g << shift <= 128 else 1.95
    per_piece = 0.18 if g << own <= 8 else 0.27
    at = min(range(1, sms), key=lambda i: max(11 + pieces * per_piece / i, 11 + units * per_unit / (sms - i)))
    return min(sms - at, units)


RAGGED = [("even", [64], [4096], [1] * 64), ("idle", [64], [4096], [0 if i % 8 == 3 else 1 for i in range(64)]),
          ("half-idle", [64], [4096], [i % 2 for i in range(64)]), ("drafts", [13, 11], [4001, 2003], [4 if i % 2 else 1 for i in range(24)]),
          ("one-draft", [48], [4096], [4] + [1] * 47), ("front", [40, 8], [4096, 700], [1] * 48)]


@pytest.mark.parametrize("groups,share,new", [c[1:] for c in RAGGED], ids=[c[0] for c in RAGGED])
def test_the_passes_divide_the_sms_by_the_same_work(kv8, groups, share, new):
    """Idle sequences, drafts of different lengths, new tokens that begin among the shared ones: the prefix pass
    takes the CTAs that the suffix pass leaves it."""
    own = [40 + 13 * (i % 50) for i in range(len(new))]
    s = Shared(kv8, groups, share, own, new, seed=71)
    if len(groups) == 2 and groups[1] == 8:              # these begin before the shared positions end
        s.lens[41:44] = [600, 300, 2]
        s.batch.lens.copy_(ints(s.lens))
    s.batch_tokens = sum(new)
    ws = workspace(s)
    out = s.cache.attention(s.batch, s.q, workspace=ws, prefix=s.prefix)
    check(s, out)
    assert shared(ws) and s.cache.get_error() == 0
    sms = min(torch.cuda.get_device_properties(0).multi_processor_count, MAX_CTAS)
    assert abs(prefix_ctas(s, ws) - best_split(s, groups, share, sms)) <= 1


def run(s, prefix=None, **kw):
    """The call on a fresh workspace; it has to share."""
    ws = workspace(s)
    out = s.cache.attention(s.batch, s.q, workspace=ws, prefix=prefix or s.prefix, **kw)
    assert shared(ws)
    return out


def check_some(s, out, rng, n=60):
    """check(), for some of the sequences: the reference takes milliseconds for each."""
    pick = set(rng.sample(range(len(s.lens)), n))
    rows = [r for b in sorted(pick) for r in range(int(s.offsets[b]), int(s.offsets[b + 1]))]
    want, bound = serving_ref.attention(s.ref(), s.table, [m if b in pick else 0 for b, m in enumerate(s.lens)], s.offsets,
                                        s.q[:int(s.offsets[-1])].double())
    assert rows and torch.all((out[rows].double() - want[rows]).abs() <= bound[rows])


def sizes(n, parts, rng):
    """`parts` group sizes of n sequences, empty ones among them."""
    cut = sorted(rng.choices(range(n + 1), k=parts - 1))
    return [b - a for a, b in zip([0] + cut, cut + [n])]


@pytest.mark.parametrize("parts,new", [(340, 2), (700, 3)], ids=["decode", "prompt"])
def test_hundreds_of_groups(kv8, parts, new):
    """1024 sequences in about as many groups as it pays for, of none to some sequences, some that share nothing, the
    last ones empty."""
    rng = random.Random(parts)
    groups = sizes(1024, parts - 20, rng) + [0] * 20
    share = [rng.choice([0, 100, 128, 260, 300]) for _ in groups]
    fresh = [0 if i % 13 == 5 else new - (i % 5 == 2) for i in range(1024)]
    s = Shared(kv8, groups, share, [new + i % 40 for i in range(1024)], fresh, (16, 1, 64), 16, seed=parts, pad=3)
    out = torch.full(s.q.shape, 5.0, dtype=torch.bfloat16, device="cuda")
    run(s, out=out)
    check_some(s, out, rng, 200)
    assert (out[int(s.offsets[-1]):] == 5).all() and s.cache.get_error() == 0


@pytest.mark.parametrize("bound", [127, 128, 300, 511, 513])
def test_a_bound_below_what_is_shared(kv8, bound):
    """Positions past the bound are each sequence's own; never a position twice, none lost."""
    s = Shared(kv8, [1000], [512], [20 + i % 50 for i in range(1000)], [2] * 1000, (32, 2, 64), seed=74)
    check_some(s, run(s, kv8.KV8Prefix(ints([0, 1000]), ints([512]), bound)), random.Random(bound))
    assert s.cache.get_error() == 0


@pytest.mark.parametrize("new", [1, 2, 4, 40])
@pytest.mark.parametrize("at", [0, 3, 31])
def test_a_missing_shared_page_is_missing_for_the_group(kv8, at, new):
    """The first sequence's row is the one that is read: a page out of range there is left out for all, one in
    another sequence's row for none."""
    from bit_expert_layer_gb300 import _abi
    s = Shared(kv8, [6, 5], [512, 256], [100 + i for i in range(11)], [new] * 11, page=16, seed=75)
    good = run(s)
    check(s, good)
    for row, bad in ((0, s.n_pages), (0, -1), (2, -1)):
        t = s.table.copy()
        t[row, at] = bad
        s.batch.page_table.copy_(ints(t))
        out = run(s)
        if row:
            assert torch.equal(out, good) and s.cache.get_error() == 0
            continue
        assert s.cache.get_error() == _abi.MOE_ERR_DEVICE_BOUNDS
        # the same without the page: it holds 16 positions that every token sees
        less, lens = s.table.copy(), list(s.lens)
        for b in range(6):
            less[b, at:-1] = s.table[b, at + 1:]
            lens[b] -= 16
        check(s, out, lens=lens, table=less)
        assert torch.equal(out[6 * new:], good[6 * new:])


@pytest.mark.parametrize("new", [1, 2, 4, 40])
def test_a_missing_own_page_is_missing_for_its_sequence(kv8, new):
    from bit_expert_layer_gb300 import _abi
    s = Shared(kv8, [6], [512], [100 + i for i in range(6)], [new] * 6, page=16, seed=76)
    good = run(s)
    for b, at in ((0, 32), (3, 34)):
        t = s.table.copy()
        t[b, at] = 2 ** 31 - 1
        s.batch.page_table.copy_(ints(t))
        out = run(s)
        assert s.cache.get_error() == _abi.MOE_ERR_DEVICE_BOUNDS
        less, lens = s.table.copy(), list(s.lens)
        less[b, at:-1] = s.table[b, at + 1:]
        lens[b] -= 16
        check(s, out, lens=lens, table=less)
        rest = [i for i in range(6 * new) if i // new != b]
        assert torch.equal(out[rest], good[rest])


@pytest.mark.parametrize("new", [1, 40])
def test_rows_that_see_nothing(kv8, new):
    """All pages out of range, shared and own: zeros."""
    s = Shared(kv8, [6], [512], [100] * 6, [new] * 6, page=64, seed=77)
    s.batch.page_table.fill_(-1)
    assert (run(s) == 0).all() and s.cache.get_error() != 0
