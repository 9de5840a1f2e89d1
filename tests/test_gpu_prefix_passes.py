"""The two passes of attention with shared prefixes: that they are taken where a test says so, how they
divide the SMs, and what they leave out.  (Results in general: test_gpu_serving.py.)"""
from __future__ import annotations

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
