"""The 8-bit key/value cache and rotary positions on the GPU against the 64-bit reference
(tests/kv8_ref.py).  Cache write and read back are exact (scales are powers of two, codes are
nearest numbers), so they are compared for equality; attention and rotary positions are held
to bounds derived from the kernels' arithmetic (RefCache.attention; `check_rope` below)."""
from __future__ import annotations

import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")
import kv8_ref  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kv8():
    from bit_expert_layer_gb300.build import build
    build()
    if not torch.cuda.is_available():
        pytest.fail("a GPU test ran without a CUDA device")
    from bit_expert_layer_gb300 import kv8
    return kv8


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Setup:
    """A cache filled with random codes, sequences of the given lengths in shuffled pages, and
    the call's token tensors as slices of one projection's output."""

    def __init__(self, kv8, lens, new, layout=(16, 2, 128), page=64, fmt="e4m3", seed=0, pad=0, n_pages=None, q_gain=2.0):
        self.hq, self.hkv, self.d = layout
        g = self.g = gen(seed)
        self.lens, self.new = list(lens), list(new)
        need = [-(-max(n, 1) // page) for n in lens]
        self.n_pages = n_pages or sum(need) + 2
        order = torch.randperm(self.n_pages, generator=g, device="cuda").cpu().numpy()
        self.table = np.full((len(lens), max(need)), -7, np.int32)     # never read past a sequence's length
        at = 0
        for i, n in enumerate(need):
            self.table[i, :n] = order[at:at + n]
            at += n
        self.offsets = np.concatenate([[0], np.cumsum(new)])
        self.t = int(self.offsets[-1]) + pad
        shape = (self.n_pages, self.hkv, page, self.d)
        if fmt == "e4m3":
            mk = lambda: torch.randn(shape, generator=g, device="cuda").mul_(60).to(torch.float8_e4m3fn).view(torch.uint8)  # noqa: E731
        else:
            mk = lambda: torch.randn(shape, generator=g, device="cuda").mul_(40).clamp_(-127, 127).round_().to(torch.int8).view(torch.uint8)  # noqa: E731
        sc = lambda lo: torch.exp2(torch.randint(lo, lo + 4, shape[:2] + (page // 16,), generator=g, device="cuda").float())  # noqa: E731
        self.cache = kv8.KV8Cache(mk(), mk(), sc(-8), sc(-9), fmt)
        self.qkv = torch.randn(self.t, self.hq + 2 * self.hkv, self.d, generator=g, device="cuda")
        self.qkv[:, :self.hq] *= q_gain
        self.qkv = self.qkv.to(torch.bfloat16)
        self.q = self.qkv[:, :self.hq]
        self.k = self.qkv[:, self.hq:self.hq + self.hkv]
        self.v = self.qkv[:, self.hq + self.hkv:]
        self.batch = kv8.KV8Batch(ints(self.table), ints(self.lens), ints(self.offsets), max_new=max(1, max(new)))

    def ref(self):
        c = self.cache
        return kv8_ref.RefCache(c.k, c.v, c.k_scale, c.v_scale, c.fmt)

    def check_attention(self, out, ref=None, scale=None):
        n = int(self.offsets[-1])
        if n == 0:
            return
        want, bound = (ref or self.ref()).attention(self.table, self.lens, self.offsets, self.q[:n].double(), scale)
        err = (out[:n].double() - want).abs()
        assert torch.isfinite(out[:n]).all()
        worst = torch.argmax((err / bound).flatten())
        assert torch.all(err <= bound), (np.unravel_index(int(worst), err.shape), float(err.flatten()[worst]),
                                         float(bound.flatten()[worst]))

    def check_cache(self, ref):
        c = self.cache
        for name, codes, scales in (("k", c.k, c.k_scale), ("v", c.v, c.v_scale)):
            assert torch.equal(scales.double(), ref.scales[name]), name
            bad = (codes != ref.codes[name]).nonzero()
            assert bad.numel() == 0, (name, bad[:4].tolist())


# ----------------------------------------------------------------------------- rotary positions
def check_rope(got, x, pos, rope_args, inv_freq, axis_of):
    """fp32 products and sums of values with relative error 2^-21 (sine and cosine within a few
    ulp of fp32, their argument within 2^-25 of a turn), then one rounding to bf16."""
    want = kv8_ref.rope(x.double(), pos, inv_freq, axis_of, rope_args["rotary"])
    half = rope_args["rotary"] // 2
    mag = torch.zeros_like(want)
    mag[:, :, :half] = x[:, :, :half].double().abs() + x[:, :, half:2 * half].double().abs()
    mag[:, :, half:2 * half] = mag[:, :, :half]
    assert torch.all((got.double() - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -20 * mag)
    assert torch.equal(got[:, :, 2 * half:], x[:, :, 2 * half:])


@pytest.mark.parametrize("t", [1, 2, 7, 64, 2049])
@pytest.mark.parametrize("d,rotary,axes,cyclic", [(128, 128, 1, False), (128, 32, 3, True), (64, 64, 3, False),
                                                  (64, 16, 2, True), (128, 96, 4, True)])
def test_rope(kv8, t, d, rotary, axes, cyclic):
    g = gen(t * 7 + d + rotary)
    half = rotary // 2
    sections = [half - (axes - 1) * (half // axes)] + [half // axes] * (axes - 1)
    rope = kv8.Rope(d, rotary, theta=1e6, sections=sections, cyclic=cyclic)
    x = torch.randn(t, 7, d, generator=g, device="cuda").to(torch.bfloat16)
    pos = torch.randint(-1000000, 1000000, (axes, t), generator=g, device="cuda", dtype=torch.int32)
    inv = [1e6 ** (-2 * j / rotary) for j in range(half)]
    axis_of = list(rope.plan.axis)[:half]
    q, k = rope(x[:, :5], x[:, 5:], pos)
    a = dict(rotary=rotary)
    check_rope(q, x[:, :5], pos, a, inv, axis_of)
    check_rope(k, x[:, 5:], pos, a, inv, axis_of)
    # in place, in a wider tensor: the other heads stay
    y = x.clone()
    rope(y[:, 1:5], y[:, 5:], pos, out=(y[:, 1:5], y[:, 5:]))
    assert torch.equal(y[:, 1:5], q[:, 1:]) and torch.equal(y[:, 5:], k) and torch.equal(y[:, 0], x[:, 0])
    # q alone
    q2, none = rope(x[:, :5], None, pos)
    assert none is None and torch.equal(q2, q)


def test_rope_given_frequencies_zero_and_special(kv8):
    inv = np.linspace(0, 9, 64)          # 0 turns nothing; above 2 pi / 2 wraps
    rope = kv8.Rope(128, inv_freq=inv)
    x = torch.randn(33, 2, 128, generator=gen(3), device="cuda").to(torch.bfloat16)
    pos = torch.arange(33, dtype=torch.int32, device="cuda")
    q, _ = rope(x, None, pos)
    check_rope(q, x, pos[None], dict(rotary=128), inv, [0] * 64)
    assert torch.equal(q[:, :, 0], x[:, :, 0]) and torch.equal(q[0], x[0])
    x[5, 1, 7] = math.inf
    q2, _ = rope(x, None, pos)
    keep = torch.ones_like(q, dtype=torch.bool)
    keep[5, 1, 7] = keep[5, 1, 71] = False
    assert torch.equal(q2[keep], q[keep])
    e, _ = rope(x[:0], None, pos[:0])
    assert e.shape == (0, 2, 128)


# ----------------------------------------------------------------------------- cache write and read back
LENS_NEW = [([1], [1]), ([16, 17, 15, 33], [1, 1, 1, 1]), ([64, 80, 97], [3, 16, 40]),
            ([130, 0, 5, 300], [130, 0, 5, 33]), ([47, 48, 49], [17, 32, 2])]


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("lens,new", LENS_NEW, ids=[str(x[1]) for x in LENS_NEW])
@pytest.mark.parametrize("layout,page", [((16, 2, 128), 64), ((3, 3, 64), 16), ((4, 1, 128), 32), ((2, 2, 64), 256)])
def test_append_and_gather(kv8, fmt, lens, new, layout, page):
    s = Setup(kv8, lens, new, layout, page, fmt, seed=len(lens) + page, pad=3)
    n = int(s.offsets[-1])
    s.k[:n] *= 0.5                      # some blocks keep their scale, others grow
    s.v[n // 2:n] *= 8
    ref = s.ref()
    ref.append(s.table, s.lens, s.offsets, s.k.double(), s.v.double())
    s.cache.append(s.batch, s.k, s.v)
    s.check_cache(ref)
    k, v = (torch.full((s.t, s.hkv, s.d), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    s.cache.gather(s.batch, s.t, out=(k, v))
    assert (k[n:] == 7).all() and (v[n:] == 7).all()
    for b, (ln, w) in enumerate(zip(lens, new)):
        if w:
            kk, vv, _ = ref.values(s.table[b], ln)
            r = slice(int(s.offsets[b]), int(s.offsets[b + 1]))
            assert torch.equal(k[r].double(), kk[ln - w:]) and torch.equal(v[r].double(), vv[ln - w:])
    assert s.cache.get_error() == 0


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_append_token_by_token(kv8, fmt):
    """33 decode steps of growing magnitude: every growth rounds the block's codes again."""
    s = Setup(kv8, [40, 7], [33, 1], fmt=fmt, seed=4)
    ref = s.ref()
    for i in range(33):
        lens = ints([8 + i, 8])
        b = kv8.KV8Batch(s.batch.page_table, lens, ints([0, 1, 1]), max_new=1)
        k = (torch.randn(1, 2, 128, generator=s.g, device="cuda") * 1.3 ** (i % 16)).to(torch.bfloat16)
        v = (torch.randn(1, 2, 128, generator=s.g, device="cuda") * 2.0 ** ((i * 7) % 16)).to(torch.bfloat16)
        ref.append(s.table, [8 + i, 8], [0, 1, 1], k.double(), v.double())
        s.cache.append(b, k, v)
    s.check_cache(ref)


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_append_extreme_values(kv8, fmt):
    """Zeros, the smallest and largest bf16 numbers, magnitudes at the borders of the scale,
    infinities and NaN; nothing that is not finite reaches the cache."""
    s = Setup(kv8, [16 * 12], [16 * 12], (2, 2, 128), fmt=fmt, seed=5)
    s.k[:16] = 0
    s.k[16:32] *= 2.0 ** -130
    s.k[32:48] *= 2.0 ** -112
    s.k[48:64] = 3.3895313892515355e38
    s.k[64:80] = torch.where(torch.arange(128, device="cuda") % 2 == 0, 3.3895313892515355e38, 2.0 ** -133)
    for i, x in enumerate((448.0, 450.0, 127.0, 127.5, 1.0)):
        s.k[80 + 16 * i:96 + 16 * i] = torch.linspace(-x, x, 128, device="cuda").to(torch.bfloat16)
        s.k[80 + 16 * i, 0, 0] = x
    ref = s.ref()
    ref.append(s.table, s.lens, s.offsets, s.k.double(), s.v.double())
    s.cache.append(s.batch, s.k, s.v)
    s.check_cache(ref)
    assert s.cache.get_error() == 0
    s.v[3, 0, 5] = math.nan
    s.v[4, 1, 6] = -math.inf
    s.v[170:, 1] = math.nan
    s.k[9, 0, :8] = math.inf
    ref.append(s.table, s.lens, s.offsets, s.k.double(), s.v.double())
    s.cache.append(s.batch, s.k, s.v)
    s.check_cache(ref)
    from bit_expert_layer_gb300 import _abi
    assert s.cache.get_error() == _abi.MOE_ERR_NONFINITE
    assert s.cache.get_error() == 0
    k, v = s.cache.gather(s.batch, s.t)
    assert torch.isfinite(k).all() and torch.isfinite(v).all()


# ----------------------------------------------------------------------------- attention
LAYOUTS = [(16, 2, 128), (7, 7, 64), (10, 2, 128), (32, 2, 64), (8, 1, 128), (3, 1, 128), (16, 1, 128)]
EDGE = [1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 500]


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("page", [16, 64])
@pytest.mark.parametrize("layout", LAYOUTS, ids=str)
def test_attention_one_token(kv8, layout, page, fmt):
    s = Setup(kv8, EDGE, [1] * len(EDGE), layout, page, fmt, seed=layout[0] + page)
    s.check_attention(s.cache.attention(s.batch, s.q))
    assert s.cache.get_error() == 0


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("layout", LAYOUTS, ids=str)
@pytest.mark.parametrize("lens,new", [([5, 40, 100], [2, 2, 2]), ([3, 64, 129], [3, 1, 2]), ([70, 9, 333], [5, 4, 8]),
                                      ([20, 300], [20, 17]), ([131, 513, 64], [131, 130, 33])],
                         ids=["two", "three", "eight", "twenty", "prompt"])
def test_attention_several_tokens(kv8, layout, fmt, lens, new):
    s = Setup(kv8, lens, new, layout, 32, fmt, seed=layout[0] + len(new), pad=2)
    out = torch.full(s.q.shape, 5.0, dtype=torch.bfloat16, device="cuda")
    s.cache.attention(s.batch, s.q, out=out)
    s.check_attention(out)
    assert (out[int(s.offsets[-1]):] == 5).all()          # rows behind the last sequence
    assert s.cache.get_error() == 0


@pytest.mark.parametrize("fmt,lens,new", [("e4m3", [32768, 4097], [1, 1]), ("int8", [20001], [1]),
                                          ("e4m3", [9000, 8192], [4, 4]), ("int8", [5000], [700]),
                                          ("e4m3", [2048], [2048])],
                         ids=["decode-32k", "decode-20k", "draft", "piece", "prompt"])
def test_attention_long(kv8, fmt, lens, new):
    s = Setup(kv8, lens, new, fmt=fmt, seed=lens[0])
    s.check_attention(s.cache.attention(s.batch, s.q))


@pytest.mark.parametrize("new", [1, 3])
def test_attention_many_sequences(kv8, new):
    """The largest batch, and more segments per CTA than warps; empty sequences among them."""
    rng = np.random.RandomState(3)
    lens = [int(x) for x in rng.choice([3, 5, 16, 40, 100, 257], 1024)]
    w = [0 if i % 17 == 5 else new for i in range(1024)]
    s = Setup(kv8, lens, w, (4, 2, 64), 16, seed=8)
    s.check_attention(s.cache.attention(s.batch, s.q))


def test_attention_rows_that_see_nothing(kv8):
    """A sequence without positions, and one with more new tokens than positions: zeros."""
    s = Setup(kv8, [0, 2, 30], [1, 5, 1], seed=9)
    out = s.cache.attention(s.batch, s.q)
    s.check_attention(out)
    assert (out[0] == 0).all() and (out[1:4] == 0).all() and (out[4:] != 0).any(-1).all()


@pytest.mark.parametrize("new", [1, 2, 40])
@pytest.mark.parametrize("page", [16, 128])
def test_attention_ignores_what_lies_behind(kv8, new, page):
    """Codes (e4m3 NaN among them) and scales past a sequence's length do not matter."""
    lens = [n for n in (50, 97, 257) if n >= new]
    s = Setup(kv8, lens, [new] * len(lens), page=page, seed=10)
    a = s.cache.attention(s.batch, s.q)
    c = s.cache
    live = torch.zeros(c.k.shape[0], c.k.shape[2], dtype=torch.bool, device="cuda")
    for row, n in zip(s.table, lens):
        for p in range(n):
            live[int(row[p // page]), p % page] = True
    dead = ~live[:, None, :, None].expand_as(c.k)
    c.k[dead] = 0x7F
    c.v[dead] = 0xFF
    blocks = ~live.view(live.shape[0], -1, 16).any(-1)[:, None].expand_as(c.k_scale)
    c.k_scale[blocks] = math.nan
    c.v_scale[blocks] = math.inf
    assert torch.equal(s.cache.attention(s.batch, s.q), a)


def test_attention_extreme_scales(kv8):
    """Value blocks of very different scales, all-zero blocks, queries of any magnitude."""
    s = Setup(kv8, [400, 400], [1, 1], (16, 2, 128), seed=11, q_gain=1.0)
    c = s.cache
    c.v_scale[:] = torch.exp2(torch.randint(-30, 10, c.v_scale.shape, generator=s.g, device="cuda").float())
    c.v_scale[int(s.table[0, 0])] = 2.0 ** -100
    c.v[int(s.table[0, 0])] = 0
    s.q[0] = 0
    s.q[1, :4] *= 2.0 ** -60
    s.check_attention(c.attention(s.batch, s.q))
    s.q[:] = 1.0
    s.q[0] *= 2.0 ** 60                    # one key takes all the weight
    c.k_scale[:] = 2.0 ** -66
    s.check_attention(c.attention(s.batch, s.q))


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("new", [1, 3, 90])
def test_attention_uneven_scales(kv8, new, fmt):
    """Blocks side by side whose scales differ by up to 2^20, for keys and values alike."""
    s = Setup(kv8, [500, 90], [new, new], (16, 2, 128), 32, fmt, seed=33, q_gain=1.0)
    c = s.cache
    for x, lo in ((c.k_scale, -26), (c.v_scale, -18)):
        x[:] = torch.exp2(torch.randint(lo, lo + 21, x.shape, generator=s.g, device="cuda").float())
    s.check_attention(c.attention(s.batch, s.q))


def test_attention_not_finite_queries_stay_in_their_rows(kv8):
    s = Setup(kv8, [100, 70, 40], [1, 3, 1], seed=12)
    a = s.cache.attention(s.batch, s.q)
    s.q[0, 3, 5] = math.nan
    s.q[2, 8, 0] = math.nan
    b = s.cache.attention(s.batch, s.q)
    keep = torch.ones(5, 16, dtype=torch.bool, device="cuda")
    keep[0, 3] = keep[2, 8] = False
    assert torch.equal(a[keep], b[keep]) and torch.isnan(b[~keep]).all()


def test_prompt_queries_that_are_not_finite_stay_in_their_rows(kv8):
    s = Setup(kv8, [700, 200], [60, 200], seed=34)
    a = s.cache.attention(s.batch, s.q)
    s.q[5, 3, 5] = math.nan
    s.q[61, 8, 0] = math.nan
    s.q[150, 15] = math.inf
    b = s.cache.attention(s.batch, s.q)
    keep = torch.ones(260, 16, dtype=torch.bool, device="cuda")
    keep[5, 3] = keep[61, 8] = keep[150, 15] = False
    assert torch.equal(a[keep], b[keep]) and torch.isnan(b[~keep]).all()


@pytest.mark.parametrize("new", [1, 4, 90])
def test_query_of_infinity_makes_its_row_nan_whatever_the_keys(kv8, new):
    """All scores minus infinity (one sign of keys in the query's infinite dim) are no row of zeros."""
    s = Setup(kv8, [150], [new], seed=35)
    s.cache.k[..., 5] = 0x38                     # 1.0 in every key
    a = s.cache.attention(s.batch, s.q)
    s.q[new - 1, 3] = 0
    s.q[new - 1, 3, 5] = -math.inf
    b = s.cache.attention(s.batch, s.q)
    keep = torch.ones(new, 16, dtype=torch.bool, device="cuda")
    keep[new - 1, 3] = False
    assert torch.equal(a[keep], b[keep]) and torch.isnan(b[~keep]).all()


@pytest.mark.parametrize("new", [1, 4, 90])
@pytest.mark.parametrize("gain, key", [(116, -100), (90, -95), (-100, 95), (-126, 118)])
def test_queries_and_keys_at_opposite_ends_of_the_range(kv8, new, gain, key):
    """The scores are of ordinary size although neither factor is."""
    s = Setup(kv8, [150, 90], [new, new], seed=36)
    s.cache.k_scale[:] = 2.0 ** key
    s.q[:] = (s.q.double() * 2.0 ** gain).to(torch.bfloat16)
    scale = 2.0 ** (-8 - gain - key)
    assert torch.isfinite(s.q).all() and 1e-30 < scale < 1e30
    s.check_attention(s.cache.attention(s.batch, s.q, scale=scale), scale=scale)


@pytest.mark.parametrize("scale", [0.02, 1.5])
def test_attention_scale(kv8, scale):
    s = Setup(kv8, [300, 33], [1, 1], seed=13, q_gain=0.5)
    s.check_attention(s.cache.attention(s.batch, s.q, scale=scale), scale=scale)


@pytest.mark.parametrize("new", [1, 40])
def test_bad_pages_lengths_and_offsets(kv8, new):
    """What is out of range on the device: left out, recorded, and nothing else changes."""
    from bit_expert_layer_gb300 import _abi
    s = Setup(kv8, [200, 300, 90], [new] * 3, page=16, seed=14)
    c, good = s.cache, s.cache.attention(s.batch, s.q)
    r1 = slice(int(s.offsets[1]), int(s.offsets[2]))
    rest = torch.ones(s.t, dtype=torch.bool, device="cuda")
    rest[r1] = False
    for page in (-1, s.n_pages, 2 ** 31 - 1, -2 ** 31):
        t = s.table.copy()
        t[1, 3] = page
        b = kv8.KV8Batch(ints(t), s.batch.lens, s.batch.offsets, s.batch.max_new)
        out = c.attention(b, s.q)
        assert c.get_error() == _abi.MOE_ERR_DEVICE_BOUNDS
        assert torch.equal(out[rest], good[rest]) and torch.isfinite(out).all()
        if new == 1:                       # the other 284 positions' attention
            keep = torch.cat([torch.arange(48), torch.arange(64, 300)]).cuda()
            k, v, _ = s.ref().values(s.table[1], 300)
            for h in (0, 9):
                p = torch.softmax(k[keep, h // 8] @ s.q[r1][0, h].double() / math.sqrt(128), 0)
                want = p @ v[keep, h // 8]
                assert ((out[r1][0, h].double() - want).abs() <= 2.0 ** -7 * (p @ v[keep, h // 8].abs())).all()
        before = c.k.clone()
        c.append(kv8.KV8Batch(ints(t[:, :4].copy()), ints([64, 64, 64]), ints([0, 0, 16, 16]), 16), s.k[:16].repeat(2, 1, 1)[:16]
                 if new > 1 else s.k[:1].repeat(16, 1, 1), s.v[:1].repeat(16, 1, 1))
        assert c.get_error() == _abi.MOE_ERR_DEVICE_BOUNDS and torch.equal(c.k, before)
    for lens in ([200, 2 ** 31 - 1, 90], [200, -5, 90]):
        b = kv8.KV8Batch(s.batch.page_table, ints(lens), s.batch.offsets, s.batch.max_new)
        out = c.attention(b, s.q)
        assert c.get_error() == _abi.MOE_ERR_DEVICE_BOUNDS and torch.equal(out[rest], good[rest])
    for off in ([0, 2 ** 30, 2, 3], [-4, 1, 2, 3], [0, 5, 2, 10 ** 9], [3, 2, 1, 0]):
        b = kv8.KV8Batch(s.batch.page_table, s.batch.lens, ints(off), s.batch.max_new)
        c.attention(b, s.q)
        assert c.get_error() == _abi.MOE_ERR_DEVICE_BOUNDS
        c.gather(b, s.t)
        assert c.get_error() == _abi.MOE_ERR_DEVICE_BOUNDS
    # more new tokens than max_new: the first ones are done
    if new > 1:
        b = kv8.KV8Batch(s.batch.page_table, s.batch.lens, s.batch.offsets, new - 7)
        out = torch.full(s.q.shape, 5.0, dtype=torch.bfloat16, device="cuda")
        c.attention(b, s.q, out=out)
        assert c.get_error() == _abi.MOE_ERR_DEVICE_BOUNDS and (out[new - 7:new] == 5).all()
    assert torch.equal(c.attention(s.batch, s.q), good) and c.get_error() == 0


def test_cache_past_4_gigabytes(kv8):
    """Pages whose byte offsets pass 2^32."""
    n_pages = (5 << 30) // (2 * 64 * 128)
    c = kv8.KV8Cache.empty(n_pages, fmt="int8")
    s = Setup(kv8, [333, 200], [333, 200], fmt="int8", seed=15)
    far = np.random.RandomState(1).permutation(np.arange(n_pages - 40, n_pages))
    table = s.table.copy()
    table[s.table >= 0] = far[s.table[s.table >= 0]]
    b = kv8.KV8Batch(ints(table), s.batch.lens, s.batch.offsets, s.batch.max_new)
    s.cache.append(s.batch, s.k, s.v)
    c.append(b, s.k, s.v)
    assert torch.equal(c.gather(b, s.t)[0], s.cache.gather(s.batch, s.t)[0])
    assert torch.equal(c.attention(b, s.q), s.cache.attention(s.batch, s.q))
    one = kv8.KV8Batch(ints(table), s.batch.lens, ints([0, 1, 2]), 1)
    ref = kv8.KV8Batch(ints(s.table), s.batch.lens, ints([0, 1, 2]), 1)
    assert torch.equal(c.attention(one, s.q[:2]), s.cache.attention(ref, s.q[:2]))
    assert c.get_error() == 0


def test_same_bits_again_and_one_workspace_for_all_shapes(kv8):
    shapes = [Setup(kv8, [5000, 300, 17], [1, 1, 1], seed=16), Setup(kv8, [700, 64], [33, 64], seed=17),
              Setup(kv8, [3000, 40], [4, 2], (10, 2, 128), seed=18), Setup(kv8, [900] * 40, [1] * 40, seed=19)]
    ws = max((s.cache.new_workspace(s.hq, s.batch.max_new) for s in shapes), key=lambda w: w.numel())
    first = [s.cache.attention(s.batch, s.q) for s in shapes]
    for _ in range(5):
        for s, a in zip(shapes, first):
            assert torch.equal(s.cache.attention(s.batch, s.q, workspace=ws), a)


def test_other_stream_and_short_wait_limit(kv8):
    from bit_expert_layer_gb300 import _abi
    s = Setup(kv8, [3000, 300], [1, 1], seed=20)
    a = s.cache.attention(s.batch, s.q)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    outs = [s.cache.attention(s.batch, s.q, stream=st) for _ in range(4)]
    st.synchronize()
    assert all(torch.equal(o, a) for o in outs)
    # a wait that gives up is recorded, and the next call is whole again
    big = Setup(kv8, [30000] * 8, [1] * 8, seed=21)
    b = big.cache.attention(big.batch, big.q)
    ws = big.cache.new_workspace(16, 1)
    _abi.moe_set_wait_limit_ns(1)
    try:
        big.cache.attention(big.batch, big.q, workspace=ws)
        torch.cuda.synchronize()
    finally:
        _abi.moe_set_wait_limit_ns(0)
    assert big.cache.get_error() == _abi.MOE_ERR_TIMEOUT
    assert torch.equal(big.cache.attention(big.batch, big.q, workspace=ws), b)
    assert big.cache.get_error() == 0


def test_prompt_with_a_short_wait_limit(kv8):
    """The prompt kernel's waits give up, too: recorded, and the next call is whole again."""
    from bit_expert_layer_gb300 import _abi
    s = Setup(kv8, [3000, 700], [600, 700], seed=23)
    a = s.cache.attention(s.batch, s.q)
    ws = s.cache.new_workspace(16, 700)
    _abi.moe_set_wait_limit_ns(1)
    try:
        s.cache.attention(s.batch, s.q, workspace=ws)
        torch.cuda.synchronize()
    finally:
        _abi.moe_set_wait_limit_ns(0)
    assert s.cache.get_error() == _abi.MOE_ERR_TIMEOUT
    assert torch.equal(s.cache.attention(s.batch, s.q, workspace=ws), a)
    assert s.cache.get_error() == 0


@pytest.mark.parametrize("new", [1, 40])
def test_two_calls_at_once(kv8, new):
    """Two streams, one cache, a workspace each."""
    s = Setup(kv8, [4000, 900, 60], [new] * 3, seed=24)
    a = s.cache.attention(s.batch, s.q)
    streams = [torch.cuda.Stream() for _ in range(2)]
    spaces = [s.cache.new_workspace(16, new) for _ in range(2)]
    torch.cuda.synchronize()
    outs = [s.cache.attention(s.batch, s.q, workspace=spaces[i % 2], stream=streams[i % 2]) for i in range(12)]
    torch.cuda.synchronize()
    assert all(torch.equal(o, a) for o in outs) and s.cache.get_error() == 0


@pytest.mark.parametrize("lens,new,bound", [([700, 33], [1, 1], 300), ([300, 40], [5, 2], 64), ([90, 64], [0, 0], 9)])
def test_a_loose_bound_on_the_new_tokens(kv8, lens, new, bound):
    s = Setup(kv8, lens, new, seed=25, pad=1)
    b = kv8.KV8Batch(s.batch.page_table, s.batch.lens, s.batch.offsets, bound)
    out = torch.full(s.q.shape, 5.0, dtype=torch.bfloat16, device="cuda")
    s.cache.attention(b, s.q, out=out)
    s.check_attention(out)
    assert (out[int(s.offsets[-1]):] == 5).all() and s.cache.get_error() == 0


def test_prompts_of_the_largest_batch(kv8):
    rng = np.random.RandomState(5)
    new = [int(x) for x in rng.choice([0, 1, 17, 40], 1024)]
    s = Setup(kv8, [n + int(rng.choice([0, 3, 150])) for n in new], new, (4, 2, 64), 16, seed=26)
    s.check_attention(s.cache.attention(s.batch, s.q))
    assert s.cache.get_error() == 0


@pytest.mark.parametrize("new", [1, 6])
@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_three_million_positions(kv8, fmt, new):
    """A sequence that reads the same four pages 750 times over: what all its tokens see is, but
    for the last few positions, what one round of the pages gives (each weight 1 / 750).  Of
    sum_i p_i |v_i|: 2^-11 for the weights, (n / 128 + 64) 2^-23 < 2^-8.4 for the fp32 sums over
    n positions, 2^-8 for the last rounding; together under 2^-7."""
    s = Setup(kv8, [4096], [new], (8, 1, 64), 1024, fmt, seed=27)
    rounds = 750
    b = kv8.KV8Batch(ints(np.tile(s.table, (1, rounds))), ints([4096 * rounds]), s.batch.offsets, new)
    out = s.cache.attention(b, s.q).double()
    k, v, _ = s.ref().values(s.table[0], 4096)
    for i in range(new):
        n = torch.full((4096,), float(rounds), device="cuda", dtype=torch.float64)
        n[4096 - new + i + 1:] -= 1
        for h in range(8):
            p = torch.softmax(k[:, 0] @ s.q[i, h].double() / 8 + n.log(), 0)
            assert ((out[i, h] - p @ v[:, 0]).abs() <= 2.0 ** -7 * (p @ v[:, 0].abs())).all()
    assert s.cache.get_error() == 0


def test_captured_prompt(kv8):
    s = Setup(kv8, [300, 77], [120, 33], seed=28)
    ws = s.cache.new_workspace(16, 120)
    want = s.cache.attention(s.batch, s.q, workspace=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = s.cache.attention(s.batch, s.q, workspace=ws)
    for lens in ([300, 77], [411, 200], [120, 33]):
        s.lens = [min(a, 5 * 64 if i == 0 else 2 * 64) for i, a in enumerate(lens)]
        s.batch.lens.copy_(ints(s.lens))
        out.zero_()
        graph.replay()
        s.check_attention(out)
    s.batch.lens.copy_(ints([300, 77]))
    graph.replay()
    assert torch.equal(out, want) and s.cache.get_error() == 0


def test_refusals(kv8):
    s = Setup(kv8, [40, 30], [1, 1], seed=22)
    bad = [lambda: kv8.KV8Batch(s.batch.page_table.long(), s.batch.lens, s.batch.offsets, 1),
           lambda: kv8.KV8Batch(s.batch.page_table, s.batch.lens[:1], s.batch.offsets, 1),
           lambda: kv8.KV8Batch(s.batch.page_table, s.batch.lens, s.batch.offsets.cpu(), 1),
           lambda: kv8.KV8Cache(s.cache.k, s.cache.v, s.cache.k_scale[:1], s.cache.v_scale),
           lambda: kv8.KV8Cache(s.cache.k, s.cache.v, s.cache.k_scale, s.cache.v_scale, "fp4"),
           lambda: kv8.KV8Cache(s.cache.k.bfloat16(), s.cache.v, s.cache.k_scale, s.cache.v_scale),
           lambda: s.cache.append(s.batch, s.k.float(), s.v), lambda: s.cache.append(s.batch, s.k, s.v[:1]),
           lambda: s.cache.append(s.batch, s.q, s.v), lambda: s.cache.attention(s.batch, s.q.transpose(0, 1)),
           lambda: s.cache.attention(s.batch, s.q[..., ::2]), lambda: s.cache.attention(s.batch, s.q, out=s.q),
           lambda: s.cache.attention(s.batch, s.q.half()), lambda: s.cache.gather(s.batch, 3, out=(s.k, s.v)),
           lambda: kv8.Rope(128, sections=[64])(s.q, s.k, ints([[1, 2], [3, 4]])),
           lambda: kv8.Rope(64)(s.q, s.k, ints([1, 2]))]
    for i, f in enumerate(bad):
        with pytest.raises(ValueError):
            f()
            pytest.fail(f"call {i} was not refused")
    from bit_expert_layer_gb300 import _abi
    with pytest.raises(_abi.MoEError) as e:
        s.cache.attention(s.batch, s.q, workspace=torch.zeros(64, dtype=torch.uint8, device="cuda"))
    assert e.value.status == _abi.MOE_ERR_WORKSPACE
    assert s.cache.attention(s.batch, s.q[:0]).shape == (0, 16, 128)
    assert s.cache.get_error() == 0


# ----------------------------------------------------------------------------- together
def test_what_a_call_describes_cannot_be_replaced(kv8):
    """A new tensor under an old name would leave the library with the old one's address."""
    s = Setup(kv8, [20], [1])
    out = s.cache.attention(s.batch, s.q)
    for obj, names in ((s.batch, ("page_table", "lens", "offsets", "max_new")), (s.cache, ("k", "v_scale", "error", "fmt")),
                       (kv8.Rope(), ("plan", "head_size"))):
        for name in names:
            with pytest.raises(AttributeError):
                setattr(obj, name, getattr(obj, name))
    s.batch.lens.fill_(10)                       # in place is how they change
    assert not torch.equal(s.cache.attention(s.batch, s.q), out)
    s.cache.attention(s.batch, s.q[:0])          # another number of rows, and back
    s.batch.lens.fill_(20)
    assert torch.equal(s.cache.attention(s.batch, s.q), out)


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_prompt_then_decode(kv8, fmt):
    """As a model uses them: rotary positions, cache write and attention, first two prompts of
    different length, then single tokens, against the same steps in 64 bits."""
    g = gen(30)
    rope = kv8.Rope(128, 32, theta=1e7, sections=[8, 4, 4], cyclic=True)
    inv = [1e7 ** (-2 * j / 32) for j in range(16)]
    axis_of = list(rope.plan.axis)[:16]
    cache = kv8.KV8Cache.empty(16, fmt=fmt)
    ref = kv8_ref.RefCache(cache.k, cache.v, cache.k_scale, cache.v_scale, fmt)
    table = np.random.RandomState(2).permutation(16).reshape(2, 8).astype(np.int32)
    ws = cache.new_workspace(16, 150)
    lens = [0, 0]
    for new in [(150, 41)] + [(1, 1)] * 20 + [(5, 0), (1, 3)]:
        lens = [a + n for a, n in zip(lens, new)]
        off = [0, new[0], sum(new)]
        qkv = torch.randn(sum(new), 20, 128, generator=g, device="cuda").to(torch.bfloat16)
        pos = torch.randint(0, 3000, (3, sum(new)), generator=g, device="cuda", dtype=torch.int32)
        q, k = rope(qkv[:, :16], qkv[:, 16:18], pos)
        check_rope(q, qkv[:, :16], pos, dict(rotary=32), inv, axis_of)
        check_rope(k, qkv[:, 16:18], pos, dict(rotary=32), inv, axis_of)
        b = kv8.KV8Batch(ints(table), ints(lens), ints(off), max_new=max(new))
        cache.append(b, k, qkv[:, 18:])
        ref.append(table, lens, off, k.double(), qkv[:, 18:].double())
        out = cache.attention(b, q, workspace=ws)
        want, bound = ref.attention(table, lens, off, q.double())
        assert ((out.double() - want).abs() <= bound).all()
    assert torch.equal(cache.k, ref.codes["k"]) and torch.equal(cache.v, ref.codes["v"])
    assert cache.get_error() == 0


def test_captured_decode_step_follows_its_inputs(kv8):
    """A decode step captured once and replayed with other lengths, pages and tokens, while an
    eager call of another shape uses the same workspace in between."""
    s = Setup(kv8, [200, 700, 33], [1, 1, 1], seed=31)
    other = Setup(kv8, [900, 64], [1, 1], seed=32)
    rope = kv8.Rope(128)
    pos = torch.zeros(3, dtype=torch.int32, device="cuda")
    ws = s.cache.new_workspace(16, 1)

    def step():
        q, k = rope(s.q, s.k, pos)
        s.cache.append(s.batch, k, s.v)
        return s.cache.attention(s.batch, q, workspace=ws), q, k
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, q, k = step()
    want_other = other.cache.attention(other.batch, other.q)
    for i in range(3):
        s.lens = [17 + 5 * i, 640 + 20 * i, 1 + i]
        s.batch.lens.copy_(ints(s.lens))
        s.table[1] = np.roll(s.table[1], 1)
        s.batch.page_table.copy_(ints(s.table))
        pos.copy_(ints([n - 1 for n in s.lens]))
        s.qkv.copy_(torch.randn(s.qkv.shape, generator=s.g, device="cuda"))
        ref = s.ref()
        graph.replay()
        assert torch.equal(other.cache.attention(other.batch, other.q, workspace=ws), want_other)
        ref.append(s.table, s.lens, s.offsets, k.double(), s.v.double())
        s.check_cache(ref)
        want, bound = ref.attention(s.table, s.lens, s.offsets, q.double())
        assert ((out.double() - want).abs() <= bound).all()
    assert s.cache.get_error() == 0


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("layout", [(16, 2, 128), (16, 1, 128), (7, 7, 64)], ids=str)
@pytest.mark.parametrize("n, new", [(100, 400), (0, 2048), (126, 129), (0, 129), (3, 4), (0, 1)])
def test_fewer_positions_than_new_tokens(kv8, n, new, layout, fmt):
    """The tokens that stand before position 0 get zeros, the others theirs, the sequences beside
    them all of theirs, and the length is recorded."""
    from bit_expert_layer_gb300 import _abi
    s = Setup(kv8, [300, n, 1000], [new % 40 + 1, new, 70 if new > 8 else 1], layout, 32, fmt, seed=n + new)
    out = torch.full(s.q.shape, 5.0, dtype=torch.bfloat16, device="cuda")
    s.cache.attention(s.batch, s.q, out=out)
    assert s.cache.get_error() == _abi.MOE_ERR_DEVICE_BOUNDS
    s.check_attention(out)
    r0 = int(s.offsets[1])
    assert (out[r0:r0 + new - n] == 0).all() and (out[r0 + new - n:] != 0).any(-1).all()


def one_row(s, b, h, q, scale=None):
    """(p, v, e) float64: weights, values and value-scale exponents of query q [d] of head h over all
    positions of sequence b, by the definition."""
    n = s.lens[b]
    k, v, vs = s.ref().values(s.table[b], n)
    g = h // (s.hq // s.hkv)
    return torch.softmax(k[:, g] @ q.double() * (scale or 1 / math.sqrt(s.d)), 0), v[:, g], vs[:, g].log2()


def shared_pages(kv8, n, seqs, new, layout, fmt, seed, page=64):
    """One cached sequence of n positions, read by `seqs` sequences of `new` new tokens each: so many
    tiles that a single run of work holds (nearly) all positions of a row."""
    one = Setup(kv8, [n], [1], layout, page, fmt, seed=seed)
    s = Setup(kv8, [n] * 2, [new] * 2, layout, page, fmt, seed=seed, n_pages=2 * -(-n // page))
    s.cache, s.n_pages = one.cache, one.n_pages
    s.lens, s.new = [n] * seqs, [new] * seqs
    s.table = np.tile(one.table, (seqs, 1))
    s.offsets = np.arange(seqs + 1) * new
    s.t = seqs * new
    s.q = torch.randn(s.t, s.hq, s.d, generator=s.g, device="cuda").to(torch.bfloat16)
    s.batch = kv8.KV8Batch(ints(s.table), ints(s.lens), ints(s.offsets), max_new=new)
    return s


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("seqs, new, layout", [(152, 5, (8, 1, 128)), (608, 1, (16, 2, 128)), (608, 2, (16, 2, 64)),
                                               (1, 1, (16, 2, 128)), (1, 90, (16, 2, 64))])
def test_long_runs_of_zero_values(kv8, seqs, new, layout, fmt):
    """36 thousand positions whose values are all zero (the smallest scale there is), scored 2^7.9
    above the first ones, and 500 others after them with as high a score: the rows' sums of weights
    pass no range.  Of sum_i p_i |v_i|: 2^-11 for the weights, the scores' 2^-22 (8 + 128) twice,
    2^-21 twice for the exponential, 2^-23 (36500 / 128 + 64) for fp32 sums, all under 2^-10; and one
    rounding."""
    n, last = 36500, 500
    s = shared_pages(kv8, n, seqs, new, layout, fmt, 40)
    c = s.cache
    pos = torch.arange(n, device="cuda")
    pg, at = torch.tensor(s.table[0], device="cuda").long()[pos // 64], pos % 64
    c.k.zero_()
    c.k[pg[128:], :, at[128:], 0] = 0x38 if fmt == "e4m3" else 1          # 1
    c.k_scale.fill_(1)
    zero = (n - last) // 16 * 16
    c.v[pg[:zero], :, at[:zero]] = 0
    c.v_scale[pg[:zero:16], :, at[:zero:16] // 16] = 2.0 ** -100
    s.q.zero_()
    s.q[:, :, 0] = 1
    scale = 7.9 * math.log(2)
    out = c.attention(s.batch, s.q, scale=scale).double()
    for g in range(s.hkv):
        h = g * s.hq // s.hkv
        p, v, _ = one_row(s, 0, h, s.q[0, h], scale)
        for i in range(new):
            w = p.clone()
            w[n - new + i + 1:] = 0
            w /= w.sum()
            want, mag = w @ v, w @ v.abs()
            assert ((out[i::new, h] - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -10 * mag).all()
    assert c.get_error() == 0


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("new", [1, 4, 90])
@pytest.mark.parametrize("unit", [16, 128])
@pytest.mark.parametrize("low, high", [(-100, 60), (-100, 115), (-60, 20), (-100, 0)])
def test_zero_values_beside_large_ones(kv8, new, low, high, unit, fmt):
    """Every second 16 (or 128) positions have values of zero and the smallest scales, the others
    large ones: the zeros' weights count in full."""
    s = Setup(kv8, [700, 130], [new, new], (16, 2, 128), 16, fmt, seed=41, q_gain=1.0)
    c = s.cache
    c.v_scale[:] = 2.0 ** high
    for b, n in enumerate(s.lens):
        for i in range(0, n, 16):
            if i // unit % 2 == 0:
                c.v[int(s.table[b, i // 16])] = 0
                c.v_scale[int(s.table[b, i // 16])] = 2.0 ** low
    s.check_attention(c.attention(s.batch, s.q))


@pytest.mark.parametrize("new", [1, 4, 90])
@pytest.mark.parametrize("score", [2.0 ** 20, 2.0 ** 28, 1e31, 3e38, 1e45, -2.0 ** 20, -2.0 ** 28, -1e31, -3e38, -1e45])
def test_scores_of_any_size(kv8, new, score):
    """Equal scores of any size, past fp32's range too, are equal weights; one that is larger by an
    eighth has all the weight.  2^-10 of sum_i p_i |v_i| and one rounding, as for ordinary scores."""
    s = Setup(kv8, [1000, 200, new], [new] * 3, seed=42)
    c = s.cache
    c.k.zero_()
    c.k[..., 0] = 0x38                                   # 1, next: 1.125
    e = 0 if abs(score) < 1e30 else 60
    c.k_scale.fill_(2.0 ** e)
    s.q.zero_()
    s.q[:, :, 0] = math.copysign(2.0 ** e, score)
    scale = float(np.float32(abs(score) / 4.0 ** e))
    a = c.attention(s.batch, s.q, scale=scale).double()
    at = 64 + 37                                         # of the second sequence
    c.k[int(s.table[1, 1]), :, 37, 0] = 0x39 if score > 0 else 0x37
    b = c.attention(s.batch, s.q, scale=scale).double()
    for j in range(3):
        v = s.ref().values(s.table[j], s.lens[j])[1]
        for i in range(new):
            see = s.lens[j] - new + i + 1
            r = int(s.offsets[j]) + i
            for h in (0, 9):
                x = v[:see, h // 8]
                want, mag = x.mean(0), x.abs().mean(0)
                assert ((a[r, h] - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -10 * mag).all()
                if j == 1 and see > at and abs(score) < 3e38:
                    want, mag = x[at], x[at].abs()
                assert ((b[r, h] - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -10 * mag).all()
    assert c.get_error() == 0


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("n, share", [(32768, 0.99), (32768, 0.999), (131072, 0.99), (131072, 0.999), (8192, 0.9999),
                                      (8192, 0.9999999)])
@pytest.mark.parametrize("zeros", [0, 4096])
@pytest.mark.parametrize("seqs, new, layout", [(152, 5, (8, 1, 128)), (608, 1, (16, 2, 128)), (608, 2, (16, 2, 64)),
                                               (1, 1, (16, 2, 128)), (1, 40, (8, 1, 64))])
def test_a_position_that_takes_nearly_all_the_weight(kv8, seqs, new, layout, zeros, n, share, fmt):
    """A sink: the first position has nearly all the weight and a value of zero, so that the row is
    what the many small weights make of theirs, the first of which may be zeros, too, of the smallest
    scale there is.  The row's error is under 2^-7 of the row, by the
    Euclidean norm: one rounding to bf16 is at most 2^-8 of each element, the rest is small beside it."""
    s = shared_pages(kv8, n, seqs, new, layout, fmt, 43)
    c = s.cache
    c.k[..., 0] = 0
    first = int(s.table[0, 0])
    c.k[first, :, 0] = 0
    c.k[first, :, 0, 0] = 0x7E if fmt == "e4m3" else 127
    c.v[first, :, 0] = 0
    pages = torch.tensor(s.table[0], device="cuda").long()[:zeros // 64]
    c.v[pages] = 0
    c.v_scale[pages] = 2.0 ** -100
    s.q[:, :, 0] = 0
    k, v, _ = s.ref().values(s.table[0], n)
    rows = sorted({0, 1, s.t // 2, s.t - 1} & set(range(s.t)))
    scale = 1 / math.sqrt(s.d)
    for h in range(s.hq):                                # each row's own share, the other rows 1 / 2
        g = h // (s.hq // s.hkv)
        lse = torch.logsumexp(k[1:, g] @ s.q[rows, h].double().T * scale, 0)
        t = (lse + math.log(share / (1 - share))) / (k[0, g, 0] * scale)
        s.q[:, h, 0] = float(t.median())
        s.q[rows, h, 0] = t.to(torch.bfloat16)
    out = c.attention(s.batch, s.q).double()
    for r in rows:
        see = n - new + r % new + 1
        for h in (0, s.hq - 1):
            g = h // (s.hq // s.hkv)
            p = torch.softmax(k[:see, g] @ s.q[r, h].double() * scale, 0)
            want, lost = p @ v[:see, g], 0.0
            assert abs(math.log((1 - float(p[0])) / (1 - share))) < 0.3
            if (1 - share) / n < 2.0 ** -32:
                # The 128 positions of the sink's own tile meet it in one product, in which it is
                # 2^7: theirs are under 2^(7 - 32) = 2^-25 there, what fp16 rounds to zero or to
                # 2^-24, and are off by up to 2^-25, or 2^-32 of the sink's weight, times the scales'
                # ratio of at most 2^3.
                lost = (p[1:128].clamp_max(2.0 ** -29) @ v[1:128, g].abs()).norm()
            err = (out[r, h] - want).norm()
            assert err <= 2.0 ** -7 * want.norm() + lost, (r, h, float(err / want.norm()))
    assert c.get_error() == 0


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("seqs, new, layout", [(152, 5, (8, 1, 128)), (608, 1, (16, 2, 128)), (1, 1, (16, 2, 128))])
def test_one_block_of_large_values(kv8, seqs, new, layout, fmt):
    """A block whose scale is 2^10 times the others', all of it in one dim: the other dims keep
    their bits."""
    n = 32768
    s = shared_pages(kv8, n, seqs, new, layout, fmt, 44)
    c = s.cache
    c.v_scale.fill_(2.0 ** -9)
    pg = int(s.table[0, 2])
    c.v[pg, :, 16:32] = 0
    c.v[pg, :, 16:32, 7] = 0x7E if fmt == "e4m3" else 127
    c.v_scale[pg, :, 1] = 2.0
    out = c.attention(s.batch, s.q).double()
    keep = torch.arange(s.d, device="cuda") != 7
    for r in sorted({0, s.t - 1}):
        for h in (0, s.hq - 1):
            see = n - new + r % new + 1
            k, v, _ = s.ref().values(s.table[0], see)
            g = h // (s.hq // s.hkv)
            p = torch.softmax(k[:, g] @ s.q[r, h].double() / math.sqrt(s.d), 0)
            want = p @ v[:, g]
            assert (out[r, h] - want)[keep].norm() <= 2.0 ** -7 * want[keep].norm()
            assert (out[r, h] - want)[7].abs() <= 2.0 ** -7 * want[7].abs()


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("over, new", [(1, 1), (3, 5), (5, 5), (40, 60), (2 ** 31 - 1 - 128, 60)])
def test_lengths_past_the_page_table_move_no_token(kv8, over, new, fmt):
    """A sequence with more positions than its row of the page table: the tokens past its end are
    left out, the others stand where they would have, and no cached position changes."""
    from bit_expert_layer_gb300 import _abi
    cap = 128
    s = Setup(kv8, [200, cap, 90], [3, new, 20], page=64, fmt=fmt, seed=45)
    table = s.table[:, :2].copy()
    lens = [100, cap + over, 90]
    b = kv8.KV8Batch(ints(table), ints(lens), s.batch.offsets, s.batch.max_new)
    ref = s.ref()
    r = [int(x) for x in s.offsets]
    fit = max(new - over, 0)                                     # tokens before the end
    rows = list(range(r[0], r[1])) + list(range(r[1], r[1] + fit)) + list(range(r[2], r[3]))
    off = [0, 3, 3 + fit, 23 + fit]
    ref.append(table, [100, cap, 90], off, s.k[rows].double(), s.v[rows].double())
    s.cache.append(b, s.k, s.v)
    assert s.cache.get_error() == _abi.MOE_ERR_DEVICE_BOUNDS
    s.check_cache(ref)
    k, v = (torch.full((s.t, s.hkv, s.d), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    s.cache.gather(b, s.t, out=(k, v))
    assert s.cache.get_error() == _abi.MOE_ERR_DEVICE_BOUNDS
    assert (k[r[1] + fit:r[2]] == 7).all() and (v[r[1] + fit:r[2]] == 7).all()
    for i, n, w, row in ((0, 100, 3, r[0]), (1, cap, fit, r[1]), (2, 90, 20, r[2])):
        kk, vv, _ = ref.values(table[i], n)
        assert torch.equal(k[row:row + w].double(), kk[n - w:]) and torch.equal(v[row:row + w].double(), vv[n - w:])
    out = torch.full(s.q.shape, 5.0, dtype=torch.bfloat16, device="cuda")
    s.cache.attention(b, s.q, out=out)
    assert s.cache.get_error() == _abi.MOE_ERR_DEVICE_BOUNDS
    assert (out[r[1] + fit:r[2]] == 5).all()
    want, bound = ref.attention(table, [100, cap, 90], off, s.q[rows].double())
    assert ((out[rows].double() - want).abs() <= bound).all()


@pytest.mark.parametrize("offsets", [[0, 4, 2, 9], [0, 3, 6, 40], [-2, 3, 6, 9], [0, 2 ** 30, 6, 9]])
def test_offsets_out_of_range_write_nothing(kv8, offsets):
    """A sequence whose offsets contradict the call's rows: none of its positions is written, and no
    row of its own in the outputs."""
    from bit_expert_layer_gb300 import _abi
    s = Setup(kv8, [100, 80, 90], [3, 3, 3], seed=46)
    good = [0 <= a <= b <= s.t for a, b in zip(offsets, offsets[1:])]
    b = kv8.KV8Batch(s.batch.page_table, s.batch.lens, ints(offsets), 9)
    before = s.ref()
    s.cache.append(b, s.k, s.v)
    assert s.cache.get_error() == _abi.MOE_ERR_DEVICE_BOUNDS
    out = torch.full(s.q.shape, 5.0, dtype=torch.bfloat16, device="cuda")
    s.cache.attention(b, s.q, out=out)
    assert s.cache.get_error() == _abi.MOE_ERR_DEVICE_BOUNDS
    mine = torch.zeros(s.t, dtype=torch.bool, device="cuda")
    for i, ok in enumerate(good):
        pages = torch.tensor(s.table[i][s.table[i] >= 0], device="cuda").long()
        if ok:
            mine[offsets[i]:offsets[i + 1]] = True
        else:
            assert torch.equal(s.cache.k[pages], before.codes["k"][pages])
            assert torch.equal(s.cache.v_scale[pages].double(), before.scales["v"][pages])
    assert (out[~mine] == 5).all()


@pytest.mark.parametrize("new", [1, 4, 90])
def test_not_finite_queries_beside_zero_values(kv8, new):
    """Zero blocks of values among others, of small and of large scales: the other rows keep their bits."""
    s = Setup(kv8, [200, 130], [new, new], seed=47)
    c = s.cache
    c.v[:, :, 16:32] = 0
    c.v_scale[:, :, 1] = 2.0 ** -100
    for high in (-9, 20):
        c.v_scale[:, :, 0] = 2.0 ** high
        a = c.attention(s.batch, s.q)
        q = s.q.clone()
        q[new - 1, 3, 5] = math.nan
        q[2 * new - 1, 8, 0] = -math.inf
        b = c.attention(s.batch, q)
        keep = torch.ones(2 * new, 16, dtype=torch.bool, device="cuda")
        keep[new - 1, 3] = keep[2 * new - 1, 8] = False
        assert torch.equal(a[keep], b[keep]) and torch.isnan(b[~keep]).all()
