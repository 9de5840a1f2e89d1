"""Torch-facing wrappers of the 8-bit key/value cache (``include/gqa_kv8.h``): the paged
cache, the batch that every call describes its sequences with, page tables built on the
device, and rotary positions with or without norms of the heads.

One decode step of a model's attention::

    rope = kv8.Rope(head_size=128, rotary=128, theta=1e7)
    cache = kv8.KV8Cache.empty(n_pages=4096, fmt="e4m3")
    ws = cache.new_workspace(n_q_heads=16, max_new=1)
    batch = kv8.KV8Batch(page_table, lens, offsets, max_new=1)   # lens count the new tokens
    q, k = rope(q, k, positions)
    cache.append(batch, k, v)
    out = cache.attention(batch, q, workspace=ws)

with ``window=`` and ``sinks=`` for a sliding window, or ``prefix=KV8Prefix(groups, shared, max_shared)``
where sequences begin alike.  A server's step begins with its page tables::

    pages = kv8.KV8Pages.all_free(n_pages, page_size=64, n_seqs=64, max_pages=512)
    offsets, positions, slots = pages.step(new, n_tokens)        # new: int32 [n_seqs], on the device
    batch = kv8.KV8Batch(pages.table, pages.lens, offsets, max_new)

PyTorch supplies device memory and streams only; each method is one C call on the current
stream of the tensors' device.  Tensors are checked here for type, shape, layout and device,
sizes and alignment by the library; a refused call raises before anything is enqueued.  What
only the device can see is collected in the cache's error word (``get_error``).
"""
from __future__ import annotations

import ctypes

import torch

from . import _abi
from ._abi import GqaKv8Batch, GqaKv8Cache, GqaKv8Pages, GqaKv8PagesState, GqaKv8Prefix, GqaNorm

BLOCK = 16                                   # positions that share a scale
FORMATS = {"e4m3": _abi.GQA_KV8_E4M3, "int8": _abi.GQA_KV8_INT8}
_BF16 = torch.bfloat16
_empty, _current_device = torch.empty, torch.cuda.current_device
_INT = torch.int32


def _elsewhere(device: torch.device, stream):
    """None where `device` and the stream to use are the current ones; else what makes them so
    for a call, so that what the call allocates belongs to the stream that uses it."""
    if stream is not None:
        if stream.device != device:
            raise ValueError(f"the stream is on {stream.device}, the tensors on {device}")
        return torch.cuda.stream(stream)
    return None if device.index == _current_device() else torch.cuda.device(device)


def _handle(index: int) -> int:
    """The current stream's handle (torch.cuda.current_stream takes 2 us to wrap it)."""
    return torch._C._cuda_getCurrentRawStream(index)


def _rows(x: torch.Tensor, name: str, heads: int, head_size: int, device) -> int:
    """The row stride of a [T, heads, head_size] tensor whose rows are contiguous."""
    shape = x.shape
    if x.dtype is not _BF16 or len(shape) != 3 or x.device != device:
        raise ValueError(f"{name}: a 3-dimensional bfloat16 tensor on {device} is wanted")
    t, h, d = shape
    if h != heads or d != head_size:
        raise ValueError(f"{name}: shape [T, {heads}, {head_size}] is wanted, got {list(shape)}")
    st, sh, sd = x.stride()
    if (sd != 1 and d > 1) or (sh != d and h > 1):
        raise ValueError(f"{name}: the heads of a row have to be contiguous")
    return st if t > 1 else h * d


def _ints(x: torch.Tensor, name: str, dim: int, device=None) -> torch.Tensor:
    if x.dtype != torch.int32 or x.dim() != dim or not x.is_contiguous() or not x.is_cuda or \
            (device is not None and x.device != device):
        raise ValueError(f"{name}: a contiguous {dim}-dimensional int32 CUDA tensor"
                         f"{'' if device is None else f' on {device}'} is wanted")
    return x


class _Fixed:
    """Attributes are set once: the C description made from them would not follow."""

    def __setattr__(self, name, value):
        if name in self.__dict__:
            raise AttributeError(f"{name} is fixed; make a new {type(self).__name__}, or change its tensor in place")
        self.__dict__[name] = value


class KV8Batch(_Fixed):
    """The sequences of a call: ``page_table`` int32 [n_seqs, max_pages], ``lens`` int32
    [n_seqs] (cached positions, the call's tokens among them), ``offsets`` int32
    [n_seqs + 1] (sequence b's tokens are rows offsets[b] .. offsets[b + 1] - 1), and
    ``max_new``, a bound on the new tokens of one sequence.  The tensors stay on the device
    and may be changed in place between calls, also under a captured graph."""

    def __init__(self, page_table: torch.Tensor, lens: torch.Tensor, offsets: torch.Tensor, max_new: int):
        self.page_table = _ints(page_table, "page_table", 2)
        self.device = page_table.device
        self.lens = _ints(lens, "lens", 1, self.device)
        self.offsets = _ints(offsets, "offsets", 1, self.device)
        n = page_table.shape[0]
        if lens.shape[0] != n or offsets.shape[0] != n + 1:
            raise ValueError(f"page_table has {n} rows: lens has to have {n} entries and offsets {n + 1}")
        self.max_new = int(max_new)
        self._c = {}

    def c(self, n_tokens: int):
        """The C description (by reference) for token tensors of n_tokens rows."""
        ref = self._c.get(n_tokens)
        if ref is None:
            c = GqaKv8Batch(self.page_table.data_ptr(), self.lens.data_ptr(), self.offsets.data_ptr(),
                            self.page_table.shape[0], self.page_table.shape[1], n_tokens, self.max_new)
            ref = ctypes.byref(c)
            self._c.clear()
            self._c[n_tokens] = ref
        return ref


class KV8Prefix(_Fixed):
    """Sequences that begin alike: sequences ``groups[i]`` .. ``groups[i + 1] - 1`` share their first
    ``shared[i]`` positions (int32 [n_groups + 1] and [n_groups], on the device; they may be
    changed in place between calls, also under a captured graph).  ``max_shared`` is a bound on the
    shared lengths, by which a call decides whether sharing pays.  Give it where it is known: without
    it (0) a call counts on what a row of the batch's page table holds, and where much less is shared
    it takes some 9 us more than without a prefix (short prompts up to twice as long).  Give the
    groups that there are, too, not a list padded with empty ones: each counts as work."""

    def __init__(self, groups: torch.Tensor, shared: torch.Tensor, max_shared: int = 0):
        self.groups = _ints(groups, "groups", 1)
        self.device = groups.device
        self.shared = _ints(shared, "shared", 1, self.device)
        n = shared.shape[0]
        if n < 1 or groups.shape[0] != n + 1:
            raise ValueError(f"shared has {n} entries: one at least is wanted, and groups has to have {n + 1}")
        self.max_shared = int(max_shared)
        if not 0 <= self.max_shared <= 1 << 24:
            raise ValueError(f"max_shared {max_shared}: 0 .. 2^24 is wanted")
        self._c = ctypes.byref(GqaKv8Prefix(groups.data_ptr(), shared.data_ptr(), n, self.max_shared))


class KV8Pages(_Fixed):
    """Which pages of a pool each sequence holds, kept on the device: ``table`` int32 [n_seqs,
    max_pages], ``free`` int32 [n_pages] (a stack), and the state that a step changes: ``lens``
    int32 [n_seqs] (cached positions), ``held`` int32 [n_seqs] (pages in the sequence's row)
    and ``n_free`` int32 [1].  Sequences that begin with pages of another one's (a shared
    prefix) say how many in ``borrowed`` int32 [n_seqs]; those are not given back, and new tokens
    have to begin behind them: a sequence whose tokens do not is recorded and done.  Lower its entry
    (in place) after a step that keeps less than them, and after the one that ends it.  ``control``
    is the pool's error word and a ticket, zero at first (made here if it is not given)."""

    def __init__(self, table: torch.Tensor, free: torch.Tensor, page_size: int, lens: torch.Tensor, held: torch.Tensor,
                 n_free: torch.Tensor, borrowed: torch.Tensor | None = None, control: torch.Tensor | None = None):
        self.table = _ints(table, "table", 2)
        self.device = dev = table.device
        n = table.shape[0]
        self.free, self.lens, self.held = _ints(free, "free", 1, dev), _ints(lens, "lens", 1, dev), _ints(held, "held", 1, dev)
        self.n_free = _ints(n_free, "n_free", 1, dev)
        self.borrowed = None if borrowed is None else _ints(borrowed, "borrowed", 1, dev)
        for name, x, m in (("lens", lens, n), ("held", held, n), ("n_free", n_free, 1), ("borrowed", borrowed, n)):
            if x is not None and x.shape[0] != m:
                raise ValueError(f"{name}: {m} entries are wanted, got {x.shape[0]}")
        self.page_size = int(page_size)
        self.control = torch.zeros(2, dtype=_INT, device=dev) if control is None else control
        words = self.control.view(_INT) if self.control.dtype is torch.uint32 else self.control
        if _ints(words, "control", 1, dev).shape[0] < 2:
            raise ValueError(f"control: 2 entries are wanted, got {words.shape[0]}")
        self._pages = ctypes.byref(GqaKv8Pages(table.data_ptr(), free.data_ptr(), self.control.data_ptr(), n, table.shape[1],
                                               free.shape[0], self.page_size))
        self._state = ctypes.byref(GqaKv8PagesState(lens.data_ptr(), held.data_ptr(), n_free.data_ptr()))

    @classmethod
    def all_free(cls, n_pages: int, page_size: int = 64, n_seqs: int = 64, max_pages: int = 512, device="cuda") -> "KV8Pages":
        """A pool of which no page is held; the first to be taken is page 0."""
        zeros = lambda *s: torch.zeros(s, dtype=_INT, device=device)  # noqa: E731
        free = torch.arange(n_pages - 1, -1, -1, dtype=_INT, device=device)
        return cls(zeros(n_seqs, max_pages), free, page_size, zeros(n_seqs), zeros(n_seqs), zeros(1) + n_pages)

    def fork(self) -> "KV8Pages":
        """Another state over the same table and free list, equal to this one for now: for
        ``step(into=...)``.  Only steps from one of them may follow once it has been stepped in place."""
        return KV8Pages(self.table, self.free, self.page_size, self.lens.clone(), self.held.clone(), self.n_free.clone(),
                        self.borrowed, self.control)

    def step(self, new: torch.Tensor, n_tokens: int, keep: torch.Tensor | None = None, out=None,
             into: "KV8Pages | None" = None, stream=None):
        """Every sequence keeps its first ``keep`` positions (int32 [n_seqs]; None: all; 0: it is
        done, and gives its pages back), adds ``new`` tokens (int32 [n_seqs]) and gets the pages
        for them.  Writes the state after it into ``into`` (None: in place) and returns
        (offsets [n_seqs + 1], positions [n_tokens], slots [n_tokens]), int32; rows at or past
        offsets[n_seqs] are left as they were.  A slot is page * page_size + place in the page,
        -1 for a token without a page (the free list ran out, which ``get_error`` tells)."""
        dev = self.device
        there = _elsewhere(dev, stream)
        if there is not None:
            with there:
                return self.step(new, n_tokens, keep, out, into)
        n = self.table.shape[0]
        if _ints(new, "new", 1, dev).shape[0] != n or (keep is not None and _ints(keep, "keep", 1, dev).shape[0] != n):
            raise ValueError(f"new, keep: {n} entries are wanted")
        if into is None:
            into = self
        elif into.table is not self.table or into.free is not self.free:
            raise ValueError("into: a fork of these pages is wanted")
        if out is None:
            out = (_empty(n + 1, dtype=_INT, device=dev), _empty(n_tokens, dtype=_INT, device=dev),
                   _empty(n_tokens, dtype=_INT, device=dev))
        else:
            for name, x, m in zip(("offsets", "positions", "slots"), out, (n + 1, n_tokens, n_tokens)):
                if _ints(x, name, 1, dev).shape[0] != m:
                    raise ValueError(f"{name}: {m} entries are wanted")
        _abi.gqa_kv8_pages_step(self._pages, self._state, into._state, 0 if keep is None else keep.data_ptr(),
                                new.data_ptr(), 0 if self.borrowed is None else self.borrowed.data_ptr(), out[0].data_ptr(),
                                out[1].data_ptr(), out[2].data_ptr(), n_tokens, _handle(dev.index))
        return out

    def get_error(self) -> int:
        """Synchronises, then reads and clears the pool's error word (a status of ``_abi.STATUS``)."""
        with torch.cuda.device(self.device):
            return _abi.gqa_kv8_pages_get_error(self._pages)


class KV8Cache(_Fixed):
    """A paged 8-bit cache over caller-owned tensors: ``k``, ``v`` one byte per number
    [n_pages, n_kv_heads, page_size, head_size], ``k_scale``, ``v_scale`` float32
    [n_pages, n_kv_heads, page_size / 16]."""

    def __init__(self, k: torch.Tensor, v: torch.Tensor, k_scale: torch.Tensor, v_scale: torch.Tensor,
                 fmt: str = "e4m3"):
        if fmt not in FORMATS:
            raise ValueError(f"format {fmt!r}: one of {sorted(FORMATS)} is wanted")
        if k.dim() != 4 or k.shape[2] % BLOCK:
            raise ValueError("k: [n_pages, n_kv_heads, page_size, head_size] is wanted, page_size a multiple of 16")
        for name, x in (("k", k), ("v", v)):
            if x.element_size() != 1 or x.shape != k.shape or not x.is_contiguous() or x.device != k.device or \
                    not x.is_cuda:
                raise ValueError(f"{name}: a contiguous CUDA tensor of bytes of k's shape is wanted")
        scales = (k.shape[0], k.shape[1], k.shape[2] // BLOCK)
        for name, x in (("k_scale", k_scale), ("v_scale", v_scale)):
            if x.dtype != torch.float32 or tuple(x.shape) != scales or not x.is_contiguous() or x.device != k.device:
                raise ValueError(f"{name}: a contiguous float32 tensor of shape {list(scales)} on {k.device} is wanted")
        self.k, self.v, self.k_scale, self.v_scale, self.fmt = k, v, k_scale, v_scale, fmt
        self.device = k.device
        self.n_pages, self.n_kv_heads, self.page_size, self.head_size = k.shape
        self.error = torch.zeros(1, dtype=torch.int32, device=k.device)
        self._c = ctypes.byref(GqaKv8Cache(
            k.data_ptr(), v.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(), self.error.data_ptr(), self.n_pages,
            self.page_size, self.n_kv_heads, self.head_size, FORMATS[fmt]))

    @classmethod
    def empty(cls, n_pages: int, n_kv_heads: int = 2, page_size: int = 64, head_size: int = 128, fmt: str = "e4m3",
              device="cuda") -> "KV8Cache":
        shape = (n_pages, n_kv_heads, page_size, head_size)
        k, v = (torch.zeros(shape, dtype=torch.uint8, device=device) for _ in range(2))
        ks, vs = (torch.ones(shape[:2] + (page_size // BLOCK,), dtype=torch.float32, device=device) for _ in range(2))
        return cls(k, v, ks, vs, fmt)

    def _batch(self, batch: KV8Batch, n_tokens: int):
        if batch.device != self.device:
            raise ValueError(f"the batch is on {batch.device}, the cache on {self.device}")
        return batch.c(n_tokens)

    def append(self, batch: KV8Batch, k: torch.Tensor, v: torch.Tensor, stream=None) -> None:
        """Quantise the new tokens' keys and values (bf16 [T, n_kv_heads, head_size], rows may
        be slices of a wider tensor) and write them into the cache."""
        dev = self.device
        there = _elsewhere(dev, stream)
        if there is not None:
            with there:
                return self.append(batch, k, v)
        ks = _rows(k, "k", self.n_kv_heads, self.head_size, dev)
        vs = _rows(v, "v", self.n_kv_heads, self.head_size, dev)
        t = k.shape[0]
        if v.shape[0] != t:
            raise ValueError(f"k has {t} rows and v {v.shape[0]}")
        _abi.gqa_kv8_append(self._c, self._batch(batch, t), k.data_ptr(), ks, v.data_ptr(), vs, _handle(dev.index))

    def gather(self, batch: KV8Batch, n_tokens: int, out=None, stream=None):
        """The batch's rows read back: (k, v), bf16 [n_tokens, n_kv_heads, head_size].  Rows at
        or past offsets[n_seqs] stay as they are."""
        dev = self.device
        there = _elsewhere(dev, stream)
        if there is not None:
            with there:
                return self.gather(batch, n_tokens, out)
        if out is None:
            shape = (n_tokens, self.n_kv_heads, self.head_size)
            out = (_empty(shape, dtype=_BF16, device=dev), _empty(shape, dtype=_BF16, device=dev))
        else:
            for name, x in zip(("k_out", "v_out"), out):
                _rows(x, name, self.n_kv_heads, self.head_size, dev)
                if x.shape[0] != n_tokens or not x.is_contiguous():
                    raise ValueError(f"{name}: a contiguous tensor of {n_tokens} rows is wanted")
        _abi.gqa_kv8_gather(self._c, self._batch(batch, n_tokens), out[0].data_ptr(), out[1].data_ptr(),
                            _handle(dev.index))
        return out

    def new_workspace(self, n_q_heads: int, max_new: int, prefix_tokens: int = 0) -> torch.Tensor:
        """A zero-filled workspace for attention calls of up to max_new new tokens per sequence; for calls
        with a prefix, of up to prefix_tokens tokens in all."""
        n = _abi.gqa_kv8_prefix_workspace_bytes(self._c, n_q_heads, max_new, prefix_tokens) if prefix_tokens else \
            _abi.gqa_kv8_workspace_bytes(self._c, n_q_heads, max_new)
        if n == 0:
            raise ValueError("configuration refused")
        return torch.zeros(n, dtype=torch.uint8, device=self.device)

    def attention(self, batch: KV8Batch, q: torch.Tensor, scale: float = 0.0, out: torch.Tensor | None = None,
                  workspace: torch.Tensor | None = None, stream=None, *, window: int | None = None, sinks: int = 0,
                  prefix: KV8Prefix | None = None) -> torch.Tensor:
        """Causal attention of the new tokens' queries (bf16 [T, n_q_heads, head_size]) over
        the cache, their own positions among it; scale 0 means 1 / sqrt(head_size).  The
        workspace is allocated for the call if none is given.

        With ``window`` a token sees the last `window` positions, its own among them, and its
        sequence's first ``sinks``.  With ``prefix`` the positions that sequences share are
        worked on once for all of them (see ``KV8Prefix``; the workspace is then one for
        ``prefix_tokens``); not together with a window."""
        dev = self.device
        there = _elsewhere(dev, stream)
        if there is not None:
            with there:
                return self.attention(batch, q, scale, out, workspace, window=window, sinks=sinks, prefix=prefix)
        if window is None and sinks or window is not None and prefix is not None:
            raise ValueError("sinks go with a window, and a prefix without one")
        shape = q.shape
        heads = shape[1] if len(shape) == 3 else 0
        qs = _rows(q, "q", heads, self.head_size, dev)
        if out is None:
            out = _empty(shape, dtype=_BF16, device=dev)
        elif out.shape != shape or out.dtype is not _BF16 or out.device != dev or not out.is_contiguous():
            raise ValueError("out: a contiguous bfloat16 tensor of q's shape is wanted")
        if workspace is None:
            workspace = self.new_workspace(heads, batch.max_new, 0 if prefix is None else shape[0])
        elif workspace.device != dev or not workspace.is_contiguous():
            raise ValueError(f"workspace: a contiguous tensor on {dev} is wanted")
        c, where = self._batch(batch, shape[0]), (out.data_ptr(), workspace.data_ptr(), workspace.nbytes, _handle(dev.index))
        if window is not None:
            _abi.gqa_kv8_window_attention(self._c, c, q.data_ptr(), qs, heads, scale, window, sinks, *where)
        elif prefix is not None:
            if prefix.device != dev:
                raise ValueError(f"the prefix is on {prefix.device}, the cache on {dev}")
            _abi.gqa_kv8_prefix_attention(self._c, c, prefix._c, q.data_ptr(), qs, heads, scale, *where)
        else:
            _abi.gqa_kv8_attention(self._c, c, q.data_ptr(), qs, heads, scale, *where)
        return out

    def get_error(self) -> int:
        """Synchronises, then reads and clears the error word (a status of ``_abi.STATUS``)."""
        with torch.cuda.device(self.device):
            return _abi.gqa_kv8_get_error(self._c)


class Rope(_Fixed):
    """Rotary positions: pair j (elements j and j + rotary / 2 of a head) turns by
    pos[axis(j)] * inv_freq[j].  ``sections`` gives each axis its number of pairs (one axis
    by default); ``cyclic`` deals the pairs out to the axes in turn instead of in runs."""

    _norm = None

    def __init__(self, head_size: int = 128, rotary: int | None = None, theta: float = 10000.0, inv_freq=None,
                 sections=None, cyclic: bool = False):
        self.plan = _abi.gqa_rope_plan_init(head_size, head_size if rotary is None else rotary, theta, inv_freq,
                                            sections, cyclic)
        self.head_size, self.n_axes = self.plan.head_size, self.plan.n_axes
        self._plan = ctypes.byref(self.plan)

    def __call__(self, q: torch.Tensor, k: torch.Tensor | None, pos: torch.Tensor, out=None, stream=None):
        """q, k: bf16 [T, heads, head_size] (rows may be slices of a wider tensor; k may be
        None); pos: int32 [n_axes, T], or [T] with one axis; out: (q_out, k_out), which may
        be q and k themselves.  Returns (q_out, k_out)."""
        dev, d, shape, at = q.device, self.head_size, q.shape, pos.shape
        if not q.is_cuda or len(shape) != 3:
            raise ValueError("q: a 3-dimensional bfloat16 CUDA tensor is wanted")
        there = _elsewhere(dev, stream)
        if there is not None:
            with there:
                return self(q, k, pos, out)
        t, hq, _ = shape
        hk = ks = kp = 0
        qs = _rows(q, "q", hq, d, dev)
        if k is not None:
            if k.dim() != 3 or k.shape[0] != t:
                raise ValueError(f"k: [{t}, heads, {d}] is wanted")
            hk, kp = k.shape[1], k.data_ptr()
            ks = _rows(k, "k", hk, d, dev)
        if at != (self.n_axes, t) and (self.n_axes != 1 or at != (t,)):
            raise ValueError(f"pos: shape [{self.n_axes}, {t}] is wanted, got {list(at)}")
        if pos.dtype is not torch.int32 or pos.device != dev or not pos.is_contiguous():
            raise ValueError(f"pos: a contiguous int32 tensor on {dev} is wanted")
        qos, kos = hq * d, hk * d
        if out is None:
            qo = _empty((t, hq, d), dtype=_BF16, device=dev)
            ko = None if k is None else _empty((t, hk, d), dtype=_BF16, device=dev)
        else:
            qo, ko = out
            if (k is None) != (ko is None) or qo.shape != q.shape or (k is not None and ko.shape != k.shape):
                raise ValueError("out: tensors of q's and k's shapes are wanted")
            qos = _rows(qo, "q_out", hq, d, dev)
            if ko is not None:
                kos = _rows(ko, "k_out", hk, d, dev)
        args = (q.data_ptr(), qs, hq, kp, ks, hk, pos.data_ptr(), t, qo.data_ptr(), qos, 0 if ko is None else ko.data_ptr(),
                kos, _handle(dev.index))
        if self._norm is None:
            _abi.gqa_rope(self._plan, *args)
        else:
            if self._norm_device is not None and self._norm_device != dev:
                raise ValueError(f"the weights are on {self._norm_device}, q on {dev}")
            _abi.gqa_norm_rope(self._plan, self._norm, *args)
        return qo, ko


class NormRope(Rope):
    """Norms of the heads and rotary positions in one pass: every head x of q and k becomes
    x / sqrt(mean(x^2) + eps) * (weight + offset), with q's and k's own weights ([head_size], both
    bf16 or both fp32; None: ones), and turns as ``rope`` has it.  Called as a Rope."""

    def __init__(self, rope: Rope, q_weight: torch.Tensor | None = None, k_weight: torch.Tensor | None = None,
                 eps: float = 1e-6, offset: float = 0.0):
        given = [w for w in (q_weight, k_weight) if w is not None]
        for w in given:
            if w.dtype not in (_BF16, torch.float32) or w.dtype != given[0].dtype or w.device != given[0].device or \
                    not w.is_cuda or w.shape != (rope.head_size,) or not w.is_contiguous():
                raise ValueError(f"weights: contiguous bfloat16 or float32 CUDA tensors of [{rope.head_size}], alike, are wanted")
        if not 0.0 <= eps <= 1e30 or not abs(offset) <= 1e30:
            raise ValueError(f"eps {eps}, offset {offset}: finite numbers are wanted, eps 0 at least")
        self.plan, self._plan, self.head_size, self.n_axes = rope.plan, rope._plan, rope.head_size, rope.n_axes
        self.q_weight, self.k_weight, self.eps, self.offset = q_weight, k_weight, float(eps), float(offset)
        self._norm_device = given[0].device if given else None
        self._norm = ctypes.byref(GqaNorm(0 if q_weight is None else q_weight.data_ptr(),
                                          0 if k_weight is None else k_weight.data_ptr(),
                                          1 if given and given[0].dtype is torch.float32 else 0, eps, offset))
