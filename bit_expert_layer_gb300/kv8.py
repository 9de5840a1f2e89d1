"""Torch-facing wrappers of the 8-bit key/value cache (``include/gqa_kv8.h``): the paged
cache, the batch that every call describes its sequences with, and rotary positions.

One decode step of a model's attention::

    rope = kv8.Rope(head_size=128, rotary=128, theta=1e7)
    cache = kv8.KV8Cache.empty(n_pages=4096, fmt="e4m3")
    ws = cache.new_workspace(n_q_heads=16, max_new=1)
    batch = kv8.KV8Batch(page_table, lens, offsets, max_new=1)   # lens count the new tokens
    q, k = rope(q, k, positions)
    cache.append(batch, k, v)
    out = cache.attention(batch, q, workspace=ws)

PyTorch supplies device memory and streams only; each method is one C call on the current
stream of the tensors' device.  Tensors are checked here for type, shape, layout and device,
sizes and alignment by the library; a refused call raises before anything is enqueued.  What
only the device can see is collected in the cache's error word (``get_error``).
"""
from __future__ import annotations

import ctypes

import torch

from . import _abi
from ._abi import GqaKv8Batch, GqaKv8Cache

BLOCK = 16                                   # positions that share a scale
FORMATS = {"e4m3": _abi.GQA_KV8_E4M3, "int8": _abi.GQA_KV8_INT8}
_BF16 = torch.bfloat16
_empty, _current_device = torch.empty, torch.cuda.current_device


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

    def new_workspace(self, n_q_heads: int, max_new: int) -> torch.Tensor:
        """A zero-filled workspace for attention calls of up to max_new new tokens per sequence."""
        n = _abi.gqa_kv8_workspace_bytes(self._c, n_q_heads, max_new)
        if n == 0:
            raise ValueError("configuration refused")
        return torch.zeros(n, dtype=torch.uint8, device=self.device)

    def attention(self, batch: KV8Batch, q: torch.Tensor, scale: float = 0.0, out: torch.Tensor | None = None,
                  workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
        """Causal attention of the new tokens' queries (bf16 [T, n_q_heads, head_size]) over
        the cache, their own positions among it; scale 0 means 1 / sqrt(head_size).  The
        workspace is allocated for the call if none is given."""
        dev = self.device
        there = _elsewhere(dev, stream)
        if there is not None:
            with there:
                return self.attention(batch, q, scale, out, workspace)
        shape = q.shape
        heads = shape[1] if len(shape) == 3 else 0
        qs = _rows(q, "q", heads, self.head_size, dev)
        if out is None:
            out = _empty(shape, dtype=_BF16, device=dev)
        elif out.shape != shape or out.dtype is not _BF16 or out.device != dev or not out.is_contiguous():
            raise ValueError("out: a contiguous bfloat16 tensor of q's shape is wanted")
        if workspace is None:
            workspace = self.new_workspace(heads, batch.max_new)
        elif workspace.device != dev or not workspace.is_contiguous():
            raise ValueError(f"workspace: a contiguous tensor on {dev} is wanted")
        _abi.gqa_kv8_attention(self._c, self._batch(batch, shape[0]), q.data_ptr(), qs, heads, scale, out.data_ptr(),
                               workspace.data_ptr(), workspace.nbytes, _handle(dev.index))
        return out

    def get_error(self) -> int:
        """Synchronises, then reads and clears the error word (a status of ``_abi.STATUS``)."""
        with torch.cuda.device(self.device):
            return _abi.gqa_kv8_get_error(self._c)


class Rope(_Fixed):
    """Rotary positions: pair j (elements j and j + rotary / 2 of a head) turns by
    pos[axis(j)] * inv_freq[j].  ``sections`` gives each axis its number of pairs (one axis
    by default); ``cyclic`` deals the pairs out to the axes in turn instead of in runs."""

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
        _abi.gqa_rope(self._plan, q.data_ptr(), qs, hq, kp, ks, hk, pos.data_ptr(), t, qo.data_ptr(), qos,
                      0 if ko is None else ko.data_ptr(), kos, _handle(dev.index))
        return qo, ko
