"""ctypes binding of latent attention (C ABI in ``include/moe_w4a8_latent.h``).

The attention operators of a layer that keeps one latent vector per token for
all heads: its norm, the rotations and the store of its row in a paged cache
(``moe_w4a8_latent_append``), and causal attention of a ragged batch over such
rows in the absorbed form (``moe_w4a8_latent_attention``).  Argument
marshalling only, as in ``attention``.
"""
from __future__ import annotations

import ctypes

import torch

from . import binding
from .attention import _DTYPES, HeadPrep, _aligned, _device, _stream
from .binding import MoeError, alloc_workspace

_lib = None


class _LatentBatch(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int64) for n in (
        "n_seqs", "n_heads", "latent_dim", "rot_dim", "page_size", "n_pages", "table_width", "max_q_len", "max_kv_len", "dtype",
        "page_stride", "row_stride")]
    _fields_ += [(n, ctypes.c_void_p) for n in ("cache", "block_table", "q_start", "kv_len")]


def _load():
    global _lib
    if _lib is None:
        lib = binding._load()
        p, i64, sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_size_t
        lib.moe_w4a8_latent_append.argtypes = [p, p, i64, p, i64, p, i64, p, i64, i64, p, i64, i64, p]
        lib.moe_w4a8_latent_append.restype = ctypes.c_int
        lib.moe_w4a8_latent_attention_workspace_size.argtypes = [p]
        lib.moe_w4a8_latent_attention_workspace_size.restype = sz
        lib.moe_w4a8_latent_attention.argtypes = [p, i64, p, i64, i64, p, i64, i64, p, ctypes.c_float, p, sz, p]
        lib.moe_w4a8_latent_attention.restype = ctypes.c_int
        _lib = lib
    return _lib


class LatentBatch:
    """A paged cache of latent rows and the ragged batch that uses it.

    cache: [pages, page_size, latent_dim + rot_dim], bf16 or fp16, any page and row strides that are multiples of 16 bytes; the
    last rot_dim components of a row are the key part that carries the position.  block_table [seqs, width], q_start
    [seqs + 1], kv_len [seqs]: contiguous int32 CUDA tensors, whose contents may change from call to call (the handle reads
    none of them on the host).  max_q_len and max_kv_len bound the batch's lengths (default for the latter: all that a row
    of the table can hold); they choose a kernel and a launch size, not the result.
    """

    def __init__(self, cache, block_table, q_start, kv_len, n_heads: int, latent_dim: int, max_q_len: int, max_kv_len: int | None = None):
        if cache.dtype not in _DTYPES:
            raise TypeError(f"cache: dtype {cache.dtype}, expected torch.bfloat16 or torch.float16")
        if not cache.is_cuda:
            raise ValueError("cache must be a CUDA tensor")
        if cache.dim() != 3:
            raise ValueError(f"cache: shape {tuple(cache.shape)}, expected [pages, page_size, latent_dim + rot_dim]")
        if cache.stride(2) != 1:
            raise ValueError("cache: the components of a row must be contiguous")
        pages, page, row = cache.shape
        if not 0 < latent_dim <= row:
            raise ValueError(f"latent_dim {latent_dim} of rows of {row} components")
        if block_table.dim() != 2:
            raise ValueError("block_table must be [seqs, width]")
        seqs, width = block_table.shape
        binding._need(block_table, "block_table", torch.int32)
        binding._need(q_start, "q_start", torch.int32, (seqs + 1,))
        binding._need(kv_len, "kv_len", torch.int32, (seqs,))
        self.device = binding._one_device("LatentBatch", (cache, block_table, q_start, kv_len))
        self._index = self.device.index
        self.dtype = cache.dtype
        self.n_heads, self.latent_dim, self.rot_dim = int(n_heads), int(latent_dim), row - int(latent_dim)
        self.cache = cache
        self.block_table, self.q_start, self.kv_len = block_table, q_start, kv_len
        if max_kv_len is None:
            max_kv_len = max(1, width * page)
        # (a stride over a single page or row says nothing)
        row_stride = cache.stride(1) if page > 1 else (row + 7) // 8 * 8
        page_stride = cache.stride(0) if pages > 1 else 0
        self._c = _LatentBatch(seqs, n_heads, latent_dim, self.rot_dim, page, pages, width, max_q_len, max_kv_len, _DTYPES[self.dtype],
                               page_stride, row_stride, cache.data_ptr(), block_table.data_ptr(), q_start.data_ptr(), kv_len.data_ptr())
        self._p = ctypes.addressof(self._c)
        self._prep = None  # the HeadPrep that was found to fit
        lib = _load()
        if _device() == self._index:
            self._workspace = lib.moe_w4a8_latent_attention_workspace_size(self._p)
        else:
            with torch.cuda.device(self._index):
                self._workspace = lib.moe_w4a8_latent_attention_workspace_size(self._p)
        if self._workspace == 0:  # sizes or strides that the operators refuse
            raise MoeError("moe_w4a8_latent_attention_workspace_size", 1)

    @property
    def max_q_len(self) -> int:
        """The bound on a sequence's new tokens.  May be set between calls: it is a hint to the next one."""
        return self._c.max_q_len

    @max_q_len.setter
    def max_q_len(self, n: int):
        if n < 1:
            raise ValueError(f"max_q_len {n}: at least 1")
        self._c.max_q_len = n

    def workspace_size(self) -> int:
        """Bytes of workspace of moe_w4a8_latent_attention for this batch, whatever its tokens."""
        return self._workspace

    def alloc_workspace(self) -> torch.Tensor:
        return alloc_workspace(self.workspace_size(), self.device)

    def _refuse(self, t, name, shape):
        """Why `t` is not a tensor of this batch of that shape."""
        if t is None:
            raise ValueError(f"{name} is required")
        if t.dtype is not self.dtype:
            raise TypeError(f"{name}: dtype {t.dtype}, expected {self.dtype}")
        if t.device != self.device:
            raise ValueError(f"{name} is on {t.device}, the cache on {self.device}")
        if t.shape != shape:
            raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {shape}")
        raise ValueError(f"{name}: its last dimension must be contiguous")

    def _rows2(self, t, name, shape):
        """(address, token stride) of a tensor of this batch."""
        # (one test on the way of every call; what was wrong is found out in _refuse)
        if t is not None and t.shape == shape and t.dtype is self.dtype and t.get_device() == self._index:
            ts, es = t.stride()
            if es == 1:
                return t.data_ptr(), ts
        self._refuse(t, name, shape)

    def _rows3(self, t, name, shape):
        """(address, token stride, head stride) of a tensor of this batch."""
        if t is not None and t.shape == shape and t.dtype is self.dtype and t.get_device() == self._index:
            ts, hs, es = t.stride()
            if es == 1:
                return t.data_ptr(), ts, hs
        self._refuse(t, name, shape)


def _enqueue(fn: str, index: int, *args):
    """Calls `fn` with `args` and the current stream of device `index`, with that device current."""
    with torch.cuda.device(index):
        status = getattr(_load(), fn)(*args, _stream(index))
    if status != 0:
        raise MoeError(fn, status)


def _fit(batch: LatentBatch, prep: HeadPrep):
    """Whether a HeadPrep goes with a batch, looked at once for the two."""
    if prep._index >= 0 and prep._index != batch._index:
        raise ValueError(f"HeadPrep is on {prep.device}, the cache on {batch.device}")
    if prep.q_weight is not None:
        raise ValueError("latent queries have no norm of their own: q_weight must be None")
    if prep.k_weight is not None and prep.k_weight.numel() != batch.latent_dim:
        raise ValueError(f"a norm weight of {prep.k_weight.numel()} components, latent vectors of {batch.latent_dim}")
    if (0 if prep.cos_sin is None else prep.cos_sin.shape[1]) != batch.rot_dim:
        raise ValueError(f"the table of HeadPrep has to be as wide as the key part, {batch.rot_dim}")
    batch._prep = prep


def moe_w4a8_latent_append(batch: LatentBatch, prep: HeadPrep, latent, k_rot=None, q_rot=None, q_rot_out=None):
    """Norms the latent vectors, turns the key parts and the queries' rotated parts, stores the rows in the cache.

    latent [tokens, latent_dim], k_rot [tokens, rot_dim] (with token strides: parts of one projection's rows), q_rot and
    q_rot_out [tokens, heads, rot_dim], any strides that are multiples of 16 bytes; q_rot_out may be q_rot.  prep: its
    k_weight [latent_dim] is the weight of the latent vector's norm (None: no norm), its table as wide as rot_dim.  A cache
    without a key part (rot_dim 0) takes latent alone.
    """
    n, rot = latent.shape[0], batch.rot_dim
    if batch._prep is not prep:
        _fit(batch, prep)
    if prep.positions is not None and prep.positions.shape != (n,):
        raise ValueError(f"positions: shape {tuple(prep.positions.shape)}, expected {(n,)}")
    row = batch._rows2(latent, "latent", (n, batch.latent_dim))
    if rot:
        heads = (n, batch.n_heads, rot)
        args = (batch._p, prep._p, n, *row, *batch._rows2(k_rot, "k_rot", (n, rot)), *batch._rows3(q_rot, "q_rot", heads),
                *batch._rows3(q_rot_out, "q_rot_out", heads))
    else:
        if not (k_rot is None and q_rot is None and q_rot_out is None):
            raise ValueError("rows without a key part: k_rot, q_rot and q_rot_out must be None")
        args = (batch._p, prep._p, n, *row, None, 0, None, 0, 0, None, 0, 0)
    if _lib is None or _device() != batch._index:
        _enqueue("moe_w4a8_latent_append", batch._index, *args)
    elif status := _lib.moe_w4a8_latent_append(*args, _stream(batch._index)):
        raise MoeError("moe_w4a8_latent_append", status)
    return q_rot_out


def moe_w4a8_latent_attention(batch: LatentBatch, q, out, lse=None, scale: float | None = None, *, workspace):
    """Causal attention of the batch's tokens over its cache of latent rows (which holds theirs already).

    q [tokens, heads, latent_dim + rot_dim], out [tokens, heads, latent_dim]; lse [tokens, heads] float32, the log-sum-exp of
    each row's scaled scores, or None; out and lse must not overlap q or the cache; scale defaults to (latent_dim + rot_dim)^-1/2, which is seldom what a model wants: its
    scale goes by the size of the heads before the absorption.  workspace: batch.alloc_workspace().
    """
    n, h, dc = q.shape[0], batch.n_heads, batch.latent_dim
    at = None
    if lse is not None:
        if lse.dtype is not torch.float32 or lse.shape != (n, h) or not lse.is_contiguous():
            raise ValueError(f"lse must be a contiguous float32 tensor of shape {(n, h)}")
        if lse.get_device() != batch._index:
            raise ValueError(f"lse is on {lse.device}, the cache on {batch.device}")
        at = lse.data_ptr()
    if workspace.get_device() != batch._index:
        raise ValueError(f"workspace is on {workspace.device}, the cache on {batch.device}")
    row = dc + batch.rot_dim
    args = (batch._p, n, *batch._rows3(q, "q", (n, h, row)), *batch._rows3(out, "out", (n, h, dc)), at, row ** -0.5 if scale is None else scale,
            *_aligned(workspace))
    if _lib is None or _device() != batch._index:
        _enqueue("moe_w4a8_latent_attention", batch._index, *args)
    elif status := _lib.moe_w4a8_latent_attention(*args, _stream(batch._index)):
        raise MoeError("moe_w4a8_latent_attention", status)
    return out
