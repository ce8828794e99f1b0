"""ctypes binding of the attention operators (C ABI in ``include/moe_w4a8_attention.h``).

The operators of a serving step that stand next to the routed experts: the
norms and the rotation of queries and keys with the store into a paged cache
(``moe_w4a8_kv_append``), and causal attention of a ragged batch over that
cache (``moe_w4a8_paged_attention``).  Argument marshalling only, as in
``binding``: tensors are checked and their addresses passed with the current
CUDA stream; every step runs in the library's kernels.
"""
from __future__ import annotations

import ctypes
import math

import torch

from . import binding
from .binding import MoeError, alloc_workspace  # noqa: F401

_DTYPES = {torch.bfloat16: 0, torch.float16: 1}
_lib = None
# the current device, and the handle of its current stream, without the objects torch.cuda makes of them
_device, _stream = torch._C._cuda_getDevice, torch._C._cuda_getCurrentRawStream


class _KVBatch(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int64) for n in (
        "n_seqs", "n_q_heads", "n_kv_heads", "head_dim", "page_size", "n_pages", "table_width", "max_q_len", "max_kv_len",
        "dtype", "k_page_stride", "k_row_stride", "k_head_stride", "v_page_stride", "v_row_stride", "v_head_stride")]
    _fields_ += [(n, ctypes.c_void_p) for n in ("k_cache", "v_cache", "block_table", "q_start", "kv_len")]


class _HeadPrep(ctypes.Structure):
    _fields_ = [("cos_sin", ctypes.c_void_p), ("table_rows", ctypes.c_int64), ("rot_dim", ctypes.c_int64),
                ("interleaved", ctypes.c_int64), ("q_weight", ctypes.c_void_p), ("k_weight", ctypes.c_void_p),
                ("positions", ctypes.c_void_p), ("eps", ctypes.c_float), ("weight_offset", ctypes.c_float)]


def _load():
    global _lib
    if _lib is None:
        lib = binding._load()
        p, i64, sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_size_t
        lib.moe_w4a8_kv_append.argtypes = [p, p, i64, p, i64, i64, p, i64, i64, p, i64, i64, p, i64, i64, p]
        lib.moe_w4a8_kv_append.restype = ctypes.c_int
        lib.moe_w4a8_paged_attention_workspace_size.argtypes = [p]
        lib.moe_w4a8_paged_attention_workspace_size.restype = sz
        lib.moe_w4a8_paged_attention.argtypes = [p, i64, p, i64, i64, p, i64, i64, p, ctypes.c_float, i64, p, sz, p]
        lib.moe_w4a8_paged_attention.restype = ctypes.c_int
        _lib = lib
    return _lib


def _check_cache(t, name):
    if t.dtype not in _DTYPES:
        raise TypeError(f"{name}: dtype {t.dtype}, expected torch.bfloat16 or torch.float16")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dim() != 4:
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected [pages, page_size, kv_heads, head_dim]")
    if t.stride(3) != 1:
        raise ValueError(f"{name}: the components of a head must be contiguous")


class KVBatch:
    """A paged key/value cache and the ragged batch that uses it.

    k_cache, v_cache: [pages, page_size, kv_heads, head_dim], bf16 or fp16, any page, row and head strides that are
    multiples of 16 bytes (a head-major cache is passed as its ``permute(0, 2, 1, 3)``).  block_table [seqs, width],
    q_start [seqs + 1], kv_len [seqs]: contiguous int32 CUDA tensors, whose contents may change from call to call (the
    handle reads none of them on the host).  max_q_len and max_kv_len bound the batch's lengths (default for the
    latter: all that a row of the table can hold); they choose a kernel and a launch size, not the result.  Where the
    table is wide and the batch's contexts are known to be short (below 768 positions, or 16 MB of cache in
    all), a max_kv_len that says so saves a call of few rows some microseconds.
    """

    def __init__(self, k_cache, v_cache, block_table, q_start, kv_len, n_q_heads: int, max_q_len: int,
                 max_kv_len: int | None = None):
        _check_cache(k_cache, "k_cache")
        _check_cache(v_cache, "v_cache")
        if v_cache.dtype != k_cache.dtype:
            raise TypeError(f"v_cache: dtype {v_cache.dtype}, expected {k_cache.dtype}")
        if v_cache.shape != k_cache.shape:
            raise ValueError(f"v_cache: shape {tuple(v_cache.shape)}, expected {tuple(k_cache.shape)}")
        pages, page, hkv, d = k_cache.shape
        if block_table.dim() != 2:
            raise ValueError("block_table must be [seqs, width]")
        seqs, width = block_table.shape
        binding._need(block_table, "block_table", torch.int32)
        binding._need(q_start, "q_start", torch.int32, (seqs + 1,))
        binding._need(kv_len, "kv_len", torch.int32, (seqs,))
        self.device = binding._one_device("KVBatch", (k_cache, v_cache, block_table, q_start, kv_len))
        self._index = self.device.index
        self.dtype = k_cache.dtype
        self.n_q_heads, self.n_kv_heads, self.head_dim = int(n_q_heads), hkv, d
        self.k_cache, self.v_cache = k_cache, v_cache
        self.block_table, self.q_start, self.kv_len = block_table, q_start, kv_len
        if max_kv_len is None:
            max_kv_len = max(1, width * page)
        ks, vs = k_cache.stride(), v_cache.stride()
        self._c = _KVBatch(seqs, n_q_heads, hkv, d, page, pages, width, max_q_len, max_kv_len, _DTYPES[self.dtype],
                           ks[0], ks[1], ks[2], vs[0], vs[1], vs[2], k_cache.data_ptr(), v_cache.data_ptr(),
                           block_table.data_ptr(), q_start.data_ptr(), kv_len.data_ptr())
        self._p = ctypes.addressof(self._c)
        lib = _load()
        if _device() == self._index:
            self._workspace = lib.moe_w4a8_paged_attention_workspace_size(self._p)
        else:
            with torch.cuda.device(self._index):
                self._workspace = lib.moe_w4a8_paged_attention_workspace_size(self._p)
        if self._workspace == 0:  # sizes or strides that the operators refuse
            raise MoeError("moe_w4a8_paged_attention_workspace_size", 1)

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
        """Bytes of workspace of moe_w4a8_paged_attention for this batch, whatever its tokens."""
        return self._workspace

    def alloc_workspace(self) -> torch.Tensor:
        return alloc_workspace(self.workspace_size(), self.device)

    def _rows(self, t, name, n, heads):
        """(address, token stride, head stride) of a [n, heads, head_dim] tensor of this batch."""
        # (one test on the way of every call; what was wrong is found out below)
        if t.shape == (n, heads, self.head_dim) and t.dtype is self.dtype and t.get_device() == self._index:
            ts, hs, es = t.stride()
            if es == 1:
                return t.data_ptr(), ts, hs
        if t.dtype is not self.dtype:
            raise TypeError(f"{name}: dtype {t.dtype}, expected {self.dtype}")
        if t.device != self.device:
            raise ValueError(f"{name} is on {t.device}, the cache on {self.device}")
        if t.shape != (n, heads, self.head_dim):
            raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {(n, heads, self.head_dim)}")
        raise ValueError(f"{name}: the components of a head must be contiguous")


class HeadPrep:
    """What moe_w4a8_kv_append does to the heads of queries and keys.

    cos_sin [positions, rot_dim] float32 (``rope_table``), or None for no rotation; its first rot_dim components of a
    head are turned, in pairs (i, i + rot_dim / 2), or (2i, 2i + 1) if interleaved.  q_weight, k_weight [head_dim]
    float32: weights of the root-mean-square norm of each head, or None for none; weight_offset is added to them (1 for
    weights held as their distance from one).  positions [tokens] int32: rows of cos_sin to use in place of the tokens'
    positions in the cache.
    """

    def __init__(self, cos_sin=None, interleaved: bool = False, q_weight=None, k_weight=None, eps: float = 1e-6,
                 weight_offset: float = 0.0, positions=None):
        rows, rot = 0, 0
        if cos_sin is not None:
            binding._need(cos_sin, "cos_sin", torch.float32)
            if cos_sin.dim() != 2:
                raise ValueError("cos_sin must be [positions, rot_dim]")
            rows, rot = cos_sin.shape
        for w, name in ((q_weight, "q_weight"), (k_weight, "k_weight")):
            if w is not None:
                binding._need(w, name, torch.float32)
                if w.dim() != 1:
                    raise ValueError(f"{name} must be [head_dim]")
        if positions is not None:
            binding._need(positions, "positions", torch.int32)
        given = tuple(t for t in (cos_sin, q_weight, k_weight, positions) if t is not None)
        self.device = binding._one_device("HeadPrep", given) if given else None
        self.cos_sin, self.q_weight, self.k_weight, self.positions = cos_sin, q_weight, k_weight, positions
        dims = {w.numel() for w in (q_weight, k_weight) if w is not None}
        if len(dims) > 1:
            raise ValueError(f"q_weight and k_weight of different sizes: {sorted(dims)}")
        self._weight_dim = dims.pop() if dims else 0
        self._index = self.device.index if given else -1
        at = [None if t is None else t.data_ptr() for t in (cos_sin, q_weight, k_weight, positions)]
        self._c = _HeadPrep(at[0], rows, rot, int(interleaved), at[1], at[2], at[3], eps, weight_offset)
        self._p = ctypes.addressof(self._c)


def rope_table(positions: int, rot_dim: int, base: float = 10000.0, device="cuda", scaling: str | None = None,
               factor: float = 1.0, original: int | None = None, beta_fast: float = 32.0, beta_slow: float = 1.0):
    """The table of HeadPrep: [positions, rot_dim] float32, cosines then sines, computed in 64 bits.

    Pair i turns by p * base^(-2i / rot_dim) at position p.  scaling for contexts longer than the trained ones:
    "linear" divides every angle by `factor`; "ntk" raises the base to base * factor^(rot_dim / (rot_dim - 2)), so that
    the slowest pair's angle is divided by `factor` and the fastest's stays; "yarn" divides the angle of a pair that
    makes less than `beta_slow` turns over the `original` context, keeps that of one that makes more than `beta_fast`
    turns, blends between, and scales cosines and sines by 0.1 ln(factor) + 1 (so scores by its square).  The blend is
    linear in the number of turns, as the method's publication has it; programs that blend linearly in the pair's index
    between rounded bounds get slightly other angles for the pairs between, and their checkpoints were trained with those.
    """
    if rot_dim < 2 or rot_dim % 2 or positions < 1:
        raise ValueError(f"rope_table: positions {positions} and rot_dim {rot_dim}: at least 1, and even and at least 2")
    if factor < 1.0:
        raise ValueError(f"rope_table: factor {factor} below 1")
    size = 1.0
    if scaling == "ntk":
        if rot_dim < 4:
            raise ValueError("rope_table: ntk scaling needs rot_dim of 4 or more")
        base = base * factor ** (rot_dim / (rot_dim - 2))
    freq = base ** (-torch.arange(0, rot_dim, 2, dtype=torch.float64) / rot_dim)
    if scaling == "linear":
        freq = freq / factor
    elif scaling == "yarn":
        if original is None:
            raise ValueError("rope_table: yarn scaling needs the original context length")
        turns = original * freq / (2 * math.pi)
        keep = ((turns - beta_slow) / (beta_fast - beta_slow)).clamp(0.0, 1.0)
        freq = freq / factor * (1 - keep) + freq * keep
        size = 0.1 * math.log(factor) + 1.0
    elif scaling not in (None, "ntk"):
        raise ValueError(f"rope_table: unknown scaling {scaling!r}")
    angle = torch.arange(positions, dtype=torch.float64)[:, None] * freq
    return (torch.cat([angle.cos(), angle.sin()], dim=1) * size).float().to(device)


def _enqueue(fn: str, index: int, *args):
    """Calls `fn` with `args` and the current stream of device `index`, with that device current."""
    with torch.cuda.device(index):
        status = getattr(_load(), fn)(*args, _stream(index))
    if status != 0:
        raise MoeError(fn, status)


def moe_w4a8_kv_append(batch: KVBatch, prep: HeadPrep, q, k, v, q_out):
    """Norms and turns the heads of q and k, stores k and v in the cache at the tokens' positions, q in q_out.

    q [tokens, q_heads, head_dim], k, v [tokens, kv_heads, head_dim], q_out as q: any token and head strides that are
    multiples of 16 bytes.  q_out may be q.
    """
    n = q.shape[0]
    hq, hkv = batch.n_q_heads, batch.n_kv_heads
    if prep._index >= 0 and prep._index != batch._index:
        raise ValueError(f"HeadPrep is on {prep.device}, the cache on {batch.device}")
    if prep._weight_dim and prep._weight_dim != batch.head_dim:
        raise ValueError(f"norm weights of {prep._weight_dim} components, heads of {batch.head_dim}")
    if prep.positions is not None and prep.positions.shape != (n,):
        raise ValueError(f"positions: shape {tuple(prep.positions.shape)}, expected {(n,)}")
    args = (batch._p, prep._p, n, *batch._rows(q, "q", n, hq), *batch._rows(k, "k", n, hkv), *batch._rows(v, "v", n, hkv),
            *batch._rows(q_out, "q_out", n, hq))
    if _lib is None or _device() != batch._index:
        _enqueue("moe_w4a8_kv_append", batch._index, *args)
    elif status := _lib.moe_w4a8_kv_append(*args, _stream(batch._index)):
        raise MoeError("moe_w4a8_kv_append", status)
    return q_out


def _aligned(ws):
    """(address, bytes) of the 256-byte aligned part of a workspace."""
    if ws.dtype is not torch.uint8 or not ws.is_contiguous():
        binding._need(ws, "workspace", torch.uint8)
    base = ws.data_ptr()
    at = (base + 255) & -256
    return at, max(0, ws.numel() - (at - base))


def moe_w4a8_paged_attention(batch: KVBatch, q, out, lse=None, scale: float | None = None, window: int = 0, *, workspace):
    """Causal attention of the batch's tokens over its cache (which holds their keys and values already).

    q, out [tokens, q_heads, head_dim]; lse [tokens, q_heads] float32, the log-sum-exp of each row's scaled scores, or
    None; scale defaults to head_dim^-1/2; window > 0 limits a token to the last `window` positions, its own among
    them.  workspace: batch.alloc_workspace().
    """
    n = q.shape[0]
    hq = batch.n_q_heads
    at = None
    if lse is not None:
        if lse.dtype is not torch.float32 or lse.shape != (n, hq) or not lse.is_contiguous():
            raise ValueError(f"lse must be a contiguous float32 tensor of shape {(n, hq)}")
        if lse.get_device() != batch._index:
            raise ValueError(f"lse is on {lse.device}, the cache on {batch.device}")
        at = lse.data_ptr()
    if workspace.get_device() != batch._index:
        raise ValueError(f"workspace is on {workspace.device}, the cache on {batch.device}")
    args = (batch._p, n, *batch._rows(q, "q", n, hq), *batch._rows(out, "out", n, hq), at,
            batch.head_dim ** -0.5 if scale is None else scale, window, *_aligned(workspace))
    if _lib is None or _device() != batch._index:
        _enqueue("moe_w4a8_paged_attention", batch._index, *args)
    elif status := _lib.moe_w4a8_paged_attention(*args, _stream(batch._index)):
        raise MoeError("moe_w4a8_paged_attention", status)
    return out
