"""Python binding of libpkv: the C entry points under the same names.

Only argument marshalling happens here (tensor pointers, the current CUDA
stream, status checks).  Every step of the computation runs in the library's
CUDA kernels; torch supplies device memory and streams.
"""
from __future__ import annotations

import ctypes
import struct
from typing import List, Optional, Sequence, Tuple

import torch

from . import _lib
from ._lib import lib

_DTYPES = {torch.bfloat16: _lib.BF16, torch.float32: _lib.F32, torch.uint8: _lib.FP4, torch.float8_e4m3fn: _lib.FP8}
_QUANTISED = (torch.uint8, torch.float8_e4m3fn)  # caches held in 4 and in 8 bits


def _stream(stream=None) -> int:
    """The handle of `stream`, or of the current stream of the current device."""
    if stream is not None:
        return stream.cuda_stream
    return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    if t is None:
        return None
    return t.data_ptr()


def _contig(t: torch.Tensor, name: str) -> torch.Tensor:
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t


class PagedKVCache:
    """Per-layer paged K/V pools plus one block table, and their descriptor.

    Pools are (num_blocks, 16, kv_heads, head_dim) tensors of bf16 or fp32
    (the layout of vLLM-Omni's SenseNova-U1 PagedDecodeCache), or, for a cache
    held in 4 bits, uint8 (num_blocks, kv_heads, 9 * head_dim), or, in 8 bits,
    float8_e4m3fn (num_blocks, kv_heads, 16 * head_dim + 16), with head_dim
    64, 128 or 256 (the page formats are in include/pkv.h; 8-bit pools start zeroed); the block
    table is int32 (max_seqs, max_blocks_per_seq).  first_valid, optional
    int32 (max_seqs,), is each sequence's first non-padding position for
    left-padded batches (tiny-llm kv_cache.py, SlotKVCache): the attention
    calls hide earlier keys and let a padding row see only its own key.  The
    tensors are owned by this object; the descriptor only points at them.
    """

    def __init__(self, k: Sequence[torch.Tensor], v: Sequence[torch.Tensor], block_table: torch.Tensor,
                 ring_rows: int = 0, bucket: Optional[int] = None, generation: int = 0,
                 first_valid: Optional[torch.Tensor] = None):
        if len(k) != len(v) or not k:
            raise ValueError("k and v need one tensor per layer")
        shape, dtype = k[0].shape, k[0].dtype
        if dtype not in _DTYPES:
            raise ValueError(f"unsupported dtype {dtype}")
        for t in list(k) + list(v):
            if t.shape != shape or t.dtype != dtype or not t.is_contiguous():
                raise ValueError("every pool must be contiguous with the same shape and dtype")
        if dtype in _QUANTISED:
            if dtype == torch.uint8:
                if len(shape) != 3 or shape[2] % 9:
                    raise ValueError("4-bit pools are uint8 (num_blocks, kv_heads, 9 * head_dim)")
                kv_heads, head_dim = int(shape[1]), int(shape[2]) // 9
            else:
                if len(shape) != 3 or shape[2] % 16 or shape[2] < 32:
                    raise ValueError("8-bit pools are float8_e4m3fn (num_blocks, kv_heads, 16 * head_dim + 16)")
                kv_heads, head_dim = int(shape[1]), int(shape[2]) // 16 - 1
            if any(t.get_device() != k[0].get_device() for t in [*k, *v, block_table] + ([] if first_valid is None else [first_valid])):
                raise ValueError("the pools and tables of a quantised cache are on one device")
        else:
            if len(shape) != 4 or shape[1] != _lib.BLOCK_SIZE:
                raise ValueError("pools are (num_blocks, 16, kv_heads, head_dim)")
            kv_heads, head_dim = int(shape[2]), int(shape[3])
        if block_table.dtype != torch.int32 or block_table.dim() != 2:
            raise ValueError("block_table is int32 (max_seqs, max_blocks_per_seq)")
        self.k: List[torch.Tensor] = list(k)
        self.v: List[torch.Tensor] = list(v)
        self.block_table = _contig(block_table, "block_table")
        if first_valid is not None and (first_valid.dtype != torch.int32 or first_valid.dim() != 1
                                        or first_valid.shape[0] != block_table.shape[0]):
            raise ValueError("first_valid is int32 (max_seqs,)")
        self.first_valid = None if first_valid is None else _contig(first_valid, "first_valid")
        self.ring_rows = int(ring_rows)
        self.generation = int(generation)
        nb = shape[0]
        self.bucket = int(bucket) if bucket is not None else int(block_table.shape[1]) * _lib.BLOCK_SIZE
        self._kp = (ctypes.c_void_p * len(k))(*[t.data_ptr() for t in self.k])
        self._vp = (ctypes.c_void_p * len(v))(*[t.data_ptr() for t in self.v])
        self.desc = _lib.CacheDesc(
            num_layers=len(k), kv_heads=kv_heads, head_dim=head_dim, dtype=_DTYPES[dtype], num_blocks=nb,
            max_seqs=block_table.shape[0], max_blocks_per_seq=block_table.shape[1], ring_rows=self.ring_rows,
            reserved0=0, k=ctypes.cast(self._kp, ctypes.c_void_p), v=ctypes.cast(self._vp, ctypes.c_void_p),
            block_table=block_table.data_ptr(), bucket=self.bucket, generation=self.generation,
            first_valid=_ptr(self.first_valid))
        self._ref = ctypes.byref(self.desc)
        self._quantised = dtype in _QUANTISED
        self._kv_heads, self._head_dim, self._device = kv_heads, head_dim, k[0].get_device()
        # the type of q, k_new and v_new rows: the cache's, bf16 for a quantised cache
        self.row_dtype = torch.bfloat16 if self._quantised else dtype

    @classmethod
    def allocate(cls, num_layers: int, kv_heads: int, head_dim: int, bucket: int, dtype=torch.bfloat16,
                 device="cuda", generation: int = 0) -> "PagedKVCache":
        """Zeroed single-sequence cache behind an identity table (one bucket); dtype torch.uint8: held in 4 bits, torch.float8_e4m3fn: in 8."""
        nb = (bucket + _lib.BLOCK_SIZE - 1) // _lib.BLOCK_SIZE
        shape = (nb, kv_heads, 9 * head_dim if dtype == torch.uint8 else 16 * head_dim + 16) if dtype in _QUANTISED else (nb, _lib.BLOCK_SIZE, kv_heads, head_dim)
        k = [torch.zeros(shape, dtype=dtype, device=device) for _ in range(num_layers)]
        v = [torch.zeros(shape, dtype=dtype, device=device) for _ in range(num_layers)]
        bt = torch.arange(nb, dtype=torch.int32, device=device).unsqueeze(0)
        return cls(k, v, bt, bucket=bucket, generation=generation)

    @property
    def num_layers(self) -> int:
        return len(self.k)

    @property
    def kv_heads(self) -> int:
        return self._kv_heads

    @property
    def head_dim(self) -> int:
        return self._head_dim

    @property
    def dtype(self) -> torch.dtype:
        return self.k[0].dtype

    def ref(self):
        return self._ref

    def reusable_for(self, num_layers, kv_heads, head_dim, dtype, length) -> bool:
        """Same shape and the length fits the current bucket (PagedDecodeCache.reusable_for)."""
        return (self.num_layers == num_layers and self.kv_heads == kv_heads and self.head_dim == head_dim
                and self.dtype == dtype and bucket_for(length) <= self.bucket)


def bucket_for(length: int) -> int:
    return int(lib.pkv_bucket_for(int(length)))


def new_err_flags(device="cuda") -> torch.Tensor:
    return torch.zeros(1, dtype=torch.int32, device=device)


def rope_inv_freq(rot_dim: int, theta: float = 10000.0, scaling: str = "none", factor: float = 1.0,
                  trained_len: float = 0.0, beta_fast: float = 32.0, beta_slow: float = 1.0) -> Tuple[torch.Tensor, float]:
    """pkv_rope_inv_freq: (float64 frequencies on the host, factor on the sines and cosines).

    scaling: "none", "linear" (positions / factor), "ntk" (a larger theta) or
    "yarn" (by parts, from the trained context length).
    """
    kinds = {"none": _lib.ROPE_PLAIN, "linear": _lib.ROPE_LINEAR, "ntk": _lib.ROPE_NTK, "yarn": _lib.ROPE_YARN}
    if scaling not in kinds:
        raise ValueError(f"scaling is one of {sorted(kinds)}")
    freq = torch.empty(max(int(rot_dim) // 2, 1), dtype=torch.float64)
    mscale = ctypes.c_double()
    _lib.check("pkv_rope_inv_freq", lib.pkv_rope_inv_freq(int(rot_dim), float(theta), kinds[scaling], float(factor),
                                                          float(trained_len), float(beta_fast), float(beta_slow),
                                                          _ptr(freq), ctypes.addressof(mscale)))
    return freq, float(mscale.value)


def rope_axes(sections: Sequence[int], dealt: bool = False) -> List[int]:
    """The axis of every column pair, for Rope's axes, from the number of pairs each axis turns.

    Axis after axis (the first sections[0] pairs turn with axis 0, ...), or
    dealt: to the axes in turn, passing over those that have all their pairs
    (0, 1, 2, 0, 1, 2, ..).
    """
    left = [int(n) for n in sections]
    if not 1 <= len(left) <= _lib.ROPE_AXES or min(left) < 0 or sum(left) == 0:
        raise ValueError(f"sections are the pairs of 1 to {_lib.ROPE_AXES} axes, none negative")
    if not dealt:
        return [a for a, n in enumerate(left) for _ in range(n)]
    out: List[int] = []
    while any(left):
        for a, n in enumerate(left):
            if n:
                left[a] -= 1
                out.append(a)
    return out


class Rope:
    """What norm_rope and norm_rope_append do to a head: RMSNorm by a weight, then a rotation.

    inv_freq: radians a position of each column pair (rot_dim = 2 *
    len(inv_freq), at most head_dim), from rope_inv_freq or a model's own;
    None for no rotation.  interleaved: pairs (2i, 2i + 1) instead of (i, i +
    rot_dim / 2).  mscale multiplies the rotated columns.  q_weight /
    k_weight: (head_dim,) of the rows' type, or None for no norm of that
    side.  Made once per model or layer; it keeps its tensors.

    axes: for rows with a position on each of several axes (time, height and
    width of images and video), the axis of every pair, as from rope_axes;
    positions are then (rows, number of axes), the highest of `axes` and one.
    """

    def __init__(self, inv_freq: Optional[torch.Tensor] = None, interleaved: bool = False, mscale: float = 1.0,
                 q_weight: Optional[torch.Tensor] = None, k_weight: Optional[torch.Tensor] = None, eps: float = 1e-6,
                 device=None, axes: Optional[Sequence[int]] = None):
        self.turns = self.axis = None
        self.num_axes = 1
        n = 0
        if inv_freq is not None:
            if inv_freq.dim() != 1 or inv_freq.numel() == 0:
                raise ValueError("inv_freq is (rot_dim / 2,)")
            n = int(inv_freq.numel())
            host = inv_freq.detach().to("cpu", torch.float64).contiguous()
            turns = torch.empty(n, dtype=torch.int64)
            _lib.check("pkv_rope_turns", lib.pkv_rope_turns(_ptr(host), n, _ptr(turns)))
            if device is None:
                device = inv_freq.device if inv_freq.is_cuda else "cuda"
            self.turns = turns.to(device)
        if axes is not None:
            axes = [int(a) for a in axes]
            if len(axes) != n or n == 0 or min(axes) < 0 or max(axes) >= _lib.ROPE_AXES:
                raise ValueError(f"axes names an axis below {_lib.ROPE_AXES} for each of the {n} pairs")
            self.num_axes = max(axes) + 1
            if self.num_axes > 1:
                self.axis = torch.tensor(axes, dtype=torch.uint8).to(device)
        for name, w in (("q_weight", q_weight), ("k_weight", k_weight)):
            if w is not None and (w.dim() != 1 or w.dtype not in (torch.bfloat16, torch.float32)):
                raise ValueError(f"{name} is (head_dim,) of bf16 or fp32")
        self.q_weight = None if q_weight is None else _contig(q_weight, "q_weight")
        self.k_weight = None if k_weight is None else _contig(k_weight, "k_weight")
        self.rot_dim, self.interleaved, self.mscale, self.eps = 2 * n, bool(interleaved), float(mscale), float(eps)
        self.desc = _lib.RopeDesc(turns=_ptr(self.turns), rot_dim=self.rot_dim, interleaved=int(self.interleaved),
                                  mscale=self.mscale, eps=self.eps, q_weight=_ptr(self.q_weight),
                                  k_weight=_ptr(self.k_weight), axis=_ptr(self.axis), num_axes=self.num_axes, reserved0=0)

        given = [t for t in (self.turns, self.q_weight, self.k_weight) if t is not None]
        weights = [w for w in (self.q_weight, self.k_weight) if w is not None]
        if any(t.get_device() != given[0].get_device() for t in given) or any(
                w.dtype != weights[0].dtype or w.numel() != weights[0].numel() for w in weights):
            raise ValueError("the norm weights and frequencies are on one device, the weights of one type and size")
        self._device = given[0].get_device() if given else None
        self._dtype, self._dim = (weights[0].dtype, weights[0].numel()) if weights else (None, None)
        self._ref = ctypes.byref(self.desc)

    def check(self, dtype: torch.dtype, head_dim: int, device: int) -> None:
        """Raises unless this applies to rows of dtype and head_dim on CUDA device `device`."""
        if self.rot_dim > head_dim:
            raise ValueError(f"rot_dim {self.rot_dim} is above head_dim {head_dim}")
        if self._device is not None and self._device != device:
            raise ValueError("the frequencies and norm weights are on another device than the rows")
        if self._dtype is not None and (self._dtype is not dtype or self._dim != head_dim):
            raise ValueError("norm weights are (head_dim,) of the rows' type")


# struct pkv_rows as bytes (native sizes and alignment): cheaper to make than a ctypes structure
_ROWS = struct.Struct("6Q6q2iQ")
assert _ROWS.size == ctypes.sizeof(_lib.RowsDesc)


def _row_stride(t: torch.Tensor, name: str, shape, dtype: torch.dtype, device: int) -> int:
    """Elements between the rows of t, whose heads and columns are contiguous and whose rows are apart as they like."""
    if t.shape != shape or t.dtype is not dtype or t.get_device() != device:
        raise ValueError(f"{name} is {tuple(shape)} of {dtype} on device {device}")
    s0, s1, s2 = t.stride()
    rows, heads, dim = shape
    if (s2 != 1 and dim > 1) or (s1 != dim and heads > 1):
        raise ValueError(f"the heads of a row of {name} must be contiguous")
    return s0 if rows > 1 else heads * dim


def _rows_desc(q, k, v, q_out, k_out, v_out, positions, kv_heads, head_dim, dtype, device, axes=1) -> bytes:
    shape = (q if q is not None else k).shape
    if len(shape) != 3:
        raise ValueError("rows are (rows, heads, head_dim)")
    rows, hq = shape[0], 0
    kv = (rows, kv_heads, head_dim)
    qp = kp = vp = qop = kop = vop = pos = 0
    qs = ks = vs = qos = kos = vos = 0
    if q is not None:
        hq = shape[1]
        heads = (rows, hq, head_dim)
        qs, qp = _row_stride(q, "q", heads, dtype, device), q.data_ptr()
        qos, qop = (qs, qp) if q_out is q else (_row_stride(q_out, "q_out", heads, dtype, device), q_out.data_ptr())
    elif q_out is not None:
        raise ValueError("q_out without q")
    if k is not None:
        ks, kp = _row_stride(k, "k", kv, dtype, device), k.data_ptr()
    if v is not None:
        vs, vp = _row_stride(v, "v", kv, dtype, device), v.data_ptr()
    if k_out is not None:
        kos, kop = _row_stride(k_out, "k_out", kv, dtype, device), k_out.data_ptr()
    if v_out is not None:
        vos, vop = _row_stride(v_out, "v_out", kv, dtype, device), v_out.data_ptr()
    if positions is not None:
        want = (rows,) if axes == 1 else (rows, axes)
        if positions.shape != want or positions.dtype is not torch.int32 or positions.get_device() != device:
            raise ValueError(f"positions is int32 {want} on device {device}")
        pos = _contig(positions, "positions").data_ptr()
    return _ROWS.pack(qp, kp, vp, qop, kop, vop, qs, ks, vs, qos, kos, vos, hq, rows, pos)


def _raw_stream(device: int, stream) -> int:
    """The handle of `stream` or of the device's current stream, for a launch on it as the current device."""
    if device < 0:
        raise ValueError("the tensors are not on a CUDA device")
    return stream.cuda_stream if stream is not None else torch._C._cuda_getCurrentRawStream(device)


def _launch(name: str, fn, args, device: int, stream) -> None:
    """fn(*args, stream) with `device` current, whichever is."""
    handle = _raw_stream(device, stream)
    if device == torch._C._cuda_getDevice():
        st = fn(*args, handle)
    else:
        with torch.cuda.device(device):
            st = fn(*args, handle)
    if st:
        _lib.check(name, st)


def _on_device(device: int, name: str, fn, args, stream, allowed=(_lib.OK,)) -> int:
    """The status of fn(*args, stream) with `device` current; with the current one where it is -1 (host memory)."""
    if device < 0 or device == torch._C._cuda_getDevice():
        return _lib.check(name, fn(*args, _stream(stream)), allowed)
    with torch.cuda.device(device):
        return _lib.check(name, fn(*args, _stream(stream)), allowed)


def norm_rope(rope: Rope, q: Optional[torch.Tensor], k: Optional[torch.Tensor], positions: Optional[torch.Tensor],
              q_out: Optional[torch.Tensor] = None, k_out: Optional[torch.Tensor] = None, stream=None) -> None:
    """pkv_norm_rope: norm and rotation of rows that go to no cache.

    q (rows, q_heads, head_dim) and k (rows, kv_heads, head_dim), bf16 or fp32,
    either may be None; rows may be strided (a slice of a projection's output).
    positions: int32 (rows,), or (rows, axes) with a Rope of several axes.
    Without q_out / k_out the rows are changed in place.
    """
    some = q if q is not None else k
    if some is None or some.dim() != 3:
        raise ValueError("q or k is (rows, heads, head_dim)")
    dim, dtype, dev = int(some.shape[2]), some.dtype, some.get_device()
    if dtype is not torch.bfloat16 and dtype is not torch.float32:
        raise ValueError(f"unsupported dtype {dtype}")
    if k is None and k_out is not None:
        raise ValueError("k_out without k")
    rope.check(dtype, dim, dev)
    kv = int(k.shape[1]) if k is not None and k.dim() == 3 else 0
    d = _rows_desc(q, k, None, q_out if q_out is not None else q, k_out if k_out is not None else k, None, positions, kv, dim,
                   dtype, dev, rope.num_axes)
    _launch("pkv_norm_rope", lib.pkv_norm_rope, (rope._ref, _DTYPES[dtype], dim, kv, d), dev, stream)


def norm_rope_append(cache: PagedKVCache, layer: int, rope: Optional[Rope], q: Optional[torch.Tensor], k_new: torch.Tensor,
                     v_new: torch.Tensor, seq_info: torch.Tensor, q_out: Optional[torch.Tensor], err: torch.Tensor,
                     window: int = 0, positions: Optional[torch.Tensor] = None, k_out: Optional[torch.Tensor] = None,
                     v_out: Optional[torch.Tensor] = None, stream=None) -> None:
    """pkv_norm_rope_append: norm and rotation of q and k, and the append of k and v, in one pass.

    q goes to q_out (None: in place).  positions (rows,) int32, or (rows, axes)
    with a Rope of several axes, overrides the angles' positions; by default a
    row's position in the cache, on every axis.  k_out / v_out
    get the rows as the cache holds them.  Rows may be strided.
    """
    dev, dtype, dim = cache._device, cache.row_dtype, cache._head_dim
    if rope is not None:
        rope.check(dtype, dim, dev)
    segments = _check_segments(cache, seq_info, err)
    d = _rows_desc(q, k_new, v_new, q if q_out is None else q_out, k_out, v_out, positions, cache._kv_heads, dim, dtype, dev,
                   1 if rope is None else rope.num_axes)
    _launch("pkv_norm_rope_append", lib.pkv_norm_rope_append,
            (cache._ref, layer, None if rope is None else rope._ref, d, _contig(seq_info, "seq_info").data_ptr(), segments, window, err.data_ptr()),
            dev, stream)


_BF16, _F32, _I32 = torch.bfloat16, torch.float32, torch.int32  # (short calls are bound by what the host looks up)


def _check_new(cache: PagedKVCache, rows: int, k_new: torch.Tensor, v_new: torch.Tensor) -> None:
    """New rows for a quantised cache, heads and columns of a row apart or as one dimension."""
    shape, heads, dim, dev = k_new.shape, cache._kv_heads, cache._head_dim, cache._device
    if (k_new.dtype is not _BF16 or v_new.dtype is not _BF16 or v_new.shape != shape
            or (shape != (rows, heads, dim) and shape != (rows, heads * dim)) or k_new.get_device() != dev or v_new.get_device() != dev):
        raise ValueError(f"rows for a quantised cache are bf16, k_new and v_new ({rows}, {heads}, {dim}) on the cache's device")


def _check_segments(cache: PagedKVCache, seq_info: torch.Tensor, err: torch.Tensor) -> int:
    """The segment table and error flags of a call: the number of segments."""
    shape, dev = seq_info.shape, cache._device
    if seq_info.dtype is not _I32 or len(shape) != 2 or shape[1] != 4 or seq_info.get_device() != dev or err.get_device() != dev:
        raise ValueError("seq_info is int32 (segments, 4), and err with it on the cache's device")
    return shape[0]


def _check_fp4(cache: PagedKVCache, q, k_new, v_new, seq_info, out, lse, err) -> None:
    """The tensors of an attention call over a quantised cache."""
    shape, kind, dev = q.shape, out.dtype, cache._device
    if (len(shape) != 3 or shape[2] != cache._head_dim or q.dtype is not _BF16 or (kind is not _F32 and kind is not _BF16) or out.shape != shape
            or q.get_device() != dev or out.get_device() != dev):
        raise ValueError(f"over a quantised cache q is bf16 (rows, heads, {cache._head_dim}) and out fp32 or bf16 of the same shape, on its device")
    if lse is not None and (lse.dtype is not _F32 or lse.numel() != shape[0] * shape[1] or not lse.is_contiguous() or lse.get_device() != dev):
        raise ValueError("lse is fp32 (rows, heads), contiguous, on the cache's device")
    _check_segments(cache, seq_info, err)
    if k_new is not None:
        _check_new(cache, shape[0], k_new, v_new)


def append(cache: PagedKVCache, layer: int, k_new: torch.Tensor, v_new: torch.Tensor, seq_info: torch.Tensor,
           err: torch.Tensor, window: int = 0, stream=None) -> None:
    rows = int(k_new.shape[0])
    if cache._quantised:
        _check_new(cache, rows, k_new, v_new)
        _check_segments(cache, seq_info, err)
    _on_device(cache._device, "pkv_append", lib.pkv_append, (
        cache.ref(), layer, _ptr(_contig(k_new, "k_new")), _ptr(_contig(v_new, "v_new")), rows,
        _ptr(_contig(seq_info, "seq_info")), int(seq_info.shape[0]), int(window), _ptr(err)), stream)


# Bounds (segments x kv heads x row tiles x keys) from which a launch over a quantised cache
# may use a workspace; pkv_attend_workspace_bytes decides.
_FP4_WORKSPACE_FROM = 1 << 18


def fp4_keys(max_kv: int, max_q_len: int, window: int) -> int:
    """Keys of a segment at most: the bound that decides how a launch over a quantised cache is cut."""
    return min(max_kv, window + max_q_len) if window > 0 else max_kv


def _fp4_workspace(cache, hq, segments, max_q_len, max_kv, window, flags, stream):
    """A workspace for one call over a quantised cache, or None: a large launch merges its shared ranges through it.

    Each call takes its own from torch's allocator, so eager calls on several
    streams share nothing.  A captured call's comes from the graph's memory pool:
    graphs captured into one pool must not run at the same time, unless their
    calls were given workspaces of their own (DecodeStep keeps one).
    """
    keys = max_kv if window <= 0 else fp4_keys(max_kv, max_q_len, window)
    tiles = -(-hq * max_q_len // (8 * cache._kv_heads))  # of 8 query rows, at most
    if segments * cache._kv_heads * tiles * keys < _FP4_WORKSPACE_FROM:
        return None
    n = attend_workspace_bytes(cache, hq, segments, max_q_len, keys, 0, flags)
    if n <= 0:
        return None
    if stream is None:
        return torch.empty(n, dtype=torch.uint8, device=cache.k[0].device)
    with torch.cuda.stream(stream):  # the allocator orders a block's users by the stream it was taken on
        return torch.empty(n, dtype=torch.uint8, device=cache.k[0].device)


def _attend(fn_name, cache, layer, q, k_new, v_new, seq_info, out, lse, err, max_q_len, max_kv, scale, causal,
            window, num_splits, flags, stream, workspace):
    shape, segments = q.shape, seq_info.shape[0]
    max_q_len, max_kv, window = int(max_q_len), int(max_kv), int(window)
    if out.dtype is _BF16:
        flags |= _lib.FLAG_OUT_BF16
    dev = cache._device  # -1 on the host (a call that is refused)
    if dev >= 0 and dev != torch._C._cuda_getDevice():
        with torch.cuda.device(dev):
            return _attend(fn_name, cache, layer, q, k_new, v_new, seq_info, out, lse, err, max_q_len, max_kv, scale, causal,
                           window, num_splits, flags, stream, workspace)
    if cache._quantised:
        _check_fp4(cache, q, k_new, v_new, seq_info, out, lse, err)
        if workspace is None and num_splits == 0:
            workspace = _fp4_workspace(cache, shape[1], segments, max_q_len, max_kv, window, flags, stream)
    new = ()
    if fn_name == "pkv_append_attend":
        new = (_contig(k_new, "k_new").data_ptr(), _contig(v_new, "v_new").data_ptr())
    ws, ws_bytes = (None, 0) if workspace is None else (workspace.data_ptr(), workspace.numel() * workspace.element_size())
    handle = torch._C._cuda_getCurrentRawStream(dev) if stream is None and dev >= 0 else _stream(stream)
    st = getattr(lib, fn_name)(
        cache._ref, layer, _contig(q, "q").data_ptr(), *new, shape[1], shape[0], _contig(seq_info, "seq_info").data_ptr(), segments,
        max_q_len, max_kv, int(num_splits), float(scale), 1 if causal else 0, window, _contig(out, "out").data_ptr(),
        None if lse is None else lse.data_ptr(), ws, ws_bytes, err.data_ptr(), int(flags), handle)
    if st:
        _lib.check(fn_name, st)


def attend_varlen(cache: PagedKVCache, layer: int, q: torch.Tensor, seq_info: torch.Tensor, out: torch.Tensor,
                  err: torch.Tensor, max_q_len: int, max_kv: int, scale: float, causal: bool = False,
                  window: int = 0, lse: Optional[torch.Tensor] = None, num_splits: int = 0, flags: int = 0,
                  stream=None, workspace: Optional[torch.Tensor] = None) -> None:
    _attend("pkv_attend_varlen", cache, layer, q, None, None, seq_info, out, lse, err, max_q_len, max_kv, scale,
            causal, window, num_splits, flags, stream, workspace)


def attend_prompt(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, seq_info: torch.Tensor, out: torch.Tensor, err: torch.Tensor,
                  max_len: int, scale: float, causal: bool = True, window: int = 0, lse: Optional[torch.Tensor] = None,
                  stream=None) -> None:
    """pkv_attend_prompt: attention of packed whole prompts over their own rows.

    q (rows, q_heads, head_dim), k and v (rows, kv_heads, head_dim), bf16; rows
    may be strided (slices of a projection's output).  out: fp32 or bf16, like
    q, and apart from it.  seq_info's segments have kv_end == q_len; max_len bounds it.
    """
    if q.dim() != 3 or k.dim() != 3:
        raise ValueError("q, k and v are (rows, heads, head_dim)")
    (rows, hq, dim), hkv, dev = q.shape, int(k.shape[1]), q.get_device()
    qs = _row_stride(q, "q", (rows, hq, dim), _BF16, dev)
    ks, vs = [_row_stride(t, name, (rows, hkv, dim), _BF16, dev) for t, name in ((k, "k"), (v, "v"))]
    if out.shape != q.shape or (out.dtype is not _F32 and out.dtype is not _BF16) or not out.is_contiguous() or out.get_device() != dev:
        raise ValueError("out is fp32 or bf16 of q's shape, contiguous, on its device")
    if lse is not None and (lse.dtype is not _F32 or lse.shape != (rows, hq) or not lse.is_contiguous() or lse.get_device() != dev):
        raise ValueError("lse is fp32 (rows, heads), contiguous, on q's device")
    if seq_info.dtype is not _I32 or seq_info.dim() != 2 or seq_info.shape[1] != 4 or seq_info.get_device() != dev or err.get_device() != dev:
        raise ValueError("seq_info is int32 (segments, 4), and err with it on q's device")
    d = _ROWS.pack(q.data_ptr(), k.data_ptr(), v.data_ptr(), 0, 0, 0, qs, ks, vs, 0, 0, 0, hq, rows, 0)
    _launch("pkv_attend_prompt", lib.pkv_attend_prompt,
            (dim, hkv, d, _contig(seq_info, "seq_info").data_ptr(), seq_info.shape[0], int(max_len), float(scale), 1 if causal else 0, int(window),
             out.data_ptr(), _ptr(lse), err.data_ptr(), _lib.FLAG_OUT_BF16 if out.dtype is _BF16 else 0), dev, stream)


def append_attend(cache: PagedKVCache, layer: int, q: torch.Tensor, k_new: torch.Tensor, v_new: torch.Tensor,
                  seq_info: torch.Tensor, out: torch.Tensor, err: torch.Tensor, max_q_len: int, max_kv: int,
                  scale: float, causal: bool = False, window: int = 0, lse: Optional[torch.Tensor] = None,
                  num_splits: int = 0, flags: int = 0, stream=None, workspace: Optional[torch.Tensor] = None) -> None:
    _attend("pkv_append_attend", cache, layer, q, k_new, v_new, seq_info, out, lse, err, max_q_len, max_kv, scale,
            causal, window, num_splits, flags, stream, workspace)


def append_attend_noalloc(cache: PagedKVCache, layer: int, q: torch.Tensor, k_new: torch.Tensor,
                          v_new: torch.Tensor, seq_info: torch.Tensor, out: torch.Tensor, err: torch.Tensor,
                          max_q_len: int, max_kv: int, scale: float, causal: bool = False, window: int = 0,
                          lse: Optional[torch.Tensor] = None, num_splits: int = 0, flags: int = 0,
                          stream=None) -> None:
    """pkv_append_attend_noalloc: append_attend merging its splits in the library's fixed scratch."""
    rows, hq = int(q.shape[0]), int(q.shape[1])
    if cache._quantised:
        _check_fp4(cache, q, k_new, v_new, seq_info, out, lse, err)
    if out.dtype == torch.bfloat16:
        flags |= _lib.FLAG_OUT_BF16
    _on_device(cache._device, "pkv_append_attend_noalloc", lib.pkv_append_attend_noalloc, (
        cache.ref(), layer, _ptr(_contig(q, "q")), _ptr(_contig(k_new, "k_new")), _ptr(_contig(v_new, "v_new")),
        hq, rows, _ptr(_contig(seq_info, "seq_info")), int(seq_info.shape[0]), int(max_q_len), int(max_kv),
        int(num_splits), float(scale), int(bool(causal)), int(window), _ptr(_contig(out, "out")), _ptr(lse),
        _ptr(err), int(flags)), stream)


def attend_workspace_bytes(cache: PagedKVCache, num_q_heads: int, num_segments: int, max_q_len: int, max_kv: int,
                           num_splits: int = 0, flags: int = 0) -> int:
    """pkv_attend_workspace_bytes: workspace the attention calls need for these bounds (0: none)."""
    args = (cache.ref(), int(num_q_heads), int(num_segments), int(max_q_len), int(max_kv), int(num_splits), int(flags))
    if cache._device < 0 or cache._device == torch._C._cuda_getDevice():
        n = int(lib.pkv_attend_workspace_bytes(*args))
    else:
        with torch.cuda.device(cache._device):
            n = int(lib.pkv_attend_workspace_bytes(*args))
    if n < 0:
        _lib.check("pkv_attend_workspace_bytes", n)
    return n


def new_workspace(cache: PagedKVCache, num_q_heads: int, num_segments: int, max_q_len: int, max_kv: int,
                  num_splits: int = 0, flags: int = 0) -> Optional[torch.Tensor]:
    """A zero-filled workspace for these bounds on the cache's device, or None if none is needed."""
    n = attend_workspace_bytes(cache, num_q_heads, num_segments, max_q_len, max_kv, num_splits, flags)
    return torch.zeros(n, dtype=torch.uint8, device=cache.k[0].device) if n > 0 else None


def seq_clone(cache: PagedKVCache, src_col: int, dst_col: int, n: int, err: torch.Tensor, stream=None) -> None:
    """pkv_seq_clone: copy positions 0..n-1 of block-table row src_col to dst_col in every layer."""
    _on_device(cache._device, "pkv_seq_clone", lib.pkv_seq_clone, (cache.ref(), int(src_col), int(dst_col), int(n), _ptr(err)), stream)


def rewind(cache: PagedKVCache, seq_info: torch.Tensor, amount: torch.Tensor, err: torch.Tensor, window: int = 0,
           stream=None) -> None:
    """pkv_rewind: kv_end -= amount per segment on the device, bounded by the ring floor."""
    _on_device(cache._device, "pkv_rewind", lib.pkv_rewind, (cache.ref(), _ptr(_contig(seq_info, "seq_info")), int(seq_info.shape[0]),
                                                            _ptr(_contig(amount, "amount")), int(window), _ptr(err)), stream)


def seqinfo_from_seqused(cu_seqlens_q: torch.Tensor, seqused_k: torch.Tensor, out: torch.Tensor,
                         stream=None) -> None:
    n = int(seqused_k.shape[0])
    _on_device(out.get_device(), "pkv_seqinfo_from_seqused", lib.pkv_seqinfo_from_seqused,
               (_ptr(cu_seqlens_q), _ptr(seqused_k), n, _ptr(out)), stream)


def advance(seq_info: torch.Tensor, stream=None) -> None:
    _on_device(seq_info.get_device(), "pkv_advance", lib.pkv_advance, (_ptr(seq_info), int(seq_info.shape[0])), stream)


def resize_bucket(old: PagedKVCache, new: PagedKVCache, old_len: int, stream=None) -> int:
    """Copy the first old_len tokens of every layer; bumps new.generation on success."""
    st = _on_device(new._device, "pkv_resize_bucket", lib.pkv_resize_bucket, (old.ref(), new.ref(), int(old_len)), stream,
                    (_lib.OK, _lib.SAME_BUCKET))
    new.generation = int(new.desc.generation)
    return st


def load_prefix(cache: PagedKVCache, keys: Sequence[torch.Tensor], values: Sequence[torch.Tensor],
                stream=None) -> bool:
    """keys/values: per layer [S, H, D] views (any strides with D contiguous).  False if empty."""
    if not keys or keys[0] is None or keys[0].shape[0] == 0:
        return False
    n = int(keys[0].shape[0])
    ss, sh, sd = keys[0].stride()
    if sd != 1:
        raise ValueError("head_dim must be contiguous")
    for t in list(keys) + list(values):
        if t.stride() != (ss, sh, 1) or t.shape != keys[0].shape or t.dtype != cache.dtype:
            raise ValueError("all prefix tensors need the same shape, strides and dtype")
    kp = (ctypes.c_void_p * len(keys))(*[t.data_ptr() for t in keys])
    vp = (ctypes.c_void_p * len(values))(*[t.data_ptr() for t in values])
    st = _on_device(cache._device, "pkv_load_prefix", lib.pkv_load_prefix,
                    (cache.ref(), ctypes.cast(kp, ctypes.c_void_p), ctypes.cast(vp, ctypes.c_void_p), n, ss, sh), stream, (_lib.OK, _lib.EMPTY))
    return st == _lib.OK


def to_contiguous(cache: PagedKVCache, layer: int, n: int, keys_out: torch.Tensor, values_out: torch.Tensor,
                  stream=None) -> None:
    """keys_out / values_out: contiguous [kv_heads, n, head_dim] of the cache's row_dtype (an 8-bit cache's stored values)."""
    if cache.dtype == torch.float8_e4m3fn:
        want = (cache._kv_heads, int(n), cache._head_dim)
        for t in (keys_out, values_out):
            if t.shape != want or t.dtype is not _BF16 or not t.is_contiguous() or t.get_device() != cache._device:
                raise ValueError(f"keys_out and values_out are bf16 {want}, contiguous, on the cache's device")
    _on_device(cache._device, "pkv_to_contiguous", lib.pkv_to_contiguous, (cache.ref(), layer, int(n), _ptr(keys_out), _ptr(values_out)),
               stream)
