"""ctypes binding over the 4-bit KV cache of libpod_attn.so (argument marshalling only).

The C ABI is ``include/pod_kv4.h``: quantising rows of K and V into a paged
cache of 4-bit codes (:meth:`PodKv4.write`), reading rows back
(:meth:`PodKv4.read`), single-token attention over the cache
(:meth:`PodKv4.decode`), and the step before all of them, the per-head norm of
q and k with the position rotation (:func:`qk_norm_rope`).

Lengths, positions and tables are device tensors, so every call can be captured
into a CUDA graph and replayed with what its tensors hold then. As in
:mod:`.pod_attn` there is no fallback: a missing library raises.
"""
from __future__ import annotations

import ctypes
from typing import Optional

import torch

from .pod_attn import POD_OK, PodError, load_library

PAGE_SIZE = 16
DTYPES = {torch.bfloat16: 0, torch.float16: 1}

# Every symbol include/pod_kv4.h declares.
EXPORTED = ("pod_qk_norm_rope", "pod_kv4_record_bytes", "pod_kv4_create", "pod_kv4_write",
            "pod_kv4_read", "pod_kv4_decode", "pod_kv4_destroy")

_i, _ll, _vp = ctypes.c_int, ctypes.c_longlong, ctypes.c_void_p


class Kv4Config(ctypes.Structure):
    _fields_ = [("num_qo_heads", _i), ("num_kv_heads", _i), ("head_dim", _i), ("group_size", _i),
                ("dtype", _i), ("page_size", _i), ("max_decode_reqs", _i), ("device", _i)]


class Kv4RowsArgs(ctypes.Structure):
    _fields_ = [("num_reqs", _i), ("num_rows", _i), ("cu_rows", _vp), ("start", _vp), ("k", _vp),
                ("v", _vp), ("k_row_stride", _ll), ("k_head_stride", _ll), ("v_row_stride", _ll),
                ("v_head_stride", _ll), ("pool", _vp), ("pool_blocks", _ll), ("block_table", _vp),
                ("block_table_stride", _i)]


class Kv4DecodeArgs(ctypes.Structure):
    _fields_ = [("num_reqs", _i), ("ctx_lens", _vp), ("q", _vp), ("o", _vp), ("lse", _vp),
                ("pool", _vp), ("pool_blocks", _ll), ("block_table", _vp),
                ("block_table_stride", _i)]


class QkArgs(ctypes.Structure):
    _fields_ = [("num_qo_heads", _i), ("num_kv_heads", _i), ("head_dim", _i), ("rot_dim", _i),
                ("interleaved", _i), ("dtype", _i), ("device", _i), ("num_rows", _i), ("q", _vp),
                ("k", _vp), ("q_out", _vp), ("k_out", _vp), ("q_row_stride", _ll),
                ("q_head_stride", _ll), ("k_row_stride", _ll), ("k_head_stride", _ll),
                ("q_out_row_stride", _ll), ("q_out_head_stride", _ll), ("k_out_row_stride", _ll),
                ("k_out_head_stride", _ll), ("q_weight", _vp), ("k_weight", _vp),
                ("eps", ctypes.c_float), ("positions", _vp), ("cos_sin", _vp),
                ("max_position", _ll)]


_bound = None


def _library() -> ctypes.CDLL:
    global _bound
    if _bound is None:
        lib = load_library()
        lib.pod_qk_norm_rope.argtypes = [ctypes.POINTER(QkArgs), _vp]
        lib.pod_kv4_record_bytes.argtypes = [_i, _i]
        lib.pod_kv4_create.argtypes = [ctypes.POINTER(_vp), ctypes.POINTER(Kv4Config)]
        lib.pod_kv4_write.argtypes = [_vp, ctypes.POINTER(Kv4RowsArgs), _vp]
        lib.pod_kv4_read.argtypes = [_vp, ctypes.POINTER(Kv4RowsArgs), _vp]
        lib.pod_kv4_decode.argtypes = [_vp, ctypes.POINTER(Kv4DecodeArgs), _vp]
        lib.pod_kv4_destroy.argtypes = [_vp]
        for name in EXPORTED:
            getattr(lib, name).restype = ctypes.c_int
        _bound = lib
    return _bound


def _need(ok: bool, what: str) -> None:
    if not ok:
        raise ValueError(what)


def _on(t: torch.Tensor, device: int, dtype, name: str) -> int:
    """The pointer of a CUDA tensor of the given device and type."""
    if not (t.is_cuda and t.get_device() == device and t.dtype == dtype):
        raise ValueError("%s: expected a %s CUDA tensor on device %d" % (name, dtype, device))
    return t.data_ptr()


def _flat(t: torch.Tensor, device: int, dtype, name: str) -> int:
    """The pointer of a contiguous one."""
    if not t.is_contiguous():
        raise ValueError("%s: expected a contiguous tensor" % name)
    return _on(t, device, dtype, name)


def _stream_of(stream, device: int) -> int:
    return int((torch.cuda.current_stream(device) if stream is None else stream).cuda_stream)


def record_bytes(head_dim: int, group_size: int) -> int:
    """Bytes of one (page, KV head) record."""
    n = int(_library().pod_kv4_record_bytes(int(head_dim), int(group_size)))
    if n < 0:
        raise PodError(n, "pod_kv4_record_bytes")
    return n


class PodKv4:
    """One library context (``pod_kv4_create`` ... ``pod_kv4_destroy``)."""

    def __init__(self, num_qo_heads: int, num_kv_heads: int, head_dim: int, *,
                 group_size: int = 64, dtype: torch.dtype = torch.bfloat16,
                 max_decode_reqs: int = 1024, device: int = 0):
        self._lib = _library()
        self._h = None
        _need(dtype in DTYPES, "dtype: bfloat16 or float16")
        self.cfg = Kv4Config(num_qo_heads, num_kv_heads, head_dim, group_size, DTYPES[dtype],
                             PAGE_SIZE, max_decode_reqs, device)
        h = _vp()
        rc = self._lib.pod_kv4_create(ctypes.byref(h), ctypes.byref(self.cfg))
        if rc != POD_OK:
            raise PodError(rc, "pod_kv4_create")
        self._h = h
        self.dtype = dtype
        self.device = int(device)
        self.record = record_bytes(head_dim, group_size)

    def new_pool(self, pool_blocks: int) -> torch.Tensor:
        """A zeroed pool (every code and pair stands for 0)."""
        return torch.zeros(pool_blocks, self.cfg.num_kv_heads, self.record, dtype=torch.uint8,
                           device="cuda:%d" % self.device)

    # -- argument structs (each keeps its tensors alive)
    def _cache(self, a, pool, block_table, num_reqs) -> None:
        _need(pool.dim() == 3 and tuple(pool.shape[1:]) == (self.cfg.num_kv_heads, self.record),
              "pool: expected [blocks, num_kv_heads, %d]" % self.record)
        _need(block_table.dim() == 2 and block_table.shape[0] == num_reqs,
              "block_table: expected [num_reqs, pages]")
        a.num_reqs = num_reqs
        a.pool = _flat(pool, self.device, torch.uint8, "pool")
        a.pool_blocks = pool.shape[0]
        a.block_table = _flat(block_table, self.device, torch.int32, "block_table")
        a.block_table_stride = block_table.shape[1]

    def rows_args(self, cu_rows, start, k, v, pool, block_table) -> Kv4RowsArgs:
        """``k``, ``v``: [rows, Hk, d], any row and head strides that are multiples of 8."""
        a = Kv4RowsArgs()
        n = start.numel()
        _need(cu_rows.numel() == n + 1, "cu_rows: expected num_reqs + 1 entries")
        self._cache(a, pool, block_table, n)
        shape = k.shape
        _need(len(shape) == 3 and shape == v.shape and
              tuple(shape[1:]) == (self.cfg.num_kv_heads, self.cfg.head_dim),
              "k, v: expected [rows, num_kv_heads, head_dim]")
        ks, vs = k.stride(), v.stride()
        _need(ks[2] == 1 and vs[2] == 1, "k, v: expected adjacent channels")
        a.num_rows = shape[0]
        a.cu_rows = _flat(cu_rows, self.device, torch.int32, "cu_rows")
        a.start = _flat(start, self.device, torch.int32, "start")
        a.k, a.v = _on(k, self.device, self.dtype, "k"), _on(v, self.device, self.dtype, "v")
        a.k_row_stride, a.k_head_stride, a.v_row_stride, a.v_head_stride = ks[0], ks[1], vs[0], vs[1]
        a._keep = (cu_rows, start, k, v, pool, block_table)
        return a

    def decode_args(self, ctx_lens, q, o, lse, pool, block_table) -> Kv4DecodeArgs:
        a = Kv4DecodeArgs()
        n = ctx_lens.numel()
        H, d = self.cfg.num_qo_heads, self.cfg.head_dim
        _need(q.shape == (n, H, d) and o.shape == (n, H, d),
              "q, o: expected [num_reqs, num_qo_heads, head_dim]")
        _need(lse.shape == (n, H), "lse: expected [num_reqs, num_qo_heads]")
        self._cache(a, pool, block_table, n)
        a.ctx_lens = _flat(ctx_lens, self.device, torch.int32, "ctx_lens")
        a.q, a.o = _flat(q, self.device, self.dtype, "q"), _flat(o, self.device, self.dtype, "o")
        a.lse = _flat(lse, self.device, torch.float32, "lse")
        a._keep = (ctx_lens, q, o, lse, pool, block_table)
        return a

    # -- calls
    def _call(self, name, args, stream) -> None:
        _need(self._h is not None, "the context is closed")
        rc = getattr(self._lib, name)(self._h, ctypes.byref(args), _stream_of(stream, self.device))
        if rc != POD_OK:
            raise PodError(rc, name)

    def write(self, args: Kv4RowsArgs, stream=None) -> None:
        self._call("pod_kv4_write", args, stream)

    def read(self, args: Kv4RowsArgs, stream=None) -> None:
        self._call("pod_kv4_read", args, stream)

    def decode(self, args: Kv4DecodeArgs, stream=None) -> None:
        self._call("pod_kv4_decode", args, stream)

    def close(self) -> int:
        if getattr(self, "_h", None):
            rc = int(self._lib.pod_kv4_destroy(self._h))
            self._h = None
            return rc
        return POD_OK

    def __del__(self):  # pragma: no cover
        try:
            self.close()
        except Exception:
            pass


def rope_table(max_position: int, rot_dim: int, base: float = 10000.0, *,
               device="cuda") -> torch.Tensor:
    """The table :func:`qk_norm_rope` takes: [max_position, rot_dim] fp32, the
    cosines of a position and then its sines, of the angles
    ``position * base ** (-2 i / rot_dim)``, computed in fp64 (in fp32 the angle
    of position 10^6 would be off by 0.03)."""
    freq = torch.pow(float(base), -torch.arange(0, rot_dim, 2, dtype=torch.float64,
                                                device=device) / rot_dim)
    angle = torch.arange(max_position, dtype=torch.float64, device=device)[:, None] * freq
    return torch.cat([angle.cos(), angle.sin()], 1).float()


def norm_rope_args(q: Optional[torch.Tensor], k: Optional[torch.Tensor], positions: torch.Tensor,
                   cos_sin: torch.Tensor, *, q_out: Optional[torch.Tensor] = None,
                   k_out: Optional[torch.Tensor] = None,
                   q_weight: Optional[torch.Tensor] = None,
                   k_weight: Optional[torch.Tensor] = None, eps: float = 1e-6,
                   interleaved: bool = False) -> QkArgs:
    """``q`` [rows, H, d] and ``k`` [rows, Hk, d] (either may be None), with any
    row and head strides that are multiples of 8. Without ``q_out`` / ``k_out``
    the rows are replaced in place; without a weight that side is only rotated."""
    a = QkArgs()
    some = q if q is not None else k
    _need(some is not None, "q or k is needed")
    device, dtype, rows, d = some.get_device(), some.dtype, some.shape[0], some.shape[-1]
    _need(dtype in DTYPES, "q, k: bfloat16 or float16")
    for name, x, out, w in (("q", q, q_out, q_weight), ("k", k, k_out, k_weight)):
        if x is None:
            continue
        out = x if out is None else out
        _need(x.dim() == 3 and x.shape[0] == rows and x.shape[2] == d and out.shape == x.shape,
              "%s: expected [rows, heads, head_dim], and its output alike" % name)
        xs, os = x.stride(), out.stride()
        _need(xs[2] == 1 and os[2] == 1, "%s: expected adjacent channels" % name)
        setattr(a, name, _on(x, device, dtype, name))
        setattr(a, name + "_out", _on(out, device, dtype, name + "_out"))
        setattr(a, name + "_row_stride", xs[0])
        setattr(a, name + "_head_stride", xs[1])
        setattr(a, name + "_out_row_stride", os[0])
        setattr(a, name + "_out_head_stride", os[1])
        if w is not None:
            _need(w.shape == (d,), "%s_weight: expected [head_dim]" % name)
            setattr(a, name + "_weight", _flat(w, device, dtype, name + "_weight"))
    a.num_qo_heads = 0 if q is None else q.shape[1]
    a.num_kv_heads = 0 if k is None else k.shape[1]
    _need(positions.shape == (rows,), "positions: expected [rows]")
    _need(cos_sin.dim() == 2, "cos_sin: expected [max_position, rot_dim]")
    a.head_dim, a.rot_dim, a.num_rows = d, cos_sin.shape[1], rows
    a.interleaved, a.dtype, a.device, a.eps = int(interleaved), DTYPES[dtype], device, eps
    a.positions = _flat(positions, device, torch.int32, "positions")
    a.cos_sin = _flat(cos_sin, device, torch.float32, "cos_sin")
    a.max_position = cos_sin.shape[0]
    a._keep = (q, k, positions, cos_sin, q_out, k_out, q_weight, k_weight)
    return a


def qk_norm_rope(args: QkArgs, stream=None) -> None:
    """``pod_qk_norm_rope``: per-head RMS norm of q and k and the rotation, in one launch."""
    rc = _library().pod_qk_norm_rope(ctypes.byref(args), _stream_of(stream, args.device))
    if rc != POD_OK:
        raise PodError(rc, "pod_qk_norm_rope")
