"""ctypes binding over the 4-bit KV cache of libpod_attn.so (argument marshalling only).

The C ABI is ``include/pod_kv4.h``: quantising rows of K and V into a paged
cache of 4-bit codes (:meth:`PodKv4.write`), reading rows back
(:meth:`PodKv4.read`), single-token attention over the cache
(:meth:`PodKv4.decode`), and the step before all of them, the per-head norm of
q and k with the position rotation (:func:`qk_norm_rope`).

Their lengths, positions and tables are device tensors, so each can be captured
into a CUDA graph and replayed with what its tensors hold then (of
:meth:`PodKv4.hybrid`, calls without prefills can). As in
:mod:`.pod_attn` there is no fallback: a missing library raises.
"""
from __future__ import annotations

import ctypes
import struct
from typing import Optional, Sequence

import torch

from .pod_attn import POD_ECAPACITY, POD_EUNSUPPORTED, POD_OK, PodAttention, PodError, load_library

PAGE_SIZE = 16
_I32, _U8, _F32 = torch.int32, torch.uint8, torch.float32
DTYPES = {torch.bfloat16: 0, torch.float16: 1}

# Every symbol include/pod_kv4.h declares.
EXPORTED = ("pod_qk_norm_rope", "pod_kv4_record_bytes", "pod_kv4_create", "pod_kv4_write",
            "pod_kv4_read", "pod_kv4_decode", "pod_kv4_status", "pod_kv4_destroy")

_i, _u, _ll, _vp = ctypes.c_int, ctypes.c_uint, ctypes.c_longlong, ctypes.c_void_p


class Kv4Config(ctypes.Structure):
    _fields_ = [("num_qo_heads", _i), ("num_kv_heads", _i), ("head_dim", _i), ("group_size", _i),
                ("dtype", _i), ("page_size", _i), ("max_decode_reqs", _i), ("device", _i),
                ("flags", _u)]


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


# The C structs are filled with struct.pack, in one call: setting the fields of a
# ctypes.Structure one by one takes longer than the launch.
_CODES = {_i: "i", _ll: "q", _vp: "P", ctypes.c_float: "f"}


def _packer(cls) -> struct.Struct:
    fmt = "".join(_CODES[t] for _, t in cls._fields_)
    n = struct.calcsize(fmt)
    packer = struct.Struct(fmt + "%dx" % (ctypes.sizeof(cls) - n))
    assert packer.size == ctypes.sizeof(cls)
    return packer


_pack_rows = _packer(Kv4RowsArgs).pack
_pack_decode = _packer(Kv4DecodeArgs).pack
_pack_qk = _packer(QkArgs).pack


class Args:
    """The C struct of one call, what that call is (its kind, and the shapes that the struct
    does not hold), and the tensors it points into."""

    __slots__ = ("struct", "call", "device", "keep")

    def __init__(self, packed: bytes, call: tuple, device: int, keep: tuple):
        self.struct, self.call, self.device, self.keep = packed, call, device, keep


_bound = None


def _library() -> ctypes.CDLL:
    global _bound
    if _bound is None:
        lib = load_library()
        lib.pod_qk_norm_rope.argtypes = [_vp, _vp]
        lib.pod_kv4_record_bytes.argtypes = [_i, _i]
        lib.pod_kv4_create.argtypes = [ctypes.POINTER(_vp), ctypes.POINTER(Kv4Config)]
        lib.pod_kv4_write.argtypes = [_vp, _vp, _vp]
        lib.pod_kv4_read.argtypes = [_vp, _vp, _vp]
        lib.pod_kv4_decode.argtypes = [_vp, _vp, _vp]
        lib.pod_kv4_status.argtypes = [_vp, _vp]
        lib.pod_kv4_destroy.argtypes = [_vp]
        for name in EXPORTED:
            getattr(lib, name).restype = ctypes.c_int
        _bound = lib
    return _bound


def _need(ok: bool, what: str) -> None:
    if not ok:
        raise ValueError(what)


def _refuse(device: int, tensors) -> None:
    """Says which (name, tensor, dtype) is no CUDA tensor of that type on that device, or not
    contiguous (a name that ends in "=" need not be)."""
    for name, t, dtype in tensors:
        if t.dtype is not dtype or t.get_device() != device or device < 0:
            raise ValueError("%s: expected a %s CUDA tensor on device %d"
                             % (name.rstrip("="), dtype, device))
        if name[-1] != "=" and not t.is_contiguous():
            raise ValueError("%s: expected a contiguous tensor" % name)


def _raw_stream(stream, device: int) -> int:
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(device)
    return int(stream.cuda_stream)


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
                 max_decode_reqs: int = 1024, device: int = 0, flags: int = 0):
        self._lib = _library()
        self._h = None
        _need(dtype in DTYPES, "dtype: bfloat16 or float16")
        self.cfg = Kv4Config(num_qo_heads, num_kv_heads, head_dim, group_size, DTYPES[dtype],
                             PAGE_SIZE, max_decode_reqs, device, flags)
        h = _vp()
        rc = self._lib.pod_kv4_create(ctypes.byref(h), ctypes.byref(self.cfg))
        if rc != POD_OK:
            raise PodError(rc, "pod_kv4_create")
        self._h = h.value
        self.dtype = dtype
        self.device = int(device)
        self.record = record_bytes(head_dim, group_size)
        self._per_page = (int(num_kv_heads), self.record)
        self._kv = (int(num_kv_heads), int(head_dim))
        self._qo = (int(num_qo_heads), int(head_dim))
        self._rows_call = ("rows", self._kv, self.record, dtype, self.device)
        self._decode_call = ("decode", self._qo, self._kv, self.record, dtype, self.device)

    def new_pool(self, pool_blocks: int) -> torch.Tensor:
        """A zeroed pool (every code and pair stands for 0)."""
        return torch.zeros(pool_blocks, self.cfg.num_kv_heads, self.record, dtype=torch.uint8,
                           device="cuda:%d" % self.device)

    # -- arguments (each keeps its tensors alive)
    def _cache(self, pool, block_table, num_reqs):
        """(blocks in the pool, pages in a row of the table)"""
        ps, ts = pool.shape, block_table.shape
        if ps[1:] != self._per_page:
            raise ValueError("pool: expected [blocks, num_kv_heads, %d]" % self.record)
        if len(ts) != 2 or ts[0] != num_reqs:
            raise ValueError("block_table: expected [num_reqs, pages]")
        return ps[0], ts[1]

    def rows_args(self, cu_rows, start, k, v, pool, block_table) -> Args:
        """``k``, ``v``: [rows, Hk, d], any row and head strides that are multiples of 8."""
        dev, dtype = self.device, self.dtype
        if not (k.dtype is dtype and v.dtype is dtype and cu_rows.dtype is _I32
                and start.dtype is _I32 and pool.dtype is _U8 and block_table.dtype is _I32
                and k.get_device() == dev and v.get_device() == dev
                and cu_rows.get_device() == dev and start.get_device() == dev
                and pool.get_device() == dev and block_table.get_device() == dev
                and cu_rows.is_contiguous() and start.is_contiguous()
                and pool.is_contiguous() and block_table.is_contiguous()):
            _refuse(dev, (("cu_rows", cu_rows, _I32), ("start", start, _I32), ("k=", k, dtype),
                          ("v=", v, dtype), ("pool", pool, _U8), ("block_table", block_table, _I32)))
        n, shape, ks, vs = start.numel(), k.shape, k.stride(), v.stride()
        blocks, pages = self._cache(pool, block_table, n)
        if cu_rows.numel() != n + 1:
            raise ValueError("cu_rows: expected num_reqs + 1 entries")
        if len(shape) != 3 or shape != v.shape or shape[1:] != self._kv:
            raise ValueError("k, v: expected [rows, num_kv_heads, head_dim]")
        if ks[2] != 1 or vs[2] != 1:
            raise ValueError("k, v: expected adjacent channels")
        return Args(_pack_rows(n, shape[0], cu_rows.data_ptr(), start.data_ptr(), k.data_ptr(),
                               v.data_ptr(), ks[0], ks[1], vs[0], vs[1], pool.data_ptr(), blocks,
                               block_table.data_ptr(), pages),
                    self._rows_call, dev, (cu_rows, start, k, v, pool, block_table))

    def decode_args(self, ctx_lens, q, o, lse, pool, block_table) -> Args:
        dev, dtype = self.device, self.dtype
        if not (q.dtype is dtype and o.dtype is dtype and lse.dtype is _F32
                and ctx_lens.dtype is _I32 and pool.dtype is _U8 and block_table.dtype is _I32
                and q.get_device() == dev and o.get_device() == dev and lse.get_device() == dev
                and ctx_lens.get_device() == dev and pool.get_device() == dev
                and block_table.get_device() == dev
                and q.is_contiguous() and o.is_contiguous() and lse.is_contiguous()
                and ctx_lens.is_contiguous() and pool.is_contiguous()
                and block_table.is_contiguous()):
            _refuse(dev, (("ctx_lens", ctx_lens, _I32), ("q", q, dtype), ("o", o, dtype),
                          ("lse", lse, _F32), ("pool", pool, _U8), ("block_table", block_table, _I32)))
        n, shape = ctx_lens.numel(), q.shape
        blocks, pages = self._cache(pool, block_table, n)
        if shape != (n, *self._qo) or o.shape != shape:
            raise ValueError("q, o: expected [num_reqs, num_qo_heads, head_dim]")
        if lse.shape != shape[:2]:
            raise ValueError("lse: expected [num_reqs, num_qo_heads]")
        return Args(_pack_decode(n, ctx_lens.data_ptr(), q.data_ptr(), o.data_ptr(),
                                 lse.data_ptr(), pool.data_ptr(), blocks, block_table.data_ptr(),
                                 pages),
                    self._decode_call, dev, (ctx_lens, q, o, lse, pool, block_table))

    # -- calls
    def write(self, args: Args, stream=None) -> None:
        if args.call is not self._rows_call and args.call != self._rows_call:
            raise ValueError("write: expected rows_args of this cache's shape")
        rc = self._lib.pod_kv4_write(self._h, args.struct, _raw_stream(stream, self.device))
        if rc != POD_OK:
            self._failed(rc, "pod_kv4_write")

    def read(self, args: Args, stream=None) -> None:
        if args.call is not self._rows_call and args.call != self._rows_call:
            raise ValueError("read: expected rows_args of this cache's shape")
        rc = self._lib.pod_kv4_read(self._h, args.struct, _raw_stream(stream, self.device))
        if rc != POD_OK:
            self._failed(rc, "pod_kv4_read")

    def decode(self, args: Args, stream=None) -> None:
        if args.call is not self._decode_call and args.call != self._decode_call:
            raise ValueError("decode: expected decode_args of this cache's shape")
        rc = self._lib.pod_kv4_decode(self._h, args.struct, _raw_stream(stream, self.device))
        if rc != POD_OK:
            self._failed(rc, "pod_kv4_decode")

    def hybrid(self, pod: PodAttention, qkv, positions, cos_sin, *, chunk_lens: Sequence[int],
               prior_lens: Sequence[int], cu_rows, start, ctx_lens, pool, block_table,
               q_weight=None, k_weight=None, eps: float = 1e-6, interleaved: bool = False,
               stream=None):
        """One layer's attention of a hybrid batch over the 4-bit cache: the counterpart of
        :meth:`PodAttention.hybrid` from the projection's output on. Returns O and LSE.

        ``qkv`` [rows, H + 2 Hk, d] holds the chunks of the prefill requests and then one row
        for each decode; its k heads are normed and rotated in place (q's in a tensor of their
        own). ``chunk_lens`` and ``prior_lens`` are host lengths as in :meth:`PodAttention.prefill_args`; ``cu_rows``,
        ``start`` and ``block_table`` cover all requests, the prefills first, and ``ctx_lens``
        the decodes (their new token included). The new K and V go into the cache; decodes
        attend over it; the prefills' contexts are read back for ``pod``, a context of the
        contiguous layout, which takes bf16 (an fp16 cache has decodes only).

        Asynchronous like the calls it makes. What can be refused is refused before anything is
        enqueued. A call without prefills can be captured; one with prefills, whose plan is made
        on the host, raises POD_EUNSUPPORTED then."""
        H, Hk, d = self.cfg.num_qo_heads, self.cfg.num_kv_heads, self.cfg.head_dim
        chunk_lens, prior_lens = [int(n) for n in chunk_lens], [int(n) for n in prior_lens]
        if len(prior_lens) != len(chunk_lens) or min(chunk_lens + prior_lens, default=0) < 0:
            raise ValueError("chunk_lens, prior_lens: expected as many of each, none negative")
        n_pre, rows = len(chunk_lens), qkv.shape[0]
        chunk_rows = sum(chunk_lens)
        if qkv.dim() != 3 or qkv.shape[1:] != (H + 2 * Hk, d):
            raise ValueError("qkv: expected [rows, num_qo_heads + 2 num_kv_heads, head_dim]")
        if rows != chunk_rows + ctx_lens.numel() or start.numel() != n_pre + ctx_lens.numel():
            raise ValueError("qkv, start: expected the chunks' rows and one for each decode")
        if n_pre and (pod.paged or self.dtype is not torch.bfloat16):
            raise ValueError("prefills: expected a contiguous-layout context and bfloat16")
        # prefill_args hands on pointers alone: the context has to read and write what is behind them
        if n_pre and any(getattr(pod.cfg, x) != getattr(self.cfg, x) for x in
                         ("num_qo_heads", "num_kv_heads", "head_dim", "device")):
            raise ValueError("pod: expected a context of this cache's heads, head_dim and device")
        # K is rotated in place and the cache written before decodes and prefills are called: what
        # they would refuse is refused here, ahead of the first launch
        lens = [p + c for p, c in zip(prior_lens, chunk_lens)]
        n_all = start.numel()
        if (ctx_lens.numel() > self.cfg.max_decode_reqs or rows > 1 << 30 or sum(lens) > 1 << 30
                or n_all * (block_table.shape[-1] + 8) > 2 ** 31 - 1 or block_table.shape[-1] > 1 << 26
                or pool.shape[0] * Hk > 2 ** 31 - 1
                or chunk_rows and (n_pre > pod.cfg.max_prefill_reqs
                                   or chunk_rows > pod.cfg.max_prefill_tokens
                                   or any(c and n > pod.cfg.max_kv_tokens
                                          for c, n in zip(chunk_lens, lens)))):
            raise PodError(POD_ECAPACITY, "PodKv4.hybrid")
        if pool.shape[0] == 0 or pool.data_ptr() % 16:
            raise ValueError("pool: expected pages, 16-byte aligned")
        _need(self._h is not None and not (chunk_rows and pod._h is None), "the context is closed")
        if stream is None:
            stream = torch.cuda.current_stream(self.device)
        with torch.cuda.stream(stream):
            if chunk_rows and torch.cuda.is_current_stream_capturing():
                raise PodError(POD_EUNSUPPORTED, "PodKv4.hybrid of prefills in a captured stream")
            q = torch.empty(rows, H, d, dtype=self.dtype, device=qkv.device)
            o = torch.empty_like(q)
            lse = torch.empty(rows, H, dtype=torch.float32, device=qkv.device)
            k, v = qkv[:, H:H + Hk], qkv[:, H + Hk:]
            rope = norm_rope_args(qkv[:, :H], k, positions, cos_sin, q_out=q, q_weight=q_weight,
                                  k_weight=k_weight, eps=eps, interleaved=interleaved)
            write = self.rows_args(cu_rows, start, k, v, pool, block_table)
            if rows > chunk_rows:
                decode = self.decode_args(ctx_lens, q[chunk_rows:], o[chunk_rows:],
                                          lse[chunk_rows:], pool, block_table[n_pre:])
            if chunk_rows:
                # (from pinned memory: the call does not wait for the stream)
                cu = torch.tensor([sum(lens[:i]) for i in range(n_pre + 1)] + [0] * n_pre,
                                  dtype=torch.int32, pin_memory=True)
                cu = cu.to(qkv.device, non_blocking=True)
                kc = torch.empty(sum(lens), Hk, d, dtype=self.dtype, device=qkv.device)
                vc = torch.empty_like(kc)
                read = self.rows_args(cu[:n_pre + 1], cu[n_pre + 1:], kc, vc, pool,
                                      block_table[:n_pre])
                prefill = pod.prefill_args(chunk_lens, prior_lens, q[:chunk_rows], o[:chunk_rows],
                                           lse[:chunk_rows], k=list(kc.split(lens)),
                                           v=list(vc.split(lens)))
            qk_norm_rope(rope, stream)
            self.write(write, stream)
            if rows > chunk_rows:
                self.decode(decode, stream)
            if chunk_rows:
                self.read(read, stream)
                pod.prefill_only(prefill, stream)
        return o, lse

    def status(self, stream=None) -> int:
        """``pod_kv4_status``: synchronises the stream; POD_ETIMEOUT after a wait that ran out."""
        return int(self._lib.pod_kv4_status(self._h, _raw_stream(stream, self.device)))

    def _failed(self, rc: int, name: str) -> None:
        _need(self._h is not None, "the context is closed")
        raise PodError(rc, name)

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


_NOTHING = (0, 0, 0, 0, 0, 0, 0)  # a side that is left out
_ROPE_CALL = ("norm_rope",)


def _side(name, x, out, weight, rows, d, dtype, device):
    """(heads, rows, output, the four strides) of q or k, and its weight."""
    if out is None:
        out = x
    if not (x.dtype is dtype and out.dtype is dtype and device >= 0
            and x.get_device() == device and out.get_device() == device):
        _refuse(device, ((name + "=", x, dtype), (name + "_out=", out, dtype)))
    shape, xs, os = x.shape, x.stride(), out.stride()
    if len(shape) != 3 or shape[0] != rows or shape[2] != d or out.shape != shape:
        raise ValueError("%s: expected [rows, heads, head_dim], and its output alike" % name)
    if xs[2] != 1 or os[2] != 1:
        raise ValueError("%s: expected adjacent channels" % name)
    w = 0
    if weight is not None:
        if weight.dtype is not dtype or weight.get_device() != device or not weight.is_contiguous():
            _refuse(device, ((name + "_weight", weight, dtype),))
        if weight.shape != (d,):
            raise ValueError("%s_weight: expected [head_dim]" % name)
        w = weight.data_ptr()
    return (shape[1], x.data_ptr(), out.data_ptr(), xs[0], xs[1], os[0], os[1]), w


def norm_rope_args(q: Optional[torch.Tensor], k: Optional[torch.Tensor], positions: torch.Tensor,
                   cos_sin: torch.Tensor, *, q_out: Optional[torch.Tensor] = None,
                   k_out: Optional[torch.Tensor] = None,
                   q_weight: Optional[torch.Tensor] = None,
                   k_weight: Optional[torch.Tensor] = None, eps: float = 1e-6,
                   interleaved: bool = False) -> Args:
    """``q`` [rows, H, d] and ``k`` [rows, Hk, d] (either may be None), with any
    row and head strides that are multiples of 8. Without ``q_out`` / ``k_out``
    the rows are replaced in place; without a weight that side is only rotated."""
    some = q if q is not None else k
    if some is None:
        raise ValueError("q or k is needed")
    device, dtype, size = some.get_device(), some.dtype, some.shape
    rows, d = size[0], size[-1]
    if dtype not in DTYPES:
        raise ValueError("q, k: bfloat16 or float16")
    qs, qw = (_NOTHING, 0) if q is None else _side("q", q, q_out, q_weight, rows, d, dtype, device)
    ks, kw = (_NOTHING, 0) if k is None else _side("k", k, k_out, k_weight, rows, d, dtype, device)
    if not (positions.dtype is _I32 and cos_sin.dtype is _F32
            and positions.get_device() == device and cos_sin.get_device() == device
            and positions.is_contiguous() and cos_sin.is_contiguous()):
        _refuse(device, (("positions", positions, _I32), ("cos_sin", cos_sin, _F32)))
    angles = cos_sin.shape
    if positions.shape != (rows,):
        raise ValueError("positions: expected [rows]")
    if len(angles) != 2:
        raise ValueError("cos_sin: expected [max_position, rot_dim]")
    far, rot = angles
    return Args(_pack_qk(qs[0], ks[0], d, rot, 1 if interleaved else 0, DTYPES[dtype], device, rows,
                         qs[1], ks[1], qs[2], ks[2], qs[3], qs[4], ks[3], ks[4], qs[5], qs[6],
                         ks[5], ks[6], qw, kw, eps, positions.data_ptr(), cos_sin.data_ptr(), far),
                _ROPE_CALL, device, (q, k, positions, cos_sin, q_out, k_out, q_weight, k_weight))


def qk_norm_rope(args: Args, stream=None) -> None:
    """``pod_qk_norm_rope``: per-head RMS norm of q and k and the rotation, in one launch."""
    if args.call is not _ROPE_CALL and args.call != _ROPE_CALL:
        raise ValueError("qk_norm_rope: expected norm_rope_args")
    rc = _library().pod_qk_norm_rope(args.struct, _raw_stream(stream, args.device))
    if rc != POD_OK:
        raise PodError(rc, "pod_qk_norm_rope")
