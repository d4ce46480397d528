"""The 4-bit KV cache on the host: symbols, the record's size, and every argument that is refused
before anything is enqueued (no GPU needed)."""
import ctypes
import os
import re
import subprocess

import pytest
import torch

import kv4_ref as ref
from hybrid_prefill_decode_pod_b200 import build as B
from hybrid_prefill_decode_pod_b200 import pod_attn as pa
from hybrid_prefill_decode_pod_b200 import pod_kv4 as p4

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PAST_THE_CHECKS = (pa.POD_OK, pa.POD_ECUDA)   # ECUDA: there is no device here


@pytest.fixture(scope="module")
def lib():
    B.build()
    return p4._library()


@pytest.fixture(scope="module")
def harness(tmp_path_factory):
    out = str(tmp_path_factory.mktemp("kv4") / "kv4_harness.so")
    subprocess.check_call([B.nvcc(), "-std=c++17", "-shared", "-Xcompiler", "-fPIC", "-I", B.INCLUDE, "-I", B.CSRC,
                           "-o", out, os.path.join(ROOT, "tests", "kv4_harness.cpp"), "-lcudart"])
    h = ctypes.CDLL(out)
    h.harness_ctx.restype = ctypes.c_void_p
    h.harness_ctx.argtypes = [ctypes.POINTER(p4.Kv4Config)]
    h.harness_free.argtypes = [ctypes.c_void_p]
    vp = ctypes.c_void_p
    h.pod_qk_norm_rope.argtypes = [ctypes.POINTER(p4.QkArgs), vp]
    for name, t in (("write", p4.Kv4RowsArgs), ("read", p4.Kv4RowsArgs), ("decode", p4.Kv4DecodeArgs)):
        getattr(h, "pod_kv4_" + name).argtypes = [vp, ctypes.POINTER(t), vp]
    return h


@pytest.fixture(scope="module")
def ctx(harness):
    c = harness.harness_ctx(ctypes.byref(p4.Kv4Config(32, 8, 128, 64, 0, 16, 64, 0)))
    yield c
    harness.harness_free(c)


def test_header_and_library_agree(lib):
    text = open(os.path.join(ROOT, "include", "pod_kv4.h")).read()
    syms = re.findall(r"POD_API\s+[\w\s\*]*?\b(pod_\w+)\s*\(", text)
    assert sorted(set(syms)) == sorted(p4.EXPORTED)
    raw = ctypes.CDLL(pa.LIB_PATH)
    assert all(hasattr(raw, s) for s in syms)


@pytest.mark.parametrize("d,group", [(64, 32), (64, 64), (128, 32), (128, 64), (128, 128)])
def test_record_layout_is_whole(lib, d, group):
    n = p4.record_bytes(d, group)
    assert n == 16 * d + 128 * d // group and n % 16 == 0
    code, pair = ref.places(d, group)
    assert torch.equal(code.flatten().sort().values, torch.arange(32 * d))
    assert pair.max() == (n - 16 * d) // 4 - 1
    # a byte never holds two tokens
    owner = {}
    for t in range(16):
        for b in (code[:, t] // 2).flatten().tolist():
            assert owner.setdefault(b, t) == t


@pytest.mark.parametrize("d,group", [(96, 32), (64, 128), (128, 16), (128, 0), (0, 0), (256, 64)])
def test_record_bytes_refuses(lib, d, group):
    assert lib.pod_kv4_record_bytes(d, group) == pa.POD_EUNSUPPORTED


@pytest.mark.parametrize("kw,code", [
    (dict(num_qo_heads=0), pa.POD_EINVAL), (dict(num_kv_heads=3), pa.POD_EINVAL), (dict(max_decode_reqs=0), pa.POD_EINVAL),
    (dict(head_dim=96), pa.POD_EUNSUPPORTED), (dict(group_size=48), pa.POD_EUNSUPPORTED), (dict(num_kv_heads=2), pa.POD_EUNSUPPORTED),
    (dict(page_size=32), pa.POD_EUNSUPPORTED), (dict(dtype=2), pa.POD_EUNSUPPORTED), (dict(head_dim=64, group_size=128), pa.POD_EUNSUPPORTED),
    (dict(max_decode_reqs=4097), pa.POD_ECAPACITY),
])
def test_create_refuses(lib, kw, code):
    base = dict(num_qo_heads=32, num_kv_heads=8, head_dim=128, group_size=64, dtype=0, page_size=16, max_decode_reqs=64, device=0)
    base.update(kw)
    h = ctypes.c_void_p()
    assert lib.pod_kv4_create(ctypes.byref(h), ctypes.byref(p4.Kv4Config(*base.values()))) == code and not h.value


def test_null_arguments(lib):
    h = ctypes.c_void_p()
    assert lib.pod_kv4_create(None, None) == pa.POD_EINVAL
    assert lib.pod_kv4_create(ctypes.byref(h), None) == pa.POD_EINVAL
    assert lib.pod_qk_norm_rope(None, None) == pa.POD_EINVAL
    for f in (lib.pod_kv4_write, lib.pod_kv4_read, lib.pod_kv4_decode):
        assert f(None, None, None) == pa.POD_EINVAL
    assert lib.pod_kv4_destroy(None) == pa.POD_OK


def rows(**kw):
    a = dict(num_reqs=2, num_rows=10, cu_rows=0x1000, start=0x2000, k=0x10000, v=0x20000, k_row_stride=1024, k_head_stride=128,
             v_row_stride=1024, v_head_stride=128, pool=0x100000, pool_blocks=100, block_table=0x3000, block_table_stride=7)
    a.update(kw)
    return p4.Kv4RowsArgs(**a)


BAD_ROWS = [
    (dict(num_reqs=-1), pa.POD_EINVAL), (dict(num_rows=-1), pa.POD_EINVAL), (dict(cu_rows=None), pa.POD_EINVAL), (dict(start=None), pa.POD_EINVAL),
    (dict(k=None), pa.POD_EINVAL), (dict(v=None), pa.POD_EINVAL), (dict(pool=None), pa.POD_EINVAL), (dict(block_table=None), pa.POD_EINVAL),
    (dict(k=0x10008), pa.POD_EINVAL), (dict(v=0x20002), pa.POD_EINVAL), (dict(pool=0x100008), pa.POD_EINVAL), (dict(cu_rows=0x1002), pa.POD_EINVAL),
    (dict(k_row_stride=1020), pa.POD_EINVAL), (dict(v_head_stride=-128), pa.POD_EINVAL), (dict(pool_blocks=0), pa.POD_EINVAL),
    (dict(block_table_stride=-1), pa.POD_EINVAL), (dict(pool_blocks=1 << 29), pa.POD_ECAPACITY), (dict(num_reqs=1 << 30), pa.POD_ECAPACITY),
    (dict(num_rows=(1 << 30) + 1), pa.POD_ECAPACITY),
]


@pytest.mark.parametrize("kw,code", BAD_ROWS)
@pytest.mark.parametrize("name", ["write", "read"])
def test_rows_refused(harness, ctx, name, kw, code):
    before = harness.harness_launches()
    assert getattr(harness, "pod_kv4_" + name)(ctx, ctypes.byref(rows(**kw)), None) == code
    assert harness.harness_launches() == before


@pytest.mark.parametrize("kw,read_ok", [
    (dict(), True), (dict(k_row_stride=0), False), (dict(k_head_stride=0), False), (dict(v_head_stride=64), False),
    (dict(k_row_stride=512), False),                       # rows of 8 heads that overlap
    (dict(k_row_stride=128, k_head_stride=1280), True),    # heads outermost
    (dict(num_rows=1, k_row_stride=3), True),              # the stride of a single row says nothing
])
def test_rows_strides(harness, ctx, kw, read_ok):
    """Any rows may be read twice or overlap; rows that are written may not."""
    assert harness.pod_kv4_write(ctx, ctypes.byref(rows(**kw)), None) in PAST_THE_CHECKS
    rc = harness.pod_kv4_read(ctx, ctypes.byref(rows(**kw)), None)
    assert rc in PAST_THE_CHECKS if read_ok else rc == pa.POD_EINVAL


def test_rows_of_nothing(harness, ctx):
    for name in ("write", "read"):
        for kw in (dict(num_reqs=0, start=None, block_table=None), dict(num_rows=0, k=None, v=None)):
            assert getattr(harness, "pod_kv4_" + name)(ctx, ctypes.byref(rows(**kw)), None) == pa.POD_OK


@pytest.mark.parametrize("kw,code", [
    (dict(), None), (dict(block_table_stride=0), None), (dict(num_reqs=0, q=None), pa.POD_OK), (dict(num_reqs=-1), pa.POD_EINVAL),
    (dict(num_reqs=65), pa.POD_ECAPACITY),
    (dict(ctx_lens=None), pa.POD_EINVAL), (dict(q=None), pa.POD_EINVAL), (dict(o=None), pa.POD_EINVAL), (dict(lse=None), pa.POD_EINVAL),
    (dict(q=0x10004), pa.POD_EINVAL), (dict(o=0x20008), pa.POD_EINVAL), (dict(lse=0x30002), pa.POD_EINVAL), (dict(ctx_lens=0x1001), pa.POD_EINVAL),
    (dict(pool=0x100004), pa.POD_EINVAL), (dict(pool_blocks=-4), pa.POD_EINVAL), (dict(pool_blocks=1 << 28), pa.POD_ECAPACITY),
    (dict(block_table_stride=1 << 27), pa.POD_ECAPACITY),
])
def test_decode_refused(harness, ctx, kw, code):
    a = dict(num_reqs=2, ctx_lens=0x1000, q=0x10000, o=0x20000, lse=0x30000, pool=0x100000, pool_blocks=100, block_table=0x3000, block_table_stride=7)
    a.update(kw)
    rc = harness.pod_kv4_decode(ctx, ctypes.byref(p4.Kv4DecodeArgs(**a)), None)
    assert rc == code if code is not None else rc in PAST_THE_CHECKS


@pytest.mark.parametrize("kw,code", [
    (dict(), None), (dict(num_rows=0, q=None), pa.POD_OK), (dict(num_qo_heads=0, q=None, q_out=None), None), (dict(q_out=0x10000), None),
    (dict(num_qo_heads=0, num_kv_heads=0), pa.POD_OK), (dict(q_weight=None, k_weight=None), None), (dict(q_row_stride=0), None),
    (dict(head_dim=80), pa.POD_EUNSUPPORTED), (dict(rot_dim=0), pa.POD_EUNSUPPORTED), (dict(rot_dim=24), pa.POD_EUNSUPPORTED),
    (dict(rot_dim=144), pa.POD_EUNSUPPORTED), (dict(dtype=5), pa.POD_EUNSUPPORTED), (dict(interleaved=2), pa.POD_EINVAL),
    (dict(eps=-1.0), pa.POD_EINVAL), (dict(eps=float("nan")), pa.POD_EINVAL), (dict(max_position=-1), pa.POD_EINVAL), (dict(num_rows=-1), pa.POD_EINVAL),
    (dict(q=None), pa.POD_EINVAL), (dict(k_out=None), pa.POD_EINVAL), (dict(positions=None), pa.POD_EINVAL), (dict(cos_sin=None), pa.POD_EINVAL),
    (dict(cos_sin=0x4004), pa.POD_EINVAL), (dict(q_weight=0x5002), pa.POD_EINVAL), (dict(k=0x20008), pa.POD_EINVAL),
    (dict(q_out_row_stride=0), pa.POD_EINVAL), (dict(q_head_stride=4), pa.POD_EINVAL), (dict(k_out_head_stride=64), pa.POD_EINVAL),
    (dict(q_out=0x10000, q_out_row_stride=8192), pa.POD_EINVAL),   # in place with other strides
    (dict(num_rows=(1 << 30) + 1), pa.POD_ECAPACITY), (dict(num_qo_heads=1 << 17), pa.POD_ECAPACITY),
])
def test_norm_rope_refused(harness, kw, code):
    a = dict(num_qo_heads=32, num_kv_heads=8, head_dim=128, rot_dim=128, interleaved=0, dtype=0, device=0, num_rows=10, q=0x10000, k=0x20000,
             q_out=0x30000, k_out=0x40000, q_row_stride=4096, q_head_stride=128, k_row_stride=1024, k_head_stride=128,
             q_out_row_stride=4096, q_out_head_stride=128, k_out_row_stride=1024, k_out_head_stride=128, q_weight=0x5000, k_weight=0x6000,
             eps=1e-6, positions=0x7000, cos_sin=0x4000, max_position=100)
    a.update(kw)
    rc = harness.pod_qk_norm_rope(ctypes.byref(p4.QkArgs(**a)), None)
    assert rc == code if code is not None else rc in PAST_THE_CHECKS


@pytest.fixture(scope="module")
def split(harness):
    """pod_kv4_split.h's functions over a batch: blocks of each request and the KV heads."""
    ll, i32, ptr = ctypes.c_longlong, ctypes.c_int, ctypes.POINTER(ctypes.c_int)
    for name, res, args in (("begin", ll, [ll, i32, i32]), ("cost", i32, [i32]), ("workers", i32, [ll, i32, i32]), ("snap", ll, [ptr, i32, i32, ll]),
                            ("cut", ll, [ptr, ptr, i32, i32, ll]), ("worker", i32, [ptr, i32, i32, i32, i32, i32, i32]),
                            ("place", None, [ptr, i32, i32, ll, ptr])):
        f = getattr(harness, "harness_" + name)
        f.restype, f.argtypes = res, args
    return harness


def prefix(xs):
    return (ctypes.c_int * (len(xs) + 1))(*[sum(xs[:i]) for i in range(len(xs) + 1)])


BATCHES = [([1], 1), ([0, 5, 0, 0, 17, 1, 0], 3), ([100] * 9, 8), ([4000, 1], 2), ([0, 0, 33], 5), ([1, 2, 3, 4, 5, 6, 7, 64] * 5, 2)]


@pytest.mark.parametrize("lens,Hk", BATCHES)
def test_places_on_the_line(split, lens, Hk):
    first, out = prefix(lens), (ctypes.c_int * 4)()
    want = [(r, h, b, n) for r, n in enumerate(lens) for h in range(Hk) for b in range(n)]
    for x in range(len(want)):
        split.harness_place(first, len(lens), Hk, x, out)
        assert tuple(out) == want[x]


@pytest.mark.parametrize("lens,Hk", BATCHES)
@pytest.mark.parametrize("ctas,least", [(148, 16), (7, 16), (1, 16), (296, 16)])
def test_work_is_cut_into_parts_of_equal_cost(split, lens, Hk, ctas, least):
    """Each block belongs to one worker, the one that kv4_worker names; every worker has one; the parts' costs differ by one."""
    R, W = len(lens), sum(lens) * Hk
    costs = [split.harness_cost(n) for n in lens]
    assert all(c == (0 if n == 0 else (n + 3) // 4 * 4 + 4) for c, n in zip(costs, lens))
    first, cost, V = prefix(lens), prefix(costs), sum(costs) * Hk
    N = split.harness_workers(W, ctas, least)
    assert 1 <= N <= ctas and (N == 1 or W // N >= least)
    at = [split.harness_begin(V, N, c) for c in range(N + 1)]
    assert at[0] == 0 and at[-1] == V and max(b - a for a, b in zip(at, at[1:])) <= V // N + 1
    cut = [split.harness_cut(first, cost, R, Hk, v) for v in at]
    assert cut[0] == 0 and cut[-1] == W and all(a < b for a, b in zip(cut, cut[1:]))
    x = 0
    for r, n in enumerate(lens):
        for h in range(Hk):
            for b in range(n):
                c = split.harness_worker(cost, R, Hk, N, r, h, b)
                assert cut[c] <= x < cut[c + 1]
                x += 1
    # a worker's warps: in order, from its first block to its last
    for a, b in zip(at, at[1:]):
        inner = [split.harness_cut(first, cost, R, Hk, a + split.harness_begin(b - a, 8, i)) for i in range(9)]
        assert inner == sorted(inner) and inner[0] == cut[at.index(a)] and inner[-1] == cut[at.index(b)]


@pytest.mark.parametrize("lens,Hk", BATCHES)
@pytest.mark.parametrize("N", [1, 5, 148])
def test_cuts_moved_to_segment_boundaries(split, lens, Hk, N):
    """In order, by no more than half a segment, and no segment lies in two parts."""
    R = len(lens)
    costs = [split.harness_cost(n) for n in lens]
    first, cost, V = prefix(lens), prefix(costs), sum(costs) * Hk
    ends = {sum(costs[:r]) * Hk + h * c for r, c in enumerate(costs) for h in range(Hk + 1)}
    blocks = {sum(lens[:r]) * Hk + h * n for r, n in enumerate(lens) for h in range(Hk + 1)}
    at = [split.harness_begin(V, N, c) for c in range(N + 1)]
    moved = [split.harness_snap(cost, R, Hk, v) for v in at]
    assert moved[0] == 0 and moved[-1] == V and moved == sorted(moved) and set(moved) <= ends
    assert all(2 * abs(m - v) <= max(costs) for m, v in zip(moved, at))
    assert {split.harness_cut(first, cost, R, Hk, v) for v in moved} <= blocks


def test_work_of_the_largest_calls(split):
    """The products of the cut stay in 64 bits at the largest tables: 2^31 blocks of 512 heads."""
    n, Hk, N = 2 ** 31 - 1 - 64, 512, 148 * 4
    first, cost = prefix([n]), prefix([split.harness_cost(n)])
    V = cost[1] * Hk
    assert split.harness_cut(first, cost, 1, Hk, V) == n * Hk
    for c in (0, 1, 300, N - 1):
        v = split.harness_begin(V, N, c)
        assert v == c * V // N
        x = split.harness_cut(first, cost, 1, Hk, v)
        h, blk = divmod(x, n)
        assert split.harness_worker(cost, 1, Hk, N, 0, h, blk) == c


def test_rope_table_is_exact_far_out():
    t = p4.rope_table(200001, 64, 10000.0, device="cpu")
    assert t.shape == (200001, 64) and t.dtype == torch.float32
    import math
    for pos, i in ((200000, 0), (199999, 3), (123456, 31)):
        a = pos * 10000.0 ** (-2 * i / 64)
        assert abs(t[pos, i].item() - math.cos(a)) < 1e-7 and abs(t[pos, 32 + i].item() - math.sin(a)) < 1e-7


def test_packed_structs_are_the_c_structs():
    """What the binding packs is what the ctypes mirror of the header's struct reads."""
    for cls, pack in ((p4.Kv4RowsArgs, p4._pack_rows), (p4.Kv4DecodeArgs, p4._pack_decode), (p4.QkArgs, p4._pack_qk)):
        values = [float(i) + 0.5 if t is ctypes.c_float else 1000 + i for i, (_, t) in enumerate(cls._fields_)]
        got = cls.from_buffer_copy(pack(*values))
        assert [getattr(got, name) for name, _ in cls._fields_] == values


def test_binding_refuses_tensors_of_the_host():
    x = torch.zeros(2, 4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        p4.norm_rope_args(x, x, torch.zeros(2, dtype=torch.int32), torch.zeros(5, 64))


@pytest.mark.parametrize("flags,code", [(4, pa.POD_EUNSUPPORTED), (1, pa.POD_EUNSUPPORTED)])
def test_create_refuses_flags(lib, flags, code):
    h = ctypes.c_void_p()
    assert lib.pod_kv4_create(ctypes.byref(h), ctypes.byref(p4.Kv4Config(32, 8, 128, 64, 0, 16, 64, 0, flags))) == code and not h.value


def test_status_of_nothing(lib):
    assert lib.pod_kv4_status(None, None) == pa.POD_EINVAL


def unopened(cls, cfg, **kw):
    """A binding object without a library context: for what is refused before any call."""
    x = object.__new__(cls)
    x.cfg, x._h = cfg, None
    for k, v in kw.items():
        setattr(x, k, v)
    return x


def hybrid_call(pod_cfg=(), **kw):
    """PodKv4.hybrid of two chunks and a decode on host tensors, 8 / 2 heads of 128."""
    kv = unopened(p4.PodKv4, p4.Kv4Config(8, 2, 128, 64, 0, 16, 4, 0), dtype=torch.bfloat16, device=0, record=2304, _per_page=(2, 2304),
                  _kv=(2, 128), _qo=(8, 128))
    cfg = dict(num_qo_heads=8, num_kv_heads=2, head_dim=128, kv_layout=0, page_size=0, max_prefill_reqs=2, max_prefill_tokens=64, max_decode_reqs=1,
               max_kv_tokens=128, device=0, flags=0)
    cfg.update(pod_cfg)
    pod = unopened(pa.PodAttention, pa.Config(*cfg.values()), paged=False)
    chunks, n = kw.pop("chunk_lens", [5, 3]), kw.pop("decodes", 1)
    rows = max(0, sum(chunks)) + n
    i32 = lambda k: torch.zeros(k, dtype=torch.int32)  # noqa: E731
    a = dict(qkv=torch.zeros(rows, 12, 128, dtype=torch.bfloat16), positions=i32(rows), cos_sin=torch.zeros(200, 128), chunk_lens=chunks,
             prior_lens=[10, 0], cu_rows=i32(len(chunks) + n + 1), start=i32(len(chunks) + n), ctx_lens=i32(n),
             pool=torch.zeros(20, 2, 2304, dtype=torch.uint8), block_table=torch.zeros(len(chunks) + n, 8, dtype=torch.int32))
    a.update(kw)
    return kv.hybrid(pod, **a)


@pytest.mark.parametrize("cfg", [dict(num_qo_heads=16), dict(num_kv_heads=8), dict(head_dim=64), dict(device=1)])
def test_hybrid_refuses_another_shapes_context(cfg):
    with pytest.raises(ValueError, match="pod: expected a context of this cache's heads"):
        hybrid_call(cfg)


@pytest.mark.parametrize("kw", [dict(prior_lens=[10]), dict(prior_lens=[10, 0, 7]), dict(prior_lens=[]), dict(prior_lens=[10, -1]),
                                dict(chunk_lens=[9, -1])])
def test_hybrid_refuses_lengths_that_do_not_fit(kw):
    """A short list of prior lengths would be read behind its end."""
    with pytest.raises(ValueError, match="chunk_lens, prior_lens"):
        hybrid_call(**kw)


@pytest.mark.parametrize("pod_cfg,kw", [
    (dict(), dict(decodes=5)),                                   # the cache's context takes 4 decodes
    (dict(), dict(chunk_lens=[1] * 3, prior_lens=[0] * 3)), (dict(max_prefill_tokens=7), dict()), (dict(max_kv_tokens=14), dict()),
    (dict(max_kv_tokens=2), dict(chunk_lens=[0, 1], prior_lens=[0, 2])),
])
def test_hybrid_refuses_sizes_before_it_changes_anything(pod_cfg, kw):
    with pytest.raises(pa.PodError) as e:
        hybrid_call(pod_cfg, **kw)
    assert e.value.code == pa.POD_ECAPACITY


@pytest.mark.parametrize("pool", [torch.zeros(0, 2, 2304, dtype=torch.uint8), torch.zeros(2 * 2304 + 8, dtype=torch.uint8)[8:].view(1, 2, 2304)])
def test_hybrid_refuses_a_pool_that_no_call_takes(pool):
    with pytest.raises(ValueError, match="pool"):
        hybrid_call(pool=pool)


def test_hybrid_of_closed_contexts():
    with pytest.raises(ValueError, match="closed"):
        hybrid_call()


def test_arguments_of_another_call_are_refused():
    """Their structs would be read as something else: other kinds, other heads, records, types and devices."""
    calls = {"rows": ("rows", (2, 128), 2304, torch.bfloat16, 0), "decode": ("decode", (8, 128), (2, 128), 2304, torch.bfloat16, 0)}
    kv = unopened(p4.PodKv4, p4.Kv4Config(8, 2, 128, 64, 0, 16, 4, 0), _rows_call=calls["rows"], _decode_call=calls["decode"])
    others = [("rows", (4, 128), 2304, torch.bfloat16, 0), ("rows", (2, 128), 2560, torch.bfloat16, 0), ("rows", (2, 128), 2304, torch.float16, 0),
              ("rows", (2, 128), 2304, torch.bfloat16, 1), ("decode", (16, 128), (2, 128), 2304, torch.bfloat16, 0), p4._ROPE_CALL]
    for name, f, own in (("write", kv.write, "rows"), ("read", kv.read, "rows"), ("decode", kv.decode, "decode"), ("qk_norm_rope", p4.qk_norm_rope, None)):
        for call in others + list(calls.values()):
            if call != calls.get(own) and not (own is None and call == p4._ROPE_CALL):
                with pytest.raises(ValueError, match=name + ": expected"):
                    f(p4.Args(b"", call, 0, ()))
