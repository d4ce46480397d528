"""The 4-bit KV cache on the GPU against its formulas in 64 bits."""
import math

import pytest
import torch

import kv4_ref as ref
from hybrid_prefill_decode_pod_b200 import pod_attn as pa
from hybrid_prefill_decode_pod_b200 import pod_kv4 as p4

pytestmark = pytest.mark.gpu

BF, HF = torch.bfloat16, torch.float16
GROUPS = [(64, 32), (64, 64), (128, 32), (128, 64), (128, 128)]


def gen(seed):
    return torch.Generator().manual_seed(seed)


def table_for(pages, blocks, g):
    """A block table with the pages of each request anywhere in the pool; the rest is -1."""
    ids = torch.randperm(blocks, generator=g)[:sum(pages)].to(torch.int32)
    t = torch.full((len(pages), max(pages + [1])), -1, dtype=torch.int32)
    at = 0
    for r, n in enumerate(pages):
        t[r, :n] = ids[at:at + n]
        at += n
    return t


def random_pool(blocks, Hk, d, group, g, wild=False):
    """Records of random codes and pairs; `wild`: pairs of any bits, NaN and infinities too."""
    rec = p4.record_bytes(d, group)
    pool = torch.randint(0, 256, (blocks, Hk, rec), generator=g, dtype=torch.uint8)
    if not wild:
        n = (rec - 16 * d) // 4
        s = 0.05 + 0.3 * torch.rand(blocks, Hk, n, generator=g)
        m = -s * (7.5 + torch.randn(blocks, Hk, n, generator=g))
        pool[..., 16 * d:] = torch.stack([s, m], -1).half().flatten(-2).contiguous().view(torch.uint8)
    return pool


def rows_case(lens, starts, blocks, seed):
    g = gen(seed)
    pages = [-(-(s + n) // 16) for s, n in zip(starts, lens)]
    table = table_for(pages, blocks, g)
    cu = torch.tensor([sum(lens[:i]) for i in range(len(lens) + 1)], dtype=torch.int32)
    return table, cu, torch.tensor(starts, dtype=torch.int32)


def row_places(lens, starts, table):
    """(page id, offset) of each row."""
    out = []
    for r, (n, s) in enumerate(zip(lens, starts)):
        out += [(int(table[r, p // 16]), p % 16) for p in range(s, s + n)]
    return out


# (the last two: more than 31 requests end in 16 rows, and more than 33 * 33 requests)
LENS = [([1], [0]), ([1, 1, 1, 1, 1], [15, 16, 0, 31, 77]), ([16, 32], [0, 16]),
        ([0, 5, 0, 40, 17, 0], [3, 14, 0, 8, 1, 0]), ([100, 1, 16], [7, 1000, 9]),
        ([0] * 40 + [3] + [0] * 70 + [2, 1] + [0] * 5, [0] * 40 + [14] + [0] * 70 + [2, 0] + [7] * 5),
        ([0, 1] * 20 + [0] * 1200 + [18] + [0] * 3, [i % 48 for i in range(40)] + [0] * 1200 + [13] + [0] * 3)]


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("d,group", GROUPS)
@pytest.mark.parametrize("lens,starts", LENS)
def test_write_places_the_codes_and_leaves_the_rest(lens, starts, d, group, dtype):
    Hk = 3
    table, cu, start = rows_case(lens, starts, 90, 1)
    rows = sum(lens)
    g = gen(2)
    qkv = (torch.randn(rows + 3, 2 * Hk, d, generator=g) * torch.rand(rows + 3, 2 * Hk, 1, generator=g) * 4).to(dtype)
    before = random_pool(90, Hk, d, group, g, wild=True)
    pool, x = before.cuda(), qkv.cuda()
    kv = p4.PodKv4(Hk, Hk, d, group_size=group, dtype=dtype)
    # three rows behind the last request
    kv.write(kv.rows_args(cu.cuda(), start.cuda(), x[:, :Hk], x[:, Hk:], pool, table.cuda()))
    after = pool.cpu()
    n, s, m, border = ref.quantised(qkv[:rows].unflatten(1, (2, Hk)), group)   # rows, 2, Hk, d
    gn, gs, gm = ref.unpack(after, d, group)                                   # blocks, Hk, 2, PAGE, d
    at = row_places(lens, starts, table)
    page, off = torch.tensor([a[0] for a in at]), torch.tensor([a[1] for a in at])
    pick = lambda y: y[page, :, :, off].transpose(1, 2)                        # noqa: E731
    assert torch.equal(pick(gs), s) and torch.equal(pick(gm), m)
    far = (pick(gn) - n).abs()
    assert far[border > 1e-5].max() == 0 and far.max() <= 1
    # every other token as it was
    written = torch.zeros(90, 16, dtype=torch.bool)
    written[page, off] = True
    code, pair = ref.places(d, group)
    same = (before == after).all(1)
    keep = torch.zeros(90, before.shape[-1], dtype=torch.bool)
    for t in range(16):
        bytes_t = torch.cat([(code[:, t] // 2).flatten(), 16 * d + 4 * pair[:, t].flatten(), 16 * d + 4 * pair[:, t].flatten() + 1,
                             16 * d + 4 * pair[:, t].flatten() + 2, 16 * d + 4 * pair[:, t].flatten() + 3]).unique()
        keep[:, bytes_t] = ~written[:, t:t + 1]
    assert same[keep].all()


@pytest.mark.parametrize("dtype", [BF, HF])
def test_write_special_values(dtype):
    """Constant groups, subnormals, values beyond fp16, infinities and NaN."""
    d, group = 64, 32
    x = torch.randn(8, 1, d, generator=gen(3))
    x[0] = 0
    x[1] = 3.5
    x[2] *= 1e-7
    x[3] *= 20000
    x[4, 0, 5] = math.inf
    x[5, 0, 40] = math.nan
    x[6, 0, 0] = -math.inf
    x[7] = 1.0
    x[7, 0, 3] = 1.0 + 2.0 ** -7
    x = x.to(dtype)
    if dtype == BF:
        x[3, 0, 1] = 1e38
    kv = p4.PodKv4(1, 1, d, group_size=group, dtype=dtype)
    pool = kv.new_pool(1)
    cu, start = torch.tensor([0, 8], dtype=torch.int32).cuda(), torch.tensor([0], dtype=torch.int32).cuda()
    tab = torch.zeros(1, 1, dtype=torch.int32).cuda()
    xc = x.cuda()
    kv.write(kv.rows_args(cu, start, xc, xc, pool, tab))
    n, s, m, border = ref.quantised(x, group)
    gn, gs, gm = (y[0, 0, :, :8] for y in ref.unpack(pool.cpu(), d, group))
    for kvi in range(2):
        assert torch.equal(gs[kvi].nan_to_num(-1), s[:, 0].nan_to_num(-1))
        assert torch.equal(gm[kvi].nan_to_num(-1), m[:, 0].nan_to_num(-1))
        far = (gn[kvi] - n[:, 0]).abs()
        far[s[:, 0].isnan()] = 0
        assert far[border[:, 0] > 1e-5].max() == 0 and far.max() <= 1
    k, v = torch.zeros_like(xc), torch.zeros_like(xc)
    kv.read(kv.rows_args(cu, start, k, v, pool, tab))
    assert torch.equal(k.isnan().cpu(), s.isnan()) and torch.equal(k.nan_to_num(9), v.nan_to_num(9))


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("d,group", GROUPS)
@pytest.mark.parametrize("lens,starts", LENS)
def test_read_gives_the_rounded_values(lens, starts, d, group, dtype):
    Hk = 3
    table, cu, start = rows_case(lens, starts, 90, 4)
    rows = sum(lens)
    pool = random_pool(90, Hk, d, group, gen(5))
    kv = p4.PodKv4(Hk, Hk, d, group_size=group, dtype=dtype)
    out = torch.full((rows + 2, 2 * Hk, d), 7.0, dtype=dtype).cuda()
    kv.read(kv.rows_args(cu.cuda(), start.cuda(), out[:, :Hk], out[:, Hk:], pool.cuda(), table.cuda()))
    val = ref.values(pool, d, group)
    at = row_places(lens, starts, table)
    page, off = torch.tensor([a[0] for a in at]), torch.tensor([a[1] for a in at])
    want = val[page, :, :, off].transpose(1, 2).flatten(1, 2).float().to(dtype)
    got = out.cpu()
    assert torch.equal(got[:rows], want)
    assert (got[rows:] == 7).all()


def test_rows_without_a_place():
    """Positions outside the table and pages outside the pool: not written, read as NaN."""
    d, group, Hk = 128, 64, 2
    kv = p4.PodKv4(Hk, Hk, d, group_size=group)
    table = torch.tensor([[1, -1], [4, 2], [3, 0], [0, 3]], dtype=torch.int32).cuda()   # 4 is outside
    start = torch.tensor([0, 8, 30, -3], dtype=torch.int32).cuda()
    cu = torch.tensor([0, 20, 36, 40, 45], dtype=torch.int32).cuda()
    x = torch.randn(45, Hk, d, generator=gen(6)).to(BF).cuda()
    pool = kv.new_pool(4)
    kv.write(kv.rows_args(cu, start, x, x, pool, table))
    k, v = torch.zeros_like(x), torch.zeros_like(x)
    kv.read(kv.rows_args(cu, start, k, v, pool, table))
    bad = torch.zeros(45, dtype=torch.bool)
    bad[16:20] = True           # page -1
    bad[20:28] = True           # page 4
    bad[38:40] = True           # positions 32, 33 of a row of two pages
    bad[40:43] = True           # positions -3 .. -1
    for y in (k, v):
        assert torch.equal(y.isnan().all(-1).all(-1).cpu(), bad) and torch.equal(y.isnan().any(-1).any(-1).cpu(), bad)
    assert (k[~bad.cuda()].float() - x[~bad.cuda()].float()).abs().max() < 0.5


def check_decode(q, pool, table, lens, d, group, o, lse):
    want, wlse, parts = ref.attend(q.cpu(), pool.cpu(), table.cpu(), lens, d, group)
    bo, bl = ref.attend_bounds(want, wlse, parts, q.dtype)
    o, lse = o.cpu().double(), lse.cpu().double()
    empty = torch.tensor(lens) == 0
    assert (o[empty] == 0).all() and (lse[empty] == -math.inf).all()
    assert ((o - want).abs() <= bo)[~empty].all(), ((o - want).abs() / bo).max()
    assert ((lse - wlse).abs() <= bl)[~empty].all(), ((lse - wlse).abs() / bl)[~empty].max()


def run_decode(kv, q, pool, table, lens, stream=None):
    o = torch.full_like(q, math.nan)
    lse = torch.full(q.shape[:2], math.nan, device=q.device)
    kv.decode(kv.decode_args(lens, q, o, lse, pool, table), stream)
    return o, lse


def decode_case(lens, H, Hk, d, group, dtype, seed, blocks=None):
    g = gen(seed)
    pages = [-(-n // 16) for n in lens]
    blocks = blocks or sum(pages) + 3
    pool = random_pool(blocks, Hk, d, group, g)
    table = table_for(pages, blocks, g)
    # what lies behind a length is of any bits
    wild = random_pool(blocks, Hk, d, group, g, wild=True)
    code, pair = ref.places(d, group)
    used = torch.zeros(blocks, dtype=torch.bool)
    for r, n in enumerate(lens):
        used[table[r, :pages[r]].long()] = True
        if n % 16:
            page = int(table[r, n // 16])
            for t in range(n % 16, 16):
                at = torch.cat([(code[:, t] // 2).flatten()] + [16 * d + 4 * pair[:, t].flatten() + b for b in range(4)])
                pool[page][:, at] = wild[page][:, at]
    pool[~used] = wild[~used]
    q = (torch.randn(len(lens), H, d, generator=g) * 1.5).to(dtype)
    return q, pool, table


DECODE = [
    # lens, H, Hk
    ([1], 1, 1), ([16], 8, 1), ([17, 1, 0, 15], 4, 2), ([40, 77, 128, 200], 4, 2),
    ([0, 0], 2, 2), ([3000], 8, 1), ([513, 64, 2048, 31, 33, 1000], 6, 2), ([700] * 9, 15, 3), ([5000, 1, 4096], 14, 2),
    (list(range(0, 130)), 8, 8),
]


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("d,group", GROUPS)
@pytest.mark.parametrize("lens,H,Hk", DECODE)
def test_decode_matches_the_formula(lens, H, Hk, d, group, dtype):
    q, pool, table = decode_case(lens, H, Hk, d, group, dtype, 7)
    kv = p4.PodKv4(H, Hk, d, group_size=group, dtype=dtype)
    qc, pc, tc = q.cuda(), pool.cuda(), table.cuda()
    lc = torch.tensor(lens, dtype=torch.int32).cuda()
    o, lse = run_decode(kv, qc, pc, tc, lc)
    check_decode(q, pool, table, lens, d, group, o, lse)
    again = run_decode(kv, qc, pc, tc, lc)   # the order of the parts does not change a bit
    assert torch.equal(o, again[0]) and torch.equal(lse, again[1])


@pytest.mark.parametrize("R,H,Hk", [(4096, 2, 1), (1500, 3, 3)])
def test_decode_of_many_short_requests(R, H, Hk):
    """More requests than threads, empty ones among them; the largest number a context admits."""
    lens = [(7 * i) % 5 * (i % 3) for i in range(R)]
    lens[R // 2] = 300
    q, pool, table = decode_case(lens, H, Hk, 64, 32, BF, 19)
    kv = p4.PodKv4(H, Hk, 64, group_size=32, max_decode_reqs=R)
    o, lse = run_decode(kv, q.cuda(), pool.cuda(), table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda())
    check_decode(q, pool, table, lens, 64, 32, o, lse)


def test_shared_pages_may_be_read_by_many():
    """A common prefix: several requests list the same pages, also twice in one row."""
    d, group, H, Hk = 128, 64, 4, 2
    q, pool, table = decode_case([64, 64, 64], H, Hk, d, group, BF, 20)
    table[1] = table[0]
    table[2, 1:] = table[2, :1]
    lens = [64, 50, 64]
    kv = p4.PodKv4(H, Hk, d, group_size=group)
    o, lse = run_decode(kv, q.cuda(), pool.cuda(), table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda())
    check_decode(q, pool, table, lens, d, group, o, lse)
    cu, start = torch.tensor([0, 64, 114, 178], dtype=torch.int32).cuda(), torch.zeros(3, dtype=torch.int32).cuda()
    k, v = (torch.zeros(178, Hk, d, dtype=BF, device="cuda") for _ in range(2))
    kv.read(kv.rows_args(cu, start, k, v, pool.cuda(), table.cuda()))
    assert torch.equal(k[64:114], k[:50]) and torch.equal(v[114:130], v[130:146])


def test_two_graphs_on_one_context_replayed_in_turn():
    """They share the workspace, one after the other on one stream."""
    cases = [decode_case(lens, 8, 1, 128, 128, HF, 21 + i) for i, lens in enumerate(([5000, 40], [900] * 7))]
    kv, graphs, outs = p4.PodKv4(8, 1, 128, group_size=128, dtype=HF), [], []
    held = []
    for (q, pool, table), lens in zip(cases, ([5000, 40], [900] * 7)):
        args = [q.cuda(), pool.cuda(), table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda()]
        run_decode(kv, *args)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = run_decode(kv, *args)
        held.append(args)
        graphs.append(g)
        outs.append(out)
    for i in (0, 1, 1, 0, 1):
        outs[i][0].fill_(7)
        graphs[i].replay()
    for out, args, lens, (q, pool, table) in zip(outs, held, ([5000, 40], [900] * 7), cases):
        eager = run_decode(kv, *args)
        assert torch.equal(out[0], eager[0]) and torch.equal(out[1], eager[1])
        check_decode(q, pool, table, lens, 128, 128, *eager)


def test_decode_extreme_queries():
    """A query of zeros, ones of very large and very small values, and a NaN: each row by itself."""
    d, group, H, Hk = 128, 64, 4, 1
    lens = [100] * 6
    q, pool, table = decode_case(lens, H, Hk, d, group, BF, 8)
    q[0] = 0
    q[1] *= 1e6
    q[2] *= 1e-20
    q[3, :, 1:] = 0
    q[4, :, :7] *= 1e4
    q[5, 2, 9] = math.nan
    kv = p4.PodKv4(H, Hk, d, group_size=group)
    o, lse = run_decode(kv, q.cuda(), pool.cuda(), table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda())
    assert o[5, 2].isnan().all() and lse[5, 2].isnan()
    assert not o[5, [0, 1, 3]].isnan().any() and not o[:5].isnan().any()
    check_decode(q[:5], pool, table[:5], lens[:5], d, group, o[:5], lse[:5])


def test_decode_keys_of_nan_and_bad_pages_touch_their_request_only():
    d, group, H, Hk = 128, 32, 8, 2
    lens = [300, 300, 5000, 40, 300]
    q, pool, table = decode_case(lens, H, Hk, d, group, BF, 9)
    table[1, 7] = pool.shape[0]
    table[2, 200] = -5
    pool[int(table[4, 3]), 1, 16 * d:16 * d + 4] = 255   # s, m of one token's first group of K, head 1
    lc = torch.tensor(lens, dtype=torch.int32).cuda()
    kv = p4.PodKv4(H, Hk, d, group_size=group)
    o, lse = run_decode(kv, q.cuda(), pool.cuda(), table.cuda(), lc)
    assert o[[1, 2]].isnan().all() and lse[[1, 2]].isnan().all()
    assert o[4, 4:].isnan().all() and lse[4, 4:].isnan().all() and not o[4, :4].isnan().any()
    ok = [0, 3]
    check_decode(q[ok], pool, table[ok], [lens[i] for i in ok], d, group, o[ok], lse[ok])


def test_decode_lengths_beyond_the_table_are_cut():
    q, pool, table = decode_case([64, 64], 4, 2, 64, 64, HF, 10)
    kv = p4.PodKv4(4, 2, 64, group_size=64, dtype=HF)
    lens = torch.tensor([2 ** 31 - 1, -7], dtype=torch.int32).cuda()
    o, lse = run_decode(kv, q.cuda(), pool.cuda(), table.cuda(), lens)
    check_decode(q, pool, table, [64, 0], 64, 64, o, lse)


def test_decode_far_pages():
    """Records whose byte offsets pass 32 bits."""
    d, group, H, Hk = 128, 64, 4, 4
    lens = [200, 50]
    q, small, table = decode_case(lens, H, Hk, d, group, BF, 11)
    blocks = (1 << 33) // (Hk * small.shape[-1])
    kv = p4.PodKv4(H, Hk, d, group_size=group)
    pool = torch.empty(blocks, Hk, small.shape[-1], dtype=torch.uint8, device="cuda")
    far = blocks - small.shape[0]
    pool[far:] = small.cuda()
    tc = (table + far * (table >= 0)).int().cuda()
    lc = torch.tensor(lens, dtype=torch.int32).cuda()
    o, lse = run_decode(kv, q.cuda(), pool, tc, lc)
    check_decode(q, small, table, lens, d, group, o, lse)
    cu = torch.tensor([0, 200, 250], dtype=torch.int32).cuda()
    start = torch.zeros(2, dtype=torch.int32).cuda()
    k, v = (torch.zeros(250, Hk, d, dtype=BF, device="cuda") for _ in range(2))
    kv.read(kv.rows_args(cu, start, k, v, pool, tc))
    k2, v2 = torch.zeros_like(k), torch.zeros_like(v)
    kv.read(kv.rows_args(cu, start, k2, v2, small.cuda(), table.cuda()))
    assert torch.equal(k, k2) and torch.equal(v, v2)
    kv.write(kv.rows_args(cu, start, k, v, pool, tc))
    kv.read(kv.rows_args(cu, start, k2, v2, pool, tc))
    # a value written again moves by half a step of its group at most (the rows are rounded), a step here
    assert (k2.float() - k.float()).abs().max() < 0.4


ROPE = [(1, 32, 8, 128, 128), (7, 4, 2, 64, 64), (33, 3, 1, 128, 64), (5, 2, 3, 64, 48), (65, 8, 8, 128, 16), (3, 5, 0, 128, 112), (300, 64, 8, 128, 128)]


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("norm", ["both", "none", "q"])
@pytest.mark.parametrize("rows,H,Hk,d,rot", ROPE)
def test_norm_rope(rows, H, Hk, d, rot, norm, interleaved, dtype):
    g = gen(12)
    qkv = (torch.randn(rows, H + 2 * Hk + 1, d, generator=g) * 3).to(dtype)
    qkv[0, 0] = 0
    w = [(1 + 0.3 * torch.randn(d, generator=g)).to(dtype) if norm == "both" or (norm == "q" and i == 0) else None for i in range(2)]
    table = p4.rope_table(9000, rot, 10000.0, device="cpu")
    pos = torch.randint(0, 9000, (rows,), generator=g, dtype=torch.int32)
    pos[-1] = 8999
    x = qkv.cuda()
    q, k = x[:, :H], x[:, H:H + Hk] if Hk else None
    wc = [y.cuda() if y is not None else None for y in w]
    qo = torch.empty(rows, H, d, dtype=dtype, device="cuda")
    ko = torch.empty(Hk, rows, d, dtype=dtype, device="cuda").transpose(0, 1) if Hk else None
    kw = dict(q_weight=wc[0], k_weight=wc[1] if Hk else None, eps=1e-5, interleaved=interleaved)
    p4.qk_norm_rope(p4.norm_rope_args(q, k, pos.cuda(), table.cuda(), q_out=qo, k_out=ko, **kw))
    for got, src, wt in ((qo, qkv[:, :H], w[0]), (ko, qkv[:, H:H + Hk], w[1])):
        if got is None:
            continue
        want, size = ref.norm_rope(src, wt, table, pos, 1e-5, interleaved)
        # half a step of the output; 13 fp32 roundings of 2^-24 on the way (squares and their sum
        # count half); fp16 below 2^-14 is spaced by 2^-24
        bound = ref.EPS[dtype] / 2 * want.abs() + 2.0 ** -20 * size + 2.0 ** -25
        assert ((got.cpu().double() - want).abs() <= bound).all()
    # in place
    p4.qk_norm_rope(p4.norm_rope_args(q, k, pos.cuda(), table.cuda(), **kw))
    assert torch.equal(q, qo) and (k is None or torch.equal(k, ko))
    assert torch.equal(x[:, H + Hk:].cpu(), qkv[:, H + Hk:])


def test_norm_rope_padding_and_far_positions():
    x = torch.randn(4, 3, 64, generator=gen(13)).to(BF).cuda()
    before = x.clone()
    pos = torch.tensor([3, -1, 100, 99], dtype=torch.int32).cuda()
    p4.qk_norm_rope(p4.norm_rope_args(x[:, :2], x[:, 2:], pos, p4.rope_table(100, 32)))
    assert torch.equal(x[1], before[1])
    assert x[2].isnan().all() and not x[[0, 3]].isnan().any()


def step(kv, x, pool, table, lens, cu, tab, w, bufs):
    """One decode step of a layer: norm and rotate the new token, write it, attend."""
    H, Hk = kv.cfg.num_qo_heads, kv.cfg.num_kv_heads
    q, k, o, lse = bufs
    p4.qk_norm_rope(p4.norm_rope_args(x[:, :H], x[:, H:H + Hk], lens, tab, q_out=q, k_out=k, q_weight=w, k_weight=w))
    kv.write(kv.rows_args(cu, lens, k, x[:, H + Hk:], pool, table))
    kv.decode(kv.decode_args(lens + 1, q, o, lse, pool, table))


def test_decode_steps_captured_and_replayed():
    """A chain of all operators, captured once; replays with other tokens and lengths give what eager calls give."""
    H, Hk, d, R = 8, 2, 128, 5
    kv, g = p4.PodKv4(H, Hk, d, group_size=64), gen(14)
    tab = p4.rope_table(512, d)
    w = (1 + 0.1 * torch.randn(d, generator=g)).to(BF).cuda()
    table = torch.randperm(R * 8, generator=g).reshape(R, 8).to(torch.int32).cuda()
    cu = torch.arange(R + 1, dtype=torch.int32).cuda()
    pools = [kv.new_pool(R * 8) for _ in range(2)]
    lens = torch.tensor([0, 3, 15, 16, 100], dtype=torch.int32).cuda()
    bufs = [tuple(torch.zeros(R, n, d, dtype=BF, device="cuda") for n in (H, Hk, H)) + (torch.zeros(R, H, device="cuda"),) for _ in range(2)]
    x = torch.zeros(R, H + 2 * Hk, d, dtype=BF, device="cuda")
    step(kv, x, pools[0].clone(), table, lens, cu, tab, w, bufs[0])   # warm up
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step(kv, x, pools[0], table, lens, cu, tab, w, bufs[0])
        lens += 1
    other = torch.tensor([0, 3, 15, 16, 100], dtype=torch.int32).cuda()
    history = []
    for i in range(6):
        x.copy_(torch.randn(x.shape, generator=g).to(BF))
        graph.replay()
        step(kv, x, pools[1], table, other, cu, tab, w, bufs[1])
        other += 1
        torch.cuda.synchronize()
        assert torch.equal(lens, other) and torch.equal(pools[0], pools[1])
        assert all(torch.equal(a, b) for a, b in zip(*bufs))
        history.append(bufs[1][2].clone())
    assert not torch.equal(history[0], history[1])
    q = bufs[1][0]
    check_decode(q.cpu(), pools[1].cpu(), table.cpu(), other.tolist(), d, 64, bufs[1][2], bufs[1][3])


def test_other_stream_and_two_contexts():
    """Calls on a side stream, beside calls of another context on the main one."""
    lens = [900, 100, 33]
    q, pool, table = decode_case(lens, 8, 2, 128, 64, BF, 15)
    kvs = [p4.PodKv4(8, 2, 128) for _ in range(2)]
    qc, pc, tc, lc = q.cuda(), pool.cuda(), table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    outs = []
    for _ in range(20):
        outs.append(run_decode(kvs[0], qc, pc, tc, lc))
        with torch.cuda.stream(side):
            outs.append(run_decode(kvs[1], qc, pc, tc, lc))
    torch.cuda.synchronize()
    for o, lse in outs[1:]:
        assert torch.equal(o, outs[0][0]) and torch.equal(lse, outs[0][1])
    check_decode(q, pool, table, lens, 128, 64, *outs[0])


def test_chunked_prefill_over_the_cache():
    """Norm and rotate a chunk, write it, read the whole context back and run the bf16 prefill on
    it beside the 4-bit decodes: attention over the values that the cache holds."""
    H, Hk, d, group, prior, chunk = 8, 2, 128, 32, 150, 70
    g = gen(16)
    kv = p4.PodKv4(H, Hk, d, group_size=group)
    pod = pa.PodAttention(H, Hk, d, max_prefill_reqs=1, max_prefill_tokens=chunk, max_decode_reqs=1, max_kv_tokens=512)
    pool = random_pool(40, Hk, d, group, g).cuda()
    table = torch.randperm(40, generator=g)[:16].reshape(1, 16).to(torch.int32).cuda()
    tab = p4.rope_table(512, d)
    x = torch.randn(chunk, H + 2 * Hk, d, generator=g).to(BF).cuda()
    q = torch.empty(chunk, H, d, dtype=BF, device="cuda")
    k = torch.empty(chunk, Hk, d, dtype=BF, device="cuda")
    pos = torch.arange(prior, prior + chunk, dtype=torch.int32, device="cuda")
    p4.qk_norm_rope(p4.norm_rope_args(x[:, :H], x[:, H:H + Hk], pos, tab, q_out=q, k_out=k))
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32).cuda()  # noqa: E731
    kv.write(kv.rows_args(i32(0, chunk), i32(prior), k, x[:, H + Hk:], pool, table))
    n = prior + chunk
    kc, vc = (torch.empty(n, Hk, d, dtype=BF, device="cuda") for _ in range(2))
    kv.read(kv.rows_args(i32(0, n), i32(0), kc, vc, pool, table))
    o = torch.empty_like(q)
    lse = torch.empty(chunk, H, device="cuda")
    pod.prefill_only(pod.prefill_args([chunk], [prior], q, o, lse, k=[kc], v=[vc]))
    assert pod.status() == pa.POD_OK and pod.close() == pa.POD_OK
    # the last token's row is what a decode over the cache gives
    do, dl = run_decode(kv, q[-1:].contiguous(), pool, table, i32(n))
    check_decode(q[-1:].cpu(), pool.cpu(), table.cpu(), [n], d, group, do, dl)
    val = ref.values(pool.cpu()[table.cpu()[0].long()], d, group).permute(2, 1, 0, 3, 4).flatten(2, 3)
    for t in (0, 5, chunk - 1):
        for h in (0, 7):
            kk, vv = val[0, h // 4, :prior + t + 1], val[1, h // 4, :prior + t + 1]
            sc = kk @ q[t, h].cpu().double() / math.sqrt(d)
            want = torch.softmax(sc, 0) @ vv
            # the prefill's tolerances, and the rounding of the rows that were read back (2^-8 of
            # a key moves a score by at most 2^-8 sum |q_i k_i| / sqrt(d))
            size = (kk.abs() @ q[t, h].cpu().double().abs()).max() / math.sqrt(d) * 2.0 ** -8
            assert (o[t, h].cpu().double() - want).abs().max() <= 1e-2 + (2 * size + 2.0 ** -8) * vv.abs().max()
            assert abs(lse[t, h].item() - torch.logsumexp(sc, 0).item()) <= 1e-3 + size


@pytest.mark.parametrize("d,group", [(128, 64), (64, 32)])
def test_hybrid_batch_over_the_cache(d, group):
    """PodKv4.hybrid, two steps in a row: chunks and decodes of one batch, each row against the
    formula over the values that the cache holds after the write."""
    H, Hk, g = 8, 2, gen(17)
    kv = p4.PodKv4(H, Hk, d, group_size=group)
    pod = pa.PodAttention(H, Hk, d, max_prefill_reqs=2, max_prefill_tokens=128, max_decode_reqs=1, max_kv_tokens=512)
    pool, tab = kv.new_pool(80), p4.rope_table(512, d)
    w = (1 + 0.1 * torch.randn(d, generator=g)).to(BF).cuda()
    table = torch.randperm(80, generator=g).reshape(5, 16).to(torch.int32).cuda()
    i32 = lambda v: torch.tensor(v, dtype=torch.int32).cuda()  # noqa: E731
    chunks, done = [50, 13], [0, 0]
    seen = [0, 3, 40]
    # the decodes' contexts so far
    pre = torch.randn(43, 2 * Hk, d, generator=g).to(BF).cuda()
    kv.write(kv.rows_args(i32([0, 0, 3, 43]), i32([0, 0, 0]), pre[:, :Hk], pre[:, Hk:], pool, table[2:]))
    for _ in range(2):
        rows = sum(chunks) + 3
        qkv = torch.randn(rows, H + 2 * Hk, d, generator=g).to(BF).cuda()
        before = qkv.clone()
        pos = i32([p for n, s in zip(chunks, done) for p in range(s, s + n)] + seen)
        cu = i32([0, chunks[0], sum(chunks)] + [sum(chunks) + 1 + i for i in range(3)])
        ctx = [n + 1 for n in seen]
        o, lse = kv.hybrid(pod, qkv, pos, tab, chunk_lens=chunks, prior_lens=done, cu_rows=cu, start=i32(done + seen), ctx_lens=i32(ctx),
                           pool=pool, block_table=table, q_weight=w, k_weight=w)
        assert pod.status() == pa.POD_OK
        q, _ = ref.norm_rope(before[:, :H].cpu(), w.cpu(), tab.cpu(), pos.cpu(), 1e-6, False)
        q = q.to(BF)
        check_decode(q[sum(chunks):], pool, table[2:], ctx, d, group, o[sum(chunks):], lse[sum(chunks):])
        at = 0
        for r, (n, s) in enumerate(zip(chunks, done)):
            val = ref.values(pool.cpu()[table.cpu()[r].long()], d, group).permute(2, 1, 0, 3, 4).flatten(2, 3)
            for t in (0, n // 2, n - 1):
                for h in (0, H - 1):
                    kk, vv = val[0, h * Hk // H, :s + t + 1], val[1, h * Hk // H, :s + t + 1]
                    x = q[at + t, h].double()
                    sc = kk @ x / math.sqrt(d)
                    size = (kk.abs() @ x.abs()).max() / math.sqrt(d) * 2.0 ** -8   # as in the test above
                    assert (o[at + t, h].cpu().double() - torch.softmax(sc, 0) @ vv).abs().max() <= 1e-2 + (2 * size + 2.0 ** -8) * vv.abs().max()
                    assert abs(lse[at + t, h].item() - torch.logsumexp(sc, 0).item()) <= 1e-3 + size
            at += n
        done = [s + n for s, n in zip(done, chunks)]
        seen = ctx
    assert pod.close() == pa.POD_OK
    with pytest.raises(ValueError):
        kv.hybrid(pod, qkv[:-1], pos, tab, chunk_lens=chunks, prior_lens=done, cu_rows=cu, start=i32(done + seen), ctx_lens=i32(ctx), pool=pool, block_table=table)


def test_hybrid_of_decodes_alone_and_of_a_chunk_alone():
    H, Hk, d = 4, 2, 64
    kv = p4.PodKv4(H, Hk, d)
    pod = pa.PodAttention(H, Hk, d, max_prefill_reqs=1, max_prefill_tokens=32, max_decode_reqs=1, max_kv_tokens=64)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32).cuda()  # noqa: E731
    tab, table = p4.rope_table(64, d), torch.arange(8, dtype=torch.int32).reshape(2, 4).cuda()
    x = torch.randn(20, H + 2 * Hk, d, generator=gen(18)).to(BF).cuda()
    pools = [kv.new_pool(8) for _ in range(2)]
    # a prompt of 20 tokens as one chunk, and as one chunk of 19 and a decode
    o, lse = kv.hybrid(pod, x.clone(), i32(list(range(20))), tab, chunk_lens=[20], prior_lens=[0], cu_rows=i32([0, 20]), start=i32([0]),
                       ctx_lens=i32([]), pool=pools[0], block_table=table[:1])
    kv.hybrid(pod, x[:19].clone(), i32(list(range(19))), tab, chunk_lens=[19], prior_lens=[0], cu_rows=i32([0, 19]), start=i32([0]),
              ctx_lens=i32([]), pool=pools[1], block_table=table[:1])
    o2, lse2 = kv.hybrid(pod, x[19:].clone(), i32([19]), tab, chunk_lens=[], prior_lens=[], cu_rows=i32([0, 1]), start=i32([19]),
                         ctx_lens=i32([20]), pool=pools[1], block_table=table[:1])
    assert pod.status() == pa.POD_OK and torch.equal(pools[0], pools[1])
    # the prefill's tolerance, on outputs of size 1
    assert (o[19:].float() - o2.float()).abs().max() <= 3e-2 and (lse[19:] - lse2).abs().max() <= 3e-2
    assert pod.close() == pa.POD_OK


def test_calls_with_nothing_to_do():
    kv = p4.PodKv4(4, 2, 64)
    pool = kv.new_pool(1)
    e = lambda *s, t=BF: torch.empty(*s, dtype=t, device="cuda")  # noqa: E731
    i32 = torch.int32
    kv.write(kv.rows_args(torch.zeros(1, dtype=i32).cuda(), e(0, t=i32), e(0, 2, 64), e(0, 2, 64), pool, e(0, 3, t=i32)))
    kv.read(kv.rows_args(torch.zeros(3, dtype=i32).cuda(), torch.zeros(2, dtype=i32).cuda(), e(0, 2, 64), e(0, 2, 64), pool, e(2, 3, t=i32)))
    kv.decode(kv.decode_args(e(0, t=i32), e(0, 4, 64), e(0, 4, 64), e(0, 4, t=torch.float32), pool, e(0, 3, t=i32)))
    p4.qk_norm_rope(p4.norm_rope_args(e(0, 4, 64), e(0, 2, 64), e(0, t=i32), p4.rope_table(4, 64)))
    # rows of no request
    x = torch.full((3, 2, 64), 5.0, dtype=BF, device="cuda")
    kv.read(kv.rows_args(torch.zeros(2, dtype=i32).cuda(), torch.zeros(1, dtype=i32).cuda(), x, x.clone(), pool, torch.zeros(1, 1, dtype=i32).cuda()))
    assert (x == 5).all()
    o, lse = run_decode(kv, e(2, 4, 64).zero_(), pool, e(2, 0, t=i32), torch.tensor([5, 0], dtype=i32).cuda())
    assert (o == 0).all() and (lse == -math.inf).all()


def test_context_errors():
    for kw, code in ((dict(device=99), pa.POD_EINVAL), (dict(group_size=48), pa.POD_EUNSUPPORTED)):
        with pytest.raises(pa.PodError) as e:
            p4.PodKv4(4, 2, 64, **kw)
        assert e.value.code == code
    kv = p4.PodKv4(4, 2, 64, max_decode_reqs=2)
    pool = kv.new_pool(1)
    q = torch.zeros(3, 4, 64, dtype=BF, device="cuda")
    lens, tab = torch.zeros(3, dtype=torch.int32).cuda(), torch.zeros(3, 1, dtype=torch.int32).cuda()
    with pytest.raises(pa.PodError) as e:
        run_decode(kv, q, pool, tab, lens)
    assert e.value.code == pa.POD_ECAPACITY
    with pytest.raises(ValueError):
        run_decode(kv, q.half(), pool, tab, lens)
    with pytest.raises(ValueError):
        run_decode(kv, q, pool, tab.long(), lens)
    with pytest.raises(ValueError):
        run_decode(kv, q, pool[:, :, :-1], tab, lens)
    with pytest.raises(ValueError):
        kv.rows_args(lens, lens, q, q, pool, tab)
    assert kv.close() == pa.POD_OK
    with pytest.raises(ValueError):
        run_decode(kv, q[:2], pool, tab[:2], lens[:2])


@pytest.mark.parametrize("dtype,factor", [(BF, 1e8), (BF, 1e12), (BF, 1e30), (BF, 2.0 ** 117), (HF, 8e3)])
def test_decode_scores_of_any_size(dtype, factor):
    """Scores far beyond 2^24 leave one token per row. Every tile of 64 tokens has values of another
    scale, and the long context lies in several CTAs."""
    d, group, H, Hk = 128, 64, 4, 2
    lens = [300, 1500, 40, 1]
    q, pool, table = decode_case(lens, H, Hk, d, group, dtype, 30)
    q = (q.double() * factor).to(dtype)
    par = pool[..., 16 * d:].contiguous().view(torch.float16).unflatten(-1, (2, -1))
    if dtype == HF:
        par[:, :, 0] *= 100
    for r, n in enumerate(lens):
        for blk in range(-(-n // 16)):
            page = int(table[r, blk])
            par[page, :, 1] = (par[page, :, 1].float() * 2.0 ** (3 * (blk // 4 % 5) - 8)).half().nan_to_num(0, 0, 0)
    pool[..., 16 * d:] = par.flatten(-2).contiguous().view(torch.uint8)
    # no score is near the largest: what the kernel's scores may be off is 2^-17 sum |q_i k_i| / sqrt(d)
    for r, n in enumerate(lens):
        if n == 1:
            continue
        k = ref.values(pool[table[r, :-(-n // 16)].long()], d, group).permute(2, 1, 0, 3, 4).flatten(2, 3)[0, :, :n]
        for h in range(H):
            kk, x = k[h // (H // Hk)], q[r, h].double()
            two = (kk @ x / math.sqrt(d)).topk(2).values
            assert two[0] - two[1] > max(1000, 3 * 2.0 ** -17 * (kk.abs() @ x.abs()).max() / math.sqrt(d))
    kv = p4.PodKv4(H, Hk, d, group_size=group, dtype=dtype)
    o, lse = run_decode(kv, q.cuda(), pool.cuda(), table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda())
    check_decode(q, pool, table, lens, d, group, o, lse)


@pytest.mark.parametrize("lens,H,Hk,d,group", [
    ([5000, 40, 700, 3000, 0, 300], 8, 2, 128, 64), ([5000, 40, 700, 3000, 0, 300], 8, 1, 64, 32),
    ([100, 0, 33, 900, 1024] * 40, 4, 4, 128, 32), ([17], 2, 2, 128, 128),
])
def test_waits_that_run_out(lens, H, Hk, d, group):
    """In the first call every warp gives up at one of its tiles: the rows of what it has from there
    on are NaN, the others as ever, and the status says so. The next call is right."""
    q, pool, table = decode_case(lens, H, Hk, d, group, BF, 31)
    args = q.cuda(), pool.cuda(), table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda()
    want, wlse = run_decode(p4.PodKv4(H, Hk, d, group_size=group), *args)
    kv = p4.PodKv4(H, Hk, d, group_size=group, flags=pa.FLAG_TEST_FORCE_TIMEOUT)
    o, lse = run_decode(kv, *args)
    assert kv.status() == pa.POD_ETIMEOUT and kv.status() == pa.POD_OK   # cleared by the read
    lost = lse.isnan().unflatten(1, (Hk, -1)).all(-1).repeat_interleave(H // Hk, 1)
    assert lost.any() and torch.equal(lse.isnan(), lost) and torch.equal(o.isnan(), lost.unsqueeze(-1).expand_as(o))
    assert not lost[torch.tensor(lens) == 0].any()
    assert torch.equal(o[~lost], want[~lost]) and torch.equal(lse[~lost], wlse[~lost])
    again = run_decode(kv, *args)
    assert torch.equal(again[0], want) and torch.equal(again[1], wlse)
    check_decode(q, pool, table, lens, d, group, want, wlse)
    assert kv.status() == pa.POD_OK
    run_decode(kv, *args)
    assert kv.close() == pa.POD_OK
    kv = p4.PodKv4(H, Hk, d, group_size=group, flags=pa.FLAG_TEST_FORCE_TIMEOUT)
    run_decode(kv, *args)
    assert kv.close() == pa.POD_ETIMEOUT


def test_refused_hybrid_calls_change_nothing():
    """Whatever the reason, rows and cache are as they were, and the same call put right gives what a first call gives."""
    H, Hk, d, g = 8, 2, 128, gen(32)
    kv = p4.PodKv4(H, Hk, d, max_decode_reqs=1)
    pods = [pa.PodAttention(H, Hk, d, max_prefill_reqs=2, max_prefill_tokens=tok, max_decode_reqs=1, max_kv_tokens=most)
            for tok, most in ((64, 256), (49, 256), (64, 99))]
    i32 = lambda v: torch.tensor(v, dtype=torch.int32).cuda()  # noqa: E731
    pool, tab = kv.new_pool(40), p4.rope_table(512, d)
    x = torch.randn(51, H + 2 * Hk, d, generator=g).to(BF).cuda()
    table = torch.arange(32, dtype=torch.int32).reshape(2, 16).cuda()
    a = dict(qkv=x.clone(), positions=i32(list(range(50, 100)) + [20]), cos_sin=tab, chunk_lens=[50], prior_lens=[50], cu_rows=i32([0, 50, 51]),
             start=i32([50, 20]), ctx_lens=i32([21]), pool=pool, block_table=table)
    first = kv.hybrid(pods[0], **{**a, "qkv": x.clone(), "pool": kv.new_pool(40)})
    odd = torch.zeros(pool.numel() + 8, dtype=torch.uint8, device="cuda")[8:].view(pool.shape)
    bad = [(pods[1], {}), (pods[2], {}), (pods[0], dict(cu_rows=i32([0, 51]))), (pods[0], dict(pool=odd)), (pods[0], dict(pool=pool[:, :, :-16])),
           (pods[0], dict(block_table=table[:1])), (pods[0], dict(cos_sin=tab[:, :24].contiguous())), (pods[0], dict(eps=-1.0)),
           (pods[0], dict(ctx_lens=i32([21]).long())), (pods[0], dict(q_weight=torch.ones(d, device="cuda"))),
           (pods[0], dict(chunk_lens=[49], ctx_lens=i32([20, 21]), start=i32([50, 20, 21]), cu_rows=i32([0, 49, 50, 51]),
                          block_table=table[[0, 1, 1]]))]
    for pod, kw in bad:
        with pytest.raises((ValueError, pa.PodError)):
            kv.hybrid(pod, **{**a, **kw})
        assert torch.equal(a["qkv"], x) and not pool.any() and not odd.any(), kw.keys()
    o, lse = kv.hybrid(pods[0], **a)
    assert torch.equal(o, first[0]) and torch.equal(lse, first[1])
    assert all(pod.status() == pa.POD_OK and pod.close() == pa.POD_OK for pod in pods)


def hybrid_case(kv, g, chunks=(50, 13), prior=(20, 0), seen=(0, 3, 40)):
    """Arguments of a hybrid call over a cache that holds something for every request (tables of 16 pages, 512 positions)."""
    H, Hk, d = kv.cfg.num_qo_heads, kv.cfg.num_kv_heads, kv.cfg.head_dim
    i32 = lambda v: torch.tensor(v, dtype=torch.int32).cuda()  # noqa: E731
    n, rows = len(chunks) + len(seen), sum(chunks) + len(seen)
    at = [sum(chunks[:i]) for i in range(len(chunks) + 1)]
    return dict(qkv=torch.randn(rows, H + 2 * Hk, d, generator=g).to(kv.dtype).cuda(), cos_sin=p4.rope_table(512, d),
                positions=i32([p for c, s in zip(chunks, prior) for p in range(s, s + c)] + list(seen)), chunk_lens=list(chunks), prior_lens=list(prior),
                cu_rows=i32(at + [at[-1] + 1 + i for i in range(len(seen))]), start=i32(list(prior) + list(seen)), ctx_lens=i32([s + 1 for s in seen]),
                pool=random_pool(16 * n, Hk, d, kv.cfg.group_size, g).cuda(),
                block_table=torch.randperm(16 * n, generator=g).reshape(n, 16).to(torch.int32).cuda())


def test_hybrid_on_a_stream_of_its_own_does_not_wait():
    """The call returns while the stream is still busy with what came before, and gives what it gives elsewhere."""
    kv = p4.PodKv4(8, 2, 128)
    pods = [pa.PodAttention(8, 2, 128, max_prefill_reqs=2, max_prefill_tokens=64, max_decode_reqs=1, max_kv_tokens=256) for _ in range(2)]
    a = hybrid_case(kv, gen(33))
    copies = [{**a, "qkv": a["qkv"].clone(), "pool": a["pool"].clone()} for _ in range(2)]
    want = kv.hybrid(pods[0], **copies[0])
    assert pods[0].status() == pa.POD_OK
    side = torch.cuda.Stream()
    kv.hybrid(pods[1], **{**a, "qkv": a["qkv"].clone(), "pool": a["pool"].clone()}, stream=side)   # (buffers of that stream exist)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(400_000_000)                                  # about 0.2 s
        busy = torch.cuda.Event()
        busy.record()
    got = kv.hybrid(pods[1], **copies[1], stream=side)
    assert not busy.query()
    side.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(got, want))
    assert torch.equal(copies[0]["qkv"], copies[1]["qkv"]) and torch.equal(copies[0]["pool"], copies[1]["pool"])
    assert not torch.equal(copies[0]["qkv"][:, 8:10], a["qkv"][:, 8:10])                  # k, rotated in place
    assert torch.equal(copies[0]["qkv"][:, :8], a["qkv"][:, :8]) and torch.equal(copies[0]["qkv"][:, 10:], a["qkv"][:, 10:])
    assert all(pod.status() == pa.POD_OK and pod.close() == pa.POD_OK for pod in pods)


def test_hybrid_in_a_graph():
    """Decodes are captured and replayed; prefills are refused before anything is enqueued."""
    kv = p4.PodKv4(8, 2, 128, dtype=HF)
    a = hybrid_case(kv, gen(34), chunks=(), prior=())
    pool = a["pool"].clone()
    want = kv.hybrid(None, **{**a, "qkv": a["qkv"].clone(), "pool": pool})
    qkv = torch.empty_like(a["qkv"])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = kv.hybrid(None, **{**a, "qkv": qkv})
    for _ in range(2):
        qkv.copy_(a["qkv"])
        g.replay()
        assert all(torch.equal(x, y) for x, y in zip(out, want)) and torch.equal(a["pool"], pool)
    kv = p4.PodKv4(8, 2, 128)
    pod = pa.PodAttention(8, 2, 128, max_prefill_reqs=2, max_prefill_tokens=64, max_decode_reqs=1, max_kv_tokens=256)
    a = hybrid_case(kv, gen(35))
    before = a["qkv"].clone(), a["pool"].clone()
    g2 = torch.cuda.CUDAGraph()
    with pytest.raises(pa.PodError) as e:
        with torch.cuda.graph(g2):
            kv.hybrid(pod, **a)
    assert e.value.code == pa.POD_EUNSUPPORTED
    assert torch.equal(a["qkv"], before[0]) and torch.equal(a["pool"], before[1])
    kv.hybrid(pod, **a)
    assert pod.status() == pa.POD_OK and pod.close() == pa.POD_OK


def test_finite_fp16_rows_stay_finite():
    """Groups that end near 65504, where n s + m would pass fp16: written, read back and attended over."""
    d, group = 64, 32
    x = torch.rand(16, 1, d, generator=gen(36)).to(HF)
    ends = [(0, 65504), (-65504, 65504), (60000, 65504), (65472, 65504), (-65504, -65504), (65504, 65504), (-100, 65000), (1, 65504)]
    for t in range(16):
        for half in range(2):
            lo, hi = ends[(t + half) % len(ends)]
            row = x[t, 0, half * group:(half + 1) * group]
            row.copy_((lo + (hi - lo) * row.double()).to(HF))
            row[3], row[17] = lo, hi
    assert x.isfinite().all()
    kv = p4.PodKv4(1, 1, d, group_size=group, dtype=HF)
    pool, xc = kv.new_pool(1), x.cuda()
    cu, start, tab = (torch.tensor(v, dtype=torch.int32).cuda() for v in ([0, 16], [0], [[0]]))
    kv.write(kv.rows_args(cu, start, xc, xc, pool, tab))
    k, v = torch.zeros_like(xc), torch.zeros_like(xc)
    kv.read(kv.rows_args(cu, start, k, v, pool, tab))
    n, s, m, _ = ref.quantised(x, group)
    gn, gs, gm = (y[0, 0] for y in ref.unpack(pool.cpu(), d, group))
    # the pairs: as the formula has them, or one step of fp16 lower where they would pass 65520
    over = 15 * s + m >= 65520
    lower = (s.half().view(torch.int16) - over.to(torch.int16)).view(HF).double()
    assert over.any() and not over.all()
    for i in range(2):
        assert torch.equal(gs[i], lower[:, 0]) and torch.equal(gm[i], m[:, 0])
    for y in (k, v):
        assert y.isfinite().all()
        # half a step, the 15 / 2048 of a step by which s may be rounded or one step lower by, and the output's rounding (32 below 65504)
        assert ((y.cpu().double() - x.double()).abs() <= (0.5 + 15 * 2.0 ** -10) * s + 16).all()
    q = torch.zeros(1, 1, d, dtype=HF).cuda()
    o, lse = run_decode(kv, q, pool, tab, torch.tensor([16], dtype=torch.int32).cuda())
    check_decode(q, pool, tab, [16], d, group, o, lse)
    # one token alone: its values, the largest among them
    for t in (0, 1, 5):
        one = kv.new_pool(1)
        kv.write(kv.rows_args(torch.tensor([0, 1], dtype=torch.int32).cuda(), start, xc[t:t + 1], xc[t:t + 1], one, tab))
        o, lse = run_decode(kv, q, one, tab, torch.tensor([1], dtype=torch.int32).cuda())
        assert o.isfinite().all()
        check_decode(q, one, tab, [1], d, group, o, lse)


def test_write_far_pages():
    """Records whose byte offsets pass 32 bits: new rows leave there what they leave in a small pool, whole pages and parts of pages."""
    d, group, Hk, lens, starts = 128, 64, 4, [200, 50, 3], [0, 7, 30]
    kv = p4.PodKv4(Hk, Hk, d, group_size=group)
    table, cu, start = rows_case(lens, starts, 24, 37)
    small = kv.new_pool(24)
    blocks = (1 << 33) // (Hk * kv.record)
    pool = torch.empty(blocks, Hk, kv.record, dtype=torch.uint8, device="cuda")
    far = blocks - 24
    pool[far:] = 0
    # where offsets of the low 32 bits would lead
    low = [(((far + i) * Hk * kv.record) & 0xffffffff) // (Hk * kv.record) for i in (0, 23)]
    pool[low[0]:low[1] + 2] = 0
    x = torch.randn(sum(lens), 2 * Hk, d, generator=gen(38)).to(BF).cuda()
    tc = (table + far * (table >= 0)).int().cuda()
    kv.write(kv.rows_args(cu.cuda(), start.cuda(), x[:, :Hk], x[:, Hk:], small, table.cuda()))
    kv.write(kv.rows_args(cu.cuda(), start.cuda(), x[:, :Hk], x[:, Hk:], pool, tc))
    assert torch.equal(pool[far:], small) and small.any()
    assert not pool[low[0]:low[1] + 2].any()
    k, v = torch.zeros(sum(lens), Hk, d, dtype=BF, device="cuda"), torch.zeros(sum(lens), Hk, d, dtype=BF, device="cuda")
    kv.read(kv.rows_args(cu.cuda(), start.cuda(), k, v, pool, tc))
    # half a step of a group whose range is below 10, and roundings
    assert (k.float() - x[:, :Hk].float()).abs().max() < 0.5 and (v.float() - x[:, Hk:].float()).abs().max() < 0.5


def rag(n, least, most, seed):
    g = gen(seed)
    return torch.randint(least, most + 1, (n,), generator=g).tolist()


@pytest.mark.parametrize("lens,H,Hk,d,group,dtype", [
    (rag(20, 300, 3000, 40), 8, 2, 128, 64, BF),      # 148 workers, segments over two or three CTAs
    ([0, 1100, 0] + rag(8, 1, 3000, 41) + [0], 16, 4, 128, 32, HF),
    (rag(30, 1000, 2500, 42), 8, 1, 64, 64, BF),
    ([12000] * 4, 2, 2, 64, 32, HF), ([2600] * 30, 7, 1, 128, 128, BF),
])
def test_decode_that_fills_the_grid(lens, H, Hk, d, group, dtype):
    """All CTAs at work on contexts that go over their ends: heads and tails joined between CTAs, and calls that follow on
    each other find the counters as they should."""
    assert sum(-(-n // 16) for n in lens) * Hk >= 16 * 148 and max(lens) > 1024
    assert len(lens) * Hk * int(math.sqrt(0.6 * -(-max(lens) // 16))) >= 148
    q, pool, table = decode_case(lens, H, Hk, d, group, dtype, 43)
    kv = p4.PodKv4(H, Hk, d, group_size=group, dtype=dtype)
    args = q.cuda(), pool.cuda(), table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda()
    outs = [run_decode(kv, *args) for _ in range(4)]
    check_decode(q, pool, table, lens, d, group, *outs[0])
    for o, lse in outs[1:]:
        assert torch.equal(o, outs[0][0]) and torch.equal(lse, outs[0][1])
    assert kv.status() == pa.POD_OK


def test_arguments_go_to_contexts_of_their_shape():
    """Two contexts of one shape take each other's; one of other heads or groups refuses them."""
    lens = [40, 7]
    q, pool, table = decode_case(lens, 4, 2, 64, 64, BF, 44)
    qc, pc, tc, lc = q.cuda(), pool.cuda(), table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda()
    a, b = (p4.PodKv4(4, 2, 64, group_size=64, max_decode_reqs=n) for n in (2, 9))
    o, lse = torch.empty_like(qc), torch.empty(2, 4, device="cuda")
    args = a.decode_args(lc, qc, o, lse, pc, tc)
    b.decode(args)
    check_decode(q, pool, table, lens, 64, 64, o, lse)
    for other in (p4.PodKv4(2, 2, 64), p4.PodKv4(4, 2, 64, group_size=32), p4.PodKv4(4, 2, 64, dtype=HF)):
        with pytest.raises(ValueError):
            other.decode(args)
    with pytest.raises(ValueError):
        a.write(args)
