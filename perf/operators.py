"""Cases and plain forms of the 4-bit KV cache operators: the per-head norm of queries and keys
with their rotation, writing rows into the cache and reading them back, and single-token
attention over it.

Where ``own`` is false, ``run`` computes the operators with elementary torch operations in 32 bits;
where it is true, it calls the library.

The cache is a pool of records, one for each (page of 16 tokens, KV head), uint8
``[blocks, Hk, record]``. A record holds, one after the other, the 4-bit codes of K, those of V,
and for each token and group of channels the pair (scale, least value) in fp16 of K, then of V:

* K: token t, channel 32 c + 8 j + i is in byte t d/2 + 4 (j d/32 + c) + i/2;
* V: token 8 f + 2 j + e, channel 32 c + 4 r + i is in byte
  4 ((32 f + 4 r + j) d/32 + c) + 2 e + i/2;

the lower four bits first. A code n stands for n scale + least.
"""
import functools
import math
import random

import torch

own = False

PAGE = 16
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


# ---------------------------------------------------------------- cases

def listed():
    return [
        # one new token of one sequence, a model of 32 query and 8 KV heads: the latency of a step
        dict(name="rope_one", op="rope", rows=1, H=32, Hk=8, d=128, rot=128, pairs="halves", norm=True, dtype="bf16", first=4095, step=0),
        # a decode batch of a smaller model, half of each head rotated, neighbouring channels paired
        dict(name="rope_batch", op="rope", rows=253, H=16, Hk=4, d=64, rot=32, pairs="neighbours", norm=True, dtype="fp16", first=17, step=31),
        # a long prompt of a large model, far positions
        dict(name="rope_prompt", op="rope", rows=16384, H=64, Hk=8, d=128, rot=128, pairs="halves", norm=True, dtype="bf16", first=114688, step=1),
        # a decode step: one token of each of 256 sequences goes into the cache
        dict(name="write_step", op="write", reqs=256, least=1, most=1, prior=8192, Hk=8, d=128, group=64, dtype="bf16", ctx_seed=1),
        # many short chunks that begin and end inside pages
        dict(name="write_chunks", op="write", reqs=16, least=1, most=40, prior=8192, Hk=4, d=64, group=32, dtype="fp16", ctx_seed=2),
        # a whole prompt at once
        dict(name="write_prompt", op="write", reqs=1, least=16384, most=16384, prior=0, Hk=8, d=128, group=128, dtype="bf16", ctx_seed=3),
        # a short prefix
        dict(name="read_prefix", op="read", reqs=1, least=77, most=77, Hk=2, d=64, group=64, dtype="bf16", ctx_seed=4),
        # the cached tokens of two prompts ahead of their next chunks
        dict(name="read_prior", op="read", reqs=2, least=2560, most=8704, Hk=8, d=128, group=64, dtype="fp16", ctx_seed=5),
        # the smallest batch
        dict(name="attend_tiny", op="attend", reqs=4, least=40, most=200, H=4, Hk=2, d=64, group=32, dtype="bf16", ctx_seed=6),
        # 64 sequences of 4096 tokens
        dict(name="attend_even", op="attend", reqs=64, least=4096, most=4096, H=32, Hk=8, d=128, group=64, dtype="bf16", ctx_seed=7),
        # a ragged batch
        dict(name="attend_ragged", op="attend", reqs=128, least=512, most=8192, H=32, Hk=8, d=128, group=32, dtype="fp16", ctx_seed=8),
        # few long sequences, eight query heads on each KV head
        dict(name="attend_long", op="attend", reqs=16, least=16384, most=32768, H=64, Hk=8, d=128, group=64, dtype="bf16", ctx_seed=9),
    ]


def _log(rng, least, most):
    return int(round(math.exp(rng.uniform(math.log(least), math.log(most)))))


def draw(rng):
    op = rng.choice(["rope", "write", "read", "attend"])
    d = rng.choice([64, 128, 128])
    Hk = rng.choice([1, 2, 3, 4, 8, 8, 16])
    dtype = rng.choice(["bf16", "bf16", "fp16"])
    if op == "rope":
        return dict(op=op, rows=_log(rng, 1, 12000), H=Hk * rng.choice([1, 2, 3, 4]), Hk=Hk, d=d,
                    rot=rng.choice([d, d, d // 2, d - 16]), pairs=rng.choice(["halves", "neighbours"]),
                    norm=rng.random() < 0.75, dtype=dtype, first=rng.randrange(100000), step=rng.choice([1, 1, 7]))
    group = rng.choice([g for g in (32, 64, 128) if g <= d])
    case = dict(op=op, Hk=Hk, d=d, group=group, dtype=dtype, ctx_seed=rng.randrange(1 << 30))
    if op == "attend":
        most = _log(rng, 8, 40000)
        reqs = _log(rng, 1, max(1, min(256, 1600000 // (most * Hk))))
        return dict(case, reqs=reqs, least=rng.choice([0, most // 8, most // 2, most]), most=most, H=Hk * rng.choice([1, 2, 4, 5, 7, 8]))
    most = _log(rng, 1, 12000)
    reqs = _log(rng, 1, max(1, min(256, 100000 // (most * Hk))))
    case.update(reqs=reqs, least=rng.choice([0, 1, most // 2, most]), most=most)
    return dict(case, prior=rng.choice([0, 5, 1000, 20000])) if op == "write" else case


def _lens(case):
    """How many tokens each sequence brings; at least one in all."""
    r = random.Random(case["ctx_seed"])
    return [r.randint(case["least"], case["most"]) for _ in range(case["reqs"] - 1)] + [case["most"]]


def _priors(case):
    r = random.Random(case["ctx_seed"] + 1)
    return [r.randint(0, case["prior"]) for _ in range(case["reqs"])]


def _record(case):
    return PAGE * case["d"] + 2 * PAGE * 4 * (case["d"] // case["group"])


def work(case):
    d, Hk = case["d"], case["Hk"]
    if case["op"] == "rope":
        n = case["rows"] * (case["H"] + Hk) * d
        return {"bytes": 4 * n + case["rows"] * (4 + 4 * case["rot"]) + (4 * d if case["norm"] else 0), "flops": 9 * n}
    rows = sum(_lens(case))
    cached = rows * Hk * (d + 8 * d // case["group"])
    if case["op"] == "attend":
        return {"bytes": cached + case["reqs"] * case["H"] * (4 * d + 4) + 4 * (rows // PAGE + case["reqs"]), "flops": 4 * rows * case["H"] * d}
    plain = rows * Hk * 4 * d
    if case["op"] == "write":
        return {"bytes": 2 * (plain + cached), "flops": 14 * rows * Hk * d}
    return {"bytes": plain + cached, "flops": 4 * rows * Hk * d}


# ---------------------------------------------------------------- inputs

def _quantised(x, group):
    """Codes, scale and least value of x [..., d]; in 64 bits, since a code may lie next to a border."""
    x = x.double().unflatten(-1, (-1, group))
    fine = x.isfinite().all(-1)
    x = x.clamp(-65504.0, 65504.0)
    lo, hi = x.amin(-1), x.amax(-1)
    scale = ((hi - lo) / 15.0).half()
    scale, lo = torch.where(fine, scale, math.nan), torch.where(fine, lo.half(), math.nan)
    n = ((x - lo.double().unsqueeze(-1)) / torch.where(scale > 0, scale.double(), math.inf).unsqueeze(-1)).round().clamp(0.0, 15.0)
    return n.nan_to_num(0.0).float(), scale, lo


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    dt, d, Hk = DTYPES[case["dtype"]], case["d"], case["Hk"]
    randn = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    st = {"case": case}
    if case["op"] == "rope":
        rows, H, rot = case["rows"], case["H"], case["rot"]
        # the projection's output: q, k and v of a token side by side
        qkv = (randn(rows, H + 2 * Hk, d) * 1.5).to(dt)
        st["q"], st["k"] = qkv[:, :H], qkv[:, H:H + Hk]
        st["qw"] = (1 + 0.2 * randn(d)).to(dt) if case["norm"] else None
        st["kw"] = (1 + 0.2 * randn(d)).to(dt) if case["norm"] else None
        st["pos"] = (case["first"] + case["step"] * torch.arange(rows, device="cuda")).to(torch.int32)
        far = int(case["first"] + case["step"] * rows) + 1
        angle = torch.arange(far, device="cuda", dtype=torch.float64)[:, None] * torch.pow(
            500000.0, -torch.arange(0, rot, 2, device="cuda", dtype=torch.float64) / rot)
        st["table"] = torch.cat([angle.cos(), angle.sin()], 1).float()
        return st
    lens = _lens(case)
    prior = _priors(case) if case["op"] == "write" else [0] * len(lens)
    pages = [-(-(p + n) // PAGE) for p, n in zip(prior, lens)]
    wide, blocks = max(pages), max(1, sum(pages))
    # pages lie anywhere in the pool
    ids = torch.randperm(blocks, generator=g, device="cuda", dtype=torch.int32)
    first = torch.tensor([sum(pages[:i]) for i in range(len(pages))], device="cuda")
    col = torch.arange(wide, device="cuda")
    row = first[:, None] + col
    there = col < torch.tensor(pages, device="cuda")[:, None]
    st["table"] = torch.where(there, ids[row.clamp(max=blocks - 1)], 0).int().contiguous()
    st["lens"] = torch.tensor(lens, device="cuda", dtype=torch.int32)
    st["start"] = torch.tensor(prior, device="cuda", dtype=torch.int32)
    st["cu"] = torch.tensor([sum(lens[:i]) for i in range(len(lens) + 1)], device="cuda", dtype=torch.int32)
    st["rows"] = sum(lens)
    groups = d // case["group"]
    if case["op"] == "write":
        # keys have a few channels much larger than the others
        loud = torch.exp(0.5 * randn(Hk, d))
        qkv = torch.cat([randn(st["rows"], Hk, d) * loud, randn(st["rows"], Hk, d)], 1).to(dt)
        st["k"], st["v"] = qkv[:, :Hk], qkv[:, Hk:]
        st["pool"] = torch.zeros(blocks, Hk, _record(case), device="cuda", dtype=torch.uint8)
        return st
    # what normally distributed keys and values leave: ranges of about four to six deviations in 15 steps
    codes = torch.randint(0, 256, (blocks, Hk, PAGE * d), generator=g, device="cuda", dtype=torch.uint8)
    scale = 0.25 + 0.15 * torch.rand(blocks, Hk, 2 * PAGE * groups, generator=g, device="cuda")
    least = scale * -(7.5 + 1.5 * torch.rand(blocks, Hk, 2 * PAGE * groups, generator=g, device="cuda") - 0.75)
    st["pool"] = torch.cat([codes, torch.stack([scale, least], -1).half().view(torch.uint8).reshape(blocks, Hk, -1)], -1)
    if case["op"] == "attend":
        st["q"] = (1.2 * randn(case["reqs"], case["H"], d)).to(dt)
    return st


# ---------------------------------------------------------------- the library's calls

@functools.lru_cache(maxsize=None)
def _cache(H, Hk, d, group, dtype):
    """The handle that a program keeps for its cache."""
    from hybrid_prefill_decode_pod_b200 import pod_kv4
    return pod_kv4.PodKv4(H, Hk, d, group_size=group, dtype=DTYPES[dtype], max_decode_reqs=256, device=torch.cuda.current_device())


def _run_own(st):
    from hybrid_prefill_decode_pod_b200 import pod_kv4
    case = st["case"]
    if case["op"] == "rope":
        q, k = torch.empty_like(st["q"], memory_format=torch.contiguous_format), torch.empty_like(st["k"], memory_format=torch.contiguous_format)
        pod_kv4.qk_norm_rope(pod_kv4.norm_rope_args(st["q"], st["k"], st["pos"], st["table"], q_out=q, k_out=k, q_weight=st["qw"], k_weight=st["kw"],
                                                    eps=1e-6, interleaved=case["pairs"] == "neighbours"))
        return q, k
    cache = _cache(case.get("H", case["Hk"]), case["Hk"], case["d"], case["group"], case["dtype"])
    if case["op"] == "attend":
        o, lse = torch.empty_like(st["q"]), torch.empty(st["q"].shape[:2], device="cuda", dtype=torch.float32)
        cache.decode(cache.decode_args(st["lens"], st["q"], o, lse, st["pool"], st["table"]))
        return o, lse
    if case["op"] == "write":
        cache.write(cache.rows_args(st["cu"], st["start"], st["k"], st["v"], st["pool"], st["table"]))
    k = torch.empty(st["rows"], case["Hk"], case["d"], device="cuda", dtype=DTYPES[case["dtype"]])
    v = torch.empty_like(k)
    cache.read(cache.rows_args(st["cu"], st["start"], k, v, st["pool"], st["table"]))
    return k, v


# ---------------------------------------------------------------- the plain forms

def _rotated(x, cos, sin, pairs):
    half = cos.shape[-1]
    a, b = (x[..., :half], x[..., half:2 * half]) if pairs == "halves" else (x[..., 0:2 * half:2], x[..., 1:2 * half:2])
    c, s = cos[:, None], sin[:, None]
    y = [a * c - b * s, a * s + b * c]
    y = torch.cat(y, -1) if pairs == "halves" else torch.stack(y, -1).flatten(-2)
    return torch.cat([y, x[..., 2 * half:]], -1)


def _rope(x, w, st):
    y = x.float()
    if w is not None:
        y = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + 1e-6) * w.float()
    t = st["table"][st["pos"].long()]
    cos, sin = t.chunk(2, -1)
    return _rotated(y, cos, sin, st["case"]["pairs"]).to(x.dtype)


def _values(records, d):
    """K and V [..., PAGE, d] in 32 bits of records [..., record]."""
    lead, at = records.shape[:-1], list(range(records.dim() - 1))
    codes = records[..., :PAGE * d].unsqueeze(-1)
    codes = torch.cat([codes & 15, codes >> 4], -1).reshape(*lead, 2, -1)
    k = codes[..., 0, :].reshape(*lead, PAGE, 4, d // 32, 8).transpose(-3, -2).reshape(*lead, PAGE, d)
    v = codes[..., 1, :].reshape(*lead, 2, 8, 4, d // 32, 2, 4)       # f r j c e i
    v = v.permute(*at, *[len(at) + x for x in (0, 2, 4, 3, 1, 5)]).reshape(*lead, PAGE, d)
    par = records[..., PAGE * d:].contiguous().view(torch.float16).reshape(*lead, 2, PAGE, -1, 2).float()
    of = lambda n, p: (n.unflatten(-1, (p.shape[-2], -1)).float() * p[..., 0:1] + p[..., 1:2]).flatten(-2)  # noqa: E731
    return of(k, par[..., 0, :, :, :]), of(v, par[..., 1, :, :, :])


def _attend(st):
    case = st["case"]
    d, Hk, R = case["d"], case["Hk"], case["reqs"]
    k, v = _values(st["pool"][st["table"].long()], d)                  # R, pages, Hk, PAGE, d
    k, v = (x.transpose(1, 2).reshape(R, Hk, -1, d) for x in (k, v))
    q = st["q"].float().reshape(R, Hk, -1, d)
    s = torch.matmul(q, k.transpose(-1, -2)) / math.sqrt(d)
    seen = (torch.arange(k.shape[2], device="cuda") < st["lens"][:, None])[:, None, None]
    s = torch.where(seen, s, -math.inf)
    top = s.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    p = torch.exp(s - top)
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p, v) / torch.where(total == 0, 1.0, total)
    return o.reshape(R, -1, d).to(st["q"].dtype), (top + total.log()).reshape(R, -1)


def _read(st):
    case = st["case"]
    k, v = _values(st["pool"][st["table"].long()], case["d"])
    k, v = (x.transpose(2, 3).flatten(1, 2) for x in (k, v))           # R, tokens, Hk, d
    seen = torch.arange(k.shape[1], device="cuda") < st["lens"][:, None]
    return k[seen].to(DTYPES[case["dtype"]]), v[seen].to(DTYPES[case["dtype"]])


def _write(st):
    def back(x):
        n, scale, lo = _quantised(x, st["case"]["group"])
        return (n * scale.float().unsqueeze(-1) + lo.float().unsqueeze(-1)).flatten(-2).to(x.dtype)
    return back(st["k"]), back(st["v"])


def run(state):
    if own:
        return _run_own(state)
    op = state["case"]["op"]
    if op == "rope":
        return _rope(state["q"], state["qw"], state), _rope(state["k"], state["kw"], state)
    return {"attend": _attend, "read": _read, "write": _write}[op](state)


# ---------------------------------------------------------------- 64 bits

def _exact_rope(x, w, st):
    rows, heads, d = x.shape
    y = x.double()
    if w is not None:
        y = y / ((y * y).sum(2, keepdim=True) / d + 1e-6).sqrt() * w.double()
    rot = st["table"].shape[1]
    z, out = y.clone(), st["table"][st["pos"].long()].double()
    for i in range(rot // 2):
        a, b = (i, i + rot // 2) if st["case"]["pairs"] == "halves" else (2 * i, 2 * i + 1)
        turn = torch.complex(out[:, i], out[:, rot // 2 + i])[:, None] * torch.complex(y[..., a], y[..., b])
        z[..., a], z[..., b] = turn.real, turn.imag
    return z


def _exact_back(x, group):
    parts = []
    for y in x.double().clamp(-65504.0, 65504.0).split(group, -1):
        lo, hi = y.min(-1, keepdim=True).values, y.max(-1, keepdim=True).values
        s, m = ((hi - lo) / 15).half().double(), lo.half().double()
        parts.append(m + s * torch.where(s > 0, ((y - m) / s).round().clamp(0, 15), 0.0))
    return torch.cat(parts, -1)


def _exact_page(case):
    """Where each (token, channel) of a page has its code, as an index into a record's 4-bit codes, and its pair, as one into its fp16 values."""
    d, group = case["d"], case["group"]
    t, ch = torch.arange(PAGE, device="cuda")[:, None], torch.arange(d, device="cuda")[None]
    k = t * d + 8 * ((ch % 32 // 8) * (d // 32) + ch // 32) + ch % 8
    v = PAGE * d + 8 * ((32 * (t // 8) + 4 * (ch % 32 // 4) + t % 8 // 2) * (d // 32) + ch // 32) + 4 * (t % 2) + ch % 4
    pair = 2 * (t * (d // group) + ch // group)
    return (k, pair), (v, pair + 2 * PAGE * (d // group))


def _exact_sequence(st, i, n):
    """K and V [n, Hk, d] in 64 bits of sequence i."""
    case = st["case"]
    rec = st["pool"][st["table"][i, :-(-n // PAGE)].long()]
    codes, pars = rec[..., :PAGE * case["d"]], rec[..., PAGE * case["d"]:].contiguous().view(torch.float16)
    out = []
    for code, pair in _exact_page(case):
        byte = codes[..., code // 2]
        val = (byte.int() >> (4 * (code % 2))) % 16
        val = val.double() * pars[..., pair].double() + pars[..., pair + 1].double()
        out.append(val.transpose(1, 2).reshape(-1, case["Hk"], case["d"])[:n])
    return out


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "rope":
        return _exact_rope(st["q"], st["qw"], st), _exact_rope(st["k"], st["kw"], st)
    if case["op"] == "write":
        return _exact_back(st["k"], case["group"]), _exact_back(st["v"], case["group"])
    lens = _lens(case)
    if case["op"] == "read":
        both = [_exact_sequence(st, i, n) for i, n in enumerate(lens)]
        return torch.cat([b[0] for b in both]), torch.cat([b[1] for b in both])
    R, H, d = st["q"].shape
    o = torch.zeros(R, H, d, dtype=torch.float64, device="cuda")
    lse = torch.full((R, H), -math.inf, dtype=torch.float64, device="cuda")
    for i, n in enumerate(lens):
        if n:
            k, v = _exact_sequence(st, i, n)
            q = st["q"][i].double().reshape(case["Hk"], -1, d)
            s = torch.einsum("hgd,nhd->hgn", q, k) / d ** 0.5
            lse[i] = torch.logsumexp(s, -1).reshape(H)
            o[i] = torch.einsum("hgn,nhd->hgd", torch.softmax(s, -1), v).reshape(H, d)
    return o, lse
