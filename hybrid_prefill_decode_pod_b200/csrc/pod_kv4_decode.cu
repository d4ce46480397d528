// pod_kv4_decode.cu -- single-token GQA attention over the 4-bit KV cache.
//
// Its floor is the cache's bytes: 16 D + 128 D / group for 16 tokens of one head
// (2304 at D = 128, groups of 64), which an SM's share of 6.5 TB/s brings every
// 95 cycles. What it costs is taking the codes apart: 4096 codes of such a block
// are 64 pairs for each lane, so every instruction for a pair is 64 of the
// block's about 380 issue slots. Hence
//
//  * K^T q as matrix products with the codes themselves. A code n in the low
//    bits of an fp16 is the subnormal n 2^-24, exactly: one AND makes two of
//    them (the codes in bits 4..7 are n 2^-20, undone in the query). The
//    queries are scaled by a power of two so that their largest channel lies in
//    [2^9, 2^10); 2^-31 of it is then the rounding of the others. Tokens are
//    the rows of the product and the G <= 8 heads its columns, so no row is
//    padding. Each channel group is summed by itself in fp32 and
//    score = s (sum q n) + m (sum q) joins them.
//  * V^T p as well: rows are channels, columns heads, the same subnormals
//    times the weights p s, rounded to fp16. What the rounding costs is the
//    weight's error times n - 8, not n: eight of each rounded weight are
//    taken away and sum p (m + 8 s) in fp32 puts them back unrounded. (Half
//    of the rows take whole bytes n0 + 16 n1, from which 16 n1 is taken away
//    after the sums: those are of up to 256 s and lose four of fp32's bits,
//    2^-16 of 16 s in all.) So that the weights lie high in fp16, each 64
//    tokens scale them by a power of two that brings the largest s to [2^13,
//    2^14): a weight is then off by 2^-11 of itself, or by 2^-39 of the
//    largest possible one where it is below 2^-28 of that (together below
//    2^-19 of a million tokens' weight). With bf16 weights (2^-8) the error
//    of an fp16 output was several times that of its own rounding.
//  * The running maximum and sum, scores, weights and O are fp32; one rescale
//    every 64 tokens.
//
// Work: see pod_kv4_split.h. The line of blocks is cut into parts of equal cost
// over the CTAs and each of those over its warps, so lengths need no balance
// and no plan from the host. (Cut into equal numbers of blocks, 256 contexts of
// 1 to 1000 tokens took 83 us, in order of length 160; by cost 46 and 47.)
// Warps stream their blocks, one bulk copy each, through rings of their own,
// across segments. What a warp has of a segment that it does not hold whole is
// joined first in its CTA, then, where the segment leaves the CTA, through the
// workspace by the CTA that arrives last, in the order of the tokens: the
// result does not depend on the order of arrival.
//
// Measured on B200s (a call, L2 not warm; they differ by 5 %): 64 x 4096 tokens
// of 8 KV heads, G = 4, groups of 64: 71 to 72 us, 4.2 TB/s; 16 x 16K..32K, G =
// 8: 108 to 113 us, 4.3 TB/s; 128 x 0.5K..8K, G = 4, groups of 32: 146 to 155
// us, 4.7 TB/s. The copies alone, with the joins, took 59, 85 and 120 us where
// all took 72, 113 and 156, the second 101 with its records in L2. 240 to 256
// warp instructions a block fill 44 to 48 % of the issue slots, the integer
// pipe (the ANDs) is 44 % busy, the matrix pipe 25 to 28 %: what bounds it is
// latency, two warps a scheduler that go through a tile's products, maximum,
// weights and products one after the other.
#include <algorithm>
#include <cfloat>

#include "pod_kv4.cuh"
#include "pod_kv4_split.h"
#include "pod_plan.h"
#include "pod_ptx.cuh"

namespace pod {
namespace {

// 8 warps of up to 255 registers (40 bytes spilled at D = 128, groups of 32,
// G > 4; none elsewhere): 12 of 168 issue more at a time, but spill and begin more
// pieces (113 against 118 us for the long case, 72 against 75 for 64 x 4096, before
// the last steps), 16 of 128 took 133 and 77.
constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
// Blocks of 16 tokens between two rescales: 2 took 127 us for the long case, 4
// 113, 6 and 8 no less.
constexpr int kTile = 4;
constexpr int kSlots = 8;  // blocks in a warp's ring; 10 change nothing, 5 cost 1 %
constexpr int kKeys = 4;   // blocks whose scores are taken together
constexpr int kMaxG = 8;
constexpr int kNever = -2;
constexpr int kLeast = 16;  // blocks that make another CTA worth its join
// Up to this many blocks in the longest context (1024 tokens) a segment stays in
// one CTA: the joins between CTAs take about 4 us, in which a CTA does some 64
// blocks. 16 x 1000 tokens, 8 KV heads: 16.2 us cut anywhere, 12.3 whole; 8 x 100:
// 13.7 and 9.4.
constexpr int kWhole = 64;
constexpr float kLn2 = 0.69314718055994531f, kLog2e = 1.4426950408889634f;

// d = a b + c: 16 x 16 times 16 x 8
__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                    uint32_t a3, uint32_t b0, uint32_t b1, const float (&c)[4]) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%10,%11,%12,%13};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c[0]), "f"(c[1]), "f"(c[2]),
        "f"(c[3]));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}
__device__ __forceinline__ uint32_t f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// N words of shared memory, N = 1, 2 or 4
template <int N>
__device__ __forceinline__ void lds(uint32_t (&v)[N], uint32_t at) {
  if constexpr (N == 4)
    asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]) : "r"(at));
  else if constexpr (N == 2)
    asm volatile("ld.shared.v2.b32 {%0,%1}, [%2];" : "=r"(v[0]), "=r"(v[1]) : "r"(at));
  else
    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v[0]) : "r"(at));
}
// The pairs of every REP-th group
template <int NP, int REP>
__device__ __forceinline__ void own_pairs(uint32_t (&v)[NP], uint32_t at) {
  if constexpr (REP == 1) {
    lds<NP>(v, at);
  } else {
#pragma unroll
    for (int u = 0; u < NP; ++u) {
      uint32_t x[1];
      lds<1>(x, at + u * REP * 4);
      v[u] = x[0];
    }
  }
}
// Waits for a phase of a ring slot; gives up after `budget` cycles (false).
__device__ __noinline__ bool slow_wait(uint32_t bar, uint32_t parity, long long budget) {
  const long long t0 = clock64();
  while (!mbar_try_wait(bar, parity))
    if (clock64() - t0 > budget) return false;
  return true;
}
constexpr int kStatusTimeout = -5;  // POD_ETIMEOUT
// (about 1 ms where a test makes waits run out)
__device__ __forceinline__ long long budget(const Kv4Decode& P) {
  return P.force ? kDefaultWaitBudget / 1000 : kDefaultWaitBudget;
}

// A wait of this warp ran out before its block `done`: waits for every copy that it
// still has under way (issued blocks, each by its own slot and phase), so that none
// lands in shared memory that is used for something else, and records the status.
__device__ __noinline__ void give_up(uint32_t bars, int done, int issued, int slots,
                                     const Kv4Decode& P) {
  for (int i = done; i < issued; ++i) slow_wait(bars + i % slots * 8, i / slots & 1, budget(P));
  __syncwarp();
  if ((threadIdx.x & 31) == 0) atomicExch(P.status, kStatusTimeout);
}
// The upper bytes of both halves
__device__ __forceinline__ uint32_t high_bytes(uint32_t v) { return __byte_perm(v, 0, 0x4341); }
// max or sum over the eight rows of a fragment (lanes 4 apart)
__device__ __forceinline__ float rows_max(float x) {
#pragma unroll
  for (int o = 4; o < 32; o <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
  return x;
}
__device__ __forceinline__ float rows_sum(float x) {
#pragma unroll
  for (int o = 4; o < 32; o <<= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// What a warp has of the segment at the start or the end of its blocks.
struct PieceMeta {
  int has[2];  // [0] goes on from the blocks before, [1] begins here and goes on
  int ends0;   // [0] reaches the end of its segment
  int final0;  // [0] is the warp's last piece
  int r[2], h[2];
};

// A segment that other CTAs hold parts of: this CTA's first (which does not begin
// here or goes on), or its last (which begins here and goes on). c0 .. c1 are
// the CTAs; c0 = c1 where there is none.
struct Shared {
  int r, h, c0, c1;
};

template <int D, int GROUP>
struct Shape {
  static constexpr int kRec = kv4_record_bytes(D, GROUP);
  static constexpr int NG = D / GROUP, NC = D / 32;  // channel groups, chunks of 32 channels
  static constexpr int kRing = kSlots * kRec;
  static constexpr int CG = GROUP / 32;  // chunks of a group
  // shared memory: rings, (max, sum) of the partial results, pieces, then the
  // requests' first blocks
  static constexpr int kMlOff = kWarps * kRing;  // float [warp][2][kMaxG][2]
  static constexpr int kMetaOff = kMlOff + kWarps * 2 * kMaxG * 2 * 4;
  static constexpr int kMiscOff = kMetaOff + kWarps * (int)sizeof(PieceMeta);
  // mbarrier [warp][slot]
  static constexpr int kBarOff = (kMiscOff + 3 * kWarps * 4 + 2 * (int)sizeof(Shared) + 7) / 8 * 8;
  // a record whose pairs are 0, for a tile of fewer than kTile blocks
  static constexpr int kZeroOff = (kBarOff + kWarps * kSlots * 8 + 15) / 16 * 16;
  static constexpr int kFirstOff = kZeroOff + kRec;
  static __host__ int smem(int reqs) { return kFirstOff + 2 * (reqs + 1) * 4; }
};

// REP: how often each head stands among the eight columns of the products
// (columns REP of them apart, 8 / REP heads at most). With REP > 1 a column
// takes every REP-th channel group only: its queries are 0 in the others, so one
// accumulator holds REP groups' sums, the pairs (s, m) of REP groups are applied
// by one instruction, and REP groups' weights are one operand.
template <int D, int GROUP, bool FP16, int REP>
__global__ void __launch_bounds__(kThreads, 1) kv4_decode_kernel(const Kv4Decode P) {
  using S = Shape<D, GROUP>;
  constexpr int NG = S::NG, NC = S::NC, CG = S::CG, kRec = S::kRec;
  constexpr int NP = NG / REP;           // passes over the groups
  constexpr int kPart = REP > 1 || CG == 1 ? 1 : 2;  // chunks of a group at a time in V^T p
  extern __shared__ __align__(128) unsigned char smem[];
  float* ml = reinterpret_cast<float*>(smem + S::kMlOff);
  PieceMeta* meta = reinterpret_cast<PieceMeta*>(smem + S::kMetaOff);
  int* misc = reinterpret_cast<int*>(smem + S::kMiscOff);
  Shared* out = reinterpret_cast<Shared*>(misc + 3 * kWarps);
  int* first = reinterpret_cast<int*>(smem + S::kFirstOff);
  int* cost = first + P.num_reqs + 1;
  const int tid = threadIdx.x, w = tid >> 5, lane = tid & 31, row = lane >> 2, j = lane & 3;
  // the replica and the heads of this lane's columns 2 j and 2 j + 1
  const int rep = REP == 1 ? 0 : REP == 2 ? j >> 1 : j, head0 = 2 * j % (8 / REP);
  const int R = P.num_reqs, Hk = P.Hk, G = P.G;
  const long long part_stride = (long long)G * D + 2 * kMaxG;  // floats of a partial result
  // the workspace of this CTA: its two parts for other CTAs, then one for each warp
  float* ws = P.part + blockIdx.x * (2 + kWarps) * part_stride;
  const long long cap = min((long long)P.table_stride * kKv4Page, (1LL << 31) - 16);
  const auto length = [&](int r) { return (int)min((long long)max(__ldg(P.ctx_lens + r), 0), cap); };

  // first[r], cost[r]: blocks of one head in front of request r, and their cost
  int longest = 0;
  {
    const int each = (R + kThreads - 1) / kThreads, r0 = min(tid * each, R), r1 = min(r0 + each, R);
    int sum = 0, sum_c = 0, big = 0;
    for (int r = r0; r < r1; ++r) {
      const int n = (length(r) + 15) >> 4;
      sum += n;
      sum_c += kv4_cost(n);
      big = max(big, n);
    }
    big = __reduce_max_sync(0xffffffffu, big);
    int inc = sum, inc_c = sum_c;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, inc, o), z = __shfl_up_sync(0xffffffffu, inc_c, o);
      if (lane >= o) {
        inc += y;
        inc_c += z;
      }
    }
    if (lane == 31) {
      misc[w] = inc;
      misc[kWarps + w] = inc_c;
      misc[2 * kWarps + w] = big;
    }
    if (tid < kWarps) meta[tid].has[0] = meta[tid].has[1] = 0;
    if (tid < kWarps * kSlots) mbar_init(smem_u32(smem + S::kBarOff) + tid * 8, 1);
    fence_mbar_init();
    for (int i = tid; i < kRec / 4; i += kThreads)
      reinterpret_cast<uint32_t*>(smem + S::kZeroOff)[i] = 0;
    __syncthreads();
    int before = inc - sum, before_c = inc_c - sum_c;
    for (int x = 0; x < kWarps; ++x) {
      if (x < w) {
        before += misc[x];
        before_c += misc[kWarps + x];
      }
      longest = max(longest, misc[2 * kWarps + x]);
    }
    for (int r = r0; r < r1; ++r) {
      const int n = (length(r) + 15) >> 4;
      first[r] = before;
      cost[r] = before_c;
      before += n;
      before_c += kv4_cost(n);
    }
    if (tid == kThreads - 1) {
      first[R] = before;
      cost[R] = before_c;
    }
    __syncthreads();
  }
  const long long W = (long long)first[R] * Hk;

  // empty contexts
  for (int r = blockIdx.x; r < R; r += gridDim.x) {
    if (first[r] != first[r + 1]) continue;
    uint32_t* o = reinterpret_cast<uint32_t*>(P.o + (long long)r * P.H * D);
    for (int i = tid; i < P.H * D / 2; i += kThreads) o[i] = 0;
    for (int i = tid; i < P.H; i += kThreads) P.lse[(long long)r * P.H + i] = -INFINITY;
  }
  if (W == 0) return;
  const bool whole = longest <= kWhole;
  const int cta = blockIdx.x, least = kv4_workers(W, gridDim.x, kLeast);
  // A segment of n blocks in p parts costs about n / p times 0.055 us and p times
  // 0.09 us for the join of the parts: p up to sqrt(0.6 n). One context of 30000
  // tokens of one KV head in 117 parts: 21 us, in 34 16 us.
  const long long parts = (long long)R * Hk * max(1, (int)sqrtf(0.6f * longest));
  const int N = whole ? max(least, (int)min((long long)R * Hk, (long long)gridDim.x))
                      : (int)min((long long)least, parts);
  if (cta >= N) return;

  // ------------------------------------------------ this warp's blocks
  const long long V = (long long)cost[R] * Hk;
  // lane 0 looks up the beginning, lane 1 the end
  const int end_lane = min(lane, 1);
  long long v = kv4_begin(V, N, cta + end_lane);
  if (whole) v = kv4_snap(cost, R, Hk, v);
  long long x_of = kv4_cut(first, cost, R, Hk, v);
  const long long vb = __shfl_sync(0xffffffffu, v, 0), ve = __shfl_sync(0xffffffffu, v, 1);
  const long long cb = __shfl_sync(0xffffffffu, x_of, 0), ce = __shfl_sync(0xffffffffu, x_of, 1);
  if (cb == ce) return;
  // The warps take equal numbers of blocks where the CTA has few segments (each
  // warp begins a piece anyway), equal costs where it has more than warps.
  if (ve - vb - (ce - cb) <= kKv4Start * kWarps)
    x_of = cb + kv4_begin(ce - cb, kWarps, w + end_lane);
  else
    x_of = kv4_cut(first, cost, R, Hk, vb + kv4_begin(ve - vb, kWarps, w + end_lane));
  const long long xb = __shfl_sync(0xffffffffu, x_of, 0), xe = __shfl_sync(0xffffffffu, x_of, 1);
  const int total = (int)(xe - xb);
  unsigned char* ring = smem + w * S::kRing;
  const uint32_t ring_s = smem_u32(ring), bar_s = smem_u32(smem + S::kBarOff) + w * kSlots * 8,
                 zero_s = smem_u32(smem + S::kZeroOff);

  // Lane i of `cur` has the record of block 32 b + i, of `nxt` that of the 32
  // behind; -1 where the page id lies outside the pool. (kNever, in a test: this
  // block's copy is left out.)
  Kv4Place seg{0, 0, 0, 1};  // of the first block, once every lane has it from lane 0
  const auto records = [&](int base) {
    int rec = 0;
    if (base + lane < total) {
      const Kv4Place p = kv4_place(first, R, Hk, xb + base + lane);
      if (base == 0) seg = p;
      const int page = __ldg(P.table + (long long)p.r * P.table_stride + p.blk);
      rec = page >= 0 && page < P.pool_blocks ? page * Hk + p.h : -1;
      if (P.force && base + lane == min(kTile * w, total - 1)) rec = kNever;
    }
    return rec;
  };
  int cur = records(0), nxt = records(32);
  int issued = 0, islot = 0;
  bool bad = false;  // this lane met a page id outside the pool
  // Copies the next `count` blocks into the slots they follow on: block i by lane
  // i % 32, which holds its record.
  const auto issue = [&](int count) {
    const int d = (lane - issued) & 31;
    if (d < count && issued + d < total) {
      const int rec = (issued & 31) + d < 32 ? cur : nxt;
      const int sl = islot + d >= kSlots ? islot + d - kSlots : islot + d;
      if (rec >= 0) {
        mbar_expect_tx(bar_s + sl * 8, kRec);
        bulk_load(ring_s + sl * kRec, P.pool + (long long)rec * kRec, kRec, bar_s + sl * 8);
      } else if (rec != kNever) {
        mbar_arrive(bar_s + sl * 8);
        bad = true;
      }
    }
    if ((issued & 31) + count >= 32 && issued < total) {
      cur = nxt;
      nxt = records((issued & ~31) + 64);
    }
    issued += count;
    islot = islot + count >= kSlots ? islot + count - kSlots : islot + count;
  };
  issue(kSlots);
  seg.r = __shfl_sync(0xffffffffu, seg.r, 0);
  seg.h = __shfl_sync(0xffffffffu, seg.h, 0);
  seg.blk = __shfl_sync(0xffffffffu, seg.blk, 0);
  seg.nblk = __shfl_sync(0xffffffffu, seg.nblk, 0);

  // what the CTA's ends share with others, while the first blocks are on their way
  if (lane == 0 && w < 2) {
    const Kv4Place p = kv4_place(first, R, Hk, w ? ce - 1 : cb);
    const long long x0 = (long long)Hk * first[p.r] + (long long)p.h * p.nblk;
    Shared m{p.r, p.h, 0, 0};
    if (w ? x0 >= cb && x0 + p.nblk > ce : x0 < cb) {
      m.c0 = kv4_worker(cost, R, Hk, N, p.r, p.h, 0);
      m.c1 = kv4_worker(cost, R, Hk, N, p.r, p.h, p.nblk - 1);
    }
    out[w] = m;
  }

  int slot = 0, phase = 0;  // of the next block
  bool failed = false;  // a wait of this warp ran out: what it has from there on is NaN
  for (long long x = xb; x < xe;) {
    if (x > xb) {  // the next head, or the next request that is not empty
      seg.blk = 0;
      if (++seg.h == Hk) {
        seg.h = 0;
        do {
          ++seg.r;
          seg.nblk = first[seg.r + 1] - first[seg.r];
        } while (seg.nblk == 0);
      }
    }
    const int n = (int)min((long long)(seg.nblk - seg.blk), xe - x);
    const int len = length(seg.r);
    const long long orow = (long long)seg.r * P.H + (long long)seg.h * G;

    // The queries as the second operand: column `row` is a head, chunk c's
    // channels 32 c + 8 j + i in the order in which K's codes come apart. A score
    // is p 2^24 F ln 2. (2^24 F may pass fp32 where the queries pass 2^116; cut, it
    // still makes every weight but the largest 0.)
    uint32_t qf[NC][4];
    float qs[NP][2], F[2];
    {
      const int q_head = row % (8 / REP), q_rep = row / (8 / REP);
      float q[NC][8];
      uint32_t most = 0;  // the largest magnitudes, in the queries' own type
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        uint4 v = make_uint4(0, 0, 0, 0);
        if (q_head < G)
          v = __ldg(reinterpret_cast<const uint4*>(P.q + (orow + q_head) * D + 32 * c + 8 * j));
        const uint32_t vv[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 f = row2_to_float<FP16>(vv[i]);
          q[c][2 * i] = f.x;
          q[c][2 * i + 1] = f.y;
          most = max2<FP16>(most, vv[i] & 0x7fff7fffu);
        }
      }
      most = max2<FP16>(most, __shfl_xor_sync(0xffffffffu, most, 1));
      most = max2<FP16>(most, __shfl_xor_sync(0xffffffffu, most, 2));
      most = max2<FP16>(most, most >> 16);
      const int e = __float_as_int(row2_to_float<FP16>(most).x) >> 23;  // 255 for NaN too
      const float sc = e == 0 || e == 255 ? 1.f : __int_as_float(min(263 - e, 254) << 23);
      const float f = P.scale_log2 / sc;
      float sum[NP];
#pragma unroll
      for (int u = 0; u < NP; ++u) sum[u] = 0.f;
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        const bool own = c / CG % REP == q_rep;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          q[c][i] = own ? q[c][i] * sc : 0.f;
          sum[c / CG / REP] += q[c][i];
        }
        qf[c][0] = float_to_row2<true>(q[c][0], q[c][4]);
        qf[c][1] = float_to_row2<true>(q[c][1] * 0.0625f, q[c][5] * 0.0625f);
        qf[c][2] = float_to_row2<true>(q[c][2], q[c][6]);
        qf[c][3] = float_to_row2<true>(q[c][3] * 0.0625f, q[c][7] * 0.0625f);
      }
#pragma unroll
      for (int u = 0; u < NP; ++u) {
        sum[u] += __shfl_xor_sync(0xffffffffu, sum[u], 1);
        sum[u] += __shfl_xor_sync(0xffffffffu, sum[u], 2);
        qs[u][0] = __shfl_sync(0xffffffffu, sum[u], 8 * j) * 0x1p-24f;
        qs[u][1] = __shfl_sync(0xffffffffu, sum[u], 8 * j + 4) * 0x1p-24f;
      }
      F[0] = __shfl_sync(0xffffffffu, f, 8 * j);
      F[1] = __shfl_sync(0xffffffffu, f, 8 * j + 4);
    }

    // the next segment's queries come closer meanwhile (they follow on, empty requests apart)
    if (x + n < xe && lane * 64 < G * D)
      asm volatile("prefetch.global.L1 [%0];" ::"l"(P.q + min((orow + G) * D + lane * 64, (long long)R * P.H * D - 8)));

    // State of heads head0 (x) and head0 + 1 (y): O of channels 4 row + 0..3 of the
    // own groups' chunks, this lane's part of the sums of p and of p (m + 8 s).
    float2 O[NC / REP][4], pm[NP], l = make_float2(0.f, 0.f);
    float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
    for (int c = 0; c < NC / REP; ++c)
#pragma unroll
      for (int i = 0; i < 4; ++i) O[c][i] = make_float2(0.f, 0.f);
#pragma unroll
    for (int g = 0; g < NP; ++g) pm[g] = make_float2(0.f, 0.f);

    for (int t0 = 0; t0 < n && !failed; t0 += kTile) {
      const int nb = min(kTile, n - t0);
      // lane b waits for the tile's block b
      {
        const int sl = slot + lane;
        const uint32_t bar = bar_s + (sl >= kSlots ? sl - kSlots : sl) * 8;
        const uint32_t parity = phase ^ (sl >= kSlots);
        const bool late =
            lane < nb && !mbar_try_wait(bar, parity) && !slow_wait(bar, parity, budget(P));
        __syncwarp();
        failed = __any_sync(0xffffffffu, late);
        if (failed) {
          give_up(bar_s, (int)(x - xb) + t0, min(issued, total), kSlots, P);
          break;
        }
      }
      // The blocks' records. A tile of fewer than kTile blocks takes the zero
      // record instead, so that all of the tile's work is one run of
      // independent instructions.
      uint32_t at[kTile];
#pragma unroll
      for (int b = 0; b < kTile; ++b) {
        at[b] = ring_s + slot * kRec + b * kRec;
        if (slot + b >= kSlots) at[b] -= kSlots * kRec;
      }
      if (nb < kTile) {
#pragma unroll
        for (int b = 1; b < kTile; ++b)
          if (b >= nb) at[b] = zero_s;
      }
      // tokens of the tile
      const int left = min(len - (seg.blk + t0) * kKv4Page, nb * kKv4Page);
      if (left & 15) {
        // Tokens behind the length get s = m = 0, whatever their bits say.
        __syncwarp();
        const uint32_t rec = ring_s + (slot + nb - 1 - (slot + nb > kSlots ? kSlots : 0)) * kRec;
        if ((lane & 15) >= (left & 15)) {
#pragma unroll
          for (int g = 0; g < NG; ++g)
            asm volatile("st.shared.b32 [%0], %1;" ::"r"(rec + 16 * D + lane * NG * 4 + g * 4), "r"(0) : "memory");
        }
        fence_proxy_async_smem();
        __syncwarp();
      }
      // ---- scores of the tile's tokens: rows `row`, `row` + 8 of each block
      float p[kTile][4];
      {
#pragma unroll
        for (int h = 0; h < kTile; h += kKeys) {
          uint32_t ka[kKeys][NC], kb[kKeys][NC], kp[kKeys][2][NP];
#pragma unroll
          for (int b = 0; b < kKeys; ++b) {
            own_pairs<NP, REP>(kp[b][0], at[h + b] + 16 * D + (row * NG + rep) * 4);
            own_pairs<NP, REP>(kp[b][1], at[h + b] + 16 * D + ((row + 8) * NG + rep) * 4);
            lds<NC>(ka[b], at[h + b] + lane * (D / 8));
            lds<NC>(kb[b], at[h + b] + 4 * D + lane * (D / 8));
          }
#pragma unroll
          for (int u = 0; u < NP; ++u) {
            float acc[kKeys][4];
#pragma unroll
            for (int b = 0; b < kKeys; ++b)
#pragma unroll
              for (int i = 0; i < 4; ++i) acc[b][i] = 0.f;
#pragma unroll
            for (int c = u * REP * CG; c < (u + 1) * REP * CG; ++c) {
#pragma unroll
              for (int b = 0; b < kKeys; ++b)
                mma(acc[b], ka[b][c] & 0x000f000fu, kb[b][c] & 0x000f000fu, ka[b][c] & 0x00f000f0u,
                    kb[b][c] & 0x00f000f0u, qf[c][0], qf[c][1], acc[b]);
#pragma unroll
              for (int b = 0; b < kKeys; ++b) {
                const uint32_t a8 = ka[b][c] >> 8, b8 = kb[b][c] >> 8;
                mma(acc[b], a8 & 0x000f000fu, b8 & 0x000f000fu, a8 & 0x00f000f0u, b8 & 0x00f000f0u,
                    qf[c][2], qf[c][3], acc[b]);
              }
            }
#pragma unroll
            for (int b = 0; b < kKeys; ++b) {
              const float2 sa = pair(kp[b][0][u]), sb = pair(kp[b][1][u]);
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const float2 sm = i < 2 ? sa : sb;
                const float mq = u ? fmaf(sm.y, qs[u][i & 1], p[h + b][i]) : sm.y * qs[u][i & 1];
                p[h + b][i] = fmaf(sm.x, acc[b][i], mq);
              }
            }
          }
        }
        if (REP > 1) {
#pragma unroll
          for (int b = 0; b < kTile; ++b)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              if (REP == 4) p[b][i] += __shfl_xor_sync(0xffffffffu, p[b][i], 1);
              p[b][i] += __shfl_xor_sync(0xffffffffu, p[b][i], 2);
            }
        }
      }
      if (left < kTile * kKv4Page) {
#pragma unroll
        for (int b = 0; b < kTile; ++b) {
          if (b * kKv4Page + row >= left) p[b][0] = p[b][1] = -INFINITY;
          if (b * kKv4Page + row + 8 >= left) p[b][2] = p[b][3] = -INFINITY;
        }
      }
      // ---- the largest scale of the tile's values
      float up, down;  // 2^k with s 2^k < 2^14, and 2^-k
      {
        __half2 big = __half2half2(__ushort_as_half(0));
#pragma unroll
        for (int b = 0; b < kTile; ++b) {
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            uint32_t vp[NP];
            own_pairs<NP, REP>(vp, at[b] + 16 * D + ((kKv4Page + row + 8 * y) * NG + rep) * 4);
#pragma unroll
            for (int u = 0; u < NP; ++u)
              big = __hmax2(big, __habs2(*reinterpret_cast<__half2*>(&vp[u])));
          }
        }
#pragma unroll
        for (int o = REP == 1 ? 4 : 4 / REP; o < 32; o <<= 1)
          big = __hmax2(big, __shfl_xor_sync(0xffffffffu, big, o));
        const int e = __float_as_int(__low2float(big)) >> 23;
        up = e == 0 || e == 255 ? 1.f : __int_as_float((267 - e) << 23);
        down = e == 0 || e == 255 ? 1.f : __int_as_float((e - 13) << 23);
      }
      // ---- running maximum and sum; p becomes 2^k times the weight
      const float lift = (float)((__float_as_int(up) >> 23) - 127);
      float2 alpha, base, scale;  // base: minus the maxima
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float mx = top[i];
#pragma unroll
        for (int b = 0; b < kTile; ++b) mx = max3(mx, p[b][i], p[b][i + 2]);
        mx = rows_max(mx);
        const float f = fminf(F[i] * 0x1p24f, FLT_MAX), m = mx == -INFINITY ? 0.f : -mx;
        (i ? alpha.y : alpha.x) = ex2((top[i] + m) * f);
        (i ? base.y : base.x) = m;
        (i ? scale.y : scale.x) = f;
        top[i] = mx;
      }
      // The maximum is taken away before the scale, so the largest weight is 2^k exactly,
      // whatever the size of the scores.
      float2 s = make_float2(0.f, 0.f);
#pragma unroll
      for (int b = 0; b < kTile; ++b)
#pragma unroll
        for (int y = 0; y < 4; y += 2) {
          const float2 x = fma2(add2(make_float2(p[b][y], p[b][y + 1]), base), scale,
                                make_float2(lift, lift));
          p[b][y] = ex2(x.x);
          p[b][y + 1] = ex2(x.y);
          s = add2(s, make_float2(p[b][y], p[b][y + 1]));
        }
      l = fma2(l, alpha, mul2(s, make_float2(down, down)));
      // ---- O: where a maximum moved, what is there is scaled first
      if (__any_sync(0xffffffffu, alpha.x != 1.f || alpha.y != 1.f)) {
#pragma unroll
        for (int c = 0; c < NC / REP; ++c)
#pragma unroll
          for (int i = 0; i < 4; ++i) O[c][i] = mul2(O[c][i], alpha);
#pragma unroll
        for (int u = 0; u < NP; ++u) pm[u] = mul2(pm[u], alpha);
      }
      const float2 c24 = make_float2(down * 0x1p24f, down * 0x1p24f);
      const float2 c20 = make_float2(down * 0x1p20f, down * 0x1p20f);
#pragma unroll
      for (int u = 0; u < NP; ++u) {
        uint32_t wt[kTile][2];
        float2 pmt = make_float2(0.f, 0.f);
        float off[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int b = 0; b < kTile; ++b) {
          uint32_t va[1], vb[1];
          lds<1>(va, at[b] + 16 * D + ((kKv4Page + row) * NG + u * REP + rep) * 4);
          lds<1>(vb, at[b] + 16 * D + ((kKv4Page + row + 8) * NG + u * REP + rep) * 4);
          const float2 sa = pair(va[0]), sb = pair(vb[0]);
          const float ma = fmaf(8.f, sa.x, sa.y), mb = fmaf(8.f, sb.x, sb.y);
          pmt.x = fmaf(p[b][0], ma, fmaf(p[b][2], mb, pmt.x));
          pmt.y = fmaf(p[b][1], ma, fmaf(p[b][3], mb, pmt.y));
          wt[b][0] = transpose8x8(f16x2(p[b][0] * sa.x, p[b][1] * sa.x));
          wt[b][1] = transpose8x8(f16x2(p[b][2] * sb.x, p[b][3] * sb.x));
        }
        // every row of `off` is the sum of the tile's rounded weights times -8 / 8: it
        // counts in each of the eight lanes that hold a part of pm
#pragma unroll
        for (int b = 0; b < kTile; ++b)
          mma(off, 0xbc00bc00u, 0xbc00bc00u, 0xbc00bc00u, 0xbc00bc00u, wt[b][0], wt[b][1], off);
        // Chunks c0 .. of each of the pass's groups; a column's own group counts. Rows
        // `row` take whole bytes n0 + 16 n1, rows `row` + 8 the codes 16 n1 in them; n0
        // is the difference.
#pragma unroll
        for (int c0 = 0; c0 < CG; c0 += kPart) {
          float acc[REP * kPart][2][4], zero[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int b = 0; b < kTile; ++b) {
#pragma unroll
            for (int y = 0; y < REP; ++y) {
              const int chunk = (u * REP + y) * CG + c0;
              uint32_t va[kPart], vb[kPart];
              lds<kPart>(va, at[b] + 8 * D + lane * (D / 8) + chunk * 4);
              lds<kPart>(vb, at[b] + 12 * D + lane * (D / 8) + chunk * 4);
#pragma unroll
              for (int c = 0; c < kPart; ++c) {
                float(&lo)[4] = acc[y * kPart + c][0], (&hi)[4] = acc[y * kPart + c][1];
                mma(lo, va[c] & 0x00ff00ffu, va[c] & 0x00f000f0u, vb[c] & 0x00ff00ffu,
                    vb[c] & 0x00f000f0u, wt[b][0], wt[b][1], b ? lo : zero);
                const uint32_t a8 = high_bytes(va[c]), b8 = high_bytes(vb[c]);
                mma(hi, a8, a8 & 0x00f000f0u, b8, b8 & 0x00f000f0u, wt[b][0], wt[b][1],
                    b ? hi : zero);
              }
            }
          }
#pragma unroll
          for (int c = 0; c < kPart; ++c)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              float2 a[2];
#pragma unroll
              for (int k = 0; k < 2; ++k) {
                a[k] = make_float2(acc[c][i][2 * k], acc[c][i][2 * k + 1]);
#pragma unroll
                for (int y = 1; y < REP; ++y) {
                  a[k].x = rep == y ? acc[y][i][2 * k] : a[k].x;
                  a[k].y = rep == y ? acc[y][i][2 * k + 1] : a[k].y;
                }
              }
              a[0] = fma2(a[1], make_float2(-1.f, -1.f), a[0]);
              float2(&o)[4] = O[u * CG + c0 + c];
              o[2 * i] = fma2(a[0], c24, o[2 * i]);
              o[2 * i + 1] = fma2(a[1], c20, o[2 * i + 1]);
            }
        }
        pmt = make_float2(pmt.x + off[0], pmt.y + off[1]);
        pm[u] = fma2(pmt, make_float2(down, down), pm[u]);
      }
      __syncwarp();
      issue(nb);
      slot += nb;
      if (slot >= kSlots) {
        slot -= kSlots;
        phase ^= 1;
      }
    }

    // ---- the piece is done
    l.x = rows_sum(l.x);
    l.y = rows_sum(l.y);
#pragma unroll
    for (int u = 0; u < NP; ++u) {
      pm[u].x = rows_sum(pm[u].x);
      pm[u].y = rows_sum(pm[u].y);
    }
#pragma unroll
    for (int c = 0; c < NC / REP; ++c)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        O[c][i].x += pm[c / CG].x;
        O[c][i].y += pm[c / CG].y;
      }
    // where chunk c of O lies among the head's channels
    const auto channel = [&](int c) { return 32 * ((c / CG * REP + rep) * CG + c % CG) + 4 * row; };
    if (__any_sync(0xffffffffu, bad)) {  // a bad page id, somewhere: in this piece?
      bool here = false;
      for (int i = lane; i < n; i += 32) {
        const int page = __ldg(P.table + (long long)seg.r * P.table_stride + seg.blk + i);
        here |= page < 0 || page >= P.pool_blocks;
      }
      if (__any_sync(0xffffffffu, here)) l.x = l.y = __int_as_float(0x7fffffff);
    }
    if (failed) l.x = l.y = __int_as_float(0x7fffffff);
    const auto score = [&](int i) { return top[i] * 0x1p24f * (F[i] * kLn2); };  // the largest
    const bool starts = seg.blk == 0, ends = seg.blk + n == seg.nblk;
    if (starts && ends) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int g = head0 + i;
        if (g >= G) continue;
        const float sum = i ? l.y : l.x, inv = 1.f / sum;
#pragma unroll
        for (int c = 0; c < NC / REP; ++c) {
          const auto at = [&](int k) { return (i ? O[c][k].y : O[c][k].x) * inv; };
          uint2 v;
          v.x = float_to_row2<FP16>(at(0), at(1));
          v.y = float_to_row2<FP16>(at(2), at(3));
          *reinterpret_cast<uint2*>(P.o + (orow + g) * D + channel(c)) = v;
        }
        if (row == 0 && rep == 0) P.lse[orow + g] = score(i) + logf(sum);
      }
    } else {
      // the warp's last piece lies over its ring, one before others in the workspace
      const int at = starts ? 1 : 0, final = x + n == xe;
      if (final) __syncwarp();
      float* part = final ? reinterpret_cast<float*>(ring) : ws + (2 + w) * part_stride;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int g = head0 + i;
        if (g >= G) continue;
#pragma unroll
        for (int c = 0; c < NC / REP; ++c)
          *reinterpret_cast<float4*>(part + g * D + channel(c)) =
              i ? make_float4(O[c][0].y, O[c][1].y, O[c][2].y, O[c][3].y)
                : make_float4(O[c][0].x, O[c][1].x, O[c][2].x, O[c][3].x);
        if (row == 0 && rep == 0) {
          float* m2 = ml + ((w * 2 + at) * kMaxG + g) * 2;
          m2[0] = score(i);
          m2[1] = i ? l.y : l.x;
        }
      }
      if (lane == 0) {
        meta[w].has[at] = 1;
        if (!at) {
          meta[w].ends0 = ends;
          meta[w].final0 = final;
        }
        meta[w].r[at] = seg.r;
        meta[w].h[at] = seg.h;
      }
    }
    x += n;
  }
  __syncthreads();

  // ------------------------------------------------ join the warps' pieces
  // A run is a piece that begins a segment (or goes on from the CTA before) and
  // the pieces [0] of the warps behind it up to the segment's end. The warps of
  // a run join it together, each a share of its channels.
  const bool is_warp = lane < kWarps;
  const uint32_t has0 = __ballot_sync(0xffffffffu, is_warp && meta[lane].has[0]);
  const uint32_t has1 = __ballot_sync(0xffffffffu, is_warp && meta[lane].has[1]);
  const uint32_t ends0 = __ballot_sync(0xffffffffu, is_warp && meta[lane].has[0] && meta[lane].ends0);
  const auto piece_of = [&](int y, int at) {
    return at || meta[y].final0 ? reinterpret_cast<const float*>(smem + y * S::kRing)
                                : ws + (2 + y) * part_stride;
  };
#pragma unroll
  for (int at = 0; at < 2; ++at) {
    if (!((at ? has1 : has0) >> w & 1)) continue;
    const uint32_t below = has1 & ((1u << w) - 1);
    const int from = at ? w : below ? 31 - __clz(below) : __ffs(has0) - 1;
    const int from_at = at || below ? 1 : 0;
    const uint32_t done = ends0 >> w >> at << at << w;  // ends at this warp (at = 0) or behind it
    const bool ends = done != 0, starts = from_at == 1;
    const uint32_t reach = has0 & ~((2u << from) - 1);
    const int to = ends ? __ffs(done) - 1 : reach ? 31 - __clz(reach) : from;
    // (a CTA of few blocks has warps without any among them)
    const uint32_t members = (1u << from) | (reach & ((2u << to) - 1));
    const int r = meta[w].r[at], h = meta[w].h[at];
    float* gp = ws + (starts ? 1 : 0) * part_stride;
    for (int i = __popc(members & ((1u << w) - 1)) * 32 + lane; i < G * D / 4;
         i += __popc(members) * 32) {
      const int g = i / (D / 4);
      float mx = -INFINITY;
      for (uint32_t m = members; m; m &= m - 1) {
        const int y = __ffs(m) - 1;
        mx = fmaxf(mx, ml[((y * 2 + (y == from ? from_at : 0)) * kMaxG + g) * 2]);
      }
      const float base = mx == -INFINITY ? 0.f : mx;
      float sum = 0.f;
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
      for (uint32_t m = members; m; m &= m - 1) {
        const int y = __ffs(m) - 1, y_at = y == from ? from_at : 0;
        const float* m2 = ml + ((y * 2 + y_at) * kMaxG + g) * 2;
        const float e = ex2((m2[0] - base) * kLog2e);
        const float4 v = reinterpret_cast<const float4*>(piece_of(y, y_at))[i];
        sum = fmaf(m2[1], e, sum);
        acc.x = fmaf(v.x, e, acc.x);
        acc.y = fmaf(v.y, e, acc.y);
        acc.z = fmaf(v.z, e, acc.z);
        acc.w = fmaf(v.w, e, acc.w);
      }
      if (starts && ends) {
        const long long orow = (long long)r * P.H + (long long)h * G + g;
        const float inv = 1.f / sum;
        uint2 v;
        v.x = float_to_row2<FP16>(acc.x * inv, acc.y * inv);
        v.y = float_to_row2<FP16>(acc.z * inv, acc.w * inv);
        *reinterpret_cast<uint2*>(P.o + orow * D + i % (D / 4) * 4) = v;
        if (i % (D / 4) == 0) P.lse[orow] = mx + logf(sum);
      } else {
        reinterpret_cast<float4*>(gp)[i] = acc;
        if (i % (D / 4) == 0)
          *reinterpret_cast<float2*>(gp + G * D + 2 * g) = make_float2(mx, sum);
      }
    }
  }

  // ------------------------------------------------ join the CTAs' parts
  // Thread 0 announces the head part, thread 32 the tail part. The barrier
  // orders the CTA's writes before the announcement that releases them.
  __syncthreads();
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    if (tid != k * 32) continue;
    const Shared m = out[k];
    int last = 0;
    if (m.c1 > m.c0) {
      int before;
      asm volatile("atom.acq_rel.gpu.global.add.s32 %0, [%1], 1;"
                   : "=r"(before)
                   : "l"(P.counters + m.c0)
                   : "memory");
      last = before == m.c1 - m.c0;
      if (last) P.counters[m.c0] = 0;  // as the next call finds it
    }
    misc[k] = last;
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    if (!misc[k]) continue;
    const Shared m = out[k];
    for (int i = tid; i < G * D / 4; i += kThreads) {
      const int g = i / (D / 4);
      float mx = -INFINITY, sum = 0.f;
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
      for (int c = m.c0; c <= m.c1; ++c) {
        const float* part =
            P.part + ((long long)c * (2 + kWarps) + (c == m.c0 ? 1 : 0)) * part_stride;
        const float2 m2 = __ldcg(reinterpret_cast<const float2*>(part + G * D + 2 * g));
        const float4 v = __ldcg(reinterpret_cast<const float4*>(part) + i);
        const float top = fmaxf(mx, m2.x), base = top == -INFINITY ? 0.f : top;
        const float e0 = ex2((mx - base) * kLog2e), e = ex2((m2.x - base) * kLog2e);
        mx = top;
        sum = fmaf(m2.y, e, sum * e0);
        acc.x = fmaf(v.x, e, acc.x * e0);
        acc.y = fmaf(v.y, e, acc.y * e0);
        acc.z = fmaf(v.z, e, acc.z * e0);
        acc.w = fmaf(v.w, e, acc.w * e0);
      }
      const long long orow = (long long)m.r * P.H + (long long)m.h * G + g;
      const float inv = 1.f / sum;
      uint2 v;
      v.x = float_to_row2<FP16>(acc.x * inv, acc.y * inv);
      v.y = float_to_row2<FP16>(acc.z * inv, acc.w * inv);
      *reinterpret_cast<uint2*>(P.o + orow * D + i % (D / 4) * 4) = v;
      if (i % (D / 4) == 0) P.lse[orow] = mx + logf(sum);
    }
  }
}

using Kernel = void (*)(const Kv4Decode);

struct Choice {
  Kernel kernel;
  int (*smem)(int reqs);
};

template <int D, int GROUP, int REP>
Choice of(int dtype) {
  return {dtype ? kv4_decode_kernel<D, GROUP, true, REP> : kv4_decode_kernel<D, GROUP, false, REP>,
          Shape<D, GROUP>::smem};
}

// As many replicas as there is room for beside the heads, at most one a group.
template <int D, int GROUP>
Choice choose_rep(int dtype, int G) {
  constexpr int NG = D / GROUP;
  if constexpr (NG >= 4)
    if (G <= 2) return of<D, GROUP, 4>(dtype);
  if constexpr (NG >= 2)
    if (G <= 4) return of<D, GROUP, 2>(dtype);
  return of<D, GROUP, 1>(dtype);
}

Choice choose(int D, int group, int dtype, int G) {
  if (D == 64) return group == 32 ? choose_rep<64, 32>(dtype, G) : choose_rep<64, 64>(dtype, G);
  if (group == 32) return choose_rep<128, 32>(dtype, G);
  return group == 64 ? choose_rep<128, 64>(dtype, G) : choose_rep<128, 128>(dtype, G);
}

}  // namespace

cudaError_t launch_kv4_decode(const Kv4Decode& P, int D, int group, int dtype, cudaStream_t s) {
  const Choice c = choose(D, group, dtype, P.G);
  // no more CTAs than the tables could give work to
  const long long most = (long long)P.num_reqs * P.table_stride * P.Hk;
  const int grid = std::max(kv4_workers(most, P.grid, kLeast),
                            (int)std::min((long long)P.num_reqs * P.Hk, (long long)P.grid));
  c.kernel<<<grid, kThreads, c.smem(P.num_reqs), s>>>(P);
  return cudaGetLastError();
}

cudaError_t kv4_decode_init(int D, int group, int dtype, int G, int max_reqs, int* ctas_per_sm,
                            size_t* part_floats) {
  const Choice c = choose(D, group, dtype, G);
  const int bytes = c.smem(max_reqs);
  *part_floats = (2 + kWarps) * ((size_t)G * D + 2 * kMaxG);
  cudaError_t e = cudaFuncSetAttribute(c.kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       c.smem(kKv4MaxReqs));
  if (e != cudaSuccess) return e;
  return cudaOccupancyMaxActiveBlocksPerMultiprocessor(ctas_per_sm, c.kernel, kThreads, bytes);
}

}  // namespace pod
