// pod_kv4_rows.cu -- the row operators around the 4-bit KV cache: per-head RMS
// norm with rotation, quantising rows into the cache, and reading them back.
// All three are bound by memory: a lane handles eight adjacent channels of one
// head's row (16 bytes), D / 8 lanes share a row.
#include <algorithm>

#include "pod_kv4.cuh"

namespace pod {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

template <bool FP16>
__device__ __forceinline__ void unpack8(const uint4& v, float (&x)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = row2_to_float<FP16>(w[i]);
    x[2 * i] = f.x;
    x[2 * i + 1] = f.y;
  }
}
template <bool FP16>
__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
  return make_uint4(float_to_row2<FP16>(x[0], x[1]), float_to_row2<FP16>(x[2], x[3]),
                    float_to_row2<FP16>(x[4], x[5]), float_to_row2<FP16>(x[6], x[7]));
}

// y = x / sqrt(mean(x^2) + eps) * w, then the rotation, rounded once.
//
// A warp takes some heads of one row, 256 / D of them at a time (kBatch loads in
// flight). The angle's cosines and sines belong to the row, so a lane multiplies
// them with its weights once, y_i = inv (x_i a_i + x_partner b_i), and a head
// costs two multiply-adds for each channel. The partner, rot / 2 channels away,
// comes by shuffle as it was read.
//
// 16384 rows of 72 heads of 128: 104 us, 5.9 TB/s, 91 % of the copy rate, with
// 32 warps an SM (64 registers, 16 bytes spilled for fp16 halves); 24 took 115,
// batches of 3 or 6 with 32 115 and 118, of 2 with 40 108, CTAs of 256 threads
// 105.
constexpr int kBatch = 4;
constexpr int kRopeThreads = 128;

template <int D, bool FP16, bool INTERLEAVED>
__global__ void __launch_bounds__(kRopeThreads, 8) norm_rope_kernel(const QkParams P, int parts) {
  constexpr int kLanes = D / 8, kHeads = 32 / kLanes;
  const int lane = threadIdx.x & 31, l = lane % kLanes, sub = lane / kLanes;
  const int unit = blockIdx.x * (kRopeThreads / 32) + (threadIdx.x >> 5);
  const int row = unit / parts, part = unit % parts;
  if (row >= P.num_rows) return;
  const int pos = __ldg(P.positions + row);
  if (pos < 0) return;
  const int half = P.rot / 2;
  const bool rotated = 8 * l < P.rot, first = 8 * l < half;
  const int partner = INTERLEAVED || !rotated ? lane : first ? lane + half / 8 : lane - half / 8;
#pragma unroll
  for (int side = 0; side < 2; ++side) {
    const int n = P.heads[side];
    const int each = (n + parts * kHeads - 1) / (parts * kHeads) * kHeads;
    const int h0 = part * each, h1 = min(n, h0 + each);
    if (h0 >= h1) continue;
    const bool norm = P.weight[side] != nullptr;
    float cs[8], sn[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      cs[i] = 1.f;
      sn[i] = 0.f;
    }
    if (pos >= P.max_position) {
#pragma unroll
      for (int i = 0; i < 8; ++i) cs[i] = __int_as_float(0x7fffffff);
    } else if (rotated) {
      const float* t = P.cos_sin + (long long)pos * P.rot;
      if constexpr (INTERLEAVED) {
        const float4 c = __ldg(reinterpret_cast<const float4*>(t + 4 * l));
        const float4 s = __ldg(reinterpret_cast<const float4*>(t + half + 4 * l));
        const float c4[4] = {c.x, c.y, c.z, c.w}, s4[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          cs[i] = c4[i / 2];
          sn[i] = i & 1 ? s4[i / 2] : -s4[i / 2];
        }
      } else {
        const int at = first ? 8 * l : 8 * l - half;
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          const float4 c = __ldg(reinterpret_cast<const float4*>(t + at + 4 * q));
          const float4 s = __ldg(reinterpret_cast<const float4*>(t + half + at + 4 * q));
          const float c4[4] = {c.x, c.y, c.z, c.w}, s4[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            cs[4 * q + i] = c4[i];
            sn[4 * q + i] = first ? -s4[i] : s4[i];
          }
        }
      }
    }
    float a[8], b[8];
    if (norm) {
      float w[8], wp[8];
      unpack8<FP16>(__ldg(reinterpret_cast<const uint4*>(P.weight[side] + 8 * l)), w);
#pragma unroll
      for (int i = 0; i < 8; ++i)
        wp[i] = INTERLEAVED ? w[i ^ 1] : __shfl_sync(0xffffffffu, w[i], partner);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        a[i] = w[i] * cs[i];
        b[i] = wp[i] * sn[i];
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        a[i] = cs[i];
        b[i] = sn[i];
      }
    }
    const uint16_t* in = P.in[side] + row * P.in_row[side] + 8 * l;
    uint16_t* out = P.out[side] + row * P.out_row[side] + 8 * l;
    for (int h = h0; h < h1; h += kHeads * kBatch) {
      uint4 raw[kBatch];
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        raw[k] = make_uint4(0, 0, 0, 0);
        const int hh = h + k * kHeads + sub;
        if (hh < h1) raw[k] = *reinterpret_cast<const uint4*>(in + hh * P.in_head[side]);
      }
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        const int hh = h + k * kHeads + sub;
        float x[8], y[8];
        unpack8<FP16>(raw[k], x);
        float inv = 1.f;
        if (norm) {
          float ss = 0.f;
#pragma unroll
          for (int i = 0; i < 8; ++i) ss = fmaf(x[i], x[i], ss);
#pragma unroll
          for (int o = kLanes / 2; o; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
          inv = rsqrtf(fmaf(ss, 1.0f / D, P.eps));
        }
        if constexpr (INTERLEAVED) {
#pragma unroll
          for (int i = 0; i < 8; ++i) y[i] = x[i ^ 1];
        } else {
          uint4 p;
          p.x = __shfl_sync(0xffffffffu, raw[k].x, partner);
          p.y = __shfl_sync(0xffffffffu, raw[k].y, partner);
          p.z = __shfl_sync(0xffffffffu, raw[k].z, partner);
          p.w = __shfl_sync(0xffffffffu, raw[k].w, partner);
          unpack8<FP16>(p, y);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float z = x[i] * a[i];
          x[i] = (rotated ? fmaf(y[i], b[i], z) : z) * inv;
        }
        if (hh < h1) *reinterpret_cast<uint4*>(out + hh * P.out_head[side]) = pack8<FP16>(x);
      }
    }
  }
}

// ------------------------------------------------------------ cache rows
//
// A CTA looks at 16 adjacent rows. Those at which a page begins (or a request's
// first row) stand for the rows of that page that follow, and a warp takes one
// such page of one KV head: up to 16 tokens and one record.

// Row `lane` of the CTA's 16 rows (lanes 0 .. 15).
struct Row {
  int count;           // tokens of its page from here on, 0 where it begins none
  int token;           // its token within the page
  const int* page;     // its table entry, or nullptr outside the table
};

__device__ __forceinline__ Row row_of(const Kv4Rows& P, int row0, int lane) {
  Row out{0, 0, nullptr};
  const int row = row0 + lane;
  // requests of the 16 rows: the first one's, and how many begin behind it
  const int r0 = warp_request(P.cu_rows, P.num_reqs, row0, lane);
  const int next = r0 + 1 + lane <= P.num_reqs ? __ldg(P.cu_rows + r0 + 1 + lane) : INT_MAX;
  int r = r0;
  if (__shfl_sync(0xffffffffu, next, 31) > row0 + 15) {
    int more = 0;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const int n = __popc(__ballot_sync(0xffffffffu, next <= row0 + i));
      if (lane == i) more = n;
    }
    r = r0 + more;
  } else {  // more than 31 requests end here (empty ones among them)
    int hi = P.num_reqs;
    while (hi - r > 1) {
      const int mid = (r + hi) >> 1;
      if (__ldg(P.cu_rows + mid) <= row)
        r = mid;
      else
        hi = mid;
    }
  }
  if (lane < 16 && row < P.num_rows && r < P.num_reqs) {
    const int begin = __ldg(P.cu_rows + r), end = min(__ldg(P.cu_rows + r + 1), P.num_rows);
    if (begin <= row && row < end) {
      const long long pos = (long long)__ldg(P.start + r) + row - begin;
      out.token = (int)(pos & 15);
      if (row == begin || row == 0 || out.token == 0) out.count = min(16 - out.token, end - row);
      if (pos >= 0 && (pos >> 4) < P.table_stride)
        out.page = P.table + (long long)r * P.table_stride + (pos >> 4);
    }
  }
  return out;
}

// Calls f(first row, tokens, first token, page id or -1, head) for each page and
// head of the CTA's rows, one warp each.
template <typename F>
__device__ __forceinline__ void for_pages(const Kv4Rows& P, F f) {
  const int lane = threadIdx.x & 31, row0 = blockIdx.x * 16;
  const Row mine = row_of(P, row0, lane);
  int page = -1;
  if (mine.count && mine.page) {
    page = __ldg(mine.page);
    if (page >= P.pool_blocks) page = -1;
  }
  const uint32_t begins = __ballot_sync(0xffffffffu, mine.count > 0);
  const int rank = mine.count > 0 ? __popc(begins & ((1u << lane) - 1)) : -1;
  const int heads = (P.Hk + gridDim.y - 1) / gridDim.y, h0 = blockIdx.y * heads;
  const int nh = min(heads, P.Hk - h0), units = __popc(begins) * nh;
  for (int u = threadIdx.x >> 5; u < units; u += kWarps) {
    const int i = __ffs(__ballot_sync(0xffffffffu, rank == u / nh)) - 1;
    f(row0 + i, __shfl_sync(0xffffffffu, mine.count, i), __shfl_sync(0xffffffffu, mine.token, i),
      __shfl_sync(0xffffffffu, page, i), h0 + u % nh);
  }
}

// Codes of a lane's eight values, and the pair of their group, which GROUP / 8
// adjacent lanes share (all lanes of the warp call this).
//
// The least and the largest value are taken in the row's own type, two at a
// time: low halves hold least values, high halves the negated largest. A NaN or
// an infinity shows in them. Quotients often lie on the border of two codes
// (short significands), so the product with the approximate reciprocal is
// corrected by one residual step: off by 2^-40 of itself before its rounding, it
// is exact on a border, and elsewhere the nearest fp32 number unless the quotient
// lies that near to the middle of two. Where a value lies
// outside the codes (fp16(lo) may be above lo, and values are cut to fp16's
// range) the lane takes its codes once more, with limits.
struct Quantised {
  uint32_t code;
  __half2 pair;
};

// (rarely taken: one copy for all callers)
template <bool FP16>
__device__ __noinline__ uint32_t limited_codes(uint4 raw, float s, float m) {
  float x[8];
  unpack8<FP16>(raw, x);
  uint32_t code = 0;
  for (int i = 0; i < 8; ++i)
    code |= (uint32_t)rintf(fminf(fmaxf((x[i] - m) / s, 0.f), 15.f)) << (4 * i);
  return code;
}

template <int GROUP, bool FP16>
__device__ __forceinline__ Quantised quantise(const uint4& raw) {
  const uint32_t least = min2<FP16>(min2<FP16>(raw.x, raw.y), min2<FP16>(raw.z, raw.w));
  const uint32_t most =
      max2<FP16>(max2<FP16>(raw.x, raw.y), max2<FP16>(raw.z, raw.w)) ^ 0x80008000u;
  uint32_t ends = min2<FP16>(__byte_perm(least, most, 0x5410), __byte_perm(least, most, 0x7632));
#pragma unroll
  for (int o = GROUP / 16; o; o >>= 1)
    ends = min2<FP16>(ends, __shfl_xor_sync(0xffffffffu, ends, o));
  const float2 e = row2_to_float<FP16>(ends);
  const bool fine = fabsf(e.x) < INFINITY && fabsf(e.y) < INFINITY;
  float lo = e.x, hi = -e.y;
  if (!FP16) {
    lo = fminf(fmaxf(lo, -65504.f), 65504.f);
    hi = fminf(fmaxf(hi, -65504.f), 65504.f);
  }
  // range / 15, rounded correctly: one residual step after the product with the
  // rounded 1 / 15 (Markstein's method)
  const float range = hi - lo, guess = range * (1.f / 15.f);
  const float step = fmaf(fmaf(-guess, 15.f, range), 1.f / 15.f, guess);
  Quantised q;
  const uint32_t nan = 0x7fff7fffu;
  q.pair = fine ? __halves2half2(__float2half_rn(step), __float2half_rn(lo))
                : *reinterpret_cast<const __half2*>(&nan);
  // m + 15 s may round to infinity in fp16 (0 .. 65504: s = 4368): s one step lower does not
  if (FP16 && fmaf(15.f, __low2float(q.pair), __high2float(q.pair)) >= 65520.f)
    *reinterpret_cast<uint32_t*>(&q.pair) -= 1;
  const float s = __low2float(q.pair), m = __high2float(q.pair);
  float inv;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(s));
  const float2 inv2 = make_float2(inv, inv), m2 = make_float2(-m, -m);
  const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
  const float2 s2 = make_float2(-s, -s);
  uint32_t code = 0;
#pragma unroll
  for (int i = 3; i >= 0; --i) {
    const float2 x = add2(row2_to_float<FP16>(w[i]), m2);
    float2 t = mul2(x, inv2);
    t = fma2(fma2(t, s2, x), inv2, t);
    const float2 n = add2(t, make_float2(12582912.f, 12582912.f));  // the integer in the low bits
    code = (code << 4) + __float_as_uint(n.y);
    code = (code << 4) + __float_as_uint(n.x);
  }
  code -= 0x3f400000u;  // the other bits of the eight 12582912 + n
  q.code = code;
  if (!(s > 0.f))
    q.code = 0;
  else if (fmaxf((m - e.x) * inv, (-e.y - m) * inv - 15.f) > 0.4999f)
    q.code = limited_codes<FP16>(raw, s, m);
  return q;
}

// The eight values of a word of codes. A code in the low bits of an fp16 is the
// subnormal n 2^-24 (n 2^-20 one code higher), and s 2^24 is exact.
template <bool FP16>
__device__ __forceinline__ uint4 values(uint32_t code, uint32_t sm) {
  const float2 p = pair(sm);
  const float2 s24 = make_float2(p.x * 0x1p24f, p.x * 0x1p24f);
  const float2 s20 = make_float2(p.x * 0x1p20f, p.x * 0x1p20f), m = make_float2(p.y, p.y);
  const uint32_t up = code >> 8;
  const float2 a = fma2(pair(code & 0x000f000fu), s24, m);  // channels 0 and 4
  const float2 b = fma2(pair(code & 0x00f000f0u), s20, m);
  const float2 c = fma2(pair(up & 0x000f000fu), s24, m);
  const float2 d = fma2(pair(up & 0x00f000f0u), s20, m);
  return make_uint4(float_to_row2<FP16>(a.x, b.x), float_to_row2<FP16>(c.x, d.x),
                    float_to_row2<FP16>(a.y, b.y), float_to_row2<FP16>(c.y, d.y));
}

__device__ __forceinline__ void sts32(uint32_t at, uint32_t v) {
  asm volatile("st.shared.b32 [%0], %1;" ::"r"(at), "r"(v) : "memory");
}
__device__ __forceinline__ void sts16(uint32_t at, uint32_t v) {
  asm volatile("st.shared.b16 [%0], %1;" ::"r"(at), "h"((unsigned short)v) : "memory");
}

// Its floor is the rows' bytes, D bytes of codes for 4 D of K and V. A whole page is
// put together in shared memory, since V's codes of a token lie 16 bytes apart,
// and leaves in 16-byte pieces; part of a page goes to its places directly.
//
// 16384 tokens of 8 heads of 128, kernel alone: 26 us for 85 MB (13 at the copy
// rate). 250 warp instructions for two rows of K and of V each are some 15 us of
// issue slots (65 % in use while CTAs run); the largest stall is the wait for
// memory: a warp has one page, whose first rows wait for the lookup of its request
// and page, and the CTAs make 1.7 waves. Four CTAs an SM (64 registers, 16 to 24
// bytes spilled); five took 3 % more. With the whole page's places
// computed anew for each row, through generic addresses, it took 30.
template <int D, int GROUP, bool FP16>
__global__ void __launch_bounds__(kThreads, 4) kv4_write_kernel(const Kv4Rows P) {
  constexpr int kLanes = D / 8, kRows = 32 / kLanes, NG = D / GROUP;
  constexpr int kRec = kv4_record_bytes(D, GROUP);
  __shared__ __align__(16) unsigned char stage[kWarps][kRec];
  const int lane = threadIdx.x & 31, l = lane % kLanes, sub = lane / kLanes;
  unsigned char* mine = stage[threadIdx.x >> 5];
  for_pages(P, [&](int row, int count, int token, int page, int h) {
    if (page < 0) return;
    unsigned char* rec = P.pool + ((long long)page * P.Hk + h) * kRec;
    const uint16_t* ks = P.x[0] + (row + sub) * P.row[0] + h * P.head[0] + 8 * l;
    const uint16_t* vs = P.x[1] + (row + sub) * P.row[1] + h * P.head[1] + 8 * l;
    const auto load = [&](uint4& k, uint4& v, int i) {
      if (i + sub < count) {
        k = *reinterpret_cast<const uint4*>(ks + i * P.row[0]);
        v = *reinterpret_cast<const uint4*>(vs + i * P.row[1]);
      }
    };
    uint4 k0 = make_uint4(0, 0, 0, 0), v0 = k0, k1 = k0, v1 = k0;  // two steps in flight
    load(k0, v0, 0);
    load(k1, v1, kRows);
    if (count == 16) {
      // where token `sub` goes; i tokens on (i a multiple of kRows) the places
      // differ by constants
      const uint32_t at = smem_u32(mine), k_at = at + k_code_byte<D>(sub, l),
                     v_at = at + v_code_byte<D>(sub, 2 * l),
                     p_at = at + pair_byte<D>(0, sub, 8 * l / GROUP, NG);
      const auto step = [&](int i, const uint4& kr, const uint4& vr) {
        const Quantised kq = quantise<GROUP, FP16>(kr), vq = quantise<GROUP, FP16>(vr);
        const uint32_t v_to = v_at + (32 * (i >> 3) + ((i & 7) >> 1)) * (D / 8);
        sts32(k_at + i * (D / 2), kq.code);
        sts16(v_to, vq.code);
        sts16(v_to + D / 2, vq.code >> 16);
        if (8 * l % GROUP == 0) {
          sts32(p_at + i * NG * 4, *reinterpret_cast<const uint32_t*>(&kq.pair));
          sts32(p_at + (kKv4Page + i) * NG * 4, *reinterpret_cast<const uint32_t*>(&vq.pair));
        }
      };
#pragma unroll 1
      for (int i = 0; i < 16; i += 2 * kRows) {
        step(i, k0, v0);
        load(k0, v0, i + 2 * kRows);
        step(i + kRows, k1, v1);
        load(k1, v1, i + 3 * kRows);
      }
      __syncwarp();
#pragma unroll
      for (int i = 0; i < (kRec + 511) / 512; ++i)
        if (i * 512 + lane * 16 < kRec)
          *reinterpret_cast<uint4*>(rec + i * 512 + lane * 16) =
              *reinterpret_cast<const uint4*>(mine + i * 512 + lane * 16);
      __syncwarp();
      return;
    }
#pragma unroll 1
    for (int i = 0; i < count; i += kRows) {
      const Quantised kq = quantise<GROUP, FP16>(k0), vq = quantise<GROUP, FP16>(v0);
      k0 = k1;
      v0 = v1;
      load(k1, v1, i + 2 * kRows);
      if (i + sub >= count) continue;
      const int t = token + i + sub;
      *reinterpret_cast<uint32_t*>(rec + k_code_byte<D>(t, l)) = kq.code;
      *reinterpret_cast<uint16_t*>(rec + v_code_byte<D>(t, 2 * l)) = (uint16_t)vq.code;
      *reinterpret_cast<uint16_t*>(rec + v_code_byte<D>(t, 2 * l + 1)) = (uint16_t)(vq.code >> 16);
      if (8 * l % GROUP == 0) {
        *reinterpret_cast<__half2*>(rec + pair_byte<D>(0, t, 8 * l / GROUP, NG)) = kq.pair;
        *reinterpret_cast<__half2*>(rec + pair_byte<D>(1, t, 8 * l / GROUP, NG)) = vq.pair;
      }
    }
  });
}

// The reverse: the record comes to shared memory in 16-byte pieces, the rows
// leave in 16 bytes a lane. 16366 tokens of 8 heads of 128, kernel alone: 17 us for
// 86 MB (13 at the copy rate), 1.7 waves of CTAs again; 61 % of the issue slots in
// use, the largest stall again the wait for memory.
template <int D, int GROUP, bool FP16>
__global__ void __launch_bounds__(kThreads) kv4_read_kernel(const Kv4Rows P) {
  constexpr int kLanes = D / 8, kRows = 32 / kLanes, NG = D / GROUP;
  constexpr int kRec = kv4_record_bytes(D, GROUP);
  __shared__ __align__(16) unsigned char stage[kWarps][kRec];
  const int lane = threadIdx.x & 31, l = lane % kLanes, sub = lane / kLanes;
  unsigned char* mine = stage[threadIdx.x >> 5];
  for_pages(P, [&](int row, int count, int token, int page, int h) {
    if (page >= 0) {
      const unsigned char* rec = P.pool + ((long long)page * P.Hk + h) * kRec;
      uint4 v[(kRec + 511) / 512];
#pragma unroll
      for (int i = 0; i < (kRec + 511) / 512; ++i)
        if (i * 512 + lane * 16 < kRec)
          v[i] = __ldg(reinterpret_cast<const uint4*>(rec + i * 512 + lane * 16));
#pragma unroll
      for (int i = 0; i < (kRec + 511) / 512; ++i)
        if (i * 512 + lane * 16 < kRec)
          *reinterpret_cast<uint4*>(mine + i * 512 + lane * 16) = v[i];
    }
    __syncwarp();
    uint16_t* kd = P.x[0] + (row + sub) * P.row[0] + h * P.head[0] + 8 * l;
    uint16_t* vd = P.x[1] + (row + sub) * P.row[1] + h * P.head[1] + 8 * l;
#pragma unroll 8
    for (int i = 0; i + sub < count; i += kRows) {
      const int t = token + i + sub;
      uint32_t kc = 0, vc = 0, kp = 0x7fff7fffu, vp = kp;  // NaN without a place
      if (page >= 0) {
        kc = *reinterpret_cast<const uint32_t*>(mine + k_code_byte<D>(t, l));
        vc = *reinterpret_cast<const uint16_t*>(mine + v_code_byte<D>(t, 2 * l)) |
             (uint32_t)*reinterpret_cast<const uint16_t*>(mine + v_code_byte<D>(t, 2 * l + 1)) << 16;
        kp = *reinterpret_cast<const uint32_t*>(mine + pair_byte<D>(0, t, 8 * l / GROUP, NG));
        vp = *reinterpret_cast<const uint32_t*>(mine + pair_byte<D>(1, t, 8 * l / GROUP, NG));
      }
      *reinterpret_cast<uint4*>(kd + i * P.row[0]) = values<FP16>(kc, kp);
      *reinterpret_cast<uint4*>(vd + i * P.row[1]) = values<FP16>(vc, vp);
    }
    __syncwarp();
  });
}

template <int D, bool FP16>
cudaError_t norm_rope_of(const QkParams& P, int interleaved, cudaStream_t s) {
  // Few rows are cut into parts of one batch of heads at least.
  constexpr int kHeads = 256 / D;
  const int most = std::max(P.heads[0], P.heads[1]);
  const long long want = kKv4Sms * 32;
  long long parts = std::min<long long>((want + P.num_rows - 1) / P.num_rows,
                                        (most + kHeads - 1) / kHeads);
  parts = std::max<long long>(parts, 1);
  constexpr int kUnits = kRopeThreads / 32;
  const unsigned grid = (unsigned)((P.num_rows * parts + kUnits - 1) / kUnits);
  if (interleaved)
    norm_rope_kernel<D, FP16, true><<<grid, kRopeThreads, 0, s>>>(P, (int)parts);
  else
    norm_rope_kernel<D, FP16, false><<<grid, kRopeThreads, 0, s>>>(P, (int)parts);
  return cudaGetLastError();
}

template <int D, int GROUP>
cudaError_t rows_of(const Kv4Rows& P, int dtype, bool read, cudaStream_t s) {
  // With few rows every KV head has CTAs of its own.
  const unsigned windows = (unsigned)((P.num_rows + 15) / 16);
  const dim3 grid(windows, windows >= 2 * kKv4Sms ? (P.Hk + kWarps - 1) / kWarps : P.Hk);
  if (read) {
    if (dtype)
      kv4_read_kernel<D, GROUP, true><<<grid, kThreads, 0, s>>>(P);
    else
      kv4_read_kernel<D, GROUP, false><<<grid, kThreads, 0, s>>>(P);
  } else {
    if (dtype)
      kv4_write_kernel<D, GROUP, true><<<grid, kThreads, 0, s>>>(P);
    else
      kv4_write_kernel<D, GROUP, false><<<grid, kThreads, 0, s>>>(P);
  }
  return cudaGetLastError();
}

cudaError_t rows_any(const Kv4Rows& P, int D, int group, int dtype, bool read, cudaStream_t s) {
  if (D == 64)
    return group == 32 ? rows_of<64, 32>(P, dtype, read, s) : rows_of<64, 64>(P, dtype, read, s);
  if (group == 32) return rows_of<128, 32>(P, dtype, read, s);
  return group == 64 ? rows_of<128, 64>(P, dtype, read, s) : rows_of<128, 128>(P, dtype, read, s);
}

}  // namespace

cudaError_t launch_qk_norm_rope(const QkParams& P, int D, int dtype, int interleaved,
                                cudaStream_t s) {
  if (D == 64)
    return dtype ? norm_rope_of<64, true>(P, interleaved, s)
                 : norm_rope_of<64, false>(P, interleaved, s);
  return dtype ? norm_rope_of<128, true>(P, interleaved, s)
               : norm_rope_of<128, false>(P, interleaved, s);
}

cudaError_t launch_kv4_write(const Kv4Rows& P, int D, int group, int dtype, cudaStream_t s) {
  return rows_any(P, D, group, dtype, false, s);
}
cudaError_t launch_kv4_read(const Kv4Rows& P, int D, int group, int dtype, cudaStream_t s) {
  return rows_any(P, D, group, dtype, true, s);
}

}  // namespace pod
