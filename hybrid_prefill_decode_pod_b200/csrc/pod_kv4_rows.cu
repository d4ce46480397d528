// pod_kv4_rows.cu -- the row operators around the 4-bit KV cache: per-head RMS
// norm with rotation, quantising rows into the cache, and reading them back.
// All three are bound by memory: a lane handles eight adjacent channels of one
// head's row (16 bytes), D / 8 lanes share a row.
#include "pod_kv4.cuh"

namespace pod {
namespace {

constexpr int kThreads = 256;

template <int D>
__device__ __forceinline__ float row_sum(float x) {
#pragma unroll
  for (int o = D / 16; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// y = x / sqrt(mean(x^2) + eps) * w, then the rotation, rounded once. The lane
// that holds a channel's partner (rot / 2 channels away) sends its unrounded
// values by shuffle.
template <int D, bool FP16, bool INTERLEAVED>
__global__ void __launch_bounds__(kThreads) norm_rope_kernel(const QkParams P) {
  constexpr int kLanes = D / 8;
  const int lane = threadIdx.x & 31, l = lane % kLanes;
  const int heads = P.heads[0] + P.heads[1];
  const long long total = (long long)P.num_rows * heads;
  const long long item0 = ((long long)blockIdx.x * kThreads + threadIdx.x) / kLanes;
  const bool in_range = item0 < total;
  const long long item = in_range ? item0 : total - 1;
  const int row = (int)(item / heads), hh = (int)(item % heads);
  const int side = hh >= P.heads[0], h = side ? hh - P.heads[0] : hh;
  const int pos = __ldg(P.positions + row);
  const bool live = in_range && pos >= 0;

  uint4 raw = make_uint4(0, 0, 0, 0);
  if (live)
    raw = *reinterpret_cast<const uint4*>(P.in[side] + row * P.in_row[side] + h * P.in_head[side] +
                                          8 * l);
  float x[8];
  const uint32_t rw[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = row2_to_float<FP16>(rw[i]);
    x[2 * i] = f.x;
    x[2 * i + 1] = f.y;
  }
  float ss = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) ss = fmaf(x[i], x[i], ss);
  ss = row_sum<D>(ss);
  if (P.weight[side]) {
    const float inv = 1.0f / sqrtf(ss * (1.0f / D) + P.eps);
    const uint4 wv = __ldg(reinterpret_cast<const uint4*>(P.weight[side] + 8 * l));
    const uint32_t ww[4] = {wv.x, wv.y, wv.z, wv.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = row2_to_float<FP16>(ww[i]);
      x[2 * i] = x[2 * i] * inv * f.x;
      x[2 * i + 1] = x[2 * i + 1] * inv * f.y;
    }
  }
  const int half = P.rot / 2;
  const bool rotated = 8 * l < P.rot;
  const bool angle = pos < P.max_position;
  const float* cs = P.cos_sin + (long long)(live && angle ? pos : 0) * P.rot;
  if constexpr (INTERLEAVED) {
    if (rotated && live && angle) {
      const float4 c = __ldg(reinterpret_cast<const float4*>(cs + 4 * l));
      const float4 s = __ldg(reinterpret_cast<const float4*>(cs + half + 4 * l));
      const float cc[4] = {c.x, c.y, c.z, c.w}, sn[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float a = x[2 * i], b = x[2 * i + 1];
        x[2 * i] = a * cc[i] - b * sn[i];
        x[2 * i + 1] = a * sn[i] + b * cc[i];
      }
    }
  } else {
    const bool first = 8 * l < half;
    const int partner = rotated ? (first ? lane + half / 8 : lane - half / 8) : lane;
    float y[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = __shfl_sync(0xffffffffu, x[i], partner);
    if (rotated && live && angle) {
      const int at = first ? 8 * l : 8 * l - half;
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const float4 c = __ldg(reinterpret_cast<const float4*>(cs + at + 4 * q));
        const float4 s = __ldg(reinterpret_cast<const float4*>(cs + half + at + 4 * q));
        const float cc[4] = {c.x, c.y, c.z, c.w}, sn[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int k = 4 * q + i;
          x[k] = x[k] * cc[i] + (first ? -y[k] : y[k]) * sn[i];
        }
      }
    }
  }
  if (!live) return;
  if (!angle) {
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = __int_as_float(0x7fffffff);
  }
  uint4 out;
  out.x = float_to_row2<FP16>(x[0], x[1]);
  out.y = float_to_row2<FP16>(x[2], x[3]);
  out.z = float_to_row2<FP16>(x[4], x[5]);
  out.w = float_to_row2<FP16>(x[6], x[7]);
  *reinterpret_cast<uint4*>(P.out[side] + row * P.out_row[side] + h * P.out_head[side] + 8 * l) = out;
}

// A row's token and head: item = (row, K or V, head).
struct Place {
  int row, kv, h;
  bool live;  // the row belongs to a request
  long long pos;
  unsigned char* rec;
};

template <int D>
__device__ __forceinline__ Place place_of(const Kv4Rows& P, int rec_bytes) {
  const int per_row = 2 * P.Hk;
  const long long total = (long long)P.num_rows * per_row;
  const long long item0 = ((long long)blockIdx.x * kThreads + threadIdx.x) / (D / 8);
  const long long item = item0 < total ? item0 : total - 1;
  Place p;
  p.row = (int)(item / per_row);
  const int sub = (int)(item % per_row);
  p.kv = sub >= P.Hk;
  p.h = p.kv ? sub - P.Hk : sub;
  const int r = row_request(P.cu_rows, P.num_reqs, p.row);
  p.live = item0 < total && r >= 0;
  p.pos = r >= 0 ? (long long)__ldg(P.start + r) + p.row - __ldg(P.cu_rows + r) : -1;
  p.rec = r >= 0 ? record_of(P, r, p.pos, p.h, rec_bytes) : nullptr;
  return p;
}

template <int D, int GROUP, bool FP16>
__global__ void __launch_bounds__(kThreads) kv4_write_kernel(const Kv4Rows P) {
  constexpr int kLanes = D / 8, NG = D / GROUP;
  const int l = (threadIdx.x & 31) % kLanes;
  const Place p = place_of<D>(P, kv4_record_bytes(D, GROUP));
  const bool live = p.live && p.rec != nullptr;
  uint4 raw = make_uint4(0, 0, 0, 0);
  if (live)
    raw = *reinterpret_cast<const uint4*>(P.x[p.kv] + p.row * P.row[p.kv] + p.h * P.head[p.kv] +
                                          8 * l);
  const uint32_t rw[4] = {raw.x, raw.y, raw.z, raw.w};
  float x[8], lo = 65504.f, hi = -65504.f;
  bool fine = true;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = row2_to_float<FP16>(rw[i]);
    x[2 * i] = f.x;
    x[2 * i + 1] = f.y;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    fine = fine && fabsf(x[i]) < __int_as_float(0x7f800000);
    x[i] = fminf(fmaxf(x[i], -65504.f), 65504.f);
    lo = fminf(lo, x[i]);
    hi = fmaxf(hi, x[i]);
  }
  int ok = fine;
#pragma unroll
  for (int o = GROUP / 16; o; o >>= 1) {
    lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
    hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
    ok &= __shfl_xor_sync(0xffffffffu, ok, o);
  }
  if (!live) return;
  const __half sh = ok ? __float2half_rn((hi - lo) / 15.0f) : __ushort_as_half(0x7fff);
  const __half mh = ok ? __float2half_rn(lo) : __ushort_as_half(0x7fff);
  const float s = __half2float(sh), m = __half2float(mh);
  uint32_t code = 0;
  if (s > 0.f) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      code |= (uint32_t)fminf(fmaxf(rintf((x[i] - m) / s), 0.f), 15.f) << (4 * i);
  }
  const int t = (int)(p.pos & 15);
  if (p.kv == 0) {
    *reinterpret_cast<uint32_t*>(p.rec + k_code_byte<D>(t, l)) = code;
  } else {
    *reinterpret_cast<uint16_t*>(p.rec + v_code_byte<D>(t, 2 * l)) = (uint16_t)code;
    *reinterpret_cast<uint16_t*>(p.rec + v_code_byte<D>(t, 2 * l + 1)) = (uint16_t)(code >> 16);
  }
  if (8 * l % GROUP == 0)
    *reinterpret_cast<__half2*>(p.rec + pair_byte<D>(p.kv, t, 8 * l / GROUP, NG)) =
        __halves2half2(sh, mh);
}

template <int D, int GROUP, bool FP16>
__global__ void __launch_bounds__(kThreads) kv4_read_kernel(const Kv4Rows P) {
  constexpr int kLanes = D / 8, NG = D / GROUP;
  const int l = (threadIdx.x & 31) % kLanes;
  const Place p = place_of<D>(P, kv4_record_bytes(D, GROUP));
  if (!p.live) return;
  float s = __int_as_float(0x7fffffff), m = s;
  uint32_t code = 0;
  if (p.rec) {
    const int t = (int)(p.pos & 15);
    if (p.kv == 0)
      code = *reinterpret_cast<const uint32_t*>(p.rec + k_code_byte<D>(t, l));
    else
      code = *reinterpret_cast<const uint16_t*>(p.rec + v_code_byte<D>(t, 2 * l)) |
             (uint32_t)*reinterpret_cast<const uint16_t*>(p.rec + v_code_byte<D>(t, 2 * l + 1)) << 16;
    const __half2 sm =
        *reinterpret_cast<const __half2*>(p.rec + pair_byte<D>(p.kv, t, 8 * l / GROUP, NG));
    s = __low2float(sm);
    m = __high2float(sm);
  }
  float x[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = fmaf((float)(code >> (4 * i) & 15), s, m);
  uint4 out;
  out.x = float_to_row2<FP16>(x[0], x[1]);
  out.y = float_to_row2<FP16>(x[2], x[3]);
  out.z = float_to_row2<FP16>(x[4], x[5]);
  out.w = float_to_row2<FP16>(x[6], x[7]);
  *reinterpret_cast<uint4*>(P.x[p.kv] + p.row * P.row[p.kv] + p.h * P.head[p.kv] + 8 * l) = out;
}

unsigned blocks_for(long long items, int D) {
  return (unsigned)((items * (D / 8) + kThreads - 1) / kThreads);
}

template <int D, bool FP16>
cudaError_t norm_rope_of(const QkParams& P, int interleaved, cudaStream_t s) {
  const unsigned grid = blocks_for((long long)P.num_rows * (P.heads[0] + P.heads[1]), D);
  if (interleaved)
    norm_rope_kernel<D, FP16, true><<<grid, kThreads, 0, s>>>(P);
  else
    norm_rope_kernel<D, FP16, false><<<grid, kThreads, 0, s>>>(P);
  return cudaGetLastError();
}

template <int D, int GROUP>
cudaError_t rows_of(const Kv4Rows& P, int dtype, bool read, cudaStream_t s) {
  const unsigned grid = blocks_for((long long)P.num_rows * 2 * P.Hk, D);
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
