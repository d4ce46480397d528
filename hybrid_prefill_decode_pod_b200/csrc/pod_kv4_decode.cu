// pod_kv4_decode.cu -- single-token GQA attention over the 4-bit KV cache.
#include "pod_kv4.cuh"

namespace pod {
namespace {

constexpr int kWarps = 8;
constexpr int kMaxG = 8;

// One CTA for each (request, KV head); each warp takes every eighth token with
// its own running maximum and sum, which are joined through shared memory.
template <int D, int GROUP, bool FP16>
__global__ void __launch_bounds__(kWarps * 32) kv4_decode_kernel(const Kv4Decode P) {
  constexpr int kCh = D / 32, NG = D / GROUP, kRec = kv4_record_bytes(D, GROUP);
  __shared__ float so[kWarps][kMaxG][D];
  __shared__ float sm[kWarps][kMaxG], sl[kWarps][kMaxG];
  const int r = blockIdx.x, h = blockIdx.y, w = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long long cap = (long long)P.table_stride * kKv4Page;
  const int len = (int)min((long long)max(P.ctx_lens[r], 0), cap);
  float q[kMaxG][kCh], o[kMaxG][kCh], mx[kMaxG], l[kMaxG];
#pragma unroll
  for (int g = 0; g < kMaxG; ++g) {
    mx[g] = -INFINITY;
    l[g] = 0.f;
#pragma unroll
    for (int c = 0; c < kCh; ++c) {
      o[g][c] = 0.f;
      const int ch = 32 * c + lane;
      q[g][c] = 0.f;
      if (g < P.G) {
        const float2 f = row2_to_float<FP16>(
            P.q[((long long)r * P.H + h * P.G + g) * D + ch]);
        q[g][c] = f.x;
      }
    }
  }
  for (int t = w; t < len; t += kWarps) {
    const int page = __ldg(P.table + (long long)r * P.table_stride + (t >> 4)), tt = t & 15;
    const bool good = page >= 0 && page < P.pool_blocks;
    const unsigned char* rec = P.pool + ((long long)(good ? page : 0) * P.Hk + h) * kRec;
    float k[kCh], v[kCh];
#pragma unroll
    for (int c = 0; c < kCh; ++c) {
      const int ch = 32 * c + lane;
      const int kb = rec[k_code_byte<D>(tt, ch >> 3) + ((ch & 7) >> 1)] >> (4 * (ch & 1)) & 15;
      const int vb = rec[v_code_byte<D>(tt, ch >> 2) + ((ch & 3) >> 1)] >> (4 * (ch & 1)) & 15;
      const __half2 kp = *reinterpret_cast<const __half2*>(rec + pair_byte<D>(0, tt, ch / GROUP, NG));
      const __half2 vp = *reinterpret_cast<const __half2*>(rec + pair_byte<D>(1, tt, ch / GROUP, NG));
      k[c] = fmaf((float)kb, __low2float(kp), __high2float(kp));
      v[c] = fmaf((float)vb, __low2float(vp), __high2float(vp));
      if (!good) k[c] = v[c] = __int_as_float(0x7fffffff);
    }
#pragma unroll
    for (int g = 0; g < kMaxG; ++g) {
      if (g >= P.G) break;
      float s = 0.f;
#pragma unroll
      for (int c = 0; c < kCh; ++c) s = fmaf(q[g][c], k[c], s);
#pragma unroll
      for (int x = 16; x; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
      s *= P.scale_log2;
      const float top = fmaxf(mx[g], s), base = top == -INFINITY ? 0.f : top;
      const float a = exp2f(mx[g] - base), p = exp2f(s - base);
      mx[g] = top;
      l[g] = l[g] * a + p;
#pragma unroll
      for (int c = 0; c < kCh; ++c) o[g][c] = o[g][c] * a + p * v[c];
    }
  }
#pragma unroll
  for (int g = 0; g < kMaxG; ++g) {
    sm[w][g] = mx[g];
    sl[w][g] = l[g];
#pragma unroll
    for (int c = 0; c < kCh; ++c) so[w][g][32 * c + lane] = o[g][c];
  }
  __syncthreads();
  for (int i = threadIdx.x; i < P.G * D; i += kWarps * 32) {
    const int g = i / D, ch = i % D;
    float top = -INFINITY;
    for (int x = 0; x < kWarps; ++x) top = fmaxf(top, sm[x][g]);
    const float base = top == -INFINITY ? 0.f : top;
    float sum = 0.f, acc = 0.f;
    for (int x = 0; x < kWarps; ++x) {
      const float a = exp2f(sm[x][g] - base);
      sum += sl[x][g] * a;
      acc += so[x][g][ch] * a;
    }
    const float out = len ? acc / sum : 0.f;
    const long long row = (long long)r * P.H + h * P.G + g;
    P.o[row * D + ch] = (uint16_t)float_to_row2<FP16>(out, 0.f);
    if (ch == 0) P.lse[row] = len ? top * 0.69314718055994531f + logf(sum) : -INFINITY;
  }
}

template <int D, int GROUP>
cudaError_t decode_of(const Kv4Decode& P, int dtype, cudaStream_t s) {
  const dim3 grid(P.num_reqs, P.Hk);
  if (dtype)
    kv4_decode_kernel<D, GROUP, true><<<grid, kWarps * 32, 0, s>>>(P);
  else
    kv4_decode_kernel<D, GROUP, false><<<grid, kWarps * 32, 0, s>>>(P);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_kv4_decode(const Kv4Decode& P, int D, int group, int dtype, cudaStream_t s) {
  if (D == 64)
    return group == 32 ? decode_of<64, 32>(P, dtype, s) : decode_of<64, 64>(P, dtype, s);
  if (group == 32) return decode_of<128, 32>(P, dtype, s);
  return group == 64 ? decode_of<128, 64>(P, dtype, s) : decode_of<128, 128>(P, dtype, s);
}

cudaError_t kv4_decode_init(int, int, int, int, int* ctas_per_sm, size_t* part_floats) {
  *ctas_per_sm = 1;
  *part_floats = 0;
  return cudaSuccess;
}

}  // namespace pod
