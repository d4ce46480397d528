// kv4_harness.cpp -- the argument checks of the 4-bit KV cache without a GPU.
//
// Test infrastructure: includes the library's API translation unit, with
// launchers that only count, and hands out a context made without a device.
// A call that passes its checks then ends at the device (POD_ECUDA where there
// is none) or at a counting launcher.
#include "pod_kv4_api.cpp"
#include "pod_kv4_split.h"

static int g_launches = 0;

namespace pod {
cudaError_t launch_qk_norm_rope(const QkParams&, int, int, int, cudaStream_t) { ++g_launches; return cudaSuccess; }
cudaError_t launch_kv4_write(const Kv4Rows&, int, int, int, cudaStream_t) { ++g_launches; return cudaSuccess; }
cudaError_t launch_kv4_read(const Kv4Rows&, int, int, int, cudaStream_t) { ++g_launches; return cudaSuccess; }
cudaError_t launch_kv4_decode(const Kv4Decode&, int, int, int, cudaStream_t) { ++g_launches; return cudaSuccess; }
cudaError_t kv4_decode_init(int, int, int, int, int, int*, size_t*) { return cudaErrorNotSupported; }
}  // namespace pod

extern "C" {
POD_API int harness_launches() { return g_launches; }
POD_API pod_kv4_ctx* harness_ctx(const pod_kv4_config* cfg) {
  pod_kv4_ctx* c = new pod_kv4_ctx();
  c->cfg = *cfg;
  return c;
}
POD_API long long harness_begin(long long V, int N, int c) { return kv4_begin(V, N, c); }
POD_API int harness_cost(int n) { return kv4_cost(n); }
POD_API int harness_workers(long long W, int ctas, int least) { return kv4_workers(W, ctas, least); }
POD_API long long harness_snap(const int* cost, int R, int Hk, long long v) { return kv4_snap(cost, R, Hk, v); }
POD_API long long harness_cut(const int* first, const int* cost, int R, int Hk, long long v) { return kv4_cut(first, cost, R, Hk, v); }
POD_API int harness_worker(const int* cost, int R, int Hk, int N, int r, int h, int blk) { return kv4_worker(cost, R, Hk, N, r, h, blk); }
POD_API void harness_place(const int* first, int R, int Hk, long long x, int* out) {
  const Kv4Place p = kv4_place(first, R, Hk, x);
  out[0] = p.r; out[1] = p.h; out[2] = p.blk; out[3] = p.nblk;
}
POD_API void harness_free(pod_kv4_ctx* c) { delete c; }
}
