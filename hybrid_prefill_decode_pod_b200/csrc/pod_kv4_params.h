// pod_kv4_params.h -- kernel parameters and launchers of the 4-bit KV cache.
#pragma once
#include <cuda_runtime.h>

#include <cstdint>

namespace pod {

constexpr int kKv4Page = 16;
constexpr int kKv4MaxReqs = 4096;
constexpr int kKv4Sms = 148;  // of a B200: what the row kernels' grids are shaped for

// Bytes of one (page, KV head) record: 4-bit codes of K and V, then a pair
// (scale, least value) of fp16 for each token and channel group.
__host__ __device__ constexpr int kv4_record_bytes(int D, int group) {
  return kKv4Page * D + 2 * kKv4Page * 4 * (D / group);
}

struct QkParams {
  int heads[2];              // H, Hk
  int num_rows;
  int rot;                   // rotated channels
  const uint16_t* in[2];     // q, k
  uint16_t* out[2];
  const uint16_t* weight[2];
  long long in_row[2], in_head[2], out_row[2], out_head[2];  // strides, elements
  float eps;
  const int* positions;
  const float* cos_sin;
  long long max_position;
};

struct Kv4Rows {
  int num_reqs, num_rows, Hk;
  const int* cu_rows;
  const int* start;
  uint16_t* x[2];  // k, v rows
  long long row[2], head[2];
  unsigned char* pool;
  int pool_blocks;
  const int* table;
  int table_stride;
};

struct Kv4Decode {
  int num_reqs, H, Hk, G;
  const int* ctx_lens;
  const uint16_t* q;
  uint16_t* o;
  float* lse;
  const unsigned char* pool;
  int pool_blocks;
  const int* table;
  int table_stride;
  float scale_log2;  // log2(e) / sqrt(d)
  float* part;       // workspace: split partial results
  int* counters;     // workspace: arrivals, zero between calls
  int grid;          // CTAs that the workspace is made for
  int* status;       // set where a wait runs out
  int force;         // a test's: one copy of each warp is left out
};

cudaError_t launch_qk_norm_rope(const QkParams& P, int D, int dtype, int interleaved,
                                cudaStream_t s);
cudaError_t launch_kv4_write(const Kv4Rows& P, int D, int group, int dtype, cudaStream_t s);
cudaError_t launch_kv4_read(const Kv4Rows& P, int D, int group, int dtype, cudaStream_t s);
cudaError_t launch_kv4_decode(const Kv4Decode& P, int D, int group, int dtype, cudaStream_t s);
// Resident CTAs per SM and workspace floats per CTA of the decode kernel; sets
// its shared-memory limit on the current device.
cudaError_t kv4_decode_init(int D, int group, int dtype, int G, int max_reqs, int* ctas_per_sm,
                            size_t* part_floats);

}  // namespace pod
