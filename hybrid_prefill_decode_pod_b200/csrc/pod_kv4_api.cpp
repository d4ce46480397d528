// pod_kv4_api.cpp -- C ABI and argument checks of the 4-bit KV cache. See
// include/pod_kv4.h for the contract.
#include <cuda_runtime.h>

#include <cstdint>
#include <new>

#include "pod_device.h"
#include "pod_kv4.h"
#include "pod_kv4_params.h"

using namespace pod;

struct pod_kv4_ctx {
  pod_kv4_config cfg{};
  int grid = 0;  // CTAs of the decode kernel
  float* part = nullptr;
  int* counters = nullptr;  // [grid] arrivals, then the status word
  bool force = false;       // the next decode leaves copies out (POD_FLAG_TEST_FORCE_TIMEOUT)
};

namespace {

constexpr int kMaxGroup = 8;

bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// The strides of rows [rows, heads, d]: multiples of 16 bytes, not negative
// and small enough that no offset leaves 62 bits. Written rows may not overlap.
// The stride of an axis of one entry says nothing and becomes 0.
bool strides_ok(long long& row, long long& head, long long rows, long long heads, int d,
                bool written) {
  if (rows <= 1) row = 0;
  if (heads <= 1) head = 0;
  if (row < 0 || head < 0 || row % 8 || head % 8) return false;
  if (row > (1LL << 30) || head > (1LL << 30)) return false;
  if (!written) return true;
  if (heads > 1 && head < d) return false;
  if (rows > 1 && row < d) return false;
  if (rows <= 1 || heads <= 1) return true;
  return row >= (heads - 1) * head + d || head >= (rows - 1) * row + d;
}

int check_device(int device) {
  int ndev = 0;
  if (cudaGetDeviceCount(&ndev) != cudaSuccess) return POD_ECUDA;
  return device < 0 || device >= ndev ? POD_EINVAL : POD_OK;
}

int check_shape(int d, int group) {
  if (d != 64 && d != 128) return POD_EUNSUPPORTED;
  if (group != 32 && group != 64 && group != 128) return POD_EUNSUPPORTED;
  return group > d ? POD_EUNSUPPORTED : POD_OK;
}

int check_cache(const pod_kv4_ctx* c, int num_reqs, const void* pool, long long blocks,
                const int* table, int stride) {
  if (!pool || (!table && stride) || blocks <= 0 || stride < 0) return POD_EINVAL;
  if (!aligned16(pool) || !aligned4(table)) return POD_EINVAL;
  if (blocks * c->cfg.num_kv_heads > (1LL << 31) - 1 || blocks > (1LL << 31) - 1 ||
      (long long)num_reqs * (stride + 8LL) > (1LL << 31) - 1 || stride > (1 << 26))
    return POD_ECAPACITY;
  return POD_OK;
}

int check_rows(const pod_kv4_ctx* c, const pod_kv4_rows_args* a, bool written, Kv4Rows* P) {
  if (a->num_reqs < 0 || a->num_rows < 0) return POD_EINVAL;
  if (a->num_rows > (1 << 30)) return POD_ECAPACITY;
  if (a->num_reqs == 0 || a->num_rows == 0) return POD_OK;
  if (!a->cu_rows || !a->start || !a->k || !a->v) return POD_EINVAL;
  if (!aligned4(a->cu_rows) || !aligned4(a->start) || !aligned16(a->k) || !aligned16(a->v))
    return POD_EINVAL;
  const int Hk = c->cfg.num_kv_heads, d = c->cfg.head_dim;
  P->row[0] = a->k_row_stride;
  P->row[1] = a->v_row_stride;
  P->head[0] = a->k_head_stride;
  P->head[1] = a->v_head_stride;
  for (int i = 0; i < 2; ++i)
    if (!strides_ok(P->row[i], P->head[i], a->num_rows, Hk, d, written)) return POD_EINVAL;
  const int rc =
      check_cache(c, a->num_reqs, a->pool, a->pool_blocks, a->block_table, a->block_table_stride);
  if (rc) return rc;
  P->num_reqs = a->num_reqs;
  P->num_rows = a->num_rows;
  P->Hk = Hk;
  P->cu_rows = a->cu_rows;
  P->start = a->start;
  P->x[0] = static_cast<uint16_t*>(a->k);
  P->x[1] = static_cast<uint16_t*>(a->v);
  P->pool = static_cast<unsigned char*>(a->pool);
  P->pool_blocks = (int)a->pool_blocks;
  P->table = a->block_table;
  P->table_stride = a->block_table_stride;
  return POD_OK;
}

int rows_call(pod_kv4_ctx* c, const pod_kv4_rows_args* a, bool read, void* stream) {
  if (!c || !a) return POD_EINVAL;
  Kv4Rows P{};
  const int rc = check_rows(c, a, read, &P);
  if (rc) return rc;
  if (P.num_rows == 0) return POD_OK;
  DeviceGuard guard(c->cfg.device);
  if (!guard.ok) return POD_ECUDA;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const auto f = read ? launch_kv4_read : launch_kv4_write;
  return f(P, c->cfg.head_dim, c->cfg.group_size, c->cfg.dtype, s) == cudaSuccess ? POD_OK
                                                                                 : POD_ECUDA;
}

}  // namespace

extern "C" {

int pod_qk_norm_rope(const pod_qk_args* a, void* stream) {
  if (!a) return POD_EINVAL;
  const int d = a->head_dim;
  if (a->num_qo_heads < 0 || a->num_kv_heads < 0 || a->num_rows < 0) return POD_EINVAL;
  if (d != 64 && d != 128) return POD_EUNSUPPORTED;
  if (a->rot_dim < 16 || a->rot_dim > d || a->rot_dim % 16) return POD_EUNSUPPORTED;
  if (a->dtype != POD_DTYPE_BF16 && a->dtype != POD_DTYPE_FP16) return POD_EUNSUPPORTED;
  if (a->interleaved != 0 && a->interleaved != 1) return POD_EINVAL;
  if (!(a->eps >= 0.0f) || a->max_position < 0) return POD_EINVAL;
  if (a->num_qo_heads > (1 << 16) || a->num_kv_heads > (1 << 16) || a->num_rows > (1 << 30))
    return POD_ECAPACITY;
  if (a->num_rows == 0 || a->num_qo_heads + a->num_kv_heads == 0) return POD_OK;
  if (!a->positions || !a->cos_sin || !aligned4(a->positions) || !aligned16(a->cos_sin))
    return POD_EINVAL;
  QkParams P{};
  P.heads[0] = a->num_qo_heads;
  P.heads[1] = a->num_kv_heads;
  P.num_rows = a->num_rows;
  P.rot = a->rot_dim;
  P.eps = a->eps;
  P.positions = a->positions;
  P.cos_sin = a->cos_sin;
  P.max_position = a->max_position;
  const void* in[2] = {a->q, a->k};
  void* out[2] = {a->q_out, a->k_out};
  const void* w[2] = {a->q_weight, a->k_weight};
  long long st[2][4] = {
      {a->q_row_stride, a->q_head_stride, a->q_out_row_stride, a->q_out_head_stride},
      {a->k_row_stride, a->k_head_stride, a->k_out_row_stride, a->k_out_head_stride}};
  for (int i = 0; i < 2; ++i) {
    if (P.heads[i] == 0) continue;
    if (!in[i] || !out[i] || !aligned16(in[i]) || !aligned16(out[i]) || (w[i] && !aligned16(w[i])))
      return POD_EINVAL;
    if (!strides_ok(st[i][0], st[i][1], a->num_rows, P.heads[i], d, false) ||
        !strides_ok(st[i][2], st[i][3], a->num_rows, P.heads[i], d, true))
      return POD_EINVAL;
    // in place only row by row: other strides would write rows not read yet
    if (in[i] == out[i] && (st[i][0] != st[i][2] || st[i][1] != st[i][3])) return POD_EINVAL;
    P.in[i] = static_cast<const uint16_t*>(in[i]);
    P.out[i] = static_cast<uint16_t*>(out[i]);
    P.weight[i] = static_cast<const uint16_t*>(w[i]);
    P.in_row[i] = st[i][0];
    P.in_head[i] = st[i][1];
    P.out_row[i] = st[i][2];
    P.out_head[i] = st[i][3];
  }
  const int rc = check_device(a->device);
  if (rc) return rc;
  DeviceGuard guard(a->device);
  if (!guard.ok) return POD_ECUDA;
  return launch_qk_norm_rope(P, d, a->dtype, a->interleaved, static_cast<cudaStream_t>(stream)) ==
                 cudaSuccess
             ? POD_OK
             : POD_ECUDA;
}

int pod_kv4_record_bytes(int head_dim, int group_size) {
  const int rc = check_shape(head_dim, group_size);
  return rc ? rc : kv4_record_bytes(head_dim, group_size);
}

int pod_kv4_create(pod_kv4_ctx** out, const pod_kv4_config* cfg) {
  if (!out || !cfg) return POD_EINVAL;
  *out = nullptr;
  const int H = cfg->num_qo_heads, Hk = cfg->num_kv_heads;
  if (H <= 0 || Hk <= 0 || H % Hk != 0 || cfg->max_decode_reqs < 1) return POD_EINVAL;
  int rc = check_shape(cfg->head_dim, cfg->group_size);
  if (rc) return rc;
  if (H / Hk > kMaxGroup || cfg->page_size != kKv4Page) return POD_EUNSUPPORTED;
  if (cfg->dtype != POD_DTYPE_BF16 && cfg->dtype != POD_DTYPE_FP16) return POD_EUNSUPPORTED;
  if (cfg->flags & ~POD_FLAG_TEST_FORCE_TIMEOUT) return POD_EUNSUPPORTED;
  if (cfg->max_decode_reqs > kKv4MaxReqs || Hk > 512) return POD_ECAPACITY;
  rc = check_device(cfg->device);
  if (rc) return rc;
  DeviceGuard guard(cfg->device);
  if (!guard.ok) return POD_ECUDA;
  int major = 0, minor = 0, sms = 0;
  if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, cfg->device) ||
      cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, cfg->device) ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, cfg->device))
    return POD_ECUDA;
  if (major != 10 || minor != 0) return POD_EUNSUPPORTED;  // built for sm_100a only

  pod_kv4_ctx* c = new (std::nothrow) pod_kv4_ctx();
  if (!c) return POD_ENOMEM;
  c->cfg = *cfg;
  c->force = cfg->flags & POD_FLAG_TEST_FORCE_TIMEOUT;
  int per_sm = 0;
  size_t floats = 0;
  if (kv4_decode_init(cfg->head_dim, cfg->group_size, cfg->dtype, H / Hk, cfg->max_decode_reqs,
                      &per_sm, &floats) !=
          cudaSuccess ||
      per_sm < 1) {
    delete c;
    return POD_ECUDA;
  }
  c->grid = sms * per_sm;
  if (cudaMalloc(&c->part, sizeof(float) * (floats * c->grid + 1)) != cudaSuccess ||
      cudaMalloc(&c->counters, sizeof(int) * (c->grid + 1)) != cudaSuccess ||
      cudaMemset(c->counters, 0, sizeof(int) * (c->grid + 1)) != cudaSuccess ||
      cudaDeviceSynchronize() != cudaSuccess) {
    cudaGetLastError();
    pod_kv4_destroy(c);
    return POD_ENOMEM;
  }
  *out = c;
  return POD_OK;
}

int pod_kv4_write(pod_kv4_ctx* c, const pod_kv4_rows_args* a, void* stream) {
  return rows_call(c, a, false, stream);
}

int pod_kv4_read(pod_kv4_ctx* c, const pod_kv4_rows_args* a, void* stream) {
  return rows_call(c, a, true, stream);
}

int pod_kv4_decode(pod_kv4_ctx* c, const pod_kv4_decode_args* a, void* stream) {
  if (!c || !a || a->num_reqs < 0) return POD_EINVAL;
  if (a->num_reqs > c->cfg.max_decode_reqs) return POD_ECAPACITY;
  if (a->num_reqs == 0) return POD_OK;
  if (!a->ctx_lens || !a->q || !a->o || !a->lse) return POD_EINVAL;
  if (!aligned4(a->ctx_lens) || !aligned16(a->q) || !aligned16(a->o) || !aligned4(a->lse))
    return POD_EINVAL;
  const int rc =
      check_cache(c, a->num_reqs, a->pool, a->pool_blocks, a->block_table, a->block_table_stride);
  if (rc) return rc;
  Kv4Decode P{};
  P.num_reqs = a->num_reqs;
  P.H = c->cfg.num_qo_heads;
  P.Hk = c->cfg.num_kv_heads;
  P.G = P.H / P.Hk;
  P.ctx_lens = a->ctx_lens;
  P.q = static_cast<const uint16_t*>(a->q);
  P.o = static_cast<uint16_t*>(a->o);
  P.lse = a->lse;
  P.pool = static_cast<const unsigned char*>(a->pool);
  P.pool_blocks = (int)a->pool_blocks;
  P.table = a->block_table;
  P.table_stride = a->block_table_stride;
  P.scale_log2 = 1.4426950408889634f / (c->cfg.head_dim == 128 ? 11.313708498984761f : 8.0f);
  P.part = c->part;
  P.counters = c->counters;
  P.grid = c->grid;
  P.status = c->counters + c->grid;
  P.force = c->force;
  c->force = false;
  DeviceGuard guard(c->cfg.device);
  if (!guard.ok) return POD_ECUDA;
  return launch_kv4_decode(P, c->cfg.head_dim, c->cfg.group_size, c->cfg.dtype,
                           static_cast<cudaStream_t>(stream)) == cudaSuccess
             ? POD_OK
             : POD_ECUDA;
}

int pod_kv4_status(pod_kv4_ctx* c, void* stream) {
  if (!c) return POD_EINVAL;
  DeviceGuard guard(c->cfg.device);
  if (!guard.ok) return POD_ECUDA;
  if (cudaStreamSynchronize(static_cast<cudaStream_t>(stream)) != cudaSuccess) return POD_ECUDA;
  int st = 0, *word = c->counters + c->grid;
  if (cudaMemcpy(&st, word, sizeof(int), cudaMemcpyDeviceToHost) != cudaSuccess ||
      cudaMemset(word, 0, sizeof(int)) != cudaSuccess)
    return POD_ECUDA;
  return st;
}

int pod_kv4_destroy(pod_kv4_ctx* c) {
  if (!c) return POD_OK;
  int st = POD_OK;
  {
    DeviceGuard guard(c->cfg.device);
    if (cudaDeviceSynchronize() != cudaSuccess ||
        (c->counters && cudaMemcpy(&st, c->counters + c->grid, sizeof(int),
                                   cudaMemcpyDeviceToHost) != cudaSuccess))
      st = POD_ECUDA;
    cudaFree(c->part);
    cudaFree(c->counters);
  }
  delete c;
  return st;
}

}  // extern "C"
