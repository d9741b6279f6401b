// C-ABI entry points of the paged cache: argument checks and launches (host
// code; the kernels are in smla_paged_copy.cu and smla_paged_attend.cu).
#include <cuda_runtime.h>

#include <atomic>
#include <cmath>
#include <cstdint>

#include "smla.h"
#include "smla_internal.h"

namespace smla {
namespace {

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

bool sizes_fit(const smla_paged_batch& b) {
  return b.n_rows >= 0 && b.n_rows <= (int64_t(1) << 30) && b.n_seqs >= 0 && b.n_seqs <= (1 << 24) &&
         b.page_size >= 1 && b.max_pages >= 0 && int64_t(b.max_pages) * b.page_size <= (int64_t(1) << 30);
}

// Checks of the batch; *empty when there is no row to work on.
int check_batch(const smla_paged_batch* b, bool* empty) {
  *empty = false;
  if (b == nullptr) return SMLA_ERR_NULL;
  if (!sizes_fit(*b) || b->n_pages < 0 || b->n_pages > (int64_t(1) << 31)) return SMLA_ERR_SHAPE;
  if (b->n_rows == 0 || b->n_seqs == 0) {
    *empty = true;
    return SMLA_OK;
  }
  if (!b->cu_rows || !b->seq_lens) return SMLA_ERR_NULL;
  if (b->max_pages > 0 && !b->block_table) return SMLA_ERR_NULL;
  if (b->n_pages > 0 && !b->kv_cache) return SMLA_ERR_NULL;
  if (b->page_stride < int64_t(b->page_size) * SMLA_RECORD_BYTES) return SMLA_ERR_STRIDE;
  if (b->block_table_stride < b->max_pages && b->n_seqs > 1) return SMLA_ERR_STRIDE;
  if ((b->page_stride & 15) || !aligned16(b->kv_cache)) return SMLA_ERR_ALIGN;
  return SMLA_OK;
}

int check_copy(const smla_paged_batch* b, const void* latent, int64_t latent_stride, const void* rope,
               int64_t rope_stride, int32_t dtype, bool* empty) {
  int rc = check_batch(b, empty);
  if (rc != SMLA_OK) return rc;
  if (dtype < SMLA_DTYPE_BF16 || dtype > SMLA_DTYPE_F32) return SMLA_ERR_SHAPE;
  if (*empty) return SMLA_OK;
  if (!latent || !rope) return SMLA_ERR_NULL;
  if (latent_stride < SMLA_LATENT_DIM || rope_stride < SMLA_ROPE_DIM) return SMLA_ERR_STRIDE;
  const int64_t step = dtype == SMLA_DTYPE_F32 ? 4 : 8;
  if (!aligned16(latent) || !aligned16(rope) || latent_stride % step || rope_stride % step) return SMLA_ERR_ALIGN;
  return SMLA_OK;
}

int check_attend(const smla_paged_attend_params* p, bool* empty) {
  if (p == nullptr) return SMLA_ERR_NULL;
  // (the kernels scale by sm_scale * log2(e) in f32: an infinite factor would make 0 * inf of scores of 0)
  if (p->num_heads < 1 || p->num_heads > SMLA_PAGED_MAX_HEADS || !std::isfinite(p->sm_scale * kLog2e))
    return SMLA_ERR_SHAPE;
  int rc = check_batch(&p->batch, empty);
  if (rc != SMLA_OK || *empty) return rc;
  if (!p->q || !p->out) return SMLA_ERR_NULL;
  const int64_t h = p->num_heads;
  if (p->q_stride_row < 0 || p->q_stride_head < 0 || p->out_stride_row < 0 || p->out_stride_head < 0)
    return SMLA_ERR_STRIDE;
  if (h > 1 && (p->q_stride_head < SMLA_QK_DIM || p->out_stride_head < SMLA_LATENT_DIM)) return SMLA_ERR_STRIDE;
  if (p->batch.n_rows > 1 && (p->q_stride_row < (h - 1) * p->q_stride_head + SMLA_QK_DIM ||
                              p->out_stride_row < (h - 1) * p->out_stride_head + SMLA_LATENT_DIM))
    return SMLA_ERR_STRIDE;
  if (!aligned16(p->q) || !aligned16(p->out)) return SMLA_ERR_ALIGN;
  if ((p->q_stride_row | p->q_stride_head | p->out_stride_row | p->out_stride_head) & 7) return SMLA_ERR_ALIGN;
  return SMLA_OK;
}

// The current device's SM count, and whether it can run the kernels; asked once
// per device (a call can take less time on the GPU than the queries here).
constexpr int kMaxDevices = 64;
std::atomic<int32_t> g_sms[kMaxDevices];  // 0: not asked yet, -1: not an sm_103

int device_sms(int* n) {
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return SMLA_ERR_DEVICE;
  int32_t v = g_sms[dev].load(std::memory_order_relaxed);
  if (v == 0) {
    int count = 0;
    if (cudaDeviceGetAttribute(&count, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return SMLA_ERR_DEVICE;
    v = smla_device_check() == SMLA_OK && count >= 2 ? count : -1;
    g_sms[dev].store(v, std::memory_order_relaxed);
  }
  if (v < 0) return SMLA_ERR_DEVICE;
  *n = v;
  return SMLA_OK;
}

}  // namespace
}  // namespace smla

using namespace smla;

extern "C" {

int smla_paged_write(const smla_paged_batch* batch, const void* latent, int64_t latent_stride, const void* rope,
                     int64_t rope_stride, int32_t dtype, void* stream) {
  bool empty;
  int rc = check_copy(batch, latent, latent_stride, rope, rope_stride, dtype, &empty);
  if (rc != SMLA_OK || empty) return rc;
  int sms = 0;
  rc = device_sms(&sms);
  if (rc != SMLA_OK) return rc;
  const cudaError_t err =
      launch_paged_write(*batch, latent, latent_stride, rope, rope_stride, dtype, static_cast<cudaStream_t>(stream));
  return err == cudaSuccess ? SMLA_OK : SMLA_ERR_LAUNCH;
}

int smla_paged_read(const smla_paged_batch* batch, void* latent, int64_t latent_stride, void* rope,
                    int64_t rope_stride, int32_t dtype, void* stream) {
  bool empty;
  int rc = check_copy(batch, latent, latent_stride, rope, rope_stride, dtype, &empty);
  if (rc != SMLA_OK || empty) return rc;
  int sms = 0;
  rc = device_sms(&sms);
  if (rc != SMLA_OK) return rc;
  const cudaError_t err =
      launch_paged_read(*batch, latent, latent_stride, rope, rope_stride, dtype, static_cast<cudaStream_t>(stream));
  return err == cudaSuccess ? SMLA_OK : SMLA_ERR_LAUNCH;
}

size_t smla_paged_attend_workspace_size(const smla_paged_attend_params* params) {
  int sms = 0;
  if (params == nullptr || params->num_heads < 1 || params->num_heads > SMLA_PAGED_MAX_HEADS) return 0;
  const smla_paged_batch& b = params->batch;
  // (the sizes alone: pointers may still be unset here)
  if (!sizes_fit(b) || b.n_rows == 0 || b.n_seqs == 0 || device_sms(&sms) != SMLA_OK) return 0;
  return size_t(paged_attend_plan(*params, sms).total);
}

int smla_paged_attend(const smla_paged_attend_params* params, void* workspace, size_t workspace_bytes, void* stream) {
  bool empty;
  int rc = check_attend(params, &empty);
  if (rc != SMLA_OK || empty) return rc;
  int sms = 0;
  rc = device_sms(&sms);
  if (rc != SMLA_OK) return rc;
  const AttendPlan plan = paged_attend_plan(*params, sms);
  if (workspace == nullptr || uint64_t(workspace_bytes) < uint64_t(plan.total)) return SMLA_ERR_WORKSPACE;
  if (reinterpret_cast<uintptr_t>(workspace) & 255u) return SMLA_ERR_ALIGN;
  const cudaError_t err = launch_paged_attend(*params, plan, workspace, static_cast<cudaStream_t>(stream));
  return err == cudaSuccess ? SMLA_OK : SMLA_ERR_LAUNCH;
}

}  // extern "C"
