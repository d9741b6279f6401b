// Internal declarations shared by the translation units of libsmla.so.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "smla.h"

namespace smla {

// A launch that answers for itself: cudaGetLastError behind a launch would report, and take
// away, an error that another part of the process left.  (One of its own is taken away: the status
// of the call carries it.)  `dependent`: see launch_dependent.
template <typename... Params, typename... Args>
inline cudaError_t launch_kernel(bool dependent, void (*kernel)(Params...), dim3 grid, unsigned threads, size_t smem,
                                 cudaStream_t stream, const Args&... args) {
  cudaLaunchConfig_t config{};
  config.gridDim = grid;
  config.blockDim = dim3(threads);
  config.dynamicSmemBytes = smem;
  config.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  config.attrs = attr;
  config.numAttrs = dependent ? 1 : 0;
  const cudaError_t err = cudaLaunchKernelEx(&config, kernel, Params(args)...);
  if (err != cudaSuccess) cudaGetLastError();
  return err;
}
template <typename... Params, typename... Args>
inline cudaError_t launch(void (*kernel)(Params...), dim3 grid, unsigned threads, size_t smem, cudaStream_t stream,
                          const Args&... args) {
  return launch_kernel(false, kernel, grid, threads, smem, stream, args...);
}

constexpr int kRecordBytes = SMLA_RECORD_BYTES;
constexpr int kLatent = SMLA_LATENT_DIM;
constexpr int kRope = SMLA_ROPE_DIM;
constexpr int kQK = SMLA_QK_DIM;
constexpr int kScaleOffset = 512;
constexpr int kRopeOffset = 528;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
// Rows shared by at most this many CTAs are merged inside the native-fp8
// decode kernel (by the CTA whose part completes the row); rows of more parts
// are left to the merge kernel when the plan launches it.
constexpr int kMaxInKernelParts = 4;

// Workspace offsets of one plan (see smla_decode_workspace_size in smla.h).
struct WorkspaceLayout {
  int64_t ticket_off, rowtile_off, o_off, ml_off, nv_off, lens_off, total;
};

WorkspaceLayout workspace_layout(int32_t n_q, int32_t heads, int32_t slots, bool trim_lens);

// Everything a decode kernel needs, resolved on the host.
struct DecodeLaunch {
  smla_decode_params p;
  smla_plan_info plan;
  WorkspaceLayout ws;
  void* workspace;
  cudaStream_t stream;
};

// Host-side argument checks of smla_decode (SMLA_OK or a negative status);
// nothing is enqueued.
int check_decode_params(const smla_decode_params* p);

struct DecodeArgs;

// Kernel launchers (one per translation unit).  Return a cudaError_t.
cudaError_t launch_decode_simt(const DecodeLaunch& L);
cudaError_t launch_decode_tc(const DecodeLaunch& L);
cudaError_t launch_decode_fp8(const DecodeLaunch& L);
// The row-trim pass before a tensor-core decode (when plan.trim_kernel; it
// points args.lens at the trimmed lengths) and the merge of shared rows after it.
cudaError_t launch_trim(const DecodeLaunch& L, DecodeArgs& args);
cudaError_t launch_merge(const DecodeLaunch& L, const DecodeArgs& args);
// Heads and tile length of the native-fp8 kernel.
bool fp8_kernel_supports(int num_heads);
int fp8_tile_len();
int fp8_head_groups(int num_heads);
// Pipeline wait limits of the tensor-core kernels (0: their 2 s default) and
// the timeout-path test switch (see smla_set_wait_limit).
cudaError_t fp8_set_wait_limit(uint64_t ns, int stall);
cudaError_t tc_set_wait_limit(uint64_t ns, int stall);
cudaError_t launch_pack(const void* latent, int64_t latent_stride, const void* rope,
                        int64_t rope_stride, int64_t n, void* kv_out, cudaStream_t stream);

// The paged cache.  Workspace of one attend call: per worker (a pair of CTAs, or a
// CTA of the other kernels) a merge job (16 bytes), two partials' (m, l) of
// part_rows rows, and their O.
struct AttendPlan {
  int32_t workers, part_rows;
  int32_t start_slots, merge_tiles;  // slots of a row tile's start; row tiles that may be shared
  int32_t narrow;  // rows of a tile: 16 few-row kernel, 32 and 64 narrow kernel; 0: the pair kernel
  int64_t merge_off, ml_off, o_off, total;
};
AttendPlan paged_attend_plan(const smla_paged_attend_params& p, int num_sms);
// The token rows that a row sees beside the history: bit j of its mask, its sequence's
// row j (a tree); without masks (words < 0) all that the causal edge leaves.
struct TreeMasks {
  const uint32_t* mask = nullptr;
  int64_t stride = 0;
  int32_t words = -1;
};
cudaError_t launch_paged_attend(const smla_paged_attend_params& p, const TreeMasks& tree, const AttendPlan& plan,
                                void* workspace, cudaStream_t stream);
cudaError_t paged_set_wait_limit(uint64_t ns, int stall);
cudaError_t launch_paged_write(const smla_paged_batch& b, const void* latent, int64_t latent_stride, const void* rope,
                               int64_t rope_stride, int32_t dtype, cudaStream_t stream);
cudaError_t launch_paged_read(const smla_paged_batch& b, void* latent, int64_t latent_stride, void* rope,
                              int64_t rope_stride, int32_t dtype, cudaStream_t stream);
cudaError_t launch_paged_append(const smla_paged_append_params& p, cudaStream_t stream);
// (of the batch: cu_rows, seq_lens and the sizes)
cudaError_t launch_paged_tree(const smla_paged_batch& b, const int32_t* parents, uint32_t* mask, int64_t mask_stride,
                              int32_t mask_words, int32_t* positions, cudaStream_t stream);
cudaError_t launch_paged_accept(const smla_paged_batch& b, const int32_t* path, int64_t path_stride, int32_t path_len,
                                int32_t* new_lens, cudaStream_t stream);

}  // namespace smla
