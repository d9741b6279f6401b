// The paged cache's writer with the position rotation on the way (smla_paged_append):
// new rows' records with their rope rotated, and their queries' rope rotated into q.
//
// Pair k of a row at rotation position p turns by p * inv_freq[k] radians:
//   (x, y) -> scale (x cos - y sin, x sin + y cos).
// The angle is needed modulo a turn, which a float product loses at far positions (f32 has
// steps of 2^-7 radians at 10^5).  In turns, as a fixed-point fraction of 64 bits, the product
// with an integer position is a 64-bit multiplication that drops whole turns by itself:
// exact but for the factor's own 2^-64, 2^-34 turns at position 2^30.  Its upper 32 bits go to
// sincospif, which takes half turns, as an f32: rounded by 2^-26 turns at most.
//
// What bounds it: HBM at many rows (65536 rows, 16 heads, f32, 597 MB, L2 flushed: 98 us = 6.1
// TB/s, 91% of the measured copy peak; 32 trees of up to 60 rows, 128 heads, 42 MB: 7.0 us from
// L2, 12 flushed), at few the chain row -> sequence -> page -> record (64 rows, 16 heads:
// 2.45 us).  A row's queries are warps of their own, 16 heads each, so that 128 heads of one
// row are spread; all loads set out before the row's sequence is looked for.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "smla_internal.h"
#include "smla_paged.cuh"
#include "smla_paged_copy.cuh"

namespace smla {
namespace {

constexpr int kWarps = 8;
constexpr int kPairs = kRope / 2;  // a lane's each
constexpr int kLanesPerHead = 4;   // a lane takes 8 neighbouring pairs
constexpr int kHeadsPerStep = 32 / kLanesPerHead;
constexpr int kSteps = 2;
constexpr int kHeadsPerWarp = kHeadsPerStep * kSteps;

struct AppendArgs {
  PagedArgs b;
  const uint8_t* latent;
  int64_t latent_stride;  // bytes, like all of these
  const uint8_t* rope;
  int64_t rope_stride;
  const uint64_t* turns;
  const int32_t* positions;
  const uint8_t* q;
  int64_t q_row, q_head;
  uint8_t* q_out;
  int64_t q_out_row, q_out_head;
  float scale;
  int32_t heads;
};

// Cosine and sine, times the scale, of a pair that turns so far a position.
__device__ __forceinline__ float2 rotation(const AppendArgs& a, uint64_t turns, int32_t pos) {
  const uint64_t turn = turns * uint64_t(int64_t(pos));
  float s, c;
  sincospif(float(int32_t(turn >> 32)) * 0x1p-31f, &s, &c);
  return make_float2(c * a.scale, s * a.scale);
}

__device__ __forceinline__ void rotate(float& x, float& y, float c, float s) {
  const float u = fmaf(x, c, -(y * s));
  y = fmaf(x, s, y * c);
  x = u;
}

// One value of a row of the token tensors, as f32.
template <int kDtype>
__device__ __forceinline__ float load_value(const uint8_t* row, int i) {
  if constexpr (kDtype == SMLA_DTYPE_F32) return reinterpret_cast<const float*>(row)[i];
  else if constexpr (kDtype == SMLA_DTYPE_F16) return __half2float(reinterpret_cast<const __half*>(row)[i]);
  else return __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(row)[i]);
}

// A warp a row's record (blockIdx.y = 0) or the queries of 16 of its heads.
template <int kDtype, bool kInterleaved>
__global__ void __launch_bounds__(32 * kWarps) paged_append_kernel(const __grid_constant__ AppendArgs a) {
  using E = Elem<kDtype>;
  constexpr int kChunks = 16 / E::kPer;  // a lane's of a head
  wait_for_primary();
  const int lane = threadIdx.x & 31;
  const int64_t row64 = int64_t(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  if (row64 >= a.b.n_rows) return;
  const int32_t row = int32_t(row64);
  const bool record = blockIdx.y == 0;
  // the row sets out before its sequence is looked for
  uint4 lat[E::kSteps], q[kSteps][kChunks];
  float x = 0.f, y = 0.f;
  // lane's pair of the record's rope
  const int i0 = kInterleaved ? 2 * lane : lane, i1 = kInterleaved ? i0 + 1 : lane + kPairs;
  // pairs 8 c .. 8 c + 7 of the lane's heads lie in neighbouring chunks, or in both halves
  const int c = lane & (kLanesPerHead - 1);
  const int head0 = (int(blockIdx.y) - 1) * kHeadsPerWarp + lane / kLanesPerHead;
  auto chunk_at = [&](int j) {
    return kInterleaved ? kChunks * c + j : kChunks / 2 * c + j % (kChunks / 2) + j / (kChunks / 2) * (2 * kChunks);
  };
  if (record) {
    const uint8_t* src = a.latent + row * a.latent_stride + lane * 16;
#pragma unroll
    for (int i = 0; i < E::kSteps; ++i) lat[i] = __ldcs(reinterpret_cast<const uint4*>(src + i * 512));
    x = load_value<kDtype>(a.rope + row * a.rope_stride, i0);
    y = load_value<kDtype>(a.rope + row * a.rope_stride, i1);
  } else {
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
      const int head = head0 + i * kHeadsPerStep;
      const uint8_t* src = a.q + row * a.q_row + head * a.q_head;
#pragma unroll
      for (int j = 0; j < kChunks; ++j)
        if (head < a.heads) q[i][j] = __ldcs(reinterpret_cast<const uint4*>(src + chunk_at(j) * 16));
    }
  }
  const uint64_t turns = load_fresh_u64(a.turns + lane);  // of pair `lane`
  const int32_t given = a.positions != nullptr ? load_i32<kFresh>(a.positions + row) : 0;
  const int32_t b = seq_of_row<kFresh>(a.b, row);
  const int32_t end = cu_at<kFresh>(a.b, b + 1);
  if (row >= end || cu_at<kFresh>(a.b, b) > row) return;  // no sequence's row
  const int32_t pos = seq_len_at<kFresh>(a.b, b) - (end - row);
  const float2 cs = rotation(a, turns, a.positions != nullptr ? given : pos);
  if (record) {
    uint64_t at = 0;
    if (lane == 0) at = reinterpret_cast<uint64_t>(record_at<kFresh>(a.b, b, pos));
    uint8_t* rec = reinterpret_cast<uint8_t*>(__shfl_sync(0xffffffffu, at, 0));
    if (rec == nullptr) return;
    write_latent<kDtype>(rec, lat);
    rotate(x, y, cs.x, cs.y);
    const __nv_bfloat162 v = __floats2bfloat162_rn(x, y);
    if constexpr (kInterleaved) {
      *reinterpret_cast<__nv_bfloat162*>(rec + kRopeOffset + 4 * lane) = v;
    } else {
      *reinterpret_cast<__nv_bfloat16*>(rec + kRopeOffset + 2 * lane) = v.x;
      *reinterpret_cast<__nv_bfloat16*>(rec + kRopeOffset + 2 * (lane + kPairs)) = v.y;
    }
    return;
  }
  float co[8], si[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    co[k] = __shfl_sync(0xffffffffu, cs.x, 8 * c + k);
    si[k] = __shfl_sync(0xffffffffu, cs.y, 8 * c + k);
  }
#pragma unroll
  for (int i = 0; i < kSteps; ++i) {
    const int head = head0 + i * kHeadsPerStep;
    if (head >= a.heads) break;
    float v[16];
#pragma unroll
    for (int j = 0; j < kChunks; ++j)
      unpack<kDtype>(q[i][j], *reinterpret_cast<float(*)[E::kPer]>(v + j * E::kPer));
    uint32_t w[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) rotate(v[kInterleaved ? 2 * k : k], v[kInterleaved ? 2 * k + 1 : k + 8], co[k], si[k]);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const __nv_bfloat162 p = __floats2bfloat162_rn(v[2 * k], v[2 * k + 1]);
      w[k] = *reinterpret_cast<const uint32_t*>(&p);
    }
    uint8_t* dst = a.q_out + row * a.q_out_row + head * a.q_out_head;
    *reinterpret_cast<uint4*>(dst + (kInterleaved ? 2 * c : c) * 16) = make_uint4(w[0], w[1], w[2], w[3]);
    *reinterpret_cast<uint4*>(dst + (kInterleaved ? 2 * c + 1 : c + 4) * 16) = make_uint4(w[4], w[5], w[6], w[7]);
  }
}

template <int kDtype>
cudaError_t append_typed(const AppendArgs& a, bool interleaved, cudaStream_t st) {
  const dim3 grid(unsigned((int64_t(a.b.n_rows) + kWarps - 1) / kWarps),
                  unsigned(1 + (a.heads + kHeadsPerWarp - 1) / kHeadsPerWarp));
  if (interleaved) return launch_dependent(paged_append_kernel<kDtype, true>, grid, 32 * kWarps, 0, st, a);
  return launch_dependent(paged_append_kernel<kDtype, false>, grid, 32 * kWarps, 0, st, a);
}

}  // namespace

cudaError_t launch_paged_append(const smla_paged_append_params& p, cudaStream_t st) {
  AppendArgs a{};
  const int64_t size = p.dtype == SMLA_DTYPE_F32 ? 4 : 2;
  a.b = make_paged_args(p.batch);
  a.latent = static_cast<const uint8_t*>(p.latent);
  a.latent_stride = p.latent_stride * size;
  a.rope = static_cast<const uint8_t*>(p.rope);
  a.rope_stride = p.rope_stride * size;
  a.turns = p.turns;
  a.positions = p.positions;
  a.q = static_cast<const uint8_t*>(p.q_rope);
  a.q_row = p.q_rope_stride_row * size;
  a.q_head = p.q_rope_stride_head * size;
  a.q_out = static_cast<uint8_t*>(p.q_out);
  a.q_out_row = p.q_out_stride_row * 2;
  a.q_out_head = p.q_out_stride_head * 2;
  a.scale = p.rope_scale;
  a.heads = p.num_heads;
  if (p.dtype == SMLA_DTYPE_BF16) return append_typed<SMLA_DTYPE_BF16>(a, p.interleaved != 0, st);
  if (p.dtype == SMLA_DTYPE_F16) return append_typed<SMLA_DTYPE_F16>(a, p.interleaved != 0, st);
  return append_typed<SMLA_DTYPE_F32>(a, p.interleaved != 0, st);
}

}  // namespace smla
