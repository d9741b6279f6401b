// The paged cache's writer and reader (smla_paged_write, smla_paged_read).
//
// Writer, per block of 128 latent values: scale = pow2ceil(max(amax, 1e-4) / 448),
// code = E4M3(x / scale); 1 / scale is a power of two, so the quotient is exact
// and each value is rounded once.  Reader: value = e4m3 * scale in f32, rounded
// once to the output's type.
//
// A warp takes a token row (in large 16-bit reads two).  Lane l handles the
// 16-byte chunks l, l + 32, ... of a row of the token tensor (8 values of a 16-bit
// type, 4 of f32), so every access of a warp covers a contiguous range on both
// sides; a scale block is 16 or all 32 lanes of one chunk step.  The writer loads
// its row before it looks for the record.
//
// What bounds them: at few rows the chain row -> sequence -> page -> record
// (2.0 us for one row, 2.3 us for 64, graph replays), at many rows HBM: 131072
// rows in pages of 64, bytes of both sides / time: write bf16 39.1 us = 6.1 TB/s,
// write f32 58.4 us = 6.6 TB/s, read bf16 38.2 us = 6.2 TB/s, read f32 60.3 us =
// 6.4 TB/s.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "smla_internal.h"
#include "smla_paged.cuh"
#include "smla_paged_copy.cuh"

namespace smla {
namespace {

constexpr int kWarps = 8;

// Lane j's record of token row base + j (j < kRows): nullptr for a masked
// position; *has is whether the row belongs to a sequence.  A row behind the first
// one's sequence is most often the next one's; if it is not, empty sequences lie
// between, through which the warp searches again (walking through 2^20 of them took
// 72 ms).
template <int kRows>
__device__ __forceinline__ uint8_t* locate(const PagedArgs& a, int32_t base, bool* has) {
  const int lane = threadIdx.x & 31;
  int32_t b = seq_of_row(a, base);
  const int32_t r = base + lane;
  const bool mine = lane < kRows && r < a.n_rows;
  int32_t end = mine ? cu_at(a, b + 1) : 0;
  if constexpr (kRows > 1) {
    if (mine && end <= r && b + 1 < a.n_seqs) end = cu_at(a, ++b + 1);
    uint32_t behind = __ballot_sync(0xffffffffu, mine && end <= r && b + 1 < a.n_seqs);
    for (; behind != 0; behind &= behind - 1) {
      const int j = __ffs(behind) - 1;
      const int32_t s = seq_of_row(a, base + j);
      if (lane == j) b = s, end = cu_at(a, s + 1);
    }
  }
  *has = mine && r < end && cu_at(a, b) <= r;
  return *has ? record_at(a, b, seq_len_at(a, b) - (end - r)) : nullptr;
}

template <int kDtype>
__global__ void __launch_bounds__(32 * kWarps)
paged_write_kernel(const __grid_constant__ PagedArgs a, const uint8_t* __restrict__ latent, int64_t latent_stride,
                   const uint8_t* __restrict__ rope, int64_t rope_stride) {
  using E = Elem<kDtype>;
  const int lane = threadIdx.x & 31;
  const int64_t row = int64_t(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  if (row >= a.n_rows) return;
  const uint8_t* src = latent + row * latent_stride * E::kBytes + lane * 16;
  uint4 lat[E::kSteps], rp;
#pragma unroll
  for (int i = 0; i < E::kSteps; ++i) lat[i] = __ldcs(reinterpret_cast<const uint4*>(src + i * 512));
  if (lane < E::kRopeLanes)
    rp = __ldcs(reinterpret_cast<const uint4*>(rope + row * rope_stride * E::kBytes + lane * 16));
  bool has;
  const uint64_t mine = reinterpret_cast<uint64_t>(locate<1>(a, int32_t(row), &has));
  uint8_t* rec = reinterpret_cast<uint8_t*>(__shfl_sync(0xffffffffu, mine, 0));
  if (rec == nullptr) return;
  write_latent<kDtype>(rec, lat);
  if (lane < E::kRopeLanes) {
    if constexpr (kDtype == SMLA_DTYPE_BF16) {
      *reinterpret_cast<uint4*>(rec + kRopeOffset + lane * 16) = rp;
    } else {
      float x[E::kPer];
      unpack<kDtype>(rp, x);
      uint32_t w[E::kPer / 2];
#pragma unroll
      for (int k = 0; k < E::kPer / 2; ++k) {
        const __nv_bfloat162 v = __floats2bfloat162_rn(x[2 * k], x[2 * k + 1]);
        w[k] = *reinterpret_cast<const uint32_t*>(&v);
      }
      if constexpr (E::kPer == 8)
        *reinterpret_cast<uint4*>(rec + kRopeOffset + lane * 16) = make_uint4(w[0], w[1], w[2], w[3]);
      else
        *reinterpret_cast<uint2*>(rec + kRopeOffset + lane * 8) = make_uint2(w[0], w[1]);
    }
  }
}

template <int kRows, int kDtype>
__global__ void __launch_bounds__(32 * kWarps)
paged_read_kernel(const __grid_constant__ PagedArgs a, uint8_t* __restrict__ latent, int64_t latent_stride,
                  uint8_t* __restrict__ rope, int64_t rope_stride) {
  using E = Elem<kDtype>;
  constexpr int kCodes = E::kPer / 4;  // 32-bit words of codes per chunk
  const int lane = threadIdx.x & 31;
  const int64_t base64 = (int64_t(blockIdx.x) * kWarps + (threadIdx.x >> 5)) * kRows;
  if (base64 >= a.n_rows) return;
  const int32_t base = int32_t(base64);
  bool has;
  const uint64_t mine = reinterpret_cast<uint64_t>(locate<kRows>(a, base, &has));
  const uint32_t rows = __ballot_sync(0xffffffffu, has);
  uint32_t code[kRows][E::kSteps][kCodes];
  float scale[kRows][E::kSteps];
  uint32_t rp[kRows][E::kPer / 2];
#pragma unroll
  for (int j = 0; j < kRows; ++j) {
    const uint8_t* rec = reinterpret_cast<const uint8_t*>(__shfl_sync(0xffffffffu, mine, j));
#pragma unroll
    for (int i = 0; i < E::kSteps; ++i) {
      const int chunk = lane + 32 * i;
#pragma unroll
      for (int k = 0; k < kCodes; ++k) code[j][i][k] = 0;
      scale[j][i] = 0.f;
      if (rec != nullptr) {
        if constexpr (kCodes == 2) {
          const uint2 v = *reinterpret_cast<const uint2*>(rec + chunk * 8);
          code[j][i][0] = v.x;
          code[j][i][1] = v.y;
        } else {
          code[j][i][0] = *reinterpret_cast<const uint32_t*>(rec + chunk * 4);
        }
        scale[j][i] = *reinterpret_cast<const float*>(rec + kScaleOffset + 4 * (chunk * E::kPer / 128));
      }
    }
#pragma unroll
    for (int k = 0; k < E::kPer / 2; ++k) rp[j][k] = 0;
    if (rec != nullptr && lane < E::kRopeLanes) {
      if constexpr (E::kPer == 8) {
        const uint4 v = *reinterpret_cast<const uint4*>(rec + kRopeOffset + lane * 16);
        rp[j][0] = v.x, rp[j][1] = v.y, rp[j][2] = v.z, rp[j][3] = v.w;
      } else {
        const uint2 v = *reinterpret_cast<const uint2*>(rec + kRopeOffset + lane * 8);
        rp[j][0] = v.x, rp[j][1] = v.y;
      }
    }
  }
#pragma unroll
  for (int j = 0; j < kRows; ++j) {
    if (!((rows >> j) & 1u)) continue;  // no sequence's row
    uint8_t* dst = latent + int64_t(base + j) * latent_stride * E::kBytes + lane * 16;
#pragma unroll
    for (int i = 0; i < E::kSteps; ++i) {
      float x[E::kPer];
#pragma unroll
      for (int k = 0; k < kCodes; ++k) e4m3x4_to_f32(code[j][i][k], x + 4 * k);
#pragma unroll
      for (int k = 0; k < E::kPer; ++k) x[k] *= scale[j][i];
      *reinterpret_cast<uint4*>(dst + i * 512) = pack<kDtype>(x);
    }
    if (lane < E::kRopeLanes) {
      float x[E::kPer];
#pragma unroll
      for (int k = 0; k < E::kPer / 2; ++k) {
        x[2 * k] = __uint_as_float(rp[j][k] << 16);
        x[2 * k + 1] = __uint_as_float(rp[j][k] & 0xFFFF0000u);
      }
      uint4 v = pack<kDtype>(x);
      if constexpr (kDtype == SMLA_DTYPE_BF16) v = make_uint4(rp[j][0], rp[j][1], rp[j][2], rp[j][3]);  // bit for bit
      *reinterpret_cast<uint4*>(rope + int64_t(base + j) * rope_stride * E::kBytes + lane * 16) = v;
    }
  }
}

// Rows of 16-bit reads above which a warp takes two, so that their loads fly
// together (one row a warp / two, us: 1216 rows 2.58 / 2.72, 4864 rows 3.21 / 3.08,
// 131072 rows 40.8 / 38.2).  Writes and f32 reads take one at every size (two:
// bf16 write 39.1 -> 40.1 us, f32 write 58.4 -> 59.6, f32 read 60.4 -> 61.3 at
// 131072 rows; four: 68.6 for the f32 write).
constexpr int64_t kOneRowLimit = 2432;

unsigned grid_of(const PagedArgs& a, int rows) {
  return unsigned((int64_t(a.n_rows) + kWarps * rows - 1) / (kWarps * rows));
}

template <int kDtype>
cudaError_t write_typed(const PagedArgs& a, const uint8_t* lat, int64_t ls, const uint8_t* rope, int64_t rs, cudaStream_t st) {
  return launch(paged_write_kernel<kDtype>, dim3(grid_of(a, 1)), 32 * kWarps, 0, st, a, lat, ls, rope, rs);
}

template <int kDtype>
cudaError_t read_typed(const PagedArgs& a, uint8_t* lat, int64_t ls, uint8_t* rope, int64_t rs, cudaStream_t st) {
  if constexpr (kDtype != SMLA_DTYPE_F32) {
    if (a.n_rows > kOneRowLimit)
      return launch(paged_read_kernel<2, kDtype>, dim3(grid_of(a, 2)), 32 * kWarps, 0, st, a, lat, ls, rope, rs);
  }
  return launch(paged_read_kernel<1, kDtype>, dim3(grid_of(a, 1)), 32 * kWarps, 0, st, a, lat, ls, rope, rs);
}

}  // namespace

cudaError_t launch_paged_write(const smla_paged_batch& b, const void* latent, int64_t ls, const void* rope, int64_t rs,
                               int32_t dtype, cudaStream_t st) {
  const PagedArgs a = make_paged_args(b);
  const uint8_t* l = static_cast<const uint8_t*>(latent);
  const uint8_t* r = static_cast<const uint8_t*>(rope);
  if (dtype == SMLA_DTYPE_BF16) return write_typed<SMLA_DTYPE_BF16>(a, l, ls, r, rs, st);
  if (dtype == SMLA_DTYPE_F16) return write_typed<SMLA_DTYPE_F16>(a, l, ls, r, rs, st);
  return write_typed<SMLA_DTYPE_F32>(a, l, ls, r, rs, st);
}

cudaError_t launch_paged_read(const smla_paged_batch& b, void* latent, int64_t ls, void* rope, int64_t rs,
                              int32_t dtype, cudaStream_t st) {
  const PagedArgs a = make_paged_args(b);
  uint8_t* l = static_cast<uint8_t*>(latent);
  uint8_t* r = static_cast<uint8_t*>(rope);
  if (dtype == SMLA_DTYPE_BF16) return read_typed<SMLA_DTYPE_BF16>(a, l, ls, r, rs, st);
  if (dtype == SMLA_DTYPE_F16) return read_typed<SMLA_DTYPE_F16>(a, l, ls, r, rs, st);
  return read_typed<SMLA_DTYPE_F32>(a, l, ls, r, rs, st);
}

}  // namespace smla
