// Drafted-token trees over the paged cache: the nodes' masks and positions from
// their parents (smla_paged_tree), and the accepted path's records moved up behind the
// history (smla_paged_accept).
#include <cuda_runtime.h>

#include <cstdint>

#include "smla_internal.h"
#include "smla_paged.cuh"

namespace smla {
namespace {

// ---- masks and positions ----
//
// With p(i) the parent of node i, the mask of i is {i} and the mask of p(i), its position
// past + the number of ancestors.  A thread takes a node and walks up its ancestors; a
// parent is a lower node than its child (anything else is a root), so the walk ends, and
// the mask's words are met from the last to the first.  The block's nodes collect 32 words
// each in shared memory at a time, which then leave row after row.
//
// Bound: the walk, a chain of look-ups.  It reads a copy of the parents in shared memory that
// holds each node's parent and grandparent, so that a look-up goes two nodes up; the bits are
// set by shared-memory atomics, whose results nobody waits for (sequences of more than 2048
// nodes: one node at a time, through L1).  7 trees of up to 500 nodes, 40 deep: 5.0 us (12.8
// with one node a look-up and the words stored by each thread as it walks); 64 of 60: 2.5 us.

constexpr int kTreeThreads = 128;
constexpr int kTreeWords = 32;
constexpr int kTreePitch = kTreeWords + 1;  // (a column's threads hit different banks)
constexpr int kStagedNodes = 2048;

__global__ void __launch_bounds__(kTreeThreads)
paged_tree_kernel(const __grid_constant__ PagedArgs a, const int32_t* parents, uint32_t* mask,
                  int64_t mask_stride, int32_t mask_words, int32_t* positions) {
  __shared__ int2 staged[kStagedNodes];  // parent and grandparent, -1: none
  __shared__ uint32_t bits[kTreeThreads * kTreePitch];
  wait_for_primary();
  const int32_t b = blockIdx.x, tid = threadIdx.x;
  const int32_t row0 = cu_at<kFresh>(a, b), n = cu_at<kFresh>(a, b + 1) - row0;
  const int32_t step = gridDim.y * kTreeThreads;
  if (int32_t(blockIdx.y) * kTreeThreads >= n) return;
  const int32_t past = seq_len_at<kFresh>(a, b) - n;
  const bool near = n <= kStagedNodes;
  bool odd = false;
  // the parent of a node, -1 for a root
  auto parent = [&](int32_t i) {
    const int32_t up = load_i32<kFresh>(parents + row0 + i);
    odd |= up >= i;
    return up < i && up >= 0 ? up : -1;
  };
  if (near) {
#pragma unroll 4
    for (int32_t i = tid; i < n; i += kTreeThreads) staged[i].x = parent(i);
    __syncthreads();
#pragma unroll 4
    for (int32_t i = tid; i < n; i += kTreeThreads) {
      const int32_t up = staged[i].x;
      staged[i].y = up >= 0 ? staged[up].x : -1;
    }
    __syncthreads();
  }
  for (int32_t i0 = blockIdx.y * kTreeThreads; i0 < n; i0 += step) {
    const int32_t i = i0 + tid;
    int32_t at = i < n ? i : -1, depth = -1;
    if (mask_words > 0 && at >> 5 >= mask_words) odd = true;
    // words [w0, w0 + 32) of these nodes, from the last ones down; without a mask one round
    const int32_t last = mask_words > 0 ? (mask_words - 1) / kTreeWords * kTreeWords : 0;
    for (int32_t w0 = last; w0 >= 0; w0 -= kTreeWords) {
      const int32_t words = min(mask_words - w0, kTreeWords), lo = 32 * w0;
      for (int32_t w = 0; w < words; ++w) bits[tid * kTreePitch + w] = 0;
      auto meet = [&](int32_t node) {
        const int32_t w = (node >> 5) - w0;
        if (w < words) atomicOr(&bits[tid * kTreePitch + w], 1u << (node & 31));
        ++depth;
      };
      if (near) {
        while (at >= lo) {
          const int2 up = staged[at];
          meet(at);
          at = up.x;
          if (at >= lo) {
            meet(at);
            at = up.y;
          }
        }
      } else {
        while (at >= lo) {
          meet(at);
          at = parent(at);
        }
      }
      if (words <= 0) continue;
      __syncthreads();
      // a row by as many lanes as the next power of two above its words
      const int32_t shift = words > 1 ? 32 - __clz(words - 1) : 0;
      const int32_t w = tid & ((1 << shift) - 1), rows = min(n - i0, kTreeThreads);
      uint32_t* out = mask + int64_t(row0 + i0) * mask_stride + w0 + w;
      if (w < words) {
#pragma unroll 4
        for (int32_t r = tid >> shift; r < rows; r += kTreeThreads >> shift) out[r * mask_stride] = bits[r * kTreePitch + w];
      }
      __syncthreads();
    }
    if (positions != nullptr && i < n) positions[row0 + i] = past + depth;
  }
  if (odd && a.status) atomicOr(a.status, SMLA_STATUS_INDEX_OOB);
}

// ---- the accepted path ----
//
// Record of node path[i] -> position past + i.  The path rises, so path[i] >= i: a
// record's new place is never that of a node that comes later in the path, and 32 steps
// of the path at a time may be moved one after the other, each batch read whole
// before it is written.  A block a sequence, a warp 4 records of a batch.  Bound: the chain path ->
// page -> record (64 trees of 60: 2.2 us, 7 of up to 500 with paths of up to 60: 2.9).

constexpr int kAcceptWarps = 8;
constexpr int kPerWarp = 32 / kAcceptWarps;
constexpr int kRecordChunks = kRecordBytes / 16;  // 41: a lane's one or two

__global__ void __launch_bounds__(32 * kAcceptWarps)
paged_accept_kernel(const __grid_constant__ PagedArgs a, const int32_t* path, int64_t path_stride,
                    int32_t path_len, int32_t* new_lens) {
  wait_for_primary();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int32_t b = blockIdx.x;
  const int32_t row0 = cu_at<kFresh>(a, b), n = max(cu_at<kFresh>(a, b + 1) - row0, 0);
  const int32_t past = seq_len_at<kFresh>(a, b) - n;  // (new_lens may be seq_lens)
  const int32_t* steps = path + int64_t(b) * path_stride;
  int32_t accepted = 0, before = -1;
  for (int32_t i0 = 0; i0 < path_len; i0 += 32) {
    // lane l: step i0 + l; the path ends at the first step that is no higher node
    const int32_t i = i0 + lane;
    const int32_t node = i < path_len ? load_i32<kFresh>(steps + i) : -1;
    int32_t last = __shfl_up_sync(0xffffffffu, node, 1);
    if (lane == 0) last = before;
    const uint32_t bad = __ballot_sync(0xffffffffu, node < 0 || node >= n || node <= last);
    const int32_t good = bad ? __ffs(bad) - 1 : 32;
    if (warp == 0 && lane == good && node >= 0 && a.status) atomicOr(a.status, SMLA_STATUS_INDEX_OOB);
    uint8_t* from = nullptr;
    uint8_t* to = nullptr;
    if (lane < good && node != i && lane / kPerWarp == warp) {
      from = record_at<kFresh>(a, b, past + node);
      to = record_at<kFresh>(a, b, past + i);
    }
    uint4 v[kPerWarp][2];
    uint8_t* dst[kPerWarp];
#pragma unroll
    for (int k = 0; k < kPerWarp; ++k) {
      const int src_lane = warp * kPerWarp + k;
      const uint8_t* src = reinterpret_cast<const uint8_t*>(
          __shfl_sync(0xffffffffu, reinterpret_cast<uint64_t>(from), src_lane));
      dst[k] = reinterpret_cast<uint8_t*>(__shfl_sync(0xffffffffu, reinterpret_cast<uint64_t>(to), src_lane));
      if (src == nullptr) dst[k] = nullptr;
      if (dst[k] == nullptr) continue;
      v[k][0] = *reinterpret_cast<const uint4*>(src + lane * 16);
      if (lane < kRecordChunks - 32) v[k][1] = *reinterpret_cast<const uint4*>(src + 512 + lane * 16);
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kPerWarp; ++k) {
      if (dst[k] == nullptr) continue;
      *reinterpret_cast<uint4*>(dst[k] + lane * 16) = v[k][0];
      if (lane < kRecordChunks - 32) *reinterpret_cast<uint4*>(dst[k] + 512 + lane * 16) = v[k][1];
    }
    accepted += good;
    if (good < 32) break;
    before = __shfl_sync(0xffffffffu, node, 31);
  }
  __syncthreads();  // (every thread has read the length)
  if (threadIdx.x == 0) new_lens[b] = max(past + accepted, 0);
}

}  // namespace

cudaError_t launch_paged_tree(const smla_paged_batch& b, const int32_t* parents, uint32_t* mask, int64_t mask_stride,
                              int32_t mask_words, int32_t* positions, cudaStream_t st) {
  const PagedArgs a = make_paged_args(b);
  // blocks beside each other for one sequence: one round for up to twice the mean of their
  // rows (7 trees of 125 to 500 nodes: 4.9 us, by the mean itself 7.0)
  const int64_t twice = 2 * ((b.n_rows + b.n_seqs - 1) / b.n_seqs);
  const int64_t split = (twice + kTreeThreads - 1) / kTreeThreads;
  const dim3 grid(unsigned(b.n_seqs), unsigned(split < 1024 ? split : 1024));
  return launch_dependent(paged_tree_kernel, grid, kTreeThreads, 0, st, a, parents, mask, mask_stride, mask_words, positions);
}

cudaError_t launch_paged_accept(const smla_paged_batch& b, const int32_t* path, int64_t path_stride, int32_t path_len,
                                int32_t* new_lens, cudaStream_t st) {
  const PagedArgs a = make_paged_args(b);
  return launch_dependent(paged_accept_kernel, dim3(unsigned(b.n_seqs)), 32 * kAcceptWarps, 0, st, a, path, path_stride,
                          path_len, new_lens);
}

}  // namespace smla
