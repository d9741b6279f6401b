// The paged cache as the device sees it: batch arguments, the sequence of a
// token row, the record of a position (see smla_paged_batch in smla.h).
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "smla_internal.h"

namespace smla {

struct PagedArgs {
  uint8_t* kv;
  int64_t n_pages, page_stride;
  const int32_t* table;
  int64_t table_stride;
  const int32_t* cu;
  const int32_t* seq_lens;
  int32_t* status;
  int32_t n_rows, n_seqs;
  int32_t page_size, max_pages;
  uint32_t page_mul, page_sh1, page_sh2;  // position / page_size by a multiplication
};

// n / d for 32-bit n and a d known on the host (Granlund and Montgomery's
// round-up method): q = (t + ((n - t) >> sh1)) >> sh2, t = hi32(mul * n).
inline void make_divider(uint32_t d, uint32_t* mul, uint32_t* sh1, uint32_t* sh2) {
  uint32_t l = 0;
  while (l < 32 && (uint64_t(1) << l) < d) ++l;  // ceil(log2 d)
  *mul = uint32_t(((uint64_t(1) << 32) * ((uint64_t(1) << l) - d)) / d + 1);
  *sh1 = l < 1 ? l : 1;
  *sh2 = l > 0 ? l - 1 : 0;
}

inline PagedArgs make_paged_args(const smla_paged_batch& b) {
  PagedArgs a{};
  a.kv = static_cast<uint8_t*>(b.kv_cache);
  a.n_pages = b.n_pages;
  a.page_stride = b.page_stride;
  a.table = b.block_table;
  a.table_stride = b.block_table_stride;
  a.cu = b.cu_rows;
  a.seq_lens = b.seq_lens;
  a.status = b.status;
  a.n_rows = int32_t(b.n_rows);
  a.n_seqs = b.n_seqs;
  a.page_size = b.page_size;
  a.max_pages = b.max_pages;
  make_divider(uint32_t(b.page_size), &a.page_mul, &a.page_sh1, &a.page_sh2);
  return a;
}

// ---- launch order ----
//
// Short kernels are launched as dependents of whatever is before them in the stream: they may
// be placed while that ends, and wait for all of it, and for its memory, before they
// read or write anything.  Every thread waits, also one without work: a grid's end then
// always means the end of those before it.  It saves 0.3 to 0.5 us of calls that take 2.5
// to 3.  (Letting the next one be placed at their start saves no more; attend kernels
// launched so were no faster, the largest 4% slower.)
__device__ __forceinline__ void wait_for_primary() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

template <typename... Params, typename... Args>
inline cudaError_t launch_dependent(void (*kernel)(Params...), dim3 grid, int threads, size_t smem, cudaStream_t stream,
                                    const Args&... args) {
  return launch_kernel(true, kernel, grid, unsigned(threads), smem, stream, args...);
}

// How a batch's arrays are read.  The read-only path is for memory that nothing writes while the
// kernel is resident, which a dependent may be while the kernel before it still writes
// (lengths by an accept, positions and masks by a tree, any of them by a copy of the user's):
// dependents load past it, behind their wait (both are volatile).
enum Loads { kReadOnly, kFresh };

template <Loads kLoads>
__device__ __forceinline__ int32_t load_i32(const int32_t* p) {
  if constexpr (kLoads == kReadOnly) return __ldg(p);
  int32_t v;
  asm volatile("ld.global.b32 %0, [%1];" : "=r"(v) : "l"(__cvta_generic_to_global(p)));
  return v;
}
__device__ __forceinline__ uint64_t load_fresh_u64(const uint64_t* p) {
  uint64_t v;
  asm volatile("ld.global.b64 %0, [%1];" : "=l"(v) : "l"(__cvta_generic_to_global(p)));
  return v;
}

__device__ __forceinline__ uint32_t page_of(const PagedArgs& a, uint32_t pos) {
  const uint32_t t = __umulhi(a.page_mul, pos);
  return (t + ((pos - t) >> a.page_sh1)) >> a.page_sh2;
}

// cu_rows[b] clamped to the token tensors' rows.
template <Loads kLoads = kReadOnly>
__device__ __forceinline__ int32_t cu_at(const PagedArgs& a, int32_t b) {
  const int32_t v = load_i32<kLoads>(a.cu + b);
  return v < 0 ? 0 : v > a.n_rows ? a.n_rows : v;
}

// Length of sequence b, at least 0.
template <Loads kLoads = kReadOnly>
__device__ __forceinline__ int32_t seq_len_at(const PagedArgs& a, int32_t b) {
  return max(load_i32<kLoads>(a.seq_lens + b), 0);
}

// Record of position pos of sequence b, or nullptr when it is masked (page ids
// >= n_pages and positions past the table are flagged).
template <Loads kLoads = kReadOnly>
__device__ __forceinline__ uint8_t* record_at(const PagedArgs& a, int32_t b, int32_t pos) {
  if (pos < 0) return nullptr;
  const uint32_t page = page_of(a, uint32_t(pos));
  if (page >= uint32_t(a.max_pages)) {
    if (a.status) atomicOr(a.status, SMLA_STATUS_INDEX_OOB);
    return nullptr;
  }
  const int32_t id = load_i32<kLoads>(a.table + int64_t(b) * a.table_stride + page);
  if (id < 0) return nullptr;
  if (id >= a.n_pages) {
    if (a.status) atomicOr(a.status, SMLA_STATUS_INDEX_OOB);
    return nullptr;
  }
  return a.kv + int64_t(id) * a.page_stride + int64_t(uint32_t(pos) - page * uint32_t(a.page_size)) * kRecordBytes;
}

// The last sequence b with cu_rows[b] <= r (0 if there is none), found by the
// whole warp: each step looks at 32 boundaries, so that 1024 sequences take
// two loads one after the other instead of a binary search's ten.
template <Loads kLoads = kReadOnly>
__device__ __forceinline__ int32_t seq_of_row(const PagedArgs& a, int32_t r) {
  const int lane = threadIdx.x & 31;
  int32_t lo = 0, n = a.n_seqs;
  while (n > 1) {
    const int32_t step = (n + 31) >> 5;
    const int32_t off = lane * step;
    const bool in = off < n && load_i32<kLoads>(a.cu + lo + off) <= r;
    const int32_t cnt = __popc(__ballot_sync(0xffffffffu, in));
    if (cnt == 0) return lo;
    lo += (cnt - 1) * step;
    n = min(step, n - (cnt - 1) * step);
  }
  return lo;
}

}  // namespace smla
