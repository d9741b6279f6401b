// Attention of new tokens over the paged cache (smla_paged_attend): chunks of a
// prompt, drafted tokens, single tokens.
//
// For token row r at position p and head h, over the visible positions t,
//   s_t = sm_scale q . k_t (576 dims),  out = sum_t e^(s_t - m) v_t / (sum_t e^(s_t - m) + e^(sink - m)),
// v_t the latent 512 dims of k_t.  All heads of all tokens of a sequence share
// its keys, so (token, head) pairs are the rows of two matrix products:
//   S[128, 64] = Q[128, 576] . K[64, 576]^T,   O[128, 512] += P[128, 64] . V[64, 512].
//
// Three kernels, by the mean number of rows of a sequence (narrow_rows): the pair
// kernel described here for chunks and drafts, further down the narrow kernel for up to
// 64 rows and the few-row kernel for up to 16.
//
// Row tiles.  A row tile is floor(128 / heads) consecutive tokens of one
// sequence with all their heads.  Its keys are the positions up to its last
// token's, in tiles of 64.
//
// CTA pairs.  An f32 accumulator of 128 x 512 alone fills the 512 TMEM columns
// of an SM, so a row tile belongs to a cluster of two CTAs and the products are
// cta_group::2 instructions with M = 128: CTA c holds rows [64 c, 64 c + 64) of
// Q, P, S and O (64 rows on 128 lanes: lanes 64.. hold the upper half of the
// columns), which takes 256 columns for O and 64 per S buffer (the two issuers'
// halves of the K-steps, 32 columns each).  As B operands each CTA supplies half
// of the N extent: its own 32 keys of the tile for QK ("K": 32 x 576), and its own
// 256 value dims of all 64 keys for PV ("V": 64 x 256, MN-major).  Every record is
// read and dequantised once, by the CTA that owns the key, into K; bulk copies
// take K's latent blocks to the V of the CTA that needs them, its own or its
// peer's (both are 128-byte-swizzled rows of 64 dims, so a 32-key block is one
// contiguous piece of 4 KB).
//
// Warps (16): 0-3 softmax and epilogue, 4-11 loaders, 12-14 issue MMAs (even CTA
// only), 15 copier.  Per tile g (stage g & 1):
//   loaders   two groups of four warps take turns at the tiles, a warp 8 of the
//             CTA's 32 keys: records into registers, dequantised there, and as soon
//             as QK(g - 2) and the copies out of its K are done, stored.  What a
//             stage waits for after that is the stores alone
//   copier    one thread: K -> V of both CTAs when PV(g - 2) is done
//   issuers   12 and 13 the even and odd K-steps of QK into two accumulators, 14
//             PV: one thread's MMAs of N = 64 follow each other at 48 cycles or
//             more, two threads' at half of that
//   softmax   a row is two threads (32 keys each) that exchange their maxima;
//             p = 2^(x - m_ref), the reference moves (and O is rescaled in TMEM)
//             only when a score exceeds it by more than 8, so p <= 2^8
//
// What bounds the pair kernel: shared memory.  A tile of 64 keys takes ~2420 cycles,
// in which the operands' reads (1248), the loaders' and softmax warps' accesses (579)
// and the bulk copies (512) keep its port busy for ~2340.  One chunk of 2048 tokens,
// 64 heads, after 8192 earlier positions: 2467 us = 1065 TFLOP/s, 56% of the measured
// bf16 peak; 7 chunks of up to 300 tokens, 16 heads, up to 4927 positions: 225 us.
// A tile of the pair takes 1.23 us when it has 128 rows of one token (128 heads).
//
// Schedule.  A row tile takes a few slots for its start (kPairStart and so on: what
// a unit's first tile and last store take, in key tiles) and one per key tile; the
// slots of all row tiles, in order, are split evenly over the workers (worker c of
// G takes [c W / G, (c + 1) W / G)).  A row tile inside one worker's range is
// finished there; a shared one leaves f32 partials (O, m, l) that a merge kernel
// joins.
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "smla_device.cuh"
#include "smla_internal.h"
#include "smla_paged.cuh"
#include "smla_ptx.cuh"

namespace smla {

// Limit of every pipeline wait in ns (0: the default), and whether the first
// softmax wait of each CTA is on a barrier that nothing signals (a test of the
// timeout path); read at kernel start.
__device__ uint64_t g_paged_wait_ns;
__device__ int32_t g_paged_stall;

namespace {

using namespace ptx;

constexpr int kTileKeys = 64;
constexpr int kOwnKeys = 32;      // keys of a tile that one CTA of the pair loads
constexpr int kPairRows = 128;
constexpr int kCtaRows = 64;
constexpr int kLoaderWarps = 4;   // of each of the two loader groups
constexpr int kKeysPerWarp = kOwnKeys / kLoaderWarps;
constexpr int kFirstLoader = 4;
constexpr int kIssuerQk = 12;  // and 13
constexpr int kIssuerPv = 14;
constexpr int kCopier = 15;
constexpr int kAttendThreads = 16 * 32;
constexpr int kStageK = 9 * kOwnKeys * 128;   // nine 64-dim blocks of 128-byte rows
constexpr int kStageV = 4 * kTileKeys * 128;  // four 64-dim blocks
constexpr int kVBlock = kTileKeys * 128;
constexpr int kOffK = 0;
constexpr int kOffV = kOffK + 2 * kStageK;
constexpr int kOffQ = kOffV + 2 * kStageV;
constexpr int kQBlock = kCtaRows * 128;
constexpr int kOffP = kOffQ + 9 * kQBlock;
constexpr int kOffMisc = kOffP + kCtaRows * 128;
// narrow and few-row kernel: K of all keys of a tile, in two stages; V is the same
// memory.  The few-row kernel keeps Q in tensor memory and takes tiles of 96 keys.
constexpr int kQRowPitch = kQK * 2 / 3 + 16;
template <int kN>
struct Narrow {
  static constexpr bool kFew = kN == 16;
  static constexpr int kKeys = kFew ? 96 : kTileKeys;  // of a tile
  static constexpr int kLoaders = kKeys / 8;
  static constexpr int kBlock = kKeys * 128;           // a 64-dim block of a tile
  static constexpr int kStage = 9 * kBlock;
  static constexpr int kOffQ = 2 * kStage;
  static constexpr int kOffP = kOffQ + (kFew ? 0 : 9 * kQBlock);
  static constexpr int kOffMisc = kOffP + (kFew ? 16 * kQRowPitch + 256 : kN * 128);  // (P of 4 KB, q on its way)
};
constexpr uint32_t kTmemQFew = 64, kTmemSFew = kTmemQFew + kQK / 2;  // behind O's 64 columns
constexpr int kNarrowThreads = 16 * 32;
constexpr int kNarrowQk = 12;  // and 13
constexpr int kNarrowPv = 14;  // and 15
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kTmemS = 256;              // the S buffers, behind O's 256 columns
// Slots of a row tile's start, by measurement (us): the pair kernel with 1 / 4 / 8 / 12
// at 32 drafts of 5 tokens, 64 heads: 88 / 80 / 76 / 76; the narrow kernel with 1 / 2 / 4
// at 4 x 64 heads: 43.7 / 42.2 / 41.3, at 64 x 64 heads over 4096: 88.2 / 86.4 / 87.9; the
// few-row kernel with 1 / 2 / 4 at 64 x 16 heads: 53.5 / 53.2 / 51.8.
constexpr int kPairStart = 8, kNarrowStart = 2, kFewStart = 4;
constexpr float kMoveMargin = 8.f;            // log2 units; p <= 2^8
constexpr uint64_t kWaitNs = 2000000000ull;
constexpr uint32_t kIdescQK = idesc_bf16(kPairRows, kTileKeys, 0, 0);
constexpr uint32_t kIdescPV = idesc_bf16(kPairRows, 256, 0, 1);

struct AttendArgs {
  PagedArgs b;
  const uint16_t* q;
  int64_t q_row, q_head;
  uint16_t* out;
  int64_t o_row, o_head;
  float* lse;
  const float* sink;
  float scale_log2;
  int32_t heads, tokens, causal;  // tokens: of a row tile
  int32_t workers;                // pairs of CTAs, or CTAs of the other kernels
  int32_t part_rows;              // rows of a partial: 128, or 64
  int32_t coverage;               // positions the block table can hold
  int32_t start_slots;            // slots of a row tile's start
  float* o_part;                  // [2 workers][part_rows][512]
  float* ml_part;                 // [2 workers][part_rows][2]
  int32_t* merge;                 // [workers][4]: rows to merge (0: none), first token row, first worker
};

struct Misc {
  uint64_t k_full[2], q_full, p_full, s_empty[2];  // used in the even CTA
  uint64_t k_ready[2], v_land[2], v_full[2];
  uint64_t qk_done[2], pv_done[2], drain, never;
  uint32_t tmem;
  int32_t dead;
  uint64_t wait_ns;
  int32_t stall;
  int32_t first_seq, first_j;
  int64_t first_slot, beg, end, total;
  int64_t warp_sum[16];
  float tmax[2][128];
  float lsum[128];
  float alpha[2][kCtaRows], factor[kCtaRows];  // narrow kernel: per row
  // per tile: a byte per 8 keys, bit: a key before the end that has no record
  uint8_t flags[4][kTileKeys / 8];
  uint8_t flags_few[4][16];  // few-row kernel: 12 are used
};
constexpr int kAttendSmem = kOffMisc + int(sizeof(Misc));
template <int kN>
constexpr int kNarrowSmem = Narrow<kN>::kOffMisc + int(sizeof(Misc));
static_assert(kAttendSmem <= 232448 && kNarrowSmem<16> <= 232448 && kNarrowSmem<64> <= 232448, "shared memory of a CTA");

// ---- launch order ----

// The merge kernel is launched as a dependent of the attend kernel: its blocks may
// be placed as soon as those of the attend kernel leave, and wait there for all of
// it to be complete.
__device__ __forceinline__ void let_dependents_launch() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_for_primary() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// ---- cluster helpers ----

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}

__device__ __forceinline__ uint32_t map_to(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// Arrives on a barrier of either CTA.  What it announces lies in this SM's own
// shared or tensor memory (and, for shared memory, a proxy fence came before), so
// no release at cluster scope is made: that would cost ~1000 cycles each time.
__device__ __forceinline__ void arrive_at(uint32_t mapped_bar) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(mapped_bar) : "memory");
}

// Whether the phase of `bar` is complete, without waiting.
__device__ __forceinline__ bool mbar_test(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}

// Copy of `bytes` from this CTA's shared memory to either CTA's, completing on
// the barrier there.
__device__ __forceinline__ void bulk_s2s(uint32_t mapped_dst, uint32_t src, uint32_t bytes, uint32_t mapped_bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.shared::cta.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(mapped_dst),
      "r"(src), "r"(bytes), "r"(mapped_bar)
      : "memory");
}

__device__ __forceinline__ void st_shared_v4(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}

__device__ __forceinline__ void mma2(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}

// A from tensor memory.
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}

// Two f32 operations in one instruction.
__device__ __forceinline__ void add2(float a0, float a1, float b0, float b1, float& r0, float& r1) {
  asm("{\n\t.reg .b64 a, b, r;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
      "add.rn.f32x2 r, a, b;\n\tmov.b64 {%0, %1}, r;\n\t}"
      : "=f"(r0), "=f"(r1)
      : "f"(a0), "f"(a1), "f"(b0), "f"(b1));
}
__device__ __forceinline__ void add2(uint32_t a0, uint32_t a1, uint32_t b0, uint32_t b1, float& r0, float& r1) {
  add2(__uint_as_float(a0), __uint_as_float(a1), __uint_as_float(b0), __uint_as_float(b1), r0, r1);
}
// r = x * m + c
__device__ __forceinline__ void fma2(float x0, float x1, float m, float c, float& r0, float& r1) {
  asm("{\n\t.reg .b64 x, m, c, r;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 m, {%4, %4};\n\tmov.b64 c, {%5, %5};\n\t"
      "fma.rn.f32x2 r, x, m, c;\n\tmov.b64 {%0, %1}, r;\n\t}"
      : "=f"(r0), "=f"(r1)
      : "f"(x0), "f"(x1), "f"(m), "f"(c));
}

// One lane of the converged warp.  What it runs alone stays uniform to the
// compiler (unlike a branch on the thread index), so that an MMA's descriptors are
// made in uniform registers: issuing one then takes 33 cycles, not 83.
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(r));
  return r != 0;
}

// Arrives once on `bar` of both CTAs when the MMAs issued so far are complete.
__device__ __forceinline__ void commit2(uint64_t* bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
          smem_u32(bar)),
      "h"(uint16_t(3))
      : "memory");
}

// Gives up the pipeline of both CTAs (see wait_for).
__device__ __noinline__ void give_up(Misc* ms, int32_t* status) {
  if (atomicExch(&ms->dead, 1) == 0 && status) atomicOr(status, SMLA_STATUS_TIMEOUT);
  uint32_t ctas;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(ctas));
  if (ctas == 2) {
    const uint32_t other = map_to(smem_u32(&ms->dead), cluster_rank() ^ 1u);
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(other), "r"(1) : "memory");
  }
}

// Waits for the phase of `bar`; false after the limit, or once the pair has
// given up.  (Out of line, like everything that a tile does not go through: the
// roles' loops compete for the instruction cache.)
__device__ __noinline__ bool wait_on(Misc* ms, int32_t* status, uint64_t* bar, uint32_t parity) {
  uint64_t t0 = 0;
  for (uint32_t i = 0;; ++i) {
    if ((i & 63u) == 0) {
      if (*reinterpret_cast<volatile int32_t*>(&ms->dead)) return false;
      const uint64_t t = globaltimer();
      if (t0 == 0) t0 = t;
      if (t - t0 > ms->wait_ns) {
        give_up(ms, status);
        return false;
      }
    }
    if (mbar_try_wait(bar, parity)) return true;
  }
}

__device__ __forceinline__ bool wait_for(Misc* ms, const AttendArgs& a, uint64_t* bar, uint32_t parity) {
  return mbar_try_wait(bar, parity) || wait_on(ms, a.b.status, bar, parity);
}

// The same for a whole warp: one answer for all lanes.
__device__ __forceinline__ bool warp_wait(Misc* ms, const AttendArgs& a, uint64_t* bar, uint32_t parity) {
  return __all_sync(0xffffffffu, wait_for(ms, a, bar, parity));
}

// The same for a warp that goes on in any case (its role ends with the last tile, also
// after a wait that gave up).  Lanes may leave the wait's loop at different turns, and
// what follows are accesses of tensor memory by the whole warp, so they meet here.
__device__ __forceinline__ void meet_after(Misc* ms, const AttendArgs& a, uint64_t* bar, uint32_t parity) {
  wait_for(ms, a, bar, parity);
  __syncwarp();
}

// A barrier of some of the block's warps, which lanes may reach from branches of
// their own: the instruction itself wants the warp converged.
__device__ __forceinline__ void group_barrier(uint32_t id, uint32_t threads) {
  __syncwarp();
  named_barrier(id, threads);
}

// ---- the schedule ----

// sum_{i < n} floor((g i + b) / 64) for g, b >= 0: the plain sum less the residues
// modulo 64, which repeat every 64 / gcd(g, 64) terms as b mod gcd, + gcd, ...
__device__ __forceinline__ int64_t tile_sum(int32_t n, int32_t g, int32_t b) {
  const int32_t gcd = min(g & -g, kTileKeys), shift = __popc(kTileKeys / gcd - 1), period = 1 << shift;
  int64_t residues = int64_t(n >> shift) * (period * (b & (gcd - 1)) + gcd * (period * (period - 1) / 2));
  int32_t r = b & (kTileKeys - 1), rest = 0;
  for (int32_t i = n & (period - 1); i > 0; --i) {
    rest += r;
    r = (r + g) & (kTileKeys - 1);
  }
  return (int64_t(n) * b + int64_t(n) * (n - 1) / 2 * g - residues - rest) / kTileKeys;
}

// n / d for n >= 0, d > 0; most are of 32 bits, in a fraction of the time.
__device__ __forceinline__ int64_t div_up_to_64(int64_t n, int64_t d) {
  if (((n | d) >> 32) == 0) return int64_t(uint32_t(n) / uint32_t(d));
  return n / d;
}

// What a sequence needs for its row tiles.
struct Seq {
  int32_t row0, rows;  // its token rows
  int32_t past;        // position of the first one (negative: rows before the sequence's start)
  int32_t tiles;       // row tiles
};

__device__ __forceinline__ Seq seq_at(const AttendArgs& a, int32_t b) {
  Seq s;
  s.row0 = cu_at(a.b, b);
  const int32_t end = cu_at(a.b, b + 1);
  s.rows = max(end - s.row0, 0);
  s.past = seq_len_at(a.b, b) - s.rows;
  s.tiles = (s.rows + a.tokens - 1) / a.tokens;
  return s;
}

// End of the visible positions of row tile j: its last token's, within the table.
__device__ __forceinline__ int32_t keys_end(const AttendArgs& a, const Seq& s, int32_t j) {
  const int32_t last = a.causal ? min((j + 1) * a.tokens, s.rows) : s.rows;
  return max(min(s.past + last, a.coverage), 0);
}

__device__ __forceinline__ int32_t key_tiles(int32_t end) { return max((end + kTileKeys - 1) / kTileKeys, 1); }

// Slots of the sequence's first j row tiles.
__device__ int64_t slots_before(const AttendArgs& a, const Seq& s, int32_t j) {
  if (j <= 0) return 0;
  if (!a.causal) return int64_t(j) * (a.start_slots + key_tiles(keys_end(a, s, 0)));
  if (j == 1) return a.start_slots + key_tiles(keys_end(a, s, 0));
  int64_t sum = int64_t(j) * a.start_slots;
  const int32_t n = min(j, s.tiles - 1);  // tiles that end at past + tokens (i + 1)
  if (j == s.tiles) sum += key_tiles(keys_end(a, s, j - 1));
  // tiles [0, lo) have one key tile, [lo, hi) follow the line, [hi, n) end at the table's end
  const int32_t G = a.tokens, P = s.past, C = a.coverage;
  int32_t lo = P <= kTileKeys ? min((kTileKeys - P) / G, n) : 0, hi = n;
  if (P > C - s.rows) hi = P < C ? max(min(int32_t((uint32_t(C - P) + uint32_t(G - 1)) / uint32_t(G)) - 1, n), lo) : lo;
  sum += lo;
  if (hi > lo) sum += tile_sum(hi - lo, G, P + G * (lo + 1) + kTileKeys - 1);
  sum += int64_t(n - hi) * key_tiles(C);
  return sum;
}

// A row tile's part that this worker works on.
struct Unit {
  int32_t seq, row0, tokens;  // its first token row and number of tokens
  int32_t pos0;               // position of that token
  int32_t end;                // end of its visible positions
  int32_t t0, t1, tiles;      // key tiles [t0, t1) of `tiles`
  int64_t slot;               // that of key tile 0
};

struct Units {
  int64_t slot, beg, end;
  int32_t seq, j;
  Seq s;

  __device__ __forceinline__ void start(const AttendArgs& a, const Misc* ms) {
    slot = ms->first_slot;
    beg = ms->beg;
    end = ms->end;
    seq = ms->first_seq;
    j = ms->first_j;
    s.tiles = 0;
    if (slot < end && seq < a.b.n_seqs) s = seq_at(a, seq);
  }

  // The next unit of this worker; false when there is none.
  __device__ __noinline__ bool next(const AttendArgs& a, Unit& u) { return next_inline(a, u); }

  __device__ __forceinline__ bool next_inline(const AttendArgs& a, Unit& u) {
    while (slot < end && seq < a.b.n_seqs) {
      if (j >= s.tiles) {
        // the next sequence; from an empty one in doubling steps, over boundaries that are
        // not above its own (one by one, 2^10 empty sequences between two others took the
        // pair kernel from 46 to 974 us)
        j = 0;
        ++seq;
        for (int32_t step = 1; s.tiles == 0 && seq + step <= a.b.n_seqs && cu_at(a.b, seq + step) <= s.row0; step *= 2)
          seq += step;
        if (seq < a.b.n_seqs) s = seq_at(a, seq);
        continue;
      }
      u.seq = seq;
      u.row0 = s.row0 + j * a.tokens;
      u.tokens = min(a.tokens, s.rows - j * a.tokens);
      u.pos0 = s.past + j * a.tokens;
      u.end = keys_end(a, s, j);
      u.tiles = key_tiles(u.end);
      slot += a.start_slots;
      u.slot = slot;
      u.t0 = int32_t(max(beg - slot, int64_t(0)));
      u.t1 = int32_t(max(min(end - slot, int64_t(u.tiles)), int64_t(0)));
      slot += u.tiles;
      ++j;
      if (u.t0 < u.t1) return true;
    }
    return false;
  }
};

// The worker's range of slots and the row tile it starts in, by all threads.
template <int kThreads>
__device__ __forceinline__ void find_range(const AttendArgs& a, Misc* ms, int32_t worker) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int32_t per = (a.b.n_seqs + kThreads - 1) / kThreads;
  const int32_t s0 = min(tid * per, a.b.n_seqs), s1 = min(s0 + per, a.b.n_seqs);
  int64_t sum = 0;
  for (int32_t s = s0; s < s1; ++s) {
    const Seq q = seq_at(a, s);
    sum += slots_before(a, q, q.tiles);
    if (worker == 0 && q.rows > 0 && q.past > a.coverage - q.rows && a.b.status)  // positions past the table
      atomicOr(a.b.status, SMLA_STATUS_INDEX_OOB);
  }
  int64_t inc = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t v = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += v;
  }
  if (lane == 31) ms->warp_sum[warp] = inc;
  __syncthreads();
  int64_t before = inc - sum, total = 0;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) {
    const int64_t v = ms->warp_sum[w];
    if (w < warp) before += v;
    total += v;
  }
  const int64_t G = max(min(int64_t(a.workers), total), int64_t(1));
  const int64_t beg = worker < G ? div_up_to_64(worker * total, G) : total;
  const int64_t end = worker < G ? div_up_to_64((worker + 1) * total, G) : total;
  if (tid == 0) {
    ms->beg = beg;
    ms->end = end;
    ms->total = total;
    if (beg >= end) ms->first_slot = end;  // nothing to do
  }
  if (beg < end && before <= beg && beg < before + sum) {
    int64_t slot = before;
    int32_t s = s0;
    Seq q = seq_at(a, s);
    int64_t n = slots_before(a, q, q.tiles);
    while (slot + n <= beg) {
      slot += n;
      q = seq_at(a, ++s);
      n = slots_before(a, q, q.tiles);
    }
    ms->first_seq = s;
    ms->first_slot = slot;
  }
  __syncthreads();
  // the last row tile of that sequence that starts at or before beg: each step looks
  // at 32 of them
  if (warp == 0 && beg < end) {
    const Seq q = seq_at(a, ms->first_seq);
    const int64_t at = beg - ms->first_slot;
    int32_t lo = 0, n = q.tiles;
    while (n > 1) {
      const int32_t step = (n + 31) >> 5, off = lane * step;
      const bool in = off < n && slots_before(a, q, lo + off) <= at;
      const int32_t last = __popc(__ballot_sync(0xffffffffu, in)) - 1;
      lo += last * step;
      n = min(step, n - last * step);
    }
    __syncwarp();
    if (lane == 0) {
      ms->first_j = lo;
      ms->first_slot += slots_before(a, q, lo);
    }
  }
}

// ---- dequantisation ----

// Two E4M3 codes (bytes of w picked by sel into the lower byte of each half) as
// bf16x2 of value * 2^-120: sign, exponent and mantissa are moved into place,
//   16 m + 256 (x - m) = 256 x - 240 m,  m = x & 0x7F,
// by multiplications, since the shifts and logic of the usual form alone keep
// the ALU pipe busy longer than the tensor work of a tile lasts; an exact product
// with scale * 2^120 does the rest (subnormals included).
__device__ __forceinline__ uint32_t place2(uint32_t w, uint32_t sel) {
  const uint32_t x = __byte_perm(w, 0, sel);
  uint32_t y;
  asm("{\n\t.reg .u32 t;\n\tmul.lo.u32 t, %2, 0xFFFFFF10;\n\tmad.lo.u32 %0, %1, 256, t;\n\t}"
      : "=r"(y)
      : "r"(x), "r"(x & 0x007F007Fu));
  return y;
}

__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// Eight codes by one scale factor (a bf16x2 pair).
__device__ __forceinline__ void dequant8(const uint2& c, uint32_t mul2, uint32_t (&v)[4]) {
  v[0] = mul_bf16x2(place2(c.x, 0x4140), mul2);
  v[1] = mul_bf16x2(place2(c.x, 0x4342), mul2);
  v[2] = mul_bf16x2(place2(c.y, 0x4140), mul2);
  v[3] = mul_bf16x2(place2(c.y, 0x4342), mul2);
}

// Running OR that has an upper bit of a byte set once a NaN code (0x7F or 0xFF)
// was met.
__device__ __forceinline__ uint32_t nan_codes(const uint2& c, uint32_t top) {
  return top | ((c.x & 0x7F7F7F7Fu) + 0x01010101u) | ((c.y & 0x7F7F7F7Fu) + 0x01010101u);
}

// Zero if a block scale takes the fast path: a power of two in [2^-120, 2^7]
// (scale * 2^120 is then a normal bf16 power of two).
__device__ __forceinline__ uint32_t odd_scale(uint32_t bits) { return (bits - (7u << 23)) & 0xC07FFFFFu; }

// The general form: bf16(e4m3 * scale), values that are not finite become zero
// and are reported.
struct Dequant8 {
  uint32_t v[4];
  uint32_t bad;
};
__device__ __noinline__ Dequant8 dequant8_any(uint32_t c0, uint32_t c1, uint32_t scale_bits) {
  const float scale = __uint_as_float(scale_bits);
  Dequant8 r;
  r.bad = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t w = i < 2 ? c0 : c1;
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(__nv_fp8x2_storage_t(w >> (16 * (i & 1))), __NV_E4M3);
    float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
    f.x = __bfloat162float(__float2bfloat16_rn(f.x * scale));
    f.y = __bfloat162float(__float2bfloat16_rn(f.y * scale));
    if (!isfinite(f.x)) f.x = 0.f, r.bad = 1;
    if (!isfinite(f.y)) f.y = 0.f, r.bad = 1;
    r.v[i] = pack_bf16x2(f.x, f.y);
  }
  return r;
}

__device__ __forceinline__ uint2 ldg_v2_now(const void* p) {
  uint2 v;
  asm volatile("ld.global.nc.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(__cvta_generic_to_global(p)));
  return v;
}

// One tile's records of a loader warp, in flight or landed.  Lane l holds the
// codes of dims [256 i + 8 l, + 8): a 16-byte chunk of bf16 each, and eight
// neighbouring lanes fill a 128-byte row of K or V.
struct Raw {
  uint2 lat[kKeysPerWarp][2];
  uint32_t scale[kKeysPerWarp][2];
  uint4 rope[2];  // lane l: 16 bytes of the rope of records l / 8 and 4 + l / 8
};

__device__ __forceinline__ void load_record(const uint8_t* p, int j, Raw& r) {
  const int lane = threadIdx.x & 31;
  r.lat[j][0] = ldg_v2_now(p + lane * 8);
  r.lat[j][1] = ldg_v2_now(p + lane * 8 + 256);
  r.scale[j][0] = ldg_u32_now(p + kScaleOffset + 4 * (lane >> 4));
  r.scale[j][1] = ldg_u32_now(p + kScaleOffset + 4 * (lane >> 4) + 8);
}

// The loads of records anywhere (rec: lane j's, 0: none, read as zeros).
__device__ __forceinline__ Raw load_scattered(uint64_t rec) {
  const int lane = threadIdx.x & 31;
  Raw r;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint64_t p = __shfl_sync(0xffffffffu, rec, 4 * i + (lane >> 3));
    r.rope[i] = make_uint4(0, 0, 0, 0);
    if (p) r.rope[i] = ldg_v4_now(reinterpret_cast<const uint8_t*>(p) + kRopeOffset + (lane & 7) * 16);
  }
#pragma unroll
  for (int j = 0; j < kKeysPerWarp; ++j) {
    const uint64_t p = __shfl_sync(0xffffffffu, rec, j);
    r.lat[j][0] = r.lat[j][1] = make_uint2(0, 0);
    r.scale[j][0] = r.scale[j][1] = 0x3F800000u;  // zeros by the fast path
    if (p) load_record(reinterpret_cast<const uint8_t*>(p), j, r);
  }
  return r;
}

// The same out of line, for the pair's loaders, whose registers are all taken
// (inline there: 248 -> 279 us at 7 chunks of 300; the call costs pages of one record
// 288 us where pages of a multiple of 8 take 222).
__device__ __noinline__ Raw load_scattered_call(uint64_t rec) { return load_scattered(rec); }

// Starts the copies of a unit's q rows of this CTA, zeros behind them, `copies`
// times over the 64 rows, by `warps` warps (w: which).  Eight lanes take a row, one
// of its 16-byte chunks in each of the nine blocks, so that all nine addresses are
// one plus constants.
__device__ __noinline__ void load_q(const AttendArgs& a, uint32_t q_at, uint32_t rank, int w, int warps, int32_t row0,
                                    int32_t rows, int copies) {
  const int lane = threadIdx.x & 31;
  for (int i = 4 * w + (lane >> 3); i < kCtaRows; i += 4 * warps) {
    const int32_t m = int32_t(rank) * kCtaRows + i % (kCtaRows / copies);
    const uint32_t dst = q_at + i * 128 + (((lane ^ i) & 7) << 4);
    if (m < rows) {
      const int32_t tok = m / a.heads;
      const uint16_t* src = a.q + int64_t(row0 + tok) * a.q_row + int64_t(m - tok * a.heads) * a.q_head + (lane & 7) * 8;
#pragma unroll
      for (int b = 0; b < kQK / 64; ++b) cp_async16(dst + b * kQBlock, src + b * 64);
    } else {
#pragma unroll
      for (int b = 0; b < kQK / 64; ++b) st_shared_v4(dst + b * kQBlock, 0, 0, 0, 0);
    }
  }
}

// The end of load_q's copies: the caller may announce them after it.
__device__ __forceinline__ void finish_q() {
  cp_async_wait_all();
  fence_proxy_async_smem();
  __syncwarp();
}

// q of a unit's up to 16 rows into tensor memory, 32 lanes by each of four warps: lane
// l gets row l % 16, so that S has all rows wherever a softmax warp looks for them.
// The rows are loaded whole by the 128 threads together and change hands in shared
// memory, a third at a time (each lane loading its own row took 4 us).
__device__ __noinline__ void load_q_tmem(const AttendArgs& a, uint32_t buf, uint32_t at, int32_t row0, int32_t rows) {
  constexpr int kThird = kQK / 8 / 3, kEach = 16 * kThird / 128;  // 16-byte chunks of a row's third, of a thread
  uint4 v[3][kEach];
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    const int32_t j = threadIdx.x + 128 * i, m = j / kThird, tok = m / a.heads;
    const uint16_t* src = a.q + int64_t(row0 + tok) * a.q_row + int64_t(m - tok * a.heads) * a.q_head + (j - m * kThird) * 8;
#pragma unroll
    for (int third = 0; third < 3; ++third) {
      v[third][i] = make_uint4(0, 0, 0, 0);
      if (m < rows) v[third][i] = ldg_v4_now(src + third * kThird * 8);
    }
  }
  const uint32_t mine = buf + (threadIdx.x & 15) * kQRowPitch;
#pragma unroll
  for (int third = 0; third < 3; ++third) {
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      const int32_t j = threadIdx.x + 128 * i, m = j / kThird;
      st_shared_v4(buf + m * kQRowPitch + (j - m * kThird) * 16, v[third][i].x, v[third][i].y, v[third][i].z, v[third][i].w);
    }
    group_barrier(1, 128);
#pragma unroll 1
    for (int c = 0; c < kThird; c += 4) {
      uint32_t x[16];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint4 w = ld_shared_v4(mine + (c + i) * 16);
        x[4 * i] = w.x, x[4 * i + 1] = w.y, x[4 * i + 2] = w.z, x[4 * i + 3] = w.w;
      }
      tmem_st16(at + 4 * (third * kThird + c), x);
    }
    group_barrier(1, 128);
  }
  tmem_wait_st();
  tc_fence_before();
}

// ---- roles ----

// A loader warp's cursor over the pair's tiles and the addresses of its 8 keys there.
struct Cursor {
  Units units;
  bool more;
  int32_t t, t0, t1, end, seq, row0, rows;  // of the cursor's unit

  __device__ __forceinline__ void next_unit(const AttendArgs& a) {
    Unit u;
    more = units.next(a, u);
    t = t0 = u.t0, t1 = u.t1, end = u.end, seq = u.seq, row0 = u.row0, rows = u.tokens * a.heads;
  }
  __device__ __forceinline__ void step(const AttendArgs& a) {
    if (more && ++t == t1) next_unit(a);
  }
  // Page id and offset at the cursor: lanes 0-7 the warp's keys, lanes 8-15 the peer
  // warp's (both CTAs need to know which keys have no record).  The id
  // is first looked at when the loads set out; in: a key before the end.
  __device__ __forceinline__ void look_up(const AttendArgs& a, int32_t rank, int w, int32_t& id, int32_t& offset,
                                          bool& in) const {
    const int lane = threadIdx.x & 31;
    id = -1;
    const int32_t owner = rank ^ (lane >> 3);
    const int32_t pos = t * kTileKeys + owner * kOwnKeys + w * kKeysPerWarp + (lane & 7);
    in = more && lane < 2 * kKeysPerWarp && pos < end;  // (the end lies within the table)
    if (in) {
      const uint32_t page = page_of(a.b, uint32_t(pos));
      offset = pos - int32_t(page) * a.b.page_size;
      id = int32_t(ldg_u32_now(a.b.table + int64_t(seq) * a.b.table_stride + page));
    }
  }
};

// The narrow and the few-row kernel's cursor: tiles of kKeys keys of the unit's keys [key0, stop), and
// a warp's 8 records there by lanes 0-7.
template <int kKeys>
struct KeyCursor {
  Units units;
  bool more;
  int32_t key, key0, stop, end, seq, row0, rows;

  __device__ __forceinline__ void next_unit(const AttendArgs& a) {
    Unit u;
    more = units.next_inline(a, u);
    key = key0 = u.t0 * kTileKeys, stop = u.t1 * kTileKeys, end = min(u.end, stop);
    seq = u.seq, row0 = u.row0, rows = u.tokens * a.heads;
  }
  __device__ __forceinline__ void step(const AttendArgs& a) {
    if (more && (key += kKeys) >= stop) next_unit(a);
  }
  __device__ __forceinline__ void look_up(const AttendArgs& a, int w, int32_t& id, int32_t& offset, bool& in) const {
    const int lane = threadIdx.x & 31;
    id = -1;
    const int32_t pos = key + w * kKeysPerWarp + (lane & 7);
    in = more && lane < kKeysPerWarp && pos < end;
    if (in) {
      const uint32_t page = page_of(a.b, uint32_t(pos));
      offset = pos - int32_t(page) * a.b.page_size;
      id = int32_t(ldg_u32_now(a.b.table + int64_t(seq) * a.b.table_stride + page));
    }
  }
};

__device__ __forceinline__ uint64_t record_address(const AttendArgs& a, int32_t id, int32_t offset) {
  if (id < 0) return 0;
  if (id >= a.b.n_pages) {
    if (a.b.status) atomicOr(a.b.status, SMLA_STATUS_INDEX_OOB);
    return 0;
  }
  return reinterpret_cast<uint64_t>(a.b.kv) + int64_t(id) * a.b.page_stride + int64_t(offset) * kRecordBytes;
}

// Whether the 8 records of lanes 0-7 lie in a row, as in pages of a multiple of 8.
__device__ __forceinline__ bool records_in_a_row(uint64_t rec, uint64_t first) {
  const int lane = threadIdx.x & 31;
  return __all_sync(0xffffffffu, lane >= kKeysPerWarp || (rec != 0 && rec == first + uint64_t(lane) * kRecordBytes));
}

// The pair's loaders: two groups of four warps take turns at the tiles, of each of
// which a CTA loads 32 keys.
__device__ __forceinline__ void loader_role(const AttendArgs& a, Misc* ms, uint32_t base, uint32_t rank) {
  const int lane = threadIdx.x & 31, index = (threadIdx.x >> 5) - kFirstLoader;
  const uint32_t group = index / kLoaderWarps;  // takes the tiles g with g % 2 == group: the stage
  const int w = index % kLoaderWarps;           // keys [8 w, 8 w + 8) of the CTA's 32
  const uint32_t q_full = map_to(smem_u32(&ms->q_full), 0), k_full = map_to(smem_u32(ms->k_full), 0);
  // where this lane's chunks go: row key = 8 w + j of block lane / 8, swizzled
  // column (lane & 7) ^ j
  const uint32_t k_at = base + kOffK + (lane >> 3) * (kOwnKeys * 128) + w * kKeysPerWarp * 128;
  const uint32_t rope_at = base + kOffK + 8 * (kOwnKeys * 128) + w * kKeysPerWarp * 128;

  // The records' addresses are looked up while the tile before is converted; their
  // loads set out as soon as its registers are free and land while the other group
  // works.
  Cursor c;
  c.units.start(a, ms);
  c.next_unit(a);
  if (group == 1) c.step(a);
  // rec: lane j's record (0: none)
  auto issue = [&](uint64_t rec, Raw& r) {
    const uint64_t first = __shfl_sync(0xffffffffu, rec, 0);
    if (records_in_a_row(rec, first)) {
      const uint8_t* p = reinterpret_cast<const uint8_t*>(first);
#pragma unroll
      for (int j = 0; j < kKeysPerWarp; ++j) load_record(p + j * kRecordBytes, j, r);
#pragma unroll
      for (int i = 0; i < 2; ++i)
        r.rope[i] = ldg_v4_now(p + (4 * i + (lane >> 3)) * kRecordBytes + kRopeOffset + (lane & 7) * 16);
    } else {
      r = load_scattered_call(rec);
    }
  };

  Raw raw;
  int32_t id, offset = 0;
  bool in;
  c.look_up(a, int32_t(rank), w, id, offset, in);
  for (uint32_t g = group; c.more; g += 2) {
    const uint64_t rec = record_address(a, id, offset);
    const uint32_t holes = __ballot_sync(0xffffffffu, rec == 0 && in);
    issue(rec, raw);
    if (c.t == c.t0) {
      // q of the unit, once the last QK of the unit before is done.  (A parity tells
      // a phase from its neighbours only, so QK(g - 3) has to be known as past, which
      // is on the other group's barrier: QK(g - 2) says so.)
      if (g >= 2 && !warp_wait(ms, a, &ms->qk_done[group], ((g - 2) >> 1) & 1)) return;
      if (g >= 1 && !warp_wait(ms, a, &ms->qk_done[group ^ 1], ((g - 1) >> 1) & 1)) return;
      load_q(a, base + kOffQ, rank, w, kLoaderWarps, c.row0, c.rows, 1);
      finish_q();
      if (lane == 0) arrive_at(q_full);
    }
    c.step(a);
    c.step(a);
    c.look_up(a, int32_t(rank), w, id, offset, in);
    // convert the landed records
    uint32_t v[kKeysPerWarp][2][4];
    uint32_t odd = 0, top = 0;
#pragma unroll
    for (int j = 0; j < kKeysPerWarp; ++j)
#pragma unroll
      for (int i = 0; i < 2; ++i) odd |= odd_scale(raw.scale[j][i]);
#pragma unroll
    for (int j = 0; j < kKeysPerWarp; ++j)
#pragma unroll
      for (int i = 0; i < 2; ++i) top = nan_codes(raw.lat[j][i], top);
    if (__any_sync(0xffffffffu, odd != 0 || (top & 0x80808080u) != 0)) {
#pragma unroll
      for (int j = 0; j < kKeysPerWarp; ++j) {
        bool bad = false;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const Dequant8 d = dequant8_any(raw.lat[j][i].x, raw.lat[j][i].y, raw.scale[j][i]);
          bad |= d.bad != 0;
#pragma unroll
          for (int k = 0; k < 4; ++k) v[j][i][k] = d.v[k];
        }
        // a latent that is not finite is zero in V, where rows that may not see the
        // key would meet it as 0 * NaN, and a NaN in the key's rope, which V lacks:
        // its scores are NaN, and the mask drops them
        if (__any_sync(0xffffffffu, bad) && lane == 8 * (j & 3)) raw.rope[j >> 2].x = 0x7FC07FC0u;
      }
    } else {
#pragma unroll
      for (int j = 0; j < kKeysPerWarp; ++j)
#pragma unroll
        for (int i = 0; i < 2; ++i)
          dequant8(raw.lat[j][i], __byte_perm(raw.scale[j][i] + (120u << 23), 0, 0x3232), v[j][i]);
    }
    if (g >= 2) {
      const uint32_t parity = ((g - 2) >> 1) & 1;
      if (!warp_wait(ms, a, &ms->qk_done[group], parity) || !warp_wait(ms, a, &ms->v_full[group], parity)) return;
    }
#pragma unroll
    for (int j = 0; j < kKeysPerWarp; ++j) {
      const uint32_t at = k_at + group * kStageK + j * 128 + ((uint32_t(lane & 7) ^ j) << 4);
      st_shared_v4(at, v[j][0][0], v[j][0][1], v[j][0][2], v[j][0][3]);
      st_shared_v4(at + 4 * (kOwnKeys * 128), v[j][1][0], v[j][1][1], v[j][1][2], v[j][1][3]);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t key = 4 * i + (lane >> 3);
      const uint4 r = raw.rope[i];
      st_shared_v4(rope_at + group * kStageK + key * 128 + ((uint32_t(lane & 7) ^ key) << 4), r.x, r.y, r.z, r.w);
    }
    if (lane < 2) ms->flags[g & 3][(rank ^ lane) * kLoaderWarps + w] = uint8_t(holes >> (8 * lane));
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) {
      mbar_arrive(&ms->k_ready[group]);
      arrive_at(k_full + 8 * group);
    }
  }
}

// The narrow and few-row kernel's loaders: all eight or twelve warps load every tile, a
// warp 8 of its keys.  Record by record: convert, store, and send the same registers
// off for the next tile's record, so that a warp's 8 records are in flight at
// nearly all times (42 KB an SM: what HBM needs at ~1 us latency).
template <int kN>
__device__ __forceinline__ void narrow_loader_role(const AttendArgs& a, Misc* ms, uint32_t base) {
  using L = Narrow<kN>;
  const int lane = threadIdx.x & 31, w = (threadIdx.x >> 5) - kFirstLoader;
  const uint32_t k_at = base + kOffK + (lane >> 3) * L::kBlock + w * kKeysPerWarp * 128;
  const uint32_t rope_at = base + kOffK + 8 * L::kBlock + w * kKeysPerWarp * 128;
  KeyCursor<L::kKeys> c;  // one tile ahead of the one that is converted
  c.units.start(a, ms);
  c.next_unit(a);
  if (!c.more) return;
  Raw raw;
  int32_t id, offset = 0;
  bool in;
  c.look_up(a, w, id, offset, in);
  uint64_t rec = record_address(a, id, offset);
  uint32_t holes = __ballot_sync(0xffffffffu, rec == 0 && in);
  raw = load_scattered(rec);
  bool starts = true, any = true;
  int32_t row0 = c.row0, rows = c.rows;
  c.step(a);
  c.look_up(a, w, id, offset, in);
  for (uint32_t g = 0; any; ++g) {
    const uint32_t stage = g & 1;
    if (!L::kFew && starts) {
      // q of the unit, once the last QK of the unit before is done (QK(g - 3), on the
      // same barrier, is past: this warp has waited for PV(g - 3))
      if (g >= 1 && !warp_wait(ms, a, &ms->qk_done[stage ^ 1], ((g - 1) >> 1) & 1)) return;
      load_q(a, base + L::kOffQ, 0, w, L::kLoaders, row0, rows, kCtaRows / kN);
    }
    rec = record_address(a, id, offset);
    const uint32_t next_holes = __ballot_sync(0xffffffffu, rec == 0 && in);
    const uint64_t first = __shfl_sync(0xffffffffu, rec, 0);
    const bool run = records_in_a_row(rec, first);
    if (g >= 2 && !warp_wait(ms, a, &ms->pv_done[stage], ((g - 2) >> 1) & 1)) return;
    uint32_t odd = 0, top = 0;
#pragma unroll
    for (int j = 0; j < kKeysPerWarp; ++j)
#pragma unroll
      for (int i = 0; i < 2; ++i) odd |= odd_scale(raw.scale[j][i]), top = nan_codes(raw.lat[j][i], top);
    const bool plain = !__any_sync(0xffffffffu, odd != 0 || (top & 0x80808080u) != 0);
    const uint32_t k = k_at + stage * L::kStage;
    uint32_t bad_keys = 0;
#pragma unroll
    for (int j = 0; j < kKeysPerWarp; ++j) {
      uint32_t v[2][4];
      if (plain) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
          dequant8(raw.lat[j][i], __byte_perm(raw.scale[j][i] + (120u << 23), 0, 0x3232), v[i]);
      } else {
        bool bad = false;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const Dequant8 d = dequant8_any(raw.lat[j][i].x, raw.lat[j][i].y, raw.scale[j][i]);
          bad |= d.bad != 0;
#pragma unroll
          for (int q = 0; q < 4; ++q) v[i][q] = d.v[q];
        }
        if (__any_sync(0xffffffffu, bad)) bad_keys |= 1u << j;
      }
      const uint32_t at = k + j * 128 + ((uint32_t(lane & 7) ^ j) << 4);
      st_shared_v4(at, v[0][0], v[0][1], v[0][2], v[0][3]);
      st_shared_v4(at + 4 * L::kBlock, v[1][0], v[1][1], v[1][2], v[1][3]);
      if (run) load_record(reinterpret_cast<const uint8_t*>(first) + j * kRecordBytes, j, raw);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t key = 4 * i + (lane >> 3);
      uint4 r = raw.rope[i];
      // (NaN in the rope of a key whose latent is not finite, as in loader_role)
      if ((lane & 7) == 0 && ((bad_keys >> key) & 1u)) r.x = 0x7FC07FC0u;
      st_shared_v4(rope_at + stage * L::kStage + key * 128 + ((uint32_t(lane & 7) ^ key) << 4), r.x, r.y, r.z, r.w);
      if (run)
        raw.rope[i] = ldg_v4_now(reinterpret_cast<const uint8_t*>(first) + key * kRecordBytes + kRopeOffset + (lane & 7) * 16);
    }
    if (!run && c.more) raw = load_scattered(rec);
    if (!L::kFew && starts) {
      finish_q();
      if (lane == 0) mbar_arrive(&ms->q_full);
    }
    if (lane == 0) (L::kFew ? ms->flags_few[g & 3] : ms->flags[g & 3])[w] = uint8_t(holes);
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) mbar_arrive(&ms->k_full[stage]);
    holes = next_holes;
    any = c.more;
    starts = c.key == c.key0;
    row0 = c.row0, rows = c.rows;
    c.step(a);
    c.look_up(a, w, id, offset, in);
    // the records of the tile after next set out for L2 (64 x 16: 52 us, without 58; one
    // by one in pages that split a warp's eight: 67 us with pages of one record, without 72)
    const bool rows_of_8 = a.b.page_size % kKeysPerWarp == 0;
    if (in && (lane == 0 || !rows_of_8) && id >= 0 && id < a.b.n_pages)
      prefetch_l2(reinterpret_cast<const uint8_t*>(record_address(a, id, offset)),
                  (rows_of_8 ? kKeysPerWarp : 1) * kRecordBytes);
  }
}

// One thread of each CTA: copies the latent blocks of K to V, dims [0, 256) to the
// even CTA's and the rest to the odd one's, and tells both CTAs when its V is
// complete (PV may read it, the loaders may overwrite the K it came from).
__device__ __forceinline__ void copier_role(const AttendArgs& a, Misc* ms, uint32_t base, uint32_t rank) {
  uint32_t land[2], full[2], v_at[2];
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    land[r] = map_to(smem_u32(ms->v_land), r);
    full[r] = map_to(smem_u32(ms->v_full), r);
    v_at[r] = map_to(base + kOffV + rank * (kOwnKeys * 128), r);
  }
  Units units;
  units.start(a, ms);
  bool more;
  int32_t t, t1;
  auto next_unit = [&]() {
    Unit u;
    more = units.next(a, u);
    t = u.t0, t1 = u.t1;
  };
  next_unit();
  uint32_t g = 0, done = 0;  // tiles copied, tiles whose V has landed here
  uint64_t t0 = 0;
  for (uint32_t idle = 1; more || done < g; ++idle) {
    const uint32_t stage = g & 1, last = done & 1;
    if (more && mbar_test(&ms->k_ready[stage], (g >> 1) & 1) &&
        (g < 2 || mbar_test(&ms->pv_done[stage], ((g - 2) >> 1) & 1))) {
      mbar_arrive_expect_tx(&ms->v_land[stage], kStageV);
#pragma unroll
      for (int b = 0; b < 4; ++b)
#pragma unroll
        for (int r = 0; r < 2; ++r)
          bulk_s2s(v_at[r] + stage * kStageV + b * kVBlock, base + kOffK + stage * kStageK + (4 * r + b) * (kOwnKeys * 128),
                   kOwnKeys * 128, land[r] + 8 * stage);
      ++g;
      if (++t == t1) next_unit();
      idle = 0;
    }
    if (done < g && mbar_test(&ms->v_land[last], (done >> 1) & 1)) {
      arrive_at(full[0] + 8 * last);
      arrive_at(full[1] + 8 * last);
      ++done;
      idle = 0;
    }
    if (idle == 0) {
      t0 = 0;
      continue;
    }
    __nanosleep(40);
    if ((idle & 63u) == 0) {
      const uint64_t now = globaltimer();
      if (t0 == 0) t0 = now;
      const bool late = now - t0 > ms->wait_ns;
      if (late) give_up(ms, a.b.status);
      if (late || *reinterpret_cast<volatile int32_t*>(&ms->dead)) {
        // copies in flight are waited for, with a limit of their own
        for (; done < g; ++done) mbar_wait(&ms->v_land[done & 1], (done >> 1) & 1, kWaitNs);
        return;
      }
    }
  }
}

// A warp of the even CTA each: K-steps which, which + 2, ... of every QK.  (The
// whole warp runs the loop, see elect_one.)
__device__ __forceinline__ void issuer_qk_role(const AttendArgs& a, Misc* ms, uint32_t base, uint32_t tmem,
                                               uint32_t which) {
  const uint64_t q0 = smem_desc(base + kOffQ, 16, 1024, kSw128);
  const uint64_t k0 = smem_desc(base + kOffK, 16, 1024, kSw128);
  Units units;
  units.start(a, ms);
  Unit u;
  uint32_t g = 0, n_units = 0;
  while (units.next(a, u)) {
    if (!warp_wait(ms, a, &ms->q_full, n_units & 1)) return;
    ++n_units;
    const int32_t t0 = u.t0, t1 = u.t1;
    for (int32_t t = t0; t < t1; ++t, ++g) {
      const uint32_t stage = g & 1;
      if (!warp_wait(ms, a, &ms->k_full[stage], (g >> 1) & 1)) return;
      if (g >= 2 && !warp_wait(ms, a, &ms->s_empty[stage], ((g - 2) >> 1) & 1)) return;
      tc_fence_after();
      const uint32_t d = tmem + kTmemS + 64 * stage + 32 * which;
      const uint64_t qd = q0 + which * 2, kd = k0 + uint64_t((stage * kStageK) >> 4) + which * 2;
      if (elect_one()) {
#pragma unroll
        for (int k = 0; k < kQK / 16; k += 2)
          mma2(d, qd + uint64_t(((k >> 2) * kQBlock + (k & 3) * 32) >> 4),
             kd + uint64_t(((k >> 2) * (kOwnKeys * 128) + (k & 3) * 32) >> 4), kIdescQK, k > 0);
        commit2(&ms->qk_done[stage]);
      }
      __syncwarp();
    }
  }
}

// A warp of the even CTA: O += P V of every tile.
__device__ __forceinline__ void issuer_pv_role(const AttendArgs& a, Misc* ms, uint32_t base, uint32_t tmem) {
  const uint64_t p0 = smem_desc(base + kOffP, 16, 1024, kSw128);
  const uint64_t v0 = smem_desc(base + kOffV, kVBlock, 1024, kSw128);
  Units units;
  units.start(a, ms);
  Unit u;
  uint32_t g = 0;
  while (units.next(a, u)) {
    const int32_t t0 = u.t0, t1 = u.t1;
    for (int32_t t = t0; t < t1; ++t, ++g) {
      const uint32_t stage = g & 1;
      if (!warp_wait(ms, a, &ms->v_full[stage], (g >> 1) & 1)) return;
      if (!warp_wait(ms, a, &ms->p_full, g & 1)) return;
      tc_fence_after();
      const uint64_t vd = v0 + uint64_t((stage * kStageV) >> 4);
      if (elect_one()) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int k = 0; k < kTileKeys / 16; ++k)
            mma2(tmem + 128 * h, p0 + uint64_t(k * 2), vd + uint64_t((h * 2 * kVBlock + k * 2048) >> 4), kIdescPV,
               (t == t0 && k == 0) ? 0u : 1u);
        commit2(&ms->pv_done[stage]);
      }
      __syncwarp();
    }
  }
}

// Output factor and LSE of a row (finish_head_v) with the sink of its head.  A sink that
// is +inf in log2 units (above 2.36e38) holds all of the weight: out = 0, where inf - inf
// would give NaN.
__device__ __forceinline__ void finish_row(const AttendArgs& a, int32_t head, float m, float l, float* factor, float* lse) {
  const float sink = a.sink != nullptr ? __ldg(a.sink + head) : 0.f;
  finish_head_v(m, l, a.sink != nullptr, sink, factor, lse);
  if (sink * kLog2e == INFINITY && l >= 0.f) *factor = 0.f;
}

// The last part of a row tile: the merge kernel joins the parts from the worker
// that holds its first key tile up to this one.
__device__ __noinline__ void name_merge(const AttendArgs& a, const Misc* ms, int32_t worker, const Unit& u) {
  const int64_t G = max(min(int64_t(a.workers), ms->total), int64_t(1));
  a.merge[worker * 4 + 1] = u.row0;
  a.merge[worker * 4 + 2] = int32_t(((u.slot + 1) * G - 1) / ms->total);
  a.merge[worker * 4] = u.tokens * a.heads;
}

__device__ __forceinline__ void softmax_role(const AttendArgs& a, Misc* ms, uint32_t base, uint32_t tmem, uint32_t rank,
                                             int32_t pair) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int row = (warp & 1) * 32 + lane;  // of this CTA
  const int half = warp >> 1;              // columns: keys [32 half, +32), dims [256 half, +256)
  const int32_t m = int32_t(rank) * kCtaRows + row;
  const int32_t tok = m / a.heads, head = m - tok * a.heads;
  const uint32_t lane_base = tmem + (uint32_t(warp) << 21);  // lane 32 warp
  const uint32_t p_full = map_to(smem_u32(&ms->p_full), 0), s_empty = map_to(smem_u32(ms->s_empty), 0);
  const uint32_t p_row = base + kOffP + row * 128;
  // scores are scaled after the mask and the maximum, so the factor has to be positive
  const float scale = a.scale_log2 == 0.f ? 1.f : fabsf(a.scale_log2);
  Units units;
  units.start(a, ms);
  Unit u;
  uint32_t g = 0;
  // (a wait that gives up does not end this role: its warps meet at named
  // barriers, so all of them run through every tile)
  if (ms->stall) meet_after(ms, a, &ms->never, 0);
  while (units.next(a, u)) {
    const bool live = m < u.tokens * a.heads;
    const int32_t see = a.causal && live ? max(min(u.pos0 + tok + 1, u.end), 0) : u.end;
    float ref = -INFINITY, l = 0.f;
    const int32_t t0 = u.t0, t1 = u.t1;
    for (int32_t t = t0; t < t1; ++t, ++g) {
      const uint32_t stage = g & 1;
      meet_after(ms, a, &ms->qk_done[stage], (g >> 1) & 1);
      tc_fence_after();
      uint32_t s[64];  // the two accumulators' 32 columns
      {
        uint32_t(&lo)[16] = *reinterpret_cast<uint32_t(*)[16]>(s);
        uint32_t(&hi)[16] = *reinterpret_cast<uint32_t(*)[16]>(s + 16);
        uint32_t(&lo2)[16] = *reinterpret_cast<uint32_t(*)[16]>(s + 32);
        uint32_t(&hi2)[16] = *reinterpret_cast<uint32_t(*)[16]>(s + 48);
        tmem_ld16(lane_base + kTmemS + 64 * stage, lo);
        tmem_ld16(lane_base + kTmemS + 64 * stage + 16, hi);
        tmem_ld16(lane_base + kTmemS + 64 * stage + 32, lo2);
        tmem_ld16(lane_base + kTmemS + 64 * stage + 48, hi2);
      }
      const uint32_t flags = *reinterpret_cast<const uint32_t*>(&ms->flags[g & 3][4 * half]);
      tmem_wait_ld();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) arrive_at(s_empty + 8 * stage);
      float x[32];  // scores before the scale (times its sign)
#pragma unroll
      for (int c = 0; c < 32; c += 2) add2(s[c], s[c + 1], s[32 + c], s[33 + c], x[c], x[c + 1]);
      if (a.scale_log2 <= 0.f) {
        const float by = a.scale_log2 < 0.f ? -1.f : 0.f;
#pragma unroll
        for (int c = 0; c < 32; ++c) x[c] *= by;
      }
      const int32_t key0 = t * kTileKeys + 32 * half;
      if (__any_sync(0xffffffffu, key0 + 32 > see) || flags) {
        // bit c: key c is seen
        const int32_t n = see - key0;
        const uint32_t seen = ~flags & (n >= 32 ? 0xffffffffu : n <= 0 ? 0u : (1u << n) - 1u);
#pragma unroll
        for (int c = 0; c < 32; ++c) x[c] = (seen >> c) & 1u ? x[c] : -INFINITY;
      }
      float tm = x[0];
#pragma unroll
      for (int c = 1; c < 32; ++c) tm = fmaxf(tm, x[c]);
      ms->tmax[stage][warp * 32 + lane] = tm;
      group_barrier(1 + (warp & 1), 64);
      tm = fmaxf(tm, ms->tmax[stage][(warp ^ 2) * 32 + lane]) * scale;
      const bool move = tm > ref + kMoveMargin;
      const float nref = move ? tm : ref;
      const float use = nref == -INFINITY ? 0.f : nref;
      const float alpha = move ? ex2(ref - use) : 1.f;
      ref = nref;
      uint32_t p[16];
      float sum0 = 0.f, sum1 = 0.f;
#pragma unroll
      for (int c = 0; c < 16; ++c) {
        float y0, y1;
        fma2(x[2 * c], x[2 * c + 1], scale, -use, y0, y1);
        y0 = ex2(y0);
        y1 = ex2(y1);
        add2(sum0, sum1, y0, y1, sum0, sum1);
        // P as the product's bf16 operand (V is bf16, and one kind::f16 product has one type);
        // the sum keeps f32.  Relative RMS error of out 0.0017-0.0022, with P in f32
        // 0.0016-0.0017 (out's own rounding); P as two bf16 terms would read V twice
        p[c] = pack_bf16x2(y0, y1);
      }
      l = l * alpha + (sum0 + sum1);
      if (g > 0) meet_after(ms, a, &ms->pv_done[(g - 1) & 1], ((g - 1) >> 1) & 1);
      if (t > t0 && __any_sync(0xffffffffu, move)) {
        tc_fence_after();
#pragma unroll 1
        for (int c = 0; c < 256; c += 16) {
          uint32_t o[16];
          tmem_ld16(lane_base + c, o);
          tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
          tmem_st16(lane_base + c, o);
        }
        tmem_wait_st();
      }
#pragma unroll
      for (int c = 0; c < 4; ++c)
        st_shared_v4(p_row + (((4 * half + c) ^ (row & 7)) << 4), p[4 * c], p[4 * c + 1], p[4 * c + 2], p[4 * c + 3]);
      fence_proxy_async_smem();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) arrive_at(p_full);
    }
    // the unit's end: row sums of the two halves, then O
    ms->lsum[warp * 32 + lane] = l;
    group_barrier(1 + (warp & 1), 64);
    l += ms->lsum[(warp ^ 2) * 32 + lane];
    meet_after(ms, a, &ms->pv_done[(g - 1) & 1], ((g - 1) >> 1) & 1);
    tc_fence_after();
    const bool whole = u.t0 == 0 && u.t1 == u.tiles;
    const int64_t part = 2 * int64_t(pair) + (u.t0 > 0 ? 0 : 1);
    float factor = 1.f;
    const int64_t tok_row = int64_t(u.row0) + tok;
    if (live && half == 0) {
      if (!whole) {
        a.ml_part[(part * a.part_rows + m) * 2] = ref;
        a.ml_part[(part * a.part_rows + m) * 2 + 1] = l;
      }
    }
    if (whole) {
      float lse;
      finish_row(a, head, ref, l, &factor, &lse);
      if (live && half == 0 && a.lse) a.lse[tok_row * a.heads + head] = lse;
    }
    uint16_t* dst = a.out + tok_row * a.o_row + int64_t(head) * a.o_head + 256 * half;
    float* pdst = a.o_part + (part * kLatent + 256 * half) * kPairRows + m * 4;  // (see paged_merge_pair_kernel)
#pragma unroll 1
    for (int c = 0; c < 256; c += 16) {
      uint32_t o[16];
      __syncwarp();  // (dead lanes skip the stores, and the load is the whole warp's)
      tmem_ld16(lane_base + c, o);
      tmem_wait_ld();
      if (live && whole) {
        uint32_t v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
          v[i] = l == 0.f ? 0u
                          : pack_bf16x2(__uint_as_float(o[2 * i]) * factor, __uint_as_float(o[2 * i + 1]) * factor);
        *reinterpret_cast<uint4*>(dst + c) = make_uint4(v[0], v[1], v[2], v[3]);
        *reinterpret_cast<uint4*>(dst + c + 8) = make_uint4(v[4], v[5], v[6], v[7]);
      } else if (live) {
#pragma unroll
        for (int i = 0; i < 16; i += 4)
          *reinterpret_cast<uint4*>(pdst + (c + i) * kPairRows) = make_uint4(o[i], o[i + 1], o[i + 2], o[i + 3]);
      }
    }
    tc_fence_before();
    if (!whole && u.t0 > 0 && u.t1 == u.tiles && rank == 0 && threadIdx.x == 0) {
      name_merge(a, ms, pair, u);
    }
  }
}

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kAttendThreads, 1)
paged_attend_kernel(const __grid_constant__ AttendArgs a) {
  extern __shared__ __align__(1024) uint8_t raw_smem[];
  const uint32_t base = smem_u32(raw_smem);
  if (base & 1023u) {  // (the operands' swizzle needs it; the same in every CTA)
    if (threadIdx.x == 0) {
      a.merge[(blockIdx.x >> 1) * 4] = 0;
      if (a.b.status) atomicOr(a.b.status, SMLA_STATUS_SMEM_LAYOUT);
    }
    return;
  }
  Misc* ms = reinterpret_cast<Misc*>(raw_smem + kOffMisc);
  const uint32_t rank = cluster_rank();
  const int32_t pair = blockIdx.x >> 1;
  const int warp = threadIdx.x >> 5;
  let_dependents_launch();
  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&ms->k_ready[i], kLoaderWarps);
      mbar_init(&ms->k_full[i], 2 * kLoaderWarps);
      mbar_init(&ms->v_land[i], 1);
      mbar_init(&ms->v_full[i], 2);
      mbar_init(&ms->s_empty[i], 8);
      mbar_init(&ms->qk_done[i], 2);
      mbar_init(&ms->pv_done[i], 1);
    }
    mbar_init(&ms->q_full, 2 * kLoaderWarps);
    mbar_init(&ms->p_full, 8);
    mbar_init(&ms->drain, 3);
    mbar_init(&ms->never, 1);
    fence_mbar_init();
    ms->dead = 0;
    ms->wait_ns = g_paged_wait_ns ? g_paged_wait_ns : kWaitNs;
    ms->stall = g_paged_stall;
    if (rank == 0) a.merge[pair * 4] = 0;
  }
  if (warp == kCopier) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&ms->tmem)),
                 "r"(kTmemCols)
                 : "memory");
    tc_fence_before();
  }
  find_range<kAttendThreads>(a, ms, pair);
  __syncthreads();
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem = ms->tmem;
  if (warp < kFirstLoader) {
    softmax_role(a, ms, base, tmem, rank, pair);
  } else if (warp < kIssuerQk) {
    loader_role(a, ms, base, rank);
  } else if (warp == kCopier) {
    if ((threadIdx.x & 31) == 0) copier_role(a, ms, base, rank);
  } else if (rank == 0) {
    if (warp == kIssuerPv) issuer_pv_role(a, ms, base, tmem);
    else issuer_qk_role(a, ms, base, tmem, uint32_t(warp - kIssuerQk));
    // every MMA has to be complete before the tensor memory and the shared
    // memory it reads go away (also after a wait that gave up); the odd CTA
    // learns of it at the cluster barrier
    __syncwarp();
    if (elect_one()) {  // (the lane that issued them: the same for the same mask)
      asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
                       smem_u32(&ms->drain))
                   : "memory");
      if (!mbar_wait(&ms->drain, 0, kWaitNs)) give_up(ms, a.b.status);
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  tc_fence_after();
  if (warp == kCopier) {
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols) : "memory");
  }
}

// ---- the narrow kernel ----
//
// Up to kN = 32 or 64 rows a tile (single tokens, a few drafted ones): no
// pair, since half of its rows or more would be empty, and each CTA loads all 64
// keys of a tile once for both products.
//   S[64, 64] = Q K^T as above (M = 64: rows 16 w .. sit in lanes 32 w .. of TMEM).
// With kN = 32 the 64 rows hold two copies of Q, so that every softmax warp finds
// its rows in its own lanes and takes kN of the 64 keys.
//   O^T[128 b .. + 128, kN] += V^T P^T, b = 0 .. 3: the four M = 128 blocks of
// dims take 4 kN columns, and V^T is the K tile read MN-major, so nothing is copied.
// Warps (16): 0-3 softmax, 4-11 loaders, 12-13 half of QK's K-steps each, 14-15
// two blocks of PV each.
//
// What bounds it: the loaders (2.1 us a tile of 64 records by eight warps at the register
// limit, the same for 17, 32 and 64 rows: 3.0 TB/s of records over all SMs), whose
// largest stall is the wait for their own global loads, and for short rows the ~10 us
// until the first scores and the partials' way through L2.  4 x 64 heads over up to 16384
// positions: 37 us; 64 x 64 heads over 4096: 88 us.

template <int kN>
__device__ __forceinline__ void narrow_softmax_role(const AttendArgs& a, Misc* ms, uint32_t base, uint32_t tmem,
                                                    int32_t worker) {
  using L = Narrow<kN>;
  constexpr int kCopies = kCtaRows / kN, kKeys = kN;  // a thread's keys of a tile
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int32_t m = (16 * warp + (lane & 15)) % kN;   // this thread's row
  const int slice = 16 * warp / kN;                   // and keys [kKeys slice, + kKeys)
  const bool mine = lane < 16;
  const int32_t tok = m / a.heads, head = m - tok * a.heads;
  const uint32_t lane_base = tmem + (uint32_t(warp) << 21);
  const uint32_t p_row = base + L::kOffP + m * 128;
  const float scale = a.scale_log2 == 0.f ? 1.f : fabsf(a.scale_log2);
  Units units;
  units.start(a, ms);
  Unit u;
  uint32_t g = 0;
  if (ms->stall) meet_after(ms, a, &ms->never, 0);
  while (units.next_inline(a, u)) {
    const int32_t rows = u.tokens * a.heads, t0 = u.t0, t1 = u.t1;
    const bool live = mine && m < rows;
    const int32_t see = a.causal && live ? max(min(u.pos0 + tok + 1, u.end), 0) : u.end;
    float ref = -INFINITY, l = 0.f;
    for (int32_t t = t0; t < t1; ++t, ++g) {
      const uint32_t stage = g & 1;
      meet_after(ms, a, &ms->qk_done[stage], (g >> 1) & 1);
      tc_fence_after();
      float x[kKeys];
      const uint32_t s_at = lane_base + kTmemS + 128 * stage + kKeys * slice;
#pragma unroll
      for (int c = 0; c < kKeys; c += 16) {
        uint32_t s0[16], s1[16];
        tmem_ld16(s_at + c, s0);
        tmem_ld16(s_at + 64 + c, s1);
        tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < 16; i += 2) add2(s0[i], s0[i + 1], s1[i], s1[i + 1], x[c + i], x[c + i + 1]);
      }
      const uint64_t flags = *reinterpret_cast<const uint64_t*>(&ms->flags[g & 3][0]) >> (kKeys * slice);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&ms->s_empty[stage]);
      if (a.scale_log2 <= 0.f) {
        const float by = a.scale_log2 < 0.f ? -1.f : 0.f;
#pragma unroll
        for (int c = 0; c < kKeys; ++c) x[c] *= by;
      }
      const int32_t n = see - t * kTileKeys - kKeys * slice;
      if (__any_sync(0xffffffffu, n < kKeys) || flags != 0) {
        const uint64_t seen = ~flags & (n >= 64 ? ~0ull : n <= 0 ? 0ull : (1ull << n) - 1ull);
#pragma unroll
        for (int c = 0; c < kKeys; ++c) x[c] = (seen >> c) & 1u ? x[c] : -INFINITY;
      }
      float tm = x[0];
#pragma unroll
      for (int c = 1; c < kKeys; ++c) tm = fmaxf(tm, x[c]);
      if (kCopies > 1) {
        ms->tmax[stage][warp * 32 + lane] = tm;
        group_barrier(1, 128);
#pragma unroll
        for (int k = 1; k < kCopies; ++k) tm = fmaxf(tm, ms->tmax[stage][(warp ^ (k * (kN / 16))) * 32 + lane]);
      }
      tm *= scale;
      const bool move = live && tm > ref + kMoveMargin;
      const float nref = move ? tm : ref;
      const float use = nref == -INFINITY ? 0.f : nref;
      const float alpha = move ? ex2(ref - use) : 1.f;
      ref = nref;
      if (mine && slice == 0) ms->alpha[stage][m] = alpha;
      __syncwarp();
      const bool moved = named_barrier_or(1, 128, move);
      uint32_t p[kKeys / 2];
      float sum0 = 0.f, sum1 = 0.f;
#pragma unroll
      for (int c = 0; c < kKeys / 2; ++c) {
        float y0, y1;
        fma2(x[2 * c], x[2 * c + 1], scale, -use, y0, y1);
        y0 = ex2(y0);
        y1 = ex2(y1);
        add2(sum0, sum1, y0, y1, sum0, sum1);
        p[c] = pack_bf16x2(y0, y1);
      }
      l = l * alpha + (sum0 + sum1);
      if (g > 0) meet_after(ms, a, &ms->pv_done[stage ^ 1], ((g - 1) >> 1) & 1);
      if (t > t0 && moved) {
        tc_fence_after();
#pragma unroll 1
        for (int c = 0; c < 4 * kN; c += 16) {
          uint32_t o[16];
          tmem_ld16(lane_base + c, o);
          tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            o[i] = __float_as_uint(__uint_as_float(o[i]) * ms->alpha[stage][(c & (kN - 1)) + i]);
          }
          tmem_st16(lane_base + c, o);
        }
        tmem_wait_st();
      }
      if (mine) {
#pragma unroll
        for (int c = 0; c < kKeys / 8; ++c)
          st_shared_v4(p_row + (((slice * (kKeys / 8) + c) ^ (m & 7)) << 4), p[4 * c], p[4 * c + 1], p[4 * c + 2],
                       p[4 * c + 3]);
      }
      fence_proxy_async_smem();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&ms->p_full);
    }
    const bool whole = t0 == 0 && t1 == u.tiles;
    const int64_t part = 2 * int64_t(worker) + (t0 > 0 ? 0 : 1);
    if (kCopies > 1) {
      ms->lsum[warp * 32 + lane] = l;
      group_barrier(1, 128);
      l = 0.f;
#pragma unroll
      for (int k = 0; k < kCopies; ++k) l += ms->lsum[(warp ^ (k * (kN / 16))) * 32 + lane];
    }
    if (mine && slice == 0) {
      float factor = 1.f;
      if (whole) {
        float lse;
        finish_row(a, head, ref, l, &factor, &lse);
        if (live && a.lse) a.lse[(int64_t(u.row0) + tok) * a.heads + head] = lse;
      } else if (live) {
        a.ml_part[(part * a.part_rows + m) * 2] = ref;
        a.ml_part[(part * a.part_rows + m) * 2 + 1] = l;
      }
      ms->factor[m] = factor;
    }
    group_barrier(1, 128);
    meet_after(ms, a, &ms->pv_done[(g - 1) & 1], ((g - 1) >> 1) & 1);
    tc_fence_after();
    // a lane has dim 128 b + 32 warp + lane of every row
    const int32_t dim = 32 * warp + lane;
    int32_t r_tok = 0, r_head = 0;
#pragma unroll 1
    for (int c = 0; c < rows; c += 16) {
      uint32_t o[4][16];
#pragma unroll
      for (int b = 0; b < 4; ++b) tmem_ld16(lane_base + b * kN + c, o[b]);
      tmem_wait_ld();
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        if (c + i >= rows) break;
        if (whole) {
          const float f = ms->factor[c + i];
          uint16_t* dst = a.out + (int64_t(u.row0) + r_tok) * a.o_row + int64_t(r_head) * a.o_head + dim;
#pragma unroll
          for (int b = 0; b < 4; ++b) dst[128 * b] = uint16_t(pack_bf16x2(__uint_as_float(o[b][i]) * f, 0.f));
        } else {
          float* dst = a.o_part + (part * a.part_rows + c + i) * kLatent + dim;
#pragma unroll
          for (int b = 0; b < 4; ++b) dst[128 * b] = __uint_as_float(o[b][i]);
        }
        if (++r_head == a.heads) r_head = 0, ++r_tok;
      }
    }
    tc_fence_before();
    if (!whole && t0 > 0 && t1 == u.tiles && threadIdx.x == 0) name_merge(a, ms, worker, u);
  }
}

// A warp each: K-steps which, which + 2, ... of every QK into an accumulator
// of its own.
__device__ __forceinline__ void narrow_qk_role(const AttendArgs& a, Misc* ms, uint32_t base, uint32_t tmem,
                                               uint32_t which) {
  const uint64_t q0 = smem_desc(base + Narrow<64>::kOffQ, 16, 1024, kSw128) + which * 2;
  const uint64_t k0 = smem_desc(base + kOffK, 16, 1024, kSw128) + which * 2;
  Units units;
  units.start(a, ms);
  Unit u;
  uint32_t g = 0, n_units = 0;
  while (units.next_inline(a, u)) {
    const int32_t t0 = u.t0, t1 = u.t1;
    if (!warp_wait(ms, a, &ms->q_full, n_units++ & 1)) return;
    for (int32_t t = t0; t < t1; ++t, ++g) {
      const uint32_t stage = g & 1;
      if (!warp_wait(ms, a, &ms->k_full[stage], (g >> 1) & 1)) return;
      if (g >= 2 && !warp_wait(ms, a, &ms->s_empty[stage], ((g - 2) >> 1) & 1)) return;
      tc_fence_after();
      const uint64_t kd = k0 + uint64_t((stage * Narrow<64>::kStage) >> 4);
      if (elect_one()) {
#pragma unroll
        for (int k = 0; k < kQK / 16; k += 2)
          mma_f16_ss(tmem + kTmemS + 128 * stage + 64 * which, q0 + uint64_t(((k >> 2) * kQBlock + (k & 3) * 32) >> 4),
                   kd + uint64_t(((k >> 2) * (kTileKeys * 128) + (k & 3) * 32) >> 4),
                   idesc_bf16(kCtaRows, kTileKeys, 0, 0), k > 0);
        mma_commit(&ms->qk_done[stage]);
      }
      __syncwarp();
    }
  }
}

// A warp each: blocks 2 which and 2 which + 1 of every O^T += V^T P^T.
template <int kN>
__device__ __forceinline__ void narrow_pv_role(const AttendArgs& a, Misc* ms, uint32_t base, uint32_t tmem,
                                               uint32_t which) {
  using L = Narrow<kN>;
  const uint64_t v0 = smem_desc(base + kOffK + which * 4 * (kTileKeys * 128), kTileKeys * 128, 1024, kSw128);
  const uint64_t p0 = smem_desc(base + L::kOffP, 16, 1024, kSw128);
  Units units;
  units.start(a, ms);
  Unit u;
  uint32_t g = 0;
  while (units.next_inline(a, u)) {
    const int32_t t0 = u.t0, t1 = u.t1;
    for (int32_t t = t0; t < t1; ++t, ++g) {
      const uint32_t stage = g & 1;
      if (!warp_wait(ms, a, &ms->p_full, g & 1)) return;
      tc_fence_after();
      const uint64_t vd = v0 + uint64_t((stage * Narrow<64>::kStage) >> 4);
      if (elect_one()) {
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
          for (int k = 0; k < kTileKeys / 16; ++k)
            mma_f16_ss(tmem + (2 * which + b) * kN, vd + uint64_t((b * 2 * (kTileKeys * 128) + k * 2048) >> 4),
                     p0 + uint64_t(k * 2), idesc_bf16(128, kN, 1, 0), (t == t0 && k == 0) ? 0u : 1u);
        mma_commit(&ms->pv_done[stage]);
      }
      __syncwarp();
    }
  }
}

template <int kN>
__global__ void __launch_bounds__(kNarrowThreads, 1) paged_attend_narrow_kernel(const __grid_constant__ AttendArgs a) {
  extern __shared__ __align__(1024) uint8_t raw_smem[];
  const uint32_t base = smem_u32(raw_smem);
  const int32_t worker = blockIdx.x;
  const int warp = threadIdx.x >> 5;
  let_dependents_launch();
  if (threadIdx.x == 0) a.merge[worker * 4] = 0;
  if (base & 1023u) {
    if (threadIdx.x == 0 && a.b.status) atomicOr(a.b.status, SMLA_STATUS_SMEM_LAYOUT);
    return;
  }
  Misc* ms = reinterpret_cast<Misc*>(raw_smem + Narrow<kN>::kOffMisc);
  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&ms->k_full[i], 2 * kLoaderWarps);
      mbar_init(&ms->s_empty[i], 4);
      mbar_init(&ms->qk_done[i], 2);
      mbar_init(&ms->pv_done[i], 2);
    }
    mbar_init(&ms->q_full, 2 * kLoaderWarps);
    mbar_init(&ms->p_full, 4);
    mbar_init(&ms->drain, 4);
    mbar_init(&ms->never, 1);
    fence_mbar_init();
    ms->dead = 0;
    ms->wait_ns = g_paged_wait_ns ? g_paged_wait_ns : kWaitNs;
    ms->stall = g_paged_stall;
  }
  if (warp == kNarrowQk) {
    tmem_alloc(&ms->tmem, kTmemCols);
    tc_fence_before();
  }
  find_range<kNarrowThreads>(a, ms, worker);
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ms->tmem;
  if (warp < kFirstLoader) {
    narrow_softmax_role<kN>(a, ms, base, tmem, worker);
  } else if (warp < kNarrowQk) {
    narrow_loader_role<kN>(a, ms, base);
  } else {
    if (warp < kNarrowPv) narrow_qk_role(a, ms, base, tmem, uint32_t(warp - kNarrowQk));
    else narrow_pv_role<kN>(a, ms, base, tmem, uint32_t(warp - kNarrowPv));
    // every MMA complete before the memory it reads goes away
    __syncwarp();
    if (elect_one()) {  // (the lane that issued them: the same for the same mask)
      mma_commit(&ms->drain);
      if (!mbar_wait(&ms->drain, 0, kWaitNs)) give_up(ms, a.b.status);
    }
  }
  cp_async_wait_all();  // (a loader whose wait gave up may have q on its way)
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kNarrowQk) {
    tmem_relinquish();
    tmem_dealloc(tmem, kTmemCols);
  }
}

// ---- the few-row kernel ----
//
// Up to 16 rows a tile: the loaders' conversion bounds the narrow kernel, so here twelve
// of the 16 warps load, in tiles of 96 keys, and warps 0-3 do the rest.  Q lies in tensor memory
// (288 columns, the A operand of S[64, 96] = Q K^T), which leaves shared memory to two
// stages of 96 keys.  S holds four copies of the 16 rows, one in each warp's lanes; a
// warp takes 24 of the keys.  Per tile: S read, maxima exchanged, P stored, then warp 0
// issues the next QK, warps 1 and 2 two blocks of O^T += V^T P^T each.
//
// 64 x 16 heads over up to 4096 positions: 53 us (131 MB of records: 2.5 TB/s; 60 us with
// eight loaders, tiles of 64 keys and Q in shared memory, 62 us with Q in tensor memory
// and a third stage instead of more loaders); one token, 16 heads, 500 positions: 15 us.
// Bound: 2.2 us a tile of 96 keys (4.3 TB/s of records over all SMs), still the loaders,
// and ~18 us of start, partials and merge.

// QK of tile g, by warp 0.
__device__ __forceinline__ void few_issue_qk(const AttendArgs& a, Misc* ms, uint64_t k0, uint32_t tmem, uint32_t g) {
  using L = Narrow<16>;
  const uint32_t stage = g & 1;
  if (warp_wait(ms, a, &ms->k_full[stage], (g >> 1) & 1)) {
    tc_fence_after();
    const uint64_t kd = k0 + uint64_t((stage * L::kStage) >> 4);
    if (elect_one()) {
#pragma unroll
      for (int k = 0; k < kQK / 16; ++k)
        mma_ts(tmem + kTmemSFew, tmem + kTmemQFew + 8 * k, kd + uint64_t(((k >> 2) * L::kBlock + (k & 3) * 32) >> 4),
               idesc_bf16(kCtaRows, L::kKeys, 0, 0), k > 0);
      mma_commit(&ms->qk_done[stage]);
    }
  }
  __syncwarp();
}

__device__ __forceinline__ void few_compute_role(const AttendArgs& a, Misc* ms, uint32_t base, uint32_t tmem,
                                                 int32_t worker) {
  using L = Narrow<16>;
  constexpr int kN = 16, kKeys = 24;  // rows; a thread's keys of a tile
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int32_t m = lane & 15;
  const int slice = warp;
  const bool mine = lane < 16;
  const int32_t tok = m / a.heads, head = m - tok * a.heads;
  const uint32_t lane_base = tmem + (uint32_t(warp) << 21);
  const uint32_t p_row = base + L::kOffP + m * 128;
  const float scale = a.scale_log2 == 0.f ? 1.f : fabsf(a.scale_log2);
  const uint64_t k0 = smem_desc(base + kOffK, 16, 1024, kSw128);
  const uint32_t pv = uint32_t(warp) - 1;  // warps 1 and 2: blocks 2 pv and 2 pv + 1
  const uint64_t v0 = smem_desc(base + kOffK + (pv & 1) * 4 * L::kBlock, L::kBlock, 1024, kSw128);
  const uint64_t p0 = smem_desc(base + L::kOffP, 16, 1024, kSw128);
  Units units;
  units.start(a, ms);
  Unit u;
  uint32_t g = 0;
  // (a wait that gives up does not end this role: its warps meet at named barriers)
  if (ms->stall) meet_after(ms, a, &ms->never, 0);
  while (units.next_inline(a, u)) {
    const int32_t rows = u.tokens * a.heads, t0 = u.t0, t1 = u.t1;
    const int32_t key0 = t0 * kTileKeys, stop = t1 * kTileKeys, end = min(u.end, stop);
    const bool live = mine && m < rows;
    const int32_t see = a.causal && live ? max(min(u.pos0 + tok + 1, end), 0) : end;
    float ref = -INFINITY, l = 0.f;
    // q (every warp has seen the last QK and PV of the unit before done)
    load_q_tmem(a, base + L::kOffP, lane_base + kTmemQFew, u.row0, rows);
    group_barrier(1, 128);
    if (warp == 0) few_issue_qk(a, ms, k0, tmem, g);
    for (int32_t key = key0; key < stop; key += L::kKeys, ++g) {
      const uint32_t stage = g & 1;
      meet_after(ms, a, &ms->qk_done[stage], (g >> 1) & 1);
      tc_fence_after();
      float x[kKeys];
      {
        uint32_t s0[16], s1[8];
        tmem_ld16(lane_base + kTmemSFew + kKeys * slice, s0);
        tmem_ld8(lane_base + kTmemSFew + kKeys * slice + 16, s1);
        tmem_wait_ld();
#pragma unroll
        for (int c = 0; c < 16; ++c) x[c] = __uint_as_float(s0[c]);
#pragma unroll
        for (int c = 0; c < 8; ++c) x[16 + c] = __uint_as_float(s1[c]);
      }
      const uint8_t* f = &ms->flags_few[g & 3][3 * slice];
      const uint32_t flags = f[0] | uint32_t(f[1]) << 8 | uint32_t(f[2]) << 16;
      if (a.scale_log2 <= 0.f) {
        const float by = a.scale_log2 < 0.f ? -1.f : 0.f;
#pragma unroll
        for (int c = 0; c < kKeys; ++c) x[c] *= by;
      }
      const int32_t n = see - key - kKeys * slice;
      if (__any_sync(0xffffffffu, n < kKeys) || flags != 0) {
        const uint32_t seen = ~flags & (n >= 32 ? ~0u : n <= 0 ? 0u : (1u << n) - 1u);
#pragma unroll
        for (int c = 0; c < kKeys; ++c) x[c] = (seen >> c) & 1u ? x[c] : -INFINITY;
      }
      float tm = x[0];
#pragma unroll
      for (int c = 1; c < kKeys; ++c) tm = fmaxf(tm, x[c]);
      ms->tmax[stage][warp * 32 + lane] = tm;
      group_barrier(1, 128);
#pragma unroll
      for (int k = 1; k < 4; ++k) tm = fmaxf(tm, ms->tmax[stage][(warp ^ k) * 32 + lane]);
      tm *= scale;
      const bool move = live && tm > ref + kMoveMargin;
      const float nref = move ? tm : ref;
      const float use = nref == -INFINITY ? 0.f : nref;
      const float alpha = move ? ex2(ref - use) : 1.f;
      ref = nref;
      uint32_t p[kKeys / 2];
      float sum0 = 0.f, sum1 = 0.f;
#pragma unroll
      for (int c = 0; c < kKeys / 2; ++c) {
        float y0, y1;
        fma2(x[2 * c], x[2 * c + 1], scale, -use, y0, y1);
        y0 = ex2(y0);
        y1 = ex2(y1);
        add2(sum0, sum1, y0, y1, sum0, sum1);
        p[c] = pack_bf16x2(y0, y1);
      }
      l = l * alpha + (sum0 + sum1);
      if (g > 0) meet_after(ms, a, &ms->pv_done[stage ^ 1], ((g - 1) >> 1) & 1);
      if (key > key0 && __any_sync(0xffffffffu, move)) {
        tc_fence_after();
#pragma unroll 1
        for (int c = 0; c < 4 * kN; c += 16) {
          uint32_t o[16];
          tmem_ld16(lane_base + c, o);
          tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < 16; ++i)
            o[i] = __float_as_uint(__uint_as_float(o[i]) * __shfl_sync(0xffffffffu, alpha, i));
          tmem_st16(lane_base + c, o);
        }
        tmem_wait_st();
      }
      if (mine) {  // P: two blocks of 64 and 32 keys
#pragma unroll
        for (int i = 0; i < kKeys / 8; ++i) {
          const int c = slice * (kKeys / 8) + i;
          st_shared_v4(p_row + (c >> 3) * (kN * 128) + (((c & 7) ^ (m & 7)) << 4), p[4 * i], p[4 * i + 1], p[4 * i + 2],
                       p[4 * i + 3]);
        }
      }
      fence_proxy_async_smem();
      tc_fence_before();
      group_barrier(2, 128);  // P is stored, S read
      if (warp == 0) {
        if (key + L::kKeys < stop) few_issue_qk(a, ms, k0, tmem, g + 1);
      } else if (warp < 3) {
        tc_fence_after();
        const uint64_t vd = v0 + uint64_t((stage * L::kStage) >> 4);
        if (elect_one()) {
#pragma unroll
          for (int b = 0; b < 2; ++b)
#pragma unroll
            for (int k = 0; k < L::kKeys / 16; ++k)
              mma_f16_ss(tmem + (2 * pv + b) * kN, vd + uint64_t((b * 2 * L::kBlock + k * 2048) >> 4),
                         p0 + uint64_t(((k >> 2) * (kN * 128) + (k & 3) * 32) >> 4), idesc_bf16(128, kN, 1, 0),
                         (key == key0 && k == 0) ? 0u : 1u);
          mma_commit(&ms->pv_done[stage]);
        }
        __syncwarp();
      }
    }
    const bool whole = t0 == 0 && t1 == u.tiles;
    const int64_t part = 2 * int64_t(worker) + (t0 > 0 ? 0 : 1);
    ms->lsum[warp * 32 + lane] = l;
    group_barrier(1, 128);
    l = 0.f;
#pragma unroll
    for (int k = 0; k < 4; ++k) l += ms->lsum[(warp ^ k) * 32 + lane];
    if (mine && slice == 0) {
      float factor = 1.f;
      if (whole) {
        float lse;
        finish_row(a, head, ref, l, &factor, &lse);
        if (live && a.lse) a.lse[(int64_t(u.row0) + tok) * a.heads + head] = lse;
      } else if (live) {
        a.ml_part[(part * a.part_rows + m) * 2] = ref;
        a.ml_part[(part * a.part_rows + m) * 2 + 1] = l;
      }
      ms->factor[m] = factor;
    }
    group_barrier(1, 128);
    meet_after(ms, a, &ms->pv_done[(g - 1) & 1], ((g - 1) >> 1) & 1);
    tc_fence_after();
    // a lane has dim 128 b + 32 warp + lane of every row
    const int32_t dim = 32 * warp + lane;
    int32_t r_tok = 0, r_head = 0;
#pragma unroll 1
    for (int c = 0; c < rows; c += 16) {
      uint32_t o[4][16];
#pragma unroll
      for (int b = 0; b < 4; ++b) tmem_ld16(lane_base + b * kN + c, o[b]);
      tmem_wait_ld();
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        if (c + i >= rows) break;
        if (whole) {
          const float f = ms->factor[c + i];
          uint16_t* dst = a.out + (int64_t(u.row0) + r_tok) * a.o_row + int64_t(r_head) * a.o_head + dim;
#pragma unroll
          for (int b = 0; b < 4; ++b) dst[128 * b] = uint16_t(pack_bf16x2(__uint_as_float(o[b][i]) * f, 0.f));
        } else {
          float* dst = a.o_part + (part * a.part_rows + c + i) * kLatent + dim;
#pragma unroll
          for (int b = 0; b < 4; ++b) dst[128 * b] = __uint_as_float(o[b][i]);
        }
        if (++r_head == a.heads) r_head = 0, ++r_tok;
      }
    }
    tc_fence_before();
    if (!whole && t0 > 0 && t1 == u.tiles && threadIdx.x == 0) name_merge(a, ms, worker, u);
  }
}

__global__ void __launch_bounds__(kNarrowThreads, 1) paged_attend_few_kernel(const __grid_constant__ AttendArgs a) {
  extern __shared__ __align__(1024) uint8_t raw_smem[];
  const uint32_t base = smem_u32(raw_smem);
  const int32_t worker = blockIdx.x;
  const int warp = threadIdx.x >> 5;
  let_dependents_launch();
  if (threadIdx.x == 0) a.merge[worker * 4] = 0;
  if (base & 1023u) {
    if (threadIdx.x == 0 && a.b.status) atomicOr(a.b.status, SMLA_STATUS_SMEM_LAYOUT);
    return;
  }
  Misc* ms = reinterpret_cast<Misc*>(raw_smem + Narrow<16>::kOffMisc);
  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&ms->k_full[i], Narrow<16>::kLoaders);
      mbar_init(&ms->qk_done[i], 1);
      mbar_init(&ms->pv_done[i], 2);
    }
    mbar_init(&ms->drain, 3);
    mbar_init(&ms->never, 1);
    fence_mbar_init();
    ms->dead = 0;
    ms->wait_ns = g_paged_wait_ns ? g_paged_wait_ns : kWaitNs;
    ms->stall = g_paged_stall;
  }
  if (warp == 3) {
    tmem_alloc(&ms->tmem, kTmemCols);
    tc_fence_before();
  }
  find_range<kNarrowThreads>(a, ms, worker);
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ms->tmem;
  if (warp < kFirstLoader) {
    few_compute_role(a, ms, base, tmem, worker);
    // every MMA complete before the memory it reads goes away
    __syncwarp();
    if (warp < 3 && elect_one()) {  // (the lane that issued them: the same for the same mask)
      mma_commit(&ms->drain);
      if (!mbar_wait(&ms->drain, 0, kWaitNs)) give_up(ms, a.b.status);
    }
  } else {
    narrow_loader_role<16>(a, ms, base);
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 3) {
    tmem_relinquish();
    tmem_dealloc(tmem, kTmemCols);
  }
}

// The worker whose job a block of a merge kernel takes: blockIdx.x, or in grids of as
// many blocks as there may be jobs (kSearch) the blockIdx.x-th that named one.
template <bool kSearch>
__device__ __forceinline__ int32_t merge_job(const AttendArgs& a) {
  if (!kSearch) return blockIdx.x;
  const int lane = threadIdx.x & 31;
  int32_t last = -1;
  for (int32_t base = 0, seen = 0; base < a.workers && last < 0; base += 256) {
    int32_t named[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int32_t w = base + 32 * i + lane;
      named[i] = w < a.workers ? a.merge[4 * w] : 0;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t mask = __ballot_sync(0xffffffffu, named[i] > 0);
      const int32_t nth = int32_t(blockIdx.x) - seen;
      if (nth >= 0 && nth < __popc(mask)) last = base + 32 * i + int32_t(__fns(mask, 0, nth + 1));
      seen += __popc(mask);
    }
  }
  return last;
}

// Joins the partials of a row tile shared between workers: with m = max_c m_c,
//   l = sum_c l_c 2^(m_c - m),  O = sum_c O_c 2^(m_c - m),
// and the sink enters once.  The parts (up to one a worker) come from L2, whose
// latency is the cost: a warp takes a quarter of a row's dims, so that a merge of
// few rows and many parts is spread over many SMs, and keeps 8 parts' loads in
// flight.  With kGroups = 2, for row tiles of many parts, two warps share a quarter's
// parts and meet in shared memory.
template <int kGroups>
__global__ void __launch_bounds__(kGroups == 1 ? 256 : 128 * kGroups) paged_merge_kernel(const __grid_constant__ AttendArgs a) {
  constexpr int kRows = kGroups == 1 ? 2 : 1;  // of a block
  constexpr int kFlight = 8;
  __shared__ float4 o_sum[kGroups][128];
  __shared__ float l_sum[kGroups];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int quarter = warp & 3, group = kGroups == 1 ? 0 : warp >> 2;
  const int32_t m = blockIdx.y * kRows + (kGroups == 1 ? warp >> 2 : 0);
  wait_for_primary();
  const int32_t last = merge_job<(kGroups > 1)>(a);
  if (last < 0) return;
  const int4 job = *reinterpret_cast<const int4*>(a.merge + last * 4);
  if (m >= job.x) return;
  const int32_t first = job.z;
  auto part_of = [&](int32_t c) -> int64_t { return (2 * int64_t(c) + (c == first ? 1 : 0)) * a.part_rows + m; };
  float mx = -INFINITY;
  for (int32_t c = first + lane; c <= last; c += 32) mx = fmaxf(mx, a.ml_part[part_of(c) * 2]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
  const float use = mx == -INFINITY ? 0.f : mx;
  float l = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  const int32_t at = 128 * quarter + 4 * lane;
  for (int32_t c0 = first + group; c0 <= last; c0 += 32 * kGroups) {
    // lane i: weight and weighted sum of part c0 + kGroups i
    float2 ml = make_float2(-INFINITY, 0.f);
    if (c0 + kGroups * lane <= last) ml = *reinterpret_cast<const float2*>(a.ml_part + part_of(c0 + kGroups * lane) * 2);
    const float wgt = ex2(ml.x - use);
    l += ml.y * wgt;
    const int32_t n = min((last - c0) / kGroups + 1, 32);
    for (int32_t i = 0; i < n; i += kFlight) {
      float4 v[kFlight];
#pragma unroll
      for (int k = 0; k < kFlight; ++k) {
        v[k] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (i + k < n)
          v[k] = __ldcg(reinterpret_cast<const float4*>(a.o_part + part_of(c0 + kGroups * (i + k)) * kLatent + at));
      }
#pragma unroll
      for (int k = 0; k < kFlight; ++k) {
        const float f = __shfl_sync(0xffffffffu, wgt, (i + k) & 31);
        if (i + k < n) o.x += v[k].x * f, o.y += v[k].y * f, o.z += v[k].z * f, o.w += v[k].w * f;
      }
    }
  }
#pragma unroll
  for (int k = 16; k > 0; k >>= 1) l += __shfl_xor_sync(0xffffffffu, l, k);
  if constexpr (kGroups > 1) {
    o_sum[group][32 * quarter + lane] = o;
    if (quarter == 0 && lane == 0) l_sum[group] = l;
    __syncthreads();
    if (group != 0) return;
#pragma unroll
    for (int g = 1; g < kGroups; ++g) {
      const float4 v = o_sum[g][32 * quarter + lane];
      o.x += v.x, o.y += v.y, o.z += v.z, o.w += v.w;
      l += l_sum[g];
    }
  }
  const int32_t tok = m / a.heads, head = m - tok * a.heads;
  const int64_t tok_row = int64_t(job.y) + tok;
  float factor, lse;
  finish_row(a, head, mx, l, &factor, &lse);
  if (lane == 0 && quarter == 0 && a.lse) a.lse[tok_row * a.heads + head] = lse;
  uint2 v = make_uint2(pack_bf16x2(o.x * factor, o.y * factor), pack_bf16x2(o.z * factor, o.w * factor));
  if (l == 0.f) v = make_uint2(0, 0);
  *reinterpret_cast<uint2*>(a.out + tok_row * a.o_row + int64_t(head) * a.o_head + at) = v;
}

// The same for the pair kernel's partials, which lie as its threads (one a row) write
// them: O of a part as [512 / 4][128 rows][4].  A lane takes a row, a warp 16 dims of
// 32 rows.  One pass: the sums are rescaled when the maximum moves.
template <int kGroups>
__global__ void __launch_bounds__(kGroups == 1 ? 256 : 128 * kGroups)
paged_merge_pair_kernel(const __grid_constant__ AttendArgs a) {
  constexpr int kDimWarps = kGroups == 1 ? 8 : 4, kDims = 16, kSplit = kLatent / (kDims * kDimWarps);
  constexpr int kFlight = 4;
  __shared__ float4 o_sum[kGroups == 1 ? 1 : kGroups][kDims / 4][kDimWarps * 32];
  __shared__ float2 ml_sum[kGroups][kDimWarps * 32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int dim_warp = warp % kDimWarps, group = warp / kDimWarps;
  const int32_t m0 = blockIdx.y / kSplit * 32, m = m0 + lane;
  const int32_t at = kDims * (blockIdx.y % kSplit * kDimWarps + dim_warp);
  wait_for_primary();
  const int32_t last = merge_job<(kGroups > 1)>(a);
  if (last < 0) return;
  const int4 job = *reinterpret_cast<const int4*>(a.merge + last * 4);
  if (m0 >= job.x) return;
  const bool live = m < job.x;
  const int32_t first = job.z;
  float mx = -INFINITY, l = 0.f;
  float4 o[kDims / 4];
#pragma unroll
  for (int i = 0; i < kDims / 4; ++i) o[i] = make_float4(0.f, 0.f, 0.f, 0.f);
  // joins one more sum with its own maximum
  auto add = [&](const float2& ml, const float4 (&v)[kDims / 4]) {
    const float nm = fmaxf(mx, ml.x), use = nm == -INFINITY ? 0.f : nm;
    const float f = ex2(mx - use), w = ex2(ml.x - use);
    mx = nm;
    l = l * f + ml.y * w;
#pragma unroll
    for (int i = 0; i < kDims / 4; ++i) {
      o[i].x = o[i].x * f + v[i].x * w, o[i].y = o[i].y * f + v[i].y * w;
      o[i].z = o[i].z * f + v[i].z * w, o[i].w = o[i].w * f + v[i].w * w;
    }
  };
  for (int32_t c0 = first + group; c0 <= last; c0 += kGroups * kFlight) {
    float2 ml[kFlight];
    float4 v[kFlight][kDims / 4];
#pragma unroll
    for (int k = 0; k < kFlight; ++k) {
      const int32_t c = c0 + kGroups * k;
      ml[k] = make_float2(-INFINITY, 0.f);
#pragma unroll
      for (int i = 0; i < kDims / 4; ++i) v[k][i] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (c > last || !live) continue;  // (rows behind the last hold nothing)
      const int64_t part = 2 * int64_t(c) + (c == first ? 1 : 0);
      ml[k] = *reinterpret_cast<const float2*>(a.ml_part + (part * kPairRows + m) * 2);
#pragma unroll
      for (int i = 0; i < kDims / 4; ++i)
        v[k][i] = __ldcg(reinterpret_cast<const float4*>(a.o_part + (part * kLatent + at + 4 * i) * kPairRows + m * 4));
    }
#pragma unroll
    for (int k = 0; k < kFlight; ++k)
      if (c0 + kGroups * k <= last) add(ml[k], v[k]);
  }
  if constexpr (kGroups > 1) {
    const int at_sum = dim_warp * 32 + lane;
    ml_sum[group][at_sum] = make_float2(mx, l);
#pragma unroll
    for (int i = 0; i < kDims / 4; ++i) o_sum[group][i][at_sum] = o[i];
    __syncthreads();
    if (group != 0) return;
#pragma unroll
    for (int g = 1; g < kGroups; ++g) {
      float4 v[kDims / 4];
#pragma unroll
      for (int i = 0; i < kDims / 4; ++i) v[i] = o_sum[g][i][at_sum];
      add(ml_sum[g][at_sum], v);
    }
  }
  if (!live) return;
  const int32_t tok = m / a.heads, head = m - tok * a.heads;
  const int64_t tok_row = int64_t(job.y) + tok;
  float factor, lse;
  finish_row(a, head, mx, l, &factor, &lse);
  if (at == 0 && a.lse) a.lse[tok_row * a.heads + head] = lse;
  uint32_t v[kDims / 2];
#pragma unroll
  for (int i = 0; i < kDims / 4; ++i) {
    v[2 * i] = l == 0.f ? 0u : pack_bf16x2(o[i].x * factor, o[i].y * factor);
    v[2 * i + 1] = l == 0.f ? 0u : pack_bf16x2(o[i].z * factor, o[i].w * factor);
  }
  uint16_t* dst = a.out + tok_row * a.o_row + int64_t(head) * a.o_head + at;
  *reinterpret_cast<uint4*>(dst) = make_uint4(v[0], v[1], v[2], v[3]);
  *reinterpret_cast<uint4*>(dst + 8) = make_uint4(v[4], v[5], v[6], v[7]);
}

}  // namespace

// Rows of a narrow tile (16, 32, 64), or 0 for the pair kernel: by the mean number
// of rows (tokens x heads) of a sequence, since the lengths themselves are on the
// device.  Any split is computed correctly by either.  Measured at 64 sequences of
// 4096 positions (graph replays, us; rows: few-row kernel / narrow tiles of 32 / of 64 /
// pair kernel):
//   16: 63 / 77 / 78 / 99    24: - / 78 / 80 / 100    32: 106 / 80 / 82 / 100
//   64: 192 / 140 / 88 / 104    96: 273 / 201 / 148 / 106    128: - / - / 154 / 108
// One kernel serves the whole call, so a batch of unlike sequences gets what its mean
// gives: 63 single tokens and one of two, 16 heads, take 77 us in tiles of 32 (63 without
// the second token); 63 tokens and a chunk of 512 177 us in one call, 63 + 97 as two;
// 255 tokens and the chunk 373, 191 + 97 as two.  Empty sequences count: a chunk of 2048
// tokens, 4 heads, takes 84 us alone or among 64 sequences, 276 among 512.
static int narrow_rows(const smla_paged_attend_params& p) {
  if (p.num_heads > kCtaRows) return 0;
  const int64_t mean = (p.batch.n_rows * p.num_heads + p.batch.n_seqs - 1) / p.batch.n_seqs;
  if (mean > kCtaRows) return 0;
  const int64_t rows = mean > p.num_heads ? mean : p.num_heads;
  return rows <= 16 ? 16 : rows <= 32 ? 32 : 64;
}

// The plan of one kernel (narrow as in AttendPlan).
static AttendPlan plan_of_kernel(const smla_paged_attend_params& p, int num_sms, int narrow) {
  AttendPlan plan{};
  const smla_paged_batch& b = p.batch;
  plan.narrow = narrow;
  plan.part_rows = plan.narrow ? kCtaRows : kPairRows;
  const int64_t tokens = (plan.narrow ? plan.narrow : kPairRows) / p.num_heads;
  const int64_t coverage = int64_t(b.max_pages) * b.page_size;
  const int64_t most_tiles = coverage > 0 ? (coverage + kTileKeys - 1) / kTileKeys : 1;
  const int64_t row_tiles = (b.n_rows + tokens - 1) / tokens + (b.n_rows < b.n_seqs ? b.n_rows : int64_t(b.n_seqs));
  plan.start_slots = plan.narrow == 16 ? kFewStart : plan.narrow ? kNarrowStart : kPairStart;
  const int64_t slots = row_tiles * (most_tiles + plan.start_slots);
  int64_t workers = plan.narrow ? num_sms : num_sms / 2;
  if (slots < workers) workers = slots;
  plan.workers = int32_t(workers < 1 ? 1 : workers);
  plan.merge_tiles = int32_t(row_tiles < plan.workers ? row_tiles : plan.workers);
  plan.merge_off = 0;
  plan.ml_off = (int64_t(plan.workers) * 16 + 255) & ~int64_t(255);
  plan.o_off = plan.ml_off + ((int64_t(plan.workers) * 2 * plan.part_rows * 8 + 255) & ~int64_t(255));
  plan.total = plan.o_off + int64_t(plan.workers) * 2 * plan.part_rows * kLatent * 4;
  return plan;
}

// The workspace is as large as the largest that any kernel would take for these sizes.
// Each kernel's grows with the rows, sequences and pages, so theirs does too, and a
// workspace for a batch serves every smaller one, whichever kernel that gets.
AttendPlan paged_attend_plan(const smla_paged_attend_params& p, int num_sms) {
  if (p.batch.n_rows <= 0 || p.batch.n_seqs <= 0) return AttendPlan{};
  AttendPlan plan = plan_of_kernel(p, num_sms, narrow_rows(p));
  for (const int narrow : {0, 16, 32, 64}) {
    if (narrow != 0 && narrow < p.num_heads) continue;
    const int64_t total = plan_of_kernel(p, num_sms, narrow).total;
    if (total > plan.total) plan.total = total;
  }
  return plan;
}

static cudaError_t launch_narrow(void (*kernel)(AttendArgs), int smem, const AttendArgs& a, cudaStream_t stream) {
  const cudaError_t err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (err != cudaSuccess) return err;
  kernel<<<a.workers, kNarrowThreads, smem, stream>>>(a);
  return cudaGetLastError();
}

static cudaError_t launch_merge(void (*kernel)(AttendArgs), const AttendArgs& a, dim3 grid, int threads,
                                cudaStream_t stream) {
  cudaLaunchConfig_t config{};
  config.gridDim = grid;
  config.blockDim = dim3(unsigned(threads));
  config.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  config.attrs = attr;
  config.numAttrs = 1;
  return cudaLaunchKernelEx(&config, kernel, a);
}

cudaError_t launch_paged_attend(const smla_paged_attend_params& p, const AttendPlan& plan, void* workspace,
                                cudaStream_t stream) {
  AttendArgs a{};
  a.b = make_paged_args(p.batch);
  a.q = static_cast<const uint16_t*>(p.q);
  a.q_row = p.q_stride_row;
  a.q_head = p.q_stride_head;
  a.out = static_cast<uint16_t*>(p.out);
  a.o_row = p.out_stride_row;
  a.o_head = p.out_stride_head;
  a.lse = p.lse;
  a.sink = p.sink;
  a.scale_log2 = p.sm_scale * kLog2e;
  a.heads = p.num_heads;
  a.tokens = (plan.narrow ? plan.narrow : kPairRows) / p.num_heads;
  a.causal = p.causal != 0;
  a.workers = plan.workers;
  a.part_rows = plan.part_rows;
  a.start_slots = plan.start_slots;
  a.coverage = p.batch.max_pages * p.batch.page_size;
  char* ws = static_cast<char*>(workspace);
  a.merge = reinterpret_cast<int32_t*>(ws + plan.merge_off);
  a.ml_part = reinterpret_cast<float*>(ws + plan.ml_off);
  a.o_part = reinterpret_cast<float*>(ws + plan.o_off);
  cudaError_t err;
  if (plan.narrow == 16) {
    err = launch_narrow(paged_attend_few_kernel, kNarrowSmem<16>, a, stream);
  } else if (plan.narrow == 32) {
    err = launch_narrow(paged_attend_narrow_kernel<32>, kNarrowSmem<32>, a, stream);
  } else if (plan.narrow == 64) {
    err = launch_narrow(paged_attend_narrow_kernel<64>, kNarrowSmem<64>, a, stream);
  } else {
    err = cudaFuncSetAttribute(paged_attend_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kAttendSmem);
    if (err != cudaSuccess) return err;
    paged_attend_kernel<<<2 * plan.workers, kAttendThreads, kAttendSmem, stream>>>(a);
    err = cudaGetLastError();
  }
  if (err != cudaSuccess || plan.workers == 1) return err;
  // Row tiles of 8 parts or more on average: several warps share a row's parts, and the
  // grid is as large as the row tiles, not as the workers (4 x 64 heads, 38 parts: 42.9 us
  // with the other form, 36.3 with this; four groups: 40.3; 2 x 2 x 64 heads in the pair
  // kernel: 23.0, 20.1, with two groups 21.5).  With fewer parts a search of the job
  // costs more than it saves (64 x 16 heads: 60 -> 64 us)
  const bool many = plan.workers >= 8 * plan.merge_tiles;
  const unsigned jobs = unsigned(many ? plan.merge_tiles : plan.workers);
  if (plan.narrow) {
    if (many) return launch_merge(paged_merge_kernel<2>, a, dim3(jobs, unsigned(plan.narrow)), 256, stream);
    return launch_merge(paged_merge_kernel<1>, a, dim3(jobs, unsigned(plan.narrow) / 2), 256, stream);
  }
  if (many) return launch_merge(paged_merge_pair_kernel<4>, a, dim3(jobs, 32), 512, stream);
  return launch_merge(paged_merge_pair_kernel<1>, a, dim3(jobs, 16), 256, stream);
}

cudaError_t paged_set_wait_limit(uint64_t ns, int stall) {
  const int32_t s = stall;
  const cudaError_t err = cudaMemcpyToSymbol(g_paged_wait_ns, &ns, sizeof(ns));
  return err != cudaSuccess ? err : cudaMemcpyToSymbol(g_paged_stall, &s, sizeof(s));
}

}  // namespace smla
