// pkv_latent_decode.cu - attention of new tokens over a paged cache of shared latents
// (the absorbed form) on tcgen05 tensor cores, two CTAs to a tile.
//
// A cache row c_t (576 values) is key to every head, and its first 512 values are the
// value: with x[t] = scale q . c_t over the keys a query sees,
//   lse = ln sum_t exp x[t],   out = sum_t exp(x[t] - lse) c_t[0:512].
// All heads of a sequence share the rows, so its query rows (tokens x heads, up to 128
// at a time) are the M axis of two products per tile of 128 keys:
//   S = Q C^T  [128 x 128 x 576],   O += P C[:, 0:512]  [128 x 512 x 128].
// With 128 query rows that is 242 operations a byte of cache, and the card's balance is
// ~290: memory bounds the kernel, if the tensor cores run close to their rate.
//
// Why a pair of CTAs (cta_group::2, M = 128). O of 128 rows is 128 x 512 fp32, the whole
// tensor memory of an SM, and S has to go somewhere. A pair halves it: each CTA holds 64
// query rows in 128 lanes (lanes 0-63: the first half of a product's columns, lanes 64-127
// the second half of the same rows), so that O takes 256 columns and two S buffers 128.
// Each CTA also brings only half of every product's B operand:
//   S:  its 64 keys of the tile, all 576 dims     (72 KB, one tile in shared memory)
//   PV: its 256 dims of the values, all 128 keys  (64 KB, one tile)
// The two overlap in content, but an operand of a pair lies at one offset in both CTAs,
// and the keys of a CTA at that offset differ for S while they agree for PV; so what both
// need is loaded twice, the second time from L2. (Measured as loads alone, with 17 slots
// of 8 KB in flight: 6.76 TB/s of distinct cache rows, 12.8 TB/s into the SMs; the copy
// bandwidth is 6.78.) The MMAs of a tile take ~2200-2500 cycles, its bytes ~3300.
//
// Roles per CTA: warps 0 and 6 load (TMA through the page table); warps 1 and 7 issue the MMAs
// (CTA 0's, for the pair); warps 2-5 are softmax and epilogue, lanes l and l + 64 sharing row l.
//
// Work: where the (sequence, 128-row block) items are no more than the pairs of CTAs, each pair
// takes one item or an equal part of one; the parts are as short as their number allows, unless
// whole items are about as short. Else the items' tiles in a row are cut into equal ranges. Parts
// of an item leave unnormalised partials, which a second kernel joins.
#include <algorithm>
#include <atomic>
#include <cfloat>
#include <cmath>

#include "pkv_latent.cuh"
#include "pkv_latent_schedule.h"

namespace pkv {
namespace {

using namespace latent;
using namespace prefill_detail;

constexpr int kKeys = 128;                 // keys of a tile
constexpr int kRows = 128;                 // query rows of an item
constexpr int kChunk = 64 * 128;           // [64 rows x 64 values], 128-byte swizzled: 8 KB
constexpr int kChunks = kRow / 64;         // 9
constexpr int kKGroups = 3;                // S's loads and barriers: three chunks at a time
constexpr int kVGroups = 2;                // PV's: the CTA's dims 0-127 and 128-255
constexpr int kLatThreads = 8 * 32;
constexpr int kAhead = 1;                  // tiles whose rows are asked for in L2 ahead
constexpr int kMaxRowsPerLaunch = 512;     // sequences of one launch

// shared memory, offsets from a 1024-aligned base
constexpr int kOffQ = 0;                              // [9 chunks][64 query rows]
constexpr int kOffK = kOffQ + kChunks * kChunk;       // [9 chunks][64 own keys]
constexpr int kOffV = kOffK + kChunks * kChunk;       // [2 key halves][4 own chunks][64 keys]
constexpr int kOffP = kOffV + 8 * kChunk;             // [2 key halves][64 query rows]
constexpr int kOffBar = kOffP + 2 * kChunk;
constexpr int kNumBars = 2 * kKGroups + 2 * kVGroups + 9;
constexpr int kOffMisc = kOffBar + kNumBars * 8;      // tmem slot, abort flag, 7 of the schedule
constexpr int kOffMax = kOffMisc + 36;                // [2][128] row maxima, [128] sums
constexpr int kLatSmem = kOffMax + 3 * 128 * 4 + 1024;  // + slack for the alignment
static_assert(kLatSmem <= kMaxDynSmem, "shared memory above the opt-in limit");

constexpr uint32_t kColS = 256;            // TMEM: O in columns 0-255, S in 256 + 64 * buffer
constexpr uint32_t kIdescS = idesc_bf16_f32(kRows, kKeys, false);
constexpr uint32_t kIdescO = idesc_bf16_f32(kRows, 256, true);

// n / d for 0 <= n < 2^31 as a product: with 2^(l-1) < d <= 2^l and m = floor(2^(31+l) / d) + 1
// (below 2^32), n m / 2^(31+l) exceeds n / d by less than 1 / d.
struct Divisor {
  uint32_t m;
  int shift;
  int d;
};
inline Divisor make_divisor(int d) {
  int l = 0;
  while ((1ll << l) < d) ++l;
  return {static_cast<uint32_t>((1ull << (31 + l)) / d + 1), 31 + l, d};
}
__device__ __forceinline__ int div_by(int n, const Divisor& v) {
  return static_cast<int>((static_cast<uint64_t>(static_cast<uint32_t>(n)) * v.m) >> v.shift);
}

struct LatentDecodeParams {
  const __nv_bfloat16* pool;
  const int32_t* page_table;
  const int32_t* batch_idx;
  const int32_t* seq_lens;
  __nv_bfloat16* out;      // [batch, n_q * heads, 512]
  float* lse;              // [batch, n_q * heads]
  float* part_o;           // [2 * workers][block_rows][512]
  float* part_ml;          // [2 * workers][block_rows][2]
  int4* part_item;         // [workers]: parts of the item that the range ends (0: none), its place
  int32_t* dev_err;
  int batch;
  Divisor heads;
  int n_q;
  int rows;                // n_q * heads
  Divisor row_blocks;      // ceil(rows / 128)
  int block_rows;          // min(rows, 128): rows of a partial
  Divisor page_size;
  int num_pages;
  int max_batch;
  int max_blocks;
  int box_rows;            // rows of one TMA box: 16, 32 or 64
  Divisor workers;         // pairs of CTAs
  float qscale;            // scale * log2(e)
};

// ------------------------------------------------------ pair instructions --

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync_all() {
  asm volatile(
      "barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::
          : "memory");
}
// The address in CTA `rank` of the pair of what lies at `p` in this one.
__device__ __forceinline__ uint32_t peer_u32(const void* p, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(smem_u32(p)), "r"(rank));
  return r;
}
// What CTA 1's softmax threads hand over to the MMAs (P and zeroed values in its shared memory; S
// that they have read and O that they have rescaled, behind tcgen05 fences) is waited for by threads
// of CTA 0. Arrives and waits have CTA scope by default and order nothing between threads of two
// CTAs, so here both have cluster scope. The release is a fence of this CTA's shared memory alone:
// an arrive with .release.cluster waits for all of the SM's memory traffic, loads by TMA included
// (64 x ~768 keys, 128 heads: 24.7 us with the fence, 30.1 with that; 16 x ~20000, 128 rows: 75.4
// and 91.6; 64 x 4096, 16 heads: 57.3 and 89.1). With CTA scope on both sides it is 24.7 and 75.5.
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t bar) {
  asm volatile(
      "fence.release.sync_restrict::shared::cta.cluster;\n\t"
      "mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar)
      : "memory");
}
__device__ __forceinline__ bool wait_phase_cluster(uint64_t* bar, uint32_t parity,
                                                   volatile int* abort_flag) {
  WaitLimit limit;
  for (;;) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity)
        : "memory");
    if (ok) return true;
    if (limit.over(abort_flag)) return false;
  }
}
// One box of a tiled load whose bytes count on a barrier of either CTA of the pair.
__device__ __forceinline__ void tma_load_3d_pair(void* dst, const CUtensorMap* map, uint32_t bar,
                                                 int x, int y, int z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y), "r"(z)
      : "memory");
}

// Arrives on the barrier at this offset in both CTAs once the MMAs issued so far are done.
__device__ __forceinline__ void commit_pair(uint64_t* bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64"
      " [%0], %1;" ::"r"(smem_u32(bar)),
      "h"(static_cast<uint16_t>(3))
      : "memory");
}

// Four K-steps of a product of the pair. a_lo, b_lo: low descriptor words of the first
// step; kStepA, kStepB: bytes from one step to the next. With the descriptors made ahead
// of the four instructions nothing is issued between them.
template <int kStepA, int kStepB>
__device__ __forceinline__ void umma4_pair(uint32_t d, uint32_t a_lo, uint32_t b_lo,
                                           uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p0, p1;\n\t.reg .b64 a<4>, b<4>;\n\t.reg .b32 x<4>, y<4>;\n\t"
      "setp.ne.b32 p0, %3, 0;\n\tsetp.eq.b32 p1, %3, %3;\n\t"
      "add.u32 x1, %1, %6;\n\tadd.u32 x2, x1, %6;\n\tadd.u32 x3, x2, %6;\n\t"
      "add.u32 y1, %2, %7;\n\tadd.u32 y2, y1, %7;\n\tadd.u32 y3, y2, %7;\n\t"
      "mov.b64 a0, {%1, %5};\n\tmov.b64 b0, {%2, %5};\n\t"
      "mov.b64 a1, {x1, %5};\n\tmov.b64 b1, {y1, %5};\n\t"
      "mov.b64 a2, {x2, %5};\n\tmov.b64 b2, {y2, %5};\n\t"
      "mov.b64 a3, {x3, %5};\n\tmov.b64 b3, {y3, %5};\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], a0, b0, %4, p0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], a1, b1, %4, p1;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], a2, b2, %4, p1;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], a3, b3, %4, p1;\n\t}" ::"r"(d),
      "r"(a_lo), "r"(b_lo), "r"(accumulate), "r"(idesc), "n"(kDescHi), "n"(kStepA >> 4),
      "n"(kStepB >> 4)
      : "memory");
}
__device__ __forceinline__ void umma1_pair(uint32_t d, uint32_t a_lo, uint32_t b_lo,
                                           uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\tsetp.ne.b32 p, %3, 0;\n\t"
      "mov.b64 a, {%1, %5};\n\tmov.b64 b, {%2, %5};\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], a, b, %4, p;\n\t}" ::"r"(d),
      "r"(a_lo), "r"(b_lo), "r"(accumulate), "r"(idesc), "n"(kDescHi)
      : "memory");
}

// Barrier of n threads that tells all of them whether v held for each.
__device__ __forceinline__ bool named_bar_all(int id, int n, bool v) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %3, 0;\n\t"
      "barrier.cta.red.and.pred q, %1, %2, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(id), "r"(n), "r"(v ? 1 : 0)
      : "memory");
  return r != 0;
}

// ------------------------------------------------------------------- work --

// Keys of a sequence's last query, 0 for padding and for rows that are refused (*err); its slot.
__device__ __forceinline__ int seq_keys(const LatentDecodeParams& p, int b, int* err, int* slot_out) {
  const int slot = __ldg(p.batch_idx + b);
  const int n = __ldg(p.seq_lens + b);
  *slot_out = slot;
  *err = 0;
  if (slot == 0) return 0;
  if (slot < 0 || slot >= p.max_batch) *err = PKV_DEV_ERR_BAD_SLOT;
  else if (n < 0 || n > p.max_blocks * p.page_size.d) *err = PKV_DEV_ERR_BAD_POS;
  return *err ? 0 : n;
}
__device__ __forceinline__ int key_tiles(int n) {
  return n / kKeys + (n % kKeys != 0);
}
// Whether the sequence of n keys ends inside a 16-key step of tile j: rows past its end, which
// may hold any bits, would take part in PV.
__device__ __forceinline__ bool ragged(int n, int j) {
  return n - j * kKeys < kKeys && (n & 15) != 0;
}

// One worker's walk over its range: an item's tiles j0 .. j1 - 1 at a time.
struct Walk {
  int x, end;          // flat tiles: behind the current segment, the range's end
  int b, base, n;      // sequence, the tiles before it, its keys
  int slot;
  int rb, nt, j0, j1;  // the segment's row block, tiles of its item, and range of tiles
};
__device__ __forceinline__ bool walk_next(const LatentDecodeParams& p, Walk& w) {
  if (w.x >= w.end) return false;
#pragma unroll 1
  for (;;) {
    w.nt = key_tiles(w.n);
    const int span = w.nt * p.row_blocks.d;
    if (w.x < w.base + span) break;
    w.base += span;
    int err;
    w.n = seq_keys(p, ++w.b, &err, &w.slot);
  }
  const int in = w.x - w.base;
  w.rb = p.row_blocks.d == 1 ? 0 : in / w.nt;
  w.j0 = in - w.rb * w.nt;
  w.j1 = min(w.nt, w.j0 + (w.end - w.x));
  w.x += w.j1 - w.j0;
  return true;
}

}  // namespace

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kLatThreads, 1)
latent_decode_kernel(const __grid_constant__ CUtensorMap qmap,
                     const __grid_constant__ CUtensorMap kmap,
                     const __grid_constant__ CUtensorMap vmap,
                     const LatentDecodeParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + kOffBar);
  uint64_t* k_full = bars;                    // [3] CTA 0: both CTAs' chunks have landed
  uint64_t* k_empty = k_full + kKGroups;      // [3] both: S has read them
  uint64_t* v_full = k_empty + kKGroups;      // [2] CTA 0: both CTAs' values have landed
  uint64_t* v_empty = v_full + kVGroups;      // [2] both: PV has read them
  uint64_t* q_full = v_empty + kVGroups;      // CTA 0
  uint64_t* q_empty = q_full + 1;             // both: the item's last S is done
  uint64_t* s_full = q_empty + 1;             // [2] both
  uint64_t* p_full = s_full + 2;              // [2] CTA 0: both CTAs' P is there, S has been read
  uint64_t* pv_done = p_full + 2;             // both
  uint64_t* o_free = pv_done + 1;             // CTA 0: both epilogues have read O
  uint64_t* v_tail = o_free + 1;              // each CTA: the values of a ragged tile
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + kOffMisc);
  volatile int* s_abort = reinterpret_cast<volatile int*>(smem + kOffMisc + 4);
  int* s_walk = reinterpret_cast<int*>(smem + kOffMisc + 8);  // [7]: the range and its first segment
  float* s_max = reinterpret_cast<float*>(smem + kOffMax);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();
  const int worker = blockIdx.x >> 1;

  if (threadIdx.x == 0) {
    for (int g = 0; g < kKGroups; ++g) {
      mbar_init(&k_full[g], 1);
      mbar_init(&k_empty[g], 1);
    }
    for (int g = 0; g < kVGroups; ++g) {
      mbar_init(&v_full[g], 1);
      mbar_init(&v_empty[g], 1);
    }
    mbar_init(q_full, 1);
    mbar_init(q_empty, 1);
    mbar_init(&s_full[0], 1);
    mbar_init(&s_full[1], 1);
    mbar_init(&p_full[0], 8);   // the four softmax warps of both CTAs
    mbar_init(&p_full[1], 8);
    mbar_init(pv_done, 1);
    mbar_init(o_free, 8);
    mbar_init(v_tail, 1);
    *s_abort = 0;
    fence_barrier_init();
    tma_prefetch_desc(&qmap);
    tma_prefetch_desc(&kmap);
    tma_prefetch_desc(&vmap);
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(tmem_slot)),
                 "r"(kTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  pdl_wait_primary();
  pdl_launch_dependents();

  // The schedule: every sequence's keys, in P's place in shared memory (no P is written before
  // all warps have read what follows); warp 0 finds this pair's range among their tiles and goes
  // on with its loads while the others read what it found. (What runs once costs mostly the
  // latency of its instructions: little code, loops not unrolled.)
  int* keys_of = reinterpret_cast<int*>(smem + kOffP);
#pragma unroll 1
  for (int b = threadIdx.x; b < p.batch; b += kLatThreads) {
    int err;
    keys_of[b] = seq_keys(p, b, &err, &keys_of[kMaxRowsPerLaunch + b]);
  }
  __syncthreads();
  if (warp == 0) {
    int total = 0, items = 0, most = 0;
#pragma unroll 1
    for (int b = lane; b < p.batch; b += 32) {
      const int nt = key_tiles(keys_of[b]);
      total += nt;
      items += nt > 0;
      most = max(most, nt);
    }
    total = __reduce_add_sync(0xffffffffu, total) * p.row_blocks.d;
    items = __reduce_add_sync(0xffffffffu, items) * p.row_blocks.d;
    most = __reduce_max_sync(0xffffffffu, most);
    const int each = div_by(total, p.workers);
    const int more = total - each * p.workers.d;
    const PartRule rule = part_rule(items, most, p.workers.d, each, more, [&](int len) {
      int n = 0;
#pragma unroll 1
      for (int b = lane; b < p.batch; b += 32) n += (key_tiles(keys_of[b]) + len - 1) / len;
      return static_cast<int>(__reduce_add_sync(0xffffffffu, n)) * p.row_blocks.d;
    });
    const bool parts = rule.parts;
    const int part_len = rule.len;
    const int reach = each >= 16 ? 1 : kCutReach;
    // what the scan counts: parts, or tiles
    const int x0 = parts ? worker : worker * each + min(worker, more);
    const int x1 = parts ? worker : x0 + each + (worker < more ? 1 : 0);
    if (lane == 0) {
      s_walk[0] = s_walk[1] = parts ? 0 : total;  // (past the last: no work)
      s_walk[6] = 0;
    }
    __syncwarp();
    int run = 0;
#pragma unroll 1
    for (int g = 0; g < p.batch && run <= x1; g += 32) {
      const int b = g + lane;
      const int n = b < p.batch ? keys_of[b] : 0;
      const int nt = key_tiles(n);
      const int unit = parts ? (nt + part_len - 1) / part_len : nt;
      const int span = unit * p.row_blocks.d;
      int incl = span;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
      }
      const int base = run + incl - span;
      run += __shfl_sync(0xffffffffu, incl, 31);
      bool first = x0 >= base && x0 < base + span;
      int walk_base = base;
      if (parts) {
        if (first) {
          const int in = x0 - base;
          const int rb = in / unit, k = in - rb * unit;
          const int len = nt / unit, longer = nt - len * unit;  // the first parts are one longer
          s_walk[0] = rb * nt + k * len + min(k, longer);
          s_walk[1] = rb * nt + (k + 1) * len + min(k + 1, longer);
          walk_base = 0;
          s_walk[6] = k > 0 && k + 1 == unit ? unit : 0;  // ends an item of that many parts
        }
      } else {
#pragma unroll 1
        for (int k = 1; k >= 0; --k) {
          const int x = k ? x1 : x0;
          if (x >= base && x < base + span) {
            const int i0 = base + (p.row_blocks.d == 1 ? 0 : (x - base) / nt * nt);
            const int i1 = i0 + nt;
            const int c = move_cut(x, i0, i1, reach);
            s_walk[k] = c;
            if (k == 0 && c > i0 && c < i1 && move_cut(x1, i0, i1, reach) >= i1) {
              // ends an item that it begins inside: as many workers before it as cuts in the item
              int u = worker;
              while (move_cut((u - 1) * each + min(u - 1, more), i0, i1, reach) > i0) --u;
              s_walk[6] = worker - u + 2;
            }
          }
        }
      }
      if (first) {
        // (a cut that moved to its item's end may lie past the sequence: the walk steps on)
        s_walk[2] = b;
        s_walk[3] = walk_base;
        s_walk[4] = n;
        s_walk[5] = keys_of[kMaxRowsPerLaunch + b];
      }
    }
    __syncwarp();
    asm volatile("barrier.cta.arrive 2, %0;" ::"n"(kLatThreads) : "memory");
  } else {
    named_bar_sync(2, kLatThreads);
  }
  Walk w;
  w.x = s_walk[0], w.end = s_walk[1], w.b = s_walk[2], w.base = s_walk[3], w.n = s_walk[4];
  w.slot = s_walk[5];
  bool more = walk_next(p, w);

  if (warp == 0 || warp == 6) {
    // ---------------------------------------------------- loads ----
    // Warp 0 brings Q and the keys for S, warp 6 the values for PV: each waits for its own
    // part of the shared memory only.
    const bool keys = warp == 0;
    const int R = p.box_rows;
    const int half_boxes = 64 / R;   // boxes of a chunk
    uint32_t tc = 0, items = 0;
    const uint32_t full0 = peer_u32(keys ? k_full : v_full, 0);
    const uint32_t q_full0 = peer_u32(q_full, 0);
    bool ok = true;
    // Boxes: the rows of a tile that lie in one page, at most 64; warp 0 loads those of this
    // CTA's half of the keys (`boxes` a tile), warp 6 those of the whole tile. Lane l holds the
    // pool row of box l % boxes of tile (window's first) + l / boxes.
    const int boxes = keys ? half_boxes : 2 * half_boxes;
    const int box_sh = __ffs(boxes) - 1;
    const int box0 = ((lane & (boxes - 1)) + (keys ? static_cast<int>(rank) * half_boxes : 0)) * R;
    const int window = 32 >> box_sh;
    // Where a page holds 64 rows one load brings all chunks of a group (loads of 8 KB one by
    // one come to 47 bytes a cycle, of 24 KB to 82 on all SMs at once); else a lane issues the
    // loads of one chunk of one box.
    const int per = R == 64 ? 1 : keys ? 3 : 2;
    for (; ok && more; more = walk_next(p, w)) {
      const int32_t* table = p.page_table + static_cast<long long>(w.slot) * p.max_blocks;
      if (keys) {
        if (lane == 0) {
          ok = items == 0 || wait_phase(q_empty, (items - 1) & 1, s_abort);
          if (ok) {
            if (rank == 0) mbar_arrive_expect_tx(q_full, 2 * kChunks * kChunk);
            tma_load_3d_pair(smem + kOffQ, &qmap, q_full0, 0,
                             w.b * p.rows + w.rb * kRows + static_cast<int>(rank) * 64, 0);
          }
        }
        ok = __shfl_sync(0xffffffffu, ok, 0);
        ++items;
      }
      int row = 0;
#pragma unroll 1
      for (int j = w.j0; ok && j < w.j1; ++j, ++tc) {
        const int in = (j - w.j0) & (window - 1);
        if (in == 0) {
          // a window's pages, all at once; page 0 as filler past the last key, and where an
          // entry names no page
          const int tile = j + (lane >> box_sh);
          const int t = tile * kKeys + box0;
          row = 0;
          if (tile < w.j1 && static_cast<uint32_t>(t) < static_cast<uint32_t>(w.n)) {
            const int block = div_by(t, p.page_size);
            const int page = __ldg(table + block);
            if (page < 0 || page >= p.num_pages) set_dev_err(p.dev_err, PKV_DEV_ERR_BAD_PAGE);
            else row = page * p.page_size.d + (t - block * p.page_size.d);
          }
        }
        if (keys) {
          const int src = __shfl_sync(0xffffffffu, row, (in << box_sh) + lane / per);
          uint8_t* dst = smem + kOffK + (lane % per) * kChunk + (lane / per) * R * 128;
#pragma unroll 1
          for (int g = 0; ok && g < kKGroups; ++g) {
            ok = tc == 0 || wait_phase(&k_empty[g], (tc - 1) & 1, s_abort);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            if (lane == 0 && rank == 0) mbar_arrive_expect_tx(&k_full[g], 2 * 3 * kChunk);
            __syncwarp();
            if (lane < per * boxes)
              tma_load_3d_pair(dst + 3 * g * kChunk, &kmap, full0 + 8 * g, 0, src,
                               3 * g + lane % per);
          }
          // The rows of a tile come from memory into L2 a tile before they are loaded: what shared
          // memory holds in flight (72 KB) does not cover the latency under load. (None / 1 / 2 / 3
          // tiles ahead, 16 and 128 heads: 64 x U[512, 1024] keys 24.3 / 23.3 / 24.6 / 25.3 and 27.0 /
          // 25.8 / 27.0 / 27.8 us, in pages of 16 rows 25.9 / 26.5 / 27.4 / 28.1 and 28.1 / 28.8 / 29.2 /
          // 29.7; 64 x U[2048, 8191] 82.0 / 75.6 / 78.9 / 81.6 and 97.3 / 92.7 / 97.3 / 99.7; one
          // sequence of 4000 15.9 / 15.8 / 15.7 / 15.8.)
          const int ahead = in + kAhead;
          const int at = lane >> box_sh;
          if (row > 0 && (at == ahead || (in == 0 && at > 0 && at < ahead)))
            asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(
                             p.pool + static_cast<long long>(row) * kRow),
                         "r"(R * kRow * 2)
                         : "memory");
        } else {
          const bool tail = ragged(w.n, j);
          const uint32_t tail_own = peer_u32(v_tail, rank);
          const int kh = lane / per >= half_boxes ? 1 : 0;  // which half of the tile's keys
          const int src = __shfl_sync(0xffffffffu, row, (in << box_sh) + lane / per);
          uint8_t* dst = smem + kOffV + (kh * 4 + lane % per) * kChunk +
                         (lane / per - kh * half_boxes) * R * 128;
#pragma unroll 1
          for (int g = 0; ok && g < kVGroups; ++g) {
            ok = tc == 0 || wait_phase(&v_empty[g], (tc - 1) & 1, s_abort);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            // the values of a ragged tile are announced to this CTA's softmax warps, which zero
            // the rows past its end, all others to the pair's MMA warp
            if (lane == 0) {
              if (tail) {
                if (g == 0) mbar_arrive_expect_tx(v_tail, 8 * kChunk);
              } else if (rank == 0) {
                mbar_arrive_expect_tx(&v_full[g], 2 * 4 * kChunk);
              }
            }
            __syncwarp();
            if (lane < per * boxes)
              tma_load_3d_pair(dst + 2 * g * kChunk, &vmap, tail ? tail_own : full0 + 8 * g, 0, src,
                               static_cast<int>(rank) * 4 + 2 * g + lane % per);
          }
        }
      }
    }
    if (!ok && lane == 0) *s_abort = 1;
  } else if (warp == 1 || warp == 7) {
    // ----------------------------------------------------- MMAs ----
    // Two streams of products share the tensor pipe, each with its own issuing thread of CTA 0
    // (both in one thread, that polled for whichever was ready, took 200 cycles a round beside the
    // softmax warps, whose code passes through the same instruction cache): S of the tiles waits for
    // rows from memory, PV for a softmax, and neither holds up the other. (64 x ~768
    // keys, 128 heads: 26.5 -> 24.6 us; 16 x ~20000, 128 rows: 77.7 -> 74.6 us.)
    if (rank == 1) {
      // The other CTA's threads issue for both. Here warp 1 notes for the join whether the worker's
      // range ends an item of several parts, and writes the rows of sequences without keys.
      if (warp == 1) {
        if (lane == 0) p.part_item[worker] = make_int4(s_walk[6], w.b, w.rb, 0);
#pragma unroll 1
        for (int b = worker; b < p.batch; b += p.workers.d) {
          int err, slot;
          if (seq_keys(p, b, &err, &slot) > 0) continue;
          if (err && lane == 0) set_dev_err(p.dev_err, err);
          const long long at = static_cast<long long>(b) * p.rows;
          uint4* o = reinterpret_cast<uint4*>(p.out + at * kLatent);
          for (long long e = lane; e < static_cast<long long>(p.rows) * (kLatent / 8); e += 32)
            o[e] = make_uint4(0u, 0u, 0u, 0u);
          for (int e = lane; e < p.rows; e += 32) p.lse[at + e] = -INFINITY;
        }
      }
    } else if (elect_one()) {
      bool ok = true;
      uint32_t tc = 0, items = 0;  // tiles, items issued
      if (warp == 1) {
        const uint32_t q_lo = desc_lo(smem_u32(smem + kOffQ), 0);
        const uint32_t k_lo = desc_lo(smem_u32(smem + kOffK), 0);
        for (; ok && more; more = walk_next(p, w)) {
          ok = wait_phase(q_full, items & 1, s_abort);
          ++items;
#pragma unroll 1
          for (int j = w.j0; ok && j < w.j1; ++j, ++tc) {
            // S goes into buffer tc & 1, which P of tile tc - 2 has been read from. (A barrier for
            // each buffer: this thread may come late, for it waits for Q too, and a barrier that two
            // tiles have completed in the meantime looks as if none had.)
            ok = tc < 2 || wait_phase_cluster(&p_full[tc & 1], ((tc >> 1) - 1) & 1, s_abort);
#pragma unroll 1
            for (int g = 0; ok && g < kKGroups; ++g) {
              ok = wait_phase(&k_full[g], tc & 1, s_abort);
              if (!ok) break;
              tc_fence_after();
#pragma unroll
              for (int c = 0; c < 3; ++c)
                umma4_pair<32, 32>(tmem + kColS + 64 * (tc & 1),
                                   q_lo + (((3 * g + c) * kChunk) >> 4),
                                   k_lo + (((3 * g + c) * kChunk) >> 4), kIdescS, g + c > 0 ? 1u : 0u);
              commit_pair(&k_empty[g]);
            }
            if (ok) commit_pair(&s_full[tc & 1]);
          }
          if (ok) commit_pair(q_empty);
        }
      } else {
        const uint32_t p_lo = desc_lo(smem_u32(smem + kOffP), 0);
        const uint32_t v_lo = desc_lo(smem_u32(smem + kOffV), kChunk);
        uint32_t fv = 0;  // tiles whose values v_full announced
        for (; ok && more; more = walk_next(p, w)) {
#pragma unroll 1
          for (int j = w.j0; ok && j < w.j1; ++j, ++tc) {
            // (before an item's first PV both epilogues have read the last item's O)
            ok = wait_phase_cluster(&p_full[tc & 1], (tc >> 1) & 1, s_abort) &&
                 (j > w.j0 || items == 0 || wait_phase_cluster(o_free, (items - 1) & 1, s_abort));
            const bool tail = ragged(w.n, j);
            const int left = w.n - j * kKeys;
            const int steps = left >= kKeys ? 8 : (left + 15) >> 4;  // of 16 keys
            const uint32_t acc = j > w.j0 ? 1u : 0u;
#pragma unroll 1
            for (int g = 0; ok && g < kVGroups; ++g) {
              ok = tail || wait_phase(&v_full[g], fv & 1, s_abort);
              if (!ok) break;
              tc_fence_after();
              const uint32_t b = v_lo + ((2 * g * kChunk) >> 4);
              const uint32_t d = tmem + 128 * g;
              if (steps == 8) {
                umma4_pair<32, 2048>(d, p_lo, b, kIdescO, acc);
                umma4_pair<32, 2048>(d, p_lo + (kChunk >> 4), b + ((4 * kChunk) >> 4), kIdescO, 1u);
              } else {
#pragma unroll 1
                for (int k = 0; k < steps; ++k) {
                  const int kh = k >> 2, ks = k & 3;
                  umma1_pair(d, p_lo + ((kh * kChunk) >> 4) + 2 * ks,
                             b + ((kh * 4 * kChunk) >> 4) + 128 * ks, kIdescO, acc | (k > 0 ? 1u : 0u));
                }
              }
              commit_pair(&v_empty[g]);
            }
            if (ok) commit_pair(pv_done);
            if (!tail) ++fv;
          }
          ++items;
        }
      }
      if (!ok) *s_abort = 1;
    }
  } else {
    // ---------------------------------------- softmax and epilogue ----
    const int tl = 32 * (warp & 3) + lane;   // TMEM lane
    const int hk = tl >> 6;                  // keys 64 hk .. of a tile, dims 256 hk .. of a row
    const int r = tl & 63;                   // row of this CTA
    const uint32_t t_lane = tmem + (static_cast<uint32_t>(tl & 96) << 16);
    const uint32_t p_full0 = peer_u32(p_full, 0);
    const uint32_t o_free0 = peer_u32(o_free, 0);
    uint8_t* prow = smem + kOffP + hk * kChunk + r * 128;
    uint32_t tc = 0, tails = 0;
    bool ok = true;
    for (; ok && more; more = walk_next(p, w)) {
      const int row = w.rb * kRows + static_cast<int>(rank) * 64 + r;  // row of the sequence
      const bool live = row < p.rows;
      const bool warp_live = __any_sync(0xffffffffu, live);
      // keys that the row sees: all but those of the drafts behind its token
      const int lim = live ? w.n - (p.n_q - 1 - div_by(row, p.heads)) : 0;
      float m_run = -INFINITY;  // running maximum of the row, raw score units
      float l_run = 0.f;        // sum over this thread's half of the keys
      bool left_together = false;
      for (int j = w.j0; j < w.j1; ++j, ++tc) {
        // a wait that gave up is told to the other warps at their next common barrier, so
        // that all four leave at the same place
        ok = ok && wait_phase(&s_full[tc & 1], (tc >> 1) & 1, s_abort);
        ok = __all_sync(0xffffffffu, ok);
        tc_fence_after();
        uint32_t s[64];
        float mx = -INFINITY;
        const int c_hi = lim - j * kKeys - hk * 64;  // visible columns of this thread's 64
        if (warp_live && ok) {
          tmem_ld32(t_lane + kColS + 64 * (tc & 1), *reinterpret_cast<uint32_t(*)[32]>(&s[0]));
          tmem_ld32(t_lane + kColS + 64 * (tc & 1) + 32,
                    *reinterpret_cast<uint32_t(*)[32]>(&s[32]));
          tmem_wait_ld();
          if (c_hi < 64) {
#pragma unroll
            for (int c = 0; c < 64; ++c)
              if (c >= c_hi) s[c] = __float_as_uint(-INFINITY);
          }
          float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int c = 0; c < 64; c += 8) {
#pragma unroll
            for (int k = 0; k < 4; ++k)
              m4[k] = fmax3(m4[k], __uint_as_float(s[c + 2 * k]), __uint_as_float(s[c + 2 * k + 1]));
          }
          mx = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3]));
        }
        // the row's two threads agree on its maximum
        float* const maxima = s_max + 128 * (tc & 1);
        maxima[tl] = mx;
        ok = named_bar_all(1, 128, ok);
        if (!ok) {
          left_together = true;
          break;
        }
        const float m_cand = fmaxf(m_run, fmaxf(mx, maxima[tl ^ 64]));
        // The maximum that the weights refer to moves only when it has grown by more than
        // 2^8: until then weights of up to 256 do no harm in bf16 and fp32, and O stays.
        const bool grow = m_run == -INFINITY ? m_cand != -INFINITY
                                             : (m_cand - m_run) * p.qscale > kRescaleThreshold;
        const float m_use = grow ? m_cand : m_run;
        const float alpha = grow ? ex2((m_run - m_use) * p.qscale) : 1.f;
        const float neg_m = m_use == -INFINITY ? 0.f : -m_use * p.qscale;
        uint32_t pk[32];
        float psum = 0.f;
        if (warp_live) {
          const unsigned long long qs2 = pack_f32x2(p.qscale, p.qscale);
          const unsigned long long nm2 = pack_f32x2(neg_m, neg_m);
          unsigned long long acc0 = 0ull, acc1 = 0ull;
#pragma unroll
          for (int c = 0; c < 64; c += 4) {
            float e[4];
#pragma unroll
            for (int u = 0; u < 2; ++u) {
              const unsigned long long x2 =
                  ffma2(pack_f32x2(__uint_as_float(s[c + 2 * u]), __uint_as_float(s[c + 2 * u + 1])),
                        qs2, nm2);
              float x0, x1;
              unpack_f32x2(x2, x0, x1);
              e[2 * u] = ex2(x0);
              e[2 * u + 1] = ex2(x1);
            }
            acc0 = fadd2(acc0, pack_f32x2(e[0], e[1]));
            acc1 = fadd2(acc1, pack_f32x2(e[2], e[3]));
            // weights in bf16 for the product (each off by at most 2^-8 of itself);
            // their sum takes them unrounded
            pk[c / 2] = pack_bf16x2(e[0], e[1]);
            pk[c / 2 + 1] = pack_bf16x2(e[2], e[3]);
          }
          float a, b, c, d;
          unpack_f32x2(acc0, a, b);
          unpack_f32x2(acc1, c, d);
          psum = (a + b) + (c + d);
        }
        l_run = l_run * alpha + psum;
        m_run = m_use;
        // P and O are free once the last PV is done
        ok = tc == 0 || wait_phase(pv_done, (tc - 1) & 1, s_abort);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) continue;
        tc_fence_after();
        if (warp_live) {
#pragma unroll
          for (int q = 0; q < 8; ++q)
            *reinterpret_cast<uint4*>(prow + ((q ^ (r & 7)) << 4)) =
                make_uint4(pk[4 * q], pk[4 * q + 1], pk[4 * q + 2], pk[4 * q + 3]);
          if (j > w.j0 && __any_sync(0xffffffffu, grow)) {
#pragma unroll 1
            for (int q = 0; q < 256; q += 32) {
              uint32_t o[32];
              tmem_ld32(t_lane + q, o);
              tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
              tmem_st32(t_lane + q, o);
            }
            tmem_wait_st();
          }
        }
        // values of rows past the last key may hold any bits: their weights are 0, but
        // 0 * NaN is not, so the rows that share a 16-key step with live ones are zeroed
        if (ragged(w.n, j)) {
          ok = __all_sync(0xffffffffu, wait_phase(v_tail, tails & 1, s_abort));
          ++tails;
          if (!ok) continue;
          const int left = w.n - j * kKeys;
          for (int q = tl; q < (16 - (left & 15)) * 32; q += 128) {
            const int key = left + (q >> 5);
            uint8_t* at = smem + kOffV + ((key >> 6) * 4 + ((q >> 3) & 3)) * kChunk +
                          (key & 63) * 128 + (q & 7) * 16;
            *reinterpret_cast<uint4*>(at) = make_uint4(0u, 0u, 0u, 0u);
          }
        }
        fence_proxy_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(p_full0 + 8 * (tc & 1));
      }
      // ---- the segment's end: O and the row's maximum and sum ----
      if (left_together) break;
      ok = ok && wait_phase(pv_done, (tc - 1) & 1, s_abort);
      float* const sums = s_max + 256;
      sums[tl] = l_run;
      ok = named_bar_all(1, 128, ok);
      tc_fence_after();
      if (ok) {
        const float l = l_run + sums[tl ^ 64];
        const bool whole = w.j0 == 0 && w.j1 == w.nt;
        const int first = w.rb * kRows + static_cast<int>(rank) * 64;  // row of this CTA's row 0
        const int live_rows = min(64, p.rows - first);
        if (live_rows > 0) {
          const bool has = live && l != 0.f;  // (a NaN among its scores: NaN)
          const float inv = has ? 1.f / l : 0.f;
          const long long at = static_cast<long long>(w.b) * p.rows + first;
          const int part = 2 * worker + (w.j0 == 0 ? 1 : 0);
          const long long pat = static_cast<long long>(part) * p.block_rows + (first - w.rb * kRows);
          if (live && hk == 0) {
            if (whole) {
              p.lse[at + r] =
                  has ? (m_run * p.qscale + __log2f(l)) * 0.69314718055994531f : -INFINITY;
            } else {
              // (-inf says that the row sees no key of the part)
              p.part_ml[2 * (pat + r)] =
                  m_run == -INFINITY && lim > w.j0 * kKeys ? -FLT_MAX : m_run;
              p.part_ml[2 * (pat + r) + 1] = l;
            }
          }
          // Through shared memory, 128 bytes of each half row a round (64 values of the result, 32
          // of a partial), so that stores fill whole lines. Each half's two warps stage and store
          // for themselves: a round at a time in P's place, or, where the worker is done, all
          // rounds in Q's and the keys'.
          const bool last = w.x >= w.end;
          uint8_t* stage = smem + (last ? kOffQ : kOffP) + hk * kChunk;
          const int rounds = whole ? 4 : 8;
          const long long row_bytes = kLatent * (whole ? 2 : 4);
          uint8_t* dst = (whole ? reinterpret_cast<uint8_t*>(p.out) + at * row_bytes
                                : reinterpret_cast<uint8_t*>(p.part_o) + pat * row_bytes) +
                         hk * (row_bytes / 2);
          const int per = last ? rounds : 1;  // rounds staged side by side
#pragma unroll 1
          for (int rd = 0; rd < rounds; ++rd) {
            uint8_t* st = stage + (last ? rd * 2 * kChunk : 0);
            if (warp_live) {
              uint32_t v[32];
              if (whole) {
                uint32_t a[64];
                tmem_ld32(t_lane + 64 * rd, *reinterpret_cast<uint32_t(*)[32]>(&a[0]));
                tmem_ld32(t_lane + 64 * rd + 32, *reinterpret_cast<uint32_t(*)[32]>(&a[32]));
                tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < 32; ++e)
                  v[e] = has ? pack_bf16x2(__uint_as_float(a[2 * e]) * inv,
                                           __uint_as_float(a[2 * e + 1]) * inv)
                             : 0u;
              } else {
                tmem_ld32(t_lane + 32 * rd, v);
                tmem_wait_ld();
              }
#pragma unroll
              for (int c = 0; c < 8; ++c)
                *reinterpret_cast<uint4*>(st + r * 128 + ((c ^ (r & 7)) << 4)) =
                    make_uint4(v[4 * c], v[4 * c + 1], v[4 * c + 2], v[4 * c + 3]);
            }
            if (rd + 1 < rounds && last) continue;
            named_bar_sync(3 + hk, 64);
            // 16-byte pieces: eight neighbouring lanes store the 128 bytes of a row and round
            const int c = r & 7;
            uint8_t* const to = dst + (rd + 1 - per) * 128 + c * 16;
#pragma unroll 1
            for (int i0 = r >> 3; i0 < live_rows; i0 += 16) {
#pragma unroll 1
              for (int k = 0; k < per; k += 4) {
                uint4 x[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                  const int sr = i0 + 8 * (i >> 2), kk = k + (i & 3);
                  if (kk < per)
                    x[i] = *reinterpret_cast<const uint4*>(stage + kk * 2 * kChunk + sr * 128 +
                                                           ((c ^ (sr & 7)) << 4));
                }
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                  const int sr = i0 + 8 * (i >> 2), kk = k + (i & 3);
                  if (kk < per && sr < live_rows)
                    *reinterpret_cast<uint4*>(to + sr * row_bytes + kk * 128) = x[i];
                }
              }
            }
            if (!last) named_bar_sync(3 + hk, 64);  // the place may be written again
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(o_free0);
      }
    }
    if (!ok) *s_abort = 1;
  }
  __syncwarp();
  if (*s_abort && threadIdx.x == 0) {
    set_dev_err(p.dev_err, PKV_DEV_ERR_TIMEOUT);
    // copies that are still in flight land before the CTA's shared memory goes back
    const uint64_t t0 = global_timer_ns();
    while (global_timer_ns() - t0 < 100000) {}
  }
  tc_fence_before();
  __syncthreads();
  // (neither CTA leaves while the other's MMAs may read its shared memory; no data is handed over,
  // so nothing waits for the results' stores)
  asm volatile(
      "barrier.cluster.arrive.relaxed.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
  if (warp == 1) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem),
                 "r"(kTmemCols)
                 : "memory");
  }
}

// Joins the partials of split items: those of the worker whose range ends the item and of the
// parts - 1 workers before it, the first of which left the partial of its last segment, the others
// that of their first. Weights are 2^(m_i - max m), their sum that of the l_i. The warps of the
// grid share the rows of all these items, where they are many enough a whole row each, else a
// quarter.
constexpr int kJoinWarps = 4;

template <int kSplit>
__device__ __forceinline__ void join_row(const LatentDecodeParams& p, const int4& item, int worker,
                                         int row_in, int split, int lane) {
  const int row = item.z * kRows + row_in;
  if (row >= p.rows) return;
  constexpr int kVecs = 4 / kSplit;  // 16-byte pieces of a lane
  const int piece = split * (128 / kSplit) + lane;
  float m = -INFINITY, l = 0.f;
  float4 o[kVecs];
#pragma unroll
  for (int e = 0; e < kVecs; ++e) o[e] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
  for (int done = 0; done < item.x; done += 32) {
    // 32 parts at a time, from the last down: lane i looks at that of worker u
    const int n = min(32, item.x - done);
    const int u = worker - done - lane;
    const int part = 2 * u + (done + lane == item.x - 1 ? 1 : 0);
    const long long pr = static_cast<long long>(part) * p.block_rows + row_in;
    const float mi = lane < n ? __ldcg(p.part_ml + 2 * pr) : -INFINITY;
    const float li = lane < n ? __ldcg(p.part_ml + 2 * pr + 1) : 0.f;
    float mx = mi;
#pragma unroll
    for (int s = 16; s > 0; s >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, s));
    const float mn = fmaxf(m, mx);
    // (-1: a range none of whose keys the row sees, which adds nothing, whatever the keys hold)
    const float take = mi == -INFINITY ? -1.f : ex2((mi - mn) * p.qscale);
    const float keep = m == -INFINITY ? 0.f : ex2((m - mn) * p.qscale);
    float ls = mi == -INFINITY ? 0.f : take * li;
#pragma unroll
    for (int s = 16; s > 0; s >>= 1) ls += __shfl_xor_sync(0xffffffffu, ls, s);
    l = l * keep + ls;
#pragma unroll
    for (int e = 0; e < kVecs; ++e) o[e].x *= keep, o[e].y *= keep, o[e].z *= keep, o[e].w *= keep;
#pragma unroll 4
    for (int i = 0; i < n; ++i) {
      const int pi = __shfl_sync(0xffffffffu, part, i);
      const float t = __shfl_sync(0xffffffffu, take, i);
      const float4* src = reinterpret_cast<const float4*>(
          p.part_o + (static_cast<long long>(pi) * p.block_rows + row_in) * kLatent);
      float4 v[kVecs];
#pragma unroll
      for (int e = 0; e < kVecs; ++e) v[e] = __ldcg(src + piece + 32 * e);
      if (t >= 0.f) {
#pragma unroll
        for (int e = 0; e < kVecs; ++e) {
          o[e].x = fmaf(v[e].x, t, o[e].x);
          o[e].y = fmaf(v[e].y, t, o[e].y);
          o[e].z = fmaf(v[e].z, t, o[e].z);
          o[e].w = fmaf(v[e].w, t, o[e].w);
        }
      }
    }
    m = mn;
  }
  const bool has = l != 0.f;
  const float inv = has ? 1.f / l : 0.f;
  const long long at = static_cast<long long>(item.y) * p.rows + row;
#pragma unroll
  for (int e = 0; e < kVecs; ++e)
    reinterpret_cast<uint2*>(p.out + at * kLatent)[piece + 32 * e] =
        has ? make_uint2(pack_bf16x2(o[e].x * inv, o[e].y * inv),
                         pack_bf16x2(o[e].z * inv, o[e].w * inv))
            : make_uint2(0u, 0u);
  if (lane == 0 && split == 0)
    p.lse[at] = has ? (m * p.qscale + __log2f(l)) * 0.69314718055994531f : -INFINITY;
}

__global__ void __launch_bounds__(kJoinWarps * 32) latent_join_kernel(const LatentDecodeParams p) {
  constexpr int kMaxWorkers = 128;
  __shared__ int4 s_item[kMaxWorkers];
  __shared__ int s_worker[kMaxWorkers];
  __shared__ int s_count;
  const int lane = threadIdx.x & 31;
  pdl_wait_primary();
  pdl_launch_dependents();
  // the items of several parts, in order of the workers that end them
  if (threadIdx.x < 32) {
    int count = 0;
    int4 item[kMaxWorkers / 32];
#pragma unroll
    for (int k = 0; k < kMaxWorkers / 32; ++k) {
      const int w = k * 32 + lane;
      item[k] = w < p.workers.d ? __ldcg(p.part_item + w) : make_int4(0, 0, 0, 0);
    }
#pragma unroll
    for (int k = 0; k < kMaxWorkers / 32; ++k) {
      const uint32_t has = __ballot_sync(0xffffffffu, item[k].x > 0);
      if (item[k].x > 0) {
        const int at = count + __popc(has & ((1u << lane) - 1u));
        s_item[at] = item[k];
        s_worker[at] = k * 32 + lane;
      }
      count += __popc(has);
    }
    if (lane == 0) s_count = count;
  }
  __syncthreads();
  const int count = s_count;
  const int warps = gridDim.x * kJoinWarps;
  const int id = blockIdx.x * kJoinWarps + (threadIdx.x >> 5);
  const int rows = count * p.block_rows;
  if (rows * 4 <= warps) {
    if (id < rows * 4) {
      const int i = (id >> 2) / p.block_rows;
      join_row<4>(p, s_item[i], s_worker[i], (id >> 2) - i * p.block_rows, id & 3, lane);
    }
  } else {
#pragma unroll 1
    for (int u = id; u < rows; u += warps) {
      const int i = u / p.block_rows;
      join_row<1>(p, s_item[i], s_worker[i], u - i * p.block_rows, 0, lane);
    }
  }
}

namespace {

// {64 values, rows, 9 chunks} view of an array of rows of 576; a box is `box_rows` rows of
// `box_chunks` chunks, 128-byte swizzled.
bool encode_rows_map(CUtensorMap* map, const void* base, long long rows, int box_rows,
                     int box_chunks) {
  prefill_host::EncodeTiledFn enc = prefill_host::encode_fn();
  const cuuint64_t dims[3] = {64u, static_cast<cuuint64_t>(rows), kChunks};
  const cuuint64_t strides[2] = {kRow * 2, 128u};
  const cuuint32_t box[3] = {64u, static_cast<cuuint32_t>(box_rows),
                             static_cast<cuuint32_t>(box_chunks)};
  const cuuint32_t estr[3] = {1u, 1u, 1u};
  return enc != nullptr &&
         enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box,
             estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

constexpr int kMaxQueries = 64;
constexpr int kMaxHeads = 1024;

bool latent_rows_ok(int batch, int n_q, int heads) {
  return batch >= 0 && n_q >= 1 && n_q <= kMaxQueries && heads >= 1 && heads <= kMaxHeads &&
         static_cast<long long>(batch) * n_q * heads <= INT_MAX;
}
// The most tiles that one sequence can have.
long long seq_tiles(const pkv_cache_desc* c, int rows) {
  return (static_cast<long long>(c->max_blocks) * c->page_size + kKeys - 1) / kKeys *
         ((rows + kRows - 1) / kRows);
}
// Rows of one launch: equal launches of at most 512 rows and 2^30 tiles. 0: one row has more.
int launch_batch(const pkv_cache_desc* c, int batch, int rows) {
  const long long most = std::min<long long>(kMaxRowsPerLaunch, (1ll << 30) / seq_tiles(c, rows));
  if (most == 0) return 0;
  const long long launches = (batch + most - 1) / most;
  return static_cast<int>(launches > 0 ? (batch + launches - 1) / launches : 1);
}
// Pairs of CTAs of a launch, and the bytes of its partials.
int launch_workers(const pkv_cache_desc* c, int batch, int rows, int sm_count) {
  return static_cast<int>(std::min<long long>(seq_tiles(c, rows) * batch, std::min(sm_count / 2, 128)));
}
size_t partial_bytes(int workers, int rows) {
  const size_t block_rows = rows < kRows ? rows : kRows;
  return static_cast<size_t>(workers) *
         (2 * block_rows * (kLatent + 2) * sizeof(float) + sizeof(int4));
}

}  // namespace
}  // namespace pkv

using namespace pkv;
using namespace pkv::latent;

extern "C" size_t pkv_latent_decode_workspace_size(const pkv_cache_desc* cache, int batch, int n_q,
                                                   int num_heads) {
  if (check_latent_cache(cache) != PKV_OK || !latent_rows_ok(batch, n_q, num_heads)) return 0;
  int sms = 0;
  if (device_info(&sms) != PKV_OK) return 0;
  const int rows = n_q * num_heads;
  const int per = launch_batch(cache, batch, rows);
  if (per == 0) return 0;
  const size_t n = partial_bytes(launch_workers(cache, per, rows, sms), rows);
  return n < 256 ? 256 : n;
}

extern "C" pkv_status pkv_latent_decode_attention(const pkv_cache_desc* cache, const void* pool,
                                                  const int32_t* page_table, const void* q,
                                                  int num_heads, const int32_t* batch_idx,
                                                  const int32_t* seq_lens, int batch, int n_q,
                                                  float scale, void* out, float* lse,
                                                  void* workspace, size_t workspace_bytes,
                                                  int32_t* dev_err, cudaStream_t stream) {
  if (const pkv_status st = check_latent_cache(cache); st != PKV_OK) return st;
  if (!latent_rows_ok(batch, n_q, num_heads) || !std::isfinite(scale) || !(scale > 0.f))
    return PKV_ERR_ARG;
  if (batch == 0) return PKV_OK;
  if (!pool || !page_table || !q || !batch_idx || !seq_lens || !out || !lse) return PKV_ERR_ARG;
  if (!is_aligned(pool, 16) || !is_aligned(q, 16) || !is_aligned(out, 16) || !is_aligned(lse, 4) ||
      !is_aligned(page_table, 4) || !is_aligned(batch_idx, 4) || !is_aligned(seq_lens, 4) ||
      !is_aligned(dev_err, 4) || !is_aligned(workspace, 256))
    return PKV_ERR_ALIGN;
  int sms = 0;
  if (const pkv_status st = device_info(&sms); st != PKV_OK) return st;
  const int rows = n_q * num_heads;
  const int per = launch_batch(cache, batch, rows);
  if (per == 0) return PKV_ERR_ARG;
  const int workers = launch_workers(cache, per, rows, sms);
  if (!workspace || workspace_bytes < partial_bytes(workers, rows)) return PKV_ERR_WORKSPACE;
  int box = 64;
  while (cache->page_size % box) box >>= 1;  // 16, 32 or 64
  const long long pool_rows = static_cast<long long>(cache->num_pages) * cache->page_size;
  CUtensorMap kmap, vmap;
  if (!encode_rows_map(&kmap, pool, pool_rows, box, box == 64 ? 3 : 1) ||
      !encode_rows_map(&vmap, pool, pool_rows, box, box == 64 ? 2 : 1))
    return PKV_ERR_ARG;
  int dev = 0;
  if (const cudaError_t e = cudaGetDevice(&dev); e != cudaSuccess) return record_cuda_status(e);
  static std::atomic<bool> attr_set[64] = {};  // per device; host threads may race to set it
  if (dev < 0 || dev >= 64) return PKV_ERR_DEVICE;
  if (!attr_set[dev].load(std::memory_order_acquire)) {
    const cudaError_t e = cudaFuncSetAttribute(
        latent_decode_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kLatSmem);
    if (e != cudaSuccess) return record_cuda_status(e);
    attr_set[dev].store(true, std::memory_order_release);
  }
  LatentDecodeParams p;
  p.pool = static_cast<const __nv_bfloat16*>(pool);
  p.page_table = page_table;
  p.dev_err = dev_err;
  p.heads = make_divisor(num_heads);
  p.n_q = n_q;
  p.rows = rows;
  p.row_blocks = make_divisor((rows + kRows - 1) / kRows);
  p.block_rows = rows < kRows ? rows : kRows;
  p.page_size = make_divisor(cache->page_size);
  p.num_pages = cache->num_pages;
  p.max_batch = cache->max_batch;
  p.max_blocks = cache->max_blocks;
  p.box_rows = box;
  p.qscale = scale * 1.4426950408889634f;
  for (int b0 = 0; b0 < batch; b0 += per) {
    const int n = batch - b0 < per ? batch - b0 : per;
    const long long first = static_cast<long long>(b0) * rows;
    const __nv_bfloat16* q0 = static_cast<const __nv_bfloat16*>(q) + first * kRow;
    p.batch_idx = batch_idx + b0;
    p.seq_lens = seq_lens + b0;
    p.out = static_cast<__nv_bfloat16*>(out) + first * kLatent;
    p.lse = lse + first;
    p.batch = n;
    const int w = launch_workers(cache, n, rows, sms);
    p.workers = make_divisor(w);
    p.part_o = static_cast<float*>(workspace);
    p.part_item = reinterpret_cast<int4*>(p.part_o + static_cast<size_t>(2 * w) * p.block_rows * kLatent);
    p.part_ml = reinterpret_cast<float*>(p.part_item + w);
    CUtensorMap qmap;
    if (!encode_rows_map(&qmap, q0, static_cast<long long>(n) * rows, 64, kChunks))
      return PKV_ERR_ARG;
    cudaError_t e = launch_kernel(latent_decode_kernel, dim3(2 * w), dim3(kLatThreads), kLatSmem,
                                  stream, true, qmap, kmap, vmap, p);
    if (e != cudaSuccess) return record_cuda_status(e);
    if (w == 1) continue;  // nothing can be split
    e = launch_kernel(latent_join_kernel, dim3(4 * sms), dim3(kJoinWarps * 32), 0, stream, true, p);
    if (e != cudaSuccess) return record_cuda_status(e);
  }
  return PKV_OK;
}
