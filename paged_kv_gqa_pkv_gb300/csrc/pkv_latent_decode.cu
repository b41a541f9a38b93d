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
// Roles per CTA: warp 0 loads (TMA through the page table); warp 1 issues the MMAs (of the
// pair: CTA 0's only); warps 2-5 are softmax and epilogue, lane l and l + 64 sharing row l.
//
// Work: the tiles of all (sequence, 128-row block) items in a row are cut into equal
// ranges, one per pair of CTAs; an item that a cut splits leaves unnormalised partials,
// which a second kernel joins. Cuts close to an item's end move there.
#include <atomic>
#include <cmath>

#include "pkv_latent.cuh"

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
constexpr int kLatThreads = 6 * 32;
constexpr int kMaxRowsPerLaunch = 512;     // sequences of one launch

// shared memory, offsets from a 1024-aligned base
constexpr int kOffQ = 0;                              // [9 chunks][64 query rows]
constexpr int kOffK = kOffQ + kChunks * kChunk;       // [9 chunks][64 own keys]
constexpr int kOffV = kOffK + kChunks * kChunk;       // [2 key halves][4 own chunks][64 keys]
constexpr int kOffP = kOffV + 8 * kChunk;             // [2 key halves][64 query rows]
constexpr int kOffBar = kOffP + 2 * kChunk;
constexpr int kNumBars = 2 * kKGroups + 2 * kVGroups + 7;
constexpr int kOffMisc = kOffBar + kNumBars * 8;      // tmem slot, abort flag, range
constexpr int kOffMax = kOffMisc + 32;                // [2][128] row maxima, [128] sums
constexpr int kLatSmem = kOffMax + 3 * 128 * 4 + 1024;  // + slack for the alignment
static_assert(kLatSmem <= kMaxDynSmem, "shared memory above the opt-in limit");

constexpr uint32_t kColS = 256;            // TMEM: O in columns 0-255, S in 256 + 64 * buffer
constexpr uint32_t kIdescS = idesc_bf16_f32(kRows, kKeys, false);
constexpr uint32_t kIdescO = idesc_bf16_f32(kRows, 256, true);

struct LatentDecodeParams {
  const int32_t* page_table;
  const int32_t* batch_idx;
  const int32_t* seq_lens;
  __nv_bfloat16* out;      // [batch, n_q * heads, 512]
  float* lse;              // [batch, n_q * heads]
  float* part_o;           // [2 * workers][block_rows][512]
  float* part_ml;          // [2 * workers][block_rows][2]
  int32_t* dev_err;
  int batch;
  int heads;
  int n_q;
  int rows;                // n_q * heads
  int row_blocks;          // ceil(rows / 128)
  int block_rows;          // min(rows, 128): rows of a partial
  int page_size;
  int num_pages;
  int max_batch;
  int max_blocks;
  int box_rows;            // rows of one TMA box: 16, 32 or 64
  int workers;             // pairs of CTAs
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
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t bar) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar)
               : "memory");
}
// Waits that see what threads of the other CTA released.
__device__ __forceinline__ bool mbar_try_wait_cluster(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}
__device__ __forceinline__ bool wait_pair(uint64_t* bar, uint32_t parity,
                                          volatile int* abort_flag) {
  if (mbar_try_wait_cluster(bar, parity)) return true;
  const uint64_t t0 = global_timer_ns();
  for (uint32_t i = 1;; ++i) {
    if (mbar_try_wait_cluster(bar, parity)) return true;
    if ((i & 63u) == 0) {
      if (*abort_flag) return false;
      if (global_timer_ns() - t0 > kWaitLimitNs) {
        *abort_flag = 1;
        return false;
      }
    }
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

// 32 bytes to global memory in one instruction: a whole sector per lane.
__device__ __forceinline__ void st_global_v8(void* a, const uint32_t (&w)[8]) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(a), "r"(w[0]),
               "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}

// ------------------------------------------------------------------- work --

// Keys of a sequence's last query; 0 for padding and for rows that are refused (*err).
__device__ __forceinline__ int seq_keys(const LatentDecodeParams& p, int b, int* err) {
  const int slot = __ldg(p.batch_idx + b);
  const int n = __ldg(p.seq_lens + b);
  *err = 0;
  if (slot == 0) return 0;
  if (slot < 0 || slot >= p.max_batch) *err = PKV_DEV_ERR_BAD_SLOT;
  else if (n < 0 || n > p.max_blocks * p.page_size) *err = PKV_DEV_ERR_BAD_POS;
  return *err ? 0 : n;
}
__device__ __forceinline__ int key_tiles(int n) {
  return n / kKeys + (n % kKeys != 0);
}

// The tiles of all items in a row: sequence by sequence, its row blocks one after another.
// A warp's view: lane l holds the tiles of sequences l * per .. l * per + per - 1.
struct Flat {
  long long total;
  long long before;  // tiles before this lane's sequences
  long long own;     // tiles of this lane's sequences
  int per;
};
__device__ __forceinline__ Flat flat_load(const LatentDecodeParams& p, int lane) {
  Flat f;
  f.per = (p.batch + 31) / 32;
  f.own = 0;
  for (int k = 0; k < f.per; ++k) {
    const int b = lane * f.per + k;
    int err;
    if (b < p.batch) f.own += static_cast<long long>(key_tiles(seq_keys(p, b, &err))) * p.row_blocks;
  }
  long long incl = f.own;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += y;
  }
  f.before = incl - f.own;
  f.total = __shfl_sync(0xffffffffu, incl, 31);
  return f;
}
// The sequence that holds flat tile x (0 <= x < total) and the tiles before it.
__device__ __forceinline__ void flat_find(const LatentDecodeParams& p, const Flat& f, int lane,
                                          long long x, int* seq, long long* base) {
  const bool mine = x >= f.before && x < f.before + f.own;
  int b = 0;
  long long at = f.before;
  if (mine) {
    for (int k = 0; k < f.per; ++k) {
      int err;
      const int s = lane * f.per + k;
      const long long n = static_cast<long long>(key_tiles(seq_keys(p, s, &err))) * p.row_blocks;
      if (x < at + n) {
        b = s;
        break;
      }
      at += n;
    }
  }
  const uint32_t who = __ballot_sync(0xffffffffu, mine);
  const int src = who ? __ffs(who) - 1 : 0;
  *seq = __shfl_sync(0xffffffffu, b, src);
  *base = __shfl_sync(0xffffffffu, at, src);
}

// The cut at flat tile x inside the item [i0, i1): where it is close to one of the item's
// ends it moves there, which saves a partial result (256 KB written and read again for
// 128 rows) for a little imbalance.
__device__ __forceinline__ long long snap_cut(long long x, long long i0, long long i1,
                                              long long total, int workers) {
  const long long near = (total / workers + 4) / 8;
  if (x - i0 <= near && x - i0 <= i1 - x) return i0;
  if (i1 - x <= near) return i1;
  return x;
}
__device__ __forceinline__ long long raw_cut(long long total, int workers, int w) {
  return total * w / workers;
}

// One worker's walk over its range: an item's tiles j0 .. j1 - 1 at a time.
struct Walk {
  long long x, end, base;  // base: tiles before sequence b
  int b;                   // the current segment's sequence
  int rb, n, nt, j0, j1;   // its row block, keys, tiles, and the range of tiles
};
__device__ __forceinline__ bool walk_next(const LatentDecodeParams& p, Walk& w) {
  if (w.x >= w.end) return false;
  long long span;
  for (;;) {
    int err;
    w.n = seq_keys(p, w.b, &err);
    w.nt = key_tiles(w.n);
    span = static_cast<long long>(w.nt) * p.row_blocks;
    if (w.x < w.base + span) break;
    w.base += span;
    ++w.b;
  }
  const long long in = w.x - w.base;
  w.rb = static_cast<int>(in / w.nt);
  w.j0 = static_cast<int>(in % w.nt);
  const long long left = w.end - w.x;
  w.j1 = left < w.nt - w.j0 ? w.j0 + static_cast<int>(left) : w.nt;
  w.x += w.j1 - w.j0;
  return true;
}

}  // namespace

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kLatThreads, 1)
latent_decode_kernel(const __grid_constant__ CUtensorMap qmap,
                     const __grid_constant__ CUtensorMap cmap, const LatentDecodeParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + kOffBar);
  uint64_t* k_full = bars;                    // [3] CTA 0: both CTAs' chunks have landed
  uint64_t* k_empty = k_full + kKGroups;      // [3] both: S has read them
  uint64_t* v_full = k_empty + kKGroups;      // [2] each CTA its own
  uint64_t* v_empty = v_full + kVGroups;      // [2] both: PV has read them
  uint64_t* q_full = v_empty + kVGroups;      // CTA 0
  uint64_t* q_empty = q_full + 1;             // both: the item's last S is done
  uint64_t* s_full = q_empty + 1;             // [2] both
  uint64_t* p_full = s_full + 2;              // CTA 0: P and the values of both CTAs are there
  uint64_t* pv_done = p_full + 1;             // both
  uint64_t* o_free = pv_done + 1;             // CTA 0: both epilogues have read O
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + kOffMisc);
  volatile int* s_abort = reinterpret_cast<volatile int*>(smem + kOffMisc + 4);
  long long* s_range = reinterpret_cast<long long*>(smem + kOffMisc + 8);  // x, end
  int* s_seq = reinterpret_cast<int*>(smem + kOffMisc + 24);
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
    mbar_init(p_full, 8);   // the four softmax warps of both CTAs
    mbar_init(pv_done, 1);
    mbar_init(o_free, 8);
    fence_barrier_init();
    tma_prefetch_desc(&qmap);
    tma_prefetch_desc(&cmap);
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(tmem_slot)),
                 "r"(kTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  pdl_wait_primary();
  pdl_launch_dependents();
  if (warp == 0) {
    const Flat f = flat_load(p, lane);
    long long cut[2], base = 0;
    int seq = 0;
#pragma unroll
    for (int k = 1; k >= 0; --k) {
      const long long x = raw_cut(f.total, p.workers, worker + k);
      cut[k] = x;
      if (x < f.total) {
        flat_find(p, f, lane, x, &seq, &base);
        int err;
        const int nt = key_tiles(seq_keys(p, seq, &err));
        const long long i0 = base + (x - base) / nt * nt;
        cut[k] = snap_cut(x, i0, i0 + nt, f.total, p.workers);
      }
    }
    // (a cut that moved to its item's end is past sequence `seq`: the walk steps on)
    if (lane == 0) {
      s_range[0] = cut[0];
      s_range[1] = cut[1];
      *s_seq = seq;
      *reinterpret_cast<long long*>(smem + kOffMax) = base;  // read before any maximum is written
      *s_abort = (p.dev_err != nullptr &&
                  (*reinterpret_cast<volatile int32_t*>(p.dev_err) & PKV_DEV_ERR_TIMEOUT))
                     ? 1
                     : 0;
    }
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  Walk w;
  w.x = s_range[0];
  w.end = s_range[1];
  w.b = *s_seq;
  w.base = *reinterpret_cast<long long*>(smem + kOffMax);
  __syncthreads();

  if (warp == 0) {
    // ---------------------------------------------------- loads ----
    const int R = p.box_rows;
    const int half_boxes = 64 / R;   // boxes of a chunk
    uint32_t tc = 0, items = 0;
    const uint32_t k_full0 = peer_u32(k_full, 0);
    const uint32_t q_full0 = peer_u32(q_full, 0);
    bool ok = true;
    while (ok && walk_next(p, w)) {
      const int slot = __ldg(p.batch_idx + w.b);
      const int32_t* table = p.page_table + static_cast<long long>(slot) * p.max_blocks;
      if (lane == 0) {
        ok = items == 0 || wait_pair(q_empty, (items - 1) & 1, s_abort);
        if (ok) {
          if (rank == 0) mbar_arrive_expect_tx(q_full, 2 * kChunks * kChunk);
          const int row = w.b * p.rows + w.rb * kRows + static_cast<int>(rank) * 64;
          for (int c = 0; c < kChunks; ++c)
            tma_load_3d_pair(smem + kOffQ + c * kChunk, &qmap, q_full0, 0, row, c);
        }
      }
      ok = __shfl_sync(0xffffffffu, ok, 0);
      ++items;
      for (int j = w.j0; ok && j < w.j1; ++j, ++tc) {
        // lane k < 128 / R: the pool row of box k of the tile; past the last key, and for
        // an entry without a page, page 0 as filler
        int row = 0;
        bool bad = false;
        if (lane < 2 * half_boxes) {
          const long long t = static_cast<long long>(j) * kKeys + lane * R;
          if (t < w.n) {
            const int blk = static_cast<int>(t) / p.page_size;
            const int page = __ldg(table + blk);
            if (page < 0 || page >= p.num_pages) bad = true;
            else row = page * p.page_size + (static_cast<int>(t) - blk * p.page_size);
          }
        }
        if (__any_sync(0xffffffffu, bad) && lane == 0) set_dev_err(p.dev_err, PKV_DEV_ERR_BAD_PAGE);
        // this CTA's keys for S: box `lane` of its half, from lane + rank * half_boxes
        const int krow =
            __shfl_sync(0xffffffffu, row, (lane + static_cast<int>(rank) * half_boxes) & 31);
        for (int g = 0; ok && g < kKGroups; ++g) {
          ok = tc == 0 || wait_pair(&k_empty[g], (tc - 1) & 1, s_abort);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          if (lane == 0 && rank == 0) mbar_arrive_expect_tx(&k_full[g], 2 * 3 * kChunk);
          __syncwarp();
          if (lane < half_boxes) {
#pragma unroll
            for (int c = 0; c < 3; ++c)
              tma_load_3d_pair(smem + kOffK + (3 * g + c) * kChunk + lane * R * 128, &cmap,
                               k_full0 + 8 * g, 0, krow, 3 * g + c);
          }
        }
        for (int g = 0; ok && g < kVGroups; ++g) {
          ok = tc == 0 || wait_pair(&v_empty[g], (tc - 1) & 1, s_abort);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          if (lane == 0) mbar_arrive_expect_tx(&v_full[g], 4 * kChunk);
          __syncwarp();
          if (lane < 2 * half_boxes) {
            const int kh = lane / half_boxes;  // which half of the tile's keys
            uint8_t* dst = smem + kOffV + (kh * 4 + 2 * g) * kChunk + (lane % half_boxes) * R * 128;
#pragma unroll
            for (int c = 0; c < 2; ++c)
              tma_load_3d(dst + c * kChunk, &cmap, &v_full[g], 0, row,
                          static_cast<int>(rank) * 4 + 2 * g + c);
          }
        }
      }
    }
    if (!ok && lane == 0) *s_abort = 1;
  } else if (warp == 1) {
    // ----------------------------------------------------- MMAs ----
    if (rank == 0) {
      const uint32_t q_lo = desc_lo(smem_u32(smem + kOffQ), 0);
      const uint32_t k_lo = desc_lo(smem_u32(smem + kOffK), 0);
      const uint32_t p_lo = desc_lo(smem_u32(smem + kOffP), 0);
      const uint32_t v_lo = desc_lo(smem_u32(smem + kOffV), kChunk);
      uint32_t tc = 0, items = 0;  // tiles whose PV has been issued; items begun
      bool ok = true;
      auto wait_w = [&](uint64_t* bar, uint32_t parity) -> bool {
        return __all_sync(0xffffffffu, wait_pair(bar, parity, s_abort));
      };
      // S of tile number t: Q C^T into buffer t & 1
      auto issue_s = [&](uint32_t t, bool last) -> bool {
#pragma unroll 1
        for (int g = 0; g < kKGroups; ++g) {
          if (!wait_w(&k_full[g], t & 1)) return false;
          tc_fence_after();
          if (elect_one()) {
#pragma unroll
            for (int c = 0; c < 3; ++c)
              umma4_pair<32, 32>(tmem + kColS + 64 * (t & 1),
                                 q_lo + (((3 * g + c) * kChunk) >> 4),
                                 k_lo + (((3 * g + c) * kChunk) >> 4), kIdescS,
                                 g + c > 0 ? 1u : 0u);
            commit_pair(&k_empty[g]);
            if (g == kKGroups - 1) {
              commit_pair(&s_full[t & 1]);
              if (last) commit_pair(q_empty);
            }
          }
          __syncwarp();
        }
        return true;
      };
      while (ok && walk_next(p, w)) {
        const int nt = w.j1 - w.j0;
        ok = wait_w(q_full, items & 1) && issue_s(tc, nt == 1);
        for (int i = 0; ok && i < nt; ++i) {
          if (i + 1 < nt) ok = issue_s(tc + 1, i + 2 == nt);
          ok = ok && wait_w(p_full, tc & 1);
          if (ok && i == 0 && items > 0) ok = wait_w(o_free, (items - 1) & 1);
          if (!ok) break;
          tc_fence_after();
          const int left = w.n - (w.j0 + i) * kKeys;
          const int steps = left >= kKeys ? 8 : (left + 15) >> 4;  // of 16 keys
          if (elect_one()) {
#pragma unroll 1
            for (int g = 0; g < kVGroups; ++g) {
              const uint32_t vg = v_lo + ((2 * g * kChunk) >> 4);
#pragma unroll 1
              for (int kh = 0; kh < 2; ++kh) {
                const uint32_t a = p_lo + ((kh * kChunk) >> 4);
                const uint32_t b = vg + ((kh * 4 * kChunk) >> 4);
                const uint32_t acc = (i > 0 || kh > 0) ? 1u : 0u;
                const int n = steps - 4 * kh;
                if (n >= 4) {
                  umma4_pair<32, 2048>(tmem + 128 * g, a, b, kIdescO, acc);
                } else {
                  for (int k = 0; k < n; ++k)
                    umma1_pair(tmem + 128 * g, a + 2 * k, b + 128 * k, kIdescO,
                               acc | (k > 0 ? 1u : 0u));
                }
              }
              commit_pair(&v_empty[g]);
            }
            commit_pair(pv_done);
          }
          __syncwarp();
          ++tc;
        }
        ++items;
      }
      if (!ok && lane == 0) *s_abort = 1;
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
    uint32_t tc = 0;
    bool ok = true;
    while (ok && walk_next(p, w)) {
      const int row = w.rb * kRows + static_cast<int>(rank) * 64 + r;  // row of the sequence
      const bool live = row < p.rows;
      const bool warp_live = __any_sync(0xffffffffu, live);
      // keys that the row sees: all but those of the drafts behind its token
      const int lim = live ? w.n - (p.n_q - 1 - row / p.heads) : 0;
      float m_run = -INFINITY;  // running maximum of the row, raw score units
      float l_run = 0.f;        // sum over this thread's half of the keys
      bool left_together = false;
      for (int j = w.j0; j < w.j1; ++j, ++tc) {
        // a wait that gave up is told to the other warps at their next common barrier, so
        // that all four leave at the same place
        ok = ok && wait_pair(&s_full[tc & 1], (tc >> 1) & 1, s_abort);
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
        // the values of both halves have landed here; P and O are free once the last PV is done
        ok = wait_or_abort(&v_full[0], tc & 1, s_abort) &&
             wait_or_abort(&v_full[1], tc & 1, s_abort) &&
             (tc == 0 || wait_pair(pv_done, (tc - 1) & 1, s_abort));
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
        const int left = w.n - j * kKeys;
        if (left < kKeys && (left & 15)) {
          const int z0 = left, nz = 16 - (left & 15);
          for (int q = tl; q < nz * 32; q += 128) {
            const int key = z0 + (q >> 5);
            uint8_t* at = smem + kOffV + ((key >> 6) * 4 + ((q >> 3) & 3)) * kChunk +
                          (key & 63) * 128 + (q & 7) * 16;
            *reinterpret_cast<uint4*>(at) = make_uint4(0u, 0u, 0u, 0u);
          }
        }
        fence_proxy_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(p_full0);
      }
      // ---- the segment's end: O and the row's maximum and sum ----
      if (left_together) break;
      ok = ok && wait_pair(pv_done, (tc - 1) & 1, s_abort);
      float* const sums = s_max + 256;
      sums[tl] = l_run;
      ok = named_bar_all(1, 128, ok);
      tc_fence_after();
      if (ok) {
        const float l = l_run + sums[tl ^ 64];
        const bool whole = w.j0 == 0 && w.j1 == w.nt;
        if (warp_live) {
          if (whole) {
            const bool has = live && l > 0.f;
            const float inv = has ? 1.f / l : 0.f;
            const long long at = static_cast<long long>(w.b) * p.rows + row;
            __nv_bfloat16* orow = p.out + at * kLatent + hk * 256;
#pragma unroll 1
            for (int q = 0; q < 256; q += 32) {
              uint32_t o[32];
              tmem_ld32(t_lane + q, o);
              tmem_wait_ld();
              if (live) {
#pragma unroll
                for (int v = 0; v < 2; ++v) {
                  uint32_t wv[8];
#pragma unroll
                  for (int e = 0; e < 8; ++e) {
                    const float a = __uint_as_float(o[16 * v + 2 * e]) * inv;
                    const float b = __uint_as_float(o[16 * v + 2 * e + 1]) * inv;
                    wv[e] = has ? pack_bf16x2(a, b) : 0u;
                  }
                  st_global_v8(orow + q + 16 * v, wv);
                }
              }
            }
            if (live && hk == 0)
              p.lse[at] = has ? (m_run * p.qscale + __log2f(l)) * 0.69314718055994531f : -INFINITY;
          } else {
            const int part = 2 * worker + (w.j0 == 0 ? 1 : 0);
            const long long at = static_cast<long long>(part) * p.block_rows + (row - w.rb * kRows);
            float* orow = p.part_o + at * kLatent + hk * 256;
#pragma unroll 1
            for (int q = 0; q < 256; q += 32) {
              uint32_t o[32];
              tmem_ld32(t_lane + q, o);
              tmem_wait_ld();
              if (live) {
#pragma unroll
                for (int v = 0; v < 4; ++v)
                  st_global_v8(orow + q + 8 * v, *reinterpret_cast<uint32_t(*)[8]>(&o[8 * v]));
              }
            }
            if (live && hk == 0) {
              p.part_ml[2 * at] = m_run;
              p.part_ml[2 * at + 1] = l;
            }
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
  cluster_sync_all();
  if (warp == 1) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem),
                 "r"(kTmemCols)
                 : "memory");
  }
}

// Joins the partials of split items, and writes the rows of sequences without keys. A warp
// takes one row: 16 of its 512 values a lane, the partials one after another (their loads do
// not depend on each other), with weights 2^(m_i - max m) and the sum of the l_i.
constexpr int kJoinWarps = 8;

__global__ void __launch_bounds__(kJoinWarps * 32) latent_join_kernel(const LatentDecodeParams p) {
  pdl_wait_primary();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int groups = (p.block_rows + kJoinWarps - 1) / kJoinWarps;
  const int item = blockIdx.x / groups;
  const int row_in = (blockIdx.x - item * groups) * kJoinWarps + (threadIdx.x >> 5);
  const int b = item / p.row_blocks;
  const int rb = item - b * p.row_blocks;
  const int row = rb * kRows + row_in;
  if (row_in >= p.block_rows || row >= p.rows) return;
  int err;
  const int n = seq_keys(p, b, &err);
  const long long at = static_cast<long long>(b) * p.rows + row;
  uint4* orow = reinterpret_cast<uint4*>(p.out + at * kLatent) + 2 * lane;
  if (n == 0) {
    if (err && lane == 0) set_dev_err(p.dev_err, err);
    orow[0] = make_uint4(0u, 0u, 0u, 0u);
    orow[1] = make_uint4(0u, 0u, 0u, 0u);
    if (lane == 0) p.lse[at] = -INFINITY;
    return;
  }
  const Flat f = flat_load(p, lane);
  // tiles before sequence b
  long long base = 0;
  {
    const int owner = b / f.per;
    long long v = f.before;
    if (lane == owner) {
      for (int s = owner * f.per; s < b; ++s) {
        int e;
        v += static_cast<long long>(key_tiles(seq_keys(p, s, &e))) * p.row_blocks;
      }
    }
    base = __shfl_sync(0xffffffffu, v, owner);
  }
  const int nt = key_tiles(n);
  const long long i0 = base + static_cast<long long>(rb) * nt, i1 = i0 + nt;
  // the first worker whose range begins inside the item
  int wf = static_cast<int>(i0 * p.workers / f.total);
  auto cut = [&](int wk) -> long long {  // of a worker whose raw cut may lie outside: i0 or i1
    const long long x = raw_cut(f.total, p.workers, wk);
    if (x <= i0) return i0;
    if (x >= i1) return i1;
    return snap_cut(x, i0, i1, f.total, p.workers);
  };
  while (wf < p.workers && cut(wf) <= i0) ++wf;
  if (wf >= p.workers || cut(wf) >= i1) return;  // one worker has the whole item
  // partials: worker wf - 1's last one, then those of the workers that begin inside
  float m = -INFINITY, l = 0.f;
  float o[16];
#pragma unroll
  for (int e = 0; e < 16; ++e) o[e] = 0.f;
  auto add = [&](int part) {
    const long long pr = static_cast<long long>(part) * p.block_rows + row_in;
    const float4* src = reinterpret_cast<const float4*>(p.part_o + pr * kLatent) + 4 * lane;
    const float4 v[4] = {src[0], src[1], src[2], src[3]};
    const float mi = p.part_ml[2 * pr], li = p.part_ml[2 * pr + 1];
    if (mi == -INFINITY) return;  // no key of this range is seen by the row
    const float mn = fmaxf(m, mi);
    const float keep = ex2((m - mn) * p.qscale), take = ex2((mi - mn) * p.qscale);
    l = l * keep + li * take;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      o[4 * e] = o[4 * e] * keep + v[e].x * take;
      o[4 * e + 1] = o[4 * e + 1] * keep + v[e].y * take;
      o[4 * e + 2] = o[4 * e + 2] * keep + v[e].z * take;
      o[4 * e + 3] = o[4 * e + 3] * keep + v[e].w * take;
    }
    m = mn;
  };
  add(2 * (wf - 1) + 1);
  for (int wk = wf; wk < p.workers; ++wk) {
    const long long c = cut(wk);
    if (c >= i1) break;
    if (wk + 1 < p.workers && cut(wk + 1) == c) continue;  // an empty range
    add(2 * wk);
  }
  const bool has = l > 0.f;
  const float inv = has ? 1.f / l : 0.f;
  uint32_t wv[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) wv[e] = has ? pack_bf16x2(o[2 * e] * inv, o[2 * e + 1] * inv) : 0u;
  orow[0] = make_uint4(wv[0], wv[1], wv[2], wv[3]);
  orow[1] = make_uint4(wv[4], wv[5], wv[6], wv[7]);
  if (lane == 0)
    p.lse[at] = has ? (m * p.qscale + __log2f(l)) * 0.69314718055994531f : -INFINITY;
}

namespace {

// {64 values, rows, 9 chunks} view of an array of rows of 576; one box is `box_rows` rows of
// one chunk, 128-byte swizzled.
bool encode_rows_map(CUtensorMap* map, const void* base, long long rows, int box_rows) {
  prefill_host::EncodeTiledFn enc = prefill_host::encode_fn();
  if (enc == nullptr) return false;
  const cuuint64_t dims[3] = {64u, static_cast<cuuint64_t>(rows), kChunks};
  const cuuint64_t strides[2] = {kRow * 2, 128u};
  const cuuint32_t box[3] = {64u, static_cast<cuuint32_t>(box_rows), 1u};
  const cuuint32_t estr[3] = {1u, 1u, 1u};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box,
             estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

constexpr int kMaxQueries = 64;
constexpr int kMaxHeads = 1024;

bool latent_rows_ok(int batch, int n_q, int heads) {
  return batch >= 0 && n_q >= 1 && n_q <= kMaxQueries && heads >= 1 && heads <= kMaxHeads &&
         static_cast<long long>(batch) * n_q * heads <= INT_MAX;
}
int launch_batch(int batch) {
  const int launches = (batch + kMaxRowsPerLaunch - 1) / kMaxRowsPerLaunch;
  return launches > 0 ? (batch + launches - 1) / launches : 0;
}
// Pairs of CTAs of a launch, and the bytes of its partials.
int launch_workers(const pkv_cache_desc* c, int batch, int rows, int sm_count) {
  const long long blocks = (static_cast<long long>(c->max_blocks) * c->page_size + kKeys - 1) / kKeys;
  const long long tiles = blocks * batch * ((rows + kRows - 1) / kRows);
  const int pairs = sm_count / 2;
  return tiles < pairs ? static_cast<int>(tiles) : pairs;
}
size_t partial_bytes(int workers, int rows) {
  const size_t block_rows = rows < kRows ? rows : kRows;
  return static_cast<size_t>(2 * workers) * block_rows * (kLatent + 2) * sizeof(float);
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
  const size_t n = partial_bytes(launch_workers(cache, launch_batch(batch), rows, sms), rows);
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
  if (!is_aligned(pool, 16) || !is_aligned(q, 16) || !is_aligned(out, 32) || !is_aligned(lse, 4) ||
      !is_aligned(page_table, 4) || !is_aligned(batch_idx, 4) || !is_aligned(seq_lens, 4) ||
      !is_aligned(dev_err, 4) || !is_aligned(workspace, 256))
    return PKV_ERR_ALIGN;
  int sms = 0;
  if (const pkv_status st = device_info(&sms); st != PKV_OK) return st;
  const int rows = n_q * num_heads;
  const int per = launch_batch(batch);
  const int workers = launch_workers(cache, per, rows, sms);
  if (!workspace || workspace_bytes < partial_bytes(workers, rows)) return PKV_ERR_WORKSPACE;
  int box = 64;
  while (cache->page_size % box) box >>= 1;  // 16, 32 or 64
  CUtensorMap cmap;
  if (!encode_rows_map(&cmap, pool, static_cast<long long>(cache->num_pages) * cache->page_size, box))
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
  p.page_table = page_table;
  p.dev_err = dev_err;
  p.heads = num_heads;
  p.n_q = n_q;
  p.rows = rows;
  p.row_blocks = (rows + kRows - 1) / kRows;
  p.block_rows = rows < kRows ? rows : kRows;
  p.page_size = cache->page_size;
  p.num_pages = cache->num_pages;
  p.max_batch = cache->max_batch;
  p.max_blocks = cache->max_blocks;
  p.box_rows = box;
  p.qscale = scale * 1.4426950408889634f;
  for (int b0 = 0; b0 < batch; b0 += per) {
    const int n = batch - b0 < per ? batch - b0 : per;
    const long long first = static_cast<long long>(b0) * rows;
    const __nv_bfloat16* q0 = static_cast<const __nv_bfloat16*>(q) + first * kRow;
    CUtensorMap qmap;
    if (!encode_rows_map(&qmap, q0, static_cast<long long>(n) * rows, 64)) return PKV_ERR_ARG;
    p.batch_idx = batch_idx + b0;
    p.seq_lens = seq_lens + b0;
    p.out = static_cast<__nv_bfloat16*>(out) + first * kLatent;
    p.lse = lse + first;
    p.batch = n;
    p.workers = launch_workers(cache, n, rows, sms);
    p.part_o = static_cast<float*>(workspace);
    p.part_ml = p.part_o + static_cast<size_t>(2 * p.workers) * p.block_rows * kLatent;
    cudaError_t e = launch_kernel(latent_decode_kernel, dim3(2 * p.workers), dim3(kLatThreads),
                                  kLatSmem, stream, true, qmap, cmap, p);
    if (e != cudaSuccess) return record_cuda_status(e);
    const long long groups = (p.block_rows + kJoinWarps - 1) / kJoinWarps;
    e = launch_kernel(latent_join_kernel,
                      dim3(static_cast<unsigned>(groups * n * p.row_blocks)),
                      dim3(kJoinWarps * 32), 0, stream, true, p);
    if (e != cudaSuccess) return record_cuda_status(e);
  }
  return PKV_OK;
}
