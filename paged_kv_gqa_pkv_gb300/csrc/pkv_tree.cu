// pkv_tree.cu - pkv_tree_attention: a tree of drafted tokens per sequence over
// the paged cache, on tcgen05.
//
// For one sequence and one kv head the queries are R = nodes x group rows (row
// r is node r / G, query head kvh * G + r % G), all over the same keys: the
// committed context, which every row sees whole, and the tree's own nodes,
// where a row sees its ancestors. So the keys stream once per (sequence, kv
// head) however large the tree is, as in the decode, while the products are
// those of a 128-row tile, as in the chunked prefill: S = Q K^T and O += P V on
// tcgen05, 128 keys at a time, P kept in tensor memory over S.
//
// Masks: a node's ancestors-or-self are one 64-bit word, built per warp from
// the parents by pointer doubling (six rounds of shuffles). A key tile that
// ends inside the context needs no mask; in the last one or two tiles a row's
// 128 visible columns are the context's low bits and its ancestor word shifted
// to the tree's place in the tile. V rows past the last node are zeroed in
// shared memory (stale slots may hold any bits, and 0 * NaN is not 0).
//
// What bounds it: the K/V stream. A 128-key tile of K and V is 64 KB, ~1.45 us
// of one SM's share of the measured copy bandwidth; its two products at 128
// rows take 0.27 us each. Both softmax warpgroups are kept busy in either of
// two forms of the kernel:
//   R <= 128 (kTwo = false): one row tile; the warpgroups take the even and the
//     odd key tiles, each with its own running maximum, sum and accumulator,
//     joined when the segment ends. One chain of product, softmax, product
//     after another would leave the tensor pipe and the loads waiting.
//   R > 128 (kTwo = true): two row tiles, one per warpgroup, over the same key
//     tiles; above 256 rows further row blocks are items of their own.
//
// Schedule: the list of all (sequence, kv head, row block) items' key tiles is
// cut into gridDim equal ranges, one per CTA; a range's pieces of items are its
// segments. An item inside one range is written out by its CTA. An item cut by
// range borders leaves one partial (unnormalised O, running maximum and sum)
// per CTA, at most two per CTA (its first and its last segment), and the merge
// kernel joins them. Partials are stored column by column, so that the rows,
// one per thread, are contiguous.
#include <atomic>
#include <cmath>

#include "pkv_prefill_common.cuh"

namespace pkv {

namespace {

using namespace prefill_detail;

constexpr int kMaxRows = 256;          // query rows of an item
constexpr int kTreeMaxBatch = 192;     // batch rows per launch (tile prefix in shared memory)
constexpr int kRing = 5;               // K/V tile slots
constexpr int kMergeThreads = 256;
constexpr int kMergeCols = 8;          // head dims per merge thread
constexpr int kMergeUnroll = 4;        // partials in flight per merge thread

// shared memory: two Q tiles (the two row tiles of an item, or in the one-tile
// form this segment's and the next one's), the K/V ring, barriers, and in the
// one-tile form the second warpgroup's maxima and sums
constexpr int kOffQ = 0;
constexpr int kOffRing = kOffQ + 2 * kTileBytes;
constexpr int kOffBar = kOffRing + kRing * kTileBytes;
// q_full[2], q_empty[2], ring_full[kRing], ring_empty[kRing], s_full[2],
// p_full[2], pv_done[2], o_free[2], x_full
constexpr int kNumBars = 4 + 2 * kRing + 9;
constexpr int kOffXch = kOffBar + kNumBars * 8;   // float2 [128]
constexpr int kOffMisc = kOffXch + 128 * 8;       // tmem slot, abort flag, scan
constexpr int kOffPrefix = kOffMisc + 8 + 40;
constexpr int kSmemBytes = kOffPrefix + (kTreeMaxBatch + 1) * 4 + 1024;
static_assert(kSmemBytes <= kMaxDynSmem, "shared memory above the opt-in limit");

struct TreeParams {
  const int32_t* page_table;
  const int32_t* parents;
  const int32_t* tree_lens;
  const int32_t* batch_idx;
  const int32_t* ctx_lens;
  void* out;
  float* lse;
  int32_t* prefix;   // workspace: [batch + 1] key tiles of the rows before each row
  float* partials;   // workspace: 2 * workers slots of slot_floats
  int32_t* dev_err;
  int batch;
  int n_nodes;
  int num_q_heads;
  int num_kv_heads;
  int group;
  int rows;          // n_nodes * group
  int row_blocks;    // items per (sequence, kv head)
  int items_per_row; // num_kv_heads * row_blocks
  int q_box_nodes;   // nodes of one Q box: min(128 / group, n_nodes)
  int page_size;
  int num_pages;
  int max_batch;
  int max_blocks;
  int box_rows;      // rows of one K/V box: min(page_size, 128)
  int workers;       // ranges of the tile list (CTAs, or teams of warps)
  int slot_rows;     // rows of a partial slot: min(rows, kMaxRows)
  int merge_split;   // merge threads that share an item's partials (a power of two)
  float qscale;      // scale * log2(e)
};

// A partial slot: O [rows][128], then m and l [rows], 16-byte aligned.
__host__ __device__ __forceinline__ int64_t slot_floats(int rows) {
  return static_cast<int64_t>(rows) * kHeadDim + (2 * rows + 3) / 4 * 4;
}

// Tiles of kTile keys of batch row b (0: nothing to attend), and the error it
// raises.
template <int kTile>
__device__ __forceinline__ int tree_row_tiles(const TreeParams& p, int b, int* err) {
  const int slot = p.batch_idx[b], ctx = p.ctx_lens[b], n = p.tree_lens[b];
  *err = 0;
  if (slot == 0) return 0;
  if (slot < 0 || slot >= p.max_batch) *err = PKV_DEV_ERR_BAD_SLOT;
  else if (n < 0 || n > p.n_nodes) *err = PKV_DEV_ERR_BAD_TREE;
  else if (ctx < 0 || static_cast<int64_t>(ctx) + n >
                          static_cast<int64_t>(p.max_blocks) * p.page_size)
    *err = PKV_DEV_ERR_BAD_POS;
  if (*err || n == 0) return 0;
  return static_cast<int>((static_cast<int64_t>(ctx) + n + kTile - 1) / kTile);
}

// One CTA's piece of an item.
struct Segment {
  int b, item;       // batch row, item within the row
  int t0, t1;        // key tiles [t0, t1) of `tiles`
  int tiles;
};

__device__ __forceinline__ void close_segment(Segment& s, int64_t left) {
  s.t1 = left < s.tiles - s.t0 ? s.t0 + static_cast<int>(left) : s.tiles;
}

// The segment that starts at tile u of the list (below u_end).
__device__ __forceinline__ Segment first_segment(const int32_t* prefix, int batch, int ipr,
                                                 int64_t u, int64_t u_end) {
  int lo = 0, hi = batch - 1;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (static_cast<int64_t>(prefix[mid + 1]) * ipr > u) hi = mid;
    else lo = mid + 1;
  }
  Segment s;
  s.b = lo;
  s.tiles = prefix[lo + 1] - prefix[lo];
  const int64_t r = u - static_cast<int64_t>(prefix[lo]) * ipr;
  s.item = static_cast<int>(r / s.tiles);
  s.t0 = static_cast<int>(r % s.tiles);
  close_segment(s, u_end - u);
  return s;
}

// The next item's segment; `left` tiles (at least one) remain in the range.
__device__ __forceinline__ Segment next_segment(Segment s, const int32_t* prefix, int ipr,
                                                int64_t left) {
  s.t0 = 0;
  if (++s.item == ipr) {
    s.item = 0;
    do {
      ++s.b;
      s.tiles = prefix[s.b + 1] - prefix[s.b];
    } while (s.tiles == 0);
  }
  close_segment(s, left);
  return s;
}

// Tiles per batch row and their prefix in s_prefix[0 .. batch], by every CTA (it
// ends before a barrier that the caller owes); CTA 0 also leaves the prefix to
// the merge.
template <int kTile>
__device__ __forceinline__ void tile_prefix(const TreeParams& p, int32_t* s_prefix, int* s_scan) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int tiles = 0;
  if (threadIdx.x < kTreeMaxBatch && static_cast<int>(threadIdx.x) < p.batch) {
    int err;
    tiles = tree_row_tiles<kTile>(p, threadIdx.x, &err);
    if (err && blockIdx.x == 0) set_dev_err(p.dev_err, err);
  }
  int incl = tiles;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += v;
  }
  if (lane == 31) s_scan[warp] = incl;
  __syncthreads();
  int before = 0;
  for (int w = 0; w < warp; ++w) before += s_scan[w];
  if (threadIdx.x < kTreeMaxBatch) {
    s_prefix[threadIdx.x + 1] = before + incl;
    if (blockIdx.x == 0 && static_cast<int>(threadIdx.x) < p.batch)
      p.prefix[threadIdx.x + 1] = before + incl;
  }
  if (threadIdx.x == 0) {
    s_prefix[0] = 0;
    if (blockIdx.x == 0) p.prefix[0] = 0;
  }
}

// The K/V stream is read once where an item's rows fit one row block: its
// loads carry an L2 evict-first policy, so the partials and the page table stay.
__device__ __forceinline__ uint64_t kv_policy(bool once) {
  uint64_t pol;
  if (once) asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(pol));
  else asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(pol));
  return pol;
}

__device__ __forceinline__ void tma_load_4d_hint(void* dst, const CUtensorMap* map, uint64_t* bar,
                                                 int x, int y, int z, int w, uint64_t pol) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1, {%3, %4, %5, %6}], [%2], %7;" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(x), "r"(y), "r"(z), "r"(w),
      "l"(pol)
      : "memory");
}

// Node `lane` and node `lane + 32` of a tree of n nodes: the word of its
// ancestors and itself, 0 for a node past n or with an invalid parent on its
// way up. Warp-collective. bad: some node below n has an invalid parent.
__device__ __forceinline__ void ancestor_words(const int32_t* parents, int n, int lane,
                                               uint64_t (&word)[2], bool& bad) {
  int up[2];
  bool wrong = false;
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int i = lane + 32 * k;
    up[k] = -1;
    word[k] = 0;
    if (i < n) {
      up[k] = parents[i];
      word[k] = 1ull << i;
      if (up[k] < -1 || up[k] >= i) {
        wrong = true;
        up[k] = -1;
        word[k] = 0;
      }
    }
  }
  bad = __any_sync(0xffffffffu, wrong);
  const uint32_t dead0 = __ballot_sync(0xffffffffu, word[0] == 0);
  const uint32_t dead1 = __ballot_sync(0xffffffffu, word[1] == 0);
  const uint64_t dead = static_cast<uint64_t>(dead1) << 32 | dead0;
  // after round r a word holds the node and its 2^r - 1 nearest ancestors, and
  // `up` the 2^r-th
#pragma unroll
  for (int r = 0; r < 6; ++r) {
    const uint64_t w0 = word[0], w1 = word[1];
    const int u0 = up[0], u1 = up[1];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int at = up[k] & 31;
      const uint64_t a0 = __shfl_sync(0xffffffffu, w0, at), a1 = __shfl_sync(0xffffffffu, w1, at);
      const int b0 = __shfl_sync(0xffffffffu, u0, at), b1 = __shfl_sync(0xffffffffu, u1, at);
      if (up[k] >= 0) {
        word[k] |= up[k] < 32 ? a0 : a1;
        // a parent that is itself cut off contributes no word of its own
        word[k] |= 1ull << up[k];
        up[k] = up[k] < 32 ? b0 : b1;
      }
    }
  }
#pragma unroll
  for (int k = 0; k < 2; ++k)
    if ((word[k] & dead) != 0) word[k] = 0;
}

// Bits 32 w .. 32 w + 31 of the visible columns of a tile whose columns
// [0, off) are context and column off + a is node a (off may be negative or
// past the tile).
__device__ __forceinline__ uint32_t visible_word(int w, int off, uint64_t anc) {
  const int s = 32 * w - off;  // bit 0 of this word is node s
  uint32_t v = 0;
  if (s >= 0) v = s < 64 ? static_cast<uint32_t>(anc >> s) : 0u;
  else if (s > -32) v = (static_cast<uint32_t>(anc) << -s) | ((1u << -s) - 1u);
  else v = 0xffffffffu;
  return v;
}

}  // namespace

// 10 warps: warp 0 loads, warp 1 issues the tensor instructions, warps 2-5 and
// 6-9 are the softmax warpgroups.
template <bool kTwo>
__global__ void __launch_bounds__(kThreads, 1)
tree_attention_kernel(const __grid_constant__ CUtensorMap qmap,
                      const __grid_constant__ CUtensorMap kmap,
                      const __grid_constant__ CUtensorMap vmap, const TreeParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + kOffBar);
  uint64_t* q_full = bars + 0;              // [2]; two tiles: [0] stands for both
  uint64_t* q_empty = bars + 2;             // [2]
  uint64_t* ring_full = bars + 4;           // [kRing]
  uint64_t* ring_empty = bars + 4 + kRing;  // [kRing]
  uint64_t* s_full = bars + 4 + 2 * kRing;  // [2]
  uint64_t* p_full = s_full + 2;            // [2]
  uint64_t* pv_done = s_full + 4;           // [2]
  uint64_t* o_free = s_full + 6;            // [2]; one tile: [0] stands for both
  uint64_t* x_full = s_full + 8;            // one tile: the second warpgroup's maxima and sums
  float2* xch = reinterpret_cast<float2*>(smem + kOffXch);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + kOffMisc);
  volatile int* s_abort = reinterpret_cast<volatile int*>(smem + kOffMisc + 4);
  int* s_scan = reinterpret_cast<int*>(smem + kOffMisc + 8);
  int32_t* s_prefix = reinterpret_cast<int32_t*>(smem + kOffPrefix);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kRing; ++s) {
      mbar_init(&ring_full[s], 1);
      mbar_init(&ring_empty[s], 1);
    }
    for (int h = 0; h < 2; ++h) {
      mbar_init(&q_full[h], 1);
      mbar_init(&q_empty[h], 1);
      mbar_init(&s_full[h], 1);
      mbar_init(&p_full[h], kGroupThreads);
      mbar_init(&pv_done[h], 1);
      mbar_init(&o_free[h], kGroupThreads);
    }
    mbar_init(x_full, kGroupThreads);
    *s_abort = 0;
    fence_barrier_init();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&qmap);
    tma_prefetch_desc(&kmap);
    tma_prefetch_desc(&vmap);
  }
  if (warp == 1) tmem_alloc(tmem_slot, kTmemCols);
  pdl_wait_primary();
  pdl_launch_dependents();  // the merge waits for this grid before it reads anything

  tile_prefix<kBN>(p, s_prefix, s_scan);
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  const int ipr = p.items_per_row;
  const int64_t total = static_cast<int64_t>(s_prefix[p.batch]) * ipr;
  const int64_t per = (total + p.workers - 1) / p.workers;
  const int64_t u0 = static_cast<int64_t>(blockIdx.x) * per;
  const int64_t u_end = u0 + per < total ? u0 + per : total;

  if (warp == 0) {
    // ---------------------------------------------------- TMA producer ----
    uint32_t L = 0;   // ring loads issued
    uint32_t si = 0;  // segments
    const int R = p.box_rows;
    const int nsub = kBN / R;         // boxes per head-dim half of a key tile (1..8)
    const int tpc = 32 / nsub;        // key tiles per chunk of page-table entries
    const uint64_t pol = kv_policy(p.row_blocks == 1);
    // Pool rows of chunk c of a segment's boxes, box k of tile t0 + c * tpc + i
    // in lane i * nsub + k. Boxes past the last key, and unreserved entries
    // (flagged), read page 0 as filler.
    auto chunk_rows = [&](const Segment& sg, int c) -> int {
      const int slot = p.batch_idx[sg.b];
      const int last = p.ctx_lens[sg.b] + p.tree_lens[sg.b] - 1;  // last key
      const int j = sg.t0 + c * tpc + lane / nsub;
      const int l0 = j * kBN + (lane % nsub) * R;
      if (j >= sg.t1 || l0 > last) return 0;
      const int pg = p.page_table[static_cast<int64_t>(slot) * p.max_blocks + l0 / p.page_size];
      if (pg >= 0 && pg < p.num_pages) return pg * p.page_size + l0 % p.page_size;
      set_dev_err(p.dev_err, PKV_DEV_ERR_BAD_PAGE);
      return 0;
    };
    Segment sg;
    int next_rows = 0;
    if (u0 < u_end) {
      sg = first_segment(s_prefix, p.batch, ipr, u0, u_end);
      next_rows = chunk_rows(sg, 0);
    }
    for (int64_t u = u0; u < u_end && !*s_abort;) {
      const int n = sg.t1 - sg.t0;
      u += n;
      int rows[2] = {next_rows, 0};   // of the even and the odd chunk at hand
      rows[1] = n > tpc ? chunk_rows(sg, 1) : 0;
      Segment nx = sg;
      if (u < u_end) {
        nx = next_segment(sg, s_prefix, ipr, u_end - u);
        next_rows = chunk_rows(nx, 0);  // in flight while this segment streams
      }
      const int kvh = sg.item / p.row_blocks;
      const int rb = sg.item % p.row_blocks;
      bool ok = true;
      // Q of this segment. One tile: the other buffer than the last segment's.
      // Two tiles: the one buffer, free after the last segment's last QK, so it
      // is asked for only after the first kQDefer K/V tiles.
      auto load_q = [&]() -> bool {
        bool good = true;
        if (lane == 0) {
          constexpr int kTiles = kTwo ? 2 : 1;
          const uint32_t buf = kTwo ? 0 : si & 1, use = kTwo ? si : si >> 1;
          good = use == 0 || wait_or_abort(&q_empty[buf], (use - 1) & 1, s_abort);
          if (good) {
            mbar_arrive_expect_tx(&q_full[buf], kTiles * 2 * p.q_box_nodes * p.group * 128);
            for (int h = 0; h < kTiles; ++h) {
              const int node0 = sg.b * p.n_nodes + (rb * 2 + h) * (kBM / p.group);
              uint8_t* qd = smem + kOffQ + (kTwo ? h : buf) * kTileBytes;
              tma_load_3d(qd, &qmap, &q_full[buf], 0, kvh * p.group, node0);
              tma_load_3d(qd + kHalf, &qmap, &q_full[buf], 64, kvh * p.group, node0);
            }
          }
        }
        return __shfl_sync(0xffffffffu, good, 0);
      };
      // one 128-key tile, i tiles into the segment
      auto load = [&](const CUtensorMap* map, int i) -> bool {
        const int c = i / tpc;
        const int have = (c & 1) ? rows[1] : rows[0];
        const int lane0 = (i - c * tpc) * nsub;
        int at[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) at[k] = __shfl_sync(0xffffffffu, have, (lane0 + k) & 31);
        bool good = true;
        if (lane == 0) {
          const uint32_t s = L % kRing;
          if (L >= kRing && !wait_or_abort(&ring_empty[s], ((L / kRing) - 1) & 1, s_abort)) {
            good = false;
          } else {
            uint8_t* dst = smem + kOffRing + s * kTileBytes;
            mbar_arrive_expect_tx(&ring_full[s], kTileBytes);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              if (k < nsub) {
                tma_load_4d_hint(dst + k * R * 128, map, &ring_full[s], 0, at[k], 0, kvh, pol);
                tma_load_4d_hint(dst + kHalf + k * R * 128, map, &ring_full[s], 0, at[k], 1, kvh,
                                 pol);
              }
            }
          }
        }
        good = __shfl_sync(0xffffffffu, good, 0);
        if (good) ++L;
        return good;
      };
      // ring order = the issuer's order: the K tiles run kAhead tiles before
      // the V tiles (one per chain in flight)
      constexpr int kAhead = kTwo ? 1 : 2;
      constexpr int kQDefer = kTwo ? 3 : 0;
      int loads = 0, ik = 0;
      auto next_load = [&](const CUtensorMap* map, int i) -> bool {
        if (loads++ == kQDefer && !load_q()) return false;
        return load(map, i);
      };
      for (; ok && ik < kAhead && ik < n; ++ik) ok = next_load(&kmap, ik);
      for (int i = 0; ok && i < n; ++i) {
        if (i > 0 && i % tpc == 0) {
          // V enters chunk c: chunk c - 1 is done with, c + 1 takes its place
          const int c = i / tpc;
          const int more = (c + 1) * tpc < n ? chunk_rows(sg, c + 1) : 0;
          if (c & 1) rows[0] = more;
          else rows[1] = more;
        }
        if constexpr (kTwo) {
          if (ik < n) ok = next_load(&kmap, ik++);
          ok = ok && next_load(&vmap, i);
        } else {
          ok = next_load(&vmap, i);
          if (ok && ik < n) ok = next_load(&kmap, ik++);
        }
      }
      if (ok && loads <= kQDefer) ok = load_q();
      sg = nx;
      if (!ok && lane == 0) *s_abort = 1;
      __syncwarp();
      ++si;
      if (!ok) break;
    }
    // copies still in flight land before the CTA leaves
    if (__any_sync(0xffffffffu, *s_abort != 0) && lane == 0) {
      const uint32_t first = L > kRing ? L - kRing : 0;
      for (uint32_t l = first; l < L; ++l) mbar_wait_bounded(&ring_full[l % kRing], (l / kRing) & 1);
    }
  } else if (warp == 1) {
    // ------------------------------------------------------ MMA issuer ----
    uint32_t C = 0;             // ring slots consumed
    uint32_t si = 0;            // segments
    uint32_t pv[2] = {0, 0};    // PV products issued per chain
    const uint32_t sR = smem_u32(smem + kOffRing);
    uint32_t qd[2][8];  // the two Q tiles
    kmajor_steps(smem_u32(smem + kOffQ), qd[0]);
    kmajor_steps(smem_u32(smem + kOffQ + kTileBytes), qd[1]);
    auto wait_w = [&](uint64_t* bar, uint32_t parity) -> bool {
      return __shfl_sync(0xffffffffu, wait_or_abort(bar, parity, s_abort) ? 1 : 0, 0) != 0;
    };
    auto issue_qk = [&](int h, const uint32_t (&kb)[8]) {  // S_h = Q K^T
      if (elect_one()) {
        uint32_t qa[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) qa[e] = (kTwo ? h : si & 1) ? qd[1][e] : qd[0][e];
        umma8_ss(tmem + static_cast<uint32_t>(h * kBN), qa, kb, kIdescQK, 0u);
        umma_commit(&s_full[h]);
      }
      __syncwarp();
    };
    auto issue_pv = [&](int h, const uint32_t (&vb)[8], uint32_t acc) {  // O_h (+)= P_h V
      if (elect_one()) {
        umma8_ts(tmem + static_cast<uint32_t>(256 + h * kHeadDim),
                 tmem + static_cast<uint32_t>(h * kBN), vb, kIdescPV, acc);
        umma_commit(&pv_done[h]);
      }
      __syncwarp();
    };
    auto commit_w = [&](uint64_t* bar) {
      if (elect_one()) umma_commit(bar);
      __syncwarp();
    };
    // S_h is free once the chain's last PV has read P_h from it
    auto s_free = [&](int h) -> bool {
      return pv[h] == 0 || wait_w(&pv_done[h], (pv[h] - 1) & 1);
    };
    // the next K tile into the S of chain h
    auto next_qk = [&](int h, bool last_of_segment) -> bool {
      const uint32_t slot = C % kRing;
      bool ok = wait_w(&ring_full[slot], (C / kRing) & 1);
      ++C;
      uint32_t kb[8];
      kmajor_steps(sR + slot * kTileBytes, kb);
      ok = ok && s_free(h);
      if (!ok) return false;
      tc_fence_after();
      issue_qk(h, kb);
      commit_w(&ring_empty[slot]);
      if (last_of_segment) commit_w(&q_empty[si & 1]);
      return true;
    };
    Segment sg;
    for (int64_t u = u0; u < u_end && !*s_abort;) {
      if (u == u0) sg = first_segment(s_prefix, p.batch, ipr, u, u_end);
      else sg = next_segment(sg, s_prefix, ipr, u_end - u);
      const int n = sg.t1 - sg.t0;
      u += n;
      const int keys = p.ctx_lens[sg.b] + p.tree_lens[sg.b];
      bool ok = kTwo ? wait_w(&q_full[0], si & 1) : wait_w(&q_full[si & 1], (si >> 1) & 1);
      if constexpr (!kTwo) {
        ok = ok && next_qk(0, n == 1);
        if (ok && n > 1) ok = next_qk(1, n == 2);
      } else if (ok) {
        const uint32_t slot = C % kRing;
        ok = wait_w(&ring_full[slot], (C / kRing) & 1);
        ++C;
        uint32_t kb[8];
        kmajor_steps(sR + slot * kTileBytes, kb);
        for (int h = 0; ok && h < 2; ++h) {
          ok = s_free(h);
          if (!ok) break;
          tc_fence_after();
          issue_qk(h, kb);
        }
        if (ok) {
          commit_w(&ring_empty[slot]);
          if (n == 1) commit_w(&q_empty[0]);
        }
      }
      for (int i = 0; ok && i < n; ++i) {
        // the ring slots of this step: V_i, and the K tile kAhead further on
        const bool more = i + (kTwo ? 1 : 2) < n;
        uint32_t ck = C, cv = C;
        if constexpr (kTwo) {
          if (more) ++C;
          cv = C++;
        } else {
          ++C;
        }
        const uint32_t vslot = cv % kRing;
        if (!__all_sync(0xffffffffu,
                        wait_or_abort(&ring_full[vslot], (cv / kRing) & 1, s_abort))) {
          ok = false;
          break;
        }
        const int nvalid = min(kBN, keys - (sg.t0 + i) * kBN);
        if (nvalid < kBN) {  // rows past the last key: zero
          uint8_t* vt = smem + kOffRing + vslot * kTileBytes;
          const int chunks = (kBN - nvalid) * 16;
          for (int q = lane; q < chunks; q += 32) {
            const int r = nvalid + (q >> 4);
            const int c = q & 15;
            *reinterpret_cast<uint4*>(vt + (c >> 3) * kHalf + r * 128 + (c & 7) * 16) =
                make_uint4(0u, 0u, 0u, 0u);
          }
          fence_proxy_async_smem();
        }
        __syncwarp();
        uint32_t vb[8];
        vmn_steps(sR + vslot * kTileBytes, vb);
        if constexpr (kTwo) {
          const uint32_t kslot = ck % kRing;
          uint32_t kb[8];
          kmajor_steps(sR + kslot * kTileBytes, kb);
          if (more) ok = wait_w(&ring_full[kslot], (ck / kRing) & 1);
          for (int h = 0; h < 2 && ok; ++h) {
            ok = wait_w(&p_full[h], pv[h] & 1);
            if (ok && i == 0 && si > 0) ok = wait_w(&o_free[h], (si - 1) & 1);
            if (!ok) break;
            tc_fence_after();
            issue_pv(h, vb, i > 0 ? 1u : 0u);
            ++pv[h];
            if (more) {
              ok = s_free(h);
              if (!ok) break;
              tc_fence_after();
              issue_qk(h, kb);
            }
          }
          if (!ok) break;
          commit_w(&ring_empty[vslot]);
          if (more) {
            commit_w(&ring_empty[kslot]);
            if (i + 2 == n) commit_w(&q_empty[0]);
          }
        } else {
          const int h = i & 1;
          ok = wait_w(&p_full[h], pv[h] & 1);
          if (ok && i == 0 && si > 0) ok = wait_w(&o_free[0], (si - 1) & 1);
          if (!ok) break;
          tc_fence_after();
          issue_pv(h, vb, i > 1 ? 1u : 0u);
          ++pv[h];
          commit_w(&ring_empty[vslot]);
          if (more) ok = next_qk(h, i + 3 == n);
        }
      }
      if (!ok && lane == 0) *s_abort = 1;
      __syncwarp();
      ++si;
      if (!ok) break;
    }
  } else {
    // ---------------------------------------------------- softmax rows ----
    const int grp = (warp - 2) >> 2;
    const int lane_base = 32 * (warp & 3);
    const int row = lane_base + lane;  // of its row tile
    const uint32_t t_lane = tmem + (static_cast<uint32_t>(lane_base) << 16);
    const uint32_t t_s = t_lane + grp * kBN;
    const uint32_t t_o = t_lane + 256 + grp * kHeadDim;
    uint32_t tc[2] = {0, 0};  // key tiles per chain so far
    uint32_t si = 0;
    uint64_t word[2] = {0, 0};  // ancestor words of batch row word_b
    int word_b = -1;
    Segment sg;
    for (int64_t u = u0; u < u_end;) {
      if (__any_sync(0xffffffffu, *s_abort != 0)) break;  // warp-uniform
      if (u == u0) sg = first_segment(s_prefix, p.batch, ipr, u, u_end);
      else sg = next_segment(sg, s_prefix, ipr, u_end - u);
      const int n = sg.t1 - sg.t0;
      const bool whole = n == sg.tiles;
      const bool first_of_cta = u == u0;
      u += n;
      const int kvh = sg.item / p.row_blocks;
      const int rb = sg.item % p.row_blocks;
      const int ctx = p.ctx_lens[sg.b];
      const int r = rb * kMaxRows + (kTwo ? grp * kBM : 0) + row;  // row of the sequence
      const bool mine = r < p.rows;
      const int node = r / p.group;
      const bool warp_live = __any_sync(0xffffffffu, mine);
      uint64_t anc = 0;
      if (warp_live) {
        if (sg.b != word_b) {
          bool bad;
          ancestor_words(p.parents + static_cast<int64_t>(sg.b) * p.n_nodes, p.tree_lens[sg.b],
                         lane, word, bad);
          if (bad && lane == 0) set_dev_err(p.dev_err, PKV_DEV_ERR_BAD_TREE);
          word_b = sg.b;
        }
        const uint64_t w0 = __shfl_sync(0xffffffffu, word[0], node & 31);
        const uint64_t w1 = __shfl_sync(0xffffffffu, word[1], node & 31);
        if (mine) anc = node < 32 ? w0 : w1;
      }
      float m_run = -INFINITY;  // running max, raw score units
      float l_run = 0.f;
      bool ok = true;
      for (int i = kTwo ? 0 : grp; i < n && ok; i += kTwo ? 1 : 2) {
        if (!__all_sync(0xffffffffu, wait_or_abort(&s_full[grp], tc[grp] & 1, s_abort))) {
          ok = false;
          break;
        }
        if (warp_live) {
          tc_fence_after();
          uint32_t sr[128];
          {
            uint32_t (&a)[32] = *reinterpret_cast<uint32_t(*)[32]>(&sr[0]);
            uint32_t (&b)[32] = *reinterpret_cast<uint32_t(*)[32]>(&sr[32]);
            uint32_t (&cc)[32] = *reinterpret_cast<uint32_t(*)[32]>(&sr[64]);
            uint32_t (&d)[32] = *reinterpret_cast<uint32_t(*)[32]>(&sr[96]);
            tmem_ld32(t_s + 0, a);
            tmem_ld32(t_s + 32, b);
            tmem_ld32(t_s + 64, cc);
            tmem_ld32(t_s + 96, d);
            tmem_wait_ld();
          }
          const int off = ctx - (sg.t0 + i) * kBN;  // context columns of this tile
          float mx;
          if (off >= kBN) {
            mx = row_max_full(sr);
          } else {
            float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
            for (int w = 0; w < 4; ++w) {
              const uint32_t vis = anc != 0 ? visible_word(w, off, anc) : 0u;
#pragma unroll
              for (int q = 0; q < 32; ++q) {
                const float v =
                    (vis >> q) & 1u ? __uint_as_float(sr[32 * w + q]) : -INFINITY;
                sr[32 * w + q] = __float_as_uint(v);
                m4[q & 3] = fmaxf(m4[q & 3], v);
              }
            }
            mx = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3]));
          }
          const float m_cand = fmaxf(m_run, mx);
          const bool grow = (m_run == -INFINITY)
                                ? (m_cand != -INFINITY)
                                : ((m_cand - m_run) * p.qscale > kRescaleThreshold);
          const float m_use = grow ? m_cand : m_run;
          const float alpha = grow ? ex2((m_run - m_use) * p.qscale) : 1.f;
          const float neg_m = (m_use == -INFINITY) ? 0.f : -m_use * p.qscale;
          // (S_h of this tile was issued after the chain's previous PV had
          // completed, so O_h is at rest)
          const float psum = softmax_row_to_tmem(sr, p.qscale, neg_m, t_s);
          l_run = l_run * alpha + psum;
          m_run = m_use;
          if (i > (kTwo ? 0 : grp) && __any_sync(0xffffffffu, grow)) {
#pragma unroll
            for (int q = 0; q < kHeadDim; q += 32) {
              uint32_t o[32];
              tmem_ld32(t_o + q, o);
              tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
              tmem_st32(t_o + q, o);
            }
          }
          tmem_wait_st();
          tc_fence_before();
        }
        mbar_arrive(&p_full[grp]);
        ++tc[grp];
      }
      if constexpr (!kTwo) {
        // the other chain's tiles, for the parity of its last PV
        tc[grp ^ 1] += grp == 0 ? n / 2 : (n + 1) / 2;
      }

      // ---- the segment's end: O / l and the LSE, or a partial ----
      const bool live = mine && anc != 0;
      const int head = kvh * p.group + r % p.group;
      const int64_t orow =
          (static_cast<int64_t>(sg.b) * p.n_nodes + node) * p.num_q_heads + head;
      const int prow = kTwo ? grp * kBM + row : row;  // row of the partial slot
      // (a range that starts inside an item or at its start has its first
      // segment's partial in slot 0 of the CTA, its last one's in slot 1)
      float* slot = p.partials + (2 * static_cast<int64_t>(blockIdx.x) + (first_of_cta ? 0 : 1)) *
                                     slot_floats(p.slot_rows);
      float a0 = 1.f, a1 = 0.f;      // weights of the two accumulators (one tile)
      if constexpr (!kTwo) {
        if (grp == 1) {
          // the first warpgroup joins the two chains; this one goes on once
          // the last segment's numbers have been read
          if (ok && si > 0)
            ok = __all_sync(0xffffffffu, wait_or_abort(&o_free[0], (si - 1) & 1, s_abort));
          if (ok) xch[row] = make_float2(m_run, l_run);
          mbar_arrive(x_full);
          ++si;
          if (!ok) {
            set_dev_err(p.dev_err, PKV_DEV_ERR_TIMEOUT);
            *s_abort = 1;
            break;
          }
          continue;
        }
      }
      float m_all = m_run, l_all = l_run;
      if (ok) {
        bool got;
        if constexpr (kTwo) {
          got = wait_or_abort(&pv_done[grp], (tc[grp] - 1) & 1, s_abort);
        } else {
          got = wait_or_abort(x_full, si & 1, s_abort) &&
                wait_or_abort(&pv_done[0], (tc[0] - 1) & 1, s_abort) &&
                (n < 2 || wait_or_abort(&pv_done[1], (tc[1] - 1) & 1, s_abort));
          if (got && n > 1) {
            const float2 c1 = xch[row];
            m_all = fmaxf(m_run, c1.x);
            a0 = m_all == -INFINITY ? 0.f : ex2((m_run - m_all) * p.qscale);
            a1 = m_all == -INFINITY ? 0.f : ex2((c1.x - m_all) * p.qscale);
            l_all = l_run * a0 + c1.y * a1;
          }
        }
        if (!__all_sync(0xffffffffu, got)) ok = false;
      }
      tc_fence_after();
      const bool has = live && ok && l_all != 0.f;  // a NaN among the scores stays one
      const float inv = has ? 1.f / l_all : 0.f;
      if (warp_live && ok) {
#pragma unroll 1
        for (int c = 0; c < kHeadDim; c += 32) {
          uint32_t o[32];
          if constexpr (kTwo) {
            tmem_ld32(t_o + c, o);
            tmem_wait_ld();
          } else {
            tmem_ld32(t_lane + 256 + c, o);
            tmem_wait_ld();
            if (n > 1) {
              uint32_t o1[32];
              tmem_ld32(t_lane + 256 + kHeadDim + c, o1);
              tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < 32; ++e)
                o[e] = __float_as_uint(__uint_as_float(o[e]) * a0 + __uint_as_float(o1[e]) * a1);
            }
          }
          if (mine && whole) {
            uint4* dst = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.out) +
                                                  orow * kHeadDim + c);
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              uint4 w = make_uint4(0u, 0u, 0u, 0u);
              if (has) {
                const int e = 8 * q;
                w.x = pack_bf16x2(__uint_as_float(o[e]) * inv, __uint_as_float(o[e + 1]) * inv);
                w.y = pack_bf16x2(__uint_as_float(o[e + 2]) * inv, __uint_as_float(o[e + 3]) * inv);
                w.z = pack_bf16x2(__uint_as_float(o[e + 4]) * inv, __uint_as_float(o[e + 5]) * inv);
                w.w = pack_bf16x2(__uint_as_float(o[e + 6]) * inv, __uint_as_float(o[e + 7]) * inv);
              }
              dst[q] = w;
            }
          } else if (live) {
#pragma unroll
            for (int e = 0; e < 32; ++e)
              slot[static_cast<int64_t>(c + e) * p.slot_rows + prow] = __uint_as_float(o[e]);
          }
          __syncwarp();  // the next TMEM load is warp-collective
        }
        if (mine) {
          if (whole) {
            p.lse[orow] =
                has ? (m_all * p.qscale + __log2f(l_all)) * 0.69314718055994531f : -INFINITY;
          } else {
            // a row that sees nothing of this segment, or nothing at all, weighs 0
            float* ml = slot + static_cast<int64_t>(kHeadDim) * p.slot_rows;
            ml[prow] = has ? m_all * p.qscale : -INFINITY;
            ml[p.slot_rows + prow] = has ? l_all : 0.f;
          }
        }
      }
      tc_fence_before();
      mbar_arrive(&o_free[grp]);
      ++si;
      if (!ok) {
        set_dev_err(p.dev_err, PKV_DEV_ERR_TIMEOUT);
        *s_abort = 1;
        break;
      }
    }
  }
  if (*s_abort && threadIdx.x == 0) set_dev_err(p.dev_err, PKV_DEV_ERR_TIMEOUT);
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

// -------------------------------------------------------- few query rows --
// R <= 128 rows and short segments leave the 128-row form above waiting on its
// chain (product, softmax, product: ~3 us per key tile and warpgroup however few
// rows are live). Here the products are warp-level MMAs in the decode's
// transposed form, so the rows are the MMAs' columns (eight at a time) and the
// whole softmax stays in a warp's registers: S^T[16 keys x 8 NB rows] = K Q^T,
// O^T[128 x 8 NB] += V^T P^T. A team of T warps (T = 1, 2, 4 for R <= 32, 64, 128;
// a warp holds up to 32 rows) streams its range of 16-key tiles through a ring
// of TMA stages of its own, each warp of the team with its rows of every tile.
// The K/V fragments leave shared memory before the softmax, so a stage goes back
// to TMA early; Q's rows stay in shared memory and are read once per tile.
constexpr int kStreamTile = kDecodeTile;  // 16 keys
constexpr int kStreamWarps = 8;
constexpr int kStreamStages = 16;         // per CTA: 2 T per team
constexpr int kStreamHalf = kStreamTile * 128;
constexpr int kStreamStage = 4 * kStreamHalf;  // K and V of one tile: 8 KB

template <int NB, int T>
struct StreamCfg {
  static constexpr int kTeams = kStreamWarps / T;
  static constexpr int kStages = kStreamStages / kTeams;
  static constexpr int kQRows = T * (NB < 2 ? 2 : NB) * 8;
  static constexpr int kQHalf = kQRows * 128;
  static constexpr int kOffQ = kStreamStages * kStreamStage;
  static constexpr int kOffAnc = kOffQ + kTeams * 2 * kQHalf;          // uint64 [warps][64]
  static constexpr int kOffBar = kOffAnc + kStreamWarps * 64 * 8;
  // per team: full[kStages], empty[kStages], q_full, q_empty
  static constexpr int kBarsPerTeam = 2 * kStages + 2;
  static constexpr int kOffScan = kOffBar + kTeams * kBarsPerTeam * 8;
  static constexpr int kOffPrefix = kOffScan + kStreamWarps * 4;
  static constexpr int kSmemBytes = kOffPrefix + (kTreeMaxBatch + 1) * 4 + 1024;
};

template <int NB, int T>
__global__ void __launch_bounds__(kStreamWarps * 32, 1)
tree_stream_kernel(const __grid_constant__ CUtensorMap qmap,
                   const __grid_constant__ CUtensorMap kmap,
                   const __grid_constant__ CUtensorMap vmap, const TreeParams p) {
  using C = StreamCfg<NB, T>;
  constexpr int S = C::kStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  const int lane = threadIdx.x & 31;
  const int warp = threadIdx.x >> 5;
  const int team = warp / T, wt = warp % T;
  const bool lead = wt == 0;
  uint8_t* stages = smem + team * S * kStreamStage;
  uint8_t* sq = smem + C::kOffQ + team * 2 * C::kQHalf;
  uint64_t* anc = reinterpret_cast<uint64_t*>(smem + C::kOffAnc) + warp * 64;
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::kOffBar) + team * C::kBarsPerTeam;
  uint64_t* empty = full + S;
  uint64_t* q_full = full + 2 * S;
  uint64_t* q_empty = q_full + 1;
  int* s_scan = reinterpret_cast<int*>(smem + C::kOffScan);
  int32_t* s_prefix = reinterpret_cast<int32_t*>(smem + C::kOffPrefix);

  if (lead && lane == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], T);
    }
    mbar_init(q_full, 1);
    mbar_init(q_empty, T);
    fence_barrier_init();
  }
  if (threadIdx.x == 0) {
    tma_prefetch_desc(&qmap);
    tma_prefetch_desc(&kmap);
    tma_prefetch_desc(&vmap);
  }
  pdl_wait_primary();
  pdl_launch_dependents();
  tile_prefix<kStreamTile>(p, s_prefix, s_scan);
  __syncthreads();

  const int ipr = p.items_per_row;
  const int64_t total = static_cast<int64_t>(s_prefix[p.batch]) * ipr;
  const int64_t per = (total + p.workers - 1) / p.workers;
  const int worker = blockIdx.x * C::kTeams + team;
  const int64_t u0 = static_cast<int64_t>(worker) * per;
  const int64_t u_end = u0 + per < total ? u0 + per : total;
  if (u0 >= u_end) return;
  const int count = static_cast<int>(u_end - u0);

  // ---- the team's loads, issued by its first warp ----
  const uint64_t pol = kv_policy(true);
  Segment ps = first_segment(s_prefix, p.batch, ipr, u0, u_end);  // segment being loaded
  int pi = 0;                                                     // its next tile
  int64_t p_left = u_end - u0 - (ps.t1 - ps.t0);                  // tiles behind it
  // Pool rows of 32 tiles of a segment from tile i0 on, one per lane. Unreserved
  // entries (flagged) read page 0 as filler.
  auto tile_rows = [&](const Segment& sg, int i0) -> int {
    const int j = sg.t0 + i0 + lane;
    if (j >= sg.t1) return 0;
    const int l0 = j * kStreamTile;
    const int slot = p.batch_idx[sg.b];
    const int pg = p.page_table[static_cast<int64_t>(slot) * p.max_blocks + l0 / p.page_size];
    if (pg >= 0 && pg < p.num_pages) return pg * p.page_size + l0 % p.page_size;
    set_dev_err(p.dev_err, PKV_DEV_ERR_BAD_PAGE);
    return 0;
  };
  int rows = 0, rows_next = 0;
  Segment ns = ps;  // the segment after ps, where there is one
  auto look_ahead = [&]() {  // entries of the 32 tiles behind the ones at hand
    if (pi + 32 < ps.t1 - ps.t0) {
      rows_next = tile_rows(ps, pi + 32);
    } else if (p_left > 0) {
      ns = next_segment(ps, s_prefix, ipr, p_left);
      rows_next = tile_rows(ns, 0);
    }
  };
  bool bail = false;
  int issued = 0;
  auto issue = [&]() {  // (whole first warp) tile `issued` of the range
    if (pi == ps.t1 - ps.t0) {
      ps = ns;
      pi = 0;
      p_left -= ps.t1 - ps.t0;
    }
    if ((pi & 31) == 0) {
      rows = rows_next;
      look_ahead();
    }
    const int row = __shfl_sync(0xffffffffu, rows, pi & 31);
    const int s = issued % S;
    bool ok = true;
    if (lane == 0) {
      if (T > 1 && issued >= S) ok = mbar_wait_bounded(&empty[s], ((issued / S) - 1) & 1);
      if (ok) {
        uint8_t* st = stages + s * kStreamStage;
        mbar_arrive_expect_tx(&full[s], kStreamStage);
        tma_load_4d_hint(st, &kmap, &full[s], 0, row, 0, ps.item, pol);
        tma_load_4d_hint(st + 2 * kStreamHalf, &vmap, &full[s], 0, row, 0, ps.item, pol);
      }
    }
    if (!__shfl_sync(0xffffffffu, ok, 0)) {
      bail = true;
      return;
    }
    ++issued;
    ++pi;
  };
  // a team of one refills a stage as soon as it has read it; a larger one the
  // stage before, which the other warps have most likely left too
  constexpr int kLag = T > 1 ? 1 : 0;
  if (lead) {
    rows_next = tile_rows(ps, 0);
    for (int k = 0; k < S && k < count; ++k) issue();
  }

  const int g = lane >> 2, t = lane & 3;
  const int mtx = lane >> 3, mrow = lane & 7;
  const int row0 = wt * NB * 8;  // this warp's rows
  const uint32_t sqa = smem_u32(sq);
  auto swz16 = [](int row, int chunk) -> uint32_t {  // [16 rows x 128 dims], two swizzled halves
    return static_cast<uint32_t>((chunk >> 3) * kStreamHalf + row * 128 +
                                 (((chunk & 7) ^ (row & 7)) << 4));
  };
  auto swzq = [](int row, int chunk) -> uint32_t {
    return static_cast<uint32_t>((chunk >> 3) * C::kQHalf + row * 128 +
                                 (((chunk & 7) ^ (row & 7)) << 4));
  };
  int word_b = -1;
  int si = 0;  // segments
  int k = 0;   // tiles of the range
  Segment sg;
  for (int64_t u = u0; u < u_end && !bail; ++si) {
    if (u == u0) sg = first_segment(s_prefix, p.batch, ipr, u, u_end);
    else sg = next_segment(sg, s_prefix, ipr, u_end - u);
    const int n = sg.t1 - sg.t0;
    const bool first_of_range = u == u0;
    u += n;
    if (lead && lane == 0) {
      // Q's rows: free once every warp of the team is done with the last segment
      if (si > 0 && !mbar_wait_bounded(q_empty, (si - 1) & 1)) bail = true;
      if (!bail) {
        mbar_arrive_expect_tx(q_full, 2 * p.rows * 128);
        tma_load_3d(sq, &qmap, q_full, 0, sg.item * p.group, sg.b * p.n_nodes);
        tma_load_3d(sq + C::kQHalf, &qmap, q_full, 64, sg.item * p.group, sg.b * p.n_nodes);
      }
    }
    const int ctx = p.ctx_lens[sg.b];
    const int len = p.tree_lens[sg.b];
    if (sg.b != word_b) {
      uint64_t word[2];
      bool bad;
      ancestor_words(p.parents + static_cast<int64_t>(sg.b) * p.n_nodes, len, lane, word, bad);
      if (bad && lane == 0) set_dev_err(p.dev_err, PKV_DEV_ERR_BAD_TREE);
      __syncwarp();
      anc[lane] = word[0];
      anc[lane + 32] = word[1];
      __syncwarp();
      word_b = sg.b;
    }
    float acc[NB][8][4];
    float m_run[NB][2], l_run[NB][2];
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
      for (int mt = 0; mt < 8; ++mt)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[nb][mt][e] = 0.f;
      m_run[nb][0] = m_run[nb][1] = -INFINITY;
      l_run[nb][0] = l_run[nb][1] = 0.f;
    }
    bail = __any_sync(0xffffffffu, bail);
    if (bail || !__all_sync(0xffffffffu, mbar_wait_bounded(q_full, si & 1))) {
      bail = true;
      break;
    }
    for (int i = 0; i < n; ++i, ++k) {
      const int s = k % S;
      if (!__all_sync(0xffffffffu, mbar_wait_bounded(&full[s], (k / S) & 1))) {
        bail = true;
        break;
      }
      const uint32_t sK = smem_u32(stages + s * kStreamStage);
      const uint32_t sV = sK + 2 * kStreamHalf;

      // ---- S^T = K Q^T: 16 keys x 8 NB rows ----
      float sc[NB][4];
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int e = 0; e < 4; ++e) sc[nb][e] = 0.f;
#pragma unroll
      for (int kk = 0; kk < 8; ++kk) {
        uint32_t kf[4];
        ldsm_x4(sK + swz16((mtx & 1) * 8 + mrow, 2 * kk + (mtx >> 1)), kf[0], kf[1], kf[2], kf[3]);
#pragma unroll
        for (int np = 0; np < (NB + 1) / 2; ++np) {
          uint32_t q0, q1, q2, q3;
          ldsm_x4(sqa + swzq(row0 + (2 * np + (mtx >> 1)) * 8 + mrow, 2 * kk + (mtx & 1)), q0, q1,
                  q2, q3);
          mma_16816(sc[2 * np], kf[0], kf[1], kf[2], kf[3], q0, q1);
          if constexpr (NB > 1) mma_16816(sc[2 * np + 1], kf[0], kf[1], kf[2], kf[3], q2, q3);
        }
      }
      // ---- V's fragments, then the stage goes back ----
      uint32_t vf[8][4];
#pragma unroll
      for (int mt = 0; mt < 8; ++mt)
        ldsm_x4_trans(sV + swz16((mtx >> 1) * 8 + mrow, 2 * mt + (mtx & 1)), vf[mt][0], vf[mt][1],
                      vf[mt][2], vf[mt][3]);
      const int key0 = (sg.t0 + i) * kStreamTile;
      const bool last_tile = i == n - 1;
      fence_proxy_async_smem();
      __syncwarp();
      if (T > 1 && lane == 0) {
        mbar_arrive(&empty[s]);
        if (last_tile) mbar_arrive(q_empty);
      }
      if (T == 1 && last_tile && lane == 0) mbar_arrive(q_empty);
      if (lead && k + 1 >= kLag && issued < count && issued <= k + S - kLag) {
        issue();
        if (bail) break;
      }

      // ---- masks ----
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int e = 0; e < 4; ++e) sc[nb][e] *= p.qscale;
      if (key0 + kStreamTile > ctx) {
        const int r0 = key0 + g - ctx, r1 = r0 + 8;  // node of this lane's keys (< 0: context)
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint64_t a = anc[((row0 + nb * 8 + 2 * t + h) / p.group) & 63];
            const bool v0 = r0 < 0 ? a != 0 : (r0 < 64 && ((a >> r0) & 1ull));
            const bool v1 = r1 < 0 ? a != 0 : (r1 < 64 && ((a >> r1) & 1ull));
            if (!v0) sc[nb][h] = -INFINITY;
            if (!v1) sc[nb][2 + h] = -INFINITY;
          }
        // V of keys past the last node: stale slots may hold any bits
        const int valid = ctx + len - key0;
        auto keep = [&](int key) -> uint32_t {  // two keys of one register
          return (key < valid ? 0x0000ffffu : 0u) | (key + 1 < valid ? 0xffff0000u : 0u);
        };
        if (valid < kStreamTile) {
          const uint32_t k0 = keep(2 * t), k1 = keep(2 * t + 8);
#pragma unroll
          for (int mt = 0; mt < 8; ++mt) {
            vf[mt][0] &= k0;
            vf[mt][1] &= k0;
            vf[mt][2] &= k1;
            vf[mt][3] &= k1;
          }
        }
      }
      // ---- online softmax (log2 units); a row's maximum moves only when it
      // grows by more than kRescaleThreshold ----
      bool moved = false;
      float alpha[NB][2];
      uint32_t pb[NB][2];
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
        float mx0 = fmaxf(sc[nb][0], sc[nb][2]), mx1 = fmaxf(sc[nb][1], sc[nb][3]);
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) {
          mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, o));
          mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, o));
        }
        const float mx[2] = {mx0, mx1};
        float base[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float old = m_run[nb][h];
          const bool grow = old == -INFINITY ? mx[h] != -INFINITY : mx[h] - old > kRescaleThreshold;
          if (grow) m_run[nb][h] = mx[h];
          alpha[nb][h] = grow ? ex2(old - mx[h]) : 1.f;
          moved |= grow && old != -INFINITY;
          base[h] = m_run[nb][h] == -INFINITY ? 0.f : m_run[nb][h];
        }
        const float p0 = ex2(sc[nb][0] - base[0]), p1 = ex2(sc[nb][1] - base[1]);
        const float p2 = ex2(sc[nb][2] - base[0]), p3 = ex2(sc[nb][3] - base[1]);
        l_run[nb][0] = l_run[nb][0] * alpha[nb][0] + (p0 + p2);
        l_run[nb][1] = l_run[nb][1] * alpha[nb][1] + (p1 + p3);
        pb[nb][0] = movmatrix_trans(pack_bf16x2(p0, p1));
        pb[nb][1] = movmatrix_trans(pack_bf16x2(p2, p3));
      }
      if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
          for (int mt = 0; mt < 8; ++mt) {
            acc[nb][mt][0] *= alpha[nb][0];
            acc[nb][mt][1] *= alpha[nb][1];
            acc[nb][mt][2] *= alpha[nb][0];
            acc[nb][mt][3] *= alpha[nb][1];
          }
      }
      // ---- O^T += V^T P^T ----
#pragma unroll
      for (int mt = 0; mt < 8; ++mt)
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
          mma_16816(acc[nb][mt], vf[mt][0], vf[mt][1], vf[mt][2], vf[mt][3], pb[nb][0], pb[nb][1]);
    }
    if (bail) break;

    // ---- the segment's end: O / l and the LSE, or a partial ----
    const bool whole = n == sg.tiles;
    float* slot =
        p.partials + (2 * static_cast<int64_t>(worker) + (first_of_range ? 0 : 1)) *
                         slot_floats(p.slot_rows);
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      bool has[2];
      float inv[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float l = l_run[nb][h];
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
        const int row = row0 + nb * 8 + 2 * t + h;
        const bool mine = row < p.rows;
        has[h] = mine && anc[(row / p.group) & 63] != 0 && l != 0.f;
        inv[h] = has[h] ? 1.f / l : 0.f;
        if (mine && g == 0) {
          if (whole) {
            const int64_t orow =
                (static_cast<int64_t>(sg.b) * p.n_nodes + row / p.group) * p.num_q_heads +
                sg.item * p.group + row % p.group;
            p.lse[orow] =
                has[h] ? (m_run[nb][h] + __log2f(l)) * 0.69314718055994531f : -INFINITY;
          } else {
            float* ml = slot + static_cast<int64_t>(kHeadDim) * p.slot_rows;
            ml[row] = has[h] ? m_run[nb][h] : -INFINITY;
            ml[p.slot_rows + row] = has[h] ? l : 0.f;
          }
        }
      }
      if (whole) {
        // transposed back in registers: row g of the block, two dims per lane
        const int row = row0 + nb * 8 + g;
        __nv_bfloat16* orow =
            static_cast<__nv_bfloat16*>(p.out) +
            ((static_cast<int64_t>(sg.b) * p.n_nodes + row / p.group) * p.num_q_heads +
             sg.item * p.group + row % p.group) *
                kHeadDim +
            2 * t;
#pragma unroll
        for (int mt = 0; mt < 8; ++mt) {
          const uint32_t lo =
              movmatrix_trans(pack_bf16x2(has[0] ? acc[nb][mt][0] * inv[0] : 0.f,
                                          has[1] ? acc[nb][mt][1] * inv[1] : 0.f));
          const uint32_t hi =
              movmatrix_trans(pack_bf16x2(has[0] ? acc[nb][mt][2] * inv[0] : 0.f,
                                          has[1] ? acc[nb][mt][3] * inv[1] : 0.f));
          if (row < p.rows) {
            *reinterpret_cast<uint32_t*>(orow + 16 * mt) = lo;
            *reinterpret_cast<uint32_t*>(orow + 16 * mt + 8) = hi;
          }
        }
      } else {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int row = row0 + nb * 8 + 2 * t + h;
          if (row < p.rows) {
            float* o = slot + static_cast<int64_t>(row) * kHeadDim + g;
#pragma unroll
            for (int mt = 0; mt < 8; ++mt) {
              o[16 * mt] = acc[nb][mt][h];
              o[16 * mt + 8] = acc[nb][mt][2 + h];
            }
          }
        }
      }
    }
  }
  if (bail && lane == 0) {
    set_dev_err(p.dev_err, PKV_DEV_ERR_TIMEOUT);
    // copies still in flight land before the CTA leaves
    if (lead) {
      for (int x = issued > S ? issued - S : 0; x < issued; ++x)
        mbar_wait_bounded(&full[x % S], (x / S) & 1);
      mbar_wait_bounded(q_full, si & 1);
    }
  }
}

// Joins the partials of items cut by range borders, and writes the rows of
// items that attend nothing. grid (items, parts): a CTA takes every parts-th
// block of its item's units; a unit is a row and eight head dims (16 bytes of
// out). merge_split threads share a unit's partials where items have many, each
// taking every merge_split-th, kMergeUnroll at a time. Neighbouring threads read
// neighbouring addresses: along the head dims where a partial's O is row-major
// (kRowMajor, the streaming kernel's), along the rows where it is column-major.
template <bool kRowMajor>
__global__ void __launch_bounds__(kMergeThreads) tree_merge_kernel(const TreeParams p) {
  __shared__ float s_part[kMergeThreads][kMergeCols + 2];
  pdl_wait_primary();
  const int tid = threadIdx.x;
  const int b = blockIdx.x / p.items_per_row, item = blockIdx.x % p.items_per_row;
  const int kvh = item / p.row_blocks, rb = item % p.row_blocks;
  const int before = p.prefix[b], tiles = p.prefix[b + 1] - before;
  const int split = p.merge_split;
  const int per_block = kMergeThreads / split;
  constexpr int kVecs = kHeadDim / kMergeCols;
  const int rows = min(p.rows - rb * kMaxRows, p.slot_rows);  // of this item
  const int units = rows * kVecs;
  int w0 = 0, w1 = 0, first_slot = 0;
  if (tiles > 0) {
    const int64_t total = static_cast<int64_t>(p.prefix[p.batch]) * p.items_per_row;
    const int64_t per = (total + p.workers - 1) / p.workers;
    const int64_t u = static_cast<int64_t>(before) * p.items_per_row +
                      static_cast<int64_t>(item) * tiles;
    w0 = static_cast<int>(u / per);
    w1 = static_cast<int>((u + tiles - 1) / per);
    if (w0 == w1) return;  // one range: written out there
    first_slot = u == w0 * per ? 0 : 1;  // later ranges hold the item in their first slot
  }
  const int share = tid % split;
  const int64_t floats = slot_floats(p.slot_rows);
  for (int block = blockIdx.y; block * per_block < units; block += gridDim.y) {
    const int unit = block * per_block + tid / split;
    const bool mine = unit < units;
    const int prow = kRowMajor ? unit / kVecs : unit % rows;
    const int col = (kRowMajor ? unit % kVecs : unit / rows) * kMergeCols;
    const int r = rb * kMaxRows + prow;  // row of the sequence
    float M = -INFINITY, L = 0.f;
    float acc[kMergeCols];
#pragma unroll
    for (int e = 0; e < kMergeCols; ++e) acc[e] = 0.f;
    if (mine && tiles > 0) {
      for (int w = w0 + share; w <= w1; w += kMergeUnroll * split) {
        float m[kMergeUnroll], l[kMergeUnroll], o[kMergeUnroll][kMergeCols];
#pragma unroll
        for (int k = 0; k < kMergeUnroll; ++k) {
          const int v = w + k * split;
          m[k] = -INFINITY;
          l[k] = 0.f;
          if (v <= w1) {
            const float* s =
                p.partials + (2 * static_cast<int64_t>(v) + (v == w0 ? first_slot : 0)) * floats;
            m[k] = __ldcg(s + static_cast<int64_t>(kHeadDim) * p.slot_rows + prow);
            l[k] = __ldcg(s + static_cast<int64_t>(kHeadDim + 1) * p.slot_rows + prow);
            if constexpr (kRowMajor) {
              const float4* o4 =
                  reinterpret_cast<const float4*>(s + static_cast<int64_t>(prow) * kHeadDim + col);
              const float4 x = __ldcg(o4), y = __ldcg(o4 + 1);
              o[k][0] = x.x, o[k][1] = x.y, o[k][2] = x.z, o[k][3] = x.w;
              o[k][4] = y.x, o[k][5] = y.y, o[k][6] = y.z, o[k][7] = y.w;
            } else {
#pragma unroll
              for (int e = 0; e < kMergeCols; ++e)
                o[k][e] = __ldcg(s + static_cast<int64_t>(col + e) * p.slot_rows + prow);
            }
          }
        }
        float top = M;
#pragma unroll
        for (int k = 0; k < kMergeUnroll; ++k) top = fmaxf(top, m[k]);
        const float keep = top == -INFINITY ? 1.f : ex2(M - top);
        L *= keep;
#pragma unroll
        for (int e = 0; e < kMergeCols; ++e) acc[e] *= keep;
#pragma unroll
        for (int k = 0; k < kMergeUnroll; ++k) {
          // (where the row saw nothing its O may not have been written)
          if (l[k] != 0.f) {
            const float a = ex2(m[k] - top);
            L = fmaf(l[k], a, L);
#pragma unroll
            for (int e = 0; e < kMergeCols; ++e) acc[e] = fmaf(o[k][e], a, acc[e]);
          }
        }
        M = top;
      }
    }
    if (split > 1) {
      __syncthreads();  // the last block's numbers have been read
      s_part[tid][kMergeCols] = M;
      s_part[tid][kMergeCols + 1] = L;
#pragma unroll
      for (int e = 0; e < kMergeCols; ++e) s_part[tid][e] = acc[e];
      __syncthreads();
      if (share == 0) {
        float top = M;
        for (int k = 1; k < split; ++k) top = fmaxf(top, s_part[tid + k][kMergeCols]);
        L = 0.f;
#pragma unroll
        for (int e = 0; e < kMergeCols; ++e) acc[e] = 0.f;
        for (int k = 0; k < split; ++k) {
          const float l = s_part[tid + k][kMergeCols + 1];
          if (l == 0.f) continue;
          const float a = ex2(s_part[tid + k][kMergeCols] - top);
          L = fmaf(l, a, L);
#pragma unroll
          for (int e = 0; e < kMergeCols; ++e) acc[e] = fmaf(s_part[tid + k][e], a, acc[e]);
        }
        M = top;
      }
    }
    if (mine && share == 0) {
      const bool has = L != 0.f;
      const float inv = has ? 1.f / L : 0.f;
      const int64_t orow = (static_cast<int64_t>(b) * p.n_nodes + r / p.group) * p.num_q_heads +
                           kvh * p.group + r % p.group;
      uint4 w;
      w.x = pack_bf16x2(acc[0] * inv, acc[1] * inv);
      w.y = pack_bf16x2(acc[2] * inv, acc[3] * inv);
      w.z = pack_bf16x2(acc[4] * inv, acc[5] * inv);
      w.w = pack_bf16x2(acc[6] * inv, acc[7] * inv);
      *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.out) + orow * kHeadDim + col) = w;
      if (col == 0) p.lse[orow] = has ? (M + __log2f(L)) * 0.69314718055994531f : -INFINITY;
    }
  }
}

namespace {

using namespace prefill_host;

// {D, heads, nodes} view of q; box = 64 head dims x the group's heads x
// `nodes` nodes: rows of one kv head's queries, node by node.
bool encode_tree_q_map(CUtensorMap* map, const void* q, int heads, int64_t nodes, int group,
                       int box_nodes) {
  EncodeTiledFn enc = encode_fn();
  if (enc == nullptr) return false;
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(kHeadDim), static_cast<cuuint64_t>(heads),
                              static_cast<cuuint64_t>(nodes)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(kHeadDim) * 2,
                                 static_cast<cuuint64_t>(heads) * kHeadDim * 2};
  const cuuint32_t box[3] = {64u, static_cast<cuuint32_t>(group), static_cast<cuuint32_t>(box_nodes)};
  const cuuint32_t estr[3] = {1u, 1u, 1u};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(q), dims, strides, box,
             estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool tree_group_ok(int hq, int hkv) {
  if (hq <= 0 || hq % hkv != 0) return false;
  const int g = hq / hkv;
  return g == 1 || g == 2 || g == 4 || g == 8;
}

bool tree_page_size_ok(int ps) { return ps == 16 || ps == 32 || ps == 64 || ps % 128 == 0; }

// Batch rows per launch: equal launches of at most kTreeMaxBatch rows.
int rows_per_launch(int batch) {
  const int launches = (batch + kTreeMaxBatch - 1) / kTreeMaxBatch;
  return launches <= 1 ? batch : (batch + launches - 1) / launches;
}

struct TreeLayout {
  size_t off_partials, total;
};

// Tile prefix, then two partial slots per worker.
TreeLayout tree_layout(int rows, int workers) {
  TreeLayout l;
  l.off_partials = ((kTreeMaxBatch + 1) * 4 + 255) / 256 * 256;
  const size_t part = 2 * static_cast<size_t>(workers) *
                      static_cast<size_t>(slot_floats(rows < kMaxRows ? rows : kMaxRows)) * 4;
  l.total = l.off_partials + (part + 255) / 256 * 256;
  return l;
}

// Which kernel serves R rows: teams of T warps up to 32 T rows, the tcgen05
// forms above.
int team_warps(int rows) { return rows <= 32 ? 1 : 0; }

int tree_workers(int rows, int sms) {
  const int t = team_warps(rows);
  return t ? sms * (kStreamWarps / t) : sms;
}

template <auto kKernel>
cudaError_t launch_tree(int threads, int smem, int sms, const CUtensorMap& qmap,
                        const CUtensorMap& kmap, const CUtensorMap& vmap, const TreeParams& p,
                        int dev, cudaStream_t stream) {
  static std::atomic<bool> attr_set[64] = {};  // per device; host threads may race to set it
  if (!attr_set[dev].load(std::memory_order_acquire)) {
    const cudaError_t e =
        cudaFuncSetAttribute(kKernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    attr_set[dev].store(true, std::memory_order_release);
  }
  cudaError_t e = launch_kernel(kKernel, dim3(sms), dim3(threads), smem, stream,
                                /*programmatic=*/true, qmap, kmap, vmap, p);
  if (e != cudaSuccess) return e;
  // about 16 CTAs per SM in all, and no more per item than it has blocks of units
  const int items = p.batch * p.items_per_row;
  const int per_block = kMergeThreads / p.merge_split;
  const int blocks = (p.slot_rows * (kHeadDim / kMergeCols) + per_block - 1) / per_block;
  const int want = (16 * sms + items - 1) / items;
  return launch_kernel(team_warps(p.rows) ? tree_merge_kernel<true> : tree_merge_kernel<false>,
                       dim3(items, blocks < want ? blocks : want), dim3(kMergeThreads), 0, stream,
                       /*programmatic=*/true, p);
}

template <int NB, int T>
cudaError_t launch_stream(int sms, const CUtensorMap& qmap, const CUtensorMap& kmap,
                          const CUtensorMap& vmap, const TreeParams& p, int dev,
                          cudaStream_t stream) {
  static_assert(StreamCfg<NB, T>::kSmemBytes <= kMaxDynSmem, "shared memory above the limit");
  return launch_tree<tree_stream_kernel<NB, T>>(kStreamWarps * 32, StreamCfg<NB, T>::kSmemBytes,
                                                sms, qmap, kmap, vmap, p, dev, stream);
}

}  // namespace
}  // namespace pkv

extern "C" size_t pkv_tree_workspace_size(const pkv_cache_desc* cache, int batch, int n_nodes,
                                          int num_q_heads) {
  using namespace pkv;
  if (check_cache(cache) != PKV_OK || batch < 0) return 0;
  if (n_nodes < 1 || n_nodes > PKV_MAX_TREE_NODES) return 0;
  if (!tree_group_ok(num_q_heads, cache->num_kv_heads)) return 0;
  int sms = 0;
  if (device_info(&sms) != PKV_OK) return 0;
  const int rows = n_nodes * (num_q_heads / cache->num_kv_heads);
  return tree_layout(rows, tree_workers(rows, sms)).total;
}

extern "C" pkv_status pkv_tree_attention(
    const pkv_cache_desc* cache, const void* k_pool, const void* v_pool, const int32_t* page_table,
    const void* q, int num_q_heads, const int32_t* parents, const int32_t* tree_lens,
    const int32_t* batch_idx, const int32_t* ctx_lens, int batch, int n_nodes, float scale,
    void* out, float* lse, void* workspace, size_t workspace_bytes, int32_t* dev_err,
    cudaStream_t stream) {
  using namespace pkv;
  pkv_status st = check_cache(cache);
  if (st != PKV_OK) return st;
  if (!tree_page_size_ok(cache->page_size)) return PKV_ERR_ARG;
  if (!tree_group_ok(num_q_heads, cache->num_kv_heads)) return PKV_ERR_ARG;
  if (batch < 0 || n_nodes < 1 || n_nodes > PKV_MAX_TREE_NODES) return PKV_ERR_ARG;
  if (!std::isfinite(scale) || !(scale > 0.f)) return PKV_ERR_ARG;
  if (static_cast<int64_t>(batch) * n_nodes > INT32_MAX) return PKV_ERR_ARG;
  if (batch == 0) return PKV_OK;
  if (!k_pool || !v_pool || !page_table || !q || !parents || !tree_lens || !batch_idx ||
      !ctx_lens || !out || !lse)
    return PKV_ERR_ARG;
  if (!aligned(k_pool, 16) || !aligned(v_pool, 16) || !aligned(q, 16) || !aligned(out, 16) ||
      !aligned(lse, 4) || !aligned(page_table, 4) || !aligned(parents, 4) ||
      !aligned(tree_lens, 4) || !aligned(batch_idx, 4) || !aligned(ctx_lens, 4) ||
      !aligned(dev_err, 4))
    return PKV_ERR_ALIGN;
  int sms = 0;
  st = device_info(&sms);
  if (st != PKV_OK) return st;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return PKV_ERR_DEVICE;

  TreeParams p;
  p.group = num_q_heads / cache->num_kv_heads;
  p.rows = n_nodes * p.group;
  p.workers = tree_workers(p.rows, sms);
  const TreeLayout lay = tree_layout(p.rows, p.workers);
  if (workspace == nullptr || workspace_bytes < lay.total) return PKV_ERR_WORKSPACE;
  if (!aligned(workspace, 256)) return PKV_ERR_ALIGN;
  const int team = team_warps(p.rows);
  p.n_nodes = n_nodes;
  p.num_q_heads = num_q_heads;
  p.num_kv_heads = cache->num_kv_heads;
  p.row_blocks = (p.rows + kMaxRows - 1) / kMaxRows;
  p.items_per_row = cache->num_kv_heads * p.row_blocks;
  p.q_box_nodes = kBM / p.group < n_nodes ? kBM / p.group : n_nodes;
  p.page_size = cache->page_size;
  p.num_pages = cache->num_pages;
  p.max_batch = cache->max_batch;
  p.max_blocks = cache->max_blocks;
  p.box_rows = cache->page_size < kBN ? cache->page_size : kBN;
  p.slot_rows = p.rows < kMaxRows ? p.rows : kMaxRows;
  p.qscale = scale * 1.4426950408889634f;
  p.page_table = page_table;
  p.dev_err = dev_err;
  p.prefix = static_cast<int32_t*>(workspace);
  p.partials = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + lay.off_partials);

  CUtensorMap qmap, kmap, vmap;
  if (team != 0) {
    st = encode_pool_map(&kmap, k_pool, cache);
    if (st == PKV_OK) st = encode_pool_map(&vmap, v_pool, cache);
    if (st != PKV_OK) return st;
  } else if (!encode_pool_box_map(&kmap, k_pool, cache, p.box_rows) ||
             !encode_pool_box_map(&vmap, v_pool, cache, p.box_rows)) {
    return PKV_ERR_ARG;
  }
  const int step = rows_per_launch(batch);
  for (int b0 = 0; b0 < batch; b0 += step) {
    p.batch = batch - b0 < step ? batch - b0 : step;
    // partials of an item: about workers / items, one more for the borders
    const int64_t items = static_cast<int64_t>(p.batch) * p.items_per_row;
    p.merge_split = 1;
    while (p.merge_split < 16 && items * p.merge_split * kMergeUnroll < p.workers)
      p.merge_split *= 2;
    const int64_t node0 = static_cast<int64_t>(b0) * n_nodes;
    const int64_t row0 = node0 * num_q_heads;
    const uint8_t* qb = static_cast<const uint8_t*>(q) + row0 * kHeadDim * 2;
    if (!encode_tree_q_map(&qmap, qb, num_q_heads, static_cast<int64_t>(p.batch) * n_nodes, p.group,
                           p.q_box_nodes))
      return PKV_ERR_ARG;
    p.parents = parents + node0;
    p.tree_lens = tree_lens + b0;
    p.batch_idx = batch_idx + b0;
    p.ctx_lens = ctx_lens + b0;
    p.out = static_cast<uint8_t*>(out) + row0 * kHeadDim * 2;
    p.lse = lse + row0;
    cudaError_t e;
    if (team == 1)
      e = p.rows <= 8    ? launch_stream<1, 1>(sms, qmap, kmap, vmap, p, dev, stream)
          : p.rows <= 16 ? launch_stream<2, 1>(sms, qmap, kmap, vmap, p, dev, stream)
                         : launch_stream<4, 1>(sms, qmap, kmap, vmap, p, dev, stream);
    else if (p.rows <= kBM)
      e = launch_tree<tree_attention_kernel<false>>(kThreads, kSmemBytes, sms, qmap, kmap, vmap, p,
                                                    dev, stream);
    else
      e = launch_tree<tree_attention_kernel<true>>(kThreads, kSmemBytes, sms, qmap, kmap, vmap, p,
                                                   dev, stream);
    if (e != cudaSuccess) return record_cuda_status(e);
  }
  return PKV_OK;
}
