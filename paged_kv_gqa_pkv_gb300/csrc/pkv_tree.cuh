// pkv_tree.cuh - what the kernels of pkv_tree_attention share: the work list, the
// ancestor words, the loading warp and the layout of the partial results.
//
// For one sequence and one kv head the queries are R = nodes x group rows (row r
// is node r / G, query head kvh * G + r % G), all over the same keys: the committed
// context, which every row sees whole, and the tree's own nodes, where a row sees
// its ancestors. So the keys stream once per (sequence, kv head) however large the
// tree is (up to 256 rows; above that the rows are blocks of 256, which read the
// keys once each: a worker takes a sequence's second block after the first, when the
// other workers' keys have passed through L2. 32 sequences of ~2560 keys at 8 kv heads
// and 384 rows read 715 MB from DRAM, twice the keys' bytes).
//
// Work list: all (sequence, kv head, row block) items' key tiles in one list, cut
// into equal ranges, one per worker (a CTA, a warpgroup or a warp); a range's pieces
// of items are its segments. An item inside one range is written out by its worker.
// An item cut by range borders leaves one partial (unnormalised O, running maximum
// and sum) per worker, at most two per worker (of its first and its last segment),
// and the merge kernel joins them.
//
// Masks: a node's ancestors-or-self are one 64-bit word, built per warp from the
// parents by pointer doubling (six rounds of shuffles). A key tile that ends inside
// the context needs no mask; in the last ones a row's visible keys are the context's
// and its word shifted to the tree's place. V rows past the last node are zeroed
// before the product (stale slots may hold any bits, and 0 * NaN is not 0).
//
// Numbers: S, the maxima and sums and O are fp32. P is rounded to bf16, the type of V,
// which the MMAs take with it: 2^-8 of each weight at most, and the sums take the
// unrounded weights. Against 64 bits the output's error is 2.3e-3 of its size, of which
// its own rounding to bf16 is 1.7e-3.
#pragma once

#include <atomic>

#include "pkv_prefill_common.cuh"

namespace pkv {
namespace tree {

using namespace prefill_detail;

constexpr int kMaxRows = 256;          // query rows of an item
constexpr int kStreamWarps = 8;        // workers per CTA of the streaming form
constexpr int kTreeMaxBatch = 128;     // batch rows per launch (tile prefix in shared memory)

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
  int group;         // a power of two
  int group_shift;
  int rows;          // n_nodes * group
  int row_blocks;    // items per (sequence, kv head)
  int items_per_row; // num_kv_heads * row_blocks
  int q_box_nodes;   // nodes of one Q box: min(128 / group, n_nodes)
  int page_size;
  int num_pages;
  int max_batch;
  int max_blocks;
  int box_rows;      // rows of one K/V box: min(page_size, 128)
  int workers;       // ranges of the tile list (CTAs, chains or warps)
  int min_tiles;     // shortest range of a worker
  int slot_rows;     // rows of a partial slot
  int merge_split;   // merge threads that share an item's partials (a power of two)
  float qscale;      // scale * log2(e)
};

// A partial slot: O [rows][128], or [128][rows] in the wide form, then m and l [rows],
// 16-byte aligned. The wide form's has kMaxRows rows whatever an item's: with its
// columns a constant apart the merge spends one instruction per load.
__host__ __device__ constexpr int slot_rows(int rows) { return rows > kBM ? kMaxRows : rows; }
__host__ __device__ inline int64_t slot_floats(int rows) {
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

// a / b for a >= 0, b > 0: 64-bit division takes ~100 cycles more.
__device__ __forceinline__ int64_t divide(int64_t a, int b) {
  return a <= 0x7fffffff ? static_cast<int>(a) / b : a / b;
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

// The segment that starts at tile u of the list (below u_end). Warp-collective: the
// rows that end at or before u are counted 32 at a time (a binary search's dependent
// reads took half a microsecond of every worker's start).
__device__ __forceinline__ Segment first_segment(const int32_t* prefix, int batch, int ipr,
                                                 int64_t u, int64_t u_end) {
  const int lane = threadIdx.x & 31;
  int lo = 0;
  for (int k = 0; k < batch; k += 32)
    lo += __popc(__ballot_sync(0xffffffffu, k + lane < batch &&
                                                static_cast<int64_t>(prefix[k + lane + 1]) * ipr <= u));
  Segment s;
  s.b = lo;
  s.tiles = prefix[lo + 1] - prefix[lo];
  const int64_t r = u - static_cast<int64_t>(prefix[lo]) * ipr;
  s.item = static_cast<int>(divide(r, s.tiles));
  s.t0 = static_cast<int>(r - static_cast<int64_t>(s.item) * s.tiles);
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

// Tiles per batch row and their prefix in s_prefix[0 .. batch], by every CTA (the
// caller owes a barrier behind it; s_scan: an int per warp). CTA 0 also leaves the
// prefix to the merge.
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

// Length of a worker's range of the tile list: an equal share, but not so short
// that a partial costs more than the tiles it stands for.
__device__ __forceinline__ int64_t tiles_per_worker(const TreeParams& p, int64_t total) {
  const int64_t share = divide(total + p.workers - 1, p.workers);
  return share > p.min_tiles ? share : p.min_tiles;
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

// The loading warp of a worker: Q of each segment and its K/V tiles, in the order
// K_0, then K_{i+1} (if any) and V_i.
template <int kRing>
__device__ __forceinline__ void produce(const TreeParams& p, const CUtensorMap& qmap,
                                        const CUtensorMap& kmap, const CUtensorMap& vmap,
                                        const int32_t* s_prefix, int64_t u0, int64_t u_end,
                                        int lane, volatile int* s_abort, uint8_t* sq, int q_half,
                                        int q_tiles, uint8_t* ring, uint64_t* q_full,
                                        uint64_t* q_empty, uint64_t* ring_full,
                                        uint64_t* ring_empty) {
  const int ipr = p.items_per_row;
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
    // Q of this segment: its place is free after the last segment's last S; its
    // tiles of 128 rows are q_tiles apart (one tile of all rows, or two of 128)
    auto load_q = [&]() -> bool {
      bool good = true;
      if (lane == 0) {
        good = si == 0 || wait_or_abort(q_empty, (si - 1) & 1, s_abort);
        if (good) {
          mbar_arrive_expect_tx(q_full, q_tiles * 2 * p.q_box_nodes * p.group * 128);
          for (int h = 0; h < q_tiles; ++h) {
            const int node0 = sg.b * p.n_nodes + (rb * q_tiles + h) * p.q_box_nodes;
            uint8_t* qd = sq + h * 2 * q_half;
            tma_load_3d(qd, &qmap, q_full, 0, kvh * p.group, node0);
            tma_load_3d(qd + q_half, &qmap, q_full, 64, kvh * p.group, node0);
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
      const uint32_t s = L % kRing;
      bool good = true;
      if (lane == 0) {
        good = L < kRing || wait_or_abort(&ring_empty[s], ((L / kRing) - 1) & 1, s_abort);
        if (good) mbar_arrive_expect_tx(&ring_full[s], kTileBytes);
      }
      good = __shfl_sync(0xffffffffu, good, 0);
      if (!good) return false;
      uint8_t* dst = ring + s * kTileBytes;
#pragma unroll 1
      for (int k = 0; k < nsub; ++k) {
        const int at = __shfl_sync(0xffffffffu, have, (lane0 + k) & 31);
        if (lane == 0) {
          tma_load_4d_hint(dst + k * R * 128, map, &ring_full[s], 0, at, 0, kvh, pol);
          tma_load_4d_hint(dst + kHalf + k * R * 128, map, &ring_full[s], 0, at, 1, kvh, pol);
        }
      }
      ++L;
      return true;
    };
    // ring order = the issuers' order: K_0, then K_{i+1} (if any) and V_i; Q
    // goes out behind the first K tile, whose place is free earlier. (One copy of
    // the code for all of them: the kernels' loops have to fit the instruction cache.)
    bool ok = true;
    for (int k = 0; ok && k < 2 * n; ++k) {
      const bool is_k = k == 0 || ((k & 1) && k + 1 < 2 * n);
      const int i = is_k ? (k + 1) >> 1 : k + 1 < 2 * n ? (k >> 1) - 1 : n - 1;
      // the tile before the first V of chunk c: chunk c - 1 is done with after it, and
      // its place goes to chunk c + 1 when V enters chunk c
      if (!is_k && i > 0 && i % tpc == 0) {
        const int c = i / tpc;
        const int more = (c + 1) * tpc < n ? chunk_rows(sg, c + 1) : 0;
        if (c & 1) rows[0] = more;
        else rows[1] = more;
      }
      ok = load(is_k ? &kmap : &vmap, i);
      if (k == 0) ok = ok && load_q();
    }
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
    if (si > 0) mbar_wait_bounded(q_full, (si - 1) & 1);
  }
}

constexpr float kNoMax = -3.0e38f;  // running maximum of a row that has seen nothing

// Launches one of the attention kernels on every SM.
template <auto kKernel>
cudaError_t launch_form(int threads, int smem, int sms, const CUtensorMap& qmap,
                        const CUtensorMap& kmap, const CUtensorMap& vmap, const TreeParams& p,
                        int dev, cudaStream_t stream) {
  // the shared-memory opt-in, once per device; host threads may race to set it
  static std::atomic<bool> attr_set[64] = {};
  if (!attr_set[dev].load(std::memory_order_acquire)) {
    const cudaError_t e =
        cudaFuncSetAttribute(kKernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    attr_set[dev].store(true, std::memory_order_release);
  }
  return launch_kernel(kKernel, dim3(sms), dim3(threads), smem, stream, /*programmatic=*/true, qmap,
                       kmap, vmap, p);
}

// The forms' launches (pkv_tree_tile.cu, pkv_tree_wide.cu, pkv_tree_stream.cu).
cudaError_t launch_tile_form(const CUtensorMap& qmap, const CUtensorMap& kmap,
                             const CUtensorMap& vmap, const TreeParams& p, int sms, int dev,
                             cudaStream_t stream);
cudaError_t launch_wide_form(const CUtensorMap& qmap, const CUtensorMap& kmap,
                             const CUtensorMap& vmap, const TreeParams& p, int sms, int dev,
                             cudaStream_t stream);
cudaError_t launch_stream_form(const CUtensorMap& qmap, const CUtensorMap& kmap,
                               const CUtensorMap& vmap, const TreeParams& p, int sms, int dev,
                               cudaStream_t stream);

}  // namespace tree
}  // namespace pkv
