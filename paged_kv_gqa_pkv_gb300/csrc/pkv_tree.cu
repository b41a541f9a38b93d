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
constexpr int kTreeMaxBatch = 256;     // batch rows per launch (tile prefix in shared memory)
constexpr int kRing = 5;               // K/V tile slots
constexpr int kMergeCols = 8;          // head dims per merge CTA

// shared memory: Q (two tiles; the one-tile form leaves the second one unused
// but for the exchange of the running maxima and sums), the K/V ring, barriers
constexpr int kOffQ = 0;
constexpr int kOffRing = kOffQ + 2 * kTileBytes;
constexpr int kOffBar = kOffRing + kRing * kTileBytes;
// q_full, q_empty, ring_full[kRing], ring_empty[kRing], s_full[2], p_full[2],
// pv_done[2], o_free[2], x_full
constexpr int kNumBars = 2 + 2 * kRing + 9;
constexpr int kOffMisc = kOffBar + kNumBars * 8;  // tmem slot, abort flag, scan
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
  int workers;       // CTAs of the attention kernel
  int slot_rows;     // rows of a partial slot: min(rows, kMaxRows)
  float qscale;      // scale * log2(e)
};

__host__ __device__ __forceinline__ int64_t slot_floats(int rows) {
  return static_cast<int64_t>(rows) * (kHeadDim + 2);
}

// Key tiles of batch row b (0: nothing to attend), and the error it raises.
__device__ __forceinline__ int tree_row_tiles(const TreeParams& p, int b, int* err) {
  const int slot = p.batch_idx[b];
  *err = 0;
  if (slot == 0) return 0;
  const int ctx = p.ctx_lens[b], n = p.tree_lens[b];
  if (slot < 0 || slot >= p.max_batch) *err = PKV_DEV_ERR_BAD_SLOT;
  else if (n < 0 || n > p.n_nodes) *err = PKV_DEV_ERR_BAD_TREE;
  else if (ctx < 0 || static_cast<int64_t>(ctx) + n >
                          static_cast<int64_t>(p.max_blocks) * p.page_size)
    *err = PKV_DEV_ERR_BAD_POS;
  if (*err || n == 0) return 0;
  return static_cast<int>((static_cast<int64_t>(ctx) + n + kBN - 1) / kBN);
}

// One CTA's piece of an item.
struct Segment {
  int b, item;       // batch row, item within the row
  int t0, t1;        // key tiles [t0, t1) of `tiles`
  int tiles;
};

__device__ __forceinline__ Segment locate_segment(const int32_t* prefix, int batch, int ipr,
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
  const int64_t left = u_end - u;
  s.t1 = left < s.tiles - s.t0 ? s.t0 + static_cast<int>(left) : s.tiles;
  return s;
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
  uint64_t* q_full = bars + 0;
  uint64_t* q_empty = bars + 1;
  uint64_t* ring_full = bars + 2;           // [kRing]
  uint64_t* ring_empty = bars + 2 + kRing;  // [kRing]
  uint64_t* s_full = bars + 2 + 2 * kRing;  // [2]
  uint64_t* p_full = s_full + 2;            // [2]
  uint64_t* pv_done = s_full + 4;           // [2]
  uint64_t* o_free = s_full + 6;            // [2]; one tile: [0] stands for both
  uint64_t* x_full = s_full + 8;            // one tile: maxima and sums exchanged
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + kOffMisc);
  volatile int* s_abort = reinterpret_cast<volatile int*>(smem + kOffMisc + 4);
  int* s_scan = reinterpret_cast<int*>(smem + kOffMisc + 8);
  int32_t* s_prefix = reinterpret_cast<int32_t*>(smem + kOffPrefix);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    mbar_init(q_full, 1);
    mbar_init(q_empty, 1);
    for (int s = 0; s < kRing; ++s) {
      mbar_init(&ring_full[s], 1);
      mbar_init(&ring_empty[s], 1);
    }
    for (int h = 0; h < 2; ++h) {
      mbar_init(&s_full[h], 1);
      mbar_init(&p_full[h], kGroupThreads);
      mbar_init(&pv_done[h], 1);
      mbar_init(&o_free[h], kTwo ? kGroupThreads : 2 * kGroupThreads);
    }
    mbar_init(x_full, 2 * kGroupThreads);
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

  // ---- key tiles per batch row and their prefix (every CTA) ----
  {
    int tiles = 0;
    if (threadIdx.x < kTreeMaxBatch && static_cast<int>(threadIdx.x) < p.batch) {
      int err;
      tiles = tree_row_tiles(p, threadIdx.x, &err);
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
    if (threadIdx.x < kTreeMaxBatch) s_prefix[threadIdx.x + 1] = before + incl;
    if (threadIdx.x == 0) s_prefix[0] = 0;
  }
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  if (blockIdx.x == 0)
    for (int i = threadIdx.x; i <= p.batch; i += kThreads) p.prefix[i] = s_prefix[i];

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
    const int nsub = kBN / R;
    for (int64_t u = u0; u < u_end && !*s_abort;) {
      const Segment sg = locate_segment(s_prefix, p.batch, ipr, u, u_end);
      u += sg.t1 - sg.t0;
      const int kvh = sg.item / p.row_blocks;
      const int rb = sg.item % p.row_blocks;
      const int slot = p.batch_idx[sg.b];
      const int last = p.ctx_lens[sg.b] + p.tree_lens[sg.b] - 1;  // last key
      bool ok = true;
      if (lane == 0) {
        ok = si == 0 || wait_or_abort(q_empty, (si - 1) & 1, s_abort);
        if (ok) {
          constexpr int kTiles = kTwo ? 2 : 1;
          mbar_arrive_expect_tx(q_full, kTiles * 2 * p.q_box_nodes * p.group * 128);
          for (int h = 0; h < kTiles; ++h) {
            const int node0 = sg.b * p.n_nodes + (rb * 2 + h) * (kBM / p.group);
            uint8_t* qd = smem + kOffQ + h * kTileBytes;
            tma_load_3d(qd, &qmap, q_full, 0, kvh * p.group, node0);
            tma_load_3d(qd + kHalf, &qmap, q_full, 64, kvh * p.group, node0);
          }
        }
      }
      ok = __shfl_sync(0xffffffffu, ok, 0);
      // One 128-key tile through the page table: lane k < nsub finds the pool
      // row of box k; boxes past the last key, and unreserved entries
      // (flagged), read page 0 as filler.
      auto load = [&](const CUtensorMap* map, int j) -> bool {
        int rowk = 0;
        bool bad = false;
        if (lane < nsub) {
          const int l0 = j * kBN + lane * R;
          if (l0 <= last) {
            const int pg = p.page_table[static_cast<int64_t>(slot) * p.max_blocks + l0 / p.page_size];
            if (pg < 0 || pg >= p.num_pages) bad = true;
            else rowk = pg * p.page_size + l0 % p.page_size;
          }
        }
        if (__any_sync(0xffffffffu, bad) && lane == 0) set_dev_err(p.dev_err, PKV_DEV_ERR_BAD_PAGE);
        int rows[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) rows[k] = __shfl_sync(0xffffffffu, rowk, k);
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
                tma_load_4d(dst + k * R * 128, map, &ring_full[s], 0, rows[k], 0, kvh);
                tma_load_4d(dst + kHalf + k * R * 128, map, &ring_full[s], 0, rows[k], 1, kvh);
              }
            }
          }
        }
        ++L;
        return __shfl_sync(0xffffffffu, good, 0);
      };
      // ring order = the issuer's order: the K tiles run kAhead tiles before
      // the V tiles (one per chain in flight)
      constexpr int kAhead = kTwo ? 1 : 2;
      int jk = sg.t0;
      for (int a = 0; ok && a < kAhead && jk < sg.t1; ++a, ++jk) ok = load(&kmap, jk);
      for (int j = sg.t0; ok && j < sg.t1; ++j) {
        if constexpr (kTwo) {
          if (jk < sg.t1) ok = load(&kmap, jk++);
          ok = ok && load(&vmap, j);
        } else {
          ok = load(&vmap, j);
          if (ok && jk < sg.t1) ok = load(&kmap, jk++);
        }
      }
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
    uint32_t qd[2][8];
    kmajor_steps(smem_u32(smem + kOffQ), qd[0]);
    kmajor_steps(smem_u32(smem + kOffQ + (kTwo ? kTileBytes : 0)), qd[1]);
    auto wait_w = [&](uint64_t* bar, uint32_t parity) -> bool {
      return __shfl_sync(0xffffffffu, wait_or_abort(bar, parity, s_abort) ? 1 : 0, 0) != 0;
    };
    auto issue_qk = [&](int h, const uint32_t (&kb)[8]) {  // S_h = Q K^T
      if (elect_one()) {
        umma8_ss(tmem + static_cast<uint32_t>(h * kBN), qd[h], kb, kIdescQK, 0u);
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
    // the next K tile into the S of chain h (kTwo: of both)
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
      if (last_of_segment) commit_w(q_empty);
      return true;
    };
    for (int64_t u = u0; u < u_end && !*s_abort;) {
      const Segment sg = locate_segment(s_prefix, p.batch, ipr, u, u_end);
      const int n = sg.t1 - sg.t0;
      u += n;
      const int keys = p.ctx_lens[sg.b] + p.tree_lens[sg.b];
      bool ok = wait_w(q_full, si & 1);
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
          if (n == 1) commit_w(q_empty);
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
            if (i + 2 == n) commit_w(q_empty);
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
    float2* xch = reinterpret_cast<float2*>(smem + kOffQ + kTileBytes);  // [2][2][128], one tile
    uint32_t tc[2] = {0, 0};  // key tiles per chain so far
    uint32_t si = 0;
    for (int64_t u = u0; u < u_end;) {
      if (__any_sync(0xffffffffu, *s_abort != 0)) break;  // warp-uniform
      const Segment sg = locate_segment(s_prefix, p.batch, ipr, u, u_end);
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
        uint64_t word[2];
        bool bad;
        ancestor_words(p.parents + static_cast<int64_t>(sg.b) * p.n_nodes, p.tree_lens[sg.b], lane,
                       word, bad);
        if (bad && lane == 0 && sg.item == 0) set_dev_err(p.dev_err, PKV_DEV_ERR_BAD_TREE);
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
      float m_all = m_run, l_all = l_run;
      if (ok) {
        bool got;
        if constexpr (kTwo) {
          got = wait_or_abort(&pv_done[grp], (tc[grp] - 1) & 1, s_abort);
        } else {
          float2* x = xch + (si & 1) * 256;
          x[grp * 128 + row] = make_float2(m_run, l_run);
          mbar_arrive(x_full);
          got = wait_or_abort(x_full, si & 1, s_abort) &&
                wait_or_abort(&pv_done[0], (tc[0] - 1) & 1, s_abort) &&
                (n < 2 || wait_or_abort(&pv_done[1], (tc[1] - 1) & 1, s_abort));
          if (got) {
            const float2 c0 = x[row], c1 = n < 2 ? make_float2(-INFINITY, 0.f) : x[128 + row];
            m_all = fmaxf(c0.x, c1.x);
            a0 = m_all == -INFINITY ? 0.f : ex2((c0.x - m_all) * p.qscale);
            a1 = m_all == -INFINITY ? 0.f : ex2((c1.x - m_all) * p.qscale);
            l_all = c0.y * a0 + c1.y * a1;
          }
        }
        if (!__all_sync(0xffffffffu, got)) ok = false;
      }
      tc_fence_after();
      const bool has = live && ok && l_all != 0.f;  // a NaN among the scores stays one
      const float inv = has ? 1.f / l_all : 0.f;
      if (warp_live && ok) {
        // one tile: each warpgroup writes half of the head dims
        constexpr int kCols = kTwo ? kHeadDim : kHeadDim / 2;
        const int col0 = kTwo ? 0 : grp * kCols;
#pragma unroll 1
        for (int c = col0; c < col0 + kCols; c += 32) {
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
        if (mine && (kTwo || grp == 0)) {
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
      mbar_arrive(&o_free[kTwo ? grp : 0]);
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

// Joins the partials of items cut by range borders, and writes the rows of
// sequences that attend nothing. grid (workers + batch, 128 / kMergeCols): CTA
// (w, c) for w < workers takes the item that its range's end cuts, if it is the
// item's first range; CTA (workers + b, c) the sequence b without keys. A thread
// is a row, its columns the CTA's.
__global__ void __launch_bounds__(kMaxRows) tree_merge_kernel(const TreeParams p) {
  __shared__ int32_t s_prefix[kTreeMaxBatch + 1];
  pdl_wait_primary();
  const int c0 = blockIdx.y * kMergeCols;
  const int tid = threadIdx.x;
  if (static_cast<int>(blockIdx.x) >= p.workers) {
    const int b = blockIdx.x - p.workers;
    if (p.prefix[b + 1] != p.prefix[b]) return;
    const int64_t rows = static_cast<int64_t>(p.n_nodes) * p.num_q_heads;
    for (int64_t i = tid; i < rows; i += kMaxRows) {
      const int64_t orow = b * rows + i;
      *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.out) + orow * kHeadDim + c0) =
          make_uint4(0u, 0u, 0u, 0u);
      if (blockIdx.y == 0) p.lse[orow] = -INFINITY;
    }
    return;
  }
  for (int i = tid; i <= p.batch; i += kMaxRows) s_prefix[i] = p.prefix[i];
  __syncthreads();
  const int ipr = p.items_per_row;
  const int64_t total = static_cast<int64_t>(s_prefix[p.batch]) * ipr;
  const int64_t per = (total + p.workers - 1) / p.workers;
  const int64_t cut = (static_cast<int64_t>(blockIdx.x) + 1) * per;  // first tile of the next range
  if (cut >= total) return;
  const Segment sg = locate_segment(s_prefix, p.batch, ipr, cut, cut + 1);
  if (sg.t0 == 0) return;  // the border lies between items
  const int64_t first_tile = cut - sg.t0;
  const int w0 = static_cast<int>(first_tile / per);
  if (w0 != static_cast<int>(blockIdx.x)) return;  // an earlier range's CTA joins it
  const int w1 = static_cast<int>((first_tile + sg.tiles - 1) / per);
  const int kvh = sg.item / p.row_blocks;
  const int rb = sg.item % p.row_blocks;
  const int r = rb * kMaxRows + tid;
  if (tid >= p.slot_rows || r >= p.rows) return;
  const int64_t floats = slot_floats(p.slot_rows);
  // the item's segment in range w: w's first one unless the item starts inside w
  const bool starts_inside = first_tile != static_cast<int64_t>(w0) * per;
  auto seg = [&](int w) -> const float* {
    return p.partials + (2 * static_cast<int64_t>(w) + (w == w0 && starts_inside ? 1 : 0)) * floats;
  };
  const int64_t ml = static_cast<int64_t>(kHeadDim) * p.slot_rows + tid;
  float M = -INFINITY;
  for (int w = w0; w <= w1; ++w) M = fmaxf(M, __ldcg(seg(w) + ml));
  float acc[kMergeCols];
#pragma unroll
  for (int e = 0; e < kMergeCols; ++e) acc[e] = 0.f;
  float L = 0.f;
  for (int w = w0; w <= w1; ++w) {
    const float* s = seg(w);
    const float l = __ldcg(s + ml + p.slot_rows);
    if (l == 0.f) continue;  // the row saw nothing there (its O may not be written)
    const float a = ex2(__ldcg(s + ml) - M);
    L = fmaf(l, a, L);
#pragma unroll
    for (int e = 0; e < kMergeCols; ++e)
      acc[e] = fmaf(__ldcg(s + static_cast<int64_t>(c0 + e) * p.slot_rows + tid), a, acc[e]);
  }
  const bool has = L != 0.f;
  const float inv = has ? 1.f / L : 0.f;
  const int node = r / p.group;
  const int64_t orow = (static_cast<int64_t>(sg.b) * p.n_nodes + node) * p.num_q_heads +
                       kvh * p.group + r % p.group;
  uint4 w;
  w.x = pack_bf16x2(acc[0] * inv, acc[1] * inv);
  w.y = pack_bf16x2(acc[2] * inv, acc[3] * inv);
  w.z = pack_bf16x2(acc[4] * inv, acc[5] * inv);
  w.w = pack_bf16x2(acc[6] * inv, acc[7] * inv);
  *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.out) + orow * kHeadDim + c0) = w;
  if (blockIdx.y == 0)
    p.lse[orow] = has ? (M + __log2f(L)) * 0.69314718055994531f : -INFINITY;
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

// Tile prefix, then two partial slots per CTA.
TreeLayout tree_layout(int rows, int workers) {
  TreeLayout l;
  l.off_partials = ((kTreeMaxBatch + 1) * 4 + 255) / 256 * 256;
  const size_t part = 2 * static_cast<size_t>(workers) *
                      static_cast<size_t>(slot_floats(rows < kMaxRows ? rows : kMaxRows)) * 4;
  l.total = l.off_partials + (part + 255) / 256 * 256;
  return l;
}

template <bool kTwo>
cudaError_t launch_tree(const CUtensorMap& qmap, const CUtensorMap& kmap, const CUtensorMap& vmap,
                        const TreeParams& p, int dev, cudaStream_t stream) {
  static std::atomic<bool> attr_set[64] = {};  // per device; host threads may race to set it
  if (!attr_set[dev].load(std::memory_order_acquire)) {
    const cudaError_t e = cudaFuncSetAttribute(
        tree_attention_kernel<kTwo>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
    if (e != cudaSuccess) return e;
    attr_set[dev].store(true, std::memory_order_release);
  }
  cudaError_t e = launch_kernel(tree_attention_kernel<kTwo>, dim3(p.workers), dim3(kThreads),
                                kSmemBytes, stream, /*programmatic=*/true, qmap, kmap, vmap, p);
  if (e != cudaSuccess) return e;
  return launch_kernel(tree_merge_kernel, dim3(p.workers + p.batch, kHeadDim / kMergeCols),
                       dim3(kMaxRows), 0, stream, /*programmatic=*/true, p);
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
  return tree_layout(n_nodes * (num_q_heads / cache->num_kv_heads), sms).total;
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
  const TreeLayout lay = tree_layout(p.rows, sms);
  if (workspace == nullptr || workspace_bytes < lay.total) return PKV_ERR_WORKSPACE;
  if (!aligned(workspace, 256)) return PKV_ERR_ALIGN;
  const bool two = p.rows > kBM;
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
  p.workers = sms;
  p.slot_rows = p.rows < kMaxRows ? p.rows : kMaxRows;
  p.qscale = scale * 1.4426950408889634f;
  p.page_table = page_table;
  p.dev_err = dev_err;
  p.prefix = static_cast<int32_t*>(workspace);
  p.partials = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + lay.off_partials);

  CUtensorMap qmap, kmap, vmap;
  if (!encode_pool_box_map(&kmap, k_pool, cache, p.box_rows) ||
      !encode_pool_box_map(&vmap, v_pool, cache, p.box_rows))
    return PKV_ERR_ARG;
  const int step = rows_per_launch(batch);
  for (int b0 = 0; b0 < batch; b0 += step) {
    p.batch = batch - b0 < step ? batch - b0 : step;
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
    const cudaError_t e = two ? launch_tree<true>(qmap, kmap, vmap, p, dev, stream)
                              : launch_tree<false>(qmap, kmap, vmap, p, dev, stream);
    if (e != cudaSuccess) return record_cuda_status(e);
  }
  return PKV_OK;
}
