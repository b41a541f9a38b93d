// pkv_tree_stream.cu - tree attention of up to 8 query rows of many items, with
// warp-level MMAs.
//
// The products are warp-level MMAs in the decode's transposed form, with the rows as
// their columns: S^T[16 keys x 8 rows] = K Q^T, O^T[128 x 8] += V^T P^T, and a row's whole
// softmax stays in a warp's registers. Each warp streams its range of 16-key tiles
// through a ring of TMA stages of its own, so eight ranges per SM hide one another's
// segment ends, where the warpgroup forms wait. Bound by the K/V stream; with few items by
// their many partials. Measured against the tile form, 8 kv heads, 8 rows: 64 sequences
// of ~768 keys 39.1 / 41.6 us, of ~200 keys 19.6 / 23.6 us, 256 of ~768 keys 138 / 146 us,
// 32 of ~12000 keys 230 / 226 us. At 16 rows (two column blocks) the tile form was
// the faster: 43.3 / 42.2, 24.4 / 24.0, 146 / 147 and 238 / 227 us.
#include "pkv_tree.cuh"

namespace pkv {
namespace tree {

namespace {

constexpr int kStreamTile = kDecodeTile;  // 16 keys
constexpr int kStreamStages = 2;          // per warp
constexpr int kStreamHalf = kStreamTile * 128;
constexpr int kStreamStage = 4 * kStreamHalf;  // K and V of one tile: 8 KB

struct StreamCfg {
  static constexpr int kQRows = 8;
  static constexpr int kQHalf = kQRows * 128;
  static constexpr int kOffQ = kStreamWarps * kStreamStages * kStreamStage;
  static constexpr int kOffAnc = kOffQ + kStreamWarps * 2 * kQHalf;    // uint64 [warps][64]
  static constexpr int kOffBar = kOffAnc + kStreamWarps * 64 * 8;
  static constexpr int kBars = kStreamStages + 1;                      // full, q_full
  static constexpr int kOffScan = kOffBar + kStreamWarps * kBars * 8;
  static constexpr int kOffPrefix = kOffScan + kStreamWarps * 4;
  static constexpr int kSmemBytes = kOffPrefix + (kTreeMaxBatch + 1) * 4 + 1024;
  static_assert(kSmemBytes <= kMaxDynSmem, "rows and shared memory of one warp");
};

}  // namespace

__global__ void __launch_bounds__(kStreamWarps * 32, 1)
tree_stream_kernel(const __grid_constant__ CUtensorMap qmap,
                   const __grid_constant__ CUtensorMap kmap,
                   const __grid_constant__ CUtensorMap vmap, const TreeParams p) {
  using C = StreamCfg;
  constexpr int S = kStreamStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  const int lane = threadIdx.x & 31;
  const int warp = threadIdx.x >> 5;
  uint8_t* stages = smem + warp * S * kStreamStage;
  uint8_t* sq = smem + C::kOffQ + warp * 2 * C::kQHalf;
  uint64_t* anc = reinterpret_cast<uint64_t*>(smem + C::kOffAnc) + warp * 64;
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::kOffBar) + warp * C::kBars;
  uint64_t* q_full = full + S;
  int* s_scan = reinterpret_cast<int*>(smem + C::kOffScan);
  int32_t* s_prefix = reinterpret_cast<int32_t*>(smem + C::kOffPrefix);

  if (lane == 0) {
    for (int s = 0; s < S; ++s) mbar_init(&full[s], 1);
    mbar_init(q_full, 1);
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
  const int64_t per = tiles_per_worker(p, total);
  const int worker = blockIdx.x * kStreamWarps + warp;
  const int64_t u0 = static_cast<int64_t>(worker) * per;
  const int64_t u_end = u0 + per < total ? u0 + per : total;
  if (u0 >= u_end) return;
  const int count = static_cast<int>(u_end - u0);

  // ---- this warp's loads ----
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
  auto issue = [&]() {  // tile `issued` of the range
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
    if (lane == 0) {
      uint8_t* st = stages + s * kStreamStage;
      mbar_arrive_expect_tx(&full[s], kStreamStage);
      tma_load_4d_hint(st, &kmap, &full[s], 0, row, 0, ps.item, pol);
      tma_load_4d_hint(st + 2 * kStreamHalf, &vmap, &full[s], 0, row, 0, ps.item, pol);
    }
    ++issued;
    ++pi;
  };
  rows_next = tile_rows(ps, 0);
  for (int k = 0; k < S && k < count; ++k) issue();

  const int g = lane >> 2, t = lane & 3;
  const int mtx = lane >> 3, mrow = lane & 7;
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
    if (lane == 0) {  // Q's rows: the last segment's have been read (fenced at its end)
      mbar_arrive_expect_tx(q_full, 2 * p.rows * 128);
      tma_load_3d(sq, &qmap, q_full, 0, sg.item * p.group, sg.b * p.n_nodes);
      tma_load_3d(sq + C::kQHalf, &qmap, q_full, 64, sg.item * p.group, sg.b * p.n_nodes);
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
    float acc[8][4];
    float m_run[2], l_run[2];
#pragma unroll
    for (int mt = 0; mt < 8; ++mt)
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[mt][e] = 0.f;
    m_run[0] = m_run[1] = -INFINITY;
    l_run[0] = l_run[1] = 0.f;
    if (!__all_sync(0xffffffffu, mbar_wait_bounded(q_full, si & 1))) {
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

      // ---- S^T = K Q^T: 16 keys x 8 rows ----
      float sc[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) sc[e] = 0.f;
#pragma unroll
      for (int kq = 0; kq < 4; ++kq) {  // 32 dims: two K-steps
        uint32_t qf[4];
        ldsm_x4(sqa + swzq(mrow, 4 * kq + mtx), qf[0], qf[1], qf[2], qf[3]);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          uint32_t kf[4];
          ldsm_x4(sK + swz16((mtx & 1) * 8 + mrow, 4 * kq + 2 * e + (mtx >> 1)), kf[0], kf[1], kf[2],
                  kf[3]);
          mma_16816(sc, kf[0], kf[1], kf[2], kf[3], qf[2 * e], qf[2 * e + 1]);
        }
      }
      // ---- V's fragments, then the stage goes back ----
      uint32_t vf[8][4];
#pragma unroll
      for (int mt = 0; mt < 8; ++mt)
        ldsm_x4_trans(sV + swz16((mtx >> 1) * 8 + mrow, 2 * mt + (mtx & 1)), vf[mt][0], vf[mt][1],
                      vf[mt][2], vf[mt][3]);
      const int key0 = (sg.t0 + i) * kStreamTile;
      fence_proxy_async_smem();
      __syncwarp();
      if (issued < count) issue();

      // ---- masks ----
#pragma unroll
      for (int e = 0; e < 4; ++e) sc[e] *= p.qscale;
      if (key0 + kStreamTile > ctx) {
        const int r0 = key0 + g - ctx, r1 = r0 + 8;  // node of this lane's keys (< 0: context)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint64_t a = anc[((2 * t + h) >> p.group_shift) & 63];
          const bool v0 = r0 < 0 ? a != 0 : (r0 < 64 && ((a >> r0) & 1ull));
          const bool v1 = r1 < 0 ? a != 0 : (r1 < 64 && ((a >> r1) & 1ull));
          if (!v0) sc[h] = -INFINITY;
          if (!v1) sc[2 + h] = -INFINITY;
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
      float alpha[2];
      uint32_t pb[2];
      float mx0 = fmaxf(sc[0], sc[2]), mx1 = fmaxf(sc[1], sc[3]);
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) {
        mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, o));
        mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, o));
      }
      const float mx[2] = {mx0, mx1};
      float base[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float old = m_run[h];
        const bool grow = old == -INFINITY ? mx[h] != -INFINITY : mx[h] - old > kRescaleThreshold;
        if (grow) m_run[h] = mx[h];
        alpha[h] = grow ? ex2(old - mx[h]) : 1.f;
        moved |= grow && old != -INFINITY;
        base[h] = m_run[h] == -INFINITY ? 0.f : m_run[h];
      }
      const float p0 = ex2(sc[0] - base[0]), p1 = ex2(sc[1] - base[1]);
      const float p2 = ex2(sc[2] - base[0]), p3 = ex2(sc[3] - base[1]);
      l_run[0] = l_run[0] * alpha[0] + (p0 + p2);
      l_run[1] = l_run[1] * alpha[1] + (p1 + p3);
      pb[0] = movmatrix_trans(pack_bf16x2(p0, p1));
      pb[1] = movmatrix_trans(pack_bf16x2(p2, p3));
      if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
        for (int mt = 0; mt < 8; ++mt) {
          acc[mt][0] *= alpha[0];
          acc[mt][1] *= alpha[1];
          acc[mt][2] *= alpha[0];
          acc[mt][3] *= alpha[1];
        }
      }
      // ---- O^T += V^T P^T ----
#pragma unroll
      for (int mt = 0; mt < 8; ++mt)
        mma_16816(acc[mt], vf[mt][0], vf[mt][1], vf[mt][2], vf[mt][3], pb[0], pb[1]);
    }
    if (bail) break;

    // ---- the segment's end: O / l and the LSE, or a partial ----
    const bool whole = n == sg.tiles;
    float* slot =
        p.partials + (2 * static_cast<int64_t>(worker) + (first_of_range ? 0 : 1)) *
                         slot_floats(p.slot_rows);
    bool has[2];
    float inv[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float l = l_run[h];
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
      const int row = 2 * t + h;
      const bool mine = row < p.rows;
      has[h] = mine && anc[(row >> p.group_shift) & 63] != 0 && l != 0.f;
      inv[h] = has[h] ? 1.f / l : 0.f;
      if (mine && g == 0) {
        if (whole) {
          const int64_t orow =
              (static_cast<int64_t>(sg.b) * p.n_nodes + (row >> p.group_shift)) * p.num_q_heads +
              sg.item * p.group + (row & (p.group - 1));
          p.lse[orow] =
              has[h] ? (m_run[h] + __log2f(l)) * 0.69314718055994531f : -INFINITY;
        } else {
          float* ml = slot + static_cast<int64_t>(kHeadDim) * p.slot_rows;
          ml[row] = has[h] ? m_run[h] : -INFINITY;
          ml[p.slot_rows + row] = has[h] ? l : 0.f;
        }
      }
    }
    if (whole) {
      // transposed back in registers: row g of the block, two dims per lane
      const int row = g;
      __nv_bfloat16* orow =
          static_cast<__nv_bfloat16*>(p.out) +
          ((static_cast<int64_t>(sg.b) * p.n_nodes + (row >> p.group_shift)) * p.num_q_heads +
           sg.item * p.group + (row & (p.group - 1))) *
              kHeadDim +
          2 * t;
#pragma unroll
      for (int mt = 0; mt < 8; ++mt) {
        const uint32_t lo =
            movmatrix_trans(pack_bf16x2(has[0] ? acc[mt][0] * inv[0] : 0.f,
                                        has[1] ? acc[mt][1] * inv[1] : 0.f));
        const uint32_t hi =
            movmatrix_trans(pack_bf16x2(has[0] ? acc[mt][2] * inv[0] : 0.f,
                                        has[1] ? acc[mt][3] * inv[1] : 0.f));
        if (row < p.rows) {
          *reinterpret_cast<uint32_t*>(orow + 16 * mt) = lo;
          *reinterpret_cast<uint32_t*>(orow + 16 * mt + 8) = hi;
        }
      }
    } else {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int row = 2 * t + h;
        if (row < p.rows) {
          float* o = slot + static_cast<int64_t>(row) * kHeadDim + g;
#pragma unroll
          for (int mt = 0; mt < 8; ++mt) {
            o[16 * mt] = acc[mt][h];
            o[16 * mt + 8] = acc[mt][2 + h];
          }
        }
      }
    }
  }
  if (bail && lane == 0) {
    set_dev_err(p.dev_err, PKV_DEV_ERR_TIMEOUT);
    // copies still in flight land before the CTA leaves
    for (int x = issued > S ? issued - S : 0; x < issued; ++x)
      mbar_wait_bounded(&full[x % S], (x / S) & 1);
    mbar_wait_bounded(q_full, si & 1);
  }
}

cudaError_t launch_stream_form(const CUtensorMap& qmap, const CUtensorMap& kmap,
                               const CUtensorMap& vmap, const TreeParams& p, int sms, int dev,
                               cudaStream_t stream) {
  return launch_form<tree_stream_kernel>(kStreamWarps * 32, StreamCfg::kSmemBytes, sms, qmap, kmap,
                                         vmap, p, dev, stream);
}

}  // namespace tree
}  // namespace pkv
