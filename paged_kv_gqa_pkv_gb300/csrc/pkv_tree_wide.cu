// pkv_tree_wide.cu - tree attention of more than 128 query rows per item, on tcgen05.
//
// Here the tensor work is the larger part (0.55 us per 128-key tile and 128 rows), and
// with the rows as TMEM lanes a softmax needs no reduction across threads: one row per
// thread, two row tiles of 128, one per warpgroup, over the same key tiles; S = Q K^T, P
// over S in tensor memory, O += P V. A key tile is taken in two halves with an S each
// (kHalfKeys), so that a warpgroup's softmax of one half runs while the tensor cores
// have the other half's products: with one S per row tile, product, softmax and product
// took turns (256 rows, 8 x 32768 keys: 251 -> 215 us). There a CTA has a 256 x 128 tile
// every 2.0 us, 66 % of the matrix peak with the rows past the trees counted; what bounds
// it is the chain of a half tile (product, softmax, product, each waiting for the one
// before). On short contexts the ends of segments weigh too: 32 x ~2560 keys take 97 us, of
// which the merge of the cut items' partials, 30 MB from L2, is 13.
#include "pkv_tree.cuh"

namespace pkv {
namespace tree {

namespace {

constexpr int kHalfKeys = 64;

struct WideCfg {
  static constexpr int kThreads = 12 * 32;
  static constexpr int kRing = 5;
  static constexpr int kOffRing = 2 * kTileBytes;  // behind the two Q tiles
  static constexpr int kOffBar = kOffRing + kRing * kTileBytes;
  // q_full, q_empty, ring_full[kRing], ring_empty[kRing], then [row tile][half]:
  // s_full, p_full, pv_done; o_free[row tile]
  static constexpr int kNumBars = 2 + 2 * kRing + 12 + 2;
  static constexpr int kOffMisc = kOffBar + kNumBars * 8;
  static constexpr int kOffPrefix = kOffMisc + 8 + 48;
  static constexpr int kSmemBytes = kOffPrefix + (kTreeMaxBatch + 1) * 4 + 1024;
  static constexpr uint32_t kIdescS = idesc_bf16_f32(128, kHalfKeys, false);
  static_assert(kSmemBytes <= kMaxDynSmem, "shared memory above the opt-in limit");
};

// D (+)= sum over four K-steps of A (tensor memory, 8 columns a step) B.
__device__ __forceinline__ void umma4_ts(uint32_t d, uint32_t a, const uint32_t (&b_lo)[4],
                                         uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p0, p1;\n\t.reg .b64 b<4>;\n\t.reg .b32 t<4>;\n\t"
      "setp.ne.b32 p0, %6, 0;\n\tsetp.eq.b32 p1, %6, %6;\n\t"
      "mov.b64 b0, {%2, %8};\n\tadd.u32 t0, %1, 0;\n\t"
      "mov.b64 b1, {%3, %8};\n\tadd.u32 t1, %1, 8;\n\t"
      "mov.b64 b2, {%4, %8};\n\tadd.u32 t2, %1, 16;\n\t"
      "mov.b64 b3, {%5, %8};\n\tadd.u32 t3, %1, 24;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [t0], b0, %7, p0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [t1], b1, %7, p1;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [t2], b2, %7, p1;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [t3], b3, %7, p1;\n\t}" ::"r"(d),
      "r"(a), "r"(b_lo[0]), "r"(b_lo[1]), "r"(b_lo[2]), "r"(b_lo[3]), "r"(accumulate), "r"(idesc),
      "n"(kDescHi)
      : "memory");
}

// Bits 32 w .. 32 w + 31 of the visible columns of a run of keys whose columns
// [0, off) are context and column off + a is node a (off may be negative).
__device__ __forceinline__ uint32_t visible_word(int w, int off, uint64_t anc) {
  const int s = 32 * w - off;  // bit 0 of this word is node s
  if (s >= 0) return s < 64 ? static_cast<uint32_t>(anc >> s) : 0u;
  if (s > -32) return (static_cast<uint32_t>(anc) << -s) | ((1u << -s) - 1u);
  return 0xffffffffu;
}

// w[q]: 16-byte piece q of this lane's row. Afterwards w[k] is piece lane % 4 of the row
// of lane k of this lane's four, so that four lanes write 64 consecutive bytes of a
// row (a store of 32 rows' pieces takes the memory pipe eight times as long).
__device__ __forceinline__ void transpose4(uint4 (&w)[4], int lane) {
  auto swap = [&](uint4& a, uint4& b, int o) {  // the lane with bit o keeps b and gets the other's
    const bool up = lane & o;
    uint4 s = up ? a : b;
    s.x = __shfl_xor_sync(0xffffffffu, s.x, o);
    s.y = __shfl_xor_sync(0xffffffffu, s.y, o);
    s.z = __shfl_xor_sync(0xffffffffu, s.z, o);
    s.w = __shfl_xor_sync(0xffffffffu, s.w, o);
    if (up) a = s;
    else b = s;
  };
  swap(w[0], w[1], 1);
  swap(w[2], w[3], 1);
  swap(w[0], w[2], 2);
  swap(w[1], w[3], 2);
}

}  // namespace

__global__ void __launch_bounds__(WideCfg::kThreads, 1)
tree_wide_kernel(const __grid_constant__ CUtensorMap qmap,
                 const __grid_constant__ CUtensorMap kmap,
                 const __grid_constant__ CUtensorMap vmap, const TreeParams p) {
  using C = WideCfg;
  constexpr int kRing = C::kRing;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::kOffBar);
  uint64_t* q_full = bars + 0;
  uint64_t* q_empty = bars + 1;
  uint64_t* ring_full = bars + 2;
  uint64_t* ring_empty = ring_full + kRing;
  uint64_t* s_full = ring_empty + kRing;  // [2 h + half]
  uint64_t* p_full = s_full + 4;          // P in tensor memory, O rescaled
  uint64_t* pv_done = s_full + 8;
  uint64_t* o_free = s_full + 12;         // [h]
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::kOffMisc);
  volatile int* s_abort = reinterpret_cast<volatile int*>(smem + C::kOffMisc + 4);
  int* s_scan = reinterpret_cast<int*>(smem + C::kOffMisc + 8);
  int32_t* s_prefix = reinterpret_cast<int32_t*>(smem + C::kOffPrefix);
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int s = 0; s < 2 + 2 * kRing; ++s) mbar_init(&bars[s], 1);
    for (int s = 0; s < 4; ++s) {
      mbar_init(&s_full[s], 1);
      mbar_init(&p_full[s], kGroupThreads);
      mbar_init(&pv_done[s], 1);
    }
    mbar_init(&o_free[0], kGroupThreads);
    mbar_init(&o_free[1], kGroupThreads);
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
  uint8_t* ring = smem + C::kOffRing;
  const int ipr = p.items_per_row;
  const int64_t total = static_cast<int64_t>(s_prefix[p.batch]) * ipr;
  const int64_t per = tiles_per_worker(p, total);
  const int64_t u0 = static_cast<int64_t>(blockIdx.x) * per;
  const int64_t u_end = u0 + per < total ? u0 + per : total;

  if (warp == 0) {
    produce<kRing>(p, qmap, kmap, vmap, s_prefix, u0, u_end, lane, s_abort, smem, kHalf, 2, ring,
                   q_full, q_empty, ring_full, ring_empty);
  } else if (warp < 3) {
    // ------------------------- warp 1: S = Q K^T; warp 2: O (+)= P V ----
    const uint32_t sR = smem_u32(ring);
    uint32_t qd[2][8];
    kmajor_steps(smem_u32(smem), qd[0]);
    kmajor_steps(smem_u32(smem + kTileBytes), qd[1]);
    auto wait_w = [&](uint64_t* bar, uint32_t parity) -> bool {
      return __all_sync(0xffffffffu, wait_or_abort(bar, parity, s_abort));
    };
    uint32_t base = 0;  // ring slots of the segments before
    uint32_t si = 0;    // segments
    uint32_t done = 0;  // key tiles issued
    Segment sg;
    for (int64_t u = u0; u < u_end && !*s_abort;) {
      if (u == u0) sg = first_segment(s_prefix, p.batch, ipr, u, u_end);
      else sg = next_segment(sg, s_prefix, ipr, u_end - u);
      const int n = sg.t1 - sg.t0;
      u += n;
      bool ok = true;
      if (warp == 1) {
        ok = wait_w(q_full, si & 1);
        for (int i = 0; ok && i < n; ++i, ++done) {
          const uint32_t at = base + (i == 0 ? 0 : 2 * i - 1), slot = at % kRing;
          ok = wait_w(&ring_full[slot], (at / kRing) & 1);
          uint32_t kb[8];
          kmajor_steps(sR + slot * kTileBytes, kb);
#pragma unroll
          for (int b = 0; b < 2; ++b) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              // P_h of the tile before sits on this S until its product is done
              if (done > 0) ok = ok && wait_w(&pv_done[2 * h + b], (done - 1) & 1);
              if (!ok) break;
              tc_fence_after();
              if (elect_one()) {
                umma8_ss(tmem + static_cast<uint32_t>(h * kBN + b * kHalfKeys), qd[h], kb,
                         C::kIdescS, 0u);
                umma_commit(&s_full[2 * h + b]);
                if (b == 1 && h == 1) {
                  umma_commit(&ring_empty[slot]);
                  if (i == n - 1) umma_commit(q_empty);
                }
              }
              __syncwarp();
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) kb[e] += (kHalfKeys * 128) >> 4;  // the second half's rows
          }
        }
      } else {
        const int keys = p.ctx_lens[sg.b] + p.tree_lens[sg.b];
        for (int i = 0; ok && i < n; ++i, ++done) {
          const uint32_t at = base + (i + 1 < n ? 2 * i + 2 : n + i), slot = at % kRing;
          ok = wait_w(&ring_full[slot], (at / kRing) & 1);
          const int nvalid = min(kBN, keys - (sg.t0 + i) * kBN);
          if (ok && nvalid < kBN) {  // rows past the last key: zero
            uint8_t* vt = ring + slot * kTileBytes;
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
          vmn_steps(sR + slot * kTileBytes, vb);
#pragma unroll
          for (int b = 0; b < 2; ++b) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              if (i == 0 && b == 0 && si > 0) ok = ok && wait_w(&o_free[h], (si - 1) & 1);
              ok = ok && wait_w(&p_full[2 * h + b], done & 1);
              if (!ok) break;
              tc_fence_after();
              const uint32_t v4[4] = {vb[4 * b], vb[4 * b + 1], vb[4 * b + 2], vb[4 * b + 3]};
              if (elect_one()) {
                umma4_ts(tmem + static_cast<uint32_t>(256 + h * kHeadDim),
                         tmem + static_cast<uint32_t>(h * kBN + b * kHalfKeys), v4, kIdescPV,
                         i > 0 || b > 0 ? 1u : 0u);
                umma_commit(&pv_done[2 * h + b]);
                if (b == 1 && h == 1) umma_commit(&ring_empty[slot]);
              }
              __syncwarp();
            }
          }
        }
      }
      base += 2 * n;
      if (!ok && lane == 0) *s_abort = 1;
      __syncwarp();
      ++si;
      if (!ok) break;
    }
  } else if (warp >= 4) {
    // ---------------------------------------------------- softmax rows ----
    const int grp = (warp - 4) >> 2;
    const int lane_base = 32 * (warp & 3);
    const int row = lane_base + lane;  // of its row tile
    const uint32_t t_lane = tmem + (static_cast<uint32_t>(lane_base) << 16);
    const uint32_t t_o = t_lane + 256 + grp * kHeadDim;
    const unsigned long long qs2 = pack_f32x2(p.qscale, p.qscale);
    uint32_t tc = 0;  // key tiles so far
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
      const bool first_of_range = u == u0;
      u += n;
      const int kvh = sg.item / p.row_blocks;
      const int rb = sg.item % p.row_blocks;
      const int ctx = p.ctx_lens[sg.b];
      const int prow = grp * kBM + row;        // row of the item
      const int r = rb * kMaxRows + prow;      // of the sequence
      const bool mine = r < p.rows;
      const int node = r >> p.group_shift;
      if (sg.b != word_b) {
        bool bad;
        ancestor_words(p.parents + static_cast<int64_t>(sg.b) * p.n_nodes, p.tree_lens[sg.b], lane,
                       word, bad);
        if (bad && lane == 0) set_dev_err(p.dev_err, PKV_DEV_ERR_BAD_TREE);
        word_b = sg.b;
      }
      const uint64_t w0 = __shfl_sync(0xffffffffu, word[0], node & 31);
      const uint64_t w1 = __shfl_sync(0xffffffffu, word[1], node & 31);
      const uint64_t anc = mine ? (node < 32 ? w0 : w1) : 0ull;
      // a warp whose rows are all past the tree leaves its S as P: the products keep
      // rows apart, and nothing of these is used
      const bool warp_live = __any_sync(0xffffffffu, anc != 0);
      float m_run = kNoMax;  // running maximum, log2 units
      float l_run = 0.f;
      bool ok = true;
      for (int j = 0; j < 2 * n && ok; ++j) {  // half tiles
        const int b = j & 1;
        const uint32_t t_s = t_lane + grp * kBN + b * kHalfKeys;
        if (!__all_sync(0xffffffffu, wait_or_abort(&s_full[2 * grp + b], tc & 1, s_abort))) {
          ok = false;
          break;
        }
        if (warp_live) {
          tc_fence_after();
          uint32_t sr[64];
          {
            uint32_t (&x)[32] = *reinterpret_cast<uint32_t(*)[32]>(&sr[0]);
            uint32_t (&y)[32] = *reinterpret_cast<uint32_t(*)[32]>(&sr[32]);
            tmem_ld32(t_s, x);
            tmem_ld32(t_s + 32, y);
            tmem_wait_ld();
          }
          const int off = ctx - (sg.t0 * kBN + j * kHalfKeys);  // context columns
          if (off < kHalfKeys) {
#pragma unroll
            for (int w = 0; w < 2; ++w) {
              const uint32_t vis = anc != 0 ? visible_word(w, off, anc) : 0u;
#pragma unroll
              for (int q = 0; q < 32; ++q)
                if (!((vis >> q) & 1u)) sr[32 * w + q] = 0xff800000u;  // -inf
            }
          }
          float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int q = 0; q < 64; q += 8)
#pragma unroll
            for (int k = 0; k < 4; ++k)
              m4[k] = fmax3(m4[k], __uint_as_float(sr[q + 2 * k]), __uint_as_float(sr[q + 2 * k + 1]));
          const float mx = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3])) * p.qscale;
          const bool grow = mx > m_run + kRescaleThreshold || (m_run == kNoMax && mx > m_run);
          float alpha = 1.f;
          if (grow) {
            alpha = m_run == kNoMax ? 0.f : ex2(m_run - mx);
            m_run = mx;
          }
          const unsigned long long nm2 = pack_f32x2(-m_run, -m_run);
          unsigned long long acc0 = 0ull, acc1 = 0ull;
#pragma unroll
          for (int c = 0; c < 2; ++c) {  // 32 keys -> 16 columns
            uint32_t pk[16];
#pragma unroll
            for (int q = 0; q < 16; ++q) {
              float x0, x1;
              unpack_f32x2(ffma2(pack_f32x2(__uint_as_float(sr[32 * c + 2 * q]),
                                            __uint_as_float(sr[32 * c + 2 * q + 1])),
                                 qs2, nm2),
                           x0, x1);
              x0 = ex2(x0);
              x1 = ex2(x1);
              if (q & 1) acc1 = fadd2(acc1, pack_f32x2(x0, x1));
              else acc0 = fadd2(acc0, pack_f32x2(x0, x1));
              pk[q] = pack_bf16x2(x0, x1);
            }
            tmem_st16(t_s + 16 * c, pk);
          }
          float s0, s1, s2, s3;
          unpack_f32x2(acc0, s0, s1);
          unpack_f32x2(acc1, s2, s3);
          l_run = l_run * alpha + ((s0 + s1) + (s2 + s3));
          if (j > 0 && __any_sync(0xffffffffu, grow)) {
            // O at rest: the product of the half before is done
            const bool got =
                wait_or_abort(&pv_done[2 * grp + (b ^ 1)], (b ? tc : tc - 1) & 1, s_abort);
            if (!__all_sync(0xffffffffu, got)) ok = false;
            tc_fence_after();
#pragma unroll 1
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
        mbar_arrive(&p_full[2 * grp + b]);
        tc += b;
      }

      // ---- the segment's end: O / l and the LSE, or a partial ----
      if (ok) {
        const bool got = wait_or_abort(&pv_done[2 * grp], (tc - 1) & 1, s_abort) &&
                         wait_or_abort(&pv_done[2 * grp + 1], (tc - 1) & 1, s_abort);
        ok = __all_sync(0xffffffffu, got);
      }
      tc_fence_after();
      const bool live = mine && anc != 0;
      const bool has = live && ok && l_run != 0.f;  // (a NaN among the scores stays one)
      const float inv = has ? 1.f / l_run : 0.f;
      const int64_t row00 = static_cast<int64_t>(sg.b) * p.n_nodes * p.num_q_heads + kvh * p.group;
      auto row_of = [&](int x) -> int64_t {  // of the output
        return row00 + (x >> p.group_shift) * p.num_q_heads + (x & (p.group - 1));
      };
      float* slot = p.partials +
                    (2 * static_cast<int64_t>(blockIdx.x) + (first_of_range ? 0 : 1)) *
                        slot_floats(kMaxRows);
      if (ok && (warp_live || whole)) {
#pragma unroll 1
        for (int c = 0; c < kHeadDim; c += 32) {
          uint32_t o[32];
          tmem_ld32(t_o + c, o);
          tmem_wait_ld();
          if (whole) {
            uint4 w[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              w[q] = make_uint4(0u, 0u, 0u, 0u);
              if (has) {
                const int e = 8 * q;
                w[q].x = pack_bf16x2(__uint_as_float(o[e]) * inv, __uint_as_float(o[e + 1]) * inv);
                w[q].y = pack_bf16x2(__uint_as_float(o[e + 2]) * inv, __uint_as_float(o[e + 3]) * inv);
                w[q].z = pack_bf16x2(__uint_as_float(o[e + 4]) * inv, __uint_as_float(o[e + 5]) * inv);
                w[q].w = pack_bf16x2(__uint_as_float(o[e + 6]) * inv, __uint_as_float(o[e + 7]) * inv);
              }
            }
            transpose4(w, lane);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const int rk = r - (lane & 3) + k;
              if (rk < p.rows)
                *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.out) +
                                          row_of(rk) * kHeadDim + c + 8 * (lane & 3)) = w[k];
            }
          } else if (live) {
#pragma unroll
            for (int e = 0; e < 32; ++e)
              slot[(c + e) * kMaxRows + prow] = __uint_as_float(o[e]);
          }
          __syncwarp();  // the next TMEM load is warp-collective
        }
      }
      if (ok && mine) {
        if (whole) {
          p.lse[row_of(r)] = has ? (m_run + __log2f(l_run)) * 0.69314718055994531f : -INFINITY;
        } else {
          float* ml = slot + kHeadDim * kMaxRows;
          ml[prow] = has ? m_run : -INFINITY;
          ml[kMaxRows + prow] = has ? l_run : 0.f;
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

cudaError_t launch_wide_form(const CUtensorMap& qmap, const CUtensorMap& kmap,
                             const CUtensorMap& vmap, const TreeParams& p, int sms, int dev,
                             cudaStream_t stream) {
  return launch_form<tree_wide_kernel>(WideCfg::kThreads, WideCfg::kSmemBytes, sms, qmap, kmap, vmap,
                                       p, dev, stream);
}

}  // namespace tree
}  // namespace pkv
