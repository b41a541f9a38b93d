// pkv_tree_tile.cu - tree attention of up to 128 query rows per item, on tcgen05.
//
// Both products are transposed: the 128 keys of a tile (then the 128 head dims) are
// the MMAs' M, the query rows their N, so few rows cost few tensor cycles: S^T = K Q^T
// and O^T += V^T P^T, with P^T in shared memory (the B operand), not over S: the next S
// is issued as soon as this one has been read, and a tile's P V product runs beside
// the next softmax. (With the rows as M and P over S a key tile took a chain of
// product, softmax, product, ~3.3 us however few rows were live.)
//
// Softmax: a thread holds four keys of two neighbouring rows in each eight. A row's
// maximum would take a reduction over the warpgroup, so it moves only when some score
// passes it by more than kRescaleThreshold (log2 units): the common tile costs one
// barrier that carries that question. P is at most 2^kRescaleThreshold, and its
// rounding to bf16 is relative, so nothing is lost by a maximum that lags.
//
// Bound by the K/V stream where contexts are long (8 x 32768 keys: 163 us at 32 rows, 169
// us at 128, 96 / 93 % of the copy bandwidth); where they are short by the ends of
// segments, in which a warpgroup joins its sums, writes its rows and takes the next
// first maximum (64 sequences x 8 kv heads of ~768 keys: 44 us at 32 rows, 68 us at
// 128). Up to 64 rows a CTA is two workers, so that one's segment ends fall into the
// other's tiles.
//
// Every step stands in the code once, rolled into loops: five roles share an SM's
// instruction cache, and what is fetched anew waits behind the K/V stream. With
// first steps and second attempts written out, warps had no instruction for a third of
// their stalls, and the short contexts took 54 and 81 us, the long ones 169 and 176.
#include "pkv_tree.cuh"

namespace pkv {
namespace tree {

namespace {

// Shared memory and tensor memory of one form. A chain is a softmax warpgroup
// with kCols of the MMAs' columns (query rows). kShare chains share a worker: an
// item's rows are split over them and they see the same key tiles. With kShare =
// 1 a CTA is two workers, each with its own range of the list and its own ring.
template <int kCols, int kShare>
struct TileCfg {
  static constexpr int kRows = kCols * kShare;          // the MMAs' N
  static constexpr int kWorkers = kShare == 1 ? 2 : 1;  // per CTA
  static constexpr int kChains = kShare * kWorkers;
  static constexpr int kThreads = 128 + 128 * kChains;
  static constexpr int kOperHalf = kRows * 128;         // [rows x 64] of Q or P
  static constexpr int kOper = 2 * kOperHalf;
  static constexpr int kOffP = kWorkers * kOper;        // Q of the workers, then P
  static constexpr int kOffRing = 2 * kWorkers * kOper;
  // 32 KB K/V slots per ring, as many as fit
  static constexpr int kRing = (224 * 1024 - kOffRing) / kTileBytes / kWorkers;
  static constexpr int kOffBar = kOffRing + kWorkers * kRing * kTileBytes;
  // per worker: q_full, q_empty, s_full, s_free, p_full, pv_done, o_free, then
  // ring_full and ring_empty
  static constexpr int kBars = 7 + 2 * kRing;
  static constexpr int kOffWords = kOffBar + kWorkers * kBars * 8;  // uint64 [workers][64]
  static constexpr int kOffMisc = kOffWords + kWorkers * 64 * 8;    // tmem slot, abort, scan
  static constexpr int kOffPrefix = kOffMisc + 8 + (kThreads / 32) * 4;
  static constexpr int kSmemBytes = kOffPrefix + (kTreeMaxBatch + 1) * 4 + 1024;
  static constexpr uint32_t kTmemCols = 2 * kChains * kCols;        // O of the chains, then S
  // S^T = K Q^T: both K-major; O^T = V^T P^T: V is dim-contiguous (A transposed)
  static constexpr uint32_t kIdescS = idesc_bf16_f32(128, kRows, false);
  static constexpr uint32_t kIdescO = idesc_bf16_f32(128, kRows, false) | (1u << 15);
  static_assert(kSmemBytes <= kMaxDynSmem, "shared memory above the opt-in limit");
};

// 16 lanes x 8 NX columns as accumulator fragments: lane 4 g + t holds, for each
// eight columns, (row g, columns 2t, 2t + 1) and (row g + 8, the same columns).
template <int NX>
__device__ __forceinline__ void tmem_ld_frag(uint32_t taddr, float (&r)[4 * NX]);
template <>
__device__ __forceinline__ void tmem_ld_frag<4>(uint32_t taddr, float (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,"
      "%15}, [%16];"
      : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]),
        "=f"(r[7]), "=f"(r[8]), "=f"(r[9]), "=f"(r[10]), "=f"(r[11]), "=f"(r[12]), "=f"(r[13]),
        "=f"(r[14]), "=f"(r[15])
      : "r"(taddr));
}
template <>
__device__ __forceinline__ void tmem_ld_frag<8>(uint32_t taddr, float (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,"
      "%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]),
        "=f"(r[7]), "=f"(r[8]), "=f"(r[9]), "=f"(r[10]), "=f"(r[11]), "=f"(r[12]), "=f"(r[13]),
        "=f"(r[14]), "=f"(r[15]), "=f"(r[16]), "=f"(r[17]), "=f"(r[18]), "=f"(r[19]), "=f"(r[20]),
        "=f"(r[21]), "=f"(r[22]), "=f"(r[23]), "=f"(r[24]), "=f"(r[25]), "=f"(r[26]), "=f"(r[27]),
        "=f"(r[28]), "=f"(r[29]), "=f"(r[30]), "=f"(r[31])
      : "r"(taddr));
}

// 16 consecutive fp32 columns of this thread's TMEM lane.
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,"
      "%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}

// Four 8 x 8 bf16 fragments to shared memory, each transposed; lane 8 i + r gives
// the address of row r of matrix i.
__device__ __forceinline__ void stsm_x4_trans(uint32_t addr, uint32_t a, uint32_t b, uint32_t c,
                                              uint32_t d) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1,%2,%3,%4};" ::"r"(addr),
               "r"(a), "r"(b), "r"(c), "r"(d)
               : "memory");
}

// Barrier of `threads` threads that also returns whether any of them passed true.
__device__ __forceinline__ bool named_bar_or(int id, int threads, bool v) {
  int any;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %3, 0;\n\t"
      "barrier.cta.red.or.pred q, %1, %2, p;\n\tselp.b32 %0, 1, 0, q;\n\t}"
      : "=r"(any)
      : "r"(id), "r"(threads), "r"(v ? 1 : 0)
      : "memory");
  return any != 0;
}

}  // namespace

// Warps 0-3 load and issue the tensor instructions, each four after them are a
// chain's softmax warpgroup. Waits are bounded; after one has given up the loops run
// on without waiting, and a worker's warpgroups leave at a segment's end, on a decision
// taken at a barrier of them all.
template <int kCols, int kShare>
__global__ void __launch_bounds__(TileCfg<kCols, kShare>::kThreads, 1)
tree_tile_kernel(const __grid_constant__ CUtensorMap qmap,
                 const __grid_constant__ CUtensorMap kmap,
                 const __grid_constant__ CUtensorMap vmap, const TreeParams p) {
  using C = TileCfg<kCols, kShare>;
  constexpr int kRing = C::kRing;
  constexpr bool kSingle = kShare == 1;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::kOffBar);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::kOffMisc);
  volatile int* s_abort = reinterpret_cast<volatile int*>(smem + C::kOffMisc + 4);
  int* s_scan = reinterpret_cast<int*>(smem + C::kOffMisc + 8);
  int32_t* s_prefix = reinterpret_cast<int32_t*>(smem + C::kOffPrefix);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;

  // the chain that this warp serves, of the worker `own` of the CTA
  const int chain = warp < 4 ? (kSingle ? warp & 1 : 0) : (warp - 4) >> 2;
  const int own = kSingle ? chain : 0;
  uint64_t* q_full = bars + own * C::kBars;
  uint64_t* q_empty = q_full + 1;
  uint64_t* s_full = q_full + 2;
  uint64_t* s_free = q_full + 3;   // S has been read
  uint64_t* p_full = q_full + 4;   // P in shared memory, O rescaled
  uint64_t* pv_done = q_full + 5;
  uint64_t* o_free = q_full + 6;   // the segment's O has been read
  uint64_t* ring_full = q_full + 7;
  uint64_t* ring_empty = ring_full + kRing;

  if (threadIdx.x == 0) {
    for (int w = 0; w < C::kWorkers; ++w) {
      uint64_t* x = bars + w * C::kBars;
      for (int k = 0; k < C::kBars; ++k)
        mbar_init(x + k, k == 3 || k == 4 || k == 6 ? kShare * kGroupThreads : 1);
    }
    *s_abort = 0;
    fence_barrier_init();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&qmap);
    tma_prefetch_desc(&kmap);
    tma_prefetch_desc(&vmap);
  }
  if (warp == 2) tmem_alloc(tmem_slot, C::kTmemCols);
  // Q's rows past the item's, which no load writes, are 0: the scores of what an earlier
  // kernel left there could send every tile through the slow path (33 of 64 rows, 64 x
  // 768 keys: 72 us after a call with large q, 63 after others)
  const int spare = (C::kRows - p.rows) * 8;  // 16-byte pieces of each half
  for (int i = threadIdx.x; i < C::kWorkers * 2 * spare; i += C::kThreads)
    *reinterpret_cast<uint4*>(smem + i / spare * C::kOperHalf + p.rows * 128 + i % spare * 16) =
        make_uint4(0u, 0u, 0u, 0u);
  fence_proxy_async_smem();
  pdl_wait_primary();
  pdl_launch_dependents();  // the merge waits for this grid before it reads anything
  tile_prefix<kBN>(p, s_prefix, s_scan);
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  uint8_t* ring = smem + C::kOffRing + own * kRing * kTileBytes;
  const int ipr = p.items_per_row;
  const int64_t total = static_cast<int64_t>(s_prefix[p.batch]) * ipr;
  const int64_t per = tiles_per_worker(p, total);
  const int worker = blockIdx.x * C::kWorkers + own;
  const int64_t u0 = static_cast<int64_t>(worker) * per;
  const int64_t u_end = u0 + per < total ? u0 + per : total;

  if (warp < C::kWorkers) {
    produce<kRing>(p, qmap, kmap, vmap, s_prefix, u0, u_end, lane, s_abort, smem + own * C::kOper,
                   C::kOperHalf, 1, ring, q_full, q_empty, ring_full, ring_empty);
  } else if (warp >= 2 && warp < 4) {
    // ----------------------------------------------------- MMA issuers ----
    // S^T = K Q^T and O^T (+)= V^T P^T. A worker of one chain has one warp for both,
    // S_{i+1} before O_i; else warp 2 issues the S and warp 3 the O products (waits
    // and issue take a warp ~0.6 us per product).
    const uint32_t sR = smem_u32(ring);
    // low descriptor words of the eight K-steps of a [rows x 128] K-major operand
    auto oper_steps = [&](uint32_t base, uint32_t (&lo)[8]) {
      const uint32_t d = desc_lo(base, 0);
#pragma unroll
      for (int kk = 0; kk < 8; ++kk) lo[kk] = d + (((kk >> 2) * C::kOperHalf + (kk & 3) * 32) >> 4);
    };
    auto wait_w = [&](uint64_t* bar, uint32_t parity) -> bool {
      return __all_sync(0xffffffffu, wait_or_abort(bar, parity, s_abort));
    };
    uint32_t base = 0;           // ring slots of the segments before
    uint32_t si = 0;             // segments
    uint32_t s_n = 0, o_n = 0;   // S and O products issued
    uint32_t qb[8], pb[8];
    oper_steps(smem_u32(smem + own * C::kOper), qb);
    oper_steps(smem_u32(smem + C::kOffP + own * C::kOper), pb);
    const uint32_t t_o = tmem + own * kCols, t_s = t_o + C::kChains * kCols;
    Segment sg;
    for (int64_t u = u0; u < u_end && !*s_abort;) {
      if (u == u0) sg = first_segment(s_prefix, p.batch, ipr, u, u_end);
      else sg = next_segment(sg, s_prefix, ipr, u_end - u);
      const int n = sg.t1 - sg.t0;
      u += n;
      const int keys = p.ctx_lens[sg.b] + p.tree_lens[sg.b];
      auto issue_s = [&](int i) -> bool {
        if (i == 0 && !wait_w(q_full, si & 1)) return false;
        const uint32_t at = base + (i == 0 ? 0 : 2 * i - 1), slot = at % kRing;
        if (!wait_w(&ring_full[slot], (at / kRing) & 1)) return false;
        uint32_t ka[8];
        kmajor_steps(sR + slot * kTileBytes, ka);
        // once the last S has been read
        if (s_n > 0 && !wait_w(s_free, (s_n - 1) & 1)) return false;
        tc_fence_after();
        if (elect_one()) {
          umma8_ss(t_s, ka, qb, C::kIdescS, 0u);
          umma_commit(s_full);
          umma_commit(&ring_empty[slot]);
          if (i == n - 1) umma_commit(q_empty);
        }
        __syncwarp();
        ++s_n;
        return true;
      };
      auto issue_o = [&](int i) -> bool {
        const uint32_t at = base + (i + 1 < n ? 2 * i + 2 : n + i), slot = at % kRing;
        if (!wait_w(&ring_full[slot], (at / kRing) & 1)) return false;
        const int nvalid = min(kBN, keys - (sg.t0 + i) * kBN);
        if (nvalid < kBN) {  // rows past the last key: zero
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
        uint32_t va[8];
        vmn_steps(sR + slot * kTileBytes, va);
        if (i == 0 && si > 0 && !wait_w(o_free, (si - 1) & 1)) return false;
        if (!wait_w(p_full, o_n & 1)) return false;
        tc_fence_after();
        if (elect_one()) {
          umma8_ss(t_o, va, pb, C::kIdescO, i > 0 ? 1u : 0u);
          umma_commit(pv_done);
          umma_commit(&ring_empty[slot]);
        }
        __syncwarp();
        ++o_n;
        return true;
      };
      bool ok = true;
      if constexpr (!kSingle) {
        for (int i = 0; ok && i < n; ++i) ok = warp == 2 ? issue_s(i) : issue_o(i);
      } else {
        for (int i = -1; ok && i < n; ++i) {
          if (i + 1 < n) ok = issue_s(i + 1);
          if (i >= 0) ok = ok && issue_o(i);
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
    constexpr int kNX = kCols / 8;
    const int quad = warp & 3;         // TMEM lanes (keys, then head dims) 32 quad ..
    const int g = lane >> 2, t = lane & 3;
    const uint32_t t_lane = tmem + (static_cast<uint32_t>(32 * quad) << 16);
    const uint32_t t_o = t_lane + chain * kCols;
    const uint32_t t_s = t_o + C::kChains * kCols;
    const int col0 = kSingle ? 0 : chain * kCols;  // this chain's first row of the operands
    uint8_t* sP = smem + C::kOffP + own * C::kOper;
    uint8_t* sMine = sP + col0 * 128;  // this chain's rows of P, first half: also scratch
    const uint32_t sPa = smem_u32(sP);
    uint64_t* words = reinterpret_cast<uint64_t*>(smem + C::kOffWords) + own * 64;
    const int bar = 1 + chain;           // this warpgroup's barrier, the worker's
    const int worker_bar = kSingle ? bar : 1 + C::kChains;
    const int tid = 32 * quad + lane;    // thread of the warpgroup
    const unsigned long long qs2 = pack_f32x2(p.qscale, p.qscale);
    uint32_t tc = 0;                     // this chain's key tiles so far
    uint32_t si = 0;
    int word_b = -1;                     // batch row of the ancestor words
    bool failed = false;                 // a wait of this thread gave up
    Segment sg;
    for (int64_t u = u0; u < u_end;) {
      if (u == u0) sg = first_segment(s_prefix, p.batch, ipr, u, u_end);
      else sg = next_segment(sg, s_prefix, ipr, u_end - u);
      const int n = sg.t1 - sg.t0;
      const bool whole = n == sg.tiles;
      const bool first_of_range = u == u0;
      u += n;
      const int kvh = sg.item / p.row_blocks;
      const int rb = sg.item % p.row_blocks;
      const int ctx = p.ctx_lens[sg.b];
      const int r0 = rb * kMaxRows + col0;  // row of this chain's column 0
      if (sg.b != word_b) {
        // (the last segment's end is a barrier of all of the worker's readers)
        uint64_t word[2];
        bool bad;
        ancestor_words(p.parents + static_cast<int64_t>(sg.b) * p.n_nodes, p.tree_lens[sg.b], lane,
                       word, bad);
        if (bad && lane == 0) set_dev_err(p.dev_err, PKV_DEV_ERR_BAD_TREE);
        if (quad == 0 && (kSingle || chain == 0)) {
          words[lane] = word[0];
          words[lane + 32] = word[1];
        }
        named_bar_sync(worker_bar, kShare * kGroupThreads);
        word_b = sg.b;
      }
      // the ancestor word of column c's row, 0: no live row
      auto column_word = [&](int c) -> uint64_t {
        const int r = r0 + c;
        return r < p.rows ? words[r >> p.group_shift] : 0ull;
      };
      // running maxima (log2 units) and sums of this thread's rows 8 c + 2 t + d
      float m_run[kNX][2], l_run[kNX][2];
#pragma unroll
      for (int c = 0; c < kNX; ++c) {
        m_run[c][0] = m_run[c][1] = kNoMax;
        l_run[c][0] = l_run[c][1] = 0.f;
      }
      for (int i = 0; i < n; ++i) {
        failed |= !wait_or_abort(s_full, tc & 1, s_abort);
        tc_fence_after();
        const int off = ctx - (sg.t0 + i) * kBN;  // context keys of this tile
        float x[2][4 * kNX];  // [16-key half][fragment]
        auto load = [&]() {
          tmem_ld_frag<kNX>(t_s, x[0]);
          tmem_ld_frag<kNX>(t_s + (16u << 16), x[1]);
          tmem_wait_ld();
          if (off < kBN) {
            // this lane's keys are 32 quad + g + 8 j: bits 8 j of a row's word (with 32
            // ones below it: the context) from bit `from` on
            const int from = max(32 * quad + g - off + 32, 0);
            const int part = from >> 5, sh = from & 31;
#pragma unroll
            for (int c = 0; c < kNX; ++c)
#pragma unroll
              for (int d = 0; d < 2; ++d) {
                const uint64_t w = column_word(8 * c + 2 * t + d);
                const uint32_t w0 = static_cast<uint32_t>(w), w1 = static_cast<uint32_t>(w >> 32);
                const uint32_t a = part == 0 ? ~0u : part == 1 ? w0 : part == 2 ? w1 : 0u;
                const uint32_t b = part == 0 ? w0 : part == 1 ? w1 : 0u;
                const uint32_t v = (w0 | w1) != 0u ? __funnelshift_r(a, b, sh) : 0u;
#pragma unroll
                for (int j = 0; j < 4; ++j)
                  if (!((v >> (8 * j)) & 1u)) x[j >> 1][4 * c + 2 * (j & 1) + d] = -INFINITY;
              }
          }
        };
        // x -> x * qscale - m; whether a score passes its row's maximum by more
        // than the threshold
        auto shift = [&]() -> bool {
          float top = -INFINITY;
#pragma unroll
          for (int c = 0; c < kNX; ++c) {
            const unsigned long long nm = pack_f32x2(-m_run[c][0], -m_run[c][1]);
#pragma unroll
            for (int hf = 0; hf < 2; ++hf)
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                float* y = &x[hf][4 * c + 2 * e];
                unpack_f32x2(ffma2(pack_f32x2(y[0], y[1]), qs2, nm), y[0], y[1]);
                top = fmax3(top, y[0], y[1]);
              }
          }
          return top > kRescaleThreshold;
        };
        for (bool slow = i == 0;; slow = true) {
          load();  // (S has not been given back yet)
          if (slow) {
            // ---- the rows' maxima of this tile, then the new running ones ----
            // P's place is free once the chain's last product has read it (and
            // the last segment's numbers have been read from it); O is at rest
            if (tc > 0) failed |= !wait_or_abort(pv_done, (tc - 1) & 1, s_abort);
            tc_fence_after();
            // the scratch is these rows' place in P: [4 warps][kCols], the factors
            float* scratch = reinterpret_cast<float*>(sMine);
            float* factor = scratch + 4 * kCols;
            float mx[kNX][2];
#pragma unroll
            for (int c = 0; c < kNX; ++c)
#pragma unroll
              for (int d = 0; d < 2; ++d)
                mx[c][d] = fmaxf(fmaxf(x[0][4 * c + d], x[0][4 * c + 2 + d]),
                                 fmaxf(x[1][4 * c + d], x[1][4 * c + 2 + d])) * p.qscale;
            // (shuffles stay in program order: all columns' of a step side by side)
#pragma unroll
            for (int o = 4; o < 32; o <<= 1)
#pragma unroll
              for (int c = 0; c < kNX; ++c)
#pragma unroll
                for (int d = 0; d < 2; ++d)
                  mx[c][d] = fmaxf(mx[c][d], __shfl_xor_sync(0xffffffffu, mx[c][d], o));
            if (g == 0) {
#pragma unroll
              for (int c = 0; c < kNX; ++c)
                *reinterpret_cast<float2*>(scratch + quad * kCols + 8 * c + 2 * t) =
                    make_float2(mx[c][0], mx[c][1]);
            }
            named_bar_sync(bar, kGroupThreads);
#pragma unroll
            for (int c = 0; c < kNX; ++c) {
              float2 all = make_float2(-INFINITY, -INFINITY);
#pragma unroll
              for (int w = 0; w < 4; ++w) {
                const float2 v = *reinterpret_cast<const float2*>(scratch + w * kCols + 8 * c + 2 * t);
                all.x = fmaxf(all.x, v.x);
                all.y = fmaxf(all.y, v.y);
              }
              if (i == 0) {  // nothing to rescale yet
                m_run[c][0] = fmaxf(all.x, kNoMax);
                m_run[c][1] = fmaxf(all.y, kNoMax);
                continue;
              }
              float f[2];
#pragma unroll
              for (int d = 0; d < 2; ++d) {
                const float old = m_run[c][d], top = d ? all.y : all.x;
                const bool grow = top > old + kRescaleThreshold || (old == kNoMax && top > old);
                f[d] = grow ? (old == kNoMax ? 0.f : ex2(old - top)) : 1.f;
                if (grow) m_run[c][d] = top;
                l_run[c][d] *= f[d];
              }
              if (quad == 0 && g == 0)
                *reinterpret_cast<float2*>(factor + 8 * c + 2 * t) = make_float2(f[0], f[1]);
            }
            named_bar_sync(bar, kGroupThreads);  // (and the scratch has been read)
            if (i > 0) {
#pragma unroll 1
              for (int c = 0; c < kCols; c += 16) {
                uint32_t o[16];
                tmem_ld16(t_o + c, o);
                tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < 16; ++e)
                  o[e] = __float_as_uint(__uint_as_float(o[e]) * factor[c + e]);
                tmem_st16(t_o + c, o);
              }
              tmem_wait_st();
              named_bar_sync(bar, kGroupThreads);  // the factors have been read
            }
          }
          const bool over = shift();
          if (slow || !named_bar_or(bar, kGroupThreads, over)) break;
        }
        tc_fence_before();
        mbar_arrive(s_free);
        if (tc > 0) failed |= !wait_or_abort(pv_done, (tc - 1) & 1, s_abort);
#pragma unroll
        for (int c = 0; c < kNX; ++c) {
          uint32_t w[4];  // keys 8 j .. of this warp's 32, the two rows packed
          unsigned long long sum = pack_f32x2(l_run[c][0], l_run[c][1]);
#pragma unroll
          for (int hf = 0; hf < 2; ++hf)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const float a = ex2(x[hf][4 * c + 2 * e]), b = ex2(x[hf][4 * c + 2 * e + 1]);
              sum = fadd2(sum, pack_f32x2(a, b));
              w[2 * hf + e] = pack_bf16x2(a, b);
            }
          unpack_f32x2(sum, l_run[c][0], l_run[c][1]);
          // row 8 c + (lane & 7) of these, keys 32 quad + 8 (lane >> 3) ..
          const int row = col0 + 8 * c + (lane & 7);
          const int chunk = 4 * quad + (lane >> 3);
          stsm_x4_trans(sPa + (chunk >> 3) * C::kOperHalf + row * 128 +
                            (((chunk & 7) ^ (row & 7)) << 4),
                        w[0], w[1], w[2], w[3]);
        }
        fence_proxy_async_smem();
        tc_fence_before();
        mbar_arrive(p_full);
        ++tc;
      }

      // ---- the segment's end: O / l and the LSE, or a partial ----
      // this warp's sums, while the last product runs
#pragma unroll
      for (int o = 4; o < 32; o <<= 1)
#pragma unroll
        for (int c = 0; c < kNX; ++c)
#pragma unroll
          for (int d = 0; d < 2; ++d)
            l_run[c][d] += __shfl_xor_sync(0xffffffffu, l_run[c][d], o);
      failed |= !wait_or_abort(pv_done, (tc - 1) & 1, s_abort);
      tc_fence_after();
      // in P's place: l [4 warps][kCols], m [kCols]; then per row the
      // accumulator's factor and the place in out (-1: none)
      float* xl = reinterpret_cast<float*>(sMine);
      float* fac = xl + 5 * kCols;
      int* place = reinterpret_cast<int*>(fac + kCols);
      if (g == 0) {
#pragma unroll
        for (int c = 0; c < kNX; ++c) {
          const int col = 8 * c + 2 * t;
          *reinterpret_cast<float2*>(xl + quad * kCols + col) =
              make_float2(l_run[c][0], l_run[c][1]);
          if (quad == 0)
            *reinterpret_cast<float2*>(xl + 4 * kCols + col) = make_float2(m_run[c][0], m_run[c][1]);
        }
      }
      named_bar_sync(bar, kGroupThreads);
      float* slot = p.partials +
                    (2 * static_cast<int64_t>(worker) + (first_of_range ? 0 : 1)) *
                        slot_floats(p.slot_rows);
      const int64_t out0 = (static_cast<int64_t>(sg.b) * p.n_nodes) * p.num_q_heads + kvh * p.group;
      if (tid < kCols) {
        const int r = r0 + tid;
        const float l = (xl[tid] + xl[kCols + tid]) + (xl[2 * kCols + tid] + xl[3 * kCols + tid]);
        const float m = xl[4 * kCols + tid];
        const bool in = r < p.rows && !failed;
        // a live row with keys (a NaN among the scores stays one)
        const bool has = in && column_word(tid) != 0 && l != 0.f;
        fac[tid] = has ? (whole ? 1.f / l : 1.f) : 0.f;
        const int rel = (r >> p.group_shift) * p.num_q_heads + (r & (p.group - 1));
        place[tid] = in ? (whole ? rel : col0 + tid) : -1;
        if (in) {
          if (whole) {
            p.lse[out0 + rel] = has ? (m + __log2f(l)) * 0.69314718055994531f : -INFINITY;
          } else {
            float* ml = slot + static_cast<int64_t>(kHeadDim) * p.slot_rows + col0 + tid;
            ml[0] = has ? m : -INFINITY;
            ml[p.slot_rows] = has ? l : 0.f;
          }
        }
      }
      named_bar_sync(bar, kGroupThreads);
      // O^T: this thread's head dim, 16 rows at a time
      const int dim = 32 * quad + lane;
      __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.out) + out0 * kHeadDim + dim;
      auto store_rows = [&](auto to_out) {
#pragma unroll 1
        for (int c = 0; c < kCols; c += 16) {
          if (r0 + c >= p.rows) break;
          uint32_t o[16];
          tmem_ld16(t_o + c, o);
          tmem_wait_ld();
#pragma unroll
          for (int e4 = 0; e4 < 16; e4 += 4) {
            const float4 f = *reinterpret_cast<const float4*>(fac + c + e4);
            const int4 at = *reinterpret_cast<const int4*>(place + c + e4);
            const float fs[4] = {f.x, f.y, f.z, f.w};
            const int as[4] = {at.x, at.y, at.z, at.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              // (a row that has seen nothing may hold anything in its accumulator)
              const float v = fs[e] != 0.f ? __uint_as_float(o[e4 + e]) * fs[e] : 0.f;
              if (decltype(to_out)::value) {
                if (as[e] >= 0) out[static_cast<uint32_t>(as[e]) * kHeadDim] = __float2bfloat16_rn(v);
              } else {
                if (as[e] >= 0) slot[static_cast<uint32_t>(as[e]) * kHeadDim + dim] = v;
              }
            }
          }
        }
      };
      if (whole) store_rows(std::true_type{});
      else store_rows(std::false_type{});
      tc_fence_before();
      mbar_arrive(o_free);
      ++si;
      // (a barrier also between these reads of P's place and the next segment's writes)
      if (named_bar_or(worker_bar, kShare * kGroupThreads, failed || *s_abort != 0)) {
        set_dev_err(p.dev_err, PKV_DEV_ERR_TIMEOUT);
        *s_abort = 1;
        break;
      }
    }
  }
  if (*s_abort && threadIdx.x == 0) set_dev_err(p.dev_err, PKV_DEV_ERR_TIMEOUT);
  tc_fence_before();
  __syncthreads();
  if (warp == 2) {
    tc_fence_after();
    tmem_dealloc(tmem, C::kTmemCols);
  }
}

namespace {
template <int kCols, int kShare>
cudaError_t launch(const CUtensorMap& qmap, const CUtensorMap& kmap, const CUtensorMap& vmap,
                   const TreeParams& p, int sms, int dev, cudaStream_t stream) {
  using C = TileCfg<kCols, kShare>;
  return launch_form<tree_tile_kernel<kCols, kShare>>(C::kThreads, C::kSmemBytes, sms, qmap, kmap,
                                                      vmap, p, dev, stream);
}
}  // namespace

cudaError_t launch_tile_form(const CUtensorMap& qmap, const CUtensorMap& kmap,
                             const CUtensorMap& vmap, const TreeParams& p, int sms, int dev,
                             cudaStream_t stream) {
  // 32 columns where they do: at 32 rows 43 against 49 us with 64 columns (64 x ~768
  // keys), 62 against 67 (32 x ~2560), 162 against 169 (8 x 32768)
  return p.rows <= 32   ? launch<32, 1>(qmap, kmap, vmap, p, sms, dev, stream)
         : p.rows <= 64 ? launch<64, 1>(qmap, kmap, vmap, p, sms, dev, stream)
                        : launch<64, 2>(qmap, kmap, vmap, p, sms, dev, stream);
}

}  // namespace tree
}  // namespace pkv
