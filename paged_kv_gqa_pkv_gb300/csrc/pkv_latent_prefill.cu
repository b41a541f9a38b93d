// pkv_latent_prefill.cu - causal attention of packed sequences in the expanded form of
// shared latents, on tcgen05 tensor cores: a head's key is its own 128 values and the
// token's 64 rotated ones (which all heads share), its value 128.
//
// For query i of the n of a sequence with m keys, over the keys t <= m - n + i:
//   x[t] = scale (q_own . k_own[t] + q_rot . k_rot[t]),
//   lse = ln sum_t exp x[t],   out = sum_t exp(x[t] - lse) v[t].
//
// An item is 256 query rows of one sequence and head, as two tiles of 128 rows that read the
// same keys. Per 128 keys the tensor cores take 2 x (12 + 8) MMAs of 128 x 128 x 16, 2560
// cycles at their rate; the 65 536 exponentials take 1024 to 2048. So the tensor pipe is the
// bound, if each tile's softmax is hidden behind the other's products.
//
// Roles of a CTA (one per SM; it takes item after item, the costly ones first): warp 0 loads keys
// and values by TMA into a ring of eight 16 KB slots (K: three slots of 64 dims x 128 keys, V: two
// of 64 keys), warp 2 the queries, one thread each of warps 1 and 3 issues the MMAs of one tile,
// warps 4-7 and 8-11 are the softmax of the two tiles, a query row per thread. Tensor memory holds
// S_0, S_1, O_0, O_1 (128 columns each); P_h, bf16, is written over S_h and read from there by the
// product with V.
//
// The two tiles' chains QK -> softmax -> PV -> QK .. are independent, each with its own issuing
// thread. (One thread that polled both chains' barriers took ~800 cycles a round beside the
// softmax warps: 6000 cycles a key tile.) A chain takes 3600 to 4200 cycles a key tile, of which
// its products run 1280: QK 1000 to 1300 from issue to S, softmax 1500 to 1900 (reading S twice, 64 columns at a
// time, in loops: with all 128 in registers the unrolled code does not stay in the instruction
// cache, 4 % slower), P's arrival to PV's end ~600, and so on. Beside a softmax each barrier
// instruction of an issuing thread takes ~100-250 cycles, for it queues behind exponentials; so
// there are few (a tile's keys have one barrier), and those that need not be waited for last are
// waited for before P. Measured with 32 heads: 24 prompts of 64 .. 1024 tokens 124 us (0.74
// PFLOP/s; the floor of their bytes is 71), 8 chunks of 512 behind 512 .. 4096 165 us (1.30
// PFLOP/s of 1.99; 172 to 179 us once the card has run them for 20 ms and lowers its clock). Tiles forced half a period apart by a barrier: 3 % slower (what each gains, the
// ring's eight slots take back: a tile's keys land where the slower tile has read values).
#include <atomic>
#include <cmath>

#include "pkv_latent.cuh"

namespace pkv {
namespace {

using namespace latent;
using namespace prefill_detail;

constexpr int kSlots = 8;
constexpr int kSlot = 128 * 128;              // 16 KB
constexpr int kQChunks = (kOwnKey + kRotated) / 64;
constexpr int kItemRows = 2 * kBM;
constexpr int kExpThreads = 12 * 32;

// shared memory, offsets from a 1024-aligned base
constexpr int kOffQ = 0;                                  // [2 tiles][3 chunks][128 rows]
constexpr int kOffRing = kOffQ + 2 * kQChunks * kSlot;
constexpr int kOffBar = kOffRing + kSlots * kSlot;
// k_full[2], k_empty[2], v_full[2], v_empty[2][2], q_full[2], q_empty[2], s_full[2], p_full[2][2],
// pv_done[2], o_free[2], tail, item_full[4], item_free[4], claim
constexpr int kAheadItems = 4;
constexpr int kNumBars = 10 + 15 + 2 * kAheadItems + 1;
constexpr int kOffMisc = kOffBar + kNumBars * 8;          // tmem slot, abort flag
constexpr int kOffItem = kOffMisc + 16;
constexpr int kItemInts = 8;
constexpr int kOffClaim = kOffItem + kAheadItems * kItemInts * 4;  // 16 bytes
constexpr int kOffSched = kOffClaim + 16;
constexpr int kExpSmem = kOffSched + kSchedMaxTiles * 2 + 1024;  // + slack for the alignment
static_assert(kExpSmem <= kMaxDynSmem, "shared memory above the opt-in limit");
static_assert(kSlots * kSlot >= kSchedSortBytes, "the sort's scratch lives in the ring");
static_assert(kOffClaim % 16 == 0, "a claim's answer is 16-byte aligned");

constexpr uint32_t kIdescS = idesc_bf16_f32(kBM, kBN, false);
constexpr uint32_t kIdescO = idesc_bf16_f32(kBM, kValue, true);

struct LatentPrefillParams {
  const int32_t* q_starts;
  const int32_t* k_starts;
  __nv_bfloat16* out;   // [tq, heads, 128]
  float* lse;           // [tq, heads]
  int32_t* dev_err;
  int n_seqs;
  int heads;
  int tq;
  int tk;
  int n_tiles;          // places for 256-row tiles: tq / 256 + n_seqs
  float qscale;         // scale * log2(e)
};

// Four K-steps, operands in shared memory.
__device__ __forceinline__ void umma4_ss(uint32_t d, uint32_t a_lo, uint32_t b_lo, uint32_t idesc,
                                         uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p0, p1;\n\t.reg .b64 a<4>, b<4>;\n\t.reg .b32 x<4>, y<4>;\n\t"
      "setp.ne.b32 p0, %3, 0;\n\tsetp.eq.b32 p1, %3, %3;\n\t"
      "add.u32 x1, %1, 2;\n\tadd.u32 x2, %1, 4;\n\tadd.u32 x3, %1, 6;\n\t"
      "add.u32 y1, %2, 2;\n\tadd.u32 y2, %2, 4;\n\tadd.u32 y3, %2, 6;\n\t"
      "mov.b64 a0, {%1, %5};\n\tmov.b64 b0, {%2, %5};\n\t"
      "mov.b64 a1, {x1, %5};\n\tmov.b64 b1, {y1, %5};\n\t"
      "mov.b64 a2, {x2, %5};\n\tmov.b64 b2, {y2, %5};\n\t"
      "mov.b64 a3, {x3, %5};\n\tmov.b64 b3, {y3, %5};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], a0, b0, %4, p0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], a1, b1, %4, p1;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], a2, b2, %4, p1;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], a3, b3, %4, p1;\n\t}" ::"r"(d),
      "r"(a_lo), "r"(b_lo), "r"(accumulate), "r"(idesc), "n"(kDescHi)
      : "memory");
}
// Four K-steps of 16 keys, P from tensor memory (8 columns a step), V from shared memory.
__device__ __forceinline__ void umma4_ts(uint32_t d, uint32_t a_tmem, uint32_t b_lo,
                                         uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p0, p1;\n\t.reg .b64 b<4>;\n\t.reg .b32 x<4>, y<4>;\n\t"
      "setp.ne.b32 p0, %3, 0;\n\tsetp.eq.b32 p1, %3, %3;\n\t"
      "add.u32 x1, %1, 8;\n\tadd.u32 x2, %1, 16;\n\tadd.u32 x3, %1, 24;\n\t"
      "add.u32 y1, %2, 128;\n\tadd.u32 y2, %2, 256;\n\tadd.u32 y3, %2, 384;\n\t"
      "mov.b64 b0, {%2, %5};\n\tmov.b64 b1, {y1, %5};\n\t"
      "mov.b64 b2, {y2, %5};\n\tmov.b64 b3, {y3, %5};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b0, %4, p0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [x1], b1, %4, p1;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [x2], b2, %4, p1;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [x3], b3, %4, p1;\n\t}" ::"r"(d),
      "r"(a_tmem), "r"(b_lo), "r"(accumulate), "r"(idesc), "n"(kDescHi)
      : "memory");
}

// exp2(s * qscale - m) of 64 columns, as bf16 pairs into 32 columns of this thread's TMEM lane;
// their sum in fp32. Scale, shift and sum run two values per instruction.
__device__ __forceinline__ float weights_to_tmem(const uint32_t (&s)[64], float qscale, float neg_m,
                                                 uint32_t t_p) {
  const unsigned long long qs2 = pack_f32x2(qscale, qscale);
  const unsigned long long nm2 = pack_f32x2(neg_m, neg_m);
  unsigned long long acc0 = 0ull, acc1 = 0ull;
  uint32_t pk[32];
#pragma unroll
  for (int c = 0; c < 64; c += 4) {
    float e[4];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const unsigned long long x2 = ffma2(
          pack_f32x2(__uint_as_float(s[c + 2 * u]), __uint_as_float(s[c + 2 * u + 1])), qs2, nm2);
      float x0, x1;
      unpack_f32x2(x2, x0, x1);
      e[2 * u] = ex2(x0);
      e[2 * u + 1] = ex2(x1);
    }
    acc0 = fadd2(acc0, pack_f32x2(e[0], e[1]));
    acc1 = fadd2(acc1, pack_f32x2(e[2], e[3]));
    pk[c / 2] = pack_bf16x2(e[0], e[1]);
    pk[c / 2 + 1] = pack_bf16x2(e[2], e[3]);
  }
  tmem_st32(t_p, pk);
  float a, b, c, d;
  unpack_f32x2(acc0, a, b);
  unpack_f32x2(acc1, c, d);
  return (a + b) + (c + d);
}

// 64 scores of a row.
__device__ __forceinline__ void load_half(uint32_t t_s, uint32_t (&s)[64]) {
  tmem_ld32(t_s, *reinterpret_cast<uint32_t(*)[32]>(&s[0]));
  tmem_ld32(t_s + 32, *reinterpret_cast<uint32_t(*)[32]>(&s[32]));
  tmem_wait_ld();
}

// 32 bytes to global memory in one instruction.
__device__ __forceinline__ void st_global_v8(void* a, const uint32_t (&w)[8]) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(a), "r"(w[0]),
               "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}

// ------------------------------------------------------------------- items --

// A place for a 256-row tile: sequence b owns the places q_starts[b] / 256 + b up to the next
// sequence's first one, as many as its rows can need. Places without rows have rows = 0.
struct Tile {
  int q0;    // its first query's token
  int rows;  // its queries
  int k0;    // the sequence's first key
  int nk;    // the sequence's keys
  int see;   // keys that its first query sees (may be negative)
};
__device__ __forceinline__ Tile tile_at(const LatentPrefillParams& p, int place) {
  Tile t;
  t.q0 = t.rows = t.k0 = t.nk = t.see = 0;
  int lo = 0, hi = p.n_seqs;  // the first sequence whose places begin past `place`
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if ((__ldg(p.q_starts + mid) >> 8) + mid <= place) lo = mid + 1;
    else hi = mid;
  }
  const int b = lo - 1;
  if (b < 0) return t;
  const int q0 = __ldg(p.q_starts + b), q1 = __ldg(p.q_starts + b + 1);
  const int k0 = __ldg(p.k_starts + b), k1 = __ldg(p.k_starts + b + 1);
  if (q0 < 0 || q1 < q0 || q1 > p.tq || k0 < 0 || k1 < k0 || k1 > p.tk) return t;
  const int i0 = (place - ((q0 >> 8) + b)) * kItemRows;
  if (i0 < 0 || i0 >= q1 - q0) return t;
  t.q0 = q0 + i0;
  t.rows = min(kItemRows, q1 - q0 - i0);
  t.k0 = k0;
  t.nk = k1 - k0;
  t.see = t.nk - (q1 - q0) + i0 + 1;
  return t;
}
// Takes the item of a block that has not started yet: its index, or -1 if there is none (no claim
// may follow that answer). answer: 16 bytes of shared memory.
__device__ __forceinline__ int claim_block(void* answer, uint64_t* bar, uint32_t parity,
                                           volatile int* abort_flag, bool* ok) {
  mbar_arrive_expect_tx(bar, 16);
  asm volatile(
      "clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128"
      " [%0], [%1];" ::"r"(smem_u32(answer)),
      "r"(smem_u32(bar))
      : "memory");
  *ok = wait_phase(bar, parity, abort_flag);
  if (!*ok) return -1;
  int x;
  asm volatile(
      "{\n\t.reg .b128 r;\n\t.reg .pred p;\n\tld.shared.b128 r, [%1];\n\t"
      "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, r;\n\tmov.b32 %0, -1;\n\t"
      "@p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %0, r;\n\t}"
      : "=r"(x)
      : "r"(smem_u32(answer))
      : "memory");
  fence_proxy_async_smem();  // (the next answer is written by the async proxy)
  return x;
}

// Looking an item's tile up takes a bisection through global memory, ~1500 cycles beside the
// softmax warps. Warp 2 does it for the items to come and leaves them in a ring in shared memory;
// every role reads them there. readers: the loads, two issuing threads, eight softmax warps.
constexpr int kItemReaders = 11;
struct Item {
  Tile x;
  int head;  // -1: no more items
};
struct ItemReader {
  const int* ring;
  uint64_t* full;
  uint64_t* free;
  int r = 0;
  // By a whole warp, or by one thread alone. kFree: the reader needs no more of it; else it says
  // so itself.
  template <bool kWarp, bool kFree = true>
  __device__ __forceinline__ bool next(Item* it, volatile int* abort_flag, bool* ok) {
    const int at = r % kAheadItems;
    *ok = wait_phase(&full[at], (r / kAheadItems) & 1, abort_flag);
    if (kWarp) *ok = __all_sync(0xffffffffu, *ok);
    if (!*ok) return false;
    const int* v = ring + at * kItemInts;
    it->x.q0 = v[0], it->x.rows = v[1], it->x.k0 = v[2], it->x.nk = v[3], it->x.see = v[4];
    it->head = v[5];
    if (kWarp) __syncwarp();
    if (kFree && (!kWarp || (threadIdx.x & 31) == 0)) mbar_arrive(&free[at]);
    ++r;
    return it->head >= 0;
  }
};
// Key tiles that row tile h of an item reads (0: none, or no rows).
__device__ __forceinline__ int key_tiles(const Tile& t, int h) {
  const int last = min(t.rows, kBM * (h + 1)) - 1;  // its last row
  if (last < kBM * h) return 0;
  const int see = min(t.see + last, t.nk);
  return see > 0 ? (see + kBN - 1) / kBN : 0;
}

}  // namespace

__global__ void __launch_bounds__(kExpThreads, 1)
latent_prefill_kernel(const __grid_constant__ CUtensorMap qmap,
                      const __grid_constant__ CUtensorMap kmap,
                      const __grid_constant__ CUtensorMap rmap,
                      const __grid_constant__ CUtensorMap vmap, const LatentPrefillParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  // [2], a key tile's by its number's parity: its keys (values) are there; both row tiles'
  // products have read them (the values: [2][2], the first and the last 64)
  uint64_t* k_full = reinterpret_cast<uint64_t*>(smem + kOffBar);
  uint64_t* k_empty = k_full + 2;
  uint64_t* v_full = k_empty + 2;
  uint64_t* v_empty = v_full + 2;
  uint64_t* q_full = v_empty + 4;  // [2]
  uint64_t* q_empty = q_full + 2;
  uint64_t* s_full = q_empty + 2;
  uint64_t* p_full = s_full + 2;   // [tile][half of its keys]: P_h is there, O_h rescaled
  uint64_t* pv_done = p_full + 4;
  uint64_t* o_free = pv_done + 2;  // the epilogue has read O_h
  uint64_t* tail = o_free + 2;     // values of a tile past whose last key there are others' rows
  uint64_t* item_full = tail + 1;              // [4]
  uint64_t* item_free = item_full + kAheadItems;  // [4]
  uint64_t* claim = item_free + kAheadItems;      // the answer to a claim has arrived
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + kOffMisc);
  volatile int* s_abort = reinterpret_cast<volatile int*>(smem + kOffMisc + 4);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int h = 0; h < 2; ++h) {
      mbar_init(&k_full[h], 1);
      mbar_init(&k_empty[h], 2);  // both row tiles'
      mbar_init(&v_full[h], 1);
      mbar_init(&v_empty[h], 2);
      mbar_init(&v_empty[2 + h], 2);
      mbar_init(&q_full[h], 1);
      mbar_init(&q_empty[h], 1);
      mbar_init(&s_full[h], 1);
      mbar_init(&p_full[2 * h], 4);  // the tile's four warps
      mbar_init(&p_full[2 * h + 1], 4);
      mbar_init(&pv_done[h], 1);
      mbar_init(&o_free[h], 4);
    }
    mbar_init(tail, 1);
    mbar_init(claim, 1);
    for (int i = 0; i < kAheadItems; ++i) {
      mbar_init(&item_full[i], 1);
      mbar_init(&item_free[i], kItemReaders);
    }
    *s_abort = 0;
    fence_barrier_init();
    tma_prefetch_desc(&qmap);
    tma_prefetch_desc(&kmap);
    tma_prefetch_desc(&rmap);
    tma_prefetch_desc(&vmap);
  }
  if (warp == 1) tmem_alloc(tmem_slot, kTmemCols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  pdl_wait_primary();
  pdl_launch_dependents();
  // starts have to ascend from 0 or more to the tokens there are (which blocks run is not known)
  for (int i = threadIdx.x; i <= p.n_seqs; i += kExpThreads) {
    const int q = __ldg(p.q_starts + i), k = __ldg(p.k_starts + i);
    const int qb = i > 0 ? __ldg(p.q_starts + i - 1) : 0, kb = i > 0 ? __ldg(p.k_starts + i - 1) : 0;
    if (q < qb || q > p.tq || k < kb || k > p.tk) set_dev_err(p.dev_err, PKV_DEV_ERR_LAYOUT);
  }
  // the places, the costly ones first, a sequence's together (as they stand where they are too
  // many to sort)
  uint16_t* const s_order = reinterpret_cast<uint16_t*>(smem + kOffSched);
  const bool sorted = p.n_tiles > 1 && p.n_tiles <= kSchedMaxTiles;
  if (sorted)
    sched_sort(
        s_order, smem + kOffRing, p.n_tiles,
        [&](int t) -> int {
          const Tile x = tile_at(p, t);
          // (an item's queries, first products and results take about 1.5 key tiles' time)
          return x.rows == 0 ? 0 : 2 * max(key_tiles(x, 0), key_tiles(x, 1)) + 3;
        },
        [&](int t) -> bool {  // the next place goes on in the same sequence
          const Tile x = tile_at(p, t), y = tile_at(p, t + 1);
          return x.rows > 0 && y.rows > 0 && y.k0 == x.k0 && y.q0 == x.q0 + kItemRows;
        });
  fence_proxy_async_smem();  // (the scratch's place goes to TMA)
  __syncthreads();
  int* const s_items = reinterpret_cast<int*>(smem + kOffItem);
  ItemReader items_ahead{s_items, item_full, item_free};
  Item it;

  // 384 threads start with 168 registers each; the softmax warps need more, the others few.
  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
    if (warp == 0) {
      // ------------------------------------------ keys and values ----
      // Tile n's keys take the ring's slots 5n .. 5n + 2 (mod 8), its values the next two: the
      // first 64 dims of the keys go where tile n - 2's last ones were (the load of tile n - 1's
      // values has waited for them), the others where its values were, half by half, and the
      // values where tile n - 1's keys were.
      uint32_t n = 0, slot = 0, tails = 0;  // tiles, the next slot, tiles with a tail
      bool ok = true;
      while (items_ahead.next<true, false>(&it, s_abort, &ok)) {
        const Tile& x = it.x;
        const int head = it.head;
        const int nt = max(key_tiles(x, 0), key_tiles(x, 1));
        // The next item is claimed on this word: late, so that no CTA holds one that another could
        // begin earlier (claimed when an item begins, chunks took 170 us instead of 164), but with
        // time to look it up.
        const int claim_at = max(nt - 2, 0);
        uint64_t* const claimed = &item_free[(items_ahead.r - 1) % kAheadItems];
        if (nt == 0 && lane == 0) mbar_arrive(claimed);
        for (int t = 0; t < nt; ++t, ++n) {
          if (t == claim_at && lane == 0) mbar_arrive(claimed);
          const uint32_t at = n & 1;
          const int key = x.k0 + t * kBN;
          const int left = x.nk - t * kBN;  // keys of the sequence from this tile on
          if (lane == 0) mbar_arrive_expect_tx(&k_full[at], kQChunks * kSlot);
#pragma unroll 1
          for (int s = 0; s < kQChunks; ++s) {
            if (s > 0 && n >= 2)
              ok = wait_phase(&v_empty[2 * (s - 1) + at], ((n >> 1) - 1) & 1, s_abort);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            uint8_t* dst = smem + kOffRing + ((slot + s) % kSlots) * kSlot;
            if (lane == 0) {
              if (s < 2) tma_load_3d(dst, &kmap, &k_full[at], 64 * s, head, key);
              else tma_load_3d(dst, &rmap, &k_full[at], 0, 0, key);
            }
          }
          if (!ok) break;
          slot = (slot + kQChunks) % kSlots;
          ok = n < 1 || wait_phase(&k_empty[at ^ 1], ((n - 1) >> 1) & 1, s_abort);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          const bool ragged = left < kBN && (left & 15) != 0;
          if (lane == 0) {
            uint64_t* bar = ragged ? tail : &v_full[at];
            mbar_arrive_expect_tx(bar, 2 * kSlot);
#pragma unroll 1
            for (int v = 0; v < 4; ++v)  // 64 keys, 64 dims at a time
              tma_load_3d(smem + kOffRing + ((slot + (v >> 1)) % kSlots) * kSlot +
                              (v & 1) * (kSlot / 2),
                          &vmap, bar, 64 * (v & 1), head, key + 64 * (v >> 1));
          }
          if (ragged) {
            // the rows past the sequence that share a 16-key step with its last ones: their
            // weights are 0, but what stands there may be NaN
            ok = __all_sync(0xffffffffu, wait_phase(tail, tails & 1, s_abort));
            ++tails;
            if (!ok) break;
            uint8_t* dst = smem + kOffRing + ((slot + (left >> 6)) % kSlots) * kSlot;
            const int z = 16 - (left & 15);
            for (int e = lane; e < z * 16; e += 32)
              *reinterpret_cast<uint4*>(dst + (e & 8) * (kSlot / 16) +
                                        ((left & 63) + (e >> 4)) * 128 + (e & 7) * 16) =
                  make_uint4(0u, 0u, 0u, 0u);
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&v_full[at]);
          }
          slot = (slot + 2) % kSlots;
        }
        if (!ok) break;
      }
      if (!ok && lane == 0) *s_abort = 1;
    } else if (warp == 2) {
      // ------------------------------------- items to come, queries ----
      if (lane == 0) {
        // The grid has a block for every item; a CTA that is running takes the items of blocks
        // that have not started, one when all its roles have begun the one before.
        uint32_t n[2] = {0u, 0u};
        bool ok = true;
        int item = blockIdx.x;
        for (int r = 0; ok; ++r) {
          const int at = r % kAheadItems;
          int* v = s_items + at * kItemInts;
          Tile x;
          x.rows = 0;
          int head = -1;
          if (item >= 0) {
            const int pos = item / p.heads;
            head = item - pos * p.heads;
            x = tile_at(p, sorted ? s_order[pos] : pos);
            v[0] = x.q0, v[1] = x.rows, v[2] = x.k0, v[3] = x.nk, v[4] = x.see;
          }
          v[5] = head;
          mbar_arrive(&item_full[at]);
          if (item < 0) break;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            if (!ok || key_tiles(x, h) == 0) continue;
            ok = n[h] == 0 || wait_phase(&q_empty[h], (n[h] - 1) & 1, s_abort);
            if (!ok) break;
            mbar_arrive_expect_tx(&q_full[h], kQChunks * kSlot);
            for (int c = 0; c < kQChunks; ++c)
              tma_load_3d(smem + kOffQ + (h * kQChunks + c) * kSlot, &qmap, &q_full[h], 64 * c, head,
                          x.q0 + kBM * h);
            ++n[h];
          }
          ok = ok && wait_phase(&item_free[at], (r / kAheadItems) & 1, s_abort);
          if (ok) item = claim_block(smem + kOffClaim, claim, r & 1, s_abort, &ok);
        }
        if (!ok) *s_abort = 1;
      }
    } else {
      // ------------------------------------------------------- MMAs ----
      // Warp 1 for tile 0, warp 3 for tile 1: each waits for its own tile's barriers only, so
      // that the tiles' products fill each other's gaps. Both wait for every slot of the ring and
      // give it back, also for the key tiles that only the other needs.
      if (elect_one()) {
        const int h = warp >> 1;
        const uint32_t t_s = tmem + kBN * h, t_o = tmem + 256 + kValue * h;
        const uint32_t q_lo = desc_lo(smem_u32(smem + kOffQ + h * kQChunks * kSlot), 0);
        const uint32_t ring_k = desc_lo(smem_u32(smem + kOffRing), 0);
        const uint32_t ring_v = desc_lo(smem_u32(smem + kOffRing), kSlot / 2);
        uint32_t n = 0;             // key tiles of this row tile
        uint32_t tc = 0, slot = 0;  // key tiles of the ring, its next slot
        uint32_t items = 0;
        bool ok = true;
        // gives a tile's slots back: when the MMAs so far are done, or at once
        auto give_back = [&](uint64_t* bar, bool mine) {
          if (mine) umma_commit(bar);
          else mbar_arrive(bar);
        };
        while (ok && items_ahead.next<false>(&it, s_abort, &ok)) {
          const Tile& x = it.x;
          const int nt = key_tiles(x, h), all = max(nt, key_tiles(x, 1 - h));
          if (all == 0) continue;
          if (nt > 0) ok = wait_phase(&q_full[h], items & 1, s_abort);
#pragma unroll 1
          for (int t = 0; ok && t < all; ++t, ++tc) {
            const bool mine = t < nt;
            const uint32_t at = tc & 1, ph = (tc >> 1) & 1;
            if (t == 0 || !mine) ok = wait_phase(&k_full[at], ph, s_abort);
            if (mine && ok) {
              // S_h = Q_h K^T, over P_h once the last PV_h has read it
              ok = n == 0 || wait_phase(&pv_done[h], (n - 1) & 1, s_abort);
              if (!ok) break;
              tc_fence_after();
#pragma unroll
              for (uint32_t s = 0; s < kQChunks; ++s)
                umma4_ss(t_s, q_lo + ((s * kSlot) >> 4),
                         ring_k + ((((slot + s) % kSlots) * kSlot) >> 4), kIdescS, s > 0 ? 1u : 0u);
              umma_commit(&s_full[h]);
              if (t + 1 == nt) umma_commit(&q_empty[h]);
            }
            give_back(&k_empty[at], mine);
            slot = (slot + kQChunks) % kSlots;
            // (what has been there long before P is waited for first)
            ok = ok && wait_phase(&v_full[at], ph, s_abort);
            if (mine) {
              // O_h += P_h V
              ok = ok && (t > 0 || items == 0 || wait_phase(&o_free[h], (items - 1) & 1, s_abort));
              const int left = x.nk - t * kBN;
              const int steps = left >= kBN ? 8 : (left + 15) >> 4;
#pragma unroll 1
              for (int v = 0; ok && v < 2; ++v) {
                const uint32_t b = ring_v + ((((slot + v) % kSlots) * kSlot) >> 4);
                const uint32_t a = t_s + 32 * v;
                const uint32_t acc = t > 0 || v > 0 ? 1u : 0u;
                const int k_n = steps - 4 * v;
                // (the next product's keys, whose wait costs nothing here)
                if (v == 1 && t + 1 < nt)
                  ok = wait_phase(&k_full[at ^ 1], ((tc + 1) >> 1) & 1, s_abort);
                ok = ok && wait_phase(&p_full[2 * h + v], n & 1, s_abort);
                if (!ok) break;
                tc_fence_after();
                if (k_n >= 4) {
                  umma4_ts(t_o, a, b, kIdescO, acc);
                } else {
#pragma unroll 1
                  for (int k = 0; k < k_n; ++k)
                    umma_bf16_ts(t_o, a + 8 * k,
                                 (static_cast<uint64_t>(kDescHi) << 32) | (b + 128u * k), kIdescO,
                                 acc | (k > 0 ? 1u : 0u));
                }
                if (v == 0) umma_commit(&v_empty[at]);
              }
              if (!ok) break;
              umma_commit(&pv_done[h]);
              ++n;
            }
            if (!mine) mbar_arrive(&v_empty[at]);
            give_back(&v_empty[2 + at], mine);
            slot = (slot + 2) % kSlots;
          }
          if (nt > 0) ++items;
        }
        if (!ok) *s_abort = 1;
      }
    }
  } else {
    // ------------------------------------------ softmax and epilogue ----
    asm volatile("setmaxnreg.inc.sync.aligned.u32 224;");
    const int h = (warp - 4) >> 2;
    const int lane_base = 32 * (warp & 3);
    const int row = lane_base + lane;  // of the tile
    const uint32_t t_lane = tmem + (static_cast<uint32_t>(lane_base) << 16);
    const uint32_t t_s = t_lane + kBN * h;
    const uint32_t t_o = t_lane + 256 + kValue * h;
    uint32_t n = 0;
    bool ok = true;
    while (ok && items_ahead.next<true>(&it, s_abort, &ok)) {
      const Tile& x = it.x;
      const int head = it.head;
      const int nt = key_tiles(x, h);
      const int i = kBM * h + row;  // of the item
      const bool live = i < x.rows;
      const int see = live ? min(x.see + i, x.nk) : 0;  // keys that the row sees
      float m_run = -INFINITY;  // the maximum that the weights refer to, raw score units
      float l_run = 0.f;
      for (int t = 0; t < nt; ++t, ++n) {
        ok = __all_sync(0xffffffffu, wait_phase(&s_full[h], n & 1, s_abort));
        if (!ok) break;
        tc_fence_after();
        const int c_hi = see - t * kBN;  // visible columns
        float mx = -INFINITY;
#pragma unroll 1
        for (int v = 0; v < 2; ++v) {
          uint32_t sr[64];
          load_half(t_s + 64 * v, sr);
          if (__any_sync(0xffffffffu, c_hi < 64 * v + 64)) {
            // hidden keys' scores go back as -inf
#pragma unroll
            for (int c = 0; c < 64; ++c)
              if (c >= c_hi - 64 * v) sr[c] = __float_as_uint(-INFINITY);
            tmem_st32(t_s + 64 * v, *reinterpret_cast<uint32_t(*)[32]>(&sr[0]));
            tmem_st32(t_s + 64 * v + 32, *reinterpret_cast<uint32_t(*)[32]>(&sr[32]));
            tmem_wait_st();
          }
          float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int c = 0; c < 64; c += 8) {
#pragma unroll
            for (int k = 0; k < 4; ++k)
              m4[k] = fmax3(m4[k], __uint_as_float(sr[c + 2 * k]), __uint_as_float(sr[c + 2 * k + 1]));
          }
          mx = fmax3(fmax3(m4[0], m4[1], mx), m4[2], m4[3]);
        }
        // (P will take S's columns 0-63, and a half of S is read just before its half of P is written:
        // P's first 32 columns lie over what has been read, its last 32 too)
        // the maximum moves only when it has grown by more than 2^8: until then weights of up
        // to 256 do no harm in bf16 and fp32, and O stays as it is
        const float m_cand = fmaxf(m_run, mx);
        const bool grow = m_run == -INFINITY ? m_cand != -INFINITY
                                             : (m_cand - m_run) * p.qscale > kRescaleThreshold;
        const float m_use = grow ? m_cand : m_run;
        const float neg_m = m_use == -INFINITY ? 0.f : -m_use * p.qscale;
        // (S_h of this tile was issued after the last PV_h had completed: O_h is at rest)
        if (t > 0 && __any_sync(0xffffffffu, grow)) {
          const float alpha = grow ? ex2((m_run - m_use) * p.qscale) : 1.f;  // 0 if m_run = -inf
          l_run *= alpha;
#pragma unroll 1
          for (int q = 0; q < kValue; q += 32) {
            uint32_t o[32];
            tmem_ld32(t_o + q, o);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
            tmem_st32(t_o + q, o);
          }
        }
        // P over the first 64 columns of S_h, in bf16 (a weight off by at most 2^-8 of itself;
        // the sum takes it unrounded), the first 64 keys' first: their product with V runs while
        // the others' weights are computed.
        m_run = m_use;
#pragma unroll 1
        for (int v = 0; v < 2; ++v) {
          uint32_t sr[64];
          load_half(t_s + 64 * v, sr);
          l_run += weights_to_tmem(sr, p.qscale, neg_m, t_s + 32 * v);
          tmem_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&p_full[2 * h + v]);
        }
      }
      // ---- O / l, LSE ----
      if (ok && nt > 0) ok = __all_sync(0xffffffffu, wait_phase(&pv_done[h], (n - 1) & 1, s_abort));
      if (!ok) break;
      tc_fence_after();
      const bool has = live && l_run != 0.f;  // (a NaN among its scores: NaN)
      const float inv = has ? 1.f / l_run : 0.f;
      const long long at = static_cast<long long>(x.q0 + i) * p.heads + head;
      __nv_bfloat16* orow = p.out + at * kValue;
#pragma unroll 1
      for (int q = 0; q < kValue; q += 32) {
        uint32_t o[32];
        if (nt > 0) {
          tmem_ld32(t_o + q, o);
          tmem_wait_ld();
        }
        if (live) {
#pragma unroll
          for (int v = 0; v < 2; ++v) {
            uint32_t wv[8];
#pragma unroll
            for (int e = 0; e < 8; ++e)
              wv[e] = has ? pack_bf16x2(__uint_as_float(o[16 * v + 2 * e]) * inv,
                                        __uint_as_float(o[16 * v + 2 * e + 1]) * inv)
                          : 0u;
            st_global_v8(orow + q + 16 * v, wv);
          }
        }
      }
      if (live)
        p.lse[at] = has ? (m_run * p.qscale + __log2f(l_run)) * 0.69314718055994531f : -INFINITY;
      if (nt > 0) {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&o_free[h]);
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
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

namespace {

// {values, heads, tokens} view with free strides (in values); a box is 64 values of one head of
// `tokens` tokens, 128-byte swizzled.
bool encode_heads_map(CUtensorMap* map, const void* base, int values, int heads, int tokens,
                      int64_t token_stride, int64_t head_stride, int box_tokens) {
  prefill_host::EncodeTiledFn enc = prefill_host::encode_fn();
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(values), static_cast<cuuint64_t>(heads),
                              static_cast<cuuint64_t>(tokens)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(head_stride) * 2,
                                 static_cast<cuuint64_t>(token_stride) * 2};
  const cuuint32_t box[3] = {64u, 1u, static_cast<cuuint32_t>(box_tokens)};
  const cuuint32_t estr[3] = {1u, 1u, 1u};
  return enc != nullptr &&
         enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box,
             estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace
}  // namespace pkv

using namespace pkv;
using namespace pkv::latent;

extern "C" pkv_status pkv_latent_prefill_attention(
    const void* q, int64_t q_token_stride, int64_t q_head_stride, const void* k_own,
    int64_t k_token_stride, int64_t k_head_stride, const void* k_rot, int64_t r_token_stride,
    const void* v, int64_t v_token_stride, int64_t v_head_stride, int num_heads,
    const int32_t* q_starts, const int32_t* k_starts, int n_seqs, int n_queries, int n_keys,
    float scale, void* out, float* lse, int32_t* dev_err, cudaStream_t stream) {
  if (num_heads <= 0 || num_heads > 65535 || n_seqs < 0 || n_queries < 0 || n_keys < 0 ||
      !std::isfinite(scale) || !(scale > 0.f))
    return PKV_ERR_ARG;
  constexpr int64_t kMaxStride = int64_t{1} << 38;  // a tensor map's limit, in values
  // (an axis of length 1 has no second place to step to)
  if (num_heads == 1) q_head_stride = k_head_stride = v_head_stride = 0;
  if (n_queries == 1) q_token_stride = 0;
  if (n_keys == 1) k_token_stride = r_token_stride = v_token_stride = 0;
  for (const int64_t s : {q_token_stride, q_head_stride, k_token_stride, k_head_stride,
                          r_token_stride, v_token_stride, v_head_stride})
    if (s < 0 || s >= kMaxStride) return PKV_ERR_ARG;
  if (n_seqs == 0 || n_queries == 0) return PKV_OK;
  const long long places = n_queries / 256 + static_cast<long long>(n_seqs);
  if (places * num_heads > INT_MAX) return PKV_ERR_ARG;
  if (!q || !q_starts || !k_starts || !out || !lse || (n_keys > 0 && (!k_own || !k_rot || !v)))
    return PKV_ERR_ARG;
  for (const int64_t s : {q_token_stride, q_head_stride, k_token_stride, k_head_stride,
                          r_token_stride, v_token_stride, v_head_stride})
    if (s % 8 != 0) return PKV_ERR_ALIGN;
  if (!is_aligned(q, 16) || !is_aligned(k_own, 16) || !is_aligned(k_rot, 16) || !is_aligned(v, 16) ||
      !is_aligned(out, 32) || !is_aligned(lse, 4) || !is_aligned(q_starts, 4) ||
      !is_aligned(k_starts, 4) || !is_aligned(dev_err, 4))
    return PKV_ERR_ALIGN;
  int sms = 0;
  if (const pkv_status st = device_info(&sms); st != PKV_OK) return st;
  CUtensorMap qmap, kmap, rmap, vmap;
  // (without keys nothing is loaded: the queries' tensor stands in for what is not there)
  const bool any = n_keys > 0;
  if (!encode_heads_map(&qmap, q, kOwnKey + kRotated, num_heads, n_queries, q_token_stride,
                        q_head_stride, kBM) ||
      !encode_heads_map(&kmap, any ? k_own : q, kOwnKey, num_heads, any ? n_keys : n_queries,
                        any ? k_token_stride : q_token_stride, any ? k_head_stride : q_head_stride,
                        kBN) ||
      !encode_heads_map(&rmap, any ? k_rot : q, kRotated, 1, any ? n_keys : n_queries,
                        any ? r_token_stride : q_token_stride, any ? r_token_stride : q_token_stride,
                        kBN) ||
      !encode_heads_map(&vmap, any ? v : q, kValue, num_heads, any ? n_keys : n_queries,
                        any ? v_token_stride : q_token_stride, any ? v_head_stride : q_head_stride, 64))
    return PKV_ERR_ARG;
  int dev = 0;
  if (const cudaError_t e = cudaGetDevice(&dev); e != cudaSuccess) return record_cuda_status(e);
  static std::atomic<bool> attr_set[64] = {};  // per device; host threads may race to set it
  if (dev < 0 || dev >= 64) return PKV_ERR_DEVICE;
  if (!attr_set[dev].load(std::memory_order_acquire)) {
    const cudaError_t e = cudaFuncSetAttribute(
        latent_prefill_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kExpSmem);
    if (e != cudaSuccess) return record_cuda_status(e);
    attr_set[dev].store(true, std::memory_order_release);
  }
  LatentPrefillParams p;
  p.q_starts = q_starts;
  p.k_starts = k_starts;
  p.out = static_cast<__nv_bfloat16*>(out);
  p.lse = lse;
  p.dev_err = dev_err;
  p.n_seqs = n_seqs;
  p.heads = num_heads;
  p.tq = n_queries;
  p.tk = n_keys;
  p.n_tiles = static_cast<int>(places);
  p.qscale = scale * 1.4426950408889634f;
  const long long items = places * num_heads;
  return record_cuda_status(launch_kernel(latent_prefill_kernel,
                                          dim3(static_cast<unsigned>(items)),
                                          dim3(kExpThreads), kExpSmem, stream, true, qmap, kmap, rmap,
                                          vmap, p));
}
