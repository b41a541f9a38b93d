// pkv_verify.cu - pkv_verify_tree: which drafted tokens the target accepts,
// and the token that follows them.
//
// At a node with target row p and draft row q the children are tried one after
// another; each refusal replaces the residual r by max(r - R q, 0) and R by its
// sum. Nested residuals collapse: max(max(p - a q, 0) - R q, 0) =
// max(p - (a + R) q, 0) for R >= 0, so the whole state at a node is one scalar a
// (a_0 = 0, R_0 = 1, a_{k+1} = a_k + R_k), and a refusal costs one pass over the
// two rows, R = sum_v max(p - a q, 0), with nothing written. An acceptance costs
// two numbers. Without draft rows a refusal only takes p(tok) off R.
//
// What bounds it: the passes' bytes (one or two rows of `vocab` values for each
// refusal and for the draw), so a row of the call is shared by a cluster of
// CTAs, each with a contiguous part of the vocabulary, whose sums meet in
// distributed shared memory; with few rows it is the latency of the walk's
// dependent steps, so every number the walk may ask for (each node's token, its
// p and q at the parent) is gathered by one thread per node up front. The first
// warp of every CTA then walks, all of the cluster's alike, and hands the other
// warps the passes; a pass costs one cluster barrier, a decision none.
//
// Arithmetic: a drawn number next to a border has to fall on the side that exact
// sums give, and fp32 sums of 10^5 terms move borders by more than a token's
// probability. A pass takes R = sum p - a sum q over the v with p > a q. Doubles are slow
// on this GPU (a warp's addition holds its SM's unit for some sixteen cycles, and the walk's
// dependent ones took about a microsecond a pass), so all of it is in unevaluated pairs of
// floats by the classical error-free sum and product (Knuth, Dekker; the product's error
// by an FMA), about 48 bits, added in a fixed order. A pass adds two values per
// instruction, four instructions a pair (Sum2; seven without its starting value: 35
// against 31 us); it is bound by instruction issue about as much as by its bytes. p and q
// are exact in fp32 whatever their type.
//
// Measured: one chain of 6 nodes, 32000 tokens, without a draft 6.3 us; 12 trees of 16
// nodes, 50257 in fp32 12.8 us; 64 trees, 151936 in bf16 29 us, of which the longest row
// spends three dependent passes (8, then ~5 us each beside the other rows') and a draw.
#include <atomic>

#include "pkv.h"
#include "pkv_launch.h"

namespace pkv {
namespace {

constexpr int kMaxWarps = 16;
constexpr int kMaxCluster = 8;
constexpr int kNodes = PKV_MAX_TREE_NODES;
constexpr int kDepth = 6;  // granules of each row in flight per thread

struct VerifyParams {
  const void* target;
  const void* draft;
  const int32_t* tokens;
  const int32_t* parents;
  const int32_t* tree_lens;
  const float* u_accept;
  const float* u_sample;
  int32_t* path;
  int32_t* out_tokens;
  int32_t* n_accepted;
  int32_t* dev_err;
  int n_nodes;
  int vocab;
  int cluster;  // CTAs per row
};

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
// (for a barrier that orders no writes)
__device__ __forceinline__ void cluster_arrive_relaxed() {
  asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  cluster_wait();
}
// Unevaluated sum of two floats.
struct Pair {
  float hi, lo;
};

// s = a + b, with the rounding error of s (exact whatever their magnitudes).
__device__ __forceinline__ Pair two_sum(float a, float b) {
  const float s = __fadd_rn(a, b);
  const float bb = __fsub_rn(s, a);
  return {s, __fadd_rn(__fsub_rn(a, __fsub_rn(s, bb)), __fsub_rn(b, bb))};
}

// Negative and NaN entries count as 0.
__device__ __forceinline__ float clean(float x) { return fmaxf(x, 0.f); }

// max(p - (ah + al) q, 0)
__device__ __forceinline__ Pair residual(float p, float q, float ah, float al) {
  const float prod = __fmul_rn(ah, q);
  const float perr = __fmaf_rn(ah, q, -prod);
  const Pair d = two_sum(p, -prod);
  const float lo = __fsub_rn(__fsub_rn(d.lo, perr), __fmul_rn(al, q));
  const Pair r = two_sum(d.hi, lo);
  const bool pos = r.hi > 0.f;
  if (p == INFINITY) return {p, 0.f};  // (the sum tells)
  return {pos ? r.hi : 0.f, pos ? r.lo : 0.f};
}

__device__ __forceinline__ void add(Pair& s, const Pair& x) {
  const Pair t = two_sum(s.hi, x.hi);
  s.hi = t.hi;
  s.lo = __fadd_rn(s.lo, __fadd_rn(t.lo, x.lo));
}

__device__ __forceinline__ Pair shfl_xor(const Pair& x, int o) {
  return {__shfl_xor_sync(0xffffffffu, x.hi, o), __shfl_xor_sync(0xffffffffu, x.lo, o)};
}

// Sum over each kLanes lanes of the warp, the same bits in all of them: the two
// partners of a step add in one order.
template <int kLanes = 32>
__device__ __forceinline__ Pair warp_sum(Pair x, int lane) {
#pragma unroll
  for (int o = 1; o < kLanes; o <<= 1) {
    const Pair y = shfl_xor(x, o);
    Pair a = (lane & o) ? y : x;
    add(a, (lane & o) ? x : y);
    x = a;
  }
  return x;
}

// Two sums at once: shuffles stay in program order, so that one sum's would wait for
// the other's additions.
template <int kLanes>
__device__ __forceinline__ void warp_sum2(Pair& x, Pair& y, int lane) {
#pragma unroll
  for (int o = 1; o < kLanes; o <<= 1) {
    const Pair u = shfl_xor(x, o), v = shfl_xor(y, o);
    const bool up = lane & o;
    Pair a = up ? u : x, b = up ? v : y;
    add(a, up ? x : u);
    add(b, up ? y : v);
    x = a;
    y = b;
  }
}

// Inclusive running sums over the lanes, for lanes below kLanes.
template <int kLanes>
__device__ __forceinline__ Pair scan(Pair x, int lane) {
#pragma unroll
  for (int o = 1; o < kLanes; o <<= 1) {
    Pair y = {__shfl_up_sync(0xffffffffu, x.hi, o), __shfl_up_sync(0xffffffffu, x.lo, o)};
    if (lane >= o) {
      add(y, x);
      x = y;
    }
  }
  return x;
}

__device__ __forceinline__ Pair shfl(const Pair& x, int from) {
  return {__shfl_sync(0xffffffffu, x.hi, from), __shfl_sync(0xffffffffu, x.lo, from)};
}

__device__ __forceinline__ Pair times(const Pair& a, const Pair& b) {
  const float prod = __fmul_rn(a.hi, b.hi);
  float err = __fmaf_rn(a.hi, b.hi, -prod);
  err = __fmaf_rn(a.hi, b.lo, __fmaf_rn(a.lo, b.hi, err));
  return two_sum(prod, err);
}

// max(a - b, 0); NaN stays
__device__ __forceinline__ Pair minus(const Pair& a, const Pair& b) {
  const Pair d = two_sum(a.hi, -b.hi);
  const Pair r = two_sum(d.hi, __fadd_rn(d.lo, __fsub_rn(a.lo, b.lo)));
  return r.hi < 0.f ? Pair{0.f, 0.f} : r;
}

// *(the same shared-memory location in CTA `rank` of the cluster) = v
__device__ __forceinline__ void cluster_store(Pair* at, uint32_t rank, const Pair& v) {
  uint32_t remote;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(smem_u32(at)), "r"(rank));
  asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(remote), "f"(v.hi), "f"(v.lo)
               : "memory");
}

// Two floats per instruction.
using Two = unsigned long long;
__device__ __forceinline__ Two pack2(float a, float b) {
  Two r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void unpack2(Two v, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ Two add2(Two a, Two b) {
  Two r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ Two fma2(Two a, Two b, Two c) {
  Two r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

// Two running pair sums side by side of x m for m of 0 or 1. They start from kBase,
// so that no summand of a probability vector passes the running sum and the
// error of each addition is the short form's three operations; values from 2 kBase
// on (of rows that sum to more than 1) are summed to fp32 accuracy.
struct Sum2 {
  static constexpr float kBase = 1.f;
  Two hi, lo;
  __device__ __forceinline__ void clear() {
    hi = pack2(kBase, kBase);
    lo = 0ull;
  }
  __device__ __forceinline__ void add(Two x, Two m) {
    const Two t = fma2(x, m, hi);
    const Two back = fma2(t, pack2(-1.f, -1.f), hi);  // hi - t, exact
    lo = add2(lo, fma2(x, m, back));
    hi = t;
  }
  __device__ __forceinline__ Pair total() const {
    Pair a, b;
    unpack2(hi, a.hi, b.hi);
    unpack2(lo, a.lo, b.lo);
    const Pair t = two_sum(__fsub_rn(a.hi, kBase), __fsub_rn(b.hi, kBase));
    return two_sum(t.hi, __fadd_rn(__fadd_rn(a.lo, b.lo), t.lo));
  }
};

// 1 where d > 0, else 0 (NaN: 0)
__device__ __forceinline__ float positive(float d) {
  float m;
  asm("set.gt.f32.f32 %0, %1, %2;" : "=f"(m) : "f"(d), "f"(0.f));
  return m;
}

// a > b, as the sums they stand for.
__device__ __forceinline__ bool above(const Pair& a, const Pair& b) {
  const Pair x = two_sum(a.hi, a.lo);
  return x.hi > b.hi || (x.hi == b.hi && x.lo > b.lo);
}

template <typename T>
struct Elem;
template <>
struct Elem<float> {
  static constexpr int kPer = 4;  // values per 16-byte granule
  static __device__ __forceinline__ float get(const float* p) { return *p; }
  // the granule with negative and NaN entries as 0, and with kFinite infinity as the
  // largest finite value
  template <bool kFinite>
  static __device__ __forceinline__ uint4 clean4(const uint4& w) {
    const auto f = [](uint32_t u) {
      const float x = fmaxf(__uint_as_float(u), 0.f);
      return __float_as_uint(kFinite ? fminf(x, 3.402823466e38f) : x);
    };
    return make_uint4(f(w.x), f(w.y), f(w.z), f(w.w));
  }
  static __device__ __forceinline__ void unpack(const uint4& w, float (&x)[4]) {
    x[0] = __uint_as_float(w.x);
    x[1] = __uint_as_float(w.y);
    x[2] = __uint_as_float(w.z);
    x[3] = __uint_as_float(w.w);
  }
};
template <>
struct Elem<__nv_bfloat16> {
  static constexpr int kPer = 8;
  static __device__ __forceinline__ float get(const __nv_bfloat16* p) { return __bfloat162float(*p); }
  template <bool kFinite>
  static __device__ __forceinline__ uint4 clean4(const uint4& w) {
    const auto f = [](uint32_t u) {
      uint32_t r;
      asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(u), "r"(0u));
      if (kFinite) asm("min.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(r), "r"(0x7F7F7F7Fu));
      return r;
    };
    return make_uint4(f(w.x), f(w.y), f(w.z), f(w.w));
  }
  static __device__ __forceinline__ void unpack(const uint4& w, float (&x)[8]) {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      x[2 * k] = bf16lo(u[k]);
      x[2 * k + 1] = bf16hi(u[k]);
    }
  }
};

// One row of `vocab` values, read in 16-byte granules from the aligned address
// at or below its start: value v sits at index v + off of the granules, and the
// first and last granule are read value by value where they hang over.
template <typename T>
struct RowView {
  const T* base;  // 16-byte aligned
  int off;        // values of the first granule in front of the row
  int end;        // off + vocab
  __device__ __forceinline__ RowView(const void* all, int64_t row, int vocab) {
    const T* start = static_cast<const T*>(all) + row * vocab;
    off = static_cast<int>((reinterpret_cast<uintptr_t>(start) & 15) / sizeof(T));
    base = start - off;
    end = off + vocab;
  }
  // granules, and those that lie inside the row: [first_whole, end_whole)
  __device__ __forceinline__ int granules() const { return (end + Elem<T>::kPer - 1) / Elem<T>::kPer; }
  __device__ __forceinline__ int first_whole() const { return off > 0 ? 1 : 0; }
  __device__ __forceinline__ int end_whole() const { return end / Elem<T>::kPer; }
  __device__ __forceinline__ bool inside(int g) const {
    return g >= first_whole() && g < end_whole();
  }
  __device__ __forceinline__ uint4 whole(int g) const {
    return *reinterpret_cast<const uint4*>(base + static_cast<int64_t>(g) * Elem<T>::kPer);
  }
  // values outside the row read as 0
  __device__ __forceinline__ void values(int g, float (&x)[Elem<T>::kPer]) const {
    if (inside(g)) {
      Elem<T>::unpack(whole(g), x);
    } else {
#pragma unroll
      for (int e = 0; e < Elem<T>::kPer; ++e) {
        const int i = g * Elem<T>::kPer + e;
        x[e] = i >= off && i < end ? Elem<T>::get(base + i) : 0.f;
      }
    }
  }
};

// What a pass sums: max(p - a q, 0) with the refused tokens left out.
struct Residual {
  Pair a;
  int n_refused;
};

enum : int { kSum, kDraw, kLeave };

struct Shared {
  int parent[kNodes], token[kNodes];
  float p[kNodes], q[kNodes], u[kNodes];
  int path[kNodes];
  int refused[kNodes];                // tokens refused at the current node (no draft rows)
  Pair warp_p[kMaxWarps];             // sums of p and q over the residual's tokens of the
  Pair warp_q[kMaxWarps];             // last pass, this CTA's warps
  Pair cta_sum[2][kMaxCluster];       // the residual's, of the last two passes, all CTAs
  // the walking warp's order to the others
  int order, node, n_refused, draw_warp, count;
  int first[kMaxWarps], last[kMaxWarps];  // of the draw, lanes per warp
  Pair a;
  Pair draw_at;  // how far into the draw's warp
};

template <typename T, bool kDraft, int kWarps>
struct Walk {
  const VerifyParams& p;
  Shared& s;
  const int64_t row0;  // this sequence's first row
  const uint32_t rank;
  const int lane, warp;
  uint4* ring;  // this thread's slots: [kDepth][p, q], kThreads apart
  int passes = 0;
  int held = -1;        // node whose rows the ring holds whole, -1: none
  bool held_q = false;  // the draft's too
  static constexpr int kThreads = kWarps * 32;

  // granules [g0, g1) of a row are warp wp's of this CTA
  // Whether a part fits the ring (the same for all warps).
  __device__ __forceinline__ bool range_of(const RowView<T>& v, int wp, int& g0, int& g1) const {
    const int total = v.granules();
    const int warps = p.cluster * kWarps;
    // (a division by warps, a power of two)
    const int per = (((total + warps - 1) >> (31 - __clz(warps))) + 31) / 32 * 32;
    const int64_t w = static_cast<int64_t>(rank) * kWarps + wp;
    g0 = static_cast<int>(w * per < total ? w * per : total);
    g1 = static_cast<int>((w + 1) * per < total ? (w + 1) * per : total);
    return per <= 32 * kDepth;
  }

  // Sums of p and q over the tokens with p > a q, a granule at a time.
  struct Sums {
    static constexpr int E = Elem<T>::kPer;
    Sum2 ps, qs;
    Two mah, mal;
    bool with_q;
    __device__ __forceinline__ Sums(const Pair& a, bool with)
        : mah(pack2(-a.hi, -a.hi)), mal(pack2(-a.lo, -a.lo)), with_q(with) {
      ps.clear();
      qs.clear();
    }
    // x, y: cleaned p and q of the tokens from `first` on
    __device__ __forceinline__ void take(const Shared& s, int first, const float (&x)[E],
                                         const float (&y)[E]) {
      if (with_q) {
#pragma unroll
        for (int e = 0; e < E; e += 2) {
          // p - a q to single rounding twice: its sign is that of the exact
          // difference unless that is below 2^-48 of its terms
          const Two x2 = pack2(x[e], x[e + 1]), y2 = pack2(y[e], y[e + 1]);
          float d0, d1;
          unpack2(fma2(mal, y2, fma2(mah, y2, x2)), d0, d1);
          const Two m = pack2(positive(d0), positive(d1));
          ps.add(x2, m);  // (an infinite p tells itself by the sum)
          qs.add(y2, m);
        }
      } else {
        float z[E];
#pragma unroll
        for (int e = 0; e < E; ++e) z[e] = 1.f;
        if constexpr (!kDraft) {
          for (int k = 0; k < s.n_refused; ++k) {
            const int at = s.refused[k] - first;
#pragma unroll
            for (int e = 0; e < E; ++e)
              if (at == e) z[e] = 0.f;
          }
        }
#pragma unroll
        for (int e = 0; e < E; e += 2) ps.add(pack2(x[e], x[e + 1]), pack2(z[e], z[e + 1]));
      }
    }
  };

  // This warp's part of the ordered sums: p and q over the tokens with p > a q.
  // A thread's granules come through kDepth slots of its own in shared memory, so
  // that a row's pass waits for memory about once (with four loads in flight
  // per thread a pass of few rows took 6.5 us for 76 KB per CTA, all of it latency).
  __device__ __forceinline__ void sum_part() {
    const RowView<T> pv(p.target, row0 + s.node, p.vocab);
    const RowView<T> qv(kDraft ? p.draft : p.target, row0 + s.node, p.vocab);
    const bool with_q = kDraft && s.a.hi != 0.f;
    int g0, g1;
    const bool fits = range_of(pv, warp, g0, g1);
    // a node's later passes find its rows where the first one left them (14.0 -> 12.7 us
    // for 12 rows; reading the draw's part from there too cost registers, and 2 %)
    const bool have = fits && held == s.node && (held_q || !with_q);
    constexpr int E = Elem<T>::kPer;
    Sums acc(s.a, with_q);
    const uint4* from_p = reinterpret_cast<const uint4*>(pv.base) + lane;
    const uint4* from_q = reinterpret_cast<const uint4*>(qv.base) + lane;
    // (the last granule may hang over the row's end: what lies behind it reads as 0)
    auto fetch = [&](int g, int slot) {
      if (g + lane < g1) {
        // (by the values that hang over: the bytes left of a row pass 32 bits)
        const int over = max((g + lane + 1) * E - pv.end, 0);
        const int bytes = 16 - over * static_cast<int>(sizeof(T));
        cp_async16_fill(ring + (2 * slot) * kThreads, from_p + g, bytes);
        if (with_q) cp_async16_fill(ring + (2 * slot + 1) * kThreads, from_q + g, bytes);
      }
      cp_async_commit();
    };
#pragma unroll
    for (int k = 0; k < kDepth; ++k)
      if (!have) fetch(g0 + 32 * k, k);
    int slot = 0;
    for (int g = g0; g < g1; g += 32) {
      cp_async_wait<kDepth - 1>();
      if (g + lane < g1) {
        float x[E], y[E];
        // (0 x infinity is not 0: q is made finite)
        const uint4 yw = with_q ? ring[(2 * slot + 1) * kThreads] : make_uint4(0u, 0u, 0u, 0u);
        Elem<T>::unpack(Elem<T>::template clean4<false>(ring[(2 * slot) * kThreads]), x);
        Elem<T>::unpack(Elem<T>::template clean4<true>(yw), y);
        if (g + lane == 0) {  // the row before ends in the first granule
#pragma unroll
          for (int e = 0; e < E; ++e)
            if (e < pv.off) x[e] = 0.f;
        }
        acc.take(s, (g + lane) * E - pv.off, x, y);
      }
      fetch(g + 32 * kDepth, slot);  // (the slot's values have been used)
      slot = slot + 1 < kDepth ? slot + 1 : 0;
    }
    cp_async_wait<0>();
    held_q = with_q || (have && held_q);
    held = fits ? s.node : -1;
    Pair sp = acc.ps.total(), sq = {0.f, 0.f};
    if (with_q) {
      sq = acc.qs.total();
      warp_sum2<32>(sp, sq, lane);
    } else {
      sp = warp_sum(sp, lane);
    }
    if (lane == 0) {
      s.warp_p[warp] = sp;
      s.warp_q[warp] = sq;
    }
  }

  // The walking warp: sum of the residual at node c over the whole vocabulary,
  // the same bits in every lane of every CTA of the cluster.
  __device__ Pair sum(int c, const Residual& r) {
    if (lane == 0) {
      s.order = kSum;
      s.node = c;
      s.n_refused = r.n_refused;
      s.a = r.a;
    }
    __syncthreads();
    sum_part();
    __syncthreads();
    // (every kWarps lanes add the same numbers in the same order)
    Pair sp = s.warp_p[lane % kWarps], sq = s.warp_q[lane % kWarps];
    warp_sum2<kWarps>(sp, sq, lane);
    const Pair mine = minus(sp, times(r.a, sq));
    Pair* slots = s.cta_sum[passes & 1];
    if (lane < p.cluster) cluster_store(&slots[rank], lane, mine);
    // one barrier per pass: the next pass writes the other half, and the one
    // after that follows a barrier that every CTA reaches after these reads
    __syncwarp();
    cluster_sync();
    ++passes;
    const int at = lane % kMaxCluster;
    return warp_sum<kMaxCluster>(at < p.cluster ? slots[at] : Pair{0.f, 0.f}, lane);
  }

  // The walking warp: which CTA and warp hold the token drawn at t of the last
  // pass's sum, and what lies in front of them: the first whose running sum passes
  // t, or where rounding leaves none the last one with any mass.
  __device__ __forceinline__ void place(const Pair& t, const Residual& r) {
    const Pair none = {0.f, 0.f};
    const Pair of_cta = lane < p.cluster ? s.cta_sum[(passes - 1) & 1][lane] : none;
    const Pair of_warp =
        lane < kWarps ? minus(s.warp_p[lane], times(r.a, s.warp_q[lane])) : none;
    const Pair ctas = scan<kMaxCluster>(of_cta, lane), warps = scan<kMaxWarps>(of_warp, lane);
    Pair base = none;
    const int cta = pick(of_cta.hi > 0.f, ctas, t, base);
    int w = -1;
    // (a sum above 0 has a token with p > a q in it, whatever its parts round to)
    if (static_cast<int>(rank) == cta)
      w = pick(lane < kWarps && s.warp_p[lane].hi > 0.f, warps, t, base);
    if (lane == 0) {
      s.order = kDraw;
      s.draw_warp = w;
      s.draw_at = minus(t, base);
    }
  }

  // Lane of the first running sum past t (from `base` on), else the last lane that
  // has any token of the residual; base becomes the sum in front of it.
  __device__ __forceinline__ int pick(bool has, const Pair& incl, const Pair& t,
                                      Pair& base) const {
    Pair here = base;
    add(here, incl);
    const uint32_t past = __ballot_sync(0xffffffffu, has && above(here, t));
    const uint32_t some = __ballot_sync(0xffffffffu, has);
    const int at = past != 0u ? __ffs(past) - 1 : 31 - __clz(some | 1u);
    if (at > 0) add(base, shfl(incl, at - 1));
    return at;
  }

  // The ordered draw, by all threads of the CTA that holds the token, over the
  // granules of the warp that held it in the pass: each thread sums a few of them,
  // the running sums pick the thread, and its warp looks at that thread's values, one
  // per lane. (One warp alone took 10 us for its 300 granules.) Returns the token in
  // one thread, -1 in the others.
  __device__ int draw() {
    const RowView<T> pv(p.target, row0 + s.node, p.vocab);
    const RowView<T> qv(kDraft ? p.draft : p.target, row0 + s.node, p.vocab);
    const Pair t = s.draw_at;
    int g0, g1;
    range_of(pv, s.draw_warp, g0, g1);
    constexpr int E = Elem<T>::kPer;
    const int per = (g1 - g0 + kWarps * 32 - 1) / (kWarps * 32);
    const int a0 = min(g0 + (32 * warp + lane) * per, g1), a1 = min(a0 + per, g1);
    const bool with_q = kDraft && s.a.hi != 0.f;
    // a granule that lies inside the row comes as it was loaded, in xw and yw
    auto cleaned = [&](int g, const uint4& xw, const uint4& yw, float (&x)[E], float (&y)[E]) {
      Elem<T>::unpack(xw, x);
      Elem<T>::unpack(yw, y);
      if (!pv.inside(g)) {
        pv.values(g, x);
        if (with_q) qv.values(g, y);
      }
#pragma unroll
      for (int e = 0; e < E; ++e) {
        x[e] = clean(x[e]);
        y[e] = fminf(clean(y[e]), 3.402823466e38f);
      }
    };
    const uint4 none = make_uint4(0u, 0u, 0u, 0u);
    auto raw_p = [&](int g) { return g < a1 && pv.inside(g) ? pv.whole(g) : none; };
    auto raw_q = [&](int g) { return with_q && g < a1 && qv.inside(g) ? qv.whole(g) : none; };
    Sums sums(s.a, with_q);
    for (int g = a0; g < a1; g += 2) {
      const uint4 xw[2] = {raw_p(g), raw_p(g + 1)}, yw[2] = {raw_q(g), raw_q(g + 1)};
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        if (g + k >= a1) break;
        float x[E], y[E];
        cleaned(g + k, xw[k], yw[k], x, y);
        sums.take(s, (g + k) * E - pv.off, x, y);
      }
    }
    const Pair all_p = sums.ps.total();
    const bool has = all_p.hi > 0.f;
    const Pair acc = minus(all_p, times(s.a, sums.qs.total()));
    const Pair incl = scan<32>(acc, lane);
    if (lane == 31) s.warp_p[warp] = incl;
    __syncthreads();
    // what lies in front of this warp, then of this thread
    const Pair warps = scan<kMaxWarps>(lane < kWarps ? s.warp_p[lane] : Pair{0.f, 0.f}, lane);
    Pair front = shfl(warps, max(warp - 1, 0));
    if (warp == 0) front = {0.f, 0.f};
    Pair here = front;
    add(here, incl);
    const uint32_t past = __ballot_sync(0xffffffffu, has && above(here, t));
    const uint32_t some = __ballot_sync(0xffffffffu, has);
    if (lane == 0) {
      s.first[warp] = past != 0u ? __ffs(past) - 1 : -1;
      s.last[warp] = some != 0u ? 31 - __clz(some) : -1;
    }
    __syncthreads();
    // the first thread whose running sum passes t, else the last with any mass
    const int f = lane < kWarps ? s.first[lane] : -1, e = lane < kWarps ? s.last[lane] : -1;
    const uint32_t fs = __ballot_sync(0xffffffffu, f >= 0), es = __ballot_sync(0xffffffffu, e >= 0);
    const int w = fs != 0u ? __ffs(fs) - 1 : 31 - __clz(es | 1u);
    const int l = __shfl_sync(0xffffffffu, fs != 0u ? f : e, w);
    // that thread's values again, one per lane of its warp
    int at = -1;
    if (warp == w) {
      const Pair up = {__shfl_up_sync(0xffffffffu, incl.hi, 1),
                       __shfl_up_sync(0xffffffffu, incl.lo, 1)};
      if (lane > 0) add(front, up);
      Pair at_front = shfl(front, l);
      const int v0 = max(__shfl_sync(0xffffffffu, a0, l) * E, pv.off);
      const int v1 = min(__shfl_sync(0xffffffffu, a1, l) * E, pv.end);
      for (int v = v0; v < v1; v += 32) {
        const int i = v + lane;
        Pair term = {0.f, 0.f};
        bool in = false;
        if (i < v1) {
          const float x = clean(Elem<T>::get(pv.base + i));
          if constexpr (kDraft) {
            const float y = with_q ? clean(Elem<T>::get(qv.base + i)) : 0.f;
            term = residual(x, y, s.a.hi, s.a.lo);
            // (the pass's own test, so that a residual with any token has one here)
            in = fmaf(-s.a.lo, y, fmaf(-s.a.hi, y, x)) > 0.f;
          } else {
            in = x > 0.f;
            for (int k = 0; k < s.n_refused; ++k) in = in && s.refused[k] + pv.off != i;
            if (in) term.hi = x;
          }
        }
        const Pair run = scan<32>(term, lane);
        Pair upto = at_front;
        add(upto, run);
        const uint32_t over = __ballot_sync(0xffffffffu, in && above(upto, t));
        const uint32_t any = __ballot_sync(0xffffffffu, in);
        // the first past t, or the last with mass where rounding leaves none
        if (any != 0u) at = v - pv.off + (over != 0u ? __ffs(over) - 1 : 31 - __clz(any));
        if (over != 0u) break;
        add(at_front, shfl(run, 31));
      }
      if (lane != 0) at = -1;
    }
    return at;
  }
};

template <typename T, bool kDraft, int kWarps>
__global__ void __launch_bounds__(kWarps * 32, 1024 / (kWarps * 32))
verify_tree_kernel(const VerifyParams p) {
  constexpr int kThreads = kWarps * 32;
  __shared__ Shared s;
  extern __shared__ __align__(16) uint4 ring[];
  pdl_wait_primary();
  const uint32_t rank = cluster_rank();
  const int b = blockIdx.x / p.cluster;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int N = p.n_nodes;
  const int64_t n0 = static_cast<int64_t>(b) * N;
  // the trees' numbers, in flight together with the tree's size
  int err = 0;
  int parent = -1, tok = 0;
  float u = 0.f;
  if (threadIdx.x >= 1 && static_cast<int>(threadIdx.x) < N) {
    parent = p.parents[n0 + threadIdx.x];
    tok = p.tokens[n0 + threadIdx.x];
    u = p.u_accept[n0 + threadIdx.x];
  }
  int len = p.tree_lens[b];
  if (len < 0 || len > N) {
    err = PKV_DEV_ERR_BAD_TREE;
    len = 0;
  }
  if (len == 0) {  // the whole cluster leaves together
    if (rank == 0) {
      for (int i = threadIdx.x; i < N; i += kThreads) p.path[n0 + i] = p.out_tokens[n0 + i] = -1;
      if (threadIdx.x == 0) {
        p.n_accepted[b] = 0;
        if (err) set_dev_err(p.dev_err, err);
      }
      __threadfence();
    }
    return;
  }
  // A CTA's shared memory may be written by the others once it is known to have
  // started: every thread says so here, and the gather covers the wait below. (A
  // releasing arrive took 0.2 to 0.4 us of a call, waiting behind the first pass
  // gained nothing.)
  __syncwarp();
  cluster_arrive_relaxed();
  if (threadIdx.x < kNodes) {
    const int i = threadIdx.x;
    float px = 0.f, qx = 0.f;
    if (i < 1 || i >= len) {
      parent = -1;
    } else {
      if (parent < -1 || parent >= i || tok < 0 || tok >= p.vocab) {
        err = PKV_DEV_ERR_BAD_TREE;
        parent = -1;
      }
      if (parent >= 0) {
        const int64_t at = (n0 + parent) * p.vocab + tok;
        px = clean(Elem<T>::get(static_cast<const T*>(p.target) + at));
        qx = kDraft ? clean(Elem<T>::get(static_cast<const T*>(p.draft) + at)) : 1.f;
      }
      if (err && rank == 0) set_dev_err(p.dev_err, err);
    }
    s.parent[i] = parent;
    s.token[i] = tok;
    s.p[i] = px;
    s.q[i] = qx;
    s.u[i] = u;
  }
  __syncthreads();
  cluster_wait();  // before any sum is stored to another CTA

  const float u_sample = p.u_sample[b];
  Walk<T, kDraft, kWarps> walk{p, s, n0, rank, lane, warp, ring + threadIdx.x};
  int count = 1;
  bool ok = false;
  if (warp == 0) {
    const int par0 = s.parent[lane], par1 = s.parent[lane + 32];
    int cur = 0;
    uint64_t on_path = 1;
    Residual r = {{0.f, 0.f}, 0};
    Pair mass = {1.f, 0.f};
    bool summed = false;  // the last pass summed the residual at hand
    while (true) {
      uint64_t kids = static_cast<uint64_t>(__ballot_sync(0xffffffffu, par0 == cur)) |
                      static_cast<uint64_t>(__ballot_sync(0xffffffffu, par1 == cur)) << 32;
      int next = -1;
      while (kids != 0) {
        const int x = __ffsll(static_cast<long long>(kids)) - 1;
        kids &= kids - 1;
        Pair rx = {s.p[x], 0.f};
        bool take;
        if (r.a.hi == 0.f && r.n_refused == 0) {
          // a node's first child, R = 1: u q against p, exactly
          const float prod = __fmul_rn(s.u[x], s.q[x]);
          const float rest = __fmaf_rn(s.u[x], s.q[x], -prod);
          take = prod < s.p[x] || (prod == s.p[x] && rest < 0.f);
        } else {
          if constexpr (kDraft) {
            rx = residual(s.p[x], s.q[x], r.a.hi, r.a.lo);
          } else {
            for (int k = 0; k < r.n_refused; ++k)
              if (s.refused[k] == s.token[x]) rx.hi = 0.f;
          }
          take = above(rx, times(times({s.u[x], 0.f}, {s.q[x], 0.f}), mass));
        }
        if (take) {
          next = x;
          break;
        }
        if constexpr (kDraft) {
          add(r.a, mass);
          r.a = two_sum(r.a.hi, r.a.lo);
          mass = walk.sum(cur, r);
          summed = true;
        } else {
          mass = minus(mass, rx);
          __syncwarp();
          if (lane == 0) s.refused[r.n_refused] = s.token[x];
          __syncwarp();
          ++r.n_refused;
        }
      }
      if (next < 0) break;
      cur = next;
      ++count;
      on_path |= 1ull << next;
      r = {{0.f, 0.f}, 0};
      mass = {1.f, 0.f};
      summed = false;
    }
    Pair total = summed ? mass : walk.sum(cur, r);
    if (total.hi == 0.f && (r.a.hi != 0.f || r.n_refused != 0)) {
      r = {{0.f, 0.f}, 0};  // nothing of the target is left: draw from all of it
      total = walk.sum(cur, r);
    }
    ok = total.hi > 0.f && total.hi <= 3.402823466e38f;
    if (ok) walk.place(times({u_sample, 0.f}, total), r);
    else if (lane == 0) s.order = kLeave;
    if (lane == 0) s.count = count;
    __syncthreads();
    if (rank == 0) {
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int i = lane + 32 * k;
        if ((on_path >> i) & 1ull) s.path[__popcll(on_path & ((1ull << i) - 1ull))] = i;
      }
      __syncwarp();
      for (int i = lane; i < N; i += 32) {
        p.path[n0 + i] = i < count ? s.path[i] : -1;
        if (i != count - 1) p.out_tokens[n0 + i] = i < count - 1 ? s.token[s.path[i + 1]] : -1;
      }
      if (lane == 0) {
        p.n_accepted[b] = count;
        if (!ok) {
          p.out_tokens[n0 + count - 1] = -1;
          set_dev_err(p.dev_err, PKV_DEV_ERR_BAD_PROBS);
        }
      }
    }
  } else {
    while (true) {
      __syncthreads();
      if (s.order != kSum) break;
      walk.sum_part();
      __syncthreads();
      cluster_sync();
    }
    count = s.count;
  }
  if (s.order == kDraw && s.draw_warp >= 0) {  // (the same in the whole CTA)
    const int drawn = walk.draw();
    if (drawn >= 0) p.out_tokens[n0 + count - 1] = drawn;
  }
  // a programmatic dependent may read the results before this grid has drained
  __threadfence();
}

// CTAs per row: a CTA reads about 60 bytes a cycle, so a long vocabulary is
// spread over eight of them.
int pick_cluster(int vocab) {
  int c = 1;
  while (c < kMaxCluster && vocab > c * 4096) c *= 2;
  return c;
}

template <typename T, bool kDraft, int kWarps>
cudaError_t launch(const VerifyParams& p, int batch, int dev, cudaStream_t stream) {
  constexpr int kRingBytes = kDepth * 2 * kWarps * 32 * 16;
  // the shared-memory opt-in, once per device; host threads may race to set it
  static std::atomic<bool> attr_set[64] = {};
  if (!attr_set[dev].load(std::memory_order_acquire)) {
    const cudaError_t e = cudaFuncSetAttribute(verify_tree_kernel<T, kDraft, kWarps>,
                                               cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               kRingBytes);
    if (e != cudaSuccess) return e;
    attr_set[dev].store(true, std::memory_order_release);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(batch) * p.cluster);
  cfg.blockDim = dim3(kWarps * 32);
  cfg.dynamicSmemBytes = kRingBytes;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = p.cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, verify_tree_kernel<T, kDraft, kWarps>, p);
}

// 16 warps a CTA while two CTAs per SM hold every row's cluster, else 8 (four CTAs
// per SM): more warps shorten a row's pass, more CTAs keep the rows in one wave.
template <typename T, bool kDraft>
cudaError_t launch_for(const VerifyParams& p, int batch, int sms, int dev, cudaStream_t stream) {
  return static_cast<int64_t>(batch) * p.cluster <= 2 * sms
             ? launch<T, kDraft, 16>(p, batch, dev, stream)
             : launch<T, kDraft, 8>(p, batch, dev, stream);
}

bool aligned(const void* q, uintptr_t a) { return (reinterpret_cast<uintptr_t>(q) % a) == 0; }

}  // namespace
}  // namespace pkv

extern "C" pkv_status pkv_verify_tree(const void* target_probs, const void* draft_probs,
                                      int probs_type, int vocab, const int32_t* draft_tokens,
                                      const int32_t* parents, const int32_t* tree_lens,
                                      const float* u_accept, const float* u_sample, int batch,
                                      int n_nodes, int32_t* path, int32_t* tokens,
                                      int32_t* n_accepted, int32_t* dev_err,
                                      cudaStream_t stream) {
  using namespace pkv;
  if (probs_type != PKV_PROBS_FP32 && probs_type != PKV_PROBS_BF16) return PKV_ERR_ARG;
  if (batch < 0 || batch > (1 << 24) || n_nodes < 1 || n_nodes > PKV_MAX_TREE_NODES)
    return PKV_ERR_ARG;
  if (vocab < 1 || vocab > (1 << 30)) return PKV_ERR_ARG;
  if (batch == 0) return PKV_OK;
  if (!target_probs || !draft_tokens || !parents || !tree_lens || !u_accept || !u_sample || !path ||
      !tokens || !n_accepted)
    return PKV_ERR_ARG;
  if (!aligned(target_probs, 16) || !aligned(draft_probs, 16) || !aligned(draft_tokens, 4) ||
      !aligned(parents, 4) || !aligned(tree_lens, 4) || !aligned(u_accept, 4) ||
      !aligned(u_sample, 4) || !aligned(path, 4) || !aligned(tokens, 4) ||
      !aligned(n_accepted, 4) || !aligned(dev_err, 4))
    return PKV_ERR_ALIGN;
  int sms = 0;
  const pkv_status st = device_info(&sms);
  if (st != PKV_OK) return st;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return PKV_ERR_DEVICE;
  VerifyParams p;
  p.target = target_probs;
  p.draft = draft_probs;
  p.tokens = draft_tokens;
  p.parents = parents;
  p.tree_lens = tree_lens;
  p.u_accept = u_accept;
  p.u_sample = u_sample;
  p.path = path;
  p.out_tokens = tokens;
  p.n_accepted = n_accepted;
  p.dev_err = dev_err;
  p.n_nodes = n_nodes;
  p.vocab = vocab;
  p.cluster = pick_cluster(vocab);
  cudaError_t e;
  if (probs_type == PKV_PROBS_FP32)
    e = draft_probs ? launch_for<float, true>(p, batch, sms, dev, stream)
                    : launch_for<float, false>(p, batch, sms, dev, stream);
  else
    e = draft_probs ? launch_for<__nv_bfloat16, true>(p, batch, sms, dev, stream)
                    : launch_for<__nv_bfloat16, false>(p, batch, sms, dev, stream);
  return record_cuda_status(e);
}
