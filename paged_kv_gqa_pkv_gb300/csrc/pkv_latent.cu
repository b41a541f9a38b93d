// pkv_latent.cu - rotary positions through strides, and the rows of a paged cache of
// shared latents: appended with their norm and rotation, read back by sequence.
//
// All three move every byte once and compute next to nothing, so memory bounds them:
// 16-byte accesses, several independent ones in flight per thread, and no more than
// one launch.
#include <cfloat>
#include <cmath>

#include "pkv_latent.cuh"

namespace pkv {
namespace {

using namespace latent;

// a*c - b*s and a*c + b*s to about one fp32 ulp of the result even where the two
// products nearly cancel: the rounding error of b*s is kept exactly (an FMA) and
// folded back in after the fused multiply-add. (Of an infinite b*s the error is
// inf - inf. The sum is infinite or NaN there, so any finite number will do.)
__device__ __forceinline__ float product_error(float b, float s, float p) {
  return fmaxf(fmaf(b, s, -p), -FLT_MAX);
}
__device__ __forceinline__ float turn_diff(float a, float c, float b, float s) {
  const float p = b * s;
  return fmaf(a, c, -p) - product_error(b, s, p);
}
__device__ __forceinline__ float turn_sum(float a, float c, float b, float s) {
  const float p = b * s;
  return fmaf(a, c, p) + product_error(b, s, p);
}

__device__ __forceinline__ void unpack8(const uint4& v, float (&x)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    x[2 * u] = bf16lo(w[u]);
    x[2 * u + 1] = bf16hi(w[u]);
  }
}
__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
  return make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                    pack_bf16x2(x[6], x[7]));
}

// Eight neighbouring values as four interleaved pairs.
__device__ __forceinline__ void turn_pairs(float (&x)[8], const float4& c, const float4& s) {
  const float cv[4] = {c.x, c.y, c.z, c.w}, sv[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    const float a = x[2 * u], b = x[2 * u + 1];
    x[2 * u] = turn_diff(a, cv[u], b, sv[u]);
    x[2 * u + 1] = turn_sum(b, cv[u], a, sv[u]);
  }
}
// Eight values of the first half with their partners of the second.
__device__ __forceinline__ void turn_halves(float (&x)[8], float (&y)[8], const float4 (&c)[2],
                                            const float4 (&s)[2]) {
  const float cv[8] = {c[0].x, c[0].y, c[0].z, c[0].w, c[1].x, c[1].y, c[1].z, c[1].w};
  const float sv[8] = {s[0].x, s[0].y, s[0].z, s[0].w, s[1].x, s[1].y, s[1].z, s[1].w};
#pragma unroll
  for (int u = 0; u < 8; ++u) {
    const float a = x[u], b = y[u];
    x[u] = turn_diff(a, cv[u], b, sv[u]);
    y[u] = turn_sum(b, cv[u], a, sv[u]);
  }
}

// ------------------------------------------------------------------- rotate --

struct RotateParams {
  const __nv_bfloat16* x;
  __nv_bfloat16* out;
  long long x_token, x_head, out_token, out_head;  // strides, in values
  const int32_t* positions;
  const float* rope_cos;
  const float* rope_sin;
  int32_t* dev_err;
  int n_tokens;
  int num_heads;
  int dims;
  int rope_len;
  int units;        // units of work of one head: 16-byte pieces, pairs of them, or pairs of values
  int head_groups;  // ceil(num_heads / kRotateHeads)
};

constexpr int kRotateThreads = 128;
// Heads per thread: they share the position's cosines and sines, which are read once
// into registers, and their loads are all in flight together.
constexpr int kRotateHeads = 2;

enum RotateForm { kPairs16, kHalves16, kPairs1, kHalves1 };

// A thread turns one unit of kRotateHeads heads of one token. The 16-byte forms take
// 8 values (interleaved) or 8 values and their 8 partners (halves); where an address,
// a stride or the number of dims does not allow that, a unit is one pair of values.
// Memory bounds it: 8191 tokens of 32 heads (69 MB) in 12.3 us, 5.6 TB/s with the launch (one head
// a thread 13.9, four 12.4; CTAs of 256 threads, which come to 2.3 waves, 13.4).
template <RotateForm kForm>
__global__ void __launch_bounds__(kRotateThreads) rotate_kernel(const RotateParams p) {
  pdl_wait_primary();
  pdl_launch_dependents();
  const long long id = static_cast<long long>(blockIdx.x) * kRotateThreads + threadIdx.x;
  const long long per_token = static_cast<long long>(p.units) * p.head_groups;
  const long long token = id / per_token;
  if (token >= p.n_tokens) return;
  const int rest = static_cast<int>(id - token * per_token);
  const int group = rest / p.units;
  const int u = rest - group * p.units;
  const int pos = __ldg(p.positions + token);
  if (pos < 0 || pos >= p.rope_len) {
    if (rest == 0) set_dev_err(p.dev_err, PKV_DEV_ERR_BAD_POS);
    return;
  }
  const int half = p.dims >> 1;
  const float* cs = p.rope_cos + static_cast<long long>(pos) * half;
  const float* sn = p.rope_sin + static_cast<long long>(pos) * half;
  const int h0 = group * kRotateHeads;
  const __nv_bfloat16* x = p.x + token * p.x_token + h0 * p.x_head;
  __nv_bfloat16* out = p.out + token * p.out_token + h0 * p.out_head;
  const int n = min(kRotateHeads, p.num_heads - h0);
  if constexpr (kForm == kPairs16) {
    uint4 v[kRotateHeads];
#pragma unroll
    for (int h = 0; h < kRotateHeads; ++h)
      if (h < n) v[h] = *reinterpret_cast<const uint4*>(x + h * p.x_head + 8 * u);
    const float4 c = __ldg(reinterpret_cast<const float4*>(cs) + u);
    const float4 s = __ldg(reinterpret_cast<const float4*>(sn) + u);
#pragma unroll
    for (int h = 0; h < kRotateHeads; ++h) {
      if (h >= n) break;
      float f[8];
      unpack8(v[h], f);
      turn_pairs(f, c, s);
      *reinterpret_cast<uint4*>(out + h * p.out_head + 8 * u) = pack8(f);
    }
  } else if constexpr (kForm == kHalves16) {
    uint4 a[kRotateHeads], b[kRotateHeads];
#pragma unroll
    for (int h = 0; h < kRotateHeads; ++h) {
      if (h >= n) break;
      a[h] = *reinterpret_cast<const uint4*>(x + h * p.x_head + 8 * u);
      b[h] = *reinterpret_cast<const uint4*>(x + h * p.x_head + half + 8 * u);
    }
    const float4* c4 = reinterpret_cast<const float4*>(cs) + 2 * u;
    const float4* s4 = reinterpret_cast<const float4*>(sn) + 2 * u;
    const float4 c[2] = {__ldg(c4), __ldg(c4 + 1)};
    const float4 s[2] = {__ldg(s4), __ldg(s4 + 1)};
#pragma unroll
    for (int h = 0; h < kRotateHeads; ++h) {
      if (h >= n) break;
      float f[8], g[8];
      unpack8(a[h], f);
      unpack8(b[h], g);
      turn_halves(f, g, c, s);
      *reinterpret_cast<uint4*>(out + h * p.out_head + 8 * u) = pack8(f);
      *reinterpret_cast<uint4*>(out + h * p.out_head + half + 8 * u) = pack8(g);
    }
  } else {
    const int d0 = kForm == kPairs1 ? 2 * u : u;
    const int d1 = kForm == kPairs1 ? 2 * u + 1 : u + half;
    const float c = __ldg(cs + u), s = __ldg(sn + u);
    for (int h = 0; h < n; ++h) {
      const float a = __bfloat162float(x[h * p.x_head + d0]);
      const float b = __bfloat162float(x[h * p.x_head + d1]);
      out[h * p.out_head + d0] = __float2bfloat16_rn(turn_diff(a, c, b, s));
      out[h * p.out_head + d1] = __float2bfloat16_rn(turn_sum(b, c, a, s));
    }
  }
}

// ------------------------------------------------------------------- append --

struct LatentAppendParams {
  __nv_bfloat16* pool;
  const int32_t* page_table;
  const __nv_bfloat16* x;
  long long x_token;  // stride of a token, in values
  const int32_t* batch_idx;
  const int32_t* input_pos;
  const float* rope_cos;
  const float* rope_sin;
  const float* norm_weight;  // null: no norm
  int32_t* dev_err;
  float norm_eps;
  int n_tokens;
  int rope_len;
  int page_size;
  int num_pages;
  int max_batch;
  int max_blocks;
};

constexpr int kAppendWarps = 4;

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// A warp takes a token: lane l holds the latent's 16-byte pieces l and l + 32, and lanes 0..7 four
// pairs each of the position part. The squares of all 512 values are summed in fp32 by shuffles (once
// more, scaled, where they leave its range); norm and rotation stay in fp32 and each value is rounded
// to bf16 once. What bounds it is the latency of two dependent reads (position, then page
// and angles) before the writes: the row is read beside the first of them, and norm and weights do
// not wait for the page. Measured in a graph: 64 tokens 2.0 us, 16384 tokens 10.2 us (38.1 MB,
// 3.7 TB/s; eight pairs a lane, for more registers and fewer warps, 10.8; CTAs of eight warps 11.5;
// two tokens a warp 13.1; the page looked at first 13.8).
template <bool kInterleaved>
__global__ void __launch_bounds__(kAppendWarps * 32)
latent_append_kernel(const LatentAppendParams p) {
  pdl_wait_primary();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int i = blockIdx.x * kAppendWarps + (threadIdx.x >> 5);
  if (i >= p.n_tokens) return;
  constexpr int kTurners = 8;  // lanes
  const int slot = __ldg(p.batch_idx + i);
  const int pos = __ldg(p.input_pos + i);
  const uint4* src = reinterpret_cast<const uint4*>(p.x + i * p.x_token);
  uint4 v0 = __ldg(src + lane), v1 = __ldg(src + 32 + lane);
  uint4 r = make_uint4(0u, 0u, 0u, 0u);  // four pairs: neighbours, or four values and their partners
  if (lane < kTurners) {
    if (kInterleaved) {
      r = __ldg(src + 64 + lane);
    } else {
      const uint2 a = __ldg(reinterpret_cast<const uint2*>(src + 64) + lane);
      const uint2 b = __ldg(reinterpret_cast<const uint2*>(src + 68) + lane);
      r = make_uint4(a.x, a.y, b.x, b.y);
    }
  }
  if (slot == 0) return;  // padding
  const int block = pos / p.page_size;
  int err = 0;
  if (slot < 0 || slot >= p.max_batch) err |= PKV_DEV_ERR_BAD_SLOT;
  if (pos < 0 || block >= p.max_blocks || pos >= p.rope_len) err |= PKV_DEV_ERR_BAD_POS;
  int page = -1;
  float4 c, s;
  if (!err) {
    page = __ldg(p.page_table + static_cast<long long>(slot) * p.max_blocks + block);
    if (lane < kTurners) {
      const long long at = static_cast<long long>(pos) * (kRotated / 2);
      c = __ldg(reinterpret_cast<const float4*>(p.rope_cos + at) + lane);
      s = __ldg(reinterpret_cast<const float4*>(p.rope_sin + at) + lane);
    }
  }
  if (p.norm_weight != nullptr) {
    float x[8], y[8];
    unpack8(v0, x);
    unpack8(v1, y);
    float ss = 0.f;
#pragma unroll
    for (int u = 0; u < 8; ++u) ss = fmaf(x[u], x[u], fmaf(y[u], y[u], ss));
    float ms = warp_sum(ss) * (1.f / kLatent) + p.norm_eps;
    float f = 1.f;
    if (!(ms >= 0x1p-100f && ms <= FLT_MAX)) {
      // Squares that left fp32's range, or are about to: once more with the values times a power of
      // two. (Every lane has the same sum. The row is read again: few registers for a rare case.)
      f = ms < 1.f ? 0x1p80f : 0x1p-70f;
      const __nv_bfloat16* own = p.x + i * p.x_token + 8 * lane;
      ss = 0.f;
#pragma unroll 1
      for (int u = 0; u < 16; ++u) {
        const float v = __bfloat162float(own[u < 8 ? u : 248 + u]) * f;
        ss = fmaf(v, v, ss);
      }
      ms = warp_sum(ss) * (1.f / kLatent) + p.norm_eps * f * f;
    }
    const float inv = rsqrtf(ms);
    const float4* w = reinterpret_cast<const float4*>(p.norm_weight);
    const float4 wa = __ldg(w + 2 * lane), wb = __ldg(w + 2 * lane + 1);
    const float4 wc = __ldg(w + 64 + 2 * lane), wd = __ldg(w + 64 + 2 * lane + 1);
    const float w0[8] = {wa.x, wa.y, wa.z, wa.w, wb.x, wb.y, wb.z, wb.w};
    const float w1[8] = {wc.x, wc.y, wc.z, wc.w, wd.x, wd.y, wd.z, wd.w};
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      x[u] = ((x[u] * f) * inv) * w0[u];
      y[u] = ((y[u] * f) * inv) * w1[u];
    }
    v0 = pack8(x);
    v1 = pack8(y);
  }
  if (!err && (page < 0 || page >= p.num_pages)) err = PKV_DEV_ERR_BAD_PAGE;
  if (err) {
    if (lane == 0) set_dev_err(p.dev_err, err);
    return;
  }
  uint4* dst = reinterpret_cast<uint4*>(
      p.pool + (static_cast<long long>(page) * p.page_size + pos % p.page_size) * kRow);
  dst[lane] = v0;
  dst[32 + lane] = v1;
  if (lane < kTurners) {
    float x[8];
    unpack8(r, x);
    if (kInterleaved) {
      turn_pairs(x, c, s);
      dst[64 + lane] = pack8(x);
    } else {
      const float cv[4] = {c.x, c.y, c.z, c.w}, sv[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const float a = x[u], b = x[u + 4];
        x[u] = turn_diff(a, cv[u], b, sv[u]);
        x[u + 4] = turn_sum(b, cv[u], a, sv[u]);
      }
      const uint4 w = pack8(x);
      reinterpret_cast<uint2*>(dst + 64)[lane] = make_uint2(w.x, w.y);
      reinterpret_cast<uint2*>(dst + 68)[lane] = make_uint2(w.z, w.w);
    }
  }
}

// ------------------------------------------------------------------- gather --

struct LatentGatherParams {
  const uint4* pool;
  const int32_t* page_table;
  const int32_t* slots;
  const int32_t* starts;
  uint4* out;
  int32_t* dev_err;
  int n_seqs;
  int total;
  int page_size;
  int num_pages;
  int max_batch;
  int max_blocks;
};

constexpr int kGatherWarps = 4;
constexpr int kGatherRows = 4;  // of a warp: nine 16-byte pieces a lane
constexpr int kRowPieces = kRow * 2 / 16;  // 72

// A warp copies kGatherRows consecutive rows of out. It finds the first one's sequence among the
// starts (32 at a time, so that up to 1024 sequences take two reads); lane l < kGatherRows steps on from
// there to row l's and looks up its page. Then all pieces of the rows are read before the first is
// written. Memory bounds it: 82 000 rows of 16 sequences in 30.8 us (189 MB, 6.1 TB/s; 8 rows a warp
// 31.8 us, 16 rows 33.9, the look-ups being cheap); the chain of starts, slot, page and row bounds
// few rows (777: 2.7 us, with 8 rows a warp 3.6).
__global__ void __launch_bounds__(kGatherWarps * 32)
latent_gather_kernel(const LatentGatherParams p) {
  constexpr int kPerLane = 9;
  static_assert(32 * kPerLane == kGatherRows * kRowPieces, "nine pieces a lane");
  pdl_wait_primary();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31;
  const long long warp = static_cast<long long>(blockIdx.x) * kGatherWarps + (threadIdx.x >> 5);
  // starts have to ascend from 0 or more to at most total
  for (long long i = warp * 32 + lane; i <= p.n_seqs;
       i += static_cast<long long>(gridDim.x) * (kGatherWarps * 32)) {
    const int s = __ldg(p.starts + i);
    const int before = i > 0 ? __ldg(p.starts + i - 1) : 0;
    if (s < before || s > p.total) set_dev_err(p.dev_err, PKV_DEV_ERR_LAYOUT);
  }
  const long long row0 = warp * kGatherRows;
  if (row0 >= p.total) return;
  // the number of starts that are at most row0: the first `lo` are, those from `hi` on are not
  int lo = 0, hi = p.n_seqs + 1;
  while (hi - lo > 0) {
    const int step = (hi - lo + 31) / 32;
    const int at = lo + lane * step;
    const bool below = at < hi && __ldg(p.starts + at) <= row0;
    const int n = __popc(__ballot_sync(0xffffffffu, below));  // (ascending: the first n lanes)
    if (n == 0) {
      hi = lo;
    } else {
      const int last = lo + (n - 1) * step;  // at most row0; the next one looked at is not
      hi = min(hi, last + step);
      lo = last + 1;
    }
  }
  long long from = -1;  // the row's place in the pool, -1: the row is not written
  const long long t = row0 + lane;
  if (lane < kGatherRows && t < p.total) {
    int b = lo - 1;
    while (b + 1 <= p.n_seqs && (b < 0 || __ldg(p.starts + b + 1) <= t)) {
      if (b < 0 && __ldg(p.starts) > t) break;
      ++b;
    }
    if (b >= 0 && b < p.n_seqs) {
      const int slot = __ldg(p.slots + b);
      const long long pos = t - max(__ldg(p.starts + b), 0);
      if (slot != 0 && pos >= 0) {
        const long long block = pos / p.page_size;
        int err = 0;
        if (slot < 0 || slot >= p.max_batch) err = PKV_DEV_ERR_BAD_SLOT;
        else if (block >= p.max_blocks) err = PKV_DEV_ERR_BAD_POS;
        if (!err) {
          const int page = __ldg(p.page_table + static_cast<long long>(slot) * p.max_blocks + block);
          if (page < 0 || page >= p.num_pages) err = PKV_DEV_ERR_BAD_PAGE;
          else from = static_cast<long long>(page) * p.page_size + pos % p.page_size;
        }
        if (err) set_dev_err(p.dev_err, err);
      }
    }
  }
  __syncwarp();
  uint4* dst = p.out + row0 * kRowPieces;
  uint4 v[kPerLane];
  bool have[kPerLane];
#pragma unroll
  for (int k = 0; k < kPerLane; ++k) {
    const int e = k * 32 + lane;
    const int r = e / kRowPieces;
    const long long src = __shfl_sync(0xffffffffu, from, r);
    have[k] = src >= 0;
    if (have[k]) v[k] = __ldg(p.pool + src * kRowPieces + (e - r * kRowPieces));
  }
#pragma unroll
  for (int k = 0; k < kPerLane; ++k)
    if (have[k]) dst[k * 32 + lane] = v[k];
}

// PKV_OK on an sm_103 device.
pkv_status check_device() {
  int sms = 0;
  return device_info(&sms);
}

}  // namespace
}  // namespace pkv

using namespace pkv;
using namespace pkv::latent;

extern "C" pkv_status pkv_rotate(const void* x, int64_t x_token_stride, int64_t x_head_stride,
                                 void* out, int64_t out_token_stride, int64_t out_head_stride,
                                 int n_tokens, int num_heads, int dims, int interleaved,
                                 const int32_t* positions, const float* rope_cos,
                                 const float* rope_sin, int rope_len, int32_t* dev_err,
                                 cudaStream_t stream) {
  constexpr int64_t kMaxStride = int64_t{1} << 40;
  if (n_tokens == 1) x_token_stride = out_token_stride = 0;  // (no second token to step to)
  if (num_heads == 1) x_head_stride = out_head_stride = 0;
  if (n_tokens < 0 || num_heads <= 0 || dims <= 0 || dims % 2 != 0 || rope_len <= 0)
    return PKV_ERR_ARG;
  if (interleaved != 0 && interleaved != 1) return PKV_ERR_ARG;
  for (const int64_t s : {x_token_stride, x_head_stride, out_token_stride, out_head_stride})
    if (s < 0 || s > kMaxStride) return PKV_ERR_ARG;
  // rows of the output must not lie on one another: the axis with the smaller stride has
  // to end before the next step of the other
  {
    const bool heads_inside = num_heads == 1 || (n_tokens > 1 && out_head_stride <= out_token_stride);
    const int64_t inner = heads_inside ? out_head_stride : out_token_stride;
    const int64_t outer = heads_inside ? out_token_stride : out_head_stride;
    const int64_t n_inner = heads_inside ? num_heads : n_tokens;
    const int64_t n_outer = heads_inside ? n_tokens : num_heads;
    if (n_inner > 1 && inner < dims) return PKV_ERR_ARG;
    if (n_outer > 1 && outer - dims < (n_inner - 1) * (n_inner > 1 ? inner : 0)) return PKV_ERR_ARG;
  }
  if (x == out && (x_token_stride != out_token_stride || x_head_stride != out_head_stride))
    return PKV_ERR_ARG;
  if (n_tokens == 0) return PKV_OK;
  if (!x || !out || !positions || !rope_cos || !rope_sin) return PKV_ERR_ARG;
  if (!is_aligned(x, 2) || !is_aligned(out, 2) || !is_aligned(positions, 4) ||
      !is_aligned(rope_cos, 4) || !is_aligned(rope_sin, 4) || !is_aligned(dev_err, 4))
    return PKV_ERR_ALIGN;
  if (const pkv_status st = check_device(); st != PKV_OK) return st;
  const int piece = interleaved ? 8 : 16;  // values of a 16-byte unit
  const bool wide = dims % piece == 0 && x_token_stride % 8 == 0 && x_head_stride % 8 == 0 &&
                    out_token_stride % 8 == 0 && out_head_stride % 8 == 0 && is_aligned(x, 16) &&
                    is_aligned(out, 16) && is_aligned(rope_cos, 16) && is_aligned(rope_sin, 16);
  RotateParams p;
  p.x = static_cast<const __nv_bfloat16*>(x);
  p.out = static_cast<__nv_bfloat16*>(out);
  p.x_token = x_token_stride;
  p.x_head = x_head_stride;
  p.out_token = out_token_stride;
  p.out_head = out_head_stride;
  p.positions = positions;
  p.rope_cos = rope_cos;
  p.rope_sin = rope_sin;
  p.dev_err = dev_err;
  p.n_tokens = n_tokens;
  p.num_heads = num_heads;
  p.dims = dims;
  p.rope_len = rope_len;
  p.units = wide ? dims / piece : dims / 2;
  p.head_groups = (num_heads + kRotateHeads - 1) / kRotateHeads;
  const long long per_token = static_cast<long long>(p.units) * p.head_groups;
  if (per_token > INT_MAX) return PKV_ERR_ARG;
  const long long blocks = (per_token * n_tokens + kRotateThreads - 1) / kRotateThreads;
  if (blocks > INT_MAX) return PKV_ERR_ARG;
  const auto kernel = wide ? (interleaved ? rotate_kernel<kPairs16> : rotate_kernel<kHalves16>)
                           : (interleaved ? rotate_kernel<kPairs1> : rotate_kernel<kHalves1>);
  return record_cuda_status(launch_kernel(kernel, dim3(static_cast<unsigned>(blocks)),
                                          dim3(kRotateThreads), 0, stream, true, p));
}

extern "C" pkv_status pkv_latent_append(const pkv_cache_desc* cache, void* pool,
                                        const int32_t* page_table, const void* x_new,
                                        int64_t x_token_stride, const int32_t* batch_idx,
                                        const int32_t* input_pos, int n_tokens,
                                        const float* rope_cos, const float* rope_sin, int rope_len,
                                        int interleaved, const float* norm_weight, float norm_eps,
                                        int32_t* dev_err, cudaStream_t stream) {
  if (const pkv_status st = check_latent_cache(cache); st != PKV_OK) return st;
  if (n_tokens < 0 || rope_len <= 0 || (interleaved != 0 && interleaved != 1)) return PKV_ERR_ARG;
  if (x_token_stride < 0 || x_token_stride > (int64_t{1} << 40)) return PKV_ERR_ARG;
  if (norm_weight != nullptr && !(std::isfinite(norm_eps) && norm_eps >= 0.f)) return PKV_ERR_ARG;
  if (n_tokens == 0) return PKV_OK;
  if (!pool || !page_table || !x_new || !batch_idx || !input_pos || !rope_cos || !rope_sin)
    return PKV_ERR_ARG;
  if (x_token_stride % 8 != 0 || !is_aligned(pool, 16) || !is_aligned(x_new, 16) ||
      !is_aligned(rope_cos, 16) || !is_aligned(rope_sin, 16) || !is_aligned(norm_weight, 16) ||
      !is_aligned(page_table, 4) || !is_aligned(batch_idx, 4) || !is_aligned(input_pos, 4) ||
      !is_aligned(dev_err, 4))
    return PKV_ERR_ALIGN;
  if (const pkv_status st = check_device(); st != PKV_OK) return st;
  LatentAppendParams p;
  p.pool = static_cast<__nv_bfloat16*>(pool);
  p.page_table = page_table;
  p.x = static_cast<const __nv_bfloat16*>(x_new);
  p.x_token = x_token_stride;
  p.batch_idx = batch_idx;
  p.input_pos = input_pos;
  p.rope_cos = rope_cos;
  p.rope_sin = rope_sin;
  p.norm_weight = norm_weight;
  p.norm_eps = norm_eps;
  p.dev_err = dev_err;
  p.n_tokens = n_tokens;
  p.rope_len = rope_len;
  p.page_size = cache->page_size;
  p.num_pages = cache->num_pages;
  p.max_batch = cache->max_batch;
  p.max_blocks = cache->max_blocks;
  const int grid = n_tokens / kAppendWarps + (n_tokens % kAppendWarps != 0);
  return record_cuda_status(
      launch_kernel(interleaved ? latent_append_kernel<true> : latent_append_kernel<false>,
                    dim3(grid), dim3(kAppendWarps * 32), 0, stream, true, p));
}

extern "C" pkv_status pkv_latent_gather(const pkv_cache_desc* cache, const void* pool,
                                        const int32_t* page_table, const int32_t* slots,
                                        const int32_t* starts, int n_seqs, int total, void* out,
                                        int32_t* dev_err, cudaStream_t stream) {
  if (const pkv_status st = check_latent_cache(cache); st != PKV_OK) return st;
  if (n_seqs < 0 || total < 0) return PKV_ERR_ARG;
  if (n_seqs == 0 || total == 0) return PKV_OK;
  if (!pool || !page_table || !slots || !starts || !out) return PKV_ERR_ARG;
  if (!is_aligned(pool, 16) || !is_aligned(out, 16) || !is_aligned(page_table, 4) ||
      !is_aligned(slots, 4) || !is_aligned(starts, 4) || !is_aligned(dev_err, 4))
    return PKV_ERR_ALIGN;
  if (const pkv_status st = check_device(); st != PKV_OK) return st;
  LatentGatherParams p;
  p.pool = static_cast<const uint4*>(pool);
  p.page_table = page_table;
  p.slots = slots;
  p.starts = starts;
  p.out = static_cast<uint4*>(out);
  p.dev_err = dev_err;
  p.n_seqs = n_seqs;
  p.total = total;
  p.page_size = cache->page_size;
  p.num_pages = cache->num_pages;
  p.max_batch = cache->max_batch;
  p.max_blocks = cache->max_blocks;
  constexpr int per_cta = kGatherWarps * kGatherRows;
  const int grid = total / per_cta + (total % per_cta != 0);
  return record_cuda_status(launch_kernel(latent_gather_kernel, dim3(grid),
                                          dim3(kGatherWarps * 32), 0, stream, true, p));
}
