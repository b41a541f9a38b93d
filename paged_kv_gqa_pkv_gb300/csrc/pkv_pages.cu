// pkv_pages.cu - the pages of the cache: pkv_update_pages (fork, reserve, copy
// on write, truncate, free), pkv_compact_pages and pkv_commit_path.
//
// The state is the page table and one count per page. There is no free list:
// a page is free when its count is 0, and the lowest free numbers are handed
// out, so a result depends on the state alone and never on the order in which
// CTAs run. Both page operators are two launches: a plan that reads the state
// and changes nothing, and an apply that takes every decision from the plan's
// snapshot, so rows need no order among themselves.
//
// The plan also splits the page counts into chunks, one CTA each: a chunk's
// CTA lists its free pages in ascending order and counts them. The apply's
// CTAs scan the chunk counts (at most kMaxChunks) in shared memory and find the
// k-th free page of the pool by a binary search, so a pool of any size is read
// once, in parallel, and no CTA waits for another.
//
// What bounds them: K/V rows are moved by 16-byte loads and stores with eight loads
// in flight per thread (the copy's bandwidth where much is moved), and
// two launches' latency where little is.
#include <climits>

#include "pkv.h"
#include "pkv_launch.h"

namespace pkv {
namespace {

constexpr int kPlanThreads = 256;
constexpr int kMaxChunks = 1024;
constexpr int kChunkPages = 4096;  // smallest chunk: 16 counts per thread

constexpr int kInFlight = 4;  // 16-byte loads per thread and pool before the first store

struct PagesParams {
  void* pool[2];  // K, V
  int32_t* page_table;
  int32_t* refs;
  const int32_t* dst;
  const int32_t* src;
  const int32_t* keep;
  const int32_t* newl;
  int32_t* num_live;
  int32_t* dev_err;
  // workspace
  int32_t* chunk_free;   // [n_chunks] free pages of each chunk
  int32_t* free_list;    // [num_pages] chunk c's free pages from c * chunk_pages on
  int32_t* live_list;    // [num_pages] (compact) its other pages, likewise
  int32_t* free_before;  // [num_pages] (compact) free pages of the chunk below this one
  int32_t* need;         // [n] (update) fresh pages of the row, -1: not served
  int32_t* tail;         // [n] (update) page whose kept rows are copied, -1: none
  uint32_t* fresh;       // [n * words] (update) blocks that get a fresh page
  int n;
  int words;             // 32-bit words per row of `fresh`
  int n_chunks;
  int chunk_pages;
  int row_vecs;          // 16-byte vectors per token row of one pool
  int page_size;
  int num_pages;
  int max_batch;
  int max_blocks;
};

__device__ __forceinline__ bool is_free(const PagesParams& p, int page) {
  return page >= 1 && page < p.num_pages && p.refs[page] == 0;
}

// Block-wide exclusive sum over kPlanThreads threads; contains __syncthreads.
__device__ __forceinline__ int block_excl(int v, int* scratch, int& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) scratch[warp] = x;
  __syncthreads();
  int before = 0, all = 0;
#pragma unroll
  for (int w = 0; w < kPlanThreads / 32; ++w) {
    if (w < warp) before += scratch[w];
    all += scratch[w];
  }
  __syncthreads();  // scratch is reused by the next scan
  total = all;
  return before + x - v;
}

// One chunk of the counts: its free pages listed in ascending order (and, for
// the compaction, its other pages, and how many free ones lie below each).
template <bool kLive>
__device__ void plan_chunk(const PagesParams& p, int c, int* scratch) {
  const int begin = c * p.chunk_pages;
  const int end = min(begin + p.chunk_pages, p.num_pages);
  constexpr int kPer = 16;
  int base = 0;
  for (int s = begin; s < end; s += kPlanThreads * kPer) {
    const int i0 = s + threadIdx.x * kPer;
    uint32_t bits = 0;
#pragma unroll
    for (int k = 0; k < kPer; ++k)
      if (i0 + k < end && is_free(p, i0 + k)) bits |= 1u << k;
    int total;
    int before = base + block_excl(__popc(bits), scratch, total);
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
      const int i = i0 + k;
      if (i >= end) break;
      if constexpr (kLive) p.free_before[i] = before;
      if ((bits >> k) & 1u) {
        p.free_list[begin + before] = i;
        ++before;
      } else if constexpr (kLive) {
        p.live_list[begin + (i - begin - before)] = i;
      }
    }
    base += total;
  }
  if (threadIdx.x == 0) p.chunk_free[c] = base;
}

// Exclusive prefix of the chunks' free counts in smem[0 .. n_chunks], the total
// last. Every thread of the CTA calls it.
__device__ __forceinline__ void scan_chunks(const PagesParams& p, int* prefix, int* scratch) {
  int base = 0;
  for (int s = 0; s < p.n_chunks; s += kPlanThreads) {
    const int c = s + threadIdx.x;
    const int v = c < p.n_chunks ? p.chunk_free[c] : 0;
    int total;
    const int before = block_excl(v, scratch, total);
    if (c < p.n_chunks) prefix[c] = base + before;
    base += total;
  }
  if (threadIdx.x == 0) prefix[p.n_chunks] = base;
  __syncthreads();
}

// The chunk that holds the k-th entry of a list counted by prefix (the largest
// c with prefix(c) <= k; chunks without entries are passed over).
template <class F>
__device__ __forceinline__ int find_chunk(int n_chunks, int k, F prefix) {
  int lo = 0, hi = n_chunks - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (prefix(mid) <= k) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

// The k-th free page, k below the number of free pages.
__device__ __forceinline__ int kth_free(const PagesParams& p, const int* prefix, int k) {
  const int c = find_chunk(p.n_chunks, k, [&](int i) { return prefix[i]; });
  return p.free_list[static_cast<int64_t>(c) * p.chunk_pages + (k - prefix[c])];
}

// Copies `vecs` 16-byte vectors of both pools, from `src` to `dst` (vector
// offsets), by the part `part` of `parts` CTAs; kInFlight loads of each pool go out
// before the first store.
__device__ __forceinline__ void copy_rows(const PagesParams& p, int64_t src, int64_t dst, int vecs,
                                          int part, int parts) {
  const int step = parts * kPlanThreads;
  const uint4* kf = static_cast<const uint4*>(p.pool[0]) + src;
  const uint4* vf = static_cast<const uint4*>(p.pool[1]) + src;
  uint4* kt = static_cast<uint4*>(p.pool[0]) + dst;
  uint4* vt = static_cast<uint4*>(p.pool[1]) + dst;
  for (int i = part * kPlanThreads + threadIdx.x; i < vecs; i += step * kInFlight) {
    uint4 k[kInFlight], v[kInFlight];
#pragma unroll
    for (int u = 0; u < kInFlight; ++u)
      if (i + u * step < vecs) {
        k[u] = kf[i + u * step];
        v[u] = vf[i + u * step];
      }
#pragma unroll
    for (int u = 0; u < kInFlight; ++u)
      if (i + u * step < vecs) {
        kt[i + u * step] = k[u];
        vt[i + u * step] = v[u];
      }
  }
}

// ------------------------------------------------------------------ update --

struct Row {
  int d, s, keep, newl;
  int kept_blocks;   // blocks that hold kept tokens
  int first;         // first block with a position in [keep, new)
  int blocks;        // blocks up to new
  bool same, writes;
};

__device__ __forceinline__ Row load_row(const PagesParams& p, int i) {
  Row r;
  r.d = p.dst[i];
  r.s = p.src[i];
  r.keep = p.keep[i];
  r.newl = p.newl[i];
  r.kept_blocks =
      static_cast<int>((static_cast<int64_t>(r.keep) + p.page_size - 1) / p.page_size);
  r.first = r.keep / p.page_size;
  r.blocks = static_cast<int>((static_cast<int64_t>(r.newl) + p.page_size - 1) / p.page_size);
  r.same = r.s == r.d;
  r.writes = r.newl > r.keep;
  return r;
}

__device__ __forceinline__ bool is_page(const PagesParams& p, int e) {
  return e >= 1 && e < p.num_pages;
}

// Row i against the state at the start of the call: which blocks need a fresh
// page, and which page's kept rows are copied.
__device__ void plan_row(const PagesParams& p, int i, int* scratch) {
  const Row r = load_row(p, i);
  int err = 0;
  const bool live = r.d != 0;
  if (live) {
    if (r.d < 0 || r.d >= p.max_batch || r.s < 0 || r.s >= p.max_batch ||
        (r.s == 0 && r.keep > 0))
      err = PKV_DEV_ERR_BAD_SLOT;
    else if (r.keep < 0 || r.newl < r.keep || r.blocks > p.max_blocks)
      err = PKV_DEV_ERR_BAD_POS;
  }
  bool clash = false;
  if (live && !err)
    for (int k = threadIdx.x; k < p.n; k += kPlanThreads) {
      const int d = p.dst[k];
      if ((k < i && d == r.d) || (k != i && !r.same && r.keep > 0 && d == r.s)) clash = true;
    }
  if (__syncthreads_or(clash)) err = PKV_DEV_ERR_BAD_SLOT;
  int count = 0;
  if (live && !err) {
    const int32_t* mine = p.page_table + static_cast<int64_t>(r.d) * p.max_blocks;
    const int32_t* from = p.page_table + static_cast<int64_t>(r.s) * p.max_blocks;
    const int lane = threadIdx.x & 31;
    bool bad = false;
    for (int w = threadIdx.x >> 5; w < p.words; w += kPlanThreads / 32) {
      const int j = 32 * w + lane;
      bool fresh = false;
      if (j < p.max_blocks) {
        const int old = mine[j];
        const bool have = is_page(p, old);
        const int uses = have ? p.refs[old] : 0;
        if (have && uses < 1) bad = true;
        if (j < r.kept_blocks) {
          const int e = from[j];
          if (!is_page(p, e) || p.refs[e] < 1) bad = true;
        }
        fresh = r.writes && j >= r.first && j < r.blocks && !(r.same && have && uses == 1);
      }
      const uint32_t bits = __ballot_sync(0xffffffffu, fresh);
      if (lane == 0) {
        p.fresh[static_cast<int64_t>(i) * p.words + w] = bits;
        count += __popc(bits);
      }
    }
    if (__syncthreads_or(bad)) err = PKV_DEV_ERR_BAD_PAGE;
  }
  int total;
  block_excl(count, scratch, total);
  if (threadIdx.x == 0) {
    const bool serve = live && !err;
    p.need[i] = serve ? total : -1;
    int tail = -1;
    if (serve && r.writes && r.keep % p.page_size != 0 &&
        ((p.fresh[static_cast<int64_t>(i) * p.words + (r.first >> 5)] >> (r.first & 31)) & 1u))
      tail = p.page_table[static_cast<int64_t>(r.s) * p.max_blocks + r.first];
    p.tail[i] = tail;
    if (err) set_dev_err(p.dev_err, err);
  }
}

__global__ void __launch_bounds__(kPlanThreads) update_plan_kernel(const PagesParams p) {
  __shared__ int scratch[kPlanThreads / 32];
  pdl_wait_primary();
  pdl_launch_dependents();  // the apply waits for this grid before it reads anything
  if (static_cast<int>(blockIdx.x) < p.n) plan_row(p, blockIdx.x, scratch);
  else plan_chunk<false>(p, blockIdx.x - p.n, scratch);
}

// grid (n, parts): every CTA of a row copies its part of the partly kept page;
// part 0 also rewrites the row's table entries and counts.
__global__ void __launch_bounds__(kPlanThreads, 3) update_apply_kernel(const PagesParams p) {
  __shared__ int scratch[kPlanThreads / 32];
  __shared__ int prefix[kMaxChunks + 1];
  pdl_wait_primary();
  // everything that the row's place depends on, in flight at once
  const int i = blockIdx.x;
  const int need = p.need[i], tail = p.tail[i];
  const Row r = load_row(p, i);
  int mine = 0;
  for (int k = threadIdx.x; k < i; k += kPlanThreads) mine += max(p.need[k], 0);
  if (need < 0 || (blockIdx.y > 0 && tail < 0)) return;
  scan_chunks(p, prefix, scratch);
  int before;  // fresh pages of the rows above
  block_excl(mine, scratch, before);
  if (need > 0 && static_cast<int64_t>(before) + need > prefix[p.n_chunks]) {
    if (blockIdx.y == 0 && threadIdx.x == 0) set_dev_err(p.dev_err, PKV_DEV_ERR_NO_PAGES);
    return;
  }
  if (blockIdx.y == 0) {
    int32_t* row = p.page_table + static_cast<int64_t>(r.d) * p.max_blocks;
    const int32_t* from = p.page_table + static_cast<int64_t>(r.s) * p.max_blocks;
    const uint32_t* fresh = p.fresh + static_cast<int64_t>(i) * p.words;
    const int lane = threadIdx.x & 31;
    for (int w = threadIdx.x >> 5; w < p.words; w += kPlanThreads / 32) {
      const uint32_t bits = fresh[w];
      int rank = 0;  // fresh blocks of the row below this word's
      for (int k = lane; k < w; k += 32) rank += __popc(fresh[k]);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) rank += __shfl_xor_sync(0xffffffffu, rank, o);
      const int j = 32 * w + lane;
      if (j >= p.max_blocks) continue;
      const int old = row[j];
      const bool get = (bits >> lane) & 1u;
      int now = -1;
      if (get)
        now = kth_free(p, prefix, before + rank + __popc(bits & ((1u << lane) - 1u)));
      else if (j < r.kept_blocks)
        now = from[j];
      else if (r.same && r.writes && j >= r.first && j < r.blocks)
        now = old;
      const bool stays = r.same && now == old;
      if (!stays) {
        if (is_page(p, old)) atomicSub(p.refs + old, 1);
        if (now >= 0) atomicAdd(p.refs + now, 1);
        row[j] = now;
      }
    }
    // a kernel that starts before this grid has drained (a programmatic
    // dependent) reads the table as written here
    __threadfence();
  }
  if (tail >= 0) {
    // the partly kept block is the row's first fresh one
    const int to = kth_free(p, prefix, before);
    const int64_t page_vecs = static_cast<int64_t>(p.page_size) * p.row_vecs;
    copy_rows(p, tail * page_vecs, to * page_vecs,
              (r.keep % p.page_size) * p.row_vecs, blockIdx.y, gridDim.y);
  }
}

// ----------------------------------------------------------------- compact --

__global__ void __launch_bounds__(kPlanThreads) compact_plan_kernel(const PagesParams p) {
  __shared__ int scratch[kPlanThreads / 32];
  pdl_wait_primary();
  pdl_launch_dependents();
  plan_chunk<true>(p, blockIdx.x, scratch);
}

constexpr int kPieceVecs = 4096;  // 64 KB of each pool per piece

// Everything is read from the plan's lists, so the counts may be rewritten while
// other CTAs still look pages up.
__global__ void __launch_bounds__(kPlanThreads) compact_apply_kernel(const PagesParams p) {
  __shared__ int scratch[kPlanThreads / 32];
  __shared__ int prefix[kMaxChunks + 1];
  pdl_wait_primary();
  scan_chunks(p, prefix, scratch);
  const int n_free = prefix[p.n_chunks];
  const int n_live = p.num_pages - n_free;
  // free pages below n_live = pages to move; live pages of the first c chunks
  int moves = 0;
  if (n_live < p.num_pages) {
    const int c = n_live / p.chunk_pages;
    moves = prefix[c] + p.free_before[n_live];
  }
  const int stay = n_live - moves;  // live pages below n_live
  auto live_prefix = [&](int c) { return c * p.chunk_pages - prefix[c]; };
  if (blockIdx.x == 0 && threadIdx.x == 0 && p.num_live != nullptr) *p.num_live = n_live;

  // table entries of pages that move
  const int64_t entries = static_cast<int64_t>(p.max_batch) * p.max_blocks;
  const int64_t step = static_cast<int64_t>(gridDim.x) * kPlanThreads;
  for (int64_t t = static_cast<int64_t>(blockIdx.x) * kPlanThreads + threadIdx.x; t < entries;
       t += step) {
    const int e = p.page_table[t];
    if (e < n_live || e >= p.num_pages) continue;
    const int c = e / p.chunk_pages;
    const int in_chunk = e - c * p.chunk_pages - p.free_before[e];  // live pages below it there
    // (a free page above its chunk's last live one has no place in the list)
    const int end = min((c + 1) * p.chunk_pages, p.num_pages);
    const int in_list = end - c * p.chunk_pages - (prefix[c + 1] - prefix[c]);
    if (in_chunk >= in_list ||
        p.live_list[static_cast<int64_t>(c) * p.chunk_pages + in_chunk] != e ||
        live_prefix(c) + in_chunk < stay) {
      set_dev_err(p.dev_err, PKV_DEV_ERR_BAD_PAGE);
      continue;
    }
    p.page_table[t] = kth_free(p, prefix, live_prefix(c) + in_chunk - stay);
  }
  __threadfence();

  const int64_t page_vecs = static_cast<int64_t>(p.page_size) * p.row_vecs;
  const int pieces = static_cast<int>((page_vecs + kPieceVecs - 1) / kPieceVecs);
  const int64_t units = static_cast<int64_t>(moves) * pieces;
  for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
    const int k = static_cast<int>(u / pieces);
    const int piece = static_cast<int>(u % pieces);
    const int c = find_chunk(p.n_chunks, stay + k, live_prefix);
    const int from =
        p.live_list[static_cast<int64_t>(c) * p.chunk_pages + (stay + k - live_prefix(c))];
    const int to = kth_free(p, prefix, k);
    const int64_t v0 = static_cast<int64_t>(piece) * kPieceVecs;
    const int nv = static_cast<int>(page_vecs - v0 < kPieceVecs ? page_vecs - v0 : kPieceVecs);
    copy_rows(p, from * page_vecs + v0, to * page_vecs + v0, nv, 0, 1);
    if (piece == 0 && threadIdx.x == 0) {
      p.refs[to] = p.refs[from];
      p.refs[from] = 0;
    }
  }
}

// ------------------------------------------------------------------ commit --

struct CommitParams {
  void* pool[2];
  const int32_t* page_table;
  const int32_t* path;
  const int32_t* n_accepted;
  const int32_t* batch_idx;
  const int32_t* ctx_lens;
  int32_t* new_lens;
  int32_t* dev_err;
  int n_nodes;
  int row_vecs;
  int page_size;
  int num_pages;
  int max_batch;
  int max_blocks;
};

constexpr int kCommitThreads = 256;
constexpr int kCommitInFlight = 16;

// One CTA per row; a thread owns one 16-byte column of the slot's K or V rows
// and moves the path's rows in ascending order, kCommitInFlight at a time: all of a
// group's loads precede its stores. In place this is safe: with path strictly
// increasing, path[j] >= j, so row ctx + i is never the source of a later j.
__global__ void __launch_bounds__(kCommitThreads) commit_path_kernel(const CommitParams p) {
  __shared__ int64_t s_src[PKV_MAX_TREE_NODES], s_dst[PKV_MAX_TREE_NODES];
  pdl_wait_primary();
  const int b = blockIdx.x;
  const int slot = p.batch_idx[b];
  const int ctx = p.ctx_lens[b];
  const int n = p.n_accepted[b];
  // (read beside the lengths, whatever they turn out to be)
  const int i = threadIdx.x;
  const int32_t* path = p.path + static_cast<int64_t>(b) * p.n_nodes;
  const int a = i < p.n_nodes ? path[i] : 0;
  const int before = i > 0 && i < p.n_nodes ? path[i - 1] : -1;
  int err = 0;
  if (slot < 0 || slot >= p.max_batch) err = PKV_DEV_ERR_BAD_SLOT;
  else if (slot > 0 && (n < 0 || n > p.n_nodes)) err = PKV_DEV_ERR_BAD_TREE;
  else if (slot > 0 && ctx < 0) err = PKV_DEV_ERR_BAD_POS;
  const bool live = slot > 0 && !err && n > 0;
  int mine = 0;
  if (live && i < n) {
    const int64_t from = static_cast<int64_t>(ctx) + a;
    const int64_t cap = static_cast<int64_t>(p.max_blocks) * p.page_size;
    if (a < 0 || a >= p.n_nodes || before >= a) {
      mine = PKV_DEV_ERR_BAD_TREE;
    } else if (from >= cap) {
      mine = PKV_DEV_ERR_BAD_POS;
    } else {
      s_src[i] = s_dst[i] = 0;
      if (a != i) {
        const int32_t* row = p.page_table + static_cast<int64_t>(slot) * p.max_blocks;
        const int to = ctx + i, fr = static_cast<int>(from);  // to < fr < 2^31
        const int ps = row[fr / p.page_size], pd = row[to / p.page_size];
        if (ps < 0 || ps >= p.num_pages || pd < 0 || pd >= p.num_pages) mine = PKV_DEV_ERR_BAD_PAGE;
        s_src[i] = static_cast<int64_t>(ps) * p.page_size + fr % p.page_size;
        s_dst[i] = static_cast<int64_t>(pd) * p.page_size + to % p.page_size;
      }
    }
  }
  // the lowest bit found stands for the row (every thread learns of any)
  const int bad = __syncthreads_or(mine != 0);
  if (mine) set_dev_err(p.dev_err, mine);
  if (err && threadIdx.x == 0) set_dev_err(p.dev_err, err);
  const bool moves = live && !bad;
  if (threadIdx.x == 0 && p.new_lens != nullptr) p.new_lens[b] = moves ? ctx + n : ctx;
  __threadfence();  // a programmatic dependent may read new_lens before this grid drains
  if (!moves) return;
  for (int c = threadIdx.x; c < 2 * p.row_vecs; c += kCommitThreads) {
    const bool k_side = c < p.row_vecs;
    uint4* pool = static_cast<uint4*>(k_side ? p.pool[0] : p.pool[1]) + (k_side ? c : c - p.row_vecs);
    for (int k0 = 0; k0 < n; k0 += kCommitInFlight) {
      uint4 v[kCommitInFlight];
#pragma unroll
      for (int u = 0; u < kCommitInFlight; ++u)
        if (k0 + u < n && s_src[k0 + u] != s_dst[k0 + u]) v[u] = pool[s_src[k0 + u] * p.row_vecs];
#pragma unroll
      for (int u = 0; u < kCommitInFlight; ++u)
        if (k0 + u < n && s_src[k0 + u] != s_dst[k0 + u]) pool[s_dst[k0 + u] * p.row_vecs] = v[u];
    }
  }
}

// -------------------------------------------------------------------- host --

bool aligned(const void* q, uintptr_t a) { return (reinterpret_cast<uintptr_t>(q) % a) == 0; }

struct PagesLayout {
  int n_chunks, chunk_pages, words;
  size_t off_free, off_a, off_b, off_c, total;
};

// Pages per chunk: a multiple of kChunkPages that keeps the chunks at kMaxChunks.
void chunk_layout(const pkv_cache_desc* c, PagesLayout& l) {
  const int64_t per = (static_cast<int64_t>(c->num_pages) + kMaxChunks - 1) / kMaxChunks;
  const int64_t size = (per + kChunkPages - 1) / kChunkPages * kChunkPages;
  l.chunk_pages = static_cast<int>(size);
  l.n_chunks = static_cast<int>((c->num_pages + size - 1) / size);
}

size_t up256(size_t x) { return (x + 255) / 256 * 256; }

PagesLayout update_layout(const pkv_cache_desc* c, int n) {
  PagesLayout l;
  chunk_layout(c, l);
  l.words = (c->max_blocks + 31) / 32;
  l.off_free = up256(static_cast<size_t>(l.n_chunks) * 4);
  l.off_a = l.off_free + up256(static_cast<size_t>(c->num_pages) * 4);
  l.off_b = l.off_a + up256(static_cast<size_t>(n) * 4);
  l.off_c = l.off_b + up256(static_cast<size_t>(n) * 4);
  l.total = l.off_c + up256(static_cast<size_t>(n) * l.words * 4);
  return l;
}

PagesLayout compact_layout(const pkv_cache_desc* c) {
  PagesLayout l;
  chunk_layout(c, l);
  const size_t list = up256(static_cast<size_t>(c->num_pages) * 4);
  l.words = 0;
  l.off_free = up256(static_cast<size_t>(l.n_chunks) * 4);
  l.off_a = l.off_free + list;
  l.off_b = l.off_a + list;
  l.off_c = l.off_b + list;
  l.total = l.off_c;
  return l;
}

PagesParams base_params(const pkv_cache_desc* c, const PagesLayout& l, void* k_pool, void* v_pool,
                        int32_t* page_table, int32_t* page_refs, void* workspace,
                        int32_t* dev_err) {
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  PagesParams p = {};
  p.pool[0] = k_pool;
  p.pool[1] = v_pool;
  p.page_table = page_table;
  p.refs = page_refs;
  p.dev_err = dev_err;
  p.chunk_free = reinterpret_cast<int32_t*>(ws);
  p.free_list = reinterpret_cast<int32_t*>(ws + l.off_free);
  p.words = l.words;
  p.n_chunks = l.n_chunks;
  p.chunk_pages = l.chunk_pages;
  p.row_vecs = c->num_kv_heads * c->head_dim * 2 / 16;
  p.page_size = c->page_size;
  p.num_pages = c->num_pages;
  p.max_batch = c->max_batch;
  p.max_blocks = c->max_blocks;
  return p;
}

}  // namespace
}  // namespace pkv

extern "C" {

size_t pkv_update_workspace_size(const pkv_cache_desc* cache, int n) {
  if (pkv::check_cache(cache) != PKV_OK || n < 0) return 0;
  return pkv::update_layout(cache, n).total;
}

size_t pkv_compact_workspace_size(const pkv_cache_desc* cache) {
  if (pkv::check_cache(cache) != PKV_OK) return 0;
  return pkv::compact_layout(cache).total;
}

pkv_status pkv_update_pages(const pkv_cache_desc* cache, void* k_pool, void* v_pool,
                            int32_t* page_table, int32_t* page_refs, const int32_t* dst_slots,
                            const int32_t* src_slots, const int32_t* keep_lens,
                            const int32_t* new_lens, int n, void* workspace,
                            size_t workspace_bytes, int32_t* dev_err, cudaStream_t stream) {
  using namespace pkv;
  pkv_status st = check_cache(cache);
  if (st != PKV_OK) return st;
  // (a page's 16-byte vectors are counted in 32 bits)
  if (n < 0 || static_cast<int64_t>(cache->page_size) * cache->num_kv_heads > (INT_MAX >> 6))
    return PKV_ERR_ARG;
  if (n == 0) return PKV_OK;
  if (!k_pool || !v_pool || !page_table || !page_refs || !dst_slots || !src_slots || !keep_lens ||
      !new_lens)
    return PKV_ERR_ARG;
  if (!aligned(k_pool, 16) || !aligned(v_pool, 16) || !aligned(page_table, 4) ||
      !aligned(page_refs, 4) || !aligned(dst_slots, 4) || !aligned(src_slots, 4) ||
      !aligned(keep_lens, 4) || !aligned(new_lens, 4) || !aligned(dev_err, 4))
    return PKV_ERR_ALIGN;
  int sms = 0;
  st = device_info(&sms);
  if (st != PKV_OK) return st;
  const PagesLayout l = update_layout(cache, n);
  if (static_cast<int64_t>(n) + l.n_chunks > INT_MAX) return PKV_ERR_ARG;
  if (workspace == nullptr || workspace_bytes < l.total) return PKV_ERR_WORKSPACE;
  if (!aligned(workspace, 256)) return PKV_ERR_ALIGN;
  PagesParams p =
      base_params(cache, l, k_pool, v_pool, page_table, page_refs, workspace, dev_err);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  p.need = reinterpret_cast<int32_t*>(ws + l.off_a);
  p.tail = reinterpret_cast<int32_t*>(ws + l.off_b);
  p.fresh = reinterpret_cast<uint32_t*>(ws + l.off_c);
  p.dst = dst_slots;
  p.src = src_slots;
  p.keep = keep_lens;
  p.newl = new_lens;
  p.n = n;
  cudaError_t e = launch_kernel(update_plan_kernel, dim3(n + l.n_chunks), dim3(kPlanThreads), 0,
                                stream, /*programmatic=*/true, p);
  if (e != cudaSuccess) return record_cuda_status(e);
  // parts per row: one CTA for each 16 KB of a page of one pool, as long as all rows'
  // parts are one wave (three CTAs per SM); at most 16
  const int64_t page_vecs = static_cast<int64_t>(p.page_size) * p.row_vecs;
  int64_t parts64 = (page_vecs + kPlanThreads * kInFlight - 1) / (kPlanThreads * kInFlight);
  const int64_t wave = 3 * static_cast<int64_t>(sms) / n;
  if (parts64 > wave) parts64 = wave;
  const unsigned parts = static_cast<unsigned>(parts64 < 1 ? 1 : parts64 > 16 ? 16 : parts64);
  e = launch_kernel(update_apply_kernel, dim3(n, parts), dim3(kPlanThreads), 0, stream,
                    /*programmatic=*/true, p);
  return record_cuda_status(e);
}

pkv_status pkv_compact_pages(const pkv_cache_desc* cache, void* k_pool, void* v_pool,
                             int32_t* page_table, int32_t* page_refs, int32_t* num_live,
                             void* workspace, size_t workspace_bytes, int32_t* dev_err,
                             cudaStream_t stream) {
  using namespace pkv;
  pkv_status st = check_cache(cache);
  if (st != PKV_OK) return st;
  if (!k_pool || !v_pool || !page_table || !page_refs) return PKV_ERR_ARG;
  if (!aligned(k_pool, 16) || !aligned(v_pool, 16) || !aligned(page_table, 4) ||
      !aligned(page_refs, 4) || !aligned(num_live, 4) || !aligned(dev_err, 4))
    return PKV_ERR_ALIGN;
  int sms = 0;
  st = device_info(&sms);
  if (st != PKV_OK) return st;
  const PagesLayout l = compact_layout(cache);
  if (workspace == nullptr || workspace_bytes < l.total) return PKV_ERR_WORKSPACE;
  if (!aligned(workspace, 256)) return PKV_ERR_ALIGN;
  PagesParams p =
      base_params(cache, l, k_pool, v_pool, page_table, page_refs, workspace, dev_err);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  p.live_list = reinterpret_cast<int32_t*>(ws + l.off_a);
  p.free_before = reinterpret_cast<int32_t*>(ws + l.off_b);
  p.num_live = num_live;
  cudaError_t e = launch_kernel(compact_plan_kernel, dim3(l.n_chunks), dim3(kPlanThreads), 0,
                                stream, /*programmatic=*/true, p);
  if (e != cudaSuccess) return record_cuda_status(e);
  e = launch_kernel(compact_apply_kernel, dim3(6 * sms), dim3(kPlanThreads), 0, stream,
                    /*programmatic=*/true, p);
  return record_cuda_status(e);
}

pkv_status pkv_commit_path(const pkv_cache_desc* cache, void* k_pool, void* v_pool,
                           const int32_t* page_table, const int32_t* path,
                           const int32_t* n_accepted, const int32_t* batch_idx,
                           const int32_t* ctx_lens, int batch, int n_nodes, int32_t* new_lens,
                           int32_t* dev_err, cudaStream_t stream) {
  using namespace pkv;
  pkv_status st = check_cache(cache);
  if (st != PKV_OK) return st;
  if (batch < 0 || n_nodes < 1 || n_nodes > PKV_MAX_TREE_NODES) return PKV_ERR_ARG;
  if (batch == 0) return PKV_OK;
  if (!k_pool || !v_pool || !page_table || !path || !n_accepted || !batch_idx || !ctx_lens)
    return PKV_ERR_ARG;
  if (!aligned(k_pool, 16) || !aligned(v_pool, 16) || !aligned(page_table, 4) ||
      !aligned(path, 4) || !aligned(n_accepted, 4) || !aligned(batch_idx, 4) ||
      !aligned(ctx_lens, 4) || !aligned(new_lens, 4) || !aligned(dev_err, 4))
    return PKV_ERR_ALIGN;
  int sms = 0;
  st = device_info(&sms);
  if (st != PKV_OK) return st;
  CommitParams p;
  p.pool[0] = k_pool;
  p.pool[1] = v_pool;
  p.page_table = page_table;
  p.path = path;
  p.n_accepted = n_accepted;
  p.batch_idx = batch_idx;
  p.ctx_lens = ctx_lens;
  p.new_lens = new_lens;
  p.dev_err = dev_err;
  p.n_nodes = n_nodes;
  p.row_vecs = cache->num_kv_heads * cache->head_dim * 2 / 16;
  p.page_size = cache->page_size;
  p.num_pages = cache->num_pages;
  p.max_batch = cache->max_batch;
  p.max_blocks = cache->max_blocks;
  return record_cuda_status(launch_kernel(commit_path_kernel, dim3(batch), dim3(kCommitThreads), 0,
                                          stream, /*programmatic=*/true, p));
}

}  // extern "C"
