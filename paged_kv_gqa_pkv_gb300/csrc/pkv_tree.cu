// pkv_tree.cu - pkv_tree_attention: the choice among the forms of its kernel, the
// merge of partial results, validation and launches.
#include <cmath>

#include "pkv_tree.cuh"

namespace pkv {
namespace tree {

namespace {
constexpr int kMergeThreads = 256;
constexpr int kMergeUnroll = 2;        // partials in flight per merge thread

// Head dims per merge thread: column-major partials are read by single floats, and 16
// dims make whole sectors of the output.
constexpr int merge_cols(bool row_major) { return row_major ? 8 : 16; }
}  // namespace

// Joins the partials of items cut by range borders, and writes the rows of
// items that attend nothing. grid (items of a row, parts, rows): a CTA takes every
// parts-th block of its item's units; a unit is a row and merge_cols head dims.
// merge_split threads share a unit's partials where items have many, each taking every
// merge_split-th, kMergeUnroll at a time. Neighbouring threads have neighbouring units,
// along the head dims where a partial's O is row-major (kRowMajor), along the rows where
// it is column-major (the wide form's), so that they read neighbouring addresses. (With a
// unit's sharers side by side, one user's 4096 keys took 20 us for 15 at 32 rows, 42 for
// 26 at 256.)
template <bool kRowMajor>
__global__ void __launch_bounds__(kMergeThreads, 4) tree_merge_kernel(const TreeParams p) {
  constexpr int kMergeCols = merge_cols(kRowMajor);
  __shared__ float s_part[kMergeThreads][kMergeCols + 2];
  pdl_wait_primary();
  const int tid = threadIdx.x;
  const int b = blockIdx.z, item = blockIdx.x;
  const int kvh = p.row_blocks == 1 ? item : item / p.row_blocks;
  const int rb = item - kvh * p.row_blocks;
  const int before = p.prefix[b], tiles = p.prefix[b + 1] - before;
  const int split = p.merge_split;
  const int per_block = kMergeThreads / split;
  constexpr int kVecs = kHeadDim / kMergeCols;
  const int rows = min(p.rows - rb * kMaxRows, p.slot_rows);  // of this item
  const int units = rows * kVecs;
  const int live = p.tree_lens[b] << p.group_shift;  // rows of the sequence's tree
  int w0 = 0, w1 = 0, first_slot = 0;
  if (tiles > 0) {
    const int64_t total = static_cast<int64_t>(p.prefix[p.batch]) * p.items_per_row;
    const int64_t per = tiles_per_worker(p, total);
    const int64_t u = static_cast<int64_t>(before) * p.items_per_row +
                      static_cast<int64_t>(item) * tiles;
    // (ranges of 2^31 tiles do not occur: a launch would read a hundred terabytes)
    w0 = static_cast<int>(divide(u, static_cast<int>(per)));
    w1 = static_cast<int>(divide(u + tiles - 1, static_cast<int>(per)));
    if (w0 == w1) return;  // one range: written out there
    first_slot = u == w0 * per ? 0 : 1;  // later ranges hold the item in their first slot
  }
  const int share = tid >> (31 - __clz(per_block));  // (a power of two)
  const int stride = kRowMajor ? p.slot_rows : kMaxRows;  // rows of a partial
  const int64_t floats = slot_floats(stride);
  for (int block = blockIdx.y; block * per_block < units; block += gridDim.y) {
    const int unit = block * per_block + (tid & (per_block - 1));
    const bool mine = unit < units;
    const int prow = kRowMajor ? unit / kVecs : unit % rows;
    const int col = (kRowMajor ? unit % kVecs : unit / rows) * kMergeCols;
    const int r = rb * kMaxRows + prow;  // row of the sequence
    float M = -INFINITY, L = 0.f;
    float acc[kMergeCols];
#pragma unroll
    for (int e = 0; e < kMergeCols; ++e) acc[e] = 0.f;
    if (mine && tiles > 0 && r < live) {
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
            m[k] = __ldcg(s + kHeadDim * stride + prow);
            l[k] = __ldcg(s + (kHeadDim + 1) * stride + prow);
            if constexpr (kRowMajor) {
              const float4* o4 =
                  reinterpret_cast<const float4*>(s + static_cast<int64_t>(prow) * kHeadDim + col);
              const float4 x = __ldcg(o4), y = __ldcg(o4 + 1);
              o[k][0] = x.x, o[k][1] = x.y, o[k][2] = x.z, o[k][3] = x.w;
              o[k][4] = y.x, o[k][5] = y.y, o[k][6] = y.z, o[k][7] = y.w;
            } else {
              const float* at = s + col * kMaxRows + prow;
#pragma unroll
              for (int e = 0; e < kMergeCols; ++e)
                o[k][e] = __ldcg(at + e * kMaxRows);
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
        for (int k = 1; k < split; ++k) top = fmaxf(top, s_part[tid + k * per_block][kMergeCols]);
        L = 0.f;
#pragma unroll
        for (int e = 0; e < kMergeCols; ++e) acc[e] = 0.f;
        for (int k = 0; k < split; ++k) {
          const float l = s_part[tid + k * per_block][kMergeCols + 1];
          if (l == 0.f) continue;
          const float a = ex2(s_part[tid + k * per_block][kMergeCols] - top);
          L = fmaf(l, a, L);
#pragma unroll
          for (int e = 0; e < kMergeCols; ++e) acc[e] = fmaf(s_part[tid + k * per_block][e], a, acc[e]);
        }
        M = top;
      }
    }
    if (mine && share == 0) {
      const bool has = L != 0.f;
      const float inv = has ? 1.f / L : 0.f;
      const int64_t orow = (static_cast<int64_t>(b) * p.n_nodes + (r >> p.group_shift)) *
                               p.num_q_heads +
                           kvh * p.group + (r & (p.group - 1));
#pragma unroll
      for (int e = 0; e < kMergeCols; e += 8) {
        uint4 w;
        w.x = pack_bf16x2(acc[e] * inv, acc[e + 1] * inv);
        w.y = pack_bf16x2(acc[e + 2] * inv, acc[e + 3] * inv);
        w.z = pack_bf16x2(acc[e + 4] * inv, acc[e + 5] * inv);
        w.w = pack_bf16x2(acc[e + 6] * inv, acc[e + 7] * inv);
        *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.out) + orow * kHeadDim + col + e) = w;
      }
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

// Items by which a form is picked: a full launch's where there are several, so
// that a workspace for a batch serves every smaller one.
int64_t launch_items(int batch, int hkv) {
  return static_cast<int64_t>(batch < kTreeMaxBatch ? batch : kTreeMaxBatch) * hkv;
}

struct TreeLayout {
  size_t off_partials, total;
};

// Tile prefix, then two partial slots per worker.
TreeLayout tree_layout(int rows, int workers) {
  TreeLayout l;
  l.off_partials = ((kTreeMaxBatch + 1) * 4 + 255) / 256 * 256;
  const size_t part = 2 * static_cast<size_t>(workers) *
                      static_cast<size_t>(slot_floats(slot_rows(rows))) * 4;
  l.total = l.off_partials + (part + 255) / 256 * 256;
  return l;
}

// The form that serves `rows` query rows per item and `items` items: the streaming
// one up to 8 rows of many items (measured against the tile form at the head of its
// file), the tile form up to 128 rows, the wide one above: 67 us at 128 rows against 68
// at 132 for 64 sequences of ~768 keys, 78 against 86 for 32 of ~2560, 168 against 211 for
// 8 of 32768, where the wide form computes twice the rows. Up to 64 rows the tile form
// has two workers per CTA; with one busy it takes 74 us for 53 (64 x ~768 keys, 64 rows) and
// 240 for 166 (8 x 32768).
enum class Form { kStream, kSingle, kShared, kWide };

Form pick_form(int rows, int64_t items, int sms) {
  if (rows <= 8 && items >= sms) return Form::kStream;
  return rows <= 64 ? Form::kSingle : rows <= 128 ? Form::kShared : Form::kWide;
}

int form_workers(Form f, int sms) {
  return f == Form::kStream ? sms * kStreamWarps : f == Form::kSingle ? 2 * sms : sms;
}

cudaError_t launch_merge(const TreeParams& p, int sms, cudaStream_t stream) {
  // about 16 CTAs per SM in all, and no more per item than it has blocks of units
  const int items = p.batch * p.items_per_row;
  const int per_block = kMergeThreads / p.merge_split;
  const bool wide = p.rows > kBM;
  const int blocks = (p.slot_rows * (kHeadDim / merge_cols(!wide)) + per_block - 1) / per_block;
  const int want = (16 * sms + items - 1) / items;
  return launch_kernel(wide ? tree_merge_kernel<false> : tree_merge_kernel<true>,
                       dim3(p.items_per_row, blocks < want ? blocks : want, p.batch),
                       dim3(kMergeThreads), 0, stream, /*programmatic=*/true, p);
}

}  // namespace
}  // namespace tree
}  // namespace pkv

extern "C" size_t pkv_tree_workspace_size(const pkv_cache_desc* cache, int batch, int n_nodes,
                                          int num_q_heads) {
  using namespace pkv;
  using namespace pkv::tree;
  if (check_cache(cache) != PKV_OK || batch < 0) return 0;
  if (n_nodes < 1 || n_nodes > PKV_MAX_TREE_NODES) return 0;
  if (!tree_group_ok(num_q_heads, cache->num_kv_heads)) return 0;
  int sms = 0;
  if (device_info(&sms) != PKV_OK) return 0;
  const int rows = n_nodes * (num_q_heads / cache->num_kv_heads);
  const Form form = pick_form(rows, launch_items(batch, cache->num_kv_heads), sms);
  return tree_layout(rows, form_workers(form, sms)).total;
}

extern "C" pkv_status pkv_tree_attention(
    const pkv_cache_desc* cache, const void* k_pool, const void* v_pool, const int32_t* page_table,
    const void* q, int num_q_heads, const int32_t* parents, const int32_t* tree_lens,
    const int32_t* batch_idx, const int32_t* ctx_lens, int batch, int n_nodes, float scale,
    void* out, float* lse, void* workspace, size_t workspace_bytes, int32_t* dev_err,
    cudaStream_t stream) {
  using namespace pkv;
  using namespace pkv::tree;
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
  p.group_shift = 0;
  while ((1 << p.group_shift) < p.group) ++p.group_shift;
  p.rows = n_nodes * p.group;
  const Form form = pick_form(p.rows, launch_items(batch, cache->num_kv_heads), sms);
  p.workers = form_workers(form, sms);
  const TreeLayout lay = tree_layout(p.rows, p.workers);
  if (workspace == nullptr || workspace_bytes < lay.total) return PKV_ERR_WORKSPACE;
  if (!aligned(workspace, 256)) return PKV_ERR_ALIGN;
  p.min_tiles = form == Form::kStream ? 8 : 1;
  p.n_nodes = n_nodes;
  p.num_q_heads = num_q_heads;
  p.num_kv_heads = cache->num_kv_heads;
  p.row_blocks = (p.rows + kMaxRows - 1) / kMaxRows;
  p.items_per_row = cache->num_kv_heads * p.row_blocks;
  p.q_box_nodes = p.rows > kBM ? kBM / p.group : n_nodes;
  p.page_size = cache->page_size;
  p.num_pages = cache->num_pages;
  p.max_batch = cache->max_batch;
  p.max_blocks = cache->max_blocks;
  p.box_rows = cache->page_size < kBN ? cache->page_size : kBN;
  p.slot_rows = slot_rows(p.rows);
  p.qscale = scale * 1.4426950408889634f;
  p.page_table = page_table;
  p.dev_err = dev_err;
  p.prefix = static_cast<int32_t*>(workspace);
  p.partials = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + lay.off_partials);

  CUtensorMap qmap, kmap, vmap;
  if (form == Form::kStream) {
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
    cudaError_t e = form == Form::kStream ? launch_stream_form(qmap, kmap, vmap, p, sms, dev, stream)
                    : form == Form::kWide ? launch_wide_form(qmap, kmap, vmap, p, sms, dev, stream)
                                          : launch_tile_form(qmap, kmap, vmap, p, sms, dev, stream);
    if (e == cudaSuccess) e = launch_merge(p, sms, stream);
    if (e != cudaSuccess) return record_cuda_status(e);
  }
  return PKV_OK;
}
