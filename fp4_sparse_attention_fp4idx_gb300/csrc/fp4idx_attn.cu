// fp4idx_attn.cu -- the entry points of attention over the 8-bit cache
// (include/fp4idx_attention.h): checks, and the choice of a kernel and of its
// work split.

#include "fp4idx_attn.cuh"

namespace fp4idx_impl {
namespace {

constexpr int kPage = FP4IDX_KV_BLOCK;

// The tensor-core kernel of 256-row items (fp4idx_attn_tiles.cu) takes dense
// calls of at least kTileFrom query rows per sequence and key head and of more
// than kTileWork query rows x 64-key tiles in all.  Measured, the kernel for few
// rows against it, us, 8 key heads; D = 128, sequences of up to 8192 keys: 16 rows
// 181 / 322, 24 rows 328 / 323, 32 rows 339 / 325, 64 rows 660 / 324; 32 rows of
// 64 sequences x 2048 keys 131 / 135, of 16 x 8192 132 / 120, of 16 x 32768 274 /
// 303; D = 64, 32 rows, the same four: 213 / 252, 84 / 101, 84 / 92, 168 / 242; a
// window of 4096 + 4, 48 sequences x 4 key heads, D = 64 76 / 90, D = 128 97 / 114.
// So up to 32 rows the first is 10% slower at most, up to 44% faster at 32 rows
// and up to 78% at 16.
// Of 500 keys and 500 tokens x 4 rows, 4 sequences x 2 key heads (840 row-tiles a
// CTA) 28 / 40, x 8 key heads (3370) 93 / 39.
constexpr int64_t kTileFrom = 33;
constexpr int64_t kTileWork = 1200 * kMaxGrid;
constexpr int64_t kTileRows = 256;

// Query rows of an item of the kernel for few rows (fp4idx_attn_rows.cu).
int64_t item_rows(int64_t rows, int64_t head_dim) {
  return rows <= 8 ? 8 : rows <= 16 || head_dim == 128 ? 16 : 32;
}

struct Workspace {
  int64_t part_lse, cuts, total;  // offsets in bytes; partial outputs at 0
};

// Two partial outputs per CTA (an item cut at its share's start and one at
// its end), and the cut items.
Workspace workspace_of(int64_t rows, int64_t head_dim) {
  Workspace w;
  w.part_lse = 2 * kMaxGrid * rows * head_dim * 4;
  w.cuts = w.part_lse + 2 * kMaxGrid * rows * 4;
  w.total = w.cuts + (kMaxGrid * 16 + 255) / 256 * 256;
  return w;
}

bool workspace_args_ok(int64_t batch, int64_t max_q, int64_t num_heads, int64_t kv_heads,
                       int64_t head_dim) {
  return batch >= 0 && max_q >= 1 && kv_heads >= 1 && num_heads >= kv_heads &&
         num_heads % kv_heads == 0 && (head_dim == 64 || head_dim == 128) &&
         batch < (1ll << 31) && max_q < (1ll << 31) && num_heads < (1ll << 20) &&
         max_q < (1ll << 31) / num_heads &&
         (batch == 0 || max_q * num_heads + kv_heads < (1ll << 31) / batch);
}

// Checks that both forms make, and the arguments they share.
fp4idx_status common_args(AttnArgs& a, const void* q, int64_t q_token_stride,
                          int64_t q_head_stride, int dtype, const fp4idx_kv_cache* cache,
                          const int32_t* block_table, int64_t block_table_stride,
                          float softmax_scale, void* out, float* lse, int64_t items,
                          int64_t max_q, int64_t num_tokens, int64_t num_heads, void* workspace,
                          size_t workspace_bytes, uint32_t* err_flags, bool sparse,
                          int64_t tiles, bool no_pages) {
  const fp4idx_status cs = check_cache(cache);
  if (cs == FP4IDX_ERR_NULL || !q || (!block_table && !no_pages) || !out || !workspace)
    return FP4IDX_ERR_NULL;
  if (cs == FP4IDX_ERR_SHAPE || num_heads < 1 || num_heads % cache->kv_heads ||
      num_tokens >= (1ll << 31) ||
      !workspace_args_ok(items, max_q, num_heads, cache->kv_heads, cache->head_dim))
    return FP4IDX_ERR_SHAPE;
  const int64_t rows = max_q * (num_heads / cache->kv_heads);
  const bool few = sparse || rows < kTileFrom || items * cache->kv_heads * rows * tiles <= kTileWork;
  const int64_t R = few ? item_rows(rows, cache->head_dim) : kTileRows;
  const Workspace w = workspace_of(R, cache->head_dim);
  if (workspace_bytes < (size_t)w.total) return FP4IDX_ERR_SCRATCH;
  if (!dtype_ok(dtype) || !isfinite(softmax_scale)) return FP4IDX_ERR_ARG;
  if (cs != FP4IDX_OK || !aligned(q, 16) || q_token_stride % 8 || q_head_stride % 8 ||
      !aligned(block_table, 4) || !aligned(out, 16) || !aligned(lse, 4) ||
      !aligned(workspace, 16) || !aligned(err_flags, 4))
    return FP4IDX_ERR_ALIGN;
  a.q = static_cast<const uint16_t*>(q);
  a.q_ts = q_token_stride;
  a.q_hs = q_head_stride;
  a.half = dtype == FP4IDX_FP16;
  a.kc = cache->k_codes;
  a.vc = cache->v_codes;
  a.ks = cache->k_scale;
  a.vs = cache->v_scale;
  a.num_blocks = cache->num_blocks;
  a.cstride = cache->code_block_stride;
  a.sstride = cache->scale_block_stride;
  a.table = block_table;
  a.tstride = block_table_stride;
  a.batch = (int32_t)items;
  a.max_q = (int32_t)max_q;
  a.T = (int32_t)num_tokens;
  a.Hq = (int32_t)num_heads;
  a.Hkv = cache->kv_heads;
  a.G = (int32_t)(num_heads / cache->kv_heads);
  a.R = (int32_t)R;
  a.rc_max = (int32_t)((max_q * a.G + a.R - 1) / a.R);
  a.scale_log2 = softmax_scale * kLog2e;
  a.out = static_cast<uint16_t*>(out);
  a.lse = lse;
  uint8_t* const ws = static_cast<uint8_t*>(workspace);
  a.part_out = reinterpret_cast<float*>(ws);
  a.part_lse = reinterpret_cast<float*>(ws + w.part_lse);
  a.cuts = reinterpret_cast<int4*>(ws + w.cuts);
  a.err = err_flags;
  return FP4IDX_OK;
}

// Testing hook: what the next launch withholds (-1: nothing), taken once.
std::atomic<int64_t> g_attention_withhold{-1};

// `max_tiles`: 64-key tiles of an item, at most.
fp4idx_status launch(AttnArgs& a, int head_dim, bool sparse, int64_t max_tiles, void* stream) {
  a.withhold = -1;
  if (g_attention_withhold.load(std::memory_order_relaxed) >= 0) {
    const int64_t w = g_attention_withhold.exchange(-1);
    if (w < (1ll << 30)) a.withhold = (int32_t)w;
  }
  const int64_t items = (int64_t)a.batch * a.Hkv * a.rc_max;
  // The tensor-core kernel always cuts; the other one's dense form decides
  // again by the lengths, of which the bound is taken for the longest here and
  // the mean for less.
  const int64_t total = sparse ? items * max_tiles : items * max_tiles * 3 / 4;
  a.split = a.R == kTileRows || worth_cutting(items, total, max_tiles, a.R, kMaxGrid, sparse);
  const int64_t units = a.split ? items * max_tiles : items;
  const int grid = units < kMaxGrid ? (int)units : kMaxGrid;
  if (a.R == kTileRows)
    return launch_tiles(a, head_dim, grid, static_cast<cudaStream_t>(stream));
  return launch_rows(a, head_dim, sparse, grid, static_cast<cudaStream_t>(stream));
}

}  // namespace

void attention_withhold_next(int64_t index) { g_attention_withhold.store(index); }

}  // namespace fp4idx_impl

using namespace fp4idx_impl;

extern "C" size_t fp4idx_attention_workspace_bytes(int64_t batch, int64_t max_q,
                                                   int64_t num_heads, int64_t kv_heads,
                                                   int64_t head_dim) {
  if (!workspace_args_ok(batch, max_q, num_heads, kv_heads, head_dim)) return 0;
  const int64_t rows = max_q * (num_heads / kv_heads);
  return (size_t)workspace_of(rows < kTileFrom ? item_rows(rows, head_dim) : kTileRows, head_dim)
      .total;
}

extern "C" fp4idx_status fp4idx_paged_attention_fp8(
    const void* q, int64_t q_token_stride, int64_t q_head_stride, int dtype,
    const fp4idx_kv_cache* cache, const int32_t* block_table, int64_t block_table_stride,
    const int32_t* context_lens, const int32_t* q_starts, int64_t max_q, int64_t max_context,
    int64_t window, int64_t sinks, float softmax_scale, void* out, float* lse, int64_t batch,
    int64_t num_tokens, int64_t num_heads, void* workspace, size_t workspace_bytes,
    uint32_t* err_flags, void* stream) {
  if (batch < 0 || num_tokens < 0 || max_context < 0 || (batch == 0 && num_tokens > 0))
    return FP4IDX_ERR_SHAPE;
  if (batch == 0 || num_tokens == 0) return FP4IDX_OK;
  if (!context_lens) return FP4IDX_ERR_NULL;
  if (!q_starts) {
    if (num_tokens % batch) return FP4IDX_ERR_SHAPE;
    max_q = num_tokens / batch;
  }
  if (max_q < 1 || max_context >= (1 << 30) || max_q >= (1 << 30) ||
      block_table_stride < (max_context + kPage - 1) / kPage)
    return FP4IDX_ERR_SHAPE;
  if (window < 0 || sinks < 0) return FP4IDX_ERR_ARG;
  AttnArgs a = {};
  // a window that holds every context is no window
  a.window = window < max_context ? (int32_t)window : 0;
  a.sinks = (int32_t)(sinks < max_context ? sinks : max_context);
  int64_t tiles = (max_context + kPage - 1) / kPage;
  if (a.window > 0) {
    const int64_t seen = (a.window + max_q + kPage - 1) / kPage + 1 + (a.sinks + kPage - 1) / kPage;
    if (seen < tiles) tiles = seen;
  }
  if (tiles < 1) tiles = 1;
  const fp4idx_status st =
      common_args(a, q, q_token_stride, q_head_stride, dtype, cache, block_table,
                  block_table_stride, softmax_scale, out, lse, batch, max_q, num_tokens, num_heads,
                  workspace, workspace_bytes, err_flags, false, tiles, max_context == 0);
  if (st != FP4IDX_OK) return st;
  if (!aligned(context_lens, 4) || !aligned(q_starts, 4)) return FP4IDX_ERR_ALIGN;
  a.ctx = context_lens;
  a.starts = q_starts;
  a.max_context = (int32_t)max_context;
  return launch(a, cache->head_dim, false, tiles, stream);
}

extern "C" fp4idx_status fp4idx_sparse_attention_fp8(
    const void* q, int64_t q_token_stride, int64_t q_head_stride, int dtype,
    const fp4idx_kv_cache* cache, const int32_t* block_table, int64_t block_table_stride,
    int64_t block_table_pages, const int32_t* seq_ids, const int32_t* indices,
    int64_t indices_stride, int64_t num_selected, float softmax_scale, void* out, float* lse,
    int64_t batch, int64_t num_tokens, int64_t num_heads, void* workspace, size_t workspace_bytes,
    uint32_t* err_flags, void* stream) {
  if (batch < 0 || num_tokens < 0 || num_selected < 0 || (batch == 0 && num_tokens > 0))
    return FP4IDX_ERR_SHAPE;
  if (num_tokens == 0) return FP4IDX_OK;
  if (!indices && num_selected > 0) return FP4IDX_ERR_NULL;
  if ((!seq_ids && num_tokens % batch) || batch >= (1ll << 31) || num_selected >= (1 << 30) ||
      (num_tokens > 1 && indices_stride < num_selected) || block_table_pages < 0 ||
      block_table_pages >= (1 << 24) || (batch > 1 && block_table_stride < block_table_pages))
    return FP4IDX_ERR_SHAPE;
  AttnArgs a = {};
  const fp4idx_status st = common_args(a, q, q_token_stride, q_head_stride, dtype, cache,
                                       block_table, block_table_stride, softmax_scale, out, lse,
                                       num_tokens, 1, num_tokens, num_heads, workspace,
                                       workspace_bytes, err_flags, true, 1,
                                       block_table_pages == 0);
  if (st != FP4IDX_OK) return st;
  if (!aligned(seq_ids, 4) || !aligned(indices, 4)) return FP4IDX_ERR_ALIGN;
  a.seq_ids = seq_ids;
  a.indices = indices;
  a.idx_stride = indices_stride;
  a.nsel = (int32_t)num_selected;
  a.table_pages = (int32_t)block_table_pages;
  a.num_seqs = (int32_t)batch;
  a.per_seq = seq_ids ? 1 : (int32_t)(num_tokens / batch);
  const int64_t tiles = (num_selected + kPage - 1) / kPage;
  return launch(a, cache->head_dim, true, tiles < 1 ? 1 : tiles, stream);
}
