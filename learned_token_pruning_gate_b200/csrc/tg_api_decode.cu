// C ABI of the decoding calls: argument validation and dispatch.  What the tables,
// lengths and parents hold is device memory, which the kernels check themselves.
#include "tg_internal.cuh"

using namespace tg;

namespace {

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// The pages' geometry: log2 of the page size in *shift.
tg_status check_pages(int32_t n_pages, int32_t page_size, int32_t max_pages, int32_t* shift) {
  if (n_pages < 0 || max_pages < 0)
    return set_error(TG_ERR_INVALID_ARG, "n_pages=%d max_pages=%d", n_pages, max_pages);
  if (page_size != 16 && page_size != 32 && page_size != 64 && page_size != 128)
    return set_error(TG_ERR_UNSUPPORTED, "page_size=%d (supported: 16, 32, 64, 128)", page_size);
  if (n_pages > (1 << 20) || max_pages > (1 << 20))
    return set_error(TG_ERR_UNSUPPORTED, "n_pages=%d max_pages=%d exceed 2^20", n_pages, max_pages);
  *shift = page_size == 16 ? 4 : page_size == 32 ? 5 : page_size == 64 ? 6 : 7;
  return TG_OK;
}

tg_status check_batch(int32_t batch, const char* name) {
  if (batch < 0) return set_error(TG_ERR_INVALID_ARG, "%s=%d is negative", name, batch);
  if (batch > TG_MAX_SEQS)
    return set_error(TG_ERR_UNSUPPORTED, "%s=%d exceeds TG_MAX_SEQS=%d", name, batch, TG_MAX_SEQS);
  return TG_OK;
}

tg_status check_heads(tg_dtype dtype, int32_t n_q_heads, int32_t n_kv_heads, int32_t head_dim) {
  if (dtype != TG_BF16 && dtype != TG_FP32) return set_error(TG_ERR_DTYPE, "dtype %d", dtype);
  if (n_q_heads <= 0 || n_kv_heads <= 0 || n_q_heads % n_kv_heads != 0)
    return set_error(TG_ERR_SHAPE, "n_q_heads=%d n_kv_heads=%d", n_q_heads, n_kv_heads);
  if (n_q_heads > 512) return set_error(TG_ERR_UNSUPPORTED, "n_q_heads=%d exceeds 512", n_q_heads);
  if (head_dim != 64 && head_dim != 128)
    return set_error(TG_ERR_UNSUPPORTED, "head_dim=%d (supported: 64, 128)", head_dim);
  return TG_OK;
}

bool overlap(const void* a, size_t na, const void* b, size_t nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return na > 0 && nb > 0 && x < y + nb && y < x + na;
}

struct Span {
  const void* p;
  size_t bytes;
  const char* name;
};

// No output may lie in another output or in an input, but for out[i] == in[i] exactly where `same` says so.
tg_status check_spans(const Span* in, int n_in, const Span* out, int n_out, const int* same) {
  for (int i = 0; i < n_out; ++i) {
    for (int j = 0; j < i; ++j)
      if (overlap(out[i].p, out[i].bytes, out[j].p, out[j].bytes))
        return set_error(TG_ERR_INVALID_ARG, "%s overlaps %s", out[i].name, out[j].name);
    for (int j = 0; j < n_in; ++j) {
      if (!in[j].p || !overlap(out[i].p, out[i].bytes, in[j].p, in[j].bytes)) continue;
      if (same[i] == j && out[i].p == in[j].p) continue;
      return set_error(TG_ERR_INVALID_ARG, "%s overlaps %s", out[i].name, in[j].name);
    }
  }
  return TG_OK;
}

tg_status status_word(uint32_t** w) {
  *w = device_status_word();
  return *w ? TG_OK : set_error(TG_ERR_CUDA, "cannot resolve the device status word");
}

}  // namespace

extern "C" {

tg_status tg_paged_attention_workspace_bytes(tg_dtype dtype, int32_t batch, int32_t n_q_heads,
                                             int32_t n_kv_heads, int32_t head_dim, size_t* bytes_out) {
  if (!bytes_out) return set_error(TG_ERR_INVALID_ARG, "bytes_out is NULL");
  *bytes_out = 0;
  tg_status r = check_heads(dtype, n_q_heads, n_kv_heads, head_dim);
  if (r != TG_OK || (r = check_batch(batch, "batch")) != TG_OK) return r;
  if (batch > 0) *bytes_out = paged_attention_workspace_bytes(dtype, batch, n_q_heads, n_kv_heads, head_dim);
  return TG_OK;
}

tg_status tg_paged_attention(const void* q, const void* k_pages, const void* v_pages, tg_dtype dtype,
                             int32_t batch, int32_t n_q_heads, int32_t n_kv_heads, int32_t head_dim,
                             int32_t n_pages, int32_t page_size, const int32_t* table,
                             int32_t max_pages, const int32_t* lens, const float* logsig_pages,
                             const float* gain, const float* temp, void* out, float* lse,
                             void* workspace, size_t workspace_bytes, tg_stream_t stream) {
  PagedAttnArgs a = {};
  tg_status r = check_heads(dtype, n_q_heads, n_kv_heads, head_dim);
  if (r != TG_OK || (r = check_batch(batch, "batch")) != TG_OK ||
      (r = check_pages(n_pages, page_size, max_pages, &a.page_shift)) != TG_OK)
    return r;
  // (the kernel counts tiles of at least 64 keys in 32 bits)
  if (static_cast<int64_t>(batch) * max_pages * page_size > (int64_t{1} << 36))
    return set_error(TG_ERR_UNSUPPORTED, "batch x max_pages x page_size = %lld exceeds 2^36",
                     static_cast<long long>(static_cast<int64_t>(batch) * max_pages * page_size));
  if (batch == 0) return TG_OK;
  if (!q || !lens || !gain || !temp || !out || (max_pages > 0 && !table) ||
      (n_pages > 0 && (!k_pages || !v_pages)))
    return set_error(TG_ERR_INVALID_ARG, "null pointer");
  if (!aligned16(q) || !aligned16(k_pages) || !aligned16(v_pages) || !aligned16(out))
    return set_error(TG_ERR_ALIGNMENT, "q, k_pages, v_pages and out must be 16-byte aligned");
  size_t need = 0;
  if (workspace) {
    need = paged_attention_workspace_bytes(dtype, batch, n_q_heads, n_kv_heads, head_dim);
    if (workspace_bytes < need)
      return set_error(TG_ERR_WORKSPACE, "paged attention workspace: %zu bytes given, %zu needed",
                       workspace_bytes, need);
    if (!aligned16(workspace)) return set_error(TG_ERR_ALIGNMENT, "workspace must be 16-byte aligned");
  }
  const size_t rows = static_cast<size_t>(batch) * n_q_heads, esz = dtype == TG_BF16 ? 2 : 4;
  const size_t tokens = static_cast<size_t>(n_pages) * page_size, pool_bytes = tokens * n_kv_heads * head_dim * esz;
  const Span in[] = {{q, rows * head_dim * esz, "q"}, {k_pages, pool_bytes, "k_pages"},
                     {v_pages, pool_bytes, "v_pages"}, {table, 4 * static_cast<size_t>(batch) * max_pages, "table"},
                     {lens, 4 * static_cast<size_t>(batch), "lens"}, {logsig_pages, 4 * tokens, "logsig_pages"},
                     {gain, 4 * static_cast<size_t>(n_q_heads), "gain"},
                     {temp, 4 * static_cast<size_t>(n_q_heads), "temp"}};
  const Span outs[] = {{out, rows * head_dim * esz, "out"}, {lse, lse ? 4 * rows : 0, "lse"},
                       {workspace, need, "workspace"}};
  const int same[] = {0, -1, -1};  // (a unit's query rows are read before its output is written)
  if ((r = check_spans(in, 8, outs, 3, same)) != TG_OK) return r;
  if ((r = status_word(&a.status)) != TG_OK) return r;
  a.q = q;
  a.k_pages = k_pages;
  a.v_pages = v_pages;
  a.table = table;
  a.lens = lens;
  a.logsig_pages = logsig_pages;
  a.gain = gain;
  a.temp = temp;
  a.out = out;
  a.lse = lse;
  a.batch = batch;
  a.hq = n_q_heads;
  a.hkv = n_kv_heads;
  a.n_pages = n_pages;
  a.max_pages = max_pages;
  return launch_paged_attention(a, dtype, head_dim, workspace, reinterpret_cast<cudaStream_t>(stream));
}

tg_status tg_cache_update(const int32_t* table_in, const int32_t* lens_in, int32_t batch_in,
                          const int32_t* refs_in, int32_t n_pages, int32_t page_size,
                          int32_t max_pages, const int32_t* parent, int32_t batch_out,
                          const int32_t* cu_new, int32_t* table_out, int32_t* lens_out,
                          int32_t* refs_out, int32_t* start, int32_t* copy_src, int32_t* copy_dst,
                          tg_stream_t stream) {
  CacheUpdateArgs a = {};
  tg_status r = check_batch(batch_in, "batch_in");
  if (r != TG_OK || (r = check_batch(batch_out, "batch_out")) != TG_OK ||
      (r = check_pages(n_pages, page_size, max_pages, &a.page_shift)) != TG_OK)
    return r;
  if (!parent && batch_in != batch_out)
    return set_error(TG_ERR_SHAPE, "batch_in=%d batch_out=%d without parents", batch_in, batch_out);
  if (batch_in == 0 && batch_out == 0 && refs_in == refs_out) return TG_OK;
  if ((batch_in > 0 && (!lens_in || (max_pages > 0 && !table_in))) ||
      (n_pages > 0 && (!refs_in || !refs_out)) ||
      (batch_out > 0 && (!lens_out || !start || !copy_src || !copy_dst || (max_pages > 0 && !table_out))))
    return set_error(TG_ERR_INVALID_ARG, "null pointer");
  const size_t bi = batch_in, bo = batch_out, np = n_pages, mp = max_pages;
  const Span in[] = {{table_in, 4 * bi * mp, "table_in"}, {lens_in, 4 * bi, "lens_in"},
                     {refs_in, 4 * np, "refs_in"}, {parent, 4 * bo, "parent"},
                     {cu_new, 4 * (bo + 1), "cu_new"}};
  const Span out[] = {{table_out, 4 * bo * mp, "table_out"}, {lens_out, 4 * bo, "lens_out"},
                      {refs_out, 4 * np, "refs_out"}, {start, 4 * bo, "start"},
                      {copy_src, 4 * bo, "copy_src"}, {copy_dst, 4 * bo, "copy_dst"}};
  const int same[] = {parent ? -1 : 0, parent ? -1 : 1, 2, -1, -1, -1};
  if ((r = check_spans(in, 5, out, 6, same)) != TG_OK) return r;
  if ((r = status_word(&a.status)) != TG_OK) return r;
  a.table_in = table_in;
  a.lens_in = lens_in;
  a.refs_in = refs_in;
  a.parent = parent;
  a.cu_new = cu_new;
  a.table_out = table_out;
  a.lens_out = lens_out;
  a.refs_out = refs_out;
  a.start = start;
  a.copy_src = copy_src;
  a.copy_dst = copy_dst;
  a.batch_in = batch_in;
  a.batch_out = batch_out;
  a.n_pages = n_pages;
  a.max_pages = max_pages;
  return launch_cache_update(a, reinterpret_cast<cudaStream_t>(stream));
}

tg_status tg_cache_compact(const int32_t* table_in, const int32_t* lens, int32_t batch,
                           const int32_t* refs_in, int32_t n_pages, int32_t page_size,
                           int32_t max_pages, int32_t* table_out, int32_t* refs_out, int32_t* page_map,
                           int32_t* copy_src, int32_t* copy_dst, int32_t* counts, tg_stream_t stream) {
  CacheCompactArgs a = {};
  tg_status r = check_batch(batch, "batch");
  if (r != TG_OK || (r = check_pages(n_pages, page_size, max_pages, &a.page_shift)) != TG_OK) return r;
  if (!counts || (batch > 0 && (!lens || (max_pages > 0 && (!table_in || !table_out)))) ||
      (n_pages > 0 && (!refs_in || !refs_out || !page_map || !copy_src || !copy_dst)))
    return set_error(TG_ERR_INVALID_ARG, "null pointer");
  const size_t b = batch, np = n_pages, mp = max_pages;
  const Span in[] = {{table_in, 4 * b * mp, "table_in"}, {lens, 4 * b, "lens"}, {refs_in, 4 * np, "refs_in"}};
  const Span out[] = {{table_out, 4 * b * mp, "table_out"}, {refs_out, 4 * np, "refs_out"},
                      {page_map, 4 * np, "page_map"}, {copy_src, 4 * np, "copy_src"},
                      {copy_dst, 4 * np, "copy_dst"}, {counts, 8, "counts"}};
  const int same[] = {0, 2, -1, -1, -1, -1};
  if ((r = check_spans(in, 3, out, 6, same)) != TG_OK) return r;
  if ((r = status_word(&a.status)) != TG_OK) return r;
  a.table_in = table_in;
  a.lens = lens;
  a.refs_in = refs_in;
  a.table_out = table_out;
  a.refs_out = refs_out;
  a.page_map = page_map;
  a.copy_src = copy_src;
  a.copy_dst = copy_dst;
  a.counts = counts;
  a.batch = batch;
  a.n_pages = n_pages;
  a.max_pages = max_pages;
  return launch_cache_compact(a, reinterpret_cast<cudaStream_t>(stream));
}

tg_status tg_cache_copy_pages(const tg_page_pool* pools, int32_t n_pools, int32_t n_pages,
                              const int32_t* copy_src, const int32_t* copy_dst, int32_t n_copies,
                              const int32_t* count, tg_stream_t stream) {
  if (n_pools < 0 || n_pages < 0 || n_copies < 0)
    return set_error(TG_ERR_INVALID_ARG, "n_pools=%d n_pages=%d n_copies=%d", n_pools, n_pages, n_copies);
  if (n_pools > TG_MAX_GATHER_TENSORS)
    return set_error(TG_ERR_UNSUPPORTED, "n_pools=%d exceeds %d", n_pools, TG_MAX_GATHER_TENSORS);
  if (n_pools > 0 && !pools) return set_error(TG_ERR_INVALID_ARG, "pools is null");
  int64_t items = 0;
  for (int i = 0; i < n_pools; ++i) {
    if (pools[i].page_bytes <= 0 || pools[i].layers < 0)
      return set_error(TG_ERR_SHAPE, "pool %d: page_bytes=%lld layers=%d", i,
                       static_cast<long long>(pools[i].page_bytes), pools[i].layers);
    if (pools[i].page_bytes > (int64_t{1} << 30))
      return set_error(TG_ERR_UNSUPPORTED, "pool %d: pages above 1 GiB", i);
    if (pools[i].page_bytes % 16 != 0 || !aligned16(pools[i].base))
      return set_error(TG_ERR_ALIGNMENT, "pool %d: base and page_bytes must be multiples of 16", i);
    if (n_pages > 0 && pools[i].layers > 0 && !pools[i].base)
      return set_error(TG_ERR_INVALID_ARG, "pool %d: null pointer", i);
    items += (pools[i].page_bytes / 16 + 2047) / 2048 * pools[i].layers;
  }
  if (items > INT32_MAX) return set_error(TG_ERR_UNSUPPORTED, "pools too large for one call");
  if (items == 0 || n_pages == 0 || n_copies == 0) return TG_OK;
  if (!copy_src || !copy_dst) return set_error(TG_ERR_INVALID_ARG, "null pointer");
  uint32_t* status = nullptr;
  tg_status r = status_word(&status);
  if (r != TG_OK) return r;
  return launch_cache_copy(pools, n_pools, n_pages, copy_src, copy_dst, n_copies, count, status,
                           reinterpret_cast<cudaStream_t>(stream));
}

tg_status tg_cache_append(const void* k, const void* v, const float* logsig, tg_dtype dtype, int64_t rows,
                          int32_t batch, const int32_t* cu_new, const int32_t* start,
                          int32_t n_kv_heads, int32_t head_dim, int32_t n_pages, int32_t page_size,
                          const int32_t* table, int32_t max_pages, void* k_pages, void* v_pages,
                          float* logsig_pages, tg_stream_t stream) {
  CacheAppendArgs a = {};
  if (dtype != TG_BF16 && dtype != TG_FP32) return set_error(TG_ERR_DTYPE, "dtype %d", dtype);
  tg_status r = check_batch(batch, "batch");
  if (r != TG_OK || (r = check_pages(n_pages, page_size, max_pages, &a.page_shift)) != TG_OK) return r;
  if (rows < 0 || rows > INT32_MAX)
    return set_error(TG_ERR_INVALID_ARG, "rows=%lld", static_cast<long long>(rows));
  if (n_kv_heads <= 0 || head_dim <= 0 || n_kv_heads > 1024 || head_dim > 1024)
    return set_error(TG_ERR_SHAPE, "n_kv_heads=%d head_dim=%d", n_kv_heads, head_dim);
  const int esz = dtype == TG_BF16 ? 2 : 4;
  if (head_dim * esz % 16 != 0) return set_error(TG_ERR_ALIGNMENT, "head_dim=%d is not a multiple of 16 bytes", head_dim);
  if (rows == 0 || batch == 0 || n_pages == 0 || max_pages == 0) return TG_OK;
  if (!k || !v || !cu_new || !start || !table || !k_pages || !v_pages)
    return set_error(TG_ERR_INVALID_ARG, "null pointer");
  if (!aligned16(k) || !aligned16(v) || !aligned16(k_pages) || !aligned16(v_pages))
    return set_error(TG_ERR_ALIGNMENT, "k, v, k_pages and v_pages must be 16-byte aligned");
  const size_t row_bytes = static_cast<size_t>(rows) * n_kv_heads * head_dim * esz;
  const size_t pool_bytes = static_cast<size_t>(n_pages) * page_size * n_kv_heads * head_dim * esz;
  const size_t gate_bytes = logsig_pages ? 4 * static_cast<size_t>(n_pages) * page_size : 0;
  const Span in[] = {{k, row_bytes, "k"}, {v, row_bytes, "v"}, {logsig, 4 * static_cast<size_t>(rows), "logsig"}};
  const Span out[] = {{k_pages, pool_bytes, "k_pages"}, {v_pages, pool_bytes, "v_pages"},
                      {logsig_pages, gate_bytes, "logsig_pages"}};
  const int same[] = {-1, -1, -1};
  if ((r = check_spans(in, 3, out, 3, same)) != TG_OK) return r;
  if ((r = status_word(&a.status)) != TG_OK) return r;
  a.k = k;
  a.v = v;
  a.logsig = logsig;
  a.cu_new = cu_new;
  a.start = start;
  a.table = table;
  a.k_pages = k_pages;
  a.v_pages = v_pages;
  a.logsig_pages = logsig_pages;
  a.rows = rows;
  a.batch = batch;
  a.hkv = n_kv_heads;
  a.head_bytes = head_dim * esz;
  a.n_pages = n_pages;
  a.max_pages = max_pages;
  return launch_cache_append(a, reinterpret_cast<cudaStream_t>(stream));
}

tg_status tg_gated_delta_step(const void* q, const void* k, const void* v, tg_dtype dtype,
                              const float* log_alpha, const float* beta, int32_t batch,
                              int32_t n_heads, int32_t head_dim, float eps, const float* state_in,
                              int32_t n_states, const int32_t* parent, float* state_out, void* out,
                              tg_stream_t stream) {
  if (dtype != TG_BF16 && dtype != TG_FP32) return set_error(TG_ERR_DTYPE, "dtype %d", dtype);
  if (batch < 0 || n_states < 0)
    return set_error(TG_ERR_INVALID_ARG, "batch=%d n_states=%d", batch, n_states);
  if (n_heads <= 0) return set_error(TG_ERR_SHAPE, "n_heads=%d", n_heads);
  if (head_dim != 64 && head_dim != 128)
    return set_error(TG_ERR_UNSUPPORTED, "head_dim=%d (supported: 64, 128)", head_dim);
  if (!(eps >= 0.0f)) return set_error(TG_ERR_INVALID_ARG, "eps must be >= 0");
  if (!parent && n_states < batch)
    return set_error(TG_ERR_SHAPE, "n_states=%d for batch=%d without parents", n_states, batch);
  if (static_cast<int64_t>(batch) * n_heads > INT32_MAX / 8)
    return set_error(TG_ERR_UNSUPPORTED, "batch x n_heads = %lld exceeds one launch",
                     static_cast<long long>(batch) * n_heads);
  if (batch == 0) return TG_OK;
  if (!q || !k || !v || !log_alpha || !beta || !state_out || !out || (n_states > 0 && !state_in))
    return set_error(TG_ERR_INVALID_ARG, "null pointer");
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(state_in) || !aligned16(state_out))
    return set_error(TG_ERR_ALIGNMENT, "q, k, v, state_in and state_out must be 16-byte aligned");
  const size_t heads = static_cast<size_t>(batch) * n_heads, one = 4 * static_cast<size_t>(n_heads) * head_dim * head_dim;
  const size_t row_bytes = heads * head_dim * (dtype == TG_BF16 ? 2 : 4);
  const Span in[] = {{state_in, one * n_states, "state_in"}, {q, row_bytes, "q"}, {k, row_bytes, "k"},
                     {v, row_bytes, "v"}, {log_alpha, 4 * heads, "log_alpha"}, {beta, 4 * heads, "beta"},
                     {parent, 4 * static_cast<size_t>(batch), "parent"}};
  const Span outs[] = {{state_out, one * batch, "state_out"}, {out, row_bytes, "out"}};
  const int same[] = {parent ? -1 : 0, -1};
  tg_status r = check_spans(in, 7, outs, 2, same);
  if (r != TG_OK) return r;
  uint32_t* status = nullptr;
  if ((r = status_word(&status)) != TG_OK) return r;
  return launch_delta_step(q, k, v, dtype, log_alpha, beta, batch, n_heads, head_dim, eps, state_in,
                           n_states, parent, state_out, out, status,
                           reinterpret_cast<cudaStream_t>(stream));
}

static tg_status check_beams(int32_t n_groups, int32_t beams, int32_t vocab, int32_t n_out) {
  if (n_groups < 0) return set_error(TG_ERR_INVALID_ARG, "n_groups=%d", n_groups);
  if (beams <= 0 || vocab <= 0 || n_out <= 0)
    return set_error(TG_ERR_SHAPE, "beams=%d vocab=%d n_out=%d", beams, vocab, n_out);
  if (beams > TG_MAX_BEAMS || n_out > 2 * TG_MAX_BEAMS || vocab > (1 << 20))
    return set_error(TG_ERR_UNSUPPORTED, "beams=%d n_out=%d vocab=%d (at most %d, %d, 2^20)", beams, n_out,
                     vocab, TG_MAX_BEAMS, 2 * TG_MAX_BEAMS);
  if (static_cast<int64_t>(n_groups) * beams > (1 << 20))
    return set_error(TG_ERR_UNSUPPORTED, "n_groups x beams = %lld exceeds 2^20",
                     static_cast<long long>(n_groups) * beams);
  return TG_OK;
}

tg_status tg_beam_select_workspace_bytes(int32_t n_groups, int32_t beams, int32_t vocab, int32_t n_out,
                                         size_t* bytes_out) {
  if (!bytes_out) return set_error(TG_ERR_INVALID_ARG, "bytes_out is NULL");
  *bytes_out = 0;
  tg_status r = check_beams(n_groups, beams, vocab, n_out);
  if (r != TG_OK) return r;
  *bytes_out = beam_select_workspace_bytes(n_groups, beams, vocab, n_out);
  return TG_OK;
}

tg_status tg_beam_select(const void* logits, tg_dtype dtype, const float* scores, int32_t n_groups,
                         int32_t beams, int32_t vocab, int32_t n_out, float* scores_out,
                         int32_t* parent_out, int32_t* token_out, void* workspace,
                         size_t workspace_bytes, tg_stream_t stream) {
  if (dtype != TG_BF16 && dtype != TG_FP32) return set_error(TG_ERR_DTYPE, "dtype %d", dtype);
  tg_status r = check_beams(n_groups, beams, vocab, n_out);
  if (r != TG_OK) return r;
  if (n_groups == 0) return TG_OK;
  if (!logits || !scores || !scores_out || !parent_out || !token_out)
    return set_error(TG_ERR_INVALID_ARG, "null pointer");
  const size_t need = beam_select_workspace_bytes(n_groups, beams, vocab, n_out);
  if (!workspace || workspace_bytes < need)
    return set_error(TG_ERR_WORKSPACE, "beam selection workspace: %zu bytes given, %zu needed",
                     workspace ? workspace_bytes : 0, need);
  if (!aligned16(logits) || !aligned16(workspace))
    return set_error(TG_ERR_ALIGNMENT, "logits and workspace must be 16-byte aligned");
  const size_t rows = static_cast<size_t>(n_groups) * beams, picks = 4 * static_cast<size_t>(n_groups) * n_out;
  const Span in[] = {{logits, rows * vocab * (dtype == TG_BF16 ? 2 : 4), "logits"}, {scores, 4 * rows, "scores"}};
  const Span out[] = {{scores_out, picks, "scores_out"}, {parent_out, picks, "parent_out"},
                      {token_out, picks, "token_out"}, {workspace, need, "workspace"}};
  const int same[] = {-1, -1, -1, -1};
  if ((r = check_spans(in, 2, out, 4, same)) != TG_OK) return r;
  return launch_beam_select(logits, dtype, scores, n_groups, beams, vocab, n_out, scores_out, parent_out,
                            token_out, workspace, reinterpret_cast<cudaStream_t>(stream));
}

}  // extern "C"
