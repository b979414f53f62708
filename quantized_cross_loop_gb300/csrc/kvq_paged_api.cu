// kvq_paged_api.cu — the extern "C" entry points of the paged cache (declared
// in include/kvq.h): host-side argument checks, then asynchronous launches on
// the caller's stream. Nothing here allocates device memory or synchronises.
#include <cstdarg>
#include <cstdio>
#include <cstring>
#include <utility>

#include "kvq_paged.cuh"

namespace kvq {
void set_error_message(const char* msg);
}

using namespace kvq;

namespace {

kvq_status fail(kvq_status s, const char* fmt, ...) {
  char msg[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(msg, sizeof msg, fmt, ap);
  va_end(ap);
  set_error_message(msg);
  return s;
}

kvq_status cuda_status(cudaError_t e, const char* what) {
  if (e == cudaSuccess) {
    set_error_message("");
    return KVQ_OK;
  }
  return fail(KVQ_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

kvq_status ok() { return cuda_status(cudaSuccess, ""); }

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// SMs of the current device (0: none).
int current_sms() {
  static int cache[64] = {0};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
  if (cache[dev] == 0) {
    int n = 0;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
    cache[dev] = n;
  }
  return cache[dev];
}

// The format, sizes, strides and pointers of a cache; need: which pointers the call reads.
enum { kNeedKv = 1, kNeedBounds = 2, kHeadScales = 4 };  // kHeadScales: the call reads no scales per token

bool known_dtype(int dtype) {
  return dtype == KVQ_DT_BF16 || dtype == KVQ_DT_FP16 || dtype == KVQ_DT_E4M3 || dtype == KVQ_DT_E4M3_TOKEN;
}
bool is_e4m3(int dtype) { return dtype == KVQ_DT_E4M3 || dtype == KVQ_DT_E4M3_TOKEN; }
// The type that the kernels see: where the scales lie is in the View.
int kernel_dtype(int dtype) { return is_e4m3(dtype) ? KVQ_DT_E4M3 : dtype; }

kvq_status check_cache(const kvq_paged_cache* c, int need, paged::View* v) {
  if (c == nullptr) return fail(KVQ_ERR_BAD_ARG, "cache is NULL");
  if (c->version != KVQ_FORMAT_VERSION) return fail(KVQ_ERR_UNSUPPORTED, "cache: format version %u", c->version);
  if (!known_dtype(c->dtype)) return fail(KVQ_ERR_BAD_ARG, "cache: dtype %d", c->dtype);
  if (c->head_dim != kD) return fail(KVQ_ERR_UNSUPPORTED, "cache: head_dim %d (kernels support 128)", c->head_dim);
  if (c->n_pages < 1 || c->n_heads < 1 || c->n_heads > 1024 || c->page_size < 1 || c->page_size > KVQ_PAGED_MAX_PAGE)
    return fail(KVQ_ERR_BAD_ARG, "cache: n_pages %d page_size %d n_heads %d", c->n_pages, c->page_size, c->n_heads);
  const int es = is_e4m3(c->dtype) ? 1 : 2;
  if (c->dtype == KVQ_DT_E4M3_TOKEN) {
    if (need & kHeadScales)
      return fail(KVQ_ERR_UNSUPPORTED, "cache: one with a scale per token is attended to by kvq_paged_tree_attn");
    if (c->k_scale == nullptr || c->v_scale == nullptr)
      return fail(KVQ_ERR_BAD_ARG, "cache: scales per token without k_scale or v_scale");
    if (c->key_bounds != nullptr) return fail(KVQ_ERR_BAD_ARG, "cache: key_bounds beside scales per token");
  }
  if (need & kNeedKv) {
    if (c->k == nullptr || c->v == nullptr) return fail(KVQ_ERR_BAD_ARG, "cache: k or v is NULL");
    if (!aligned16(c->k) || !aligned16(c->v)) return fail(KVQ_ERR_MISALIGNED, "cache: k and v must be 16-byte aligned");
    // strides of 16-byte steps whose places do not overlap: each dimension, from the smallest stride up, steps over
    // all that the smaller ones span
    std::pair<int64_t, int64_t> dim[3] = {
        {c->page_stride, c->n_pages}, {c->token_stride, c->page_size}, {c->head_stride, c->n_heads}};
    int64_t span = kD;
    for (int i = 0; i < 3; ++i)
      for (int j = i + 1; j < 3; ++j)
        if (dim[j].first < dim[i].first) std::swap(dim[i], dim[j]);
    for (const auto& d : dim) {
      if (d.second == 1) continue;
      if (d.first < span || d.first > (int64_t(1) << 46) / d.second)
        return fail(KVQ_ERR_BAD_ARG, "cache: strides page %lld token %lld head %lld overlap or are out of range",
                    (long long)c->page_stride, (long long)c->token_stride, (long long)c->head_stride);
      if (d.first * es % 16 != 0) return fail(KVQ_ERR_MISALIGNED, "cache: strides must be multiples of 16 bytes");
      span += d.first * (d.second - 1);
    }
  }
  if (need & kNeedBounds) {
    if (c->key_bounds == nullptr) return fail(KVQ_ERR_BAD_ARG, "cache: key_bounds is NULL");
  }
  if (c->key_bounds != nullptr && !aligned16(c->key_bounds))
    return fail(KVQ_ERR_MISALIGNED, "cache: key_bounds must be 16-byte aligned");
  if (!is_e4m3(c->dtype) && (c->k_scale != nullptr || c->v_scale != nullptr))
    return fail(KVQ_ERR_BAD_ARG, "cache: scales belong to an E4M3 cache");
  memset(v, 0, sizeof *v);
  v->k = static_cast<char*>(c->k);
  v->v = static_cast<char*>(c->v);
  v->bounds = static_cast<char*>(c->key_bounds);
  v->k_scale = c->k_scale;
  v->v_scale = c->v_scale;
  v->err = c->error;
  v->page_stride = c->n_pages > 1 ? c->page_stride * es : 0;
  v->token_stride = c->page_size > 1 ? c->token_stride * es : 0;
  v->head_stride = c->n_heads > 1 ? c->head_stride * es : 0;
  v->n_pages = c->n_pages;
  v->H = c->n_heads;
  v->ps = paged::fast_div(c->page_size);
  v->token_scales = c->dtype == KVQ_DT_E4M3_TOKEN;
  return KVQ_OK;
}

// Token, page and list positions are 32-bit numbers in the kernels, which step beyond the last one by a block's stride
// (32768 at most).
constexpr long long kMostTokens = 0x7FFFFFFFLL - 0xFFFF;
constexpr int kMostSelected = 1 << 30;

bool batch_fits(long long n_requests, int n_heads, long long max_pages) {
  return n_requests * n_heads * KVQ_PAGED_MAX_G <= 0x7FFFFFFFLL && max_pages <= kMostTokens;
}

kvq_status check_batch(const kvq_paged_cache* c, const int32_t* page_table, int max_pages, int n_requests) {
  if (n_requests < 0 || max_pages < 0) return fail(KVQ_ERR_BAD_ARG, "n_requests %d max_pages %d", n_requests, max_pages);
  if ((long long)max_pages * c->page_size > kMostTokens)
    return fail(KVQ_ERR_BAD_ARG, "max_pages %d of %d tokens: beyond 2^31 tokens", max_pages, c->page_size);
  if (!batch_fits(n_requests, c->n_heads, max_pages))
    return fail(KVQ_ERR_BAD_ARG, "n_requests %d x n_heads %d", n_requests, c->n_heads);
  if (n_requests > 0 && max_pages > 0 && page_table == nullptr) return fail(KVQ_ERR_BAD_ARG, "page_table is NULL");
  return KVQ_OK;
}

// Query heads, type, pointer and stride of a decode query.
kvq_status check_query(const kvq_paged_cache* c, int n_requests, const int32_t* seq_lens, const void* q, int q_dtype,
                       int64_t q_stride, int n_q_heads) {
  if (n_q_heads < c->n_heads || n_q_heads % c->n_heads != 0)
    return fail(KVQ_ERR_BAD_ARG, "n_q_heads %d is not a multiple of n_heads %d", n_q_heads, c->n_heads);
  if (n_q_heads / c->n_heads > KVQ_PAGED_MAX_G)
    return fail(KVQ_ERR_UNSUPPORTED, "%d query heads per KV head (at most %d)", n_q_heads / c->n_heads, KVQ_PAGED_MAX_G);
  if (q_dtype != KVQ_DT_BF16 && q_dtype != KVQ_DT_FP16) return fail(KVQ_ERR_BAD_ARG, "q_dtype %d", q_dtype);
  if (!is_e4m3(c->dtype) && q_dtype != c->dtype)
    return fail(KVQ_ERR_UNSUPPORTED, "q_dtype %d on a cache of dtype %d", q_dtype, c->dtype);
  if (n_requests > 0 && (q == nullptr || seq_lens == nullptr)) return fail(KVQ_ERR_BAD_ARG, "q or seq_lens is NULL");
  if (!aligned16(q) || q_stride % 8 != 0) return fail(KVQ_ERR_MISALIGNED, "q must be 16-byte aligned, q_stride a multiple of 8");
  if (n_requests > 1 && (q_stride < 0 || q_stride > (int64_t(1) << 40)))
    return fail(KVQ_ERR_BAD_ARG, "q_stride %lld", (long long)q_stride);
  return KVQ_OK;
}

// Rows of a ragged batch, `stride` elements apart: as far as memory could reach.
bool rows_fit(int n_rows, int64_t stride) {
  return stride >= 0 && (n_rows < 2 || stride <= (int64_t(1) << 46) / n_rows);
}
kvq_status check_rows(int n_requests, const int32_t* offsets, int n_rows) {
  if (n_rows < 0 || (offsets == nullptr && n_rows != n_requests))
    return fail(KVQ_ERR_BAD_ARG, "n_rows %d for n_requests %d%s", n_rows, n_requests, offsets ? "" : " without offsets");
  return KVQ_OK;
}

// need: what this call uses of it, no more.
kvq_status check_workspace(void* workspace, size_t bytes, size_t need) {
  if (need > 0 && (workspace == nullptr || bytes < need))
    return fail(KVQ_ERR_WORKSPACE, "workspace of %zu bytes, %zu needed", workspace ? bytes : size_t(0), need);
  if (!aligned16(workspace)) return fail(KVQ_ERR_MISALIGNED, "workspace must be 16-byte aligned");
  return KVQ_OK;
}

// kvq_paged_decode_attn (sel NULL) and kvq_paged_sparse_attn.
kvq_status attend(const kvq_paged_cache* cache, const int32_t* page_table, int max_pages, int n_requests,
                  const int32_t* seq_lens, const void* q, int q_dtype, int64_t q_stride, int n_q_heads,
                  const int32_t* sel, int n_select, float softmax_scale, float* out, float* lse, void* workspace,
                  size_t workspace_bytes, kvq_cuda_stream stream) {
  paged::AttnArgs a;
  memset(&a, 0, sizeof a);
  kvq_status st = check_cache(cache, kNeedKv | kHeadScales, &a.c);
  if (st == KVQ_OK) st = check_batch(cache, page_table, max_pages, n_requests);
  if (st == KVQ_OK) st = check_query(cache, n_requests, seq_lens, q, q_dtype, q_stride, n_q_heads);
  if (st != KVQ_OK) return st;
  if (!(softmax_scale > 0.0f) || softmax_scale > 1e30f) return fail(KVQ_ERR_BAD_ARG, "softmax_scale");
  if (n_requests == 0) return ok();
  if (out == nullptr) return fail(KVQ_ERR_BAD_ARG, "out is NULL");
  if (!aligned16(out)) return fail(KVQ_ERR_MISALIGNED, "out must be 16-byte aligned");
  a.sms = current_sms();
  if (a.sms == 0) return fail(KVQ_ERR_CUDA, "no usable CUDA device");
  st = check_workspace(workspace, workspace_bytes, paged::attn_workspace(n_requests, cache->n_heads, n_q_heads, a.sms));
  if (st != KVQ_OK) return st;
  a.table = page_table;
  a.max_pages = max_pages;
  a.B = n_requests;
  a.lens = seq_lens;
  a.q = static_cast<const char*>(q);
  a.q_stride = n_requests > 1 ? q_stride * 2 : 0;
  a.q_dtype = q_dtype;
  a.dtype = cache->dtype;
  a.Hq = n_q_heads;
  a.g = n_q_heads / cache->n_heads;
  a.sel = sel;
  a.n_select = n_select;
  a.scale = softmax_scale;
  a.out = out;
  a.lse = lse;
  a.ws = static_cast<char*>(workspace);
  return cuda_status(paged::launch_attn(a, reinterpret_cast<cudaStream_t>(stream)), "paged attention launch");
}

}  // namespace

extern "C" {

kvq_status kvq_paged_cache_init(kvq_paged_cache* c, int dtype, int n_pages, int page_size, int n_heads, int head_dim) {
  if (c == nullptr) return fail(KVQ_ERR_BAD_ARG, "cache is NULL");
  memset(c, 0, sizeof *c);
  c->version = KVQ_FORMAT_VERSION;
  c->dtype = dtype;
  c->n_pages = n_pages;
  c->page_size = page_size;
  c->n_heads = n_heads;
  c->head_dim = head_dim;
  if (!known_dtype(dtype)) return fail(KVQ_ERR_BAD_ARG, "dtype %d", dtype);
  if (n_pages < 1 || page_size < 1 || page_size > KVQ_PAGED_MAX_PAGE || n_heads < 1 || n_heads > 1024 || head_dim < 1)
    return fail(KVQ_ERR_BAD_ARG, "sizes n_pages %d page_size %d n_heads %d head_dim %d", n_pages, page_size, n_heads,
                head_dim);
  c->head_stride = head_dim;
  c->token_stride = int64_t(n_heads) * head_dim;
  c->page_stride = c->token_stride * page_size;
  return ok();
}

kvq_status kvq_paged_append(const kvq_paged_cache* cache, const int32_t* page_table, int max_pages, int n_requests,
                            const kvq_paged_rows* r, kvq_cuda_stream stream) {
  paged::View view;
  kvq_status st = check_cache(cache, kNeedKv, &view);
  if (st == KVQ_OK) st = check_batch(cache, page_table, max_pages, n_requests);
  if (st != KVQ_OK) return st;
  if (r == nullptr) return fail(KVQ_ERR_BAD_ARG, "rows is NULL");
  if (r->n_rows < 0 || (r->offsets == nullptr && r->n_rows != n_requests))
    return fail(KVQ_ERR_BAD_ARG, "n_rows %d for n_requests %d%s", r->n_rows, n_requests, r->offsets ? "" : " without offsets");
  if (r->dtype != KVQ_DT_BF16 && r->dtype != KVQ_DT_FP16) return fail(KVQ_ERR_BAD_ARG, "rows: dtype %d", r->dtype);
  if (!is_e4m3(cache->dtype) && r->dtype != cache->dtype)
    return fail(KVQ_ERR_UNSUPPORTED, "rows of dtype %d into a cache of dtype %d", r->dtype, cache->dtype);
  if (r->rotary_dim < 0 || r->rotary_dim > kD || r->rotary_dim % 8 != 0)
    return fail(KVQ_ERR_BAD_ARG, "rotary_dim %d", r->rotary_dim);
  if (r->rotary_dim > 0 && (r->rope == nullptr || r->rope_positions < 1))
    return fail(KVQ_ERR_BAD_ARG, "rotary_dim %d without a rotation table", r->rotary_dim);
  if (r->rotary_dim > 0 && !aligned16(r->rope)) return fail(KVQ_ERR_MISALIGNED, "rope must be 16-byte aligned");
  const bool has_q = r->q != nullptr;
  if (has_q) {
    if (r->q_out == nullptr) return fail(KVQ_ERR_BAD_ARG, "q without q_out");
    if (r->n_q_heads < cache->n_heads || r->n_q_heads % cache->n_heads != 0)
      return fail(KVQ_ERR_BAD_ARG, "n_q_heads %d is not a multiple of n_heads %d", r->n_q_heads, cache->n_heads);
    if (r->n_q_heads / cache->n_heads > KVQ_PAGED_MAX_G)
      return fail(KVQ_ERR_UNSUPPORTED, "%d query heads per KV head (at most %d)", r->n_q_heads / cache->n_heads,
                  KVQ_PAGED_MAX_G);
  }
  if (n_requests == 0 || r->n_rows == 0) return ok();
  if (r->start == nullptr || r->k == nullptr || r->v == nullptr) return fail(KVQ_ERR_BAD_ARG, "start, k or v is NULL");
  const void* ptrs[4] = {r->k, r->v, has_q ? r->q : nullptr, has_q ? r->q_out : nullptr};
  const int64_t strides[4] = {r->k_stride, r->v_stride, has_q ? r->q_stride : 0, has_q ? r->q_out_stride : 0};
  for (int i = 0; i < 4; ++i) {
    if (!aligned16(ptrs[i]) || strides[i] % 8 != 0)
      return fail(KVQ_ERR_MISALIGNED, "k, v, q and q_out must be 16-byte aligned, their strides multiples of 8");
    if (strides[i] < 0 || strides[i] > (int64_t(1) << 40)) return fail(KVQ_ERR_BAD_ARG, "row stride %lld", (long long)strides[i]);
  }
  if (has_q && r->n_rows > 1 && r->q_out_stride < int64_t(r->n_q_heads) * kD)
    return fail(KVQ_ERR_BAD_ARG, "q_out_stride %lld: rows overlap", (long long)r->q_out_stride);
  const int sms = current_sms();
  if (sms == 0) return fail(KVQ_ERR_CUDA, "no usable CUDA device");
  const paged::AppendArgs a = paged::append_args(view, kernel_dtype(cache->dtype), page_table, max_pages, n_requests, *r);
  return cuda_status(paged::launch_append(a, sms, reinterpret_cast<cudaStream_t>(stream)), "paged append launch");
}

size_t kvq_paged_workspace_bytes(int n_requests, int n_heads, int n_q_heads, int max_pages) {
  const int sms = current_sms();
  if (n_requests < 0 || n_heads < 1 || n_heads > 1024 || n_q_heads < n_heads || n_q_heads % n_heads != 0 ||
      n_q_heads / n_heads > KVQ_PAGED_MAX_G || max_pages < 0 || !batch_fits(n_requests, n_heads, max_pages) || sms == 0)
    return 0;
  const size_t a = paged::attn_workspace(n_requests, n_heads, n_q_heads, sms);
  const size_t b = paged::select_workspace(n_requests, n_heads, max_pages);
  return a > b ? a : b;
}

kvq_status kvq_paged_decode_attn(const kvq_paged_cache* cache, const int32_t* page_table, int max_pages,
                                 int n_requests, const int32_t* seq_lens, const void* q, int q_dtype,
                                 int64_t q_stride, int n_q_heads, float softmax_scale, float* out, float* lse,
                                 void* workspace, size_t workspace_bytes, kvq_cuda_stream stream) {
  return attend(cache, page_table, max_pages, n_requests, seq_lens, q, q_dtype, q_stride, n_q_heads, nullptr, 0,
                softmax_scale, out, lse, workspace, workspace_bytes, stream);
}

kvq_status kvq_paged_sparse_attn(const kvq_paged_cache* cache, const int32_t* page_table, int max_pages,
                                 int n_requests, const int32_t* seq_lens, const void* q, int q_dtype,
                                 int64_t q_stride, int n_q_heads, const int32_t* sel, int n_select,
                                 float softmax_scale, float* out, float* lse, void* workspace,
                                 size_t workspace_bytes, kvq_cuda_stream stream) {
  if (n_select < 1 || n_select > kMostSelected) return fail(KVQ_ERR_BAD_ARG, "n_select %d", n_select);
  if (sel == nullptr && n_requests > 0) return fail(KVQ_ERR_BAD_ARG, "sel is NULL");
  return attend(cache, page_table, max_pages, n_requests, seq_lens, q, q_dtype, q_stride, n_q_heads, sel, n_select,
                softmax_scale, out, lse, workspace, workspace_bytes, stream);
}

kvq_status kvq_paged_select(const kvq_paged_cache* cache, const int32_t* page_table, int max_pages, int n_requests,
                            const int32_t* seq_lens, const void* q, int q_dtype, int64_t q_stride, int n_q_heads,
                            int n_select, int n_first, int n_last, int32_t* sel, void* workspace,
                            size_t workspace_bytes, kvq_cuda_stream stream) {
  paged::SelectArgs a;
  memset(&a, 0, sizeof a);
  kvq_status st = check_cache(cache, kNeedBounds | kHeadScales, &a.c);
  if (st == KVQ_OK) st = check_batch(cache, page_table, max_pages, n_requests);
  if (st == KVQ_OK) st = check_query(cache, n_requests, seq_lens, q, q_dtype, q_stride, n_q_heads);
  if (st != KVQ_OK) return st;
  if (n_select < 1 || n_select > kMostSelected || n_first < 0 || n_last < 0 || (long long)n_first + n_last > n_select)
    return fail(KVQ_ERR_BAD_ARG, "n_select %d n_first %d n_last %d", n_select, n_first, n_last);
  if (n_requests == 0) return ok();
  if (sel == nullptr) return fail(KVQ_ERR_BAD_ARG, "sel is NULL");
  a.sms = current_sms();
  if (a.sms == 0) return fail(KVQ_ERR_CUDA, "no usable CUDA device");
  st = check_workspace(workspace, workspace_bytes, paged::select_workspace(n_requests, cache->n_heads, max_pages));
  if (st != KVQ_OK) return st;
  a.table = page_table;
  a.max_pages = max_pages;
  a.B = n_requests;
  a.lens = seq_lens;
  a.q = static_cast<const char*>(q);
  a.q_stride = n_requests > 1 ? q_stride * 2 : 0;
  a.q_dtype = q_dtype;
  a.dtype = cache->dtype;
  a.g = n_q_heads / cache->n_heads;
  a.n_select = n_select;
  a.n_first = n_first;
  a.n_last = n_last;
  a.sel = sel;
  a.ws = static_cast<char*>(workspace);
  return cuda_status(paged::launch_select(a, reinterpret_cast<cudaStream_t>(stream)), "page selection launch");
}

kvq_status kvq_paged_read(const kvq_paged_cache* cache, const int32_t* page_table, int max_pages, int n_requests,
                          const int32_t* start, const int32_t* offsets, int n_rows, int out_dtype, void* k_out,
                          void* v_out, int64_t k_stride, int64_t v_stride, kvq_cuda_stream stream) {
  paged::ReadArgs a;
  memset(&a, 0, sizeof a);
  kvq_status st = check_cache(cache, kNeedKv, &a.c);
  if (st == KVQ_OK) st = check_batch(cache, page_table, max_pages, n_requests);
  if (st == KVQ_OK) st = check_rows(n_requests, offsets, n_rows);
  if (st != KVQ_OK) return st;
  if (out_dtype != KVQ_DT_BF16 && out_dtype != KVQ_DT_FP16) return fail(KVQ_ERR_BAD_ARG, "out_dtype %d", out_dtype);
  if (n_requests == 0 || n_rows == 0) return ok();
  if (start == nullptr || k_out == nullptr || v_out == nullptr) return fail(KVQ_ERR_BAD_ARG, "start, k_out or v_out is NULL");
  if (!aligned16(k_out) || !aligned16(v_out) || k_stride % 8 != 0 || v_stride % 8 != 0)
    return fail(KVQ_ERR_MISALIGNED, "k_out and v_out must be 16-byte aligned, their strides multiples of 8");
  const int64_t row = int64_t(cache->n_heads) * kD;
  for (const int64_t s : {k_stride, v_stride})
    if (!rows_fit(n_rows, s) || (n_rows > 1 && s < row))
      return fail(KVQ_ERR_BAD_ARG, "row stride %lld: rows overlap or are out of range", (long long)s);
  const int sms = current_sms();
  if (sms == 0) return fail(KVQ_ERR_CUDA, "no usable CUDA device");
  a.table = page_table;
  a.max_pages = max_pages;
  a.B = n_requests;
  a.start = start;
  a.offsets = offsets;
  a.n_rows = n_rows;
  a.dtype = kernel_dtype(cache->dtype);
  a.out_dtype = out_dtype;
  a.k = static_cast<char*>(k_out);
  a.v = static_cast<char*>(v_out);
  a.k_stride = k_stride * 2;
  a.v_stride = v_stride * 2;
  return cuda_status(paged::launch_read(a, sms, reinterpret_cast<cudaStream_t>(stream)), "paged read launch");
}

size_t kvq_paged_tree_workspace_bytes(int n_requests, int n_heads, int n_q_heads, int n_rows) {
  const int sms = current_sms();
  if (n_requests < 0 || n_heads < 1 || n_heads > 1024 || n_q_heads < n_heads || n_q_heads % n_heads != 0 ||
      n_q_heads / n_heads > KVQ_PAGED_MAX_G || n_rows < 0 || !batch_fits(n_requests, n_heads, 0) || sms == 0)
    return 0;
  return paged::tree_workspace_up_to(n_requests, n_heads, n_q_heads, n_rows, sms);
}

kvq_status kvq_paged_tree_attn(const kvq_paged_cache* cache, const int32_t* page_table, int max_pages, int n_requests,
                               const int32_t* seq_lens, const int32_t* offsets, int n_rows, const uint32_t* mask,
                               int mask_words, const void* q, int q_dtype, int64_t q_stride, int n_q_heads,
                               float softmax_scale, void* out, float* lse, void* workspace, size_t workspace_bytes,
                               kvq_cuda_stream stream) {
  paged::TreeArgs a;
  memset(&a, 0, sizeof a);
  kvq_status st = check_cache(cache, kNeedKv, &a.c);
  if (st == KVQ_OK) st = check_batch(cache, page_table, max_pages, n_requests);
  if (st == KVQ_OK) st = check_rows(n_requests, offsets, n_rows);
  if (st == KVQ_OK) st = check_query(cache, n_requests > 0 && n_rows > 0 ? (n_rows > 1 ? 2 : 1) : 0, seq_lens, q, q_dtype, q_stride, n_q_heads);
  if (st != KVQ_OK) return st;
  if (!(softmax_scale > 0.0f) || softmax_scale > 1e30f) return fail(KVQ_ERR_BAD_ARG, "softmax_scale");
  if (!rows_fit(n_rows, q_stride)) return fail(KVQ_ERR_BAD_ARG, "q_stride %lld", (long long)q_stride);
  // (a mask of no rows has no address)
  if (mask_words < 0 || mask_words > KVQ_PAGED_MAX_DRAFT / 32 ||
      (mask == nullptr ? mask_words > 0 && n_rows > 0 : mask_words == 0))
    return fail(KVQ_ERR_BAD_ARG, "mask %s mask_words %d", mask == nullptr ? "NULL" : "of", mask_words);
  if (n_requests == 0 || n_rows == 0) return ok();
  if (out == nullptr) return fail(KVQ_ERR_BAD_ARG, "out is NULL");
  if (!aligned16(out)) return fail(KVQ_ERR_MISALIGNED, "out must be 16-byte aligned");
  a.sms = current_sms();
  if (a.sms == 0) return fail(KVQ_ERR_CUDA, "no usable CUDA device");
  st = check_workspace(workspace, workspace_bytes,
                       paged::tree_workspace(n_requests, cache->n_heads, n_q_heads, n_rows, a.sms));
  if (st != KVQ_OK) return st;
  a.table = page_table;
  a.max_pages = max_pages;
  a.B = n_requests;
  a.lens = seq_lens;
  a.offsets = offsets;
  a.n_rows = n_rows;
  a.mask = mask;
  a.mask_words = mask_words;
  a.g = n_q_heads / cache->n_heads;
  a.Hq = n_q_heads;
  a.q = static_cast<const char*>(q);
  a.q_stride = q_stride * 2;
  a.q_dtype = q_dtype;
  a.dtype = kernel_dtype(cache->dtype);
  a.scale = softmax_scale;
  a.out = static_cast<char*>(out);
  a.lse = lse;
  a.ws = static_cast<char*>(workspace);
  return cuda_status(paged::launch_tree(a, reinterpret_cast<cudaStream_t>(stream)), "tree attention launch");
}

kvq_status kvq_paged_tree_commit(const kvq_paged_cache* cache, const int32_t* page_table, int max_pages,
                                 int n_requests, const int32_t* seq_lens, const int32_t* accepted,
                                 const int32_t* offsets, int n_accepted, kvq_cuda_stream stream) {
  paged::CommitArgs a;
  memset(&a, 0, sizeof a);
  kvq_status st = check_cache(cache, kNeedKv, &a.c);
  if (st == KVQ_OK) st = check_batch(cache, page_table, max_pages, n_requests);
  if (st != KVQ_OK) return st;
  if (n_accepted < 0) return fail(KVQ_ERR_BAD_ARG, "n_accepted %d", n_accepted);
  if (n_requests == 0) return ok();
  if (seq_lens == nullptr || offsets == nullptr || (n_accepted > 0 && accepted == nullptr))
    return fail(KVQ_ERR_BAD_ARG, "seq_lens, offsets or accepted is NULL");
  if (current_sms() == 0) return fail(KVQ_ERR_CUDA, "no usable CUDA device");
  a.table = page_table;
  a.max_pages = max_pages;
  a.B = n_requests;
  a.lens = seq_lens;
  a.accepted = accepted;
  a.offsets = offsets;
  a.n_accepted = n_accepted;
  a.dtype = kernel_dtype(cache->dtype);
  return cuda_status(paged::launch_commit(a, reinterpret_cast<cudaStream_t>(stream)), "paged commit launch");
}

}  // extern "C"
