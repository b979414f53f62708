// kvq_paged.cuh — shared by the kernels of the paged cache (kvq_paged_*): the
// cache as the kernels see it, element conversions, division by the page size,
// and the split of a ragged batch into equal ranges of work.
#pragma once

#include <cuda_fp8.h>

#include "kvq_internal.cuh"

namespace kvq {
namespace paged {

constexpr int kBf16 = KVQ_DT_BF16, kFp16 = KVQ_DT_FP16, kE4m3 = KVQ_DT_E4M3;
constexpr int kMaxGroup = KVQ_PAGED_MAX_G;

// n / d for 0 <= n < 2^31 and 1 <= d <= 1024: with l = ceil(log2 d) and mul =
// floor(2^32 (2^l - d) / d) + 1, floor(n / d) = (umulhi(mul, n) + n) >> l
// (Granlund and Montgomery, "Division by invariant integers using
// multiplication", 1994); the sum stays below 2^32 because n < 2^31.
struct FastDiv {
  uint32_t d, mul, shift;
  __device__ __forceinline__ int div(int n) const { return int((__umulhi(mul, uint32_t(n)) + uint32_t(n)) >> shift); }
};
inline FastDiv fast_div(int d) {
  FastDiv f;
  f.d = uint32_t(d);
  f.shift = 0;
  while ((1u << f.shift) < f.d) ++f.shift;
  f.mul = uint32_t(((uint64_t(1) << 32) * ((uint64_t(1) << f.shift) - f.d)) / f.d + 1);
  return f;
}

// The cache with strides in bytes (the stride of a dimension of one entry is 0).
struct View {
  FastDiv ps;
  int32_t H;
  int32_t n_pages;
  int32_t* err;
  char* k;
  char* v;
  long long page_stride, token_stride, head_stride;
  const float* k_scale;
  const float* v_scale;
  char* bounds;  // [n_pages][H][2][128] elements, or nullptr
  // 1: E4M3 whose scales are [n_pages][H][page_size] (KVQ_DT_E4M3_TOKEN; the dtype that goes with a View is then kE4m3)
  int32_t token_scales;
};

__device__ __forceinline__ void flag(const View& c, int bits) {
  if (c.err != nullptr) atomicOr(c.err, bits);
}

template <int DT>
__host__ __device__ constexpr int elem_bytes() {
  return DT == kE4m3 ? 1 : 2;
}

// Four consecutive elements as FP32 (exact) and back (one rounding each; E4M3
// saturates at 448 and keeps NaN).
template <int DT>
__device__ __forceinline__ float4 load4(const void* p) {
  if constexpr (DT == kE4m3) {
    const uint32_t w = *reinterpret_cast<const uint32_t*>(p);
    const uint32_t a = e4m3x2_to_f16x2(w & 0xFFFFu), b = e4m3x2_to_f16x2(w >> 16);
    const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&a));
    const float2 y = __half22float2(*reinterpret_cast<const __half2*>(&b));
    return make_float4(x.x, x.y, y.x, y.y);
  } else {
    const uint2 w = *reinterpret_cast<const uint2*>(p);
    if constexpr (DT == kBf16)
      return make_float4(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xFFFF0000u), __uint_as_float(w.y << 16),
                         __uint_as_float(w.y & 0xFFFF0000u));
    const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&w.x));
    const float2 y = __half22float2(*reinterpret_cast<const __half2*>(&w.y));
    return make_float4(x.x, x.y, y.x, y.y);
  }
}

template <int DT>
__device__ __forceinline__ void store4(void* p, float4 x) {
  if constexpr (DT == kE4m3) {
    const uint32_t a = __nv_cvt_float2_to_fp8x2(make_float2(x.x, x.y), __NV_SATFINITE, __NV_E4M3);
    const uint32_t b = __nv_cvt_float2_to_fp8x2(make_float2(x.z, x.w), __NV_SATFINITE, __NV_E4M3);
    *reinterpret_cast<uint32_t*>(p) = a | (b << 16);
  } else if constexpr (DT == kBf16) {
    const __nv_bfloat162 a = __floats2bfloat162_rn(x.x, x.y), b = __floats2bfloat162_rn(x.z, x.w);
    *reinterpret_cast<uint2*>(p) =
        make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
  } else {
    const __half2 a = __floats2half2_rn(x.x, x.y), b = __floats2half2_rn(x.z, x.w);
    *reinterpret_cast<uint2*>(p) =
        make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
  }
}

// The element as it is read back after store4.
template <int DT>
__device__ __forceinline__ float4 rounded4(float4 x) {
  alignas(8) uint32_t w[2];
  store4<DT>(w, x);
  return load4<DT>(w);
}

__device__ __forceinline__ float4 times(float4 x, float s) {
  return make_float4(x.x * s, x.y * s, x.z * s, x.w * s);
}

// Tokens of request b, or -1 for a length that its table row cannot hold.
__device__ __forceinline__ int checked_len(const int32_t* lens, int b, int max_pages, const FastDiv& ps) {
  const int T = lens[b];
  return (T < 0 || (long long)T > (long long)max_pages * ps.d) ? -1 : T;
}

// Prefix sums of a count per request over the threads of a block (blockDim.x =
// NT): thread t sums the requests [t * per, (t + 1) * per). Every thread may then
// look up any position of the concatenated work.
template <int NT>
struct Prefix {
  long long pre[NT + 1];  // exclusive prefix by thread; pre[NT] is the total
  long long warp_sum[NT / 32];
};

template <int NT, typename F>
__device__ __forceinline__ void build_prefix(Prefix<NT>& S, int B, const F& count) {
  const int t = threadIdx.x, per = (B + NT - 1) / NT;
  const int b0 = min(B, t * per), b1 = min(B, b0 + per);
  long long n = 0;
  for (int b = b0; b < b1; ++b) n += count(b);
  long long x = n;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xFFFFFFFFu, x, o);
    if ((t & 31) >= o) x += y;
  }
  if ((t & 31) == 31) S.warp_sum[t >> 5] = x;
  __syncthreads();
  long long base = 0;
  for (int w = 0; w < (t >> 5); ++w) base += S.warp_sum[w];
  S.pre[t] = base + x - n;
  if (t == NT - 1) S.pre[NT] = base + x;
  __syncthreads();
}

// The request that holds work position `at` (0 <= at < total), and `at` within it.
template <int NT, typename F>
__device__ __forceinline__ int find_request(const Prefix<NT>& S, int B, const F& count, long long& at) {
  int lo = 0, hi = NT - 1;  // the last thread whose prefix is <= at (threads of no work before it share its value)
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (S.pre[mid] <= at) lo = mid;
    else hi = mid - 1;
  }
  const int per = (B + NT - 1) / NT;
  at -= S.pre[lo];
  int b = lo * per;
  for (long long n = count(b); b < B - 1 && at >= n; n = count(b)) {
    at -= n;
    ++b;
  }
  return b;
}

// Start of part c of `total` cut into n equal parts: floor(c total / n). By 32-bit
// arithmetic where that holds (64-bit divisions at the head of a kernel add up to a
// microsecond, a seventh of the shortest calls). c <= n <= 8192.
__device__ __forceinline__ long long part_start(int c, long long total, int n) {
  if (total < (1 << 19)) return uint32_t(c) * uint32_t(total) / uint32_t(n);
  return (long long)c * total / n;
}
// q = x / d and r = x % d, the same way.
__device__ __forceinline__ void divide(long long x, int d, int& q, int& r) {
  if (x <= 0x7FFFFFFF) {
    q = int(x) / d;
    r = int(x) - q * d;
  } else {
    q = int(x / d);
    r = int(x - (long long)q * d);
  }
}

// Rows of request b and the first of them, or -1 when its offsets are outside their range (no offsets: one row each).
__device__ __forceinline__ int row_range(const int32_t* offsets, int n_rows, int b, int& row0) {
  row0 = b;
  if (offsets == nullptr) return 1;
  row0 = offsets[b];
  const int row1 = offsets[b + 1];
  return row0 < 0 || row1 < row0 || row1 > n_rows ? -1 : row1 - row0;
}

// Smaller and larger ones of pairs of 16-bit numbers (BF16, or FP16, which E4M3 values
// become exactly); NaN stays.
template <int DT>
__device__ __forceinline__ uint32_t smaller(uint32_t x, uint32_t y) {
  if constexpr (DT == kBf16) {
    const __nv_bfloat162 r =
        __hmin2_nan(*reinterpret_cast<const __nv_bfloat162*>(&x), *reinterpret_cast<const __nv_bfloat162*>(&y));
    return *reinterpret_cast<const uint32_t*>(&r);
  } else {
    const __half2 r = __hmin2_nan(*reinterpret_cast<const __half2*>(&x), *reinterpret_cast<const __half2*>(&y));
    return *reinterpret_cast<const uint32_t*>(&r);
  }
}
template <int DT>
__device__ __forceinline__ uint32_t larger(uint32_t x, uint32_t y) {
  if constexpr (DT == kBf16) {
    const __nv_bfloat162 r =
        __hmax2_nan(*reinterpret_cast<const __nv_bfloat162*>(&x), *reinterpret_cast<const __nv_bfloat162*>(&y));
    return *reinterpret_cast<const uint32_t*>(&r);
  } else {
    const __half2 r = __hmax2_nan(*reinterpret_cast<const __half2*>(&x), *reinterpret_cast<const __half2*>(&y));
    return *reinterpret_cast<const uint32_t*>(&r);
  }
}

struct AppendArgs {
  View c;
  const int32_t* table;
  int32_t max_pages;
  int32_t B;
  const int32_t* start;
  const int32_t* offsets;
  int32_t n_rows;
  int32_t in_dtype;
  int32_t dtype;
  int32_t Hq;
  const char* k;
  const char* v;
  const char* q;
  char* q_out;
  long long k_stride, v_stride, q_stride, q_out_stride;  // bytes
  const float* rope;
  int32_t rope_positions;
  int32_t R;
  int32_t interleaved;
  const int32_t* positions;
};

// The arguments of an append from its checked descriptors. Positions choose rows of the
// rotation table: without one the kernels do not see them.
inline AppendArgs append_args(const View& c, int dtype, const int32_t* page_table, int max_pages, int n_requests,
                              const kvq_paged_rows& r) {
  AppendArgs a{};
  a.c = c;
  a.table = page_table;
  a.max_pages = max_pages;
  a.B = n_requests;
  a.start = r.start;
  a.offsets = r.offsets;
  a.n_rows = r.n_rows;
  a.in_dtype = r.dtype;
  a.dtype = dtype;
  a.Hq = r.n_q_heads;
  a.k = static_cast<const char*>(r.k);
  a.v = static_cast<const char*>(r.v);
  a.q = static_cast<const char*>(r.q);
  a.q_out = static_cast<char*>(r.q_out);
  a.k_stride = r.k_stride * 2;
  a.v_stride = r.v_stride * 2;
  a.q_stride = r.q_stride * 2;
  a.q_out_stride = r.q_out_stride * 2;
  a.rope = r.rope;
  a.rope_positions = r.rope_positions;
  a.R = r.rotary_dim;
  a.interleaved = r.interleaved != 0;
  a.positions = r.rotary_dim > 0 ? r.positions : nullptr;
  return a;
}

struct AttnArgs {
  const int32_t* lens;
  const int32_t* table;
  int32_t max_pages;
  int32_t B;
  int32_t lane_heads;  // KV heads of a lane of blocks (launch_attn)
  int32_t g;
  int32_t Hq;
  int32_t n_select;
  const int32_t* sel;  // [B][H][n_select], or nullptr: every page
  View c;
  const char* q;
  long long q_stride;  // bytes
  float scale;
  int32_t q_dtype;
  float* out;
  float* lse;
  char* ws;
  int32_t dtype;
  int32_t sms;
};

struct SelectArgs {
  View c;
  const int32_t* table;
  int32_t max_pages;
  int32_t B;
  const int32_t* lens;
  const char* q;
  long long q_stride;  // bytes
  int32_t q_dtype;
  int32_t dtype;
  int32_t g;
  int32_t n_select, n_first, n_last;
  int32_t* sel;
  char* ws;
  int32_t sms;
};

struct ReadArgs {
  View c;
  const int32_t* table;
  int32_t max_pages;
  int32_t B;
  const int32_t* start;
  const int32_t* offsets;
  int32_t n_rows;
  int32_t dtype;
  int32_t out_dtype;
  char* k;
  char* v;
  long long k_stride, v_stride;  // bytes
};

struct CommitArgs {
  View c;
  const int32_t* table;
  int32_t max_pages;
  int32_t B;
  const int32_t* lens;
  const int32_t* accepted;
  const int32_t* offsets;
  int32_t n_accepted;
  int32_t dtype;
};

struct TreeArgs {
  View c;
  const int32_t* table;
  int32_t max_pages;
  int32_t B;
  const int32_t* lens;
  const int32_t* offsets;
  int32_t n_rows;
  const uint32_t* mask;  // [n_rows][mask_words], or nullptr: row i sees the drafted tokens 0 .. i
  int32_t mask_words;
  int32_t g;
  int32_t Hq;
  const char* q;
  long long q_stride;  // bytes
  int32_t q_dtype;
  int32_t dtype;
  float scale;
  char* out;
  float* lse;
  char* ws;
  int32_t sms;
};

size_t tree_workspace(int B, int H, int Hq, int n_rows, int sms);        // of a call
size_t tree_workspace_up_to(int B, int H, int Hq, int n_rows, int sms);  // of any call of no more requests and rows
cudaError_t launch_read(const ReadArgs& a, int sms, cudaStream_t stream);
cudaError_t launch_commit(const CommitArgs& a, cudaStream_t stream);
cudaError_t launch_tree(const TreeArgs& a, cudaStream_t stream);

size_t attn_workspace(int B, int H, int Hq, int sms);
size_t select_workspace(int B, int H, int max_pages);
cudaError_t launch_append(const AppendArgs& a, int sms, cudaStream_t stream);
cudaError_t launch_attn(const AttnArgs& a, cudaStream_t stream);
cudaError_t launch_select(const SelectArgs& a, cudaStream_t stream);

}  // namespace paged
}  // namespace kvq
