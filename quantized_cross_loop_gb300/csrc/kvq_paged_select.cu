// kvq_paged_select.cu — the pages a query most likely finds something on.
//
// score(page) = sum_j sum_d (q_jd < 0 ? q_jd lo_d : q_jd hi_d), the sum over the
// group's query heads j of the largest q.k that the page's bounds allow. The sum
// over the heads goes into the query:
// score = sum_d up_d hi_d + down_d lo_d with up_d = sum_j max(q_jd, 0) and down_d
// = sum_j min(q_jd, 0): 256 products per page whatever the group is.
//
// The first kernel writes every page's score, in FP64, as an order-preserving key;
// the second finds the n-th largest by a radix selection and writes the pages in
// ascending order.
#include "kvq_paged.cuh"

namespace kvq {
namespace paged {
namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ uint64_t order_key(double x) {
  if (!isfinite(x)) return ~0ull - 1;  // before all finite ones; forced pages before those
  const uint64_t u = uint64_t(__double_as_longlong(x + 0.0));  // -0 counts as +0
  return (u >> 63) ? ~u : (u | (1ull << 63));
}

template <int DT, int QT>
__global__ void __launch_bounds__(kThreads) score_kernel(SelectArgs a, uint64_t* keys) {
  __shared__ double w[2][kD];  // down, up
  const int b = blockIdx.y / a.c.H, h = blockIdx.y % a.c.H;
  const int T = checked_len(a.lens, b, a.max_pages, a.c.ps);
  if (T < 0) {
    if (threadIdx.x == 0) flag(a.c, KVQ_PAGED_ERR_LENGTH);
    return;
  }
  const int pages = T == 0 ? 0 : a.c.ps.div(T - 1) + 1;
  if (pages <= a.n_select) return;
  if (threadIdx.x < 32) {
    double lo[4] = {0, 0, 0, 0}, hi[4] = {0, 0, 0, 0};
    for (int j = 0; j < a.g; ++j) {
      const float4 q = load4<QT>(a.q + (long long)b * a.q_stride + ((h * a.g + j) * kD + 4 * threadIdx.x) * 2);
      const float x[4] = {q.x, q.y, q.z, q.w};
      for (int e = 0; e < 4; ++e) {
        if (x[e] < 0.0f) lo[e] += x[e];
        else hi[e] += x[e];
      }
    }
    for (int e = 0; e < 4; ++e) {
      w[0][4 * threadIdx.x + e] = lo[e];
      w[1][4 * threadIdx.x + e] = hi[e];
    }
  }
  __syncthreads();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int p = blockIdx.x * 8 + warp; p < pages; p += gridDim.x * 8) {
    uint64_t key;
    const int page = a.table[(long long)b * a.max_pages + p];
    if (page < 0 || page >= a.c.n_pages) {
      if (lane == 0) flag(a.c, KVQ_PAGED_ERR_PAGE);
      key = 0;
    } else {
      const char* at = a.c.bounds + (((long long)page * a.c.H + h) * 2 * kD + 4 * lane) * elem_bytes<DT>();
      const float4 lo = load4<DT>(at), hi = load4<DT>(at + kD * elem_bytes<DT>());
      const double *wd = &w[0][4 * lane], *wu = &w[1][4 * lane];
      double x = wd[0] * lo.x + wd[1] * lo.y + wd[2] * lo.z + wd[3] * lo.w;
      x += wu[0] * hi.x + wu[1] * hi.y + wu[2] * hi.z + wu[3] * hi.w;
      for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xFFFFFFFFu, x, o);
      key = order_key(x);
    }
    if (p < a.n_first || p >= pages - a.n_last) key = ~0ull;
    if (lane == 0) keys[(long long)blockIdx.y * a.max_pages + p] = key;
  }
}

__global__ void __launch_bounds__(kThreads) pick_kernel(SelectArgs a, const uint64_t* all) {
  __shared__ int hist[256];
  __shared__ uint64_t s_prefix;
  __shared__ int s_left;
  __shared__ int s_sum[2][8];
  const int b = blockIdx.x / a.c.H;
  const int T = checked_len(a.lens, b, a.max_pages, a.c.ps);
  const int pages = T <= 0 ? 0 : a.c.ps.div(T - 1) + 1;
  int32_t* sel = a.sel + (long long)blockIdx.x * a.n_select;
  if (pages <= a.n_select) {
    for (int i = threadIdx.x; i < a.n_select; i += kThreads) sel[i] = i < pages ? i : -1;
    return;
  }
  const uint64_t* keys = all + (long long)blockIdx.x * a.max_pages;
  uint64_t prefix = 0, mask = 0;
  int left = a.n_select;  // still to take among the keys that match the prefix
  for (int shift = 56; shift >= 0; shift -= 8) {
    hist[threadIdx.x] = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < pages; i += kThreads) {
      const uint64_t k = keys[i];
      if ((k & mask) == prefix) atomicAdd(&hist[(k >> shift) & 255], 1);
    }
    __syncthreads();
    if (threadIdx.x == 0) {
      int bin = 255, n = left;
      while (bin > 0 && hist[bin] < n) n -= hist[bin--];
      s_prefix = prefix | (uint64_t(bin) << shift);
      s_left = n;
    }
    __syncthreads();
    prefix = s_prefix;
    left = s_left;
    mask |= 255ull << shift;
    __syncthreads();
  }
  // every key above `prefix`, and the first `left` of those equal to it
  int out = 0, eq = 0;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int i0 = 0; i0 < pages; i0 += kThreads) {
    const int i = i0 + threadIdx.x;
    const uint64_t k = i < pages ? keys[i] : 0;
    const bool same = i < pages && k == prefix, above = i < pages && k > prefix;
    const uint32_t ms = __ballot_sync(0xFFFFFFFFu, same), below = (1u << lane) - 1u;
    if (lane == 0) s_sum[0][warp] = __popc(ms);
    __syncthreads();
    int rank = eq + __popc(ms & below);
    for (int w = 0; w < 8; ++w) {
      if (w < warp) rank += s_sum[0][w];
      eq += s_sum[0][w];
    }
    const bool take = above || (same && rank < left);
    const uint32_t mt = __ballot_sync(0xFFFFFFFFu, take);
    if (lane == 0) s_sum[1][warp] = __popc(mt);
    __syncthreads();
    int at = out + __popc(mt & below);
    for (int w = 0; w < 8; ++w) {
      if (w < warp) at += s_sum[1][w];
      out += s_sum[1][w];
    }
    if (take && at < a.n_select) sel[at] = i;
    __syncthreads();
  }
}

}  // namespace

size_t select_workspace(int B, int H, int max_pages) { return 16 + size_t(B) * H * max_pages * 8; }

cudaError_t launch_select(const SelectArgs& a, cudaStream_t stream) {
  uint64_t* keys = reinterpret_cast<uint64_t*>(a.ws + 16);
  const int units = a.B * a.c.H;
  const int chunks = (a.max_pages + 63) / 64 + (a.max_pages == 0);
  const dim3 grid(chunks < 1024 ? chunks : 1024, units);
  const bool bf = a.q_dtype == kBf16;
  if (a.dtype == kBf16) score_kernel<kBf16, kBf16><<<grid, kThreads, 0, stream>>>(a, keys);
  else if (a.dtype == kFp16) score_kernel<kFp16, kFp16><<<grid, kThreads, 0, stream>>>(a, keys);
  else if (bf) score_kernel<kE4m3, kBf16><<<grid, kThreads, 0, stream>>>(a, keys);
  else score_kernel<kE4m3, kFp16><<<grid, kThreads, 0, stream>>>(a, keys);
  count_launch();
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  pick_kernel<<<units, kThreads, 0, stream>>>(a, keys);
  count_launch();
  return cudaGetLastError();
}

}  // namespace paged
}  // namespace kvq
