// kvq_paged_tree.cu — attention of several queries per request (a tree of drafted
// tokens, a chunk of a prompt, a decode step) over a paged cache.
//
// s_t = scale q.k_t over the cached tokens and the drafted ones that a row's mask
// allows, out = sum_t e^(s_t - m) v_t / l, lse = m + ln l, in one pass with a running
// maximum m and sum l.
//
// A warp per row and query head, four channels a lane.
#include "kvq_attn_common.cuh"
#include "kvq_paged.cuh"

namespace kvq {
namespace paged {
namespace {

constexpr int kThreads = 256;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

template <int DT, int QT>
__global__ void __launch_bounds__(kThreads) tree_kernel(TreeArgs a) {
  wait_prior_grid();
  allow_dependents();
  const int lane = threadIdx.x & 31, warps = gridDim.x * (kThreads / 32);
  for (long long w = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5); w < (long long)a.n_rows * a.Hq; w += warps) {
    const int row = int(w / a.Hq), hq = int(w % a.Hq), h = hq / a.g;
    int b = row, row0 = row, n = 1;
    if (a.offsets != nullptr) {
      int lo = 0, hi = a.B - 1;
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (a.offsets[mid] <= row) lo = mid;
        else hi = mid - 1;
      }
      b = lo;
      n = row_range(a.offsets, a.n_rows, b, row0);
    }
    if (n < 0) flag(a.c, KVQ_PAGED_ERR_LENGTH);
    if (n < 0 || row < row0 || row >= row0 + n) continue;
    const int i = row - row0, P = checked_len(a.lens, b, a.max_pages, a.c.ps);
    bool bad = P < 0 || P + (long long)n > (long long)a.max_pages * a.c.ps.d || n > KVQ_PAGED_MAX_DRAFT ||
               (a.mask != nullptr && n > 32 * a.mask_words);
    if (bad) flag(a.c, KVQ_PAGED_ERR_LENGTH);
    float m = -INFINITY, l = 0.0f;
    float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    const float4 q = load4<QT>(a.q + row * a.q_stride + (hq * kD + 4 * lane) * 2);
    for (int t = 0; !bad && t < P + n; ++t) {
      const int j = t - P, e = a.c.ps.div(t), page = a.table[(long long)b * a.max_pages + e];
      if (page < 0 || page >= a.c.n_pages) {
        flag(a.c, KVQ_PAGED_ERR_PAGE);
        bad = true;
        break;
      }
      if (j >= 0 && !(a.mask == nullptr ? j <= i : (a.mask[(long long)row * a.mask_words + j / 32] >> (j % 32)) & 1)) continue;
      const int place = t - e * int(a.c.ps.d);
      const long long off = (long long)page * a.c.page_stride + (long long)place * a.c.token_stride +
                            (long long)h * a.c.head_stride + 4 * lane * elem_bytes<DT>();
      float4 k = load4<DT>(a.c.k + off), v = load4<DT>(a.c.v + off);
      if constexpr (DT == kE4m3) {
        const long long s = a.c.token_scales ? ((long long)page * a.c.H + h) * int(a.c.ps.d) + place : h;
        if (a.c.k_scale != nullptr) k = times(k, a.c.k_scale[s]);
        if (a.c.v_scale != nullptr) v = times(v, a.c.v_scale[s]);
      }
      float x = q.x * k.x + q.y * k.y + q.z * k.z + q.w * k.w;
#pragma unroll
      for (int s = 16; s > 0; s >>= 1) x += __shfl_xor_sync(0xFFFFFFFFu, x, s);
      x *= a.scale * kLog2e;
      const float mx = fmaxf(m, x), base = mx == -INFINITY ? 0.0f : mx, alpha = exp2f(m - base), p = exp2f(x - base);
      m = mx;
      l = fmaf(l, alpha, p);
      o = make_float4(fmaf(p, v.x, o.x * alpha), fmaf(p, v.y, o.y * alpha), fmaf(p, v.z, o.z * alpha),
                      fmaf(p, v.w, o.w * alpha));
    }
    const float r = bad ? NAN : 1.0f / (l == 0.0f ? 1.0f : l);
    store4<QT>(a.out + ((long long)row * a.Hq + hq) * (kD * 2) + 8 * lane, bad ? make_float4(r, r, r, r) : times(o, r));
    if (a.lse != nullptr && lane == 0) a.lse[(long long)row * a.Hq + hq] = bad ? NAN : (m + log2f(l)) * kLn2;
  }
}

template <int DT, int QT>
cudaError_t launch_types(const TreeArgs& a, cudaStream_t stream) {
  const long long need = ((long long)a.n_rows * a.Hq * 32 + kThreads - 1) / kThreads, fit = 8LL * a.sms;
  count_launch();
  return launch_dependent(tree_kernel<DT, QT>, dim3(int(need < fit ? need : fit)), dim3(kThreads), 0, stream, a);
}

}  // namespace

size_t tree_workspace(int B, int H, int Hq, int n_rows, int sms) { return 16; }

cudaError_t launch_tree(const TreeArgs& a, cudaStream_t stream) {
  const bool bf = a.q_dtype == kBf16;
  if (a.dtype == kBf16) return launch_types<kBf16, kBf16>(a, stream);
  if (a.dtype == kFp16) return launch_types<kFp16, kFp16>(a, stream);
  return bf ? launch_types<kE4m3, kBf16>(a, stream) : launch_types<kE4m3, kFp16>(a, stream);
}

}  // namespace paged
}  // namespace kvq
