// kvq_paged_attn.cu — decode attention of one query per request over a paged
// cache, all pages or the selected ones.
//
// s_t = scale q.k_t, out = sum_t e^(s_t - m) v_t / l, lse = m + ln l, in one pass
// with a running maximum m and sum l. One block per (request, query head); a
// warp takes every fourth token, its lanes four channels each.
#include "kvq_paged.cuh"

namespace kvq {
namespace paged {
namespace {

constexpr int kThreads = 128;

template <int DT, int QT>
__global__ void __launch_bounds__(kThreads) attn_kernel(AttnArgs a) {
  __shared__ float sm[4], sl[4], sacc[4][kD];
  const int b = blockIdx.x / a.Hq, hq = blockIdx.x % a.Hq, h = hq / a.g;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, ps = int(a.c.ps.d);
  const int T = checked_len(a.lens, b, a.max_pages, a.c.ps);
  bool bad = T < 0;
  if (bad && threadIdx.x == 0) flag(a.c, KVQ_PAGED_ERR_LENGTH);
  const int pages = bad ? 0 : (int)(((long long)T + ps - 1) / ps);
  const int entries = a.sel != nullptr ? min(a.n_select, pages) : pages;
  const float4 q = load4<QT>(a.q + (long long)b * a.q_stride + (hq * kD + 4 * lane) * 2);
  const float ks = DT == kE4m3 && a.c.k_scale != nullptr ? a.c.k_scale[h] : 1.0f;
  const float vs = DT == kE4m3 && a.c.v_scale != nullptr ? a.c.v_scale[h] : 1.0f;
  const float scale = a.scale * ks;
  float m = -INFINITY, l = 0.0f;
  float4 acc = make_float4(0, 0, 0, 0);
  const int32_t* sel = a.sel == nullptr ? nullptr : a.sel + ((long long)b * a.c.H + h) * a.n_select;
  for (int e = 0; e < entries; ++e) {
    int lp = e;
    if (sel != nullptr) {
      lp = sel[e];
      const int before = e > 0 ? sel[e - 1] : -1;
      const bool ok = lp == -1 ? true : (lp >= 0 && lp < pages && lp > before && (e == 0 || before >= 0));
      if (!ok) {
        bad = true;
        if (threadIdx.x == 0) flag(a.c, KVQ_PAGED_ERR_SELECTION);
      }
      if (!ok || lp == -1) continue;
    }
    const int page = a.table[(long long)b * a.max_pages + lp];
    if (page < 0 || page >= a.c.n_pages) {
      bad = true;
      if (threadIdx.x == 0) flag(a.c, KVQ_PAGED_ERR_PAGE);
      continue;
    }
    const int n = min(ps, T - lp * ps);
    for (int s = warp; s < n; s += 4) {
      const long long at = (long long)page * a.c.page_stride + (long long)s * a.c.token_stride +
                           (long long)h * a.c.head_stride + 4 * lane * elem_bytes<DT>();
      const float4 k = load4<DT>(a.c.k + at), v = load4<DT>(a.c.v + at);
      float x = q.x * k.x + q.y * k.y + q.z * k.z + q.w * k.w;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xFFFFFFFFu, x, o);
      x *= scale;
      const float mn = fmaxf(m, x), base = mn == -INFINITY ? 0.0f : mn;
      const float al = expf(m - base), p = expf(x - base);
      l = l * al + p;
      acc = make_float4(acc.x * al + p * v.x, acc.y * al + p * v.y, acc.z * al + p * v.z, acc.w * al + p * v.w);
      m = mn;
    }
  }
  if (lane == 0) {
    sm[warp] = m;
    sl[warp] = l;
  }
  *reinterpret_cast<float4*>(&sacc[warp][4 * lane]) = acc;
  __syncthreads();
  const float mx = fmaxf(fmaxf(sm[0], sm[1]), fmaxf(sm[2], sm[3])), base = mx == -INFINITY ? 0.0f : mx;
  float lt = 0.0f, o = 0.0f;
  for (int w = 0; w < 4; ++w) {
    const float f = expf(sm[w] - base);
    lt += sl[w] * f;
    o += sacc[w][threadIdx.x] * f;
  }
  o = lt > 0.0f ? o / lt * vs : (lt == 0.0f ? 0.0f : NAN);
  a.out[((long long)b * a.Hq + hq) * kD + threadIdx.x] = bad ? NAN : o;
  if (a.lse != nullptr && threadIdx.x == 0) a.lse[(long long)b * a.Hq + hq] = bad ? NAN : mx + logf(lt);
}

}  // namespace

size_t attn_workspace(int B, int H, int Hq, int sms) { return 16; }

cudaError_t launch_attn(const AttnArgs& a, cudaStream_t stream) {
  const int n = a.B * a.Hq;
  const bool bf = a.q_dtype == kBf16;
  if (a.dtype == kBf16) attn_kernel<kBf16, kBf16><<<n, kThreads, 0, stream>>>(a);
  else if (a.dtype == kFp16) attn_kernel<kFp16, kFp16><<<n, kThreads, 0, stream>>>(a);
  else if (bf) attn_kernel<kE4m3, kBf16><<<n, kThreads, 0, stream>>>(a);
  else attn_kernel<kE4m3, kFp16><<<n, kThreads, 0, stream>>>(a);
  count_launch();
  return cudaGetLastError();
}

}  // namespace paged
}  // namespace kvq
