// kvq_paged_append.cu — new keys and values into the pages of a paged cache,
// keys (and queries) rotated to their position on the way, and the pages' key
// bounds kept up.
//
// Rotation of a pair (x, y) by its angle's cosine and sine: x' = x cos - y sin,
// y' = y cos + x sin, in FP32 with one rounding to the stored type. Bounds:
// min and max of the stored keys of a page per head and channel.
//
// A unit of work is (request, touched page, head), heads fastest: the H KV heads
// (K and V together) and then the query heads. Since a unit holds every new token
// of its page, the bounds need no atomics: one reader and writer per (page, head).
// Lane l of a warp holds channels 4l .. 4l+3; the partner channels of the split
// pairing come by a second load of the row, which hits L1.
#include "kvq_paged.cuh"

namespace kvq {
namespace paged {
namespace {

constexpr int kThreads = 128;
constexpr int kUnroll = 4;  // rows in flight per warp

__device__ __forceinline__ float min_nan(float a, float b) {
  float r;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float4 min_nan(float4 a, float4 b) {
  return make_float4(min_nan(a.x, b.x), min_nan(a.y, b.y), min_nan(a.z, b.z), min_nan(a.w, b.w));
}
__device__ __forceinline__ float4 max_nan(float4 a, float4 b) {
  return make_float4(max_nan(a.x, b.x), max_nan(a.y, b.y), max_nan(a.z, b.z), max_nan(a.w, b.w));
}

// New rows of request b, or -1 when its start or offsets are outside their range.
__device__ __forceinline__ int rows_of(const AppendArgs& a, int b, int& start, int& row0) {
  start = a.start[b];
  int n = 1;
  row0 = b;
  if (a.offsets != nullptr) {
    row0 = a.offsets[b];
    const int row1 = a.offsets[b + 1];
    if (row0 < 0 || row1 < row0 || row1 > a.n_rows) return -1;
    n = row1 - row0;
  }
  if (start < 0 || (long long)start + n > (long long)a.max_pages * a.c.ps.d) return -1;
  return n;
}

// Pages that request b's new rows touch.
__device__ __forceinline__ int pages_of(const AppendArgs& a, int b) {
  int start, row0;
  const int n = rows_of(a, b, start, row0);
  return n <= 0 ? 0 : a.c.ps.div(start + n - 1) - a.c.ps.div(start) + 1;
}

// One lane's four channels of a row at `p` (the head's first channel), rotated.
struct Lane {
  int d;         // first channel
  int partner;   // first channel of the partners (split pairing)
  int angle;     // first angle
  float sign;    // -1: first of its pair, +1: second
  bool rotated;
};

template <int IN>
struct Row {
  float4 x, y, cs, sn;
  __device__ __forceinline__ void load(const AppendArgs& a, const Lane& L, const char* p, long long pos) {
    x = load4<IN>(p + 2 * L.d);
    if (!L.rotated) return;
    const float* t = a.rope + pos * a.R;
    if (a.interleaved) {
      const float2 c = *reinterpret_cast<const float2*>(t + L.angle);
      const float2 s = *reinterpret_cast<const float2*>(t + a.R / 2 + L.angle);
      cs = make_float4(c.x, c.x, c.y, c.y);
      sn = make_float4(-s.x, s.x, -s.y, s.y);
    } else {
      y = load4<IN>(p + 2 * L.partner);
      cs = *reinterpret_cast<const float4*>(t + L.angle);
      sn = *reinterpret_cast<const float4*>(t + a.R / 2 + L.angle);
    }
  }
  __device__ __forceinline__ float4 rotate(const AppendArgs& a, const Lane& L) const {
    if (!L.rotated) return x;
    if (a.interleaved)
      return make_float4(x.x * cs.x + x.y * sn.x, x.y * cs.y + x.x * sn.y, x.z * cs.z + x.w * sn.z,
                         x.w * cs.w + x.z * sn.w);
    return make_float4(x.x * cs.x + L.sign * y.x * sn.x, x.y * cs.y + L.sign * y.y * sn.y,
                       x.z * cs.z + L.sign * y.z * sn.z, x.w * cs.w + L.sign * y.w * sn.w);
  }
};

__device__ __forceinline__ float4 div4(float4 x, float s) {
  return make_float4(__fdiv_rn(x.x, s), __fdiv_rn(x.y, s), __fdiv_rn(x.z, s), __fdiv_rn(x.w, s));
}

// WARPS warps share a unit's rows: 1 where a page gets a row or two (a decode
// step), the block's 4 where it gets many (their bounds joined in shared memory).
template <int DT, int IN, int WARPS>
__global__ void __launch_bounds__(kThreads) append_kernel(AppendArgs a) {
  constexpr int kGroups = kThreads / 32 / WARPS;
  __shared__ Prefix<kThreads> S;
  __shared__ float4 red[WARPS > 1 ? 2 * WARPS * 32 : 1];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, sub = warp % WARPS;
  const int heads = a.c.H + (a.q != nullptr ? a.Hq : 0);
  auto count = [&](int b) { return (long long)pages_of(a, b) * heads; };
  long long total = (long long)a.B * heads;
  if (a.offsets != nullptr) {
    build_prefix<kThreads>(S, a.B, count);
    total = S.pre[kThreads];
  }
  if (a.c.err != nullptr && blockIdx.x == 0) {
    for (int b = threadIdx.x; b < a.B; b += kThreads) {
      int start, row0;
      if (rows_of(a, b, start, row0) < 0) flag(a.c, KVQ_PAGED_ERR_LENGTH);
    }
  }
  const long long groups = (long long)gridDim.x * kGroups, me = (long long)blockIdx.x * kGroups + warp / WARPS;
  const long long u0 = me * total / groups, u1 = (me + 1) * total / groups;
  if (u0 >= u1) return;

  Lane L;
  L.d = 4 * lane;
  L.rotated = L.d < a.R;
  const bool second = L.d >= a.R / 2;
  L.partner = second ? L.d - a.R / 2 : L.d + a.R / 2;
  L.angle = a.interleaved ? L.d / 2 : (second ? L.d - a.R / 2 : L.d);
  L.sign = second ? 1.0f : -1.0f;

  long long at = u0;
  int b, hh, page_i;
  if (a.offsets == nullptr) {
    b = int(u0 / heads);
    hh = int(u0 % heads);
    page_i = 0;
  } else {
    b = find_request<kThreads>(S, a.B, count, at);
    page_i = int(at / heads);
    hh = int(at % heads);
  }
  int start = 0, row0 = 0, n = rows_of(a, b, start, row0), pages = pages_of(a, b);
  for (long long u = u0; u < u1; ++u) {
    while (pages == 0 && a.offsets != nullptr && b < a.B - 1) {  // requests that bring nothing hold no unit
      ++b;
      n = rows_of(a, b, start, row0);
      pages = pages_of(a, b);
    }
    if (n > 0) {
      const int ps = int(a.c.ps.d), page0 = a.c.ps.div(start) + page_i;
      const int first = max(start, page0 * ps), last = min(start + n, (page0 + 1) * ps);  // tokens of the page
      const int page = a.table[(long long)b * a.max_pages + page0];
      const bool page_ok = page >= 0 && page < a.c.n_pages;
      if (!page_ok && lane == 0) flag(a.c, KVQ_PAGED_ERR_PAGE);
      const bool is_q = hh >= a.c.H;
      const int h = is_q ? hh - a.c.H : hh;
      const float ks = DT == kE4m3 && !is_q && a.c.k_scale != nullptr ? a.c.k_scale[h] : 1.0f;
      const float vs = DT == kE4m3 && !is_q && a.c.v_scale != nullptr ? a.c.v_scale[h] : 1.0f;
      float4 lo = make_float4(INFINITY, INFINITY, INFINITY, INFINITY);
      float4 hi = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
      bool any = false;
      for (int t0 = first + sub; page_ok && t0 < last; t0 += WARPS * kUnroll) {
        Row<IN> r[kUnroll];
        float4 v[kUnroll];
        bool ok[kUnroll];
#pragma unroll
        for (int i = 0; i < kUnroll; ++i) {
          const int t = t0 + i * WARPS;
          ok[i] = t < last;
          if (!ok[i]) continue;
          const long long row = row0 + (t - start);
          const int pos = a.positions != nullptr ? a.positions[row] : t;
          if (a.R > 0 && (pos < 0 || pos >= a.rope_positions)) {
            ok[i] = false;
            if (lane == 0) flag(a.c, KVQ_PAGED_ERR_POSITION);
            continue;
          }
          if (is_q) {
            r[i].load(a, L, a.q + row * a.q_stride + h * 256, pos);
          } else {
            r[i].load(a, L, a.k + row * a.k_stride + h * 256, pos);
            v[i] = load4<IN>(a.v + row * a.v_stride + h * 256 + 2 * L.d);
          }
        }
        __syncwarp();  // q_out may be q: every lane has read its partners
#pragma unroll
        for (int i = 0; i < kUnroll; ++i) {
          if (!ok[i]) continue;
          const int t = t0 + i * WARPS;
          const long long row = row0 + (t - start);
          float4 x = r[i].rotate(a, L);
          if (is_q) {
            store4<IN>(a.q_out + row * a.q_out_stride + h * 256 + 2 * L.d, x);
            continue;
          }
          const long long place = (long long)page * a.c.page_stride + (long long)(t - page0 * ps) * a.c.token_stride +
                                  (long long)h * a.c.head_stride + L.d * elem_bytes<DT>();
          if constexpr (DT == kE4m3) {
            x = div4(x, ks);
            v[i] = div4(v[i], vs);
          }
          store4<DT>(a.c.k + place, x);
          store4<DT>(a.c.v + place, v[i]);
          const float4 s = rounded4<DT>(x);
          lo = min_nan(lo, s);
          hi = max_nan(hi, s);
          any = true;
        }
      }
      if (!is_q && a.c.bounds != nullptr && page_ok) {
        if constexpr (WARPS > 1) {
          red[sub * 32 + lane] = lo;
          red[(WARPS + sub) * 32 + lane] = hi;
          any = __syncthreads_or(any);
          if (sub == 0) {
            for (int w = 1; w < WARPS; ++w) {
              lo = min_nan(lo, red[w * 32 + lane]);
              hi = max_nan(hi, red[(WARPS + w) * 32 + lane]);
            }
          }
        }
        if (sub == 0 && any) {
          char* p = a.c.bounds + (((long long)page * a.c.H + h) * 2 * kD + L.d) * elem_bytes<DT>();
          if (first > page0 * ps) {
            lo = min_nan(lo, load4<DT>(p));
            hi = max_nan(hi, load4<DT>(p + kD * elem_bytes<DT>()));
          }
          store4<DT>(p, lo);
          store4<DT>(p + kD * elem_bytes<DT>(), hi);
        }
        if constexpr (WARPS > 1) __syncthreads();  // red is free again
      }
    }
    if (++hh == heads) {
      hh = 0;
      if (a.offsets == nullptr || ++page_i == pages) {
        page_i = 0;
        if (++b < a.B) {
          n = rows_of(a, b, start, row0);
          pages = pages_of(a, b);
        }
      }
    }
  }
}

template <int DT, int IN, int WARPS>
cudaError_t launch_form(const AppendArgs& a, int blocks, cudaStream_t stream) {
  append_kernel<DT, IN, WARPS><<<blocks, kThreads, 0, stream>>>(a);
  count_launch();
  return cudaGetLastError();
}

template <int DT, int IN>
cudaError_t launch_types(const AppendArgs& a, int sms, cudaStream_t stream) {
  const long long heads = a.c.H + (a.q != nullptr ? a.Hq : 0);
  const long long pages = a.offsets == nullptr ? a.B : a.n_rows / a.c.ps.d + 2 * (long long)a.B;  // at most
  const bool many = a.offsets != nullptr && a.n_rows > 8LL * a.B && a.c.ps.d > 4;
  const long long need = many ? pages * heads : (pages * heads + 3) / 4;
  const int blocks = int(need < 8LL * sms ? need : 8LL * sms);
  return many ? launch_form<DT, IN, 4>(a, blocks, stream) : launch_form<DT, IN, 1>(a, blocks, stream);
}

}  // namespace

cudaError_t launch_append(const AppendArgs& a, int sms, cudaStream_t stream) {
  const bool bf = a.in_dtype == kBf16;
  switch (a.dtype) {
    case kBf16: return launch_types<kBf16, kBf16>(a, sms, stream);
    case kFp16: return launch_types<kFp16, kFp16>(a, sms, stream);
    default: return bf ? launch_types<kE4m3, kBf16>(a, sms, stream) : launch_types<kE4m3, kFp16>(a, sms, stream);
  }
}

}  // namespace paged
}  // namespace kvq
