// kvq_paged_append.cu — new keys and values into the pages of a paged cache,
// keys (and queries) rotated to their position on the way, and the pages' key
// bounds kept up.
//
// Rotation of a pair (x, y) by its angle's cosine and sine: x' = x cos - y sin,
// y' = y cos + x sin, in FP32 with one rounding to the stored type. Bounds:
// min and max of the stored keys of a page per head and channel. Bound: HBM (each
// row is read and written once); a decode step is too small for that and bound by
// the chain of dependent loads start -> page table and rotation table -> store.
//
// A unit of work is (request, touched page, head), heads fastest: the H KV heads
// (K and V together) and then the query heads. A warp has every new token of its
// page and head, so the bounds need no atomics. Lane l holds channels 4l .. 4l+3.
// Two kernels, the host choosing by the rows a request brings on average:
//   few (up to 8)  a warp takes any units in turn, everything by plain loads;
//   many           a block takes a page and eight heads at a time, one per warp: the
//                  rotation table's rows of the page are staged once in shared
//                  memory for the eight, and a warp keeps eight rows in flight.
#include "kvq_paged.cuh"

namespace kvq {
namespace paged {
namespace {

constexpr int kFewThreads = 128;
constexpr int kFewRows = 2;        // rows in flight per warp
constexpr int kManyThreads = 256;
constexpr int kManyWarps = kManyThreads / 32;
constexpr int kManyRows = 8;
constexpr int kSlice = 64;         // rows of the rotation table staged at a time
constexpr int kManyBlocksPerSm = 3;

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

// A lane's share of the rotation.
struct Lane {
  int d;         // first channel
  int partner;   // lane that holds the partners (split pairing)
  int angle;     // first angle
  float sign;    // -1: first of its pair, +1: second
  bool rotated;
  __device__ __forceinline__ Lane(const AppendArgs& a, int lane) {
    d = 4 * lane;
    rotated = d < a.R;
    const bool second = d >= a.R / 2;
    partner = rotated ? (second ? lane - a.R / 8 : lane + a.R / 8) : lane;
    angle = a.interleaved ? d / 2 : (second ? d - a.R / 2 : d);
    sign = second ? 1.0f : -1.0f;
  }
};

struct Angles {
  float4 cs, sn;
  // t: the position's row of the rotation table (global or shared memory)
  __device__ __forceinline__ void load(const AppendArgs& a, const Lane& L, const float* t) {
    if (!L.rotated) return;
    if (a.interleaved) {
      const float2 c = *reinterpret_cast<const float2*>(t + L.angle);
      const float2 s = *reinterpret_cast<const float2*>(t + a.R / 2 + L.angle);
      cs = make_float4(c.x, c.x, c.y, c.y);
      sn = make_float4(-s.x, s.x, -s.y, s.y);
    } else {
      cs = *reinterpret_cast<const float4*>(t + L.angle);
      sn = *reinterpret_cast<const float4*>(t + a.R / 2 + L.angle);
      sn = make_float4(L.sign * sn.x, L.sign * sn.y, L.sign * sn.z, L.sign * sn.w);
    }
  }
};

template <int IN>
__device__ __forceinline__ float4 floats(uint2 w) {
  return load4<IN>(&w);
}

// The lane's four channels `w` rotated; all lanes of the warp take part.
template <int IN>
__device__ __forceinline__ float4 rotate(const AppendArgs& a, const Lane& L, const Angles& t, uint2 w) {
  const float4 x = floats<IN>(w);
  float4 y;
  if (a.interleaved) {
    y = make_float4(x.y, x.x, x.w, x.z);
  } else {
    uint2 o;
    o.x = __shfl_sync(0xFFFFFFFFu, w.x, L.partner);
    o.y = __shfl_sync(0xFFFFFFFFu, w.y, L.partner);
    y = floats<IN>(o);
  }
  if (!L.rotated) return x;
  return make_float4(x.x * t.cs.x + y.x * t.sn.x, x.y * t.cs.y + y.y * t.sn.y, x.z * t.cs.z + y.z * t.sn.z,
                     x.w * t.cs.w + y.w * t.sn.w);
}

__device__ __forceinline__ float4 div4(float4 x, float s) {
  return make_float4(__fdiv_rn(x.x, s), __fdiv_rn(x.y, s), __fdiv_rn(x.z, s), __fdiv_rn(x.w, s));
}

// What a warp does to one (page, head): where rows come from and go to.
template <int DT, int IN>
struct Unit {
  bool is_q, live;  // live: the page is in the pool
  int h, page, place0, first, last, start, row0;
  float ks, vs;
  float4 lo, hi;
  bool any;

  __device__ __forceinline__ void open(const AppendArgs& a, int b, int page_of_request, int hh, int s, int r0, int n) {
    const int ps = int(a.c.ps.d);
    start = s;
    row0 = r0;
    place0 = page_of_request * ps;
    first = max(start, place0);
    last = min(start + n, place0 + ps);
    page = a.table[(long long)b * a.max_pages + page_of_request];
    is_q = hh >= a.c.H;
    h = is_q ? hh - a.c.H : hh;
    ks = DT == kE4m3 && !is_q && a.c.k_scale != nullptr ? a.c.k_scale[h] : 1.0f;
    vs = DT == kE4m3 && !is_q && a.c.v_scale != nullptr ? a.c.v_scale[h] : 1.0f;
    lo = make_float4(INFINITY, INFINITY, INFINITY, INFINITY);
    hi = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
    any = false;
  }
  __device__ __forceinline__ void check(const AppendArgs& a) {  // (apart from open: the loads in between need no page)
    live = page >= 0 && page < a.c.n_pages;
    if (!live) flag(a.c, KVQ_PAGED_ERR_PAGE);
  }
  __device__ __forceinline__ uint2 key(const AppendArgs& a, const Lane& L, int t) const {
    const long long row = row0 + (t - start);
    const char* p = is_q ? a.q + row * a.q_stride : a.k + row * a.k_stride;
    return *reinterpret_cast<const uint2*>(p + (h * kD + L.d) * 2);
  }
  __device__ __forceinline__ uint2 value(const AppendArgs& a, const Lane& L, int t) const {
    const long long row = row0 + (t - start);
    return *reinterpret_cast<const uint2*>(a.v + row * a.v_stride + (h * kD + L.d) * 2);
  }
  __device__ __forceinline__ void put(const AppendArgs& a, const Lane& L, int t, float4 x, uint2 v) {
    if (is_q) {
      store4<IN>(a.q_out + (long long)(row0 + (t - start)) * a.q_out_stride + (h * kD + L.d) * 2, x);
      return;
    }
    const long long place = (long long)page * a.c.page_stride + (long long)(t - place0) * a.c.token_stride +
                            (long long)h * a.c.head_stride + L.d * elem_bytes<DT>();
    if constexpr (DT == kE4m3) {
      x = div4(x, ks);
      store4<DT>(a.c.v + place, div4(floats<IN>(v), vs));
    } else {
      *reinterpret_cast<uint2*>(a.c.v + place) = v;
    }
    store4<DT>(a.c.k + place, x);
    const float4 s = rounded4<DT>(x);
    lo = min_nan(lo, s);
    hi = max_nan(hi, s);
    any = true;
  }
  __device__ __forceinline__ void close(const AppendArgs& a, const Lane& L) const {
    if (is_q || !any || a.c.bounds == nullptr) return;
    char* p = a.c.bounds + (((long long)page * a.c.H + h) * 2 * kD + L.d) * elem_bytes<DT>();
    float4 l = lo, u = hi;
    if (first > place0) {  // the page held tokens before
      l = min_nan(l, load4<DT>(p));
      u = max_nan(u, load4<DT>(p + kD * elem_bytes<DT>()));
    }
    store4<DT>(p, l);
    store4<DT>(p + kD * elem_bytes<DT>(), u);
  }
};

// The row of the rotation table of token t, or -1 when it has none.
template <typename U>
__device__ __forceinline__ int position(const AppendArgs& a, const U& u, int t) {
  const int pos = a.positions != nullptr ? a.positions[u.row0 + (t - u.start)] : t;
  return a.R > 0 && (pos < 0 || pos >= a.rope_positions) ? -1 : pos;
}

__device__ __forceinline__ void flag_lengths(const AppendArgs& a) {
  if (a.c.err == nullptr || blockIdx.x != 0) return;
  for (int b = threadIdx.x; b < a.B; b += blockDim.x) {
    int start, row0;
    if (rows_of(a, b, start, row0) < 0) flag(a.c, KVQ_PAGED_ERR_LENGTH);
  }
}

template <int DT, int IN>
__global__ void __launch_bounds__(kFewThreads) append_few_kernel(AppendArgs a) {
  __shared__ Prefix<kFewThreads> S;
  const int lane = threadIdx.x & 31;
  const int heads = a.c.H + (a.q != nullptr ? a.Hq : 0);
  auto count = [&](int b) { return (long long)pages_of(a, b) * heads; };
  long long total = (long long)a.B * heads;
  if (a.offsets != nullptr) {
    build_prefix<kFewThreads>(S, a.B, count);
    total = S.pre[kFewThreads];
  }
  flag_lengths(a);
  const long long warps = (long long)gridDim.x * (kFewThreads / 32);
  const long long me = (long long)blockIdx.x * (kFewThreads / 32) + threadIdx.x / 32;
  const long long u0 = me * total / warps, u1 = (me + 1) * total / warps;
  if (u0 >= u1) return;
  const Lane L(a, lane);
  long long at = u0;
  int b, hh, page_i;
  if (a.offsets == nullptr) {
    b = int(u0 / heads);
    hh = int(u0 % heads);
    page_i = 0;
  } else {
    b = find_request<kFewThreads>(S, a.B, count, at);
    page_i = int(at / heads);
    hh = int(at % heads);
  }
  int start = 0, row0 = 0, n = rows_of(a, b, start, row0), pages = pages_of(a, b);
  for (long long w = u0; w < u1; ++w) {
    while (pages == 0 && a.offsets != nullptr && b < a.B - 1) {  // requests that bring nothing hold no unit
      ++b;
      n = rows_of(a, b, start, row0);
      pages = pages_of(a, b);
    }
    if (n > 0) {
      Unit<DT, IN> u;
      u.open(a, b, a.c.ps.div(start) + page_i, hh, start, row0, n);
      for (int t0 = u.first; t0 < u.last; t0 += kFewRows) {
        uint2 x[kFewRows], v[kFewRows];
        Angles g[kFewRows];
        bool ok[kFewRows];
#pragma unroll
        for (int i = 0; i < kFewRows; ++i) {
          const int t = t0 + i;
          ok[i] = t < u.last;
          x[i] = v[i] = make_uint2(0, 0);
          if (!ok[i]) continue;
          x[i] = u.key(a, L, t);
          if (!u.is_q) v[i] = u.value(a, L, t);
          const int pos = position(a, u, t);
          ok[i] = pos >= 0;
          if (ok[i]) g[i].load(a, L, a.rope + (long long)pos * a.R);
          else flag(a.c, KVQ_PAGED_ERR_POSITION);
        }
        u.check(a);
#pragma unroll
        for (int i = 0; i < kFewRows; ++i) {
          const float4 r = rotate<IN>(a, L, g[i], x[i]);
          if (ok[i] && u.live) u.put(a, L, t0 + i, r, v[i]);
        }
      }
      u.close(a, L);
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

template <int DT, int IN>
__global__ void __launch_bounds__(kManyThreads, kManyBlocksPerSm) append_many_kernel(AppendArgs a) {
  __shared__ Prefix<kManyThreads> S;
  __shared__ int s_pos[kSlice];  // table row of each staged row, -1: none
  extern __shared__ __align__(16) float s_rope[];  // [kSlice][R]
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int heads = a.c.H + (a.q != nullptr ? a.Hq : 0), groups = (heads + kManyWarps - 1) / kManyWarps;
  auto count = [&](int b) { return (long long)pages_of(a, b) * groups; };
  build_prefix<kManyThreads>(S, a.B, count);
  flag_lengths(a);
  const long long total = S.pre[kManyThreads];
  const long long u0 = blockIdx.x * total / gridDim.x, u1 = (blockIdx.x + 1) * total / gridDim.x;
  if (u0 >= u1) return;
  const Lane L(a, lane);
  long long at = u0;
  int b = find_request<kManyThreads>(S, a.B, count, at);
  int page_i = int(at / groups), grp = int(at % groups);
  int start = 0, row0 = 0, n = rows_of(a, b, start, row0), pages = pages_of(a, b);
  for (long long w = u0; w < u1; ++w) {
    while (pages == 0 && b < a.B - 1) {
      ++b;
      n = rows_of(a, b, start, row0);
      pages = pages_of(a, b);
    }
    if (n > 0) {  // (the same for the whole block)
      const int hh = grp * kManyWarps + warp;
      const bool active = hh < heads;
      Unit<DT, IN> u;
      u.open(a, b, a.c.ps.div(start) + page_i, active ? hh : 0, start, row0, n);
      for (int s0 = u.first; s0 < u.last; s0 += kSlice) {
        const int rows = min(kSlice, u.last - s0), per = a.R / 4;  // 16-byte chunks of a table row
        __syncthreads();  // the slice before is done with
        if (threadIdx.x < rows) {
          const int pos = position(a, u, s0 + threadIdx.x);
          s_pos[threadIdx.x] = pos;
          if (pos < 0) flag(a.c, KVQ_PAGED_ERR_POSITION);
        }
        for (int i = threadIdx.x; i < rows * per; i += kManyThreads) {
          const int r = i / per, c = i - r * per, pos = position(a, u, s0 + r);
          if (pos >= 0)
            *reinterpret_cast<float4*>(s_rope + r * a.R + 4 * c) =
                *reinterpret_cast<const float4*>(a.rope + (long long)pos * a.R + 4 * c);
        }
        __syncthreads();
        if (s0 == u.first) u.check(a);
        if (!active || !u.live) continue;
        for (int r0 = 0; r0 < rows; r0 += kManyRows) {
          uint2 x[kManyRows], v[kManyRows];
#pragma unroll
          for (int i = 0; i < kManyRows; ++i) {
            x[i] = v[i] = make_uint2(0, 0);
            if (r0 + i < rows) {
              x[i] = u.key(a, L, s0 + r0 + i);
              if (!u.is_q) v[i] = u.value(a, L, s0 + r0 + i);
            }
          }
#pragma unroll
          for (int i = 0; i < kManyRows; ++i) {
            const int r = r0 + i;
            if (r >= rows) break;
            Angles g;
            g.load(a, L, s_rope + r * a.R);
            const float4 y = rotate<IN>(a, L, g, x[i]);
            if (s_pos[r] >= 0) u.put(a, L, s0 + r, y, v[i]);
          }
        }
      }
      if (active) u.close(a, L);
    }
    if (++grp == groups) {
      grp = 0;
      if (++page_i == pages) {
        page_i = 0;
        if (++b < a.B) {
          n = rows_of(a, b, start, row0);
          pages = pages_of(a, b);
        }
      }
    }
  }
}

template <int DT, int IN>
cudaError_t launch_types(const AppendArgs& a, int sms, cudaStream_t stream) {
  const long long heads = a.c.H + (a.q != nullptr ? a.Hq : 0);
  const long long pages = a.offsets == nullptr ? a.B : a.n_rows / a.c.ps.d + 2 * (long long)a.B;  // at most
  count_launch();
  if (a.offsets != nullptr && a.n_rows > 8LL * a.B) {
    const long long need = pages * ((heads + kManyWarps - 1) / kManyWarps), fit = (long long)kManyBlocksPerSm * sms;
    append_many_kernel<DT, IN>
        <<<int(need < fit ? need : fit), kManyThreads, size_t(kSlice) * a.R * 4, stream>>>(a);
  } else {
    const long long need = (pages * heads + 3) / 4, fit = 8LL * sms;
    append_few_kernel<DT, IN><<<int(need < fit ? need : fit), kFewThreads, 0, stream>>>(a);
  }
  return cudaGetLastError();
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
