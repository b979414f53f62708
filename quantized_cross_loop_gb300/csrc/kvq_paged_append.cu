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
// Sixteen lanes (a team) hold a row of a head, eight channels each: four of the
// first half of the rotated channels and their four partners of the second, so that
// a pair never crosses lanes and a lane needs four angles; channels behind the
// rotated ones are shared out eight a lane. All new tokens of a page and head are
// one unit of work, so the bounds need no atomics.
//   one row per request  (no offsets) one launch, in which a team takes any units in
//                  turn, KV heads (K and V together) and query heads alike: 3.1 us for
//                  64 requests and 8 + 32 heads, 5.5 us by the launches below;
//   any rows       one launch for the keys and values, and one for the queries, in
//                  which a team takes four heads of a row. (Both in one launch, some
//                  blocks for each, was slower: 264 against 223 us for four prompts of
//                  8192 tokens, the blocks of an SM getting unequal shares.)
// A unit of up to 32 rows is a warp's, a larger one a block's (4 x 2048 rows, pages of
// 64: 40 us by blocks, 46 by warps; pages of 16: 50 by blocks, 40 by warps), chosen by
// each unit's own rows, and the ranges are equal in rows, not units: batches mix
// prompts with requests of one row (a prompt of 2048 and 499 single rows, pages of 256:
// 24 us; by equal counts of units, each a team's, 849).
// Rows in flight and resident warps bound these; staging the rotation table in
// shared memory for eight heads, and fetching the next rows into registers ahead of
// the arithmetic, were slower (a table's row is in L1 for the heads that follow).
#include <type_traits>

#include "kvq_attn_common.cuh"
#include "kvq_paged.cuh"

namespace kvq {
namespace paged {
namespace {

constexpr int kStepThreads = 128;
constexpr int kStepBlocksPerSm = 5;
constexpr int kTeam = 16;          // lanes of a row
constexpr int kManyThreads = 256;
constexpr int kManyWarps = kManyThreads / 32;
constexpr int kKeyBlocksPerSm = 2;    // (as many as an SM's registers hold)
constexpr int kQueryBlocksPerSm = 4;
constexpr int kKeyRows = 4;        // rows a team has in flight
constexpr int kQueryHeads = 4;     // heads a team has in flight
constexpr int kWarpRows = 32;      // rows of a unit that a warp takes by itself

// Rows that the beginning and end of a unit count for: pages of up to kWarpRows take
// a warp much the same time whatever they hold (nine prompts of up to 613 rows, pages
// of 16, with 64 and with 8: 8-bit 21.9, 24.6 us, 16-bit 21.3, 23.6), larger ones take a
// block their rows (499 single rows and 2048, with 8 and with 32: pages of 64 21.6, 36.1
// us, of 256 24.5, 39.8).
__device__ __forceinline__ int unit_rows(int ps) { return ps <= kWarpRows ? 64 : 8; }

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

// A lane's channels: a .. a + 3 and b .. b + 3.
struct Lane {
  int a, b;
  bool rotated;
  __device__ __forceinline__ Lane(const AppendArgs& g, int lane) {
    rotated = lane < g.R / 8;
    a = rotated ? 4 * lane : 8 * lane;
    b = rotated ? g.R / 2 + 4 * lane : 8 * lane + 4;
  }
};

struct Angles {
  float4 c, s;  // of the lane's four pairs
  // t: the position's row of the rotation table (global or shared memory)
  template <bool INTER>
  __device__ __forceinline__ void load(const AppendArgs& g, const Lane& L, const float* t) {
    if (!L.rotated) return;
    if constexpr (INTER) {
      const float2 c0 = *reinterpret_cast<const float2*>(t + L.a / 2), c1 = *reinterpret_cast<const float2*>(t + L.b / 2);
      t += g.R / 2;
      const float2 s0 = *reinterpret_cast<const float2*>(t + L.a / 2), s1 = *reinterpret_cast<const float2*>(t + L.b / 2);
      c = make_float4(c0.x, c0.y, c1.x, c1.y);
      s = make_float4(s0.x, s0.y, s1.x, s1.y);
    } else {
      c = *reinterpret_cast<const float4*>(t + L.a);
      s = *reinterpret_cast<const float4*>(t + L.b);  // (b = R / 2 + a: the sines lie there)
    }
  }
};

struct Raw {  // eight 16-bit channels as they come
  uint2 a, b;
};
struct Wide {
  float4 a, b;
};

__device__ __forceinline__ Raw load_raw(const char* p, const Lane& L) {
  return Raw{*reinterpret_cast<const uint2*>(p + 2 * L.a), *reinterpret_cast<const uint2*>(p + 2 * L.b)};
}

// x c - y s and y c + x s.
__device__ __forceinline__ void turn(float& x, float& y, float c, float s) {
  const float u = x;
  x = x * c - y * s;
  y = y * c + u * s;
}

template <int IN, bool INTER>
__device__ __forceinline__ Wide rotate(const Lane& L, const Angles& t, const Raw& w) {
  Wide x{load4<IN>(&w.a), load4<IN>(&w.b)};
  if (!L.rotated) return x;
  if constexpr (INTER) {
    turn(x.a.x, x.a.y, t.c.x, t.s.x);
    turn(x.a.z, x.a.w, t.c.y, t.s.y);
    turn(x.b.x, x.b.y, t.c.z, t.s.z);
    turn(x.b.z, x.b.w, t.c.w, t.s.w);
  } else {
    turn(x.a.x, x.b.x, t.c.x, t.s.x);
    turn(x.a.y, x.b.y, t.c.y, t.s.y);
    turn(x.a.z, x.b.z, t.c.z, t.s.z);
    turn(x.a.w, x.b.w, t.c.w, t.s.w);
  }
  return x;
}

// Four stored keys as two words of 16-bit pairs (E4M3 as FP16, exact), and their
// smaller and larger ones; NaN stays.
template <int DT>
__device__ __forceinline__ uint2 pairs_of(const char* p) {
  if constexpr (DT == kE4m3) {
    const uint32_t w = *reinterpret_cast<const uint32_t*>(p);
    return make_uint2(e4m3x2_to_f16x2(w & 0xFFFFu), e4m3x2_to_f16x2(w >> 16));
  } else {
    return *reinterpret_cast<const uint2*>(p);
  }
}
template <int DT>
__device__ __forceinline__ void put_pairs(char* p, uint2 x) {
  if constexpr (DT == kE4m3) store4<kE4m3>(p, load4<kFp16>(&x));
  else *reinterpret_cast<uint2*>(p) = x;
}
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

// A head's scale for storing E4M3: the code of the FP32 quotient x / s, rounded to nearest, ties to even. lo and hi are
// the scale's reciprocal less and more 2^-20, so that x lo and x hi lie on either side of the quotient (all roundings,
// of a reciprocal below FP32's normal range too, come to less than 2^-20): where both have the same code it is the
// quotient's, else (one value in some 2^15) the row's values are divided. A power of two has an exact reciprocal: lo and
// hi are that. (8-bit chunks 21.9 us; one product without the check 20.9, which stored ties wrongly; divisions out of
// line, or a branch for every four values, 22.8.)
struct Quotient {
  float lo, hi, s;
  __device__ __forceinline__ void open(const float* scale, int h) {
    s = scale != nullptr ? scale[h] : 1.0f;
    const float r = __frcp_rn(s);
    const bool exact = fmaf(r, s, -1.0f) == 0.0f;
    lo = exact ? r : r * (1.0f - 0x1p-20f);
    hi = exact ? r : r * (1.0f + 0x1p-20f);
  }
  __device__ __forceinline__ static uint32_t codes(const float4& x, float r) {
    uint32_t c;
    store4<kE4m3>(&c, times(x, r));
    return c;
  }
};
__device__ __forceinline__ uint32_t divided(const float4& x, float s) {
  uint32_t c;
  store4<kE4m3>(&c, make_float4(__fdiv_rn(x.x, s), __fdiv_rn(x.y, s), __fdiv_rn(x.z, s), __fdiv_rn(x.w, s)));
  return c;
}

// What a team does to one (page, head): where rows come from and go to.
template <int DT, int IN>
struct Unit {
  using Word = std::conditional_t<DT == kE4m3, uint32_t, uint2>;  // four stored channels
  struct Stored {
    Word k[2], v[2];
  };
  bool is_q, live;  // live: the page is in the pool
  bool any;
  int h, page, place0, first, last, start, row0;
  Quotient ks, vs;        // E4M3
  uint32_t lo[4], hi[4];  // bounds of the lane's channels, 16-bit pairs

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
    if constexpr (DT == kE4m3)
      if (!is_q) {
        ks.open(a.c.k_scale, h);
        vs.open(a.c.v_scale, h);
      }
    any = false;
    constexpr uint32_t kInf = DT == kBf16 ? 0x7F807F80u : 0x7C007C00u;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      lo[i] = kInf;
      hi[i] = kInf | 0x80008000u;
    }
  }
  __device__ __forceinline__ void check(const AppendArgs& a) {  // (apart from open: the loads in between need no page)
    live = page >= 0 && page < a.c.n_pages;
    if (!live) flag(a.c, KVQ_PAGED_ERR_PAGE);
  }
  // Where token t's row of this head is, read and (queries) written.
  __device__ __forceinline__ const char* source(const AppendArgs& a, int t) const {
    const long long row = row0 + (t - start);
    return (is_q ? a.q + row * a.q_stride : a.k + row * a.k_stride) + h * (kD * 2);
  }
  __device__ __forceinline__ const char* value(const AppendArgs& a, int t) const {
    return a.v + (row0 + (t - start)) * a.v_stride + h * (kD * 2);
  }
  __device__ __forceinline__ char* query_out(const AppendArgs& a, int t) const {
    return a.q_out + (row0 + (t - start)) * a.q_out_stride + h * (kD * 2);
  }
  __device__ __forceinline__ long long place(const AppendArgs& a, int t) const {  // in k and v
    return (long long)page * a.c.page_stride + (long long)(t - place0) * a.c.token_stride +
           (long long)h * a.c.head_stride;
  }
  __device__ __forceinline__ static void put_query(const Lane& L, char* p, const Wide& x) {
    store4<IN>(p + 2 * L.a, x.a);
    store4<IN>(p + 2 * L.b, x.b);
  }
  // A row as it is stored.
  __device__ __forceinline__ Stored stored(const Wide& x, const Raw& v) const {
    Stored r;
    if constexpr (DT == kE4m3) {
      const Wide y{load4<IN>(&v.a), load4<IN>(&v.b)};
      r.k[0] = Quotient::codes(x.a, ks.lo);
      r.k[1] = Quotient::codes(x.b, ks.lo);
      r.v[0] = Quotient::codes(y.a, vs.lo);
      r.v[1] = Quotient::codes(y.b, vs.lo);
      if (((r.k[0] ^ Quotient::codes(x.a, ks.hi)) | (r.k[1] ^ Quotient::codes(x.b, ks.hi)) |
           (r.v[0] ^ Quotient::codes(y.a, vs.hi)) | (r.v[1] ^ Quotient::codes(y.b, vs.hi))) != 0u) {
        r.k[0] = divided(x.a, ks.s);
        r.k[1] = divided(x.b, ks.s);
        r.v[0] = divided(y.a, vs.s);
        r.v[1] = divided(y.b, vs.s);
      }
    } else {
      r.v[0] = v.a;
      r.v[1] = v.b;
      store4<DT>(&r.k[0], x.a);
      store4<DT>(&r.k[1], x.b);
    }
    return r;
  }
  __device__ __forceinline__ void put(const Lane& L, char* k, char* w, const Stored& r) {
    constexpr int kE = elem_bytes<DT>();
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int at = kE * (i == 0 ? L.a : L.b);
      *reinterpret_cast<Word*>(w + at) = r.v[i];
      *reinterpret_cast<Word*>(k + at) = r.k[i];
      const uint2 y = pairs_of<DT>(reinterpret_cast<const char*>(&r.k[i]));
      lo[2 * i] = smaller<DT>(lo[2 * i], y.x);
      lo[2 * i + 1] = smaller<DT>(lo[2 * i + 1], y.y);
      hi[2 * i] = larger<DT>(hi[2 * i], y.x);
      hi[2 * i + 1] = larger<DT>(hi[2 * i + 1], y.y);
    }
    any = true;
  }
  // The bounds of the two teams of a warp joined.
  __device__ __forceinline__ void join() {
    any = __any_sync(0xFFFFFFFFu, any);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      lo[i] = smaller<DT>(lo[i], __shfl_xor_sync(0xFFFFFFFFu, lo[i], kTeam));
      hi[i] = larger<DT>(hi[i], __shfl_xor_sync(0xFFFFFFFFu, hi[i], kTeam));
    }
  }
  __device__ __forceinline__ void close(const AppendArgs& a, const Lane& L) const {
    if (is_q || !any || a.c.bounds == nullptr) return;
    constexpr int kE = elem_bytes<DT>();
    char* p = a.c.bounds + ((long long)page * a.c.H + h) * (2 * kD * kE);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      char* to = p + kE * (i == 0 ? L.a : L.b);
      uint2 l = make_uint2(lo[2 * i], lo[2 * i + 1]), u = make_uint2(hi[2 * i], hi[2 * i + 1]);
      if (first > place0) {  // the page held tokens before
        const uint2 l0 = pairs_of<DT>(to), u0 = pairs_of<DT>(to + kD * kE);
        l = make_uint2(smaller<DT>(l.x, l0.x), smaller<DT>(l.y, l0.y));
        u = make_uint2(larger<DT>(u.x, u0.x), larger<DT>(u.y, u0.y));
      }
      put_pairs<DT>(to, l);
      put_pairs<DT>(to + kD * kE, u);
    }
  }
};

// The row of the rotation table of token t, or -1 when it has none (0 without a rotation).
template <typename U>
__device__ __forceinline__ int position(const AppendArgs& a, const U& u, int t) {
  if (a.R == 0) return 0;
  const int pos = a.positions != nullptr ? a.positions[u.row0 + (t - u.start)] : t;
  return pos < 0 || pos >= a.rope_positions ? -1 : pos;
}

__device__ __forceinline__ void flag_lengths(const AppendArgs& a) {
  if (a.c.err == nullptr || blockIdx.x != 0) return;
  for (int b = threadIdx.x; b < a.B; b += blockDim.x) {
    int start, row0;
    if (rows_of(a, b, start, row0) < 0) flag(a.c, KVQ_PAGED_ERR_LENGTH);
  }
}

// One row per request, keys, values and queries: a unit is a request's head.
template <int DT, int IN, bool INTER>
__global__ void __launch_bounds__(kStepThreads, kStepBlocksPerSm) append_step_kernel(AppendArgs a) {
  wait_prior_grid();
  allow_dependents();
  const int heads = a.c.H + (a.q != nullptr ? a.Hq : 0);
  const long long total = (long long)a.B * heads;
  flag_lengths(a);
  const int teams = int(gridDim.x) * (kStepThreads / kTeam);  // at most kStepBlocksPerSm x 8 an SM
  const int me = int(blockIdx.x) * (kStepThreads / kTeam) + threadIdx.x / kTeam;
  const long long u0 = part_start(me, total, teams), u1 = part_start(me + 1, total, teams);
  if (u0 >= u1) return;
  const Lane L(a, threadIdx.x % kTeam);
  int b, hh;
  divide(u0, heads, b, hh);
  for (long long w = u0; w < u1; ++w) {
    int start, row0;
    if (rows_of(a, b, start, row0) > 0) {
      Unit<DT, IN> u;
      u.open(a, b, a.c.ps.div(start), hh, start, row0, 1);
      const Raw x = load_raw(u.source(a, start), L);
      Raw v{};
      if (!u.is_q) v = load_raw(u.value(a, start), L);
      const int pos = position(a, u, start);
      Angles g;
      if (pos >= 0) g.load<INTER>(a, L, a.rope + (long long)pos * a.R);
      else flag(a.c, KVQ_PAGED_ERR_POSITION);
      u.check(a);
      if (pos >= 0 && u.live) {
        const Wide y = rotate<IN, INTER>(L, g, x);
        if (u.is_q) {
          u.put_query(L, u.query_out(a, start), y);
        } else {
          const long long place = u.place(a, start);
          u.put(L, a.c.k + place, a.c.v + place, u.stored(y, v));
          u.close(a, L);
        }
      }
    }
    if (++hh == heads) {
      hh = 0;
      ++b;
    }
  }
}

// Keys and values of any rows: a block takes the units that start in its range of the
// work, a row counting one and a unit unit_rows() more. Its warps take the units of up
// to kWarpRows rows in turn, all of them together the others.
template <int DT, int IN, bool INTER>
__global__ void __launch_bounds__(kManyThreads, kKeyBlocksPerSm) append_keys_kernel(AppendArgs a) {
  __shared__ Prefix<kManyThreads> S;
  __shared__ uint32_t s_bound[kManyWarps][8][kTeam];
  wait_prior_grid();
  allow_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x % kTeam, ps = int(a.c.ps.d), extra = unit_rows(ps);
  auto work_of = [&](int b) {
    int start, row0;
    const int n = rows_of(a, b, start, row0);
    return n <= 0 ? 0LL : a.c.H * (n + (long long)extra * (a.c.ps.div(start + n - 1) - a.c.ps.div(start) + 1));
  };
  build_prefix<kManyThreads>(S, a.B, work_of);
  flag_lengths(a);
  const long long total = S.pre[kManyThreads];
  const bool small = ps <= kWarpRows;  // no unit is for more than a warp: each warp has a range of its own
  const int ranges = small ? int(gridDim.x) * kManyWarps : int(gridDim.x);
  const int range = small ? int(blockIdx.x) * kManyWarps + warp : int(blockIdx.x);
  const long long s0 = part_start(range, total, ranges), s1 = part_start(range + 1, total, ranges);
  if (s0 >= s1) return;
  const Lane L(a, lane);
  long long at = s0;
  int b = find_request<kManyThreads>(S, a.B, work_of, at);
  int start, row0, n, p, pages;  // the request's rows; the unit's page, and the one behind the last
  auto load = [&] {
    n = rows_of(a, b, start, row0);
    p = a.c.ps.div(start);
    pages = n <= 0 ? 0 : a.c.ps.div(start + n - 1) + 1;
  };
  auto rows = [&] { return min(start + n, (p + 1) * ps) - max(start, p * ps); };  // on page p
  load();
  const long long first = (long long)a.c.H * (min(n, (p + 1) * ps - start) + extra);  // work of the first page
  if (at >= first) {
    int skip, rest;
    divide(at - first, a.c.H * (ps + extra), skip, rest);
    p += 1 + skip;
    at = rest;
  }
  int r = rows(), h = (int(at) + r + extra - 1) / (r + extra);  // the first unit that starts here or behind
  long long pos = s0 - at + (long long)h * (r + extra);
  int turn = 0;  // the warp that takes the next unit of its own
  for (;; ++h) {
    if (h == a.c.H) {
      h = 0;
      if (++p >= pages) {
        do {
          if (++b == a.B) return;
          load();
        } while (n <= 0);
      }
      r = rows();
    }
    if (pos >= s1) return;
    pos += r + extra;
    const bool all = r > kWarpRows;
    if (!all && !small) {
      const bool mine = turn == warp;
      turn = (turn + 1) % kManyWarps;
      if (!mine) continue;
    }
    const int team = all ? threadIdx.x / kTeam : (threadIdx.x / kTeam) & 1, step = all ? kManyThreads / kTeam : 2;
    Unit<DT, IN> u;
    u.open(a, b, p, h, start, row0, n);
    u.check(a);
    for (int t0 = u.live ? u.first + team : u.last; t0 < u.last; t0 += step * kKeyRows) {
      Raw x[kKeyRows], y[kKeyRows];
      Angles g[kKeyRows];
      bool ok[kKeyRows];
#pragma unroll
      for (int i = 0; i < kKeyRows; ++i) {
        const int t = t0 + i * step;
        ok[i] = t < u.last;
        if (!ok[i]) continue;
        x[i] = load_raw(u.source(a, t), L);
        y[i] = load_raw(u.value(a, t), L);
        const int row = position(a, u, t);
        ok[i] = row >= 0;
        if (ok[i]) g[i].load<INTER>(a, L, a.rope + (long long)row * a.R);
        else flag(a.c, KVQ_PAGED_ERR_POSITION);
      }
#pragma unroll
      for (int i = 0; i < kKeyRows; ++i) {
        if (!ok[i]) continue;
        const long long place = u.place(a, t0 + i * step);
        u.put(L, a.c.k + place, a.c.v + place, u.stored(rotate<IN, INTER>(L, g[i], x[i]), y[i]));
      }
    }
    if (a.c.bounds == nullptr) continue;
    __syncwarp();
    u.join();
    if (all) {
      if ((threadIdx.x & 31) < kTeam) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          s_bound[warp][i][lane] = u.lo[i];
          s_bound[warp][4 + i][lane] = u.hi[i];
        }
      }
      u.any = __syncthreads_or(u.any);
      if (threadIdx.x < kTeam) {
        for (int v = 1; v < kManyWarps; ++v)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            u.lo[i] = smaller<DT>(u.lo[i], s_bound[v][i][lane]);
            u.hi[i] = larger<DT>(u.hi[i], s_bound[v][4 + i][lane]);
          }
      }
    }
    if (team == 0) u.close(a, L);
    if (all) __syncthreads();  // s_bound is free again
  }
}

// Queries: the new rows of all requests, concatenated and cut into equal ranges, one
// per block; a team takes four heads of a row at a time.
template <int IN, bool INTER>
__device__ __forceinline__ void append_queries(const AppendArgs& a) {
  __shared__ Prefix<kManyThreads> S;
  const int team = threadIdx.x / kTeam, quads = (a.Hq + kQueryHeads - 1) / kQueryHeads;
  auto count = [&](int b) {
    int start, row0;
    return (long long)max(0, rows_of(a, b, start, row0)) * quads;
  };
  build_prefix<kManyThreads>(S, a.B, count);
  const long long total = S.pre[kManyThreads];
  const long long i0 = part_start(blockIdx.x, total, gridDim.x), i1 = part_start(blockIdx.x + 1, total, gridDim.x);
  long long at = i0 + team;
  if (at >= i1) return;
  const Lane L(a, threadIdx.x % kTeam);
  const long long left = i1 - at;
  int b = find_request<kManyThreads>(S, a.B, count, at);
  int start = 0, row0 = 0, n = rows_of(a, b, start, row0);
  int row, quad;  // of the request
  divide(at, quads, row, quad);
  for (long long i = 0; i < left; i += kManyThreads / kTeam) {
    while (row >= n && b < a.B - 1) {
      row -= max(n, 0);
      ++b;
      n = rows_of(a, b, start, row0);
    }
    const int t = start + row, page = a.table[(long long)b * a.max_pages + a.c.ps.div(t)];
    const int pos = a.positions != nullptr ? a.positions[row0 + row] : t;
    const bool ok = a.R == 0 || (pos >= 0 && pos < a.rope_positions);
    const char* from = a.q + (long long)(row0 + row) * a.q_stride + quad * (kQueryHeads * kD * 2);
    const int heads = min(kQueryHeads, a.Hq - quad * kQueryHeads);
    Raw x[kQueryHeads];
#pragma unroll
    for (int h = 0; h < kQueryHeads; ++h)
      if (h < heads) x[h] = load_raw(from + h * (kD * 2), L);
    Angles g;
    if (ok) g.load<INTER>(a, L, a.rope + (long long)pos * a.R);
    if (ok && page >= 0 && page < a.c.n_pages) {  // (the keys' kernel flags the others)
      char* to = a.q_out + (long long)(row0 + row) * a.q_out_stride + quad * (kQueryHeads * kD * 2);
#pragma unroll
      for (int h = 0; h < kQueryHeads; ++h) {
        if (h >= heads) continue;
        const Wide y = rotate<IN, INTER>(L, g, x[h]);
        store4<IN>(to + h * (kD * 2) + 2 * L.a, y.a);
        store4<IN>(to + h * (kD * 2) + 2 * L.b, y.b);
      }
    }
    quad += kManyThreads / kTeam;
    while (quad >= quads) {
      quad -= quads;
      ++row;
    }
  }
}

// Launched behind the keys' kernel, whose results it does not need: it starts once
// that one's blocks have all waited for what came before them (whose results are then
// in memory),
// and waits for it at its end, so that whoever waits for this kernel waits for both.
template <int IN, bool INTER>
__global__ void __launch_bounds__(kManyThreads, kQueryBlocksPerSm) append_queries_kernel(AppendArgs a) {
  allow_dependents();
  append_queries<IN, INTER>(a);
  wait_prior_grid();
}

template <int DT, int IN, bool INTER>
cudaError_t launch_form(const AppendArgs& a, int sms, cudaStream_t stream) {
  const int Hq = a.q != nullptr ? a.Hq : 0;
  count_launch();
  if (a.offsets == nullptr) {
    const long long need = ((long long)a.B * (a.c.H + Hq) * kTeam + kStepThreads - 1) / kStepThreads;
    const long long fit = (long long)kStepBlocksPerSm * sms;
    return launch_dependent(append_step_kernel<DT, IN, INTER>, dim3(int(need < fit ? need : fit)),
                            dim3(kStepThreads), 0, stream, a);
  }
  // More than two query heads per KV head: half as many blocks of each kernel, so that both fit on an SM and run side
  // by side; else the queries' blocks follow the keys' (4 x 2048 rows, pages of 64, side by side and one after the
  // other: 8 + 32 heads 37.3, 40.7 us, 8 + 24 33.9, 35.7, 16 + 32 55.7, 51.9, 32 + 32 92.6, 76.6; nine prompts of up to
  // 613 rows into 8-bit pages of 16, 8 + 32 heads 21.9, 24.6; a prompt of 2048 and 499 single rows 24.5, 22.6).
  const int part = Hq > 2 * a.c.H ? 2 : 1;
  // the keys' blocks: eight units each, or (pages of more rows than a warp takes) one unit of 32 rows
  const long long units = (a.n_rows / a.c.ps.d + 2 * (long long)a.B) * a.c.H;  // at most
  const long long by_units = (units + kManyWarps - 1) / kManyWarps;
  const long long by_rows = a.c.ps.d > kWarpRows ? (long long)a.n_rows * a.c.H / 32 : 0;
  const long long need = by_units > by_rows ? by_units : by_rows, fit = (long long)kKeyBlocksPerSm * sms / part;
  const cudaError_t e = launch_dependent(append_keys_kernel<DT, IN, INTER>, dim3(int(need < fit ? need : fit)),
                                         dim3(kManyThreads), 0, stream, a);
  if (e != cudaSuccess || Hq == 0) return e;
  count_launch();
  const long long teams = a.n_rows * (long long)((Hq + kQueryHeads - 1) / kQueryHeads), per = kManyThreads / kTeam;
  const long long blocks = (teams + per - 1) / per, most = (long long)kQueryBlocksPerSm * sms / part;
  return launch_dependent(append_queries_kernel<IN, INTER>, dim3(int(blocks < most ? blocks : most)),
                          dim3(kManyThreads), 0, stream, a);
}

template <int DT, int IN>
cudaError_t launch_types(const AppendArgs& a, int sms, cudaStream_t stream) {
  return a.interleaved ? launch_form<DT, IN, true>(a, sms, stream) : launch_form<DT, IN, false>(a, sms, stream);
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
