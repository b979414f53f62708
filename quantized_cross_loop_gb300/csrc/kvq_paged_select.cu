// kvq_paged_select.cu — the pages a query most likely finds something on.
//
// score(page) = sum_j sum_d (q_jd < 0 ? q_jd lo_d : q_jd hi_d), the sum over the
// group's query heads j of the largest q.k that the page's bounds allow. The sum
// over the heads goes into the query: score = sum_d up_d hi_d + down_d lo_d with
// up_d = sum_j max(q_jd, 0) and down_d = sum_j min(q_jd, 0): 256 products per page
// and KV head whatever the group is, on the 512 bytes of its two bounds. Bound: HBM.
//
// The score kernel reads each bound once, 16 bytes a lane, and leaves the scores
// as order-preserving 32-bit keys, and a bound A of every page's sum of absolute
// terms (from the largest magnitudes of each channel: cheaper than the pages' own
// sums). An FP32 score is off by at most E = (g + 17) u A, u = 2^-24: the weights are
// sums of g terms of one sign (g - 1 roundings), a lane adds up to 16 products in two
// chains (9), five additions join the lanes (5); four more cover A's and E's own
// rounding (A has no more than 30 roundings of 2^-24 each, nothing beside 4 / 33).
// Products below FP32's normal range are off by up to 2^-150 each whatever their size,
// 256 of them by 2^-142 (sums there are exact): 2E has 2^-140 more, twice as much as
// two scores need, which covers A's and E's own steps of 2^-150.
//
// The pick kernel finds the key t of the last page that FP32 would take, by
// histograms over the keys' range. Pages above t + 2E are in, those below t - 2E are
// out by the exact scores too; if the pages between are not all taken, they are
// scored again in FP64 (products of 11-bit significands summed in 53 bits) and
// ranked, ties by page number. Two pages scarcely ever are that near: the second
// scoring costs nothing as a rule, and the order is exact always.
#include <atomic>

#include "kvq_attn_common.cuh"
#include "kvq_paged.cuh"

namespace kvq {
namespace paged {
namespace {

constexpr int kScoreThreads = 256;
constexpr int kScoreWarps = kScoreThreads / 32;
constexpr int kChunk = 8;            // pages a warp scores at a time (E4M3: twice as many): 4 KB
constexpr int kStages = 3;           // chunks in a warp's ring
constexpr int kScoreBlocksPerSm = 2;  // by shared memory: 96 KB of rings
constexpr int kFusedThreads = kScoreThreads;
constexpr int kPickThreads = 1024;
constexpr int kMostWarps = kPickThreads / 32;
constexpr int kFew = 256;            // keys of a bin ranked by comparing each with all
constexpr int kWords = 1024;         // words of 32 pages of the output's bit map
constexpr int kStagedMax = 32 * kWords;  // pages whose keys are staged in shared memory
constexpr int kBins = 2048;
constexpr int kList = 1024;          // candidates ranked in shared memory
constexpr uint32_t kFirstKey = 0xFFFFFFFFu;  // a score that is not finite
constexpr uint32_t kLastKey = 0u;            // a page outside the pool

// Monotone map of finite floats to integers (-0 counts as +0), and back.
__device__ __forceinline__ uint32_t key_of(float x) {
  if (!isfinite(x)) return kFirstKey;
  const uint32_t u = __float_as_uint(x + 0.0f);
  return (u >> 31) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ float float_of(uint32_t k) { return __uint_as_float((k >> 31) ? k & 0x7FFFFFFFu : ~k); }
__device__ __forceinline__ uint64_t key_of(double x) {
  if (!isfinite(x)) return ~0ull;
  const uint64_t u = uint64_t(__double_as_longlong(x + 0.0));
  return (u >> 63) ? ~u : (u | (1ull << 63));
}

// All pages of a unit with no more than n_select, and -1 behind them; their numbers are looked at for the error bit, by
// one of the request's units.
__device__ __forceinline__ void take_all(const SelectArgs& a, int b, int h, int pages, int32_t* sel) {
  for (int i = threadIdx.x; i < a.n_select; i += blockDim.x) sel[i] = i < pages ? i : -1;
  if (h != 0 || a.c.err == nullptr) return;
  for (int i = threadIdx.x; i < pages; i += blockDim.x) {
    const int page = a.table[(long long)b * a.max_pages + i];
    if (page < 0 || page >= a.c.n_pages) flag(a.c, KVQ_PAGED_ERR_PAGE);
  }
}

struct Workspace {
  uint32_t* keys;   // [units][max_pages rounded up to 4]
  float* largest;   // [units][chunks]: A of the chunk
  uint64_t* exact;  // [units][max_pages], candidates only
};
constexpr size_t up16(size_t n) { return (n + 15) / 16 * 16; }
__host__ __device__ constexpr size_t key_stride(int max_pages) { return (size_t(max_pages) + 3) / 4 * 4; }
__host__ __device__ inline int chunks_of(int pages, int of) { return (pages + of - 1) / of; }
inline Workspace workspace_of(char* ws, int units, int max_pages) {
  Workspace w;
  w.keys = reinterpret_cast<uint32_t*>(ws);
  char* p = ws + size_t(units) * key_stride(max_pages) * 4;
  w.largest = reinterpret_cast<float*>(p);
  w.exact = reinterpret_cast<uint64_t*>(p + up16(size_t(units) * chunks_of(max_pages, kChunk) * 4));
  return w;
}

__device__ __forceinline__ int pages_of(const SelectArgs& a, int T) { return T <= 0 ? 0 : a.c.ps.div(T - 1) + 1; }

template <int DT>
__device__ __forceinline__ const char* bounds_of(const SelectArgs& a, int page, int h) {
  return a.c.bounds + ((long long)page * a.c.H + h) * (2 * kD * elem_bytes<DT>());
}

// A 16-byte load as pairs of 16-bit values (E4M3 as FP16, exact), a pair as FP32,
// and the larger magnitudes of two pairs.
template <int DT>
struct Pairs {
  static constexpr int kN = DT == kE4m3 ? 8 : 4;
  uint32_t w[kN];
  __device__ __forceinline__ explicit Pairs(const uint4& v) {
    const uint32_t x[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (DT == kE4m3) {
        w[2 * i] = e4m3x2_to_f16x2(x[i] & 0xFFFFu);
        w[2 * i + 1] = e4m3x2_to_f16x2(x[i] >> 16);
      } else {
        w[i] = x[i];
      }
    }
  }
};
template <int DT>
__device__ __forceinline__ float2 pair_floats(uint32_t w) {
  if constexpr (DT == kBf16) return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
  return __half22float2(*reinterpret_cast<const __half2*>(&w));
}
template <int DT>
__device__ __forceinline__ uint32_t larger_magnitudes(uint32_t most, uint32_t w) {
  if constexpr (DT == kBf16) {
    const __nv_bfloat162 r = __hmax2(*reinterpret_cast<const __nv_bfloat162*>(&most),
                                     __habs2(*reinterpret_cast<const __nv_bfloat162*>(&w)));
    return *reinterpret_cast<const uint32_t*>(&r);
  } else {
    const __half2 r = __hmax2(*reinterpret_cast<const __half2*>(&most), __habs2(*reinterpret_cast<const __half2*>(&w)));
    return *reinterpret_cast<const uint32_t*>(&r);
  }
}

__device__ __forceinline__ void copy16(uint32_t dst, const char* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void wait_groups() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// A warp scores a chunk of pages at a time, from a ring of its own that 16-byte
// asynchronous copies fill, so that two chunks are on their way without registers. A
// page's bounds are 32 (16-bit) or 16 (E4M3) pieces of 16 bytes; a lane holds the
// weights of its own 8 or 16 channels of lo or hi and reads only what it copied itself.
template <int DT, int QT>
struct Scorer {
  static constexpr int kPer = DT == kE4m3 ? 16 : 8;      // channels of a lane
  static constexpr int kLanes = 2 * kD / kPer;           // lanes of a page
  static constexpr int kAtOnce = 32 / kLanes;            // pages per copy of the warp
  static constexpr int kPages = kChunk * kAtOnce;        // pages of a chunk
  static constexpr int kLoads = kChunk;
  static constexpr int kPairs = kPer / 2;
  float2 w[kPairs];
  uint32_t most[kPairs];  // largest magnitudes seen in the lane's channels

  __device__ __forceinline__ void weights(const SelectArgs& a, int b, int h, int lane) {
    const int sub = lane % kLanes, at = sub % (kLanes / 2) * kPer;
    const bool up = sub >= kLanes / 2;
#pragma unroll
    for (int e = 0; e < kPairs; ++e) {
      w[e] = make_float2(0.0f, 0.0f);
      most[e] = 0u;
    }
    const char* q = a.q + (long long)b * a.q_stride + ((long long)h * a.g * kD + at) * 2;
#pragma unroll 4
    for (int j = 0; j < a.g; ++j) {
#pragma unroll
      for (int e = 0; e < kPairs; e += 4) {
        const Pairs<QT> x(__ldg(reinterpret_cast<const uint4*>(q + (j * kD + 2 * e) * 2)));
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 y = pair_floats<QT>(x.w[i]);
          w[e + i].x += (y.x < 0.0f) == up ? 0.0f : y.x;
          w[e + i].y += (y.y < 0.0f) == up ? 0.0f : y.y;
        }
      }
    }
  }

  // A of the pages seen since weights(): no page's sum of absolute terms is larger (each channel's largest magnitude
  // counts, whichever pages they come from); the sum over the warp.
  __device__ __forceinline__ float bound() const {
    float t = 0.0f;
#pragma unroll
    for (int e = 0; e < kPairs; ++e) {
      const float2 x = pair_floats<DT>(most[e]);
      t = fmaf(fabsf(w[e].x), x.x, t);
      t = fmaf(fabsf(w[e].y), x.y, t);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) t += __shfl_xor_sync(0xFFFFFFFFu, t, o);
    return t < INFINITY ? t : INFINITY;  // (0 * inf: no bound either, and a NaN would be lost among the others)
  }

  // Page numbers of the chunk from page p0 on, one in each of kPages lanes (behind the last: the last, whose bounds A
  // has to cover anyway).
  __device__ __forceinline__ static int ids(const SelectArgs& a, int b, int p0, int pages, int lane) {
    return a.table[(long long)b * a.max_pages + min(p0 + (lane & (kPages - 1)), pages - 1)];
  }

  // Copies of the bounds of the pages `ids` into the lane's place of a stage. Returns the lanes whose page is outside
  // the pool.
  __device__ __forceinline__ static uint32_t issue(const SelectArgs& a, int h, int ids, int lane, uint32_t stage) {
    const bool ok = ids >= 0 && ids < a.c.n_pages;
    if (!ok) flag(a.c, KVQ_PAGED_ERR_PAGE);
    const int page = ok ? ids : 0;
    const char* base = bounds_of<DT>(a, 0, h) + 16 * (lane % kLanes);
    const int stride = a.c.H * (2 * kD * elem_bytes<DT>());  // of a page (H <= 1024)
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int id = __shfl_sync(0xFFFFFFFFu, page, i * kAtOnce + lane / kLanes);
      copy16(stage + i * 512 + lane * 16, base + (long long)id * stride);
    }
    return __ballot_sync(0xFFFFFFFFu, !ok);
  }

  // Scores of a stage's chunk: the key of its page `index` in each lane.
  __device__ __forceinline__ uint32_t score(uint32_t stage, uint32_t outside, int lane, int& index) {
    float v[kLoads];
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      uint4 r;
      asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                   : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
                   : "r"(stage + i * 512 + lane * 16));
      const Pairs<DT> x(r);
      float2 s = make_float2(0.0f, 0.0f);
#pragma unroll
      for (int e = 0; e < kPairs; ++e) {
        s = __ffma2_rn(w[e], pair_floats<DT>(x.w[e]), s);
        most[e] = larger_magnitudes<DT>(most[e], x.w[e]);
      }
      v[i] = s.x + s.y;
    }
    // sums over the lanes of a page: halves of the values change sides with halves of the lanes while there are any
    int n = kLoads, load = 0;
#pragma unroll
    for (int o = kLanes / 2; o >= 1; o >>= 1) {
      const bool hi = (lane & o) != 0;
      if (n > 1) {
        n /= 2;
#pragma unroll
        for (int k = 0; k < kLoads / 2; ++k) {
          if (k >= n) break;
          const float send = hi ? v[k] : v[k + n], keep = hi ? v[k + n] : v[k];
          v[k] = keep + __shfl_xor_sync(0xFFFFFFFFu, send, o);
        }
        load += hi ? n : 0;
      } else {
        v[0] += __shfl_xor_sync(0xFFFFFFFFu, v[0], o);
      }
    }
    index = load * kAtOnce + lane / kLanes;
    return (outside >> index) & 1 ? kLastKey : key_of(v[0]);
  }
};

constexpr int kRing = kStages * kChunk * 512;  // bytes per warp

template <int DT, int QT>
__global__ void __launch_bounds__(kScoreThreads, kScoreBlocksPerSm) score_kernel(SelectArgs a, Workspace ws) {
  __shared__ Prefix<kScoreThreads> S;
  extern __shared__ __align__(16) char s_ring[];
  wait_prior_grid();
  allow_dependents();
  auto count = [&](int b) {
    const int pages = pages_of(a, checked_len(a.lens, b, a.max_pages, a.c.ps));
    return pages <= a.n_select ? 0LL : (long long)chunks_of(pages, Scorer<DT, QT>::kPages);  // all taken: nothing to score
  };
  build_prefix<kScoreThreads>(S, a.B, count);
  if (a.c.err != nullptr && blockIdx.x == 0)
    for (int b = threadIdx.x; b < a.B; b += kScoreThreads)
      if (checked_len(a.lens, b, a.max_pages, a.c.ps) < 0) flag(a.c, KVQ_PAGED_ERR_LENGTH);
  // H warps side by side take the heads of the same pages, whose bounds lie side by side: a group of H warps has a
  // range of the chunks of all requests
  const int lane = threadIdx.x & 31;
  const long long total = S.pre[kScoreThreads];
  const int groups = int(gridDim.x) * kScoreWarps / a.c.H;
  const int me = int(blockIdx.x) * kScoreWarps + threadIdx.x / 32, group = me / a.c.H, h = me % a.c.H;
  if (group >= groups) return;
  const long long c0 = part_start(group, total, groups), c1 = part_start(group + 1, total, groups);
  if (c0 >= c1) return;
  long long at = c0;
  const int b = find_request<kScoreThreads>(S, a.B, count, at);
  const int pages = pages_of(a, checked_len(a.lens, b, a.max_pages, a.c.ps));
  using K = Scorer<DT, QT>;
  K score;
  // the chunk being scored (b, chunk) and the one whose pages are looked up next; a chunk's page numbers are loaded
  // one step ahead of its copies, its copies issued two steps ahead of its score
  struct Place {
    int b, chunk, pages, chunks;
  };
  auto next = [&](Place& p) {
    if (++p.chunk < p.chunks) return;
    p.chunk = 0;
    for (++p.b; p.b < a.B; ++p.b) {
      p.pages = pages_of(a, checked_len(a.lens, p.b, a.max_pages, a.c.ps));
      p.chunks = chunks_of(p.pages, K::kPages);
      if (p.pages > a.n_select) return;
    }
  };
  Place now{b, int(at), pages, chunks_of(pages, K::kPages)}, ahead = now;
  const uint32_t ring = uint32_t(__cvta_generic_to_shared(s_ring)) + (threadIdx.x / 32) * kRing;
  const int n = int(c1 - c0);
  int ids = K::ids(a, ahead.b, ahead.chunk * K::kPages, ahead.pages, lane);
  uint32_t outside[kStages] = {};
  auto fill = [&](int i, int stage) {  // chunk i of the range, if there is one
    uint32_t bad = 0;
    if (i < n) {
      bad = K::issue(a, h, ids, lane, ring + stage * (kChunk * 512));
      next(ahead);
      if (i + 1 < n) ids = K::ids(a, ahead.b, ahead.chunk * K::kPages, ahead.pages, lane);
    }
    commit();
    return bad;
  };
#pragma unroll
  for (int i = 0; i < kStages - 1; ++i) outside[i] = fill(i, i);
  score.weights(a, now.b, h, lane);
  for (int i0 = 0; i0 < n; i0 += kStages) {
#pragma unroll
    for (int e = 0; e < kStages; ++e) {
      const int i = i0 + e;
      if (i >= n) break;
      wait_groups<kStages - 2>();
      outside[(e + kStages - 1) % kStages] = fill(i + kStages - 1, (e + kStages - 1) % kStages);
      const long long unit = (long long)now.b * a.c.H + h;
      int index;
      const uint32_t key = score.score(ring + e * (kChunk * 512), outside[e], lane, index);
      const int p = now.chunk * K::kPages + index;
      if (p < now.pages) ws.keys[unit * key_stride(a.max_pages) + p] = key;
      // the warp's last chunk of the unit stands for those before
      const bool last = now.chunk + 1 == now.chunks || i + 1 == n;
      const float largest = last ? score.bound() : 0.0f;
      if (lane == 0) ws.largest[unit * chunks_of(a.max_pages, kChunk) + now.chunk] = largest;
      next(now);
      if (last && i + 1 < n) score.weights(a, now.b, h, lane);
    }
  }
}

struct Pick {
  int hist[kBins];
  alignas(16) uint32_t list_key[kList];
  uint64_t list_exact[kList];
  int list_page[kList];
  double up[kD], down[kD];
  uint32_t words[kWords];
  int warp_sum[kMostWarps];
  uint32_t warp_lo[kMostWarps], warp_hi[kMostWarps];
  float warp_a[kMostWarps];
  int n_list, left, above, bin, members;
  uint32_t t;
  uint64_t prefix;
};

// Sum over the block, and over the threads before this one.
template <int THREADS>
__device__ __forceinline__ int block_prefix(Pick& S, int x, int& before) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int y = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int z = __shfl_up_sync(0xFFFFFFFFu, y, o);
    if (lane >= o) y += z;
  }
  __syncthreads();
  if (lane == 31) S.warp_sum[warp] = y;
  __syncthreads();
  // every warp sums the warps' totals by itself
  int t = lane < THREADS / 32 ? S.warp_sum[lane] : 0, v = t;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int z = __shfl_up_sync(0xFFFFFFFFu, v, o);
    if (lane >= o) v += z;
  }
  before = y - x + __shfl_sync(0xFFFFFFFFu, v - t, warp);
  return __shfl_sync(0xFFFFFFFFu, v, 31);
}

// Exact score of a page by a warp.
template <int DT>
__device__ __forceinline__ uint64_t exact_key(const SelectArgs& a, const Pick& S, int b, int h, int p, int lane) {
  const int page = a.table[(long long)b * a.max_pages + p];
  if (page < 0 || page >= a.c.n_pages) return 0;
  const char* at = bounds_of<DT>(a, page, h) + 4 * lane * elem_bytes<DT>();
  const float4 lo = load4<DT>(at), hi = load4<DT>(at + kD * elem_bytes<DT>());
  const double *d = &S.down[4 * lane], *u = &S.up[4 * lane];
  double x = d[0] * lo.x + d[1] * lo.y + d[2] * lo.z + d[3] * lo.w;
  x += u[0] * hi.x + u[1] * hi.y + u[2] * hi.z + u[3] * hi.w;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xFFFFFFFFu, x, o);
  return key_of(x);
}

// Writes the pages p < pages <= 32 kWords with taken(p), base added, in order behind the `*out` that are there, by a
// bit map whose words are shared out among the threads. Without `out` only if they are n_select; returns whether.
template <int THREADS, typename F>
__device__ __forceinline__ bool emit(const SelectArgs& a, Pick& S, int pages, int32_t* sel, const F& taken, int base = 0,
                                     int* out = nullptr) {
  const int tid = threadIdx.x, lane = tid & 31, words = (pages + 31) / 32;
  __syncthreads();
#pragma unroll 4
  for (int w = tid / 32; w < words; w += THREADS / 32) {
    const int p = 32 * w + lane;
    const uint32_t m = __ballot_sync(0xFFFFFFFFu, p < pages && taken(p));
    if (lane == 0) S.words[w] = m;
  }
  __syncthreads();
  if (words <= 32) {  // every warp sums the words' counts by itself and writes the pages of the words it made
    const int own = lane < words ? __popc(S.words[lane]) : 0;
    int sum = own;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(0xFFFFFFFFu, sum, o);
      if (lane >= o) sum += x;
    }
    const int all = __shfl_sync(0xFFFFFFFFu, sum, 31), first = out != nullptr ? *out : 0;
    if (out == nullptr && all != a.n_select) return false;
    for (int w = tid / 32; w < words; w += THREADS / 32) {
      const uint32_t m = S.words[w];
      const int i = first + __shfl_sync(0xFFFFFFFFu, sum - own, w) + __popc(m & ((1u << lane) - 1u));
      if (((m >> lane) & 1) && i < a.n_select) sel[i] = base + 32 * w + lane;
    }
    if (out != nullptr) *out += all;
    return true;
  }
  constexpr int kOwn = (kWords + THREADS - 1) / THREADS;  // words of a thread
  uint32_t m[kOwn];
  int n = 0, before;
#pragma unroll
  for (int e = 0; e < kOwn; ++e) {
    m[e] = kOwn * tid + e < words ? S.words[kOwn * tid + e] : 0u;
    n += __popc(m[e]);
  }
  const int all = block_prefix<THREADS>(S, n, before);
  if (out == nullptr && all != a.n_select) return false;
  int i = (out != nullptr ? *out : 0) + before;
#pragma unroll
  for (int e = 0; e < kOwn; ++e)
    for (uint32_t x = m[e]; x != 0 && i < a.n_select; ++i, x &= x - 1)
      sel[i] = base + 32 * (kOwn * tid + e) + __ffs(x) - 1;
  if (out != nullptr) *out += all;
  return true;
}

// The `left`-th largest of n <= kFew keys: the smallest with fewer than `left` above it.
__device__ __forceinline__ uint32_t ranked(Pick& S, const uint32_t* keys, int n, int left) {
  if (threadIdx.x == 0) S.t = 0xFFFFFFFFu;
  __syncthreads();
  uint32_t best = 0xFFFFFFFFu;
  if ((threadIdx.x & ~31) < n) {
    const uint32_t x = threadIdx.x < n ? keys[threadIdx.x] : 0u;
    int more = 0;
#pragma unroll 8
    for (int i = 0; i < n; ++i) more += keys[i] > x;
    if (threadIdx.x < n && more < left) best = x;
    best = __reduce_min_sync(0xFFFFFFFFu, best);
    if ((threadIdx.x & 31) == 0 && best != 0xFFFFFFFFu) atomicMin(&S.t, best);
  }
  __syncthreads();
  return S.t;
}

// The same of up to 32 keys, by each warp for itself.
__device__ __forceinline__ uint32_t warp_ranked(const uint32_t* keys, int n, int left) {
  const int lane = threadIdx.x & 31;
  const uint32_t x = lane < n ? keys[lane] : 0u;
  int more = 0;
  for (int i = 0; i < n; ++i) more += __shfl_sync(0xFFFFFFFFu, x, i) > x;
  return __reduce_min_sync(0xFFFFFFFFu, lane < n && more < left ? x : 0xFFFFFFFFu);
}

// The same of up to kFew keys, by a warp, bit by bit. As many pages need no histogram (the k-th largest of 256 keys
// this way and the words of emit by each warp: 8 units 6.8 us instead of 7.4, 256 units 12.1 instead of 12.9).
__device__ __forceinline__ uint32_t bitwise_ranked(const uint32_t* keys, int n, int left) {
  constexpr int kOwn = kFew / 32;
  const int lane = threadIdx.x & 31;
  uint32_t x[kOwn], lo = 0xFFFFFFFFu, hi = 0u;
#pragma unroll
  for (int e = 0; e < kOwn; ++e) {
    const bool in = 32 * e + lane < n;
    x[e] = in ? keys[32 * e + lane] : 0u;
    if (in) lo = min(lo, x[e]);
    hi = max(hi, x[e]);
  }
  lo = __reduce_min_sync(0xFFFFFFFFu, lo);
  hi = __reduce_max_sync(0xFFFFFFFFu, hi);
#pragma unroll
  for (int e = 0; e < kOwn; ++e) x[e] = max(x[e], lo) - lo;
  uint32_t t = 0;  // the largest with `left` keys that are no smaller
  for (int bit = 31 - __clz(hi - lo); bit >= 0; --bit) {
    const uint32_t y = t | (1u << bit);
    int more = 0;
#pragma unroll
    for (int e = 0; e < kOwn; ++e) more += x[e] >= y;
    if (__reduce_add_sync(0xFFFFFFFFu, more) >= left) t = y;
  }
  return lo + t;
}

// Picks a unit's pages from its keys (`keys` is scratch: written, too); the block's threads together.
// lo and hi are the range of some of the keys that may be chosen, over the block of all.
template <int DT, int QT, int THREADS>
__device__ __forceinline__ void pick(const SelectArgs& a, Pick& S, int b, int h, int pages, uint32_t* keys,
                                     float largest, uint32_t lo, uint32_t hi, uint64_t* exact, int32_t* sel) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int f0 = a.n_first, f1 = pages - a.n_last;  // pages before f0 and from f1 on are taken anyway
  const int k = a.n_select - a.n_first - a.n_last;
  if (k == 0) {
    hi = kFirstKey;
    __syncthreads();
    for (int p = f0 + tid; p < f1; p += THREADS) keys[p] = kLastKey;  // none but those
    __syncthreads();
  } else {
    uint32_t t;
    if (f1 - f0 <= kFew) {
      if (warp == 0) {
        t = bitwise_ranked(keys + f0, f1 - f0, k);
        if (lane == 0) S.t = t;
      }
      __syncthreads();
      t = S.t;
    } else {
      lo = __reduce_min_sync(0xFFFFFFFFu, lo);
      hi = __reduce_max_sync(0xFFFFFFFFu, hi);
      if (lane == 0) {
        S.warp_lo[warp] = lo;
        S.warp_hi[warp] = hi;
      }
      for (int i = tid; i < kBins; i += THREADS) S.hist[i] = 0;
      if (tid == 0) S.n_list = 0;
      __syncthreads();  // (also: the keys are there)
      lo = __reduce_min_sync(0xFFFFFFFFu, lane < THREADS / 32 ? S.warp_lo[lane] : 0xFFFFFFFFu);
      hi = __reduce_max_sync(0xFFFFFFFFu, lane < THREADS / 32 ? S.warp_hi[lane] : 0u);
      // the k-th largest key
      int left = k;
      t = lo;
      while (lo < hi) {
        const int bits = 32 - __clz(hi - lo), shift = bits > 11 ? bits - 11 : 0;
#pragma unroll 4
        for (int p = f0 + tid; p < f1; p += THREADS) {
          const uint32_t x = keys[p];
          if (x >= lo && x <= hi) atomicAdd(&S.hist[(x - lo) >> shift], 1);
        }
        __syncthreads();
        {  // bins from the top: thread i holds the kOwn bins below kBins - kOwn i
          constexpr int kOwn = kBins / THREADS;
          int own[kOwn], n = 0, before;
#pragma unroll
          for (int e = 0; e < kOwn; ++e) {
            own[e] = S.hist[kBins - 1 - kOwn * tid - e];
            n += own[e];
          }
          block_prefix<THREADS>(S, n, before);
#pragma unroll
          for (int e = 0; e < kOwn; ++e) {
            if (before < left && left <= before + own[e]) {  // one thread, one bin
              S.bin = kBins - 1 - kOwn * tid - e;
              S.above = before;
              S.members = own[e];
            }
            before += own[e];
          }
          __syncthreads();
        }
        left -= S.above;
        lo += uint32_t(S.bin) << shift;
        if (shift == 0) hi = lo;
        else hi = min(hi, lo + ((1u << shift) - 1u));
        t = lo;
        const int members = S.members;
        if (lo < hi && members <= kFew) {
#pragma unroll 4
          for (int p = f0 + tid; p < f1; p += THREADS) {
            const uint32_t x = keys[p];
            if (x >= lo && x <= hi) S.list_key[atomicAdd(&S.n_list, 1)] = x;
          }
          __syncthreads();
          t = members <= 32 ? warp_ranked(S.list_key, members, left) : ranked(S, S.list_key, members, left);
          break;
        }
        __syncthreads();  // hist, bin and list are free again
        for (int i = tid; i < kBins; i += THREADS) S.hist[i] = 0;
        __syncthreads();
      }
    }
    // pages in doubt
    lo = hi = t;
    if (t != kFirstKey && t != kLastKey) {
      const float x = float_of(t), e = fmaf(2.0f * (float(a.g + 17) * 0x1p-24f), largest, 0x1p-140f);
      const float x0 = __fsub_rd(x, e), x1 = __fadd_ru(x, e);
      lo = x0 >= -3.4e38f ? key_of(x0) : key_of(-3.402823466e38f);
      hi = x1 <= 3.4e38f ? key_of(x1) : kFirstKey - 1u;
    }
    // as a rule the pages from the window's lower end on are as many as are wanted: written in order at once
    if (pages <= 32 * kWords && emit<THREADS>(a, S, pages, sel, [&](int p) { return p < f0 || p >= f1 || keys[p] >= lo; }))
      return;
    // the others: counted, the pages in doubt listed
    if (tid == 0) S.n_list = S.left = 0;
    __syncthreads();
    int n_above = 0;
    for (int p = f0 + tid; p < f1; p += THREADS) {
      const uint32_t x = keys[p];
      n_above += x > hi;
      if (x >= lo && x <= hi) {
        const int i = atomicAdd(&S.n_list, 1);
        if (i < kList) S.list_page[i] = p;
      }
    }
    n_above = __reduce_add_sync(0xFFFFFFFFu, n_above);
    if (lane == 0 && n_above != 0) atomicAdd(&S.left, n_above);
    if (tid < kD) {
      double up = 0.0, down = 0.0;
#pragma unroll 8
      for (int j = 0; j < a.g; ++j) {
        const uint16_t v = *reinterpret_cast<const uint16_t*>(a.q + (long long)b * a.q_stride +
                                                              ((long long)(h * a.g + j) * kD + tid) * 2);
        const float x = QT == kBf16 ? bf16_bits_to_f32(v) : f16_bits_to_f32(v);
        if (x < 0.0f) down += x;
        else up += x;
      }
      S.up[tid] = up;
      S.down[tid] = down;
    }
    __syncthreads();
    const int want = k - S.left, n_in = S.n_list;
    if (want == n_in) {  // (pages beyond the bit map)
      for (int p = f0 + tid; p < f1; p += THREADS)
        if (keys[p] >= lo && keys[p] <= hi) keys[p] = kFirstKey;
      __syncthreads();
    } else {
      if (n_in <= kList) {
        for (int i = warp; i < n_in; i += (THREADS / 32)) {
          const uint64_t x = exact_key<DT>(a, S, b, h, S.list_page[i], lane);
          if (lane == 0) S.list_exact[i] = x;
        }
        __syncthreads();
        for (int i = tid; i < n_in; i += THREADS) {
          const uint64_t x = S.list_exact[i];
          const int p = S.list_page[i];
          int rank = 0;
          for (int j = 0; j < n_in; ++j) rank += S.list_exact[j] > x || (S.list_exact[j] == x && S.list_page[j] < p);
          keys[p] = rank < want ? kFirstKey : kLastKey;
        }
      } else {  // many pages score the same, or nearly: a radix selection over the exact keys
        for (int p = f0 + warp; p < f1; p += (THREADS / 32)) {
          if (keys[p] < lo || keys[p] > hi) continue;
          const uint64_t x = exact_key<DT>(a, S, b, h, p, lane);
          if (lane == 0) exact[p] = x;
        }
        __syncthreads();
        uint64_t prefix = 0, mask = 0;
        int rest = want;  // still to take among the keys that match the prefix
        for (int shift = 56; shift >= 0; shift -= 8) {
          if (tid < 256) S.hist[tid] = 0;
          __syncthreads();
          for (int p = f0 + tid; p < f1; p += THREADS)
            if (keys[p] >= lo && keys[p] <= hi && (exact[p] & mask) == prefix)
              atomicAdd(&S.hist[int((exact[p] >> shift) & 255)], 1);
          __syncthreads();
          if (tid == 0) {
            int bin = 255, n = rest;
            while (bin > 0 && S.hist[bin] < n) n -= S.hist[bin--];
            S.prefix = prefix | (uint64_t(bin) << shift);
            S.left = n;
          }
          __syncthreads();
          prefix = S.prefix;
          rest = S.left;
          mask |= 255ull << shift;
          __syncthreads();
        }
        // above the prefix: in; equal: the first `rest` by page number (warps take runs of 32 pages in order)
        int seen = 0;
        for (int p0 = f0; p0 < f1; p0 += THREADS) {
          const int p = p0 + tid;
          const bool in = p < f1 && keys[p] >= lo && keys[p] <= hi;
          const uint64_t x = in ? exact[p] : 0;
          const bool same = in && x == prefix;
          const uint32_t m = __ballot_sync(0xFFFFFFFFu, same);
          if (lane == 0) S.warp_sum[warp] = __popc(m);
          __syncthreads();
          int rank = seen + __popc(m & ((1u << lane) - 1u));
          for (int w = 0; w < (THREADS / 32); ++w) {
            if (w < warp) rank += S.warp_sum[w];
            seen += S.warp_sum[w];
          }
          if (in) keys[p] = x > prefix || (same && rank < rest) ? kFirstKey : kLastKey;
          __syncthreads();
        }
      }
      __syncthreads();
    }
  }
  int out = 0;
  for (int base = 0; base < pages; base += 32 * kWords)  // (as many as the bit map holds at a time)
    emit<THREADS>(a, S, min(pages - base, 32 * kWords), sel, [&](int i) {
      const int p = base + i;
      return p < f0 || p >= f1 || keys[p] > hi || keys[p] == kFirstKey;
    }, base, &out);
}

template <int DT, int QT>
__global__ void __launch_bounds__(kPickThreads) pick_kernel(SelectArgs a, Workspace ws, int staged) {
  __shared__ Pick S;
  extern __shared__ __align__(16) uint32_t s_keys[];
  wait_prior_grid();
  allow_dependents();
  const long long unit = blockIdx.x;
  const int b = int(blockIdx.x) / a.c.H, h = int(blockIdx.x) % a.c.H, tid = threadIdx.x;
  const int pages = pages_of(a, checked_len(a.lens, b, a.max_pages, a.c.ps));
  int32_t* sel = a.sel + unit * a.n_select;
  if (pages <= a.n_select) return take_all(a, b, h, pages, sel);
  uint32_t* keys = ws.keys + unit * key_stride(a.max_pages);
  const float* l = ws.largest + unit * chunks_of(a.max_pages, kChunk);
  const int chunks = chunks_of(pages, Scorer<DT, QT>::kPages);
  float largest = tid < chunks ? l[tid] : 0.0f;
  uint32_t lo = 0xFFFFFFFFu, hi = 0u;
  const int f0 = a.n_first, f1 = pages - a.n_last;
#pragma unroll 2
  for (int p = 4 * tid; p < pages; p += 4 * kPickThreads) {
    const uint4 x = *reinterpret_cast<const uint4*>(keys + p);
    const uint32_t y[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (p + e >= f0 && p + e < f1) {
        lo = min(lo, y[e]);
        hi = max(hi, y[e]);
      }
    if (staged) *reinterpret_cast<uint4*>(s_keys + p) = x;
  }
  if (staged) keys = s_keys;
  for (int i = tid + kPickThreads; i < chunks; i += kPickThreads) largest = fmaxf(largest, l[i]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) largest = fmaxf(largest, __shfl_xor_sync(0xFFFFFFFFu, largest, o));
  if ((tid & 31) == 0) S.warp_a[tid >> 5] = largest;
  __syncthreads();
  for (int w = 0; w < kMostWarps; ++w) largest = fmaxf(largest, S.warp_a[w]);
  pick<DT, QT, kPickThreads>(a, S, b, h, pages, keys, largest, lo, hi, ws.exact + unit * a.max_pages, sel);
}

// Both in one: a block scores and picks a unit's pages, the keys in shared memory.
template <int DT, int QT>
__global__ void __launch_bounds__(kFusedThreads, 2) select_kernel(SelectArgs a, Workspace ws) {
  extern __shared__ __align__(16) char s_ring[];  // the rings, and in their place the pick's memory; then the keys
  Pick& S = *reinterpret_cast<Pick*>(s_ring);
  wait_prior_grid();
  allow_dependents();
  const long long unit = blockIdx.x;
  const int b = int(blockIdx.x) / a.c.H, h = int(blockIdx.x) % a.c.H, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int T = checked_len(a.lens, b, a.max_pages, a.c.ps), pages = pages_of(a, T);
  if (T < 0 && tid == 0) flag(a.c, KVQ_PAGED_ERR_LENGTH);
  int32_t* sel = a.sel + unit * a.n_select;
  if (pages <= a.n_select) return take_all(a, b, h, pages, sel);
  using K = Scorer<DT, QT>;
  K score;
  static_assert(sizeof(Pick) <= kScoreWarps * kRing, "the pick's memory takes the rings' place");
  const uint32_t ring = uint32_t(__cvta_generic_to_shared(s_ring)) + warp * kRing;
  uint32_t* keys = reinterpret_cast<uint32_t*>(s_ring + kScoreWarps * kRing);
  uint32_t lo = 0xFFFFFFFFu, hi = 0u;
  const int chunks = chunks_of(pages, K::kPages), n = chunks > warp ? (chunks - warp + kScoreWarps - 1) / kScoreWarps : 0;
  int ids = K::ids(a, b, warp * K::kPages, pages, lane);
  uint32_t outside[kStages] = {};
  auto fill = [&](int i, int stage) {  // the warp's i-th chunk, if there is one
    uint32_t bad = 0;
    if (i < n) {
      bad = K::issue(a, h, ids, lane, ring + stage * (kChunk * 512));
      if (i + 1 < n) ids = K::ids(a, b, (warp + (i + 1) * kScoreWarps) * K::kPages, pages, lane);
    }
    commit();
    return bad;
  };
#pragma unroll
  for (int i = 0; i < kStages - 1; ++i) outside[i] = fill(i, i);
  score.weights(a, b, h, lane);
  for (int i0 = 0; i0 < n; i0 += kStages) {
#pragma unroll
    for (int e = 0; e < kStages; ++e) {
      const int i = i0 + e;
      if (i >= n) break;
      wait_groups<kStages - 2>();
      outside[(e + kStages - 1) % kStages] = fill(i + kStages - 1, (e + kStages - 1) % kStages);
      int index;
      const uint32_t key = score.score(ring + e * (kChunk * 512), outside[e], lane, index);
      const int p = (warp + i * kScoreWarps) * K::kPages + index;
      if (p < pages) keys[p] = key;
      if (p >= a.n_first && p < pages - a.n_last) {
        lo = min(lo, key);
        hi = max(hi, key);
      }
    }
  }
  float largest = score.bound();
  wait_groups<0>();
  __syncthreads();  // nobody's ring is in use
  if (lane == 0) S.warp_a[warp] = largest;
  __syncthreads();
  for (int w = 0; w < (kFusedThreads / 32); ++w) largest = fmaxf(largest, S.warp_a[w]);
  pick<DT, QT, kFusedThreads>(a, S, b, h, pages, keys, largest, lo, hi, ws.exact + unit * a.max_pages, sel);
}

// One launch where a unit's pages keep a block busy for no longer than the second
// launch takes, or where there are units for half of the SMs; else the pages are
// scored by all warps of the device and picked by a second kernel. Measured (fused,
// split): 8 units of 256 pages 6.8, 9.4 us; 8 of 512 10.2, 10.8; 64 of 1024 20.5,
// 20.5; 64 of 2048 33.8, 27.6; 128 of 1024 22.3, 25.9; 256 of 2048 51, 71.
constexpr int kFusedPages = 512;       // any number of units
constexpr int kFusedManyPages = 2048;  // half as many units as SMs at least

template <int DT, int QT>
cudaError_t launch_types(const SelectArgs& a, cudaStream_t stream) {
  const int units = a.B * a.c.H;
  const Workspace ws = workspace_of(a.ws, units, a.max_pages);
  const int staged = a.max_pages <= kStagedMax;
  const size_t smem = staged ? key_stride(a.max_pages) * 4 : 0;
  constexpr int ring = kScoreWarps * kRing;
  static std::atomic<uint64_t> configured{0};  // bit: device
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (!((configured.load(std::memory_order_relaxed) >> dev) & 1)) {
    e = cudaFuncSetAttribute(select_kernel<DT, QT>, cudaFuncAttributeMaxDynamicSharedMemorySize, ring + kFusedManyPages * 4);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(score_kernel<DT, QT>, cudaFuncAttributeMaxDynamicSharedMemorySize, ring);
    if (e == cudaSuccess)  // (more than 48 KB with the static part)
      e = cudaFuncSetAttribute(pick_kernel<DT, QT>, cudaFuncAttributeMaxDynamicSharedMemorySize, kStagedMax * 4);
    if (e != cudaSuccess) return e;
    configured.fetch_or(uint64_t(1) << dev, std::memory_order_relaxed);
  }
  if (a.max_pages <= kFusedPages || (a.max_pages <= kFusedManyPages && 2 * units >= a.sms)) {
    count_launch();
    return launch_dependent(select_kernel<DT, QT>, dim3(units), dim3(kFusedThreads), ring + smem, stream, a, ws);
  }
  const long long warps = (long long)units * chunks_of(a.max_pages, Scorer<DT, QT>::kPages);  // at most
  const long long need = (warps + kScoreWarps - 1) / kScoreWarps, fit = (long long)kScoreBlocksPerSm * a.sms;
  const long long least = (a.c.H + kScoreWarps - 1) / kScoreWarps;  // one group of H warps
  const int blocks = int(need < least ? least : need < fit || fit < least ? need : fit);
  count_launch();
  e = launch_dependent(score_kernel<DT, QT>, dim3(blocks), dim3(kScoreThreads), ring, stream, a, ws);
  if (e != cudaSuccess) return e;
  count_launch();
  return launch_dependent(pick_kernel<DT, QT>, dim3(units), dim3(kPickThreads), smem, stream, a, ws, staged);
}

}  // namespace

size_t select_workspace(int B, int H, int max_pages) {
  const size_t units = size_t(B) * H;
  return units * key_stride(max_pages) * 4 + up16(units * chunks_of(max_pages, kChunk) * 4) + up16(units * max_pages * 8);
}

cudaError_t launch_select(const SelectArgs& a, cudaStream_t stream) {
  const bool bf = a.q_dtype == kBf16;
  if (a.dtype == kBf16) return launch_types<kBf16, kBf16>(a, stream);
  if (a.dtype == kFp16) return launch_types<kFp16, kFp16>(a, stream);
  return bf ? launch_types<kE4m3, kBf16>(a, stream) : launch_types<kE4m3, kFp16>(a, stream);
}

}  // namespace paged
}  // namespace kvq
