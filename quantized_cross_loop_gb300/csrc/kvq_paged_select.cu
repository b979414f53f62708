// kvq_paged_select.cu — the pages a query most likely finds something on.
//
// score(page) = sum_j sum_d (q_jd < 0 ? q_jd lo_d : q_jd hi_d), the sum over the
// group's query heads j of the largest q.k that the page's bounds allow. The sum
// over the heads goes into the query: score = sum_d up_d hi_d + down_d lo_d with
// up_d = sum_j max(q_jd, 0) and down_d = sum_j min(q_jd, 0): 256 products per page
// and KV head whatever the group is, on the 512 bytes of its two bounds. Bound: HBM.
//
// The score kernel reads each bound once, 16 bytes a lane, and leaves the scores
// as order-preserving 32-bit keys, and for every 32 pages the largest sum of
// absolute terms A. An FP32 score is off by at most E = 2^-18 A: the weights are sums
// of at most 16 terms of one sign (15 u, u = 2^-24), a lane adds up to 16 products
// (16 u), five additions join the lanes (5 u); 64 u leaves room for A's own rounding.
//
// The pick kernel finds the key t of the last page that FP32 would take, by
// histograms over the keys' range. Pages above t + 2E are in, those below t - 2E are
// out by the exact scores too; if the pages between are not all taken, they are
// scored again in FP64 (products of 11-bit significands summed in 53 bits) and
// ranked, ties by page number. Two pages scarcely ever are that near: the second
// scoring costs nothing as a rule, and the order is exact always.
#include "kvq_attn_common.cuh"
#include "kvq_paged.cuh"

namespace kvq {
namespace paged {
namespace {

constexpr int kScoreThreads = 256;
constexpr int kChunk = 16;           // pages a warp scores at a time
constexpr int kInFlight = 8;         // loads a lane has in flight
constexpr int kScoreBlocksPerSm = 4;
constexpr int kPickThreads = 512;
constexpr int kPickWarps = kPickThreads / 32;
constexpr int kBins = 2048;
constexpr int kList = 1024;          // candidates ranked in shared memory
constexpr int kStagedMax = 40960;    // pages whose keys are staged in shared memory
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

struct Workspace {
  uint32_t* keys;   // [units][max_pages]
  float* largest;   // [units][chunks]: A of the chunk
  uint64_t* exact;  // [units][max_pages], candidates only
};
constexpr size_t up16(size_t n) { return (n + 15) / 16 * 16; }
__host__ __device__ inline int chunks_of(int pages) { return (pages + kChunk - 1) / kChunk; }
inline Workspace workspace_of(char* ws, int units, int max_pages) {
  Workspace w;
  w.keys = reinterpret_cast<uint32_t*>(ws + 16);
  char* p = ws + 16 + up16(size_t(units) * max_pages * 4);
  w.largest = reinterpret_cast<float*>(p);
  w.exact = reinterpret_cast<uint64_t*>(p + up16(size_t(units) * chunks_of(max_pages) * 4));
  return w;
}

__device__ __forceinline__ int pages_of(const SelectArgs& a, int T) { return T <= 0 ? 0 : a.c.ps.div(T - 1) + 1; }

template <int DT>
__device__ __forceinline__ const char* bounds_of(const SelectArgs& a, int page, int h) {
  return a.c.bounds + ((long long)page * a.c.H + h) * (2 * kD * elem_bytes<DT>());
}

// Eight values of 16-bit type, or sixteen of E4M3, of a 16-byte load.
template <int DT>
__device__ __forceinline__ void unpack(const uint4& v, float (&x)[DT == kE4m3 ? 16 : 8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (DT == kE4m3) {
      const uint32_t a = e4m3x2_to_f16x2(w[i] & 0xFFFFu), b = e4m3x2_to_f16x2(w[i] >> 16);
      const float2 p = __half22float2(*reinterpret_cast<const __half2*>(&a));
      const float2 q = __half22float2(*reinterpret_cast<const __half2*>(&b));
      x[4 * i] = p.x;
      x[4 * i + 1] = p.y;
      x[4 * i + 2] = q.x;
      x[4 * i + 3] = q.y;
    } else if constexpr (DT == kBf16) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    } else {
      const float2 p = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
      x[2 * i] = p.x;
      x[2 * i + 1] = p.y;
    }
  }
}

// A warp scores 16 pages: a page's bounds are 32 (16-bit) or 16 (E4M3) loads of 16
// bytes, so a lane holds the weights of its own 8 or 16 channels of lo or hi, and
// one load instruction covers one or two pages.
template <int DT, int QT>
struct Scorer {
  static constexpr int kPer = DT == kE4m3 ? 16 : 8;      // channels of a lane
  static constexpr int kLanes = 2 * kD / kPer;           // lanes of a page
  static constexpr int kAtOnce = 32 / kLanes;            // pages per load
  static constexpr int kLoads = kChunk / kAtOnce;
  static constexpr int kBatch = kLoads < kInFlight ? kLoads : kInFlight;
  float w[kPer];

  __device__ __forceinline__ void weights(const SelectArgs& a, int b, int h, int lane) {
    const int sub = lane % kLanes, at = sub % (kLanes / 2) * kPer;
    const bool up = sub >= kLanes / 2;
#pragma unroll
    for (int e = 0; e < kPer; ++e) w[e] = 0.0f;
    const char* q = a.q + (long long)b * a.q_stride + ((long long)h * a.g * kD + at) * 2;
#pragma unroll 4
    for (int j = 0; j < a.g; ++j) {
#pragma unroll
      for (int e = 0; e < kPer; e += 8) {
        float x[8];
        unpack<QT>(__ldg(reinterpret_cast<const uint4*>(q + (j * kD + e) * 2)), x);
#pragma unroll
        for (int i = 0; i < 8; ++i) w[e + i] += (x[i] < 0.0f) == up ? 0.0f : x[i];
      }
    }
  }

  // Page numbers of the chunk from page p0 on, one in each lane of a half warp (0 behind the last).
  __device__ __forceinline__ static int ids(const SelectArgs& a, int b, int p0, int pages, int lane) {
    const int p = p0 + (lane & (kChunk - 1));
    return p < pages ? a.table[(long long)b * a.max_pages + p] : 0;
  }

  // Scores of the chunk whose page numbers are `page`: the key of its page `index` in each lane. The chunk's A, a
  // lane's largest sums added over the lanes, joins `largest`.
  __device__ __forceinline__ uint32_t score(const SelectArgs& a, int h, int page, int lane, int& index, float& largest) {
    if (page < 0 || page >= a.c.n_pages) {
      flag(a.c, KVQ_PAGED_ERR_PAGE);
      page = -1;
    }
    float v[kLoads], top = 0.0f;
#pragma unroll
    for (int i0 = 0; i0 < kLoads; i0 += kBatch) {
      uint4 r[kBatch];
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const int id = __shfl_sync(0xFFFFFFFFu, page, (i0 + i) * kAtOnce + lane / kLanes);
        r[i] = __ldg(reinterpret_cast<const uint4*>(bounds_of<DT>(a, id < 0 ? 0 : id, h)) + lane % kLanes);
      }
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        float x[kPer], s = 0.0f, t = 0.0f;
        unpack<DT>(r[i], x);
#pragma unroll
        for (int e = 0; e < kPer; ++e) {
          s = fmaf(w[e], x[e], s);
          t = fmaf(fabsf(w[e]), fabsf(x[e]), t);
        }
        v[i0 + i] = s;
        if (t <= 3.4e38f) top = fmaxf(top, t);  // (infinite and NaN bounds set no E: their pages' keys are exact)
      }
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
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top += __shfl_xor_sync(0xFFFFFFFFu, top, o);
    largest = fmaxf(largest, top);
    return __shfl_sync(0xFFFFFFFFu, page, index) < 0 ? kLastKey : key_of(v[0]);
  }
};

template <int DT, int QT>
__global__ void __launch_bounds__(kScoreThreads, kScoreBlocksPerSm) score_kernel(SelectArgs a, Workspace ws) {
  __shared__ Prefix<kScoreThreads> S;
  wait_prior_grid();
  allow_dependents();
  auto count = [&](int b) {
    const int pages = pages_of(a, checked_len(a.lens, b, a.max_pages, a.c.ps));
    return pages <= a.n_select ? 0LL : (long long)a.c.H * chunks_of(pages);  // all taken: nothing to score
  };
  build_prefix<kScoreThreads>(S, a.B, count);
  if (a.c.err != nullptr && blockIdx.x == 0)
    for (int b = threadIdx.x; b < a.B; b += kScoreThreads)
      if (checked_len(a.lens, b, a.max_pages, a.c.ps) < 0) flag(a.c, KVQ_PAGED_ERR_LENGTH);
  const int lane = threadIdx.x & 31;
  const long long total = S.pre[kScoreThreads], warps = (long long)gridDim.x * (kScoreThreads / 32);
  const long long me = (long long)blockIdx.x * (kScoreThreads / 32) + threadIdx.x / 32;
  const long long c0 = me * total / warps, c1 = (me + 1) * total / warps;
  if (c0 >= c1) return;
  long long at = c0;
  int b = find_request<kScoreThreads>(S, a.B, count, at);
  int pages = pages_of(a, checked_len(a.lens, b, a.max_pages, a.c.ps)), chunks = chunks_of(pages);
  int h = int(at / chunks), chunk = int(at % chunks);
  Scorer<DT, QT> K;
  bool fresh = true;
  for (long long c = c0; c < c1; ++c) {
    const int ids = K.ids(a, b, chunk * kChunk, pages, lane);
    if (fresh) K.weights(a, b, h, lane);
    fresh = false;
    const long long unit = (long long)b * a.c.H + h;
    int index;
    float largest = 0.0f;
    const uint32_t key = K.score(a, h, ids, lane, index, largest);
    const int p = chunk * kChunk + index;
    if (p < pages) ws.keys[unit * a.max_pages + p] = key;
    if (lane == 0) ws.largest[unit * chunks_of(a.max_pages) + chunk] = largest;
    if (++chunk == chunks) {
      chunk = 0;
      fresh = true;
      if (++h == a.c.H) {
        h = 0;
        for (++b; b < a.B; ++b) {
          pages = pages_of(a, checked_len(a.lens, b, a.max_pages, a.c.ps));
          chunks = chunks_of(pages);
          if (pages > a.n_select) break;
        }
      }
    }
  }
}

struct Pick {
  int hist[kBins];
  uint32_t list_key[kList];
  uint64_t list_exact[kList];
  int list_page[kList];
  double up[kD], down[kD];
  int warp_sum[kPickWarps];
  uint32_t warp_lo[kPickWarps], warp_hi[kPickWarps];
  float warp_a[kPickWarps];
  int n_list, left, above, bin, members;
  uint32_t t;
  uint64_t prefix;
};

__device__ __forceinline__ int block_sum(Pick& S, int x) {
  x = __reduce_add_sync(0xFFFFFFFFu, x);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) S.warp_sum[threadIdx.x >> 5] = x;
  __syncthreads();
  int n = 0;
  for (int w = 0; w < kPickWarps; ++w) n += S.warp_sum[w];
  return n;
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

// The `left`-th largest of up to kPickThreads keys: the one with fewer than `left` above it and enough not below.
__device__ __forceinline__ uint32_t ranked(Pick& S, const uint32_t* keys, int n, int left) {
  if (threadIdx.x < n) {
    const uint32_t x = keys[threadIdx.x];
    int more = 0, same = 0;
#pragma unroll 8
    for (int i = 0; i < n; ++i) {
      more += keys[i] > x;
      same += keys[i] == x;
    }
    if (more < left && left <= more + same) S.t = x;
  }
  __syncthreads();
  return S.t;
}

// Picks a unit's pages from its keys (`keys` is scratch: written, too); the block's threads together.
template <int DT, int QT>
__device__ __forceinline__ void pick(const SelectArgs& a, Pick& S, int b, int h, int pages, uint32_t* keys,
                                     float largest, uint64_t* exact, int32_t* sel) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int f0 = a.n_first, f1 = pages - a.n_last;  // pages before f0 and from f1 on are taken anyway
  const int k = a.n_select - a.n_first - a.n_last;
  uint32_t lo = 0xFFFFFFFFu, hi = 0u;  // window of keys in doubt; above it a page is in
  if (k == 0) {
    hi = kFirstKey;
    for (int p = f0 + tid; p < f1; p += kPickThreads) keys[p] = kLastKey;  // none but those
    __syncthreads();
  } else {
    const bool few = f1 - f0 <= kPickThreads;
    if (!few) {  // the keys' range
      for (int p = f0 + tid; p < f1; p += kPickThreads) {
        lo = min(lo, keys[p]);
        hi = max(hi, keys[p]);
      }
      lo = __reduce_min_sync(0xFFFFFFFFu, lo);
      hi = __reduce_max_sync(0xFFFFFFFFu, hi);
      if (lane == 0) {
        S.warp_lo[warp] = lo;
        S.warp_hi[warp] = hi;
      }
      __syncthreads();
      for (int w = 0; w < kPickWarps; ++w) {
        lo = min(lo, S.warp_lo[w]);
        hi = max(hi, S.warp_hi[w]);
      }
    }
    // the k-th largest key
    int left = k;
    uint32_t t = lo;
    while (lo < hi && !few) {
      const int bits = 32 - __clz(hi - lo), shift = bits > 11 ? bits - 11 : 0;
      for (int i = tid; i < kBins; i += kPickThreads) S.hist[i] = 0;
      if (tid == 0) S.n_list = 0;
      __syncthreads();
      for (int p = f0 + tid; p < f1; p += kPickThreads) {
        const uint32_t x = keys[p];
        if (x >= lo && x <= hi) atomicAdd(&S.hist[(x - lo) >> shift], 1);
      }
      __syncthreads();
      {  // bins from the top: thread i holds bins kBins - 4 i - 4 .. kBins - 4 i - 1
        int own[4], n = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          own[e] = S.hist[kBins - 1 - 4 * tid - e];
          n += own[e];
        }
        int before = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int y = __shfl_up_sync(0xFFFFFFFFu, before, o);
          if (lane >= o) before += y;
        }
        if (lane == 31) S.warp_sum[warp] = before;
        __syncthreads();
        before -= n;
        for (int w = 0; w < warp; ++w) before += S.warp_sum[w];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          if (before < left && left <= before + own[e]) {  // one thread, one bin
            S.bin = kBins - 1 - 4 * tid - e;
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
      if (lo < hi && members <= kPickThreads) {
        for (int p = f0 + tid; p < f1; p += kPickThreads) {
          const uint32_t x = keys[p];
          if (x >= lo && x <= hi) S.list_key[atomicAdd(&S.n_list, 1)] = x;
        }
        __syncthreads();
        t = ranked(S, S.list_key, members, left);
        break;
      }
      __syncthreads();  // hist, bin and list are free again
    }
    if (few) t = ranked(S, keys + f0, f1 - f0, k);
    // pages in doubt
    lo = hi = t;
    if (t != kFirstKey && t != kLastKey) {
      const float x = float_of(t), e = 2.0f * (largest * 0x1p-18f);
      const float x0 = __fsub_rd(x, e), x1 = __fadd_ru(x, e);
      lo = x0 >= -3.4e38f ? key_of(x0) : key_of(-3.402823466e38f);
      hi = x1 <= 3.4e38f ? key_of(x1) : kFirstKey - 1u;
    }
    int n_above = 0, n_in = 0;
    for (int p = f0 + tid; p < f1; p += kPickThreads) {
      n_above += keys[p] > hi;
      n_in += keys[p] >= lo && keys[p] <= hi;
    }
    n_above = block_sum(S, n_above);
    n_in = block_sum(S, n_in);
    const int want = k - n_above;
    if (want == n_in) {
      hi = lo - 1u;  // all of them (lo > 0: a page outside the pool is only taken when every page is)
      if (lo == 0u) {
        hi = 0u;
        for (int p = f0 + tid; p < f1; p += kPickThreads) keys[p] = kFirstKey;
        __syncthreads();
      }
    } else {
      if (tid < kD) {
        double up = 0.0, down = 0.0;
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
      if (tid == 0) S.n_list = 0;
      __syncthreads();
      if (n_in <= kList) {
        for (int p = f0 + tid; p < f1; p += kPickThreads)
          if (keys[p] >= lo && keys[p] <= hi) S.list_page[atomicAdd(&S.n_list, 1)] = p;
        __syncthreads();
        for (int i = warp; i < n_in; i += kPickWarps) {
          const uint64_t x = exact_key<DT>(a, S, b, h, S.list_page[i], lane);
          if (lane == 0) S.list_exact[i] = x;
        }
        __syncthreads();
        for (int i = tid; i < n_in; i += kPickThreads) {
          const uint64_t x = S.list_exact[i];
          const int p = S.list_page[i];
          int rank = 0;
          for (int j = 0; j < n_in; ++j) rank += S.list_exact[j] > x || (S.list_exact[j] == x && S.list_page[j] < p);
          keys[p] = rank < want ? kFirstKey : kLastKey;
        }
      } else {  // many pages score the same, or nearly: a radix selection over the exact keys
        for (int p = f0 + warp; p < f1; p += kPickWarps) {
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
          for (int p = f0 + tid; p < f1; p += kPickThreads)
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
        for (int p0 = f0; p0 < f1; p0 += kPickThreads) {
          const int p = p0 + tid;
          const bool in = p < f1 && keys[p] >= lo && keys[p] <= hi;
          const uint64_t x = in ? exact[p] : 0;
          const bool same = in && x == prefix;
          const uint32_t m = __ballot_sync(0xFFFFFFFFu, same);
          if (lane == 0) S.warp_sum[warp] = __popc(m);
          __syncthreads();
          int rank = seen + __popc(m & ((1u << lane) - 1u));
          for (int w = 0; w < kPickWarps; ++w) {
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
  // the pages in order: each warp a run of them, counted, then written behind the warps before
  const int run = ((pages + kPickWarps - 1) / kPickWarps + 31) / 32 * 32;
  const int p0 = min(pages, warp * run), p1 = min(pages, p0 + run);
  auto taken = [&](int p) { return p < p1 && (p < f0 || p >= f1 || keys[p] > hi || keys[p] == kFirstKey); };
  int n = 0;
  for (int p = p0; p < p1; p += 32) n += __popc(__ballot_sync(0xFFFFFFFFu, taken(p + lane)));
  __syncthreads();
  if (lane == 0) S.warp_sum[warp] = n;
  __syncthreads();
  int at = 0;
  for (int w = 0; w < warp; ++w) at += S.warp_sum[w];
  for (int p = p0; p < p1; p += 32) {
    const bool in = taken(p + lane);
    const uint32_t m = __ballot_sync(0xFFFFFFFFu, in);
    const int i = at + __popc(m & ((1u << lane) - 1u));
    if (in && i < a.n_select) sel[i] = p + lane;
    at += __popc(m);
  }
}

template <int DT, int QT>
__global__ void __launch_bounds__(kPickThreads) pick_kernel(SelectArgs a, Workspace ws, int staged) {
  __shared__ Pick S;
  extern __shared__ __align__(16) uint32_t s_keys[];
  wait_prior_grid();
  allow_dependents();
  const long long unit = blockIdx.x;
  const int b = int(unit / a.c.H), h = int(unit % a.c.H), tid = threadIdx.x;
  const int pages = pages_of(a, checked_len(a.lens, b, a.max_pages, a.c.ps));
  int32_t* sel = a.sel + unit * a.n_select;
  if (pages <= a.n_select) {  // all of them, and -1 behind
    for (int i = tid; i < a.n_select; i += kPickThreads) sel[i] = i < pages ? i : -1;
    return;
  }
  uint32_t* keys = ws.keys + unit * a.max_pages;
  if (staged) {
    for (int p = tid; p < pages; p += kPickThreads) s_keys[p] = keys[p];
    keys = s_keys;
  }
  float largest = 0.0f;
  const float* l = ws.largest + unit * chunks_of(a.max_pages);
  for (int i = tid; i < chunks_of(pages); i += kPickThreads) largest = fmaxf(largest, l[i]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) largest = fmaxf(largest, __shfl_xor_sync(0xFFFFFFFFu, largest, o));
  if ((tid & 31) == 0) S.warp_a[tid >> 5] = largest;
  __syncthreads();
  for (int w = 0; w < kPickWarps; ++w) largest = fmaxf(largest, S.warp_a[w]);
  pick<DT, QT>(a, S, b, h, pages, keys, largest, ws.exact + unit * a.max_pages, sel);
}

// Both in one: a block scores and picks a unit's pages, the keys in shared memory.
template <int DT, int QT>
__global__ void __launch_bounds__(kPickThreads, 2) select_kernel(SelectArgs a, Workspace ws) {
  __shared__ Pick S;
  extern __shared__ __align__(16) uint32_t s_keys[];
  wait_prior_grid();
  allow_dependents();
  const long long unit = blockIdx.x;
  const int b = int(unit / a.c.H), h = int(unit % a.c.H), tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int T = checked_len(a.lens, b, a.max_pages, a.c.ps), pages = pages_of(a, T);
  if (T < 0 && tid == 0) flag(a.c, KVQ_PAGED_ERR_LENGTH);
  int32_t* sel = a.sel + unit * a.n_select;
  if (pages <= a.n_select) {  // all of them, and -1 behind
    for (int i = tid; i < a.n_select; i += kPickThreads) sel[i] = i < pages ? i : -1;
    return;
  }
  Scorer<DT, QT> K;
  float largest = 0.0f;
  int ids = K.ids(a, b, warp * kChunk, pages, lane);
  K.weights(a, b, h, lane);
  for (int p0 = warp * kChunk; p0 < pages; p0 += kPickWarps * kChunk) {
    const int next = K.ids(a, b, p0 + kPickWarps * kChunk, pages, lane);
    int index;
    const uint32_t key = K.score(a, h, ids, lane, index, largest);
    if (p0 + index < pages) s_keys[p0 + index] = key;
    ids = next;
  }
  if (lane == 0) S.warp_a[warp] = largest;
  __syncthreads();
  for (int w = 0; w < kPickWarps; ++w) largest = fmaxf(largest, S.warp_a[w]);
  pick<DT, QT>(a, S, b, h, pages, s_keys, largest, ws.exact + unit * a.max_pages, sel);
}

// One launch where a unit's pages keep a block busy for no longer than the second
// launch would take, or where there are units for all SMs; else the pages are
// scored by all warps of the device and picked by a second kernel.
constexpr int kFusedPages = 256;      // any number of units
constexpr int kFusedManyPages = 2048; // at least one unit per SM

template <int DT, int QT>
cudaError_t launch_types(const SelectArgs& a, cudaStream_t stream) {
  const int units = a.B * a.c.H;
  const Workspace ws = workspace_of(a.ws, units, a.max_pages);
  const int staged = a.max_pages <= kStagedMax;
  const size_t smem = staged ? size_t(a.max_pages) * 4 : 0;
  if (a.max_pages <= kFusedPages || (a.max_pages <= kFusedManyPages && units >= a.sms)) {
    count_launch();
    return launch_dependent(select_kernel<DT, QT>, dim3(units), dim3(kPickThreads), smem, stream, a, ws);
  }
  const long long warps = (long long)units * chunks_of(a.max_pages);  // at most
  const long long need = (warps + kScoreThreads / 32 - 1) / (kScoreThreads / 32);
  const int blocks = int(need < 1 ? 1 : need < (long long)kScoreBlocksPerSm * a.sms ? need : (long long)kScoreBlocksPerSm * a.sms);
  count_launch();
  cudaError_t e = launch_dependent(score_kernel<DT, QT>, dim3(blocks), dim3(kScoreThreads), 0, stream, a, ws);
  if (e != cudaSuccess) return e;
  if (smem > 16384) {
    e = cudaFuncSetAttribute(pick_kernel<DT, QT>, cudaFuncAttributeMaxDynamicSharedMemorySize, kStagedMax * 4);
    if (e != cudaSuccess) return e;
  }
  count_launch();
  return launch_dependent(pick_kernel<DT, QT>, dim3(units), dim3(kPickThreads), smem, stream, a, ws, staged);
}

}  // namespace

size_t select_workspace(int B, int H, int max_pages) {
  const size_t units = size_t(B) * H;
  return 16 + up16(units * max_pages * 4) + up16(units * chunks_of(max_pages) * 4) + up16(units * max_pages * 8);
}

cudaError_t launch_select(const SelectArgs& a, cudaStream_t stream) {
  const bool bf = a.q_dtype == kBf16;
  if (a.dtype == kBf16) return launch_types<kBf16, kBf16>(a, stream);
  if (a.dtype == kFp16) return launch_types<kFp16, kFp16>(a, stream);
  return bf ? launch_types<kE4m3, kBf16>(a, stream) : launch_types<kE4m3, kFp16>(a, stream);
}

}  // namespace paged
}  // namespace kvq
