// kvq_paged_move.cu — rows of a paged cache back to 16-bit rows (kvq_paged_read), and
// accepted drafted tokens to their places (kvq_paged_tree_commit).
#include "kvq_attn_common.cuh"
#include "kvq_paged.cuh"

namespace kvq {
namespace paged {
namespace {

// ---------------------------------------------------------------- read
//
// Value = stored x scale (FP32), rounded once to the output's type. Bound: HBM (each
// row is read and written once).
//
// Sixteen lanes (a team) hold a row of a head, eight channels each. Work: (row, head)
// pairs in the rows' order, a block's teams side by side, so that the heads of a row
// are written together; kReadRows pairs in flight per team. Measured: eight FP16
// requests of up to 8191 rows to BF16, 8 heads, pages of 16, 138 MB moved: 24.9 us,
// 5.5 TB/s, 82% of a copy's rate; other blocks per SM x rows in flight: 1 x 8 25.3 us,
// 2 x 6 25.2, 2 x 8 26.0, 4 x 6 31.5, 4 x 8 35.5, 8 x 2 25.4. 64 tiles of 64 rows, E4M3
// with scales per token, 25 MB: 7.6 us (launch, the search for a row's request, which is
// log2 of the requests dependent loads, and range and start -> table -> row).

constexpr int kReadThreads = 256;
constexpr int kReadTeam = 16;
constexpr int kReadTeams = kReadThreads / kReadTeam;
constexpr int kReadBlocksPerSm = 4;
constexpr int kReadRows = 4;

template <int DT>
struct Eight {  // stored channels of a lane
  uint32_t w[DT == kE4m3 ? 2 : 4];
};

template <int DT>
__device__ __forceinline__ Eight<DT> load8(const char* p) {
  Eight<DT> r;
  if constexpr (DT == kE4m3) {
    const uint2 x = *reinterpret_cast<const uint2*>(p);
    r.w[0] = x.x;
    r.w[1] = x.y;
  } else {
    const uint4 x = *reinterpret_cast<const uint4*>(p);
    r.w[0] = x.x;
    r.w[1] = x.y;
    r.w[2] = x.z;
    r.w[3] = x.w;
  }
  return r;
}

template <int DT, int OUT>
__device__ __forceinline__ void store8(char* p, const Eight<DT>& x, float scale) {
  uint4 r;
  if constexpr (DT == OUT) {
    r = make_uint4(x.w[0], x.w[1], x.w[2], x.w[3]);
  } else {
    float4 a, b;
    if constexpr (DT == kE4m3) {
      a = times(load4<DT>(&x.w[0]), scale);
      b = times(load4<DT>(&x.w[1]), scale);
    } else {
      a = load4<DT>(&x.w[0]);
      b = load4<DT>(&x.w[2]);
    }
    store4<OUT>(&r.x, a);
    store4<OUT>(&r.z, b);
  }
  *reinterpret_cast<uint4*>(p) = r;
}

template <int DT, int OUT>
__global__ void __launch_bounds__(kReadThreads, kReadBlocksPerSm) read_kernel(ReadArgs a) {
  wait_prior_grid();
  allow_dependents();
  const int H = a.c.H, lane = threadIdx.x % kReadTeam;
  const long long pairs = (long long)a.n_rows * H;
  const long long p1 = part_start(blockIdx.x + 1, pairs, gridDim.x);
  long long p = part_start(blockIdx.x, pairs, gridDim.x) + threadIdx.x / kReadTeam;
  // requests that have no rows because their offsets are out of order or beyond the rows: no row leads to them
  if (a.offsets != nullptr)
#pragma unroll 1
    for (int i = blockIdx.x * kReadThreads + threadIdx.x; i < a.B; i += gridDim.x * kReadThreads) {
      int row0;
      if (row_range(a.offsets, a.n_rows, i, row0) < 0) flag(a.c, KVQ_PAGED_ERR_LENGTH);
    }
  if (p >= p1) return;
  int row, h;
  divide(p, H, row, h);
  int b = row;
  if (a.offsets != nullptr) {  // the last request whose rows begin at or before this one
    int lo = 0, hi = a.B - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (a.offsets[mid] <= row) lo = mid;
      else hi = mid - 1;
    }
    b = lo;
  }
  for (; p < p1; p += kReadRows * kReadTeams) {
    Eight<DT> k[kReadRows], v[kReadRows];
    float ks[kReadRows], vs[kReadRows];
    int at[kReadRows], head[kReadRows];
    bool mine[kReadRows], ok[kReadRows];
#pragma unroll
    for (int i = 0; i < kReadRows; ++i) {
      at[i] = row;
      head[i] = h;
      mine[i] = p + i * kReadTeams < p1;
      ok[i] = false;
      int page = -1, place = 0;
      if (mine[i]) {
        if (a.offsets != nullptr)
          while (b < a.B - 1 && a.offsets[b + 1] <= row) ++b;
        else
          b = row;
        int row0;
        const int n = row_range(a.offsets, a.n_rows, b, row0), start = a.start[b];
        mine[i] = n >= 0 && row >= row0 && row < row0 + n;
        if (mine[i]) {
          if (start < 0 || (long long)start + n > (long long)a.max_pages * a.c.ps.d) {
            flag(a.c, KVQ_PAGED_ERR_LENGTH);
          } else {
            const int t = start + row - row0, e = a.c.ps.div(t);
            place = t - e * int(a.c.ps.d);
            page = a.table[(long long)b * a.max_pages + e];
            ok[i] = page >= 0 && page < a.c.n_pages;
            if (!ok[i]) flag(a.c, KVQ_PAGED_ERR_PAGE);
          }
        }
      }
      ks[i] = vs[i] = 1.0f;
      if (ok[i]) {
        const long long off = (long long)page * a.c.page_stride + (long long)place * a.c.token_stride +
                              (long long)h * a.c.head_stride + lane * 8 * elem_bytes<DT>();
        k[i] = load8<DT>(a.c.k + off);
        v[i] = load8<DT>(a.c.v + off);
        if constexpr (DT == kE4m3) {
          const long long s = a.c.token_scales ? ((long long)page * H + h) * int(a.c.ps.d) + place : h;
          if (a.c.k_scale != nullptr) ks[i] = a.c.k_scale[s];
          if (a.c.v_scale != nullptr) vs[i] = a.c.v_scale[s];
        }
      }
      h += kReadTeams;
      while (h >= H) {
        h -= H;
        ++row;
      }
    }
#pragma unroll
    for (int i = 0; i < kReadRows; ++i) {
      if (!mine[i]) continue;
      const long long to = (long long)head[i] * (kD * 2) + lane * 16;
      char* const tk = a.k + at[i] * a.k_stride + to;
      char* const tv = a.v + at[i] * a.v_stride + to;
      if (ok[i]) {
        store8<DT, OUT>(tk, k[i], ks[i]);
        store8<DT, OUT>(tv, v[i], vs[i]);
      } else {
        constexpr uint32_t kNan = OUT == kBf16 ? 0x7FC07FC0u : 0x7E007E00u;
        *reinterpret_cast<uint4*>(tk) = *reinterpret_cast<uint4*>(tv) = make_uint4(kNan, kNan, kNan, kNan);
      }
    }
  }
}

// ---------------------------------------------------------------- commit
//
// A block per (request, KV head): it looks at the whole list first (a request is
// moved or left alone), then moves kMoveRows accepted tokens at a time, all of them
// read before any is written. That is in order, because the list ascends: the k-th
// accepted token is at place k or behind it, so what a later step reads lies behind
// what an earlier one wrote. The bounds are then taken from the keys as they are.
// Bound: latency (a few rows per request): 64 requests that keep 5 of 16 BF16 tokens,
// 8 heads, 4.8 us; 256 that keep up to 32 of 64, E4M3 with scales per token, 8.5 us: 2048
// blocks, five to an SM, are 2.7 waves of the whole chain, which reads list and table
// twice (to check them, and to move).

constexpr int kMoveThreads = 256;
constexpr int kMoveWarps = kMoveThreads / 32;

template <int DT>
struct Move {
  static constexpr int kChunks = kD * elem_bytes<DT>() / 16;  // of a row
  static constexpr int kLanes = 2 * kChunks;                  // a token's K and V
  static constexpr int kTokens = kMoveThreads / kLanes;       // side by side
  static constexpr int kEach = 4;                             // of a thread
  static constexpr int kRows = kTokens * kEach;
};

template <int DT>
__global__ void __launch_bounds__(kMoveThreads) commit_kernel(CommitArgs a) {
  using M = Move<DT>;
  __shared__ int s_src[M::kRows], s_dst[M::kRows];  // places on their pages
  __shared__ int s_page[M::kRows][2];               // pages of the pool, from and to (-1: the token stays)
  __shared__ uint4 s_bound[kMoveWarps][2][16];
  wait_prior_grid();
  allow_dependents();
  const int b = blockIdx.x / a.c.H, h = blockIdx.x % a.c.H, ps = int(a.c.ps.d), t = threadIdx.x;
  const int P = checked_len(a.lens, b, a.max_pages, a.c.ps);
  int off;
  const int m = row_range(a.offsets, a.n_accepted, b, off);
  const long long room = (long long)a.max_pages * ps;
  if (P < 0 || m < 0 || P + (long long)m > room) {
    if (t == 0) flag(a.c, KVQ_PAGED_ERR_LENGTH);
    return;
  }
  const int32_t* table = a.table + (long long)b * a.max_pages;
  int bad = 0;
  for (int i = t; i < m; i += kMoveThreads) {
    const int x = a.accepted[off + i];
    if (x < i || (i > 0 && x <= a.accepted[off + i - 1])) {
      bad |= KVQ_PAGED_ERR_SELECTION;
    } else if (P + (long long)x >= room) {
      bad |= KVQ_PAGED_ERR_LENGTH;
    } else {
      const int from = table[a.c.ps.div(P + x)], to = table[a.c.ps.div(P + i)];
      if (from < 0 || from >= a.c.n_pages || to < 0 || to >= a.c.n_pages) bad |= KVQ_PAGED_ERR_PAGE;
    }
  }
  if (bad != 0) flag(a.c, bad);
  if (__syncthreads_or(bad)) return;

  const int lane = t % M::kLanes, token = t / M::kLanes, chunk = lane % M::kChunks;
  char* const pool = lane < M::kChunks ? a.c.k : a.c.v;
  float* const scale = const_cast<float*>(lane < M::kChunks ? a.c.k_scale : a.c.v_scale);
  for (int i0 = 0; i0 < m; i0 += M::kRows) {
    if (t < M::kRows && i0 + t < m) {
      const int src = P + a.accepted[off + i0 + t], dst = P + i0 + t, e = a.c.ps.div(src), f = a.c.ps.div(dst);
      s_src[t] = src - e * ps;
      s_dst[t] = dst - f * ps;
      s_page[t][0] = table[e];
      s_page[t][1] = src == dst ? -1 : table[f];
    }
    __syncthreads();
    uint4 x[M::kEach];
    float s[M::kEach];
#pragma unroll
    for (int e = 0; e < M::kEach; ++e) {
      const int i = e * M::kTokens + token;
      if (i0 + i >= m || s_page[i][1] < 0) continue;
      x[e] = *reinterpret_cast<const uint4*>(pool + (long long)s_page[i][0] * a.c.page_stride +
                                             (long long)s_src[i] * a.c.token_stride + (long long)h * a.c.head_stride +
                                             chunk * 16);
      if (a.c.token_scales && chunk == 0) s[e] = scale[((long long)s_page[i][0] * a.c.H + h) * ps + s_src[i]];
    }
    __syncthreads();  // all of them are read
#pragma unroll
    for (int e = 0; e < M::kEach; ++e) {
      const int i = e * M::kTokens + token;
      if (i0 + i >= m || s_page[i][1] < 0) continue;
      *reinterpret_cast<uint4*>(pool + (long long)s_page[i][1] * a.c.page_stride +
                                (long long)s_dst[i] * a.c.token_stride + (long long)h * a.c.head_stride + chunk * 16) =
          x[e];
      if (a.c.token_scales && chunk == 0) scale[((long long)s_page[i][1] * a.c.H + h) * ps + s_dst[i]] = s[e];
    }
    __syncthreads();  // the list's places are free again; the keys are there for the bounds
  }
  if (a.c.bounds == nullptr) return;

  // a page at a time: sixteen lanes hold a row (eight channels each), 2 kMoveWarps rows side by side
  constexpr int kE = elem_bytes<DT>();
  constexpr uint32_t kInf = DT == kBf16 ? 0x7F807F80u : 0x7C007C00u;
  const int c = t % 16, warp = t >> 5, end = P + m;
  for (int p = a.c.ps.div(P); p * (long long)ps < end; ++p) {
    const int page = table[p], n = min(ps, end - p * ps);
    if (page < 0 || page >= a.c.n_pages) {
      if (t == 0) flag(a.c, KVQ_PAGED_ERR_PAGE);
      continue;
    }
    constexpr uint32_t kLow = kInf | 0x80008000u;
    uint4 lo = make_uint4(kInf, kInf, kInf, kInf), hi = make_uint4(kLow, kLow, kLow, kLow);
    const char* row = a.c.k + (long long)page * a.c.page_stride + (long long)h * a.c.head_stride + c * 8 * kE;
    auto join = [&](uint4& x, uint4& y, const uint4& l, const uint4& u) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        (&x.x)[i] = smaller<DT>((&x.x)[i], (&l.x)[i]);
        (&y.x)[i] = larger<DT>((&y.x)[i], (&u.x)[i]);
      }
    };
#pragma unroll 4
    for (int i = t / 16; i < n; i += kMoveThreads / 16) {
      uint4 x;
      if constexpr (DT == kE4m3) {
        const uint2 w = *reinterpret_cast<const uint2*>(row + (long long)i * a.c.token_stride);
        x = make_uint4(e4m3x2_to_f16x2(w.x & 0xFFFFu), e4m3x2_to_f16x2(w.x >> 16), e4m3x2_to_f16x2(w.y & 0xFFFFu),
                       e4m3x2_to_f16x2(w.y >> 16));
      } else {
        x = *reinterpret_cast<const uint4*>(row + (long long)i * a.c.token_stride);
      }
      join(lo, hi, x, x);
    }
    uint4 l, u;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      (&l.x)[i] = __shfl_xor_sync(0xFFFFFFFFu, (&lo.x)[i], 16);
      (&u.x)[i] = __shfl_xor_sync(0xFFFFFFFFu, (&hi.x)[i], 16);
    }
    join(lo, hi, l, u);
    if ((t & 31) < 16) {
      s_bound[warp][0][c] = lo;
      s_bound[warp][1][c] = hi;
    }
    __syncthreads();
    if (t < 16) {
      for (int w = 1; w < kMoveWarps; ++w) join(lo, hi, s_bound[w][0][c], s_bound[w][1][c]);
      char* to = a.c.bounds + ((long long)page * a.c.H + h) * (2 * kD * kE) + c * 8 * kE;
      if constexpr (DT == kE4m3) {
        uint2 y;
        store4<kE4m3>(&y.x, load4<kFp16>(&lo.x));
        store4<kE4m3>(&y.y, load4<kFp16>(&lo.z));
        *reinterpret_cast<uint2*>(to) = y;
        store4<kE4m3>(&y.x, load4<kFp16>(&hi.x));
        store4<kE4m3>(&y.y, load4<kFp16>(&hi.z));
        *reinterpret_cast<uint2*>(to + kD * kE) = y;
      } else {
        *reinterpret_cast<uint4*>(to) = lo;
        *reinterpret_cast<uint4*>(to + kD * kE) = hi;
      }
    }
    __syncthreads();  // s_bound is free again
  }
}

template <int DT, int OUT>
cudaError_t launch_read_form(const ReadArgs& a, int sms, cudaStream_t stream) {
  // blocks for the rows, and for the look at every request's offsets
  const long long rows = ((long long)a.n_rows * a.c.H + kReadTeams - 1) / kReadTeams;
  const long long requests = ((long long)a.B + kReadThreads - 1) / kReadThreads;
  const long long need = rows > requests ? rows : requests, fit = (long long)kReadBlocksPerSm * sms;
  count_launch();
  return launch_dependent(read_kernel<DT, OUT>, dim3(int(need < fit ? need : fit)), dim3(kReadThreads), 0, stream, a);
}

template <int DT>
cudaError_t launch_commit_form(const CommitArgs& a, cudaStream_t stream) {
  count_launch();
  return launch_dependent(commit_kernel<DT>, dim3(a.B * a.c.H), dim3(kMoveThreads), 0, stream, a);
}

}  // namespace

cudaError_t launch_read(const ReadArgs& a, int sms, cudaStream_t stream) {
  const bool bf = a.out_dtype == kBf16;
  switch (a.dtype) {
    case kBf16: return bf ? launch_read_form<kBf16, kBf16>(a, sms, stream) : launch_read_form<kBf16, kFp16>(a, sms, stream);
    case kFp16: return bf ? launch_read_form<kFp16, kBf16>(a, sms, stream) : launch_read_form<kFp16, kFp16>(a, sms, stream);
    default: return bf ? launch_read_form<kE4m3, kBf16>(a, sms, stream) : launch_read_form<kE4m3, kFp16>(a, sms, stream);
  }
}

cudaError_t launch_commit(const CommitArgs& a, cudaStream_t stream) {
  switch (a.dtype) {
    case kBf16: return launch_commit_form<kBf16>(a, stream);
    case kFp16: return launch_commit_form<kFp16>(a, stream);
    default: return launch_commit_form<kE4m3>(a, stream);
  }
}

}  // namespace paged
}  // namespace kvq
