// kvq_paged_attn.cu — decode attention of one query per request over a paged
// cache, all pages or the selected ones.
//
// s_t = scale q.k_t, out = sum_t e^(s_t - m) v_t / l, lse = m + ln l, in one pass
// over the cache with a running maximum m and sum l per query head.
//
// Bound: HBM. A token and KV head bring 4 D bytes (16-bit) for 4 D g flops, so a
// block must keep loads in flight and spend few instructions a byte.
//
// Work: the tiles of 64 tokens of all (request, KV head) units, concatenated and
// cut into equal ranges, one per block (two blocks an SM); lengths are read on
// the device, so a captured call follows them. A unit that lies in one block's
// range is finished there; of the others each block leaves (m, l, sum) in one of
// its two slots, and the combine kernel joins them.
//
// A warp owns 16 tokens of every tile and a ring of its own in shared memory,
// filled by 16-byte asynchronous copies, so that the main loop has no block
// barrier. Row addresses (selection, page table) are looked up one and two tiles
// ahead of their copies. Rows without a token are filled with zeros.
//
// QK^T with the heads as the 16 rows of mma.m16n8k16 and the tokens as columns:
// its result then is, register for register, the transposed operand of the second
// product out^T = V^T P^T, so the softmax weights never leave their lane.
// Exactness: products of 16-bit values are exact; P is split into parts whose sum
// is P (three of BF16, two of FP16), because one 8- or 11-bit P would cost 2^-9 or
// 2^-12 of the FP32 result. The tensor cores cut their sums off, so every 16
// tokens' product starts from zero and is added to the running sum by FP32 FMA,
// which also applies the rescaling.
// E4M3: keys and values become FP16 in registers (exact); a BF16 query is scaled
// by a power of two into FP16's range (exact down to 2^-31 of its largest).
#include <atomic>
#include <cstddef>

#include "kvq_attn_common.cuh"
#include "kvq_paged.cuh"

namespace kvq {
namespace paged {
namespace {

constexpr int kThreads = 128;
constexpr int kWarps = 4;
constexpr int kTile = 64;          // tokens per tile, 16 per warp
constexpr int kBufStride = 132;    // floats per head of the merge buffers: the lanes' columns hit distinct banks
constexpr int kBlocksPerSm = 2;
constexpr int kCombineThreads = 512;

struct Rec {  // of a block: the unit that starts in its range and ends in block `last`'s (u < 0: none)
  int32_t u, last;
};

// Workspace: Rec[n], then 2 n slots of g heads x (sum[128], m, l).
__host__ __device__ constexpr size_t recs_bytes(int n) { return (size_t(n) * sizeof(Rec) + 15) / 16 * 16; }
__host__ __device__ constexpr size_t slot_floats(int g) { return size_t(g) * (kD + 2); }

template <int DT>
struct Form {
  static constexpr int kRow = kD * elem_bytes<DT>();       // bytes of a row
  static constexpr int kStages = DT == kE4m3 ? 5 : 3;      // 96 KB (16-bit) or 80 KB of ring per block
  static constexpr int kSlice = 2 * 16 * kRow;             // a warp's K and V rows of a tile
  static constexpr int kRing = kStages * kSlice;
  static constexpr bool kHalf = DT != kBf16;               // operands are FP16
  static constexpr float kShift = kHalf ? 14.0f : 0.0f;    // weights up to 2^14: FP16 parts of small ones stay normal
};

template <int DT>
struct Smem {
  char ring[kWarps][Form<DT>::kRing];
  int mask[Form<DT>::kStages][kWarps];  // bits 0..15: rows that hold a token; bit 16: a refused row
  Prefix<kThreads> prefix;
  float m[kWarps][kMaxGroup], l[kWarps][kMaxGroup];
  float buf[2][1];  // [2][heads][kBufStride], sized at launch
};

template <int DT>
constexpr size_t smem_bytes(int nt) {
  return offsetof(Smem<DT>, buf) + size_t(2) * nt * 8 * kBufStride * 4;
}

__device__ __forceinline__ void copy16(uint32_t dst, const char* src, bool live) {
  const int n = live ? 16 : 0;  // 0: zeros
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void wait_groups() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t a) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a));
}
__device__ __forceinline__ void ldmatrix4_trans(uint32_t (&r)[4], uint32_t a) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a));
}
__device__ __forceinline__ uint4 lds16(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
  return v;
}

template <bool HALF>
__device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1) {
  if constexpr (HALF)
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                 "{%0, %1, %2, %3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                 "{%0, %1, %2, %3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t pack_half(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// (a, b) as parts whose sum is the value: hi, mid, lo of BF16 by cutting eight
// bits off at a time (exact), or hi, lo of FP16 (22 bits).
template <bool HALF>
__device__ __forceinline__ void split(float a, float b, uint32_t (&part)[3]) {
  if constexpr (HALF) {
    part[0] = pack_half(a, b);
    const float2 h = __half22float2(*reinterpret_cast<const __half2*>(&part[0]));
    part[1] = pack_half(a - h.x, b - h.y);
  } else {
#pragma unroll
    for (int i = 0; i < 3; ++i) {
      part[i] = __byte_perm(__float_as_uint(a), __float_as_uint(b), 0x7632);
      a -= __uint_as_float(__float_as_uint(a) & 0xFFFF0000u);
      b -= __uint_as_float(__float_as_uint(b) & 0xFFFF0000u);
    }
  }
}

// Tokens (of the whole cache, or of the selected pages) that a call visits of a
// request: its work is ceil(tokens / 64) tiles per KV head.
template <bool SEL>
__device__ __forceinline__ int span_of(const AttnArgs& a, int T) {
  if (T <= 0) return 0;
  if (!SEL) return T;
  return min(a.n_select, a.c.ps.div(T - 1) + 1) * int(a.c.ps.d);
}

// A position in the concatenated tiles.
template <bool SEL>
struct Cursor {
  int b, h, tile, T, span, tiles;
  __device__ __forceinline__ void load(const AttnArgs& a) {
    T = b < a.B ? checked_len(a.lens, b, a.max_pages, a.c.ps) : 0;
    span = span_of<SEL>(a, T);
    tiles = (span + kTile - 1) / kTile;
  }
  __device__ __forceinline__ void next(const AttnArgs& a) {
    if (++tile < tiles) return;
    tile = 0;
    if (++h < a.c.H) return;
    h = 0;
    do {
      ++b;
      load(a);
    } while (b < a.B && tiles == 0);
  }
};

// Where a lane's row (token lane % 16 of the warp's slice) comes from, looked up in two steps.
struct Row {
  int page;     // step one: page of the request; step two: page of the pool
  int before;   // selection: the entry before
  int place, h, b, T;
  bool live;
  int bad;      // KVQ_PAGED_ERR_* bits
};

template <bool SEL>
__device__ __forceinline__ void look_up_entry(const AttnArgs& a, const Cursor<SEL>& at, int v, Row& r) {
  const int e = a.c.ps.div(v);
  r.place = v - e * int(a.c.ps.d);
  r.h = at.h;
  r.b = at.b;
  r.T = at.T;
  r.live = v < at.span;
  r.bad = 0;
  r.page = e;
  r.before = -1;
  if (SEL && r.live) {
    const int32_t* s = a.sel + ((long long)at.b * a.c.H + at.h) * a.n_select + e;
    r.page = s[0];
    r.before = e > 0 ? s[-1] : -2;  // -2: the list begins here
  }
}

template <bool SEL>
__device__ __forceinline__ void look_up_page(const AttnArgs& a, Row& r) {
  if (SEL && r.live) {
    const int pages = a.c.ps.div(r.T - 1) + 1;  // (a live row's request has tokens)
    const bool ok = r.page == -1 || (r.page >= 0 && r.page < pages && r.page > r.before && r.before != -1);
    if (!ok) r.bad = KVQ_PAGED_ERR_SELECTION;
    r.live = ok && r.page >= 0 && r.page * int(a.c.ps.d) + r.place < r.T;
  }
  r.page = r.live ? a.table[(long long)r.b * a.max_pages + r.page] : 0;
}

template <int DT, int QT, int NT, bool SEL>
struct Block {
  using F = Form<DT>;
  const AttnArgs& a;
  Smem<DT>& S;
  const int lane, warp;
  const uint32_t ring;
  // of the current unit
  uint32_t qa[8][2 * NT];  // query operand: rows lane / 4 (and + 8)
  float o[8][4 * NT];      // running sum: channels 16 j + lane / 4 (+ 8), heads 2 (lane % 4) + {0, 1} (+ 8)
  float m[NT], l[NT], scale[NT];

  __device__ __forceinline__ Block(const AttnArgs& args, Smem<DT>& s)
      : a(args), S(s), lane(threadIdx.x & 31), warp(threadIdx.x >> 5),
        ring(uint32_t(__cvta_generic_to_shared(s.ring[threadIdx.x >> 5]))) {}

  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int j = 0; j < 8; ++j)
#pragma unroll
      for (int i = 0; i < 4 * NT; ++i) o[j][i] = 0.0f;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      m[n] = -INFINITY;
      l[n] = 0.0f;
    }
  }

  // Channels of the query operand of k-step j: 16 j + 2 q + {0, 1, 8, 9} as mma
  // numbers them; for E4M3, where a lane converts 16 consecutive key channels,
  // 16 (q + 4 (j / 4)) + 4 (j % 4) + {0 .. 3}: any order of the sum will do if
  // both operands have it.
  __device__ __forceinline__ void load_query(int b, int h) {
    const int q = lane & 3;
    const float ks = DT == kE4m3 && a.c.k_scale != nullptr ? a.c.k_scale[h] : 1.0f;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int head = lane / 4 + 8 * n;
      const char* p = a.q + (long long)b * a.q_stride + (long long)(h * a.g + head) * (kD * 2);
      scale[n] = a.scale * ks * 1.4426950408889634f;
      float top = 0.0f;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        uint2 w = make_uint2(0, 0);
        if (head < a.g) {
          if constexpr (DT == kE4m3) {
            w = *reinterpret_cast<const uint2*>(p + (16 * (q + 4 * (j / 4)) + 4 * (j % 4)) * 2);
          } else {
            w.x = *reinterpret_cast<const uint32_t*>(p + (16 * j + 2 * q) * 2);
            w.y = *reinterpret_cast<const uint32_t*>(p + (16 * j + 2 * q + 8) * 2);
          }
        }
        qa[j][2 * n] = w.x;
        qa[j][2 * n + 1] = w.y;
        if constexpr (DT == kE4m3 && QT == kBf16) {
          top = fmaxf(top, fmaxf(fabsf(__uint_as_float(w.x << 16)), fabsf(__uint_as_float(w.x & 0xFFFF0000u))));
          top = fmaxf(top, fmaxf(fabsf(__uint_as_float(w.y << 16)), fabsf(__uint_as_float(w.y & 0xFFFF0000u))));
        }
      }
      if constexpr (DT == kE4m3 && QT == kBf16) {  // BF16 to FP16 by a power of two: the largest into [2^7, 2^8)
        top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
        int e = 134 - int(__float_as_uint(top) >> 23);  // 7 - (exponent - 127)
        e = top == 0.0f || isinf(top) ? 0 : max(-120, min(120, e));
        const float f = __uint_as_float(uint32_t(127 + e) << 23);
        scale[n] *= __uint_as_float(uint32_t(127 - e) << 23);
#pragma unroll
        for (int j = 0; j < 8; ++j)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const uint32_t w = qa[j][2 * n + i];
            qa[j][2 * n + i] =
                pack_half(__uint_as_float(w << 16) * f, __uint_as_float(w & 0xFFFF0000u) * f);
          }
      }
    }
  }

  // Copies of a tile's rows of this warp into a stage.
  __device__ __forceinline__ void issue(int stage, const Row& r) {
    const bool in_pool = r.page >= 0 && r.page < a.c.n_pages;
    const bool live = r.live && in_pool;
    const int bad = r.bad | (r.live && !in_pool ? KVQ_PAGED_ERR_PAGE : 0);
    const uint32_t rows = __ballot_sync(0xFFFFFFFFu, live) & 0xFFFFu;
    const uint32_t refused = __ballot_sync(0xFFFFFFFFu, bad != 0);
    if (refused && bad) flag(a.c, bad);
    if (lane == 0) S.mask[stage][warp] = int(rows | (refused ? 0x10000u : 0u));
    const long long off = live ? (long long)r.page * a.c.page_stride + (long long)r.place * a.c.token_stride +
                                     (long long)r.h * a.c.head_stride
                               : -1;
    constexpr int kChunks = F::kRow / 16, kPer = 32 / kChunks;  // 16-byte chunks of a row, rows per instruction
    const uint32_t base = ring + stage * F::kSlice;
    const int chunk = lane % kChunks;
#pragma unroll
    for (int i = 0; i < 16 / kPer; ++i) {
      const int row = i * kPer + lane / kChunks;
      const long long x = __shfl_sync(0xFFFFFFFFu, off, row);
      const long long src = (x < 0 ? 0 : x) + chunk * 16;
      const int kc = DT == kE4m3 ? chunk ^ ((row & 1) << 2) : chunk ^ (row & 7);
      const int vc = DT == kE4m3 ? chunk ^ (((row >> 1) & 3) << 1) : chunk ^ (row & 7);
      copy16(base + row * F::kRow + kc * 16, a.c.k + src, x >= 0);
      copy16(base + 16 * F::kRow + row * F::kRow + vc * 16, a.c.v + src, x >= 0);
    }
  }

  __device__ __forceinline__ void attend(int stage) {
    const uint32_t kb = ring + stage * F::kSlice, vb = kb + 16 * F::kRow;
    const int mask = S.mask[stage][warp];
    // logits: two blocks of eight tokens, even and odd k-steps apart (independent chains)
    float s[2][2][4];
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int i = 0; i < 4; ++i) s[t][e][i] = 0.0f;
    auto qk = [&](int j, int t, uint32_t b0, uint32_t b1) {
      if constexpr (NT == 2) mma<F::kHalf>(s[t][j & 1], qa[j][0], qa[j][2], qa[j][1], qa[j][3], b0, b1);
      else mma<F::kHalf>(s[t][j & 1], qa[j][0], 0u, qa[j][1], 0u, b0, b1);
    };
    const int mr = (lane & 7) + (lane >> 4) * 8, mc = (lane >> 3) & 1;  // the lane's row and chunk of an ldmatrix
    if constexpr (DT != kE4m3) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        uint32_t r[4];
        ldmatrix4(r, kb + mr * 256 + (((2 * j + mc) ^ (mr & 7)) << 4));
        qk(j, 0, r[0], r[1]);
        qk(j, 1, r[2], r[3]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          const int row = t * 8 + lane / 4;
          const uint4 x = lds16(kb + row * 128 + ((((lane & 3) + 4 * i) ^ ((row & 1) << 2)) << 4));
          const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
          for (int j = 0; j < 4; ++j) qk(4 * i + j, t, e4m3x2_to_f16x2(w[j] & 0xFFFFu), e4m3x2_to_f16x2(w[j] >> 16));
        }
    }
    uint32_t part[2][NT][3];  // weights of the two token blocks, split
    float alpha[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      float x[2][2];
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          x[t][i] = (s[t][0][2 * n + i] + s[t][1][2 * n + i]) * scale[n];
          const int row = 8 * t + 2 * (lane & 3) + i;
          if (!((mask >> row) & 1)) x[t][i] = -INFINITY;
        }
      float mx = fmaxf(fmaxf(x[0][0], x[0][1]), fmaxf(x[1][0], x[1][1]));
      mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 1));
      mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 2));
      mx = fmaxf(m[n], mx);
      const float base = mx == -INFINITY ? 0.0f : mx;
      alpha[n] = exp2f(m[n] - base);
      m[n] = mx;
      float sum = 0.0f;
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        const float p0 = exp2f(x[t][0] - base + F::kShift), p1 = exp2f(x[t][1] - base + F::kShift);
        sum += p0 + p1;
        split<F::kHalf>(p0, p1, part[t][n]);
      }
      l[n] = l[n] * alpha[n] + sum;
      if (mask & 0x10000) l[n] = NAN;  // a refused row: the whole unit's result is NaN
    }
    float f[NT][2];  // rescaling of the heads whose sums this lane holds
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int i = 0; i < 2; ++i) f[n][i] = __shfl_sync(0xFFFFFFFFu, alpha[n], (2 * (lane & 3) + i) * 4);
    auto pv = [&](int j, const uint32_t (&v)[4]) {
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        float c[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int i = F::kHalf ? 1 : 2; i >= 0; --i)
          mma<F::kHalf>(c, v[0], v[1], v[2], v[3], part[0][n][i], part[1][n][i]);
#pragma unroll
        for (int i = 0; i < 4; ++i) o[j][4 * n + i] = o[j][4 * n + i] * f[n][i & 1] + c[i];
      }
    };
    if constexpr (DT != kE4m3) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        uint32_t v[4];
        ldmatrix4_trans(v, vb + mr * 256 + (((2 * j + mc) ^ (mr & 7)) << 4));
        pv(j, v);
      }
    } else {
      // the lane's 16 channels (chunk lane / 4) of its four tokens 2q, 2q + 1, 2q + 8, 2q + 9; the operand of step j
      // takes channels 2j and 2j + 1 of them as its rows lane / 4 and lane / 4 + 8
      uint4 x[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int row = 2 * (lane & 3) + (i & 1) + 8 * (i >> 1);
        x[i] = lds16(vb + row * 128 + (((lane >> 2) ^ (((row >> 1) & 3) << 1)) << 4));
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const uint32_t w[4] = {(&x[0].x)[k], (&x[1].x)[k], (&x[2].x)[k], (&x[3].x)[k]};
        const uint32_t lo0 = __byte_perm(w[0], w[1], 0x5140), hi0 = __byte_perm(w[0], w[1], 0x7362);
        const uint32_t lo1 = __byte_perm(w[2], w[3], 0x5140), hi1 = __byte_perm(w[2], w[3], 0x7362);
        const uint32_t even[4] = {e4m3x2_to_f16x2(lo0 & 0xFFFFu), e4m3x2_to_f16x2(lo0 >> 16),
                                  e4m3x2_to_f16x2(lo1 & 0xFFFFu), e4m3x2_to_f16x2(lo1 >> 16)};
        const uint32_t odd[4] = {e4m3x2_to_f16x2(hi0 & 0xFFFFu), e4m3x2_to_f16x2(hi0 >> 16),
                                 e4m3x2_to_f16x2(hi1 & 0xFFFFu), e4m3x2_to_f16x2(hi1 >> 16)};
        pv(2 * k, even);
        pv(2 * k + 1, odd);
      }
    }
  }

  // Channels of o[j]: c = 0 (rows lane / 4) and 1 (rows lane / 4 + 8).
  __device__ __forceinline__ int channel(int j, int c) const {
    return DT == kE4m3 ? 16 * (lane >> 2) + 2 * j + c : 16 * j + (lane >> 2) + 8 * c;
  }

  // The block's four warps joined; the result goes to out and lse, or to `slot`.
  __device__ __forceinline__ void finish(int b, int h, float* slot) {
    float* buf = reinterpret_cast<float*>(reinterpret_cast<char*>(&S) + offsetof(Smem<DT>, buf));
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      l[n] += __shfl_xor_sync(0xFFFFFFFFu, l[n], 1);
      l[n] += __shfl_xor_sync(0xFFFFFFFFu, l[n], 2);
      if ((lane & 3) == 0) {
        S.m[warp][lane / 4 + 8 * n] = m[n];
        S.l[warp][lane / 4 + 8 * n] = l[n];
      }
    }
    __syncthreads();
    auto top = [&](int head) {
      const float x = fmaxf(fmaxf(S.m[0][head], S.m[1][head]), fmaxf(S.m[2][head], S.m[3][head]));
      return x == -INFINITY ? 0.0f : x;
    };
    constexpr int kHeads = 8 * NT;
    float f[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int head = 2 * (lane & 3) + i + 8 * n;
        f[n][i] = exp2f(S.m[warp][head] - top(head));
      }
    float* mine = buf + (warp & 1) * kHeads * kBufStride;
    auto at = [&](int j, int i) -> float& {  // i = 4 n + 2 c + head bit
      return mine[(2 * (lane & 3) + (i & 1) + 8 * (i >> 2)) * kBufStride + channel(j, (i >> 1) & 1)];
    };
    if (warp >= 2) {
#pragma unroll
      for (int j = 0; j < 8; ++j)
#pragma unroll
        for (int i = 0; i < 4 * NT; ++i) at(j, i) = o[j][i] * f[i >> 2][i & 1];
    }
    __syncthreads();
    if (warp < 2) {
#pragma unroll
      for (int j = 0; j < 8; ++j)
#pragma unroll
        for (int i = 0; i < 4 * NT; ++i) at(j, i) += o[j][i] * f[i >> 2][i & 1];
    }
    __syncthreads();
    const int c = threadIdx.x;
    const float vs = DT == kE4m3 && a.c.v_scale != nullptr ? a.c.v_scale[h] : 1.0f;
    for (int j = 0; j < a.g; ++j) {
      const float mx = top(j);
      float sum = 0.0f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) sum += S.l[w][j] * exp2f(S.m[w][j] - mx);
      const float x = buf[j * kBufStride + c] + buf[(kHeads + j) * kBufStride + c];
      const bool none = fmaxf(fmaxf(S.m[0][j], S.m[1][j]), fmaxf(S.m[2][j], S.m[3][j])) == -INFINITY;
      const float at_m = none ? -INFINITY : mx - F::kShift;
      if (slot != nullptr) {
        slot[j * kD + c] = x * vs;
        if (c == 0) {
          slot[a.g * kD + 2 * j] = at_m;
          slot[a.g * kD + 2 * j + 1] = sum;
        }
      } else {
        const long long hq = (long long)b * a.Hq + h * a.g + j;
        a.out[hq * kD + c] = sum == 0.0f ? 0.0f : x * vs / sum;
        if (a.lse != nullptr && c == 0) a.lse[hq] = (at_m + log2f(sum)) * 0.6931471805599453f;
      }
    }
    __syncthreads();  // m, l and buf are free again
  }
};

template <int DT, int QT, int NT, bool SEL>
__global__ void __launch_bounds__(kThreads, kBlocksPerSm) attn_kernel(AttnArgs a) {
  using F = Form<DT>;
  extern __shared__ __align__(16) char smem[];
  Smem<DT>& S = *reinterpret_cast<Smem<DT>*>(smem);
  allow_dependents();
  const int c = blockIdx.x, n_ctas = gridDim.x;
  Rec* recs = reinterpret_cast<Rec*>(a.ws);
  float* slots = reinterpret_cast<float*>(a.ws + recs_bytes(n_ctas));
  if (threadIdx.x == 0) recs[c] = Rec{-1, 0};

  auto tiles_of = [&](int b) {
    return (long long)a.c.H * ((span_of<SEL>(a, checked_len(a.lens, b, a.max_pages, a.c.ps)) + kTile - 1) / kTile);
  };
  build_prefix<kThreads>(S.prefix, a.B, tiles_of);
  // requests without tokens, and refused ones: no block's range holds them
  for (int b = c; b < a.B; b += n_ctas) {
    const int T = checked_len(a.lens, b, a.max_pages, a.c.ps);
    if (T > 0) continue;
    const float x = T < 0 ? NAN : 0.0f;
    for (int i = threadIdx.x; i < a.Hq * kD; i += kThreads) a.out[(long long)b * a.Hq * kD + i] = x;
    if (a.lse != nullptr)
      for (int i = threadIdx.x; i < a.Hq; i += kThreads) a.lse[(long long)b * a.Hq + i] = T < 0 ? NAN : -INFINITY;
    if (T < 0 && threadIdx.x == 0) flag(a.c, KVQ_PAGED_ERR_LENGTH);
  }
  const long long W = S.prefix.pre[kThreads];
  const int C = int(W < n_ctas ? W : n_ctas);  // ranges: none is empty, so the parts of a unit are those of adjacent blocks
  if (c >= C) return;
  const long long s0 = cta_start(c, W, C), e0 = cta_start(c + 1, W, C);

  Cursor<SEL> at, ahead;
  long long in_request = s0;
  at.b = find_request<kThreads>(S.prefix, a.B, tiles_of, in_request);
  at.load(a);
  at.h = int(in_request / at.tiles);
  at.tile = int(in_request % at.tiles);
  ahead = at;

  Block<DT, QT, NT, SEL> K(a, S);
  const int row = K.warp * 16 + (K.lane & 15);
  const int n = int(e0 - s0);
  Row entry, page;  // looked up one step, and both
  bool fresh = true;
  // tile i: its selection entry is looked up at i - kStages - 1, its page at i - kStages, its copies issued at
  // i - kStages + 1
  for (int i = -F::kStages - 1; i < n; ++i) {
    if (i >= 0) {
      wait_groups<F::kStages - 2>();
      __syncwarp();  // every lane's copies have landed, and every lane has left the stage that is filled next
    }
    const int filled = i + F::kStages - 1;
    if (filled >= 0) {
      if (filled < n) K.issue(filled % F::kStages, page);
      commit();
    }
    if (filled + 1 >= 0 && filled + 1 < n) {
      page = entry;
      look_up_page<SEL>(a, page);
    }
    if (filled + 2 < n) {
      look_up_entry<SEL>(a, ahead, ahead.tile * kTile + row, entry);
      ahead.next(a);
    }
    if (i < 0) continue;
    if (fresh) {
      K.load_query(at.b, at.h);
      K.clear();
      fresh = false;
    }
    __syncwarp();  // the stage's mask
    K.attend(i % F::kStages);
    if (at.tile + 1 == at.tiles || i + 1 == n) {
      const long long ue = s0 + i + (at.tiles - at.tile), us = ue - at.tiles;  // the unit's tiles
      float* slot = nullptr;
      if (us < s0 || ue > e0) {
        slot = slots + size_t(2 * c + (us < s0 ? 0 : 1)) * slot_floats(a.g);
        if (us >= s0 && threadIdx.x == 0) recs[c] = Rec{at.b * a.c.H + at.h, cta_of(ue - 1, W, C)};
      }
      K.finish(at.b, at.h, slot);
      fresh = true;
    }
    at.next(a);
  }
}

// Joins the parts of a unit that several blocks' ranges share; block (c, j): the
// unit that starts in range c, query head j of its group. Four groups of 128
// threads take every fourth part.
__global__ void __launch_bounds__(kCombineThreads) combine_kernel(AttnArgs a, int n_ctas) {
  __shared__ float s_top[kCombineThreads / 32], s_l[4], s_x[4][kD];
  wait_prior_grid();
  const int c = blockIdx.x, j = blockIdx.y, ch = threadIdx.x & 127, grp = threadIdx.x >> 7;
  const Rec r = reinterpret_cast<const Rec*>(a.ws)[c];
  if (r.u < 0) return;
  const float* slots = reinterpret_cast<const float*>(a.ws + recs_bytes(n_ctas));
  const int parts = r.last - c + 1;  // slot 2 c + 1 of block c, slot 2 c' of the following
  auto part = [&](int i) { return slots + size_t(i == 0 ? 2 * c + 1 : 2 * (c + i)) * slot_floats(a.g); };
  float top = -INFINITY;
  for (int i = threadIdx.x; i < parts; i += kCombineThreads) top = fmaxf(top, part(i)[a.g * kD + 2 * j]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
  if ((threadIdx.x & 31) == 0) s_top[threadIdx.x >> 5] = top;
  __syncthreads();
  for (int w = 0; w < kCombineThreads / 32; ++w) top = fmaxf(top, s_top[w]);
  const float base = top == -INFINITY ? 0.0f : top;
  float l = 0.0f, x = 0.0f;
#pragma unroll 4
  for (int i = grp; i < parts; i += 4) {
    const float* p = part(i);
    const float f = exp2f(p[a.g * kD + 2 * j] - base);
    l += p[a.g * kD + 2 * j + 1] * f;
    x += p[j * kD + ch] * f;
  }
  s_x[grp][ch] = x;
  if (ch == 0) s_l[grp] = l;
  __syncthreads();
  if (grp != 0) return;
  l = (s_l[0] + s_l[1]) + (s_l[2] + s_l[3]);
  x = (s_x[0][ch] + s_x[1][ch]) + (s_x[2][ch] + s_x[3][ch]);
  const int b = r.u / a.c.H, h = r.u % a.c.H;
  const long long hq = (long long)b * a.Hq + h * a.g + j;
  a.out[hq * kD + ch] = l == 0.0f ? 0.0f : x / l;
  if (a.lse != nullptr && ch == 0) a.lse[hq] = (top + log2f(l)) * 0.6931471805599453f;
}

int blocks_of(int sms) { return sms * kBlocksPerSm; }

template <int DT, int QT, int NT, bool SEL>
cudaError_t launch_form(const AttnArgs& a, cudaStream_t stream) {
  const int smem = int(smem_bytes<DT>(NT)), n = blocks_of(a.sms);
  static std::atomic<uint64_t> configured{0};  // bit: device
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (!((configured.load(std::memory_order_relaxed) >> dev) & 1)) {
    e = cudaFuncSetAttribute(attn_kernel<DT, QT, NT, SEL>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    configured.fetch_or(uint64_t(1) << dev, std::memory_order_relaxed);
  }
  attn_kernel<DT, QT, NT, SEL><<<n, kThreads, smem, stream>>>(a);
  count_launch();
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  count_launch();
  return launch_dependent(combine_kernel, dim3(n, a.g), dim3(kCombineThreads), 0, stream, a, n);
}

template <int DT, int QT>
cudaError_t launch_types(const AttnArgs& a, cudaStream_t stream) {
  if (a.sel != nullptr) return a.g <= 8 ? launch_form<DT, QT, 1, true>(a, stream) : launch_form<DT, QT, 2, true>(a, stream);
  return a.g <= 8 ? launch_form<DT, QT, 1, false>(a, stream) : launch_form<DT, QT, 2, false>(a, stream);
}

}  // namespace

size_t attn_workspace(int B, int H, int Hq, int sms) {
  return recs_bytes(blocks_of(sms)) + 2 * size_t(blocks_of(sms)) * slot_floats(Hq / H) * 4;
}

cudaError_t launch_attn(const AttnArgs& a, cudaStream_t stream) {
  const bool bf = a.q_dtype == kBf16;
  if (a.dtype == kBf16) return launch_types<kBf16, kBf16>(a, stream);
  if (a.dtype == kFp16) return launch_types<kFp16, kFp16>(a, stream);
  return bf ? launch_types<kE4m3, kBf16>(a, stream) : launch_types<kE4m3, kFp16>(a, stream);
}

}  // namespace paged
}  // namespace kvq
