// kvq_paged_attn.cu — decode attention of one query per request over a paged
// cache, all pages or the selected ones.
//
// s_t = scale q.k_t, out = sum_t e^(s_t - m) v_t / l, lse = m + ln l, in one pass
// over the cache with a running maximum m and sum l per query head.
//
// Bound: HBM. A token and KV head bring 4 D bytes (16-bit) for 4 D g flops, so a
// block must keep loads in flight and spend few instructions a byte.
//
// Work: L blocks side by side have H / L heads each of the same tokens (a token's
// heads lie side by side in a token-major pool: read at about the same time they
// are whole DRAM pages). The tiles (64 or 128 tokens) of a lane's (request, KV
// head) units, concatenated, are cut into equal ranges, one per block of the lane
// (two blocks an SM); lengths are read on the device, so a captured call follows
// them. A unit that lies in one block's range is finished there; of the others each
// block leaves (m, l, sum) in one of its two slots, and the combine kernel joins
// them. (Joined in the same launch, by the block that finds the flags of all parts
// set, they took longer in every case: 10.1 against 8.7 us for one request of 256
// tokens, 97.8 against 90.2 us for 4 x 32768 and eight query heads: the fences and
// flags come to more than a second launch that is already waiting.)
//
// A warp owns 16 tokens of every tile and a ring of its own in shared memory,
// filled by 16-byte asynchronous copies, so that the main loop has no block
// barrier. Row addresses (selection, page table) are looked up one and two tiles
// ahead of their copies. Rows without a token are filled with zeros.
//
// QK^T with the heads as the 16 rows of mma.m16n8k16 and the tokens as columns:
// its result then is, register for register, the transposed operand of the second
// product out^T = V^T P^T, so the softmax weights never leave their lane.
// Exactness: products of 16-bit values are exact; P is split into parts, because one 8-
// or 11-bit P would cost 2^-9 or 2^-12 of the FP32 result: three of BF16, whose sum is
// P, or two of FP16, which leave out 2^-23 of a weight or 2^-39 of the unit's largest,
// whichever is more (of the product alone: the weights' sum is FP32's). A third part of
// FP16 would be half as many products again for less than FP32 sums lose anyway. The tensor
// cores cut their sums off, so every 16 tokens' product starts from zero and is added to
// the running sum by FP32 FMA, which also applies the rescaling.
// E4M3: keys and values become FP16 in registers (exact). A BF16 query becomes FP16 by
// a power of two per head that brings its largest channel into [2^15, 2^16): exact
// down to 2^-17, where FP16's step of 2^-24 is the last of eight bits. A head with a
// channel below that, 2^-32 of its largest (beside one that meets zero keys it may be
// all that counts), is found by the attention kernel (WideHeads) and attended again by
// FP32 multiply-adds, by the combine kernel: a branch or a call for such heads in the
// attention kernel's loop cost all others 1 to 30%, by the registers that it moved.
#include <atomic>

#include "kvq_attn_common.cuh"
#include "kvq_paged.cuh"

namespace kvq {
namespace paged {
namespace {

constexpr int kThreads = 128;
constexpr int kWarps = 4;
constexpr int kBufStride = 132;    // floats per head of the merge buffers: the lanes' columns hit distinct banks
constexpr int kBlocksPerSm = 2;
constexpr int kCombineThreads = 512;
constexpr int kCombineWarps = kCombineThreads / 32;
constexpr int kUnitCost = 2;       // tiles that the end of a unit takes as long as
constexpr int kMinTiles = 2;       // tiles of a block's range, once every SM has one

template <int DT, int QT>
constexpr bool kNarrow = DT == kE4m3 && QT == kBf16;  // the query becomes narrower: BF16 to FP16
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// A unit that several blocks share: the first of them and how many, `lanes` apart (u
// < 0: no such unit). Where there are no more units than blocks, unit u's is number
// u, else the one of the unit that starts in block c's range and goes on behind it
// number c.
struct Rec {
  int32_t u, first, parts, pad;
};
__host__ __device__ constexpr bool rec_per_unit(long long units, int n_ctas) { return units <= n_ctas; }

// Workspace: Rec[n], then 2 n slots of g heads x sum[128] and g x (m, l), then a byte per unit and head
// (wide_heads).
__host__ __device__ constexpr size_t slots_offset(int n) { return (size_t(n) * sizeof(Rec) + 15) / 16 * 16; }
__host__ __device__ constexpr size_t slot_floats(int g) { return size_t(g) * kD + (size_t(g) + 1) / 2 * 4; }  // (16-byte steps)

template <int DT>
struct Form {
  static constexpr int kRow = kD * elem_bytes<DT>();       // bytes of a row
  // blocks of 16 tokens in a warp's slice of a tile: 8 KB (E4M3 with one: 106 us instead of 89 for 64 ragged requests,
  // by three blocks an SM too: the softmax's own instructions come twice as often)
  static constexpr int kSteps = DT == kE4m3 ? 2 : 1;
  static constexpr int kRows = 16 * kSteps;
  static constexpr int kTile = kRows * kWarps;             // tokens per tile
  static constexpr int kStages = 3;                        // 96 KB of ring per block
  static constexpr int kSlice = 2 * kRows * kRow;          // a warp's K and V rows of a tile
  static constexpr int kRing = kStages * kSlice;
  static constexpr bool kHalf = DT != kBf16;               // operands are FP16
  static constexpr float kShift = kHalf ? 14.0f : 0.0f;    // weights up to 2^14: FP16 parts of small ones stay normal
};

template <int DT>
struct Smem {
  char ring[kWarps][Form<DT>::kRing];
  uint32_t mask[Form<DT>::kStages][kWarps];  // bit i: row i of the slice holds a token
  int refused[Form<DT>::kStages][kWarps];    // a row that the request or selection does not allow
  Prefix<kThreads> prefix;
  float m[kWarps][kMaxGroup], l[kWarps][kMaxGroup];
  float top[kMaxGroup], sum[kMaxGroup], factor[kMaxGroup];
  float buf[2 * 8 * kBufStride];  // sums of two warps, eight heads
};

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

// 2^x; results below 2^-126 are 0.
__device__ __forceinline__ float exp2_ftz(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// Four E4M3 values as two FP16 pairs (exact).
__device__ __forceinline__ void e4m3x4_to_f16(uint32_t w, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\t"
      "cvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(w));
}

__device__ __forceinline__ uint32_t pack_half(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// (a, b) as parts: hi, mid, lo of BF16 by cutting eight bits off at a time (their sum
// is the value), or hi, lo of FP16 (22 bits of it).
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
// request: its work is ceil(tokens / tile) tiles per KV head.
template <bool SEL>
__device__ __forceinline__ int span_of(const AttnArgs& a, int T) {
  if (T <= 0) return 0;
  if (!SEL) return T;
  return min(a.n_select, a.c.ps.div(T - 1) + 1) * int(a.c.ps.d);
}

// A position in the concatenated work: a unit is its tiles and kUnitCost more
// positions that stand for its merge and its query's load, so that a range of many
// short units is not longer than one of few long ones.
template <bool SEL, int TILE>
struct Cursor {
  int b, h, tile, T, span, tiles;
  long long pos;
  __device__ __forceinline__ void load(const AttnArgs& a) {
    T = b < a.B ? checked_len(a.lens, b, a.max_pages, a.c.ps) : 0;
    span = span_of<SEL>(a, T);
    tiles = (span + TILE - 1) / TILE;
  }
  __device__ __forceinline__ void next_unit(const AttnArgs& a, int h0) {  // h0: first of the lane's heads
    pos += tiles + kUnitCost - tile;
    tile = 0;
    if (++h < h0 + a.lane_heads) return;
    h = h0;
    do {
      ++b;
      load(a);
    } while (b < a.B && tiles == 0);
  }
  __device__ __forceinline__ void next(const AttnArgs& a, int h0) {
    if (tile + 1 == tiles) {
      next_unit(a, h0);
    } else {
      ++tile;
      ++pos;
    }
  }
  __device__ __forceinline__ bool before(const AttnArgs& a, long long end) const { return b < a.B && pos < end; }
};

// Where a lane's row (of the warp's slice) comes from, looked up in two steps.
struct Row {
  int page;     // step one: page of the request; step two: page of the pool
  int before;   // selection: the entry before
  int place, h, b, T;
  bool live;
  int bad;      // KVQ_PAGED_ERR_* bits
};

template <bool SEL, int TILE>
__device__ __forceinline__ void look_up_entry(const AttnArgs& a, const Cursor<SEL, TILE>& at, int v, Row& r) {
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

// The power of two that brings a BF16 number of this magnitude into [2^15, 2^16).
__device__ __forceinline__ int query_shift(float top) {
  const int e = 127 + 15 - int(__float_as_uint(top) >> 23);
  return top == 0.0f || isinf(top) ? 0 : max(-120, min(120, e));
}
__device__ __forceinline__ float power_of_two(int e) { return __uint_as_float(uint32_t(127 + e) << 23); }

// Query heads that FP16 does not hold: a byte per head that is not 0, kMaxGroup bytes per unit, behind the slots.
__device__ __forceinline__ uint8_t* wide_heads(const AttnArgs& a, int n) {
  return reinterpret_cast<uint8_t*>(a.ws + slots_offset(n) + 2 * size_t(n) * slot_floats(a.g) * 4);
}

// Finds the BF16 query heads that FP16 does not hold whole: those with a channel below 2^-17 by their power of two, or
// one that is infinite (beside which others may overflow). Block c takes the units c, c + n, ..., eight lanes a head.
struct WideHeads {
  static constexpr int kLanes = 8, kOwn = 2, kHeads = kOwn * kThreads / kLanes;
  uint4 w[kOwn][2];
  __device__ __forceinline__ static int pairs(const AttnArgs& a, int c, int n) {
    const int units = a.B * a.c.H;
    return c < units ? ((units - c + n - 1) / n) * a.g : 0;
  }
  __device__ __forceinline__ static void place(const AttnArgs& a, int c, int n, int p, int& u, int& j) {
    u = p / a.g;
    j = p - u * a.g;
    u = c + u * n;
  }
  __device__ __forceinline__ void load(const AttnArgs& a, int c, int n, int pairs, int at) {
#pragma unroll
    for (int e = 0; e < kOwn; ++e) {
      const int p = at + (e * kThreads + threadIdx.x) / kLanes;
      w[e][0] = w[e][1] = make_uint4(0u, 0u, 0u, 0u);
      if (p >= pairs) continue;
      int u, j;
      place(a, c, n, p, u, j);
      const int b = u / a.c.H, h = u - b * a.c.H;
      const char* q = a.q + (long long)b * a.q_stride + (long long)(h * a.g + j) * (kD * 2) + threadIdx.x % kLanes * 16;
      w[e][0] = *reinterpret_cast<const uint4*>(q);
      w[e][1] = *reinterpret_cast<const uint4*>(q + kD);
    }
  }
  __device__ __forceinline__ void store(const AttnArgs& a, int c, int n, int pairs, int at) const {
#pragma unroll
    for (int e = 0; e < kOwn; ++e) {
      float top = 0.0f, low = INFINITY;  // magnitudes: the largest, and the smallest that is not 0
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const uint32_t v = (&w[e][i / 8].x)[i / 2 % 4];
        const float x = fabsf(__uint_as_float(i & 1 ? v & 0xFFFF0000u : v << 16));
        top = fmaxf(top, x);
        low = fminf(low, x == 0.0f ? INFINITY : x);
      }
#pragma unroll
      for (int o = 1; o < kLanes; o *= 2) {
        top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
        low = fminf(low, __shfl_xor_sync(0xFFFFFFFFu, low, o));
      }
      const int p = at + (e * kThreads + threadIdx.x) / kLanes;
      if (p >= pairs || threadIdx.x % kLanes != 0) continue;
      int u, j;
      place(a, c, n, p, u, j);
      wide_heads(a, n)[u * kMaxGroup + j] = isinf(top) || low * power_of_two(query_shift(top)) < 0x1p-17f;
    }
  }
};

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
  __device__ __forceinline__ uint2 query_words(const char* p, int j) const {
    const int q = lane & 3;
    if constexpr (DT == kE4m3)
      return *reinterpret_cast<const uint2*>(p + (16 * (q + 4 * (j / 4)) + 4 * (j % 4)) * 2);
    else
      return make_uint2(*reinterpret_cast<const uint32_t*>(p + (16 * j + 2 * q) * 2),
                        *reinterpret_cast<const uint32_t*>(p + (16 * j + 2 * q + 8) * 2));
  }
  // scale ks 2^shift, whose parts may leave FP32's range where the logits do not (a scale of 0 would make a masked
  // place's logit NaN; with 2^-149 no logit is off by more than 2^-116).
  __device__ __forceinline__ static float scaled(float scale, float ks, int shift) {
    const uint32_t k = __float_as_uint(ks);
    const float x = ldexpf(scale * __uint_as_float((k & 0x7FFFFFu) | 0x3F800000u), int(k >> 23) - 127 + shift);
    return fminf(fmaxf(x, 0x1p-149f), 3.402823466e38f);
  }
  __device__ __forceinline__ void load_query(int b, int h) {
    const float ks = DT == kE4m3 && a.c.k_scale != nullptr ? a.c.k_scale[h] : 1.0f;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int head = lane / 4 + 8 * n;
      const char* p = a.q + (long long)b * a.q_stride + (long long)(h * a.g + head) * (kD * 2);
      scale[n] = a.scale * kLog2e;
      int shift = 0;
      float top = 0.0f;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const uint2 w = head < a.g ? query_words(p, j) : make_uint2(0, 0);
        qa[j][2 * n] = w.x;
        qa[j][2 * n + 1] = w.y;
        if constexpr (kNarrow<DT, QT>) {
          top = fmaxf(top, fmaxf(fabsf(__uint_as_float(w.x << 16)), fabsf(__uint_as_float(w.x & 0xFFFF0000u))));
          top = fmaxf(top, fmaxf(fabsf(__uint_as_float(w.y << 16)), fabsf(__uint_as_float(w.y & 0xFFFF0000u))));
        }
      }
      if constexpr (kNarrow<DT, QT>) {  // BF16 to FP16 by a power of two
        top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
        const int e = query_shift(top);
        const float f = power_of_two(e);
        shift = -e;
#pragma unroll
        for (int j = 0; j < 8; ++j)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const uint32_t w = qa[j][2 * n + i];
            qa[j][2 * n + i] = pack_half(__uint_as_float(w << 16) * f, __uint_as_float(w & 0xFFFF0000u) * f);
          }
      }
      if constexpr (DT == kE4m3) scale[n] = scaled(scale[n], ks, shift);
    }
  }

  // Copies of a tile's rows of this warp into a stage.
  __device__ __forceinline__ void issue(int stage, const Row& r) {
    const bool in_pool = r.page >= 0 && r.page < a.c.n_pages;
    const bool live = r.live && in_pool;
    const int bad = r.bad | (r.live && !in_pool ? KVQ_PAGED_ERR_PAGE : 0);
    const uint32_t rows = __ballot_sync(0xFFFFFFFFu, live) & (0xFFFFFFFFu >> (32 - F::kRows));
    const uint32_t refused = __ballot_sync(0xFFFFFFFFu, bad != 0);
    if (refused && bad) flag(a.c, bad);
    if (lane == 0) {
      S.mask[stage][warp] = rows;
      S.refused[stage][warp] = refused != 0;
    }
    const long long off = live ? (long long)r.page * a.c.page_stride + (long long)r.place * a.c.token_stride +
                                     (long long)r.h * a.c.head_stride
                               : -1;
    constexpr int kChunks = F::kRow / 16, kPer = 32 / kChunks;  // 16-byte chunks of a row, rows per instruction
    const uint32_t base = ring + stage * F::kSlice;
    const int chunk = lane % kChunks;
#pragma unroll
    for (int i = 0; i < F::kRows / kPer; ++i) {
      const int row = i * kPer + lane / kChunks;
      const long long x = __shfl_sync(0xFFFFFFFFu, off, row);
      const long long src = (x < 0 ? 0 : x) + chunk * 16;
      const int kc = DT == kE4m3 ? chunk ^ ((row & 1) << 2) : chunk ^ (row & 7);
      const int vc = DT == kE4m3 ? chunk ^ (((row >> 1) & 3) << 1) : chunk ^ (row & 7);
      copy16(base + row * F::kRow + kc * 16, a.c.k + src, x >= 0);
      copy16(base + F::kRows * F::kRow + row * F::kRow + vc * 16, a.c.v + src, x >= 0);
    }
  }

  __device__ __forceinline__ void attend(int stage) {
    constexpr int kBlocks = 2 * F::kSteps;            // of eight tokens
    constexpr int kChains = F::kSteps == 1 ? 2 : 1;   // even and odd k-steps apart, so that four chains run at once
    const uint32_t kb = ring + stage * F::kSlice, vb = kb + F::kRows * F::kRow;
    float s[kBlocks][kChains][4];
#pragma unroll
    for (int t = 0; t < kBlocks; ++t)
#pragma unroll
      for (int e = 0; e < kChains; ++e)
#pragma unroll
        for (int i = 0; i < 4; ++i) s[t][e][i] = 0.0f;
    auto qk = [&](int j, int t, uint32_t b0, uint32_t b1) {
      if constexpr (NT == 2) mma<F::kHalf>(s[t][j % kChains], qa[j][0], qa[j][2], qa[j][1], qa[j][3], b0, b1);
      else mma<F::kHalf>(s[t][j % kChains], qa[j][0], 0u, qa[j][1], 0u, b0, b1);
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
        for (int t = 0; t < kBlocks; ++t) {
          const int row = t * 8 + lane / 4;
          const uint4 x = lds16(kb + row * 128 + ((((lane & 3) + 4 * i) ^ ((row & 1) << 2)) << 4));
          const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            uint32_t b0, b1;
            e4m3x4_to_f16(w[j], b0, b1);
            qk(4 * i + j, t, b0, b1);
          }
        }
    }
    const uint32_t mask = S.mask[stage][warp];
    if (mask != (0xFFFFFFFFu >> (32 - F::kRows))) {  // some rows hold no token
#pragma unroll
      for (int t = 0; t < kBlocks; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (!((mask >> (8 * t + 2 * (lane & 3) + (i & 1))) & 1)) {
            s[t][0][i] = -INFINITY;
            if constexpr (kChains == 2) s[t][1][i] = 0.0f;  // (an infinite query times the zeros there is NaN)
          }
    }
    uint32_t part[kBlocks][NT][3];  // the weights, split
    float alpha[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      float mx = -INFINITY;
#pragma unroll
      for (int t = 0; t < kBlocks; ++t)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          if constexpr (kChains == 2) s[t][0][2 * n + i] += s[t][1][2 * n + i];
          mx = fmaxf(mx, s[t][0][2 * n + i]);
        }
      mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 1));
      mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 2));
      mx = fmaxf(m[n], mx * scale[n]);  // (scale > 0)
      const float base = mx == -INFINITY ? 0.0f : mx;
      alpha[n] = exp2_ftz(m[n] - base);
      m[n] = mx;
      float sum = 0.0f;
#pragma unroll
      for (int t = 0; t < kBlocks; ++t) {
        const float p0 = exp2_ftz(fmaf(s[t][0][2 * n], scale[n], F::kShift - base));
        const float p1 = exp2_ftz(fmaf(s[t][0][2 * n + 1], scale[n], F::kShift - base));
        sum += p0 + p1;
        split<F::kHalf>(p0, p1, part[t][n]);
      }
      l[n] = fmaf(l[n], alpha[n], sum);
      if (S.refused[stage][warp]) l[n] = NAN;  // the whole unit's result is NaN
    }
    float f[NT][2];  // rescaling of the heads whose sums this lane holds
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int i = 0; i < 2; ++i) f[n][i] = __shfl_sync(0xFFFFFFFFu, alpha[n], (2 * (lane & 3) + i) * 4);
    // products of values and weights of 16 tokens (step k), the small parts first
    auto pv = [&](float (&c)[4], int k, int n, const uint32_t (&v)[4]) {
#pragma unroll
      for (int i = F::kHalf ? 1 : 2; i >= 0; --i)
        mma<F::kHalf>(c, v[0], v[1], v[2], v[3], part[2 * k][n][i], part[2 * k + 1][n][i]);
    };
    auto add = [&](int j, int n, const float (&c)[4]) {
#pragma unroll
      for (int i = 0; i < 4; ++i) o[j][4 * n + i] = fmaf(o[j][4 * n + i], f[n][i & 1], c[i]);
    };
    if constexpr (DT != kE4m3) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        uint32_t v[4];
        ldmatrix4_trans(v, vb + mr * 256 + (((2 * j + mc) ^ (mr & 7)) << 4));
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          float c[4] = {0.0f, 0.0f, 0.0f, 0.0f};
          pv(c, 0, n, v);
          add(j, n, c);
        }
      }
    } else {
      // the lane's 16 channels (chunk lane / 4) of its four tokens 2q, 2q + 1, 2q + 8, 2q + 9 of a step; the operand
      // of product j takes channels 2j and 2j + 1 of them as its rows lane / 4 and lane / 4 + 8
      uint4 x[F::kSteps][4];
#pragma unroll
      for (int k = 0; k < F::kSteps; ++k)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int row = 16 * k + 2 * (lane & 3) + (i & 1) + 8 * (i >> 1);
          x[k][i] = lds16(vb + row * 128 + (((lane >> 2) ^ (((row >> 1) & 3) << 1)) << 4));
        }
#pragma unroll
      for (int w = 0; w < 4; ++w) {  // four channels: products 2 w and 2 w + 1
        uint32_t v[F::kSteps][2][4];
#pragma unroll
        for (int k = 0; k < F::kSteps; ++k) {
          const uint32_t y[4] = {(&x[k][0].x)[w], (&x[k][1].x)[w], (&x[k][2].x)[w], (&x[k][3].x)[w]};
#pragma unroll
          for (int i = 0; i < 2; ++i) {  // tokens 2q, 2q + 1 and 2q + 8, 2q + 9
            e4m3x4_to_f16(__byte_perm(y[2 * i], y[2 * i + 1], 0x5140), v[k][0][2 * i], v[k][0][2 * i + 1]);
            e4m3x4_to_f16(__byte_perm(y[2 * i], y[2 * i + 1], 0x7362), v[k][1][2 * i], v[k][1][2 * i + 1]);
          }
        }
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            float c[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int k = 0; k < F::kSteps; ++k) pv(c, k, n, v[k][i]);
            add(2 * w + i, n, c);
          }
      }
    }
  }

  // Channels of o[j]: c = 0 (rows lane / 4) and 1 (rows lane / 4 + 8).
  __device__ __forceinline__ int channel(int j, int c) const {
    return DT == kE4m3 ? 16 * (lane >> 2) + 2 * j + c : 16 * j + (lane >> 2) + 8 * c;
  }

  // The block's four warps joined; the result goes to out and lse, or to `slot`.
  // (Three barriers: what a slow thread still reads of one call is written in the
  // next only behind that one's first barrier.)
  __device__ __forceinline__ void finish(int b, int h, float* slot) {
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
      return fmaxf(fmaxf(S.m[0][head], S.m[1][head]), fmaxf(S.m[2][head], S.m[3][head]));
    };
    float* mine = S.buf + (warp & 1) * 8 * kBufStride;
    // (a slot's sums stay as they are: times the weights' 2^14, scaled values may leave FP32's range where the mean does
    // not)
    const float vs = DT == kE4m3 && slot == nullptr && a.c.v_scale != nullptr ? a.c.v_scale[h] : 1.0f;
    if (threadIdx.x < a.g) {
      const float mx = top(threadIdx.x), base = mx == -INFINITY ? 0.0f : mx;
      float sum = 0.0f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) sum += S.l[w][threadIdx.x] * exp2_ftz(S.m[w][threadIdx.x] - base);
      S.top[threadIdx.x] = mx - F::kShift;
      S.sum[threadIdx.x] = sum;
      S.factor[threadIdx.x] = slot != nullptr ? 1.0f : (sum == 0.0f ? 0.0f : 1.0f / sum);
    }
#pragma unroll
    for (int n = 0; n < NT; ++n) {  // eight heads at a time
      float f[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int head = 2 * (lane & 3) + i + 8 * n;
        const float mx = top(head);
        f[i] = exp2_ftz(S.m[warp][head] - (mx == -INFINITY ? 0.0f : mx));
      }
      auto at = [&](int j, int i) -> float& {  // i = 2 c + head bit
        return mine[(2 * (lane & 3) + (i & 1)) * kBufStride + channel(j, i >> 1)];
      };
      if (n > 0) __syncthreads();
      if (warp >= 2) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
#pragma unroll
          for (int i = 0; i < 4; ++i) at(j, i) = o[j][4 * n + i] * f[i & 1];
      }
      __syncthreads();
      if (warp < 2) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
#pragma unroll
          for (int i = 0; i < 4; ++i) at(j, i) += o[j][4 * n + i] * f[i & 1];
      }
      __syncthreads();
      const int c = threadIdx.x, heads = min(8, a.g - 8 * n);
      float* to = slot != nullptr ? slot + 8 * n * kD + c
                                  : a.out + ((long long)b * a.Hq + h * a.g + 8 * n) * kD + c;
#pragma unroll 4
      for (int i = 0; i < heads; ++i) {
        const float x = S.buf[i * kBufStride + c] + S.buf[(8 + i) * kBufStride + c];
        to[i * kD] = S.sum[8 * n + i] == 0.0f ? 0.0f : x * S.factor[8 * n + i] * vs;
      }
    }
    if (threadIdx.x < a.g) {
      const int j = threadIdx.x;
      if (slot != nullptr)
        *reinterpret_cast<float2*>(slot + a.g * kD + 2 * j) = make_float2(S.top[j], S.sum[j]);
      else if (a.lse != nullptr)
        a.lse[(long long)b * a.Hq + h * a.g + j] = (S.top[j] + log2f(S.sum[j])) * kLn2;
    }
  }
};

int most_blocks(int sms) { return sms * kBlocksPerSm; }

// The range that holds position x (cta_of), by 32-bit arithmetic where that holds.
__device__ __forceinline__ int range_of(long long x, long long W, int C) {
  if (W < (1 << 20)) return int((uint32_t(x + 1) * uint32_t(C) + uint32_t(W) - 1) / uint32_t(W)) - 1;
  return cta_of(x, W, C);
}

template <int DT, int QT, int NT, bool SEL>
__global__ void __launch_bounds__(kThreads, kBlocksPerSm) attn_kernel(AttnArgs a) {
  using F = Form<DT>;
  extern __shared__ __align__(16) char smem[];
  Smem<DT>& S = *reinterpret_cast<Smem<DT>*>(smem);
  wait_prior_grid();
  allow_dependents();
  // grid: (lanes, groups of blocks side by side)
  const int lanes = gridDim.x, groups = gridDim.y, group = blockIdx.y, c = group * lanes + blockIdx.x, n_ctas = lanes * groups;
  const int h0 = blockIdx.x * a.lane_heads;  // first of the lane's heads
  Rec* recs = reinterpret_cast<Rec*>(a.ws);
  float* slots = reinterpret_cast<float*>(a.ws + slots_offset(n_ctas));
  const bool per_unit = rec_per_unit((long long)a.B * a.c.H, n_ctas);
  if (!per_unit && threadIdx.x == 0) recs[c].u = -1;

  [[maybe_unused]] WideHeads heads;
  const int looker = n_ctas - 1 - c;  // (where units are few, the blocks that are left without work)
  const int pairs = kNarrow<DT, QT> ? WideHeads::pairs(a, looker, n_ctas) : 0;
  if (pairs > 0) heads.load(a, looker, n_ctas, pairs, 0);
  auto look = [&] {
    if (pairs > 0) {
      heads.store(a, looker, n_ctas, pairs, 0);
      for (int i = WideHeads::kHeads; i < pairs; i += WideHeads::kHeads) {
        heads.load(a, looker, n_ctas, pairs, i);
        heads.store(a, looker, n_ctas, pairs, i);
      }
    }
  };
  auto work_of = [&](int b) {
    const int tiles = (span_of<SEL>(a, checked_len(a.lens, b, a.max_pages, a.c.ps)) + F::kTile - 1) / F::kTile;
    return tiles > 0 ? (long long)a.lane_heads * (tiles + kUnitCost) : 0LL;
  };
  // all work W, by a warp's own scan where a lane can have a request (no barriers in the shortest calls)
  long long W, up_to = 0;  // up_to: work of the requests up to the lane's
  if (a.B <= 32) {
    const int lane = threadIdx.x & 31;
    up_to = lane < a.B ? work_of(lane) : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long x = __shfl_up_sync(0xFFFFFFFFu, up_to, o);
      if (lane >= o) up_to += x;
    }
    W = __shfl_sync(0xFFFFFFFFu, up_to, 31);
  } else {
    build_prefix<kThreads>(S.prefix, a.B, work_of);
    W = S.prefix.pre[kThreads];
  }
  // The query heads loaded above are looked at here, or, more than eight a group, behind the first copies: ragged 8-bit
  // requests, 4 heads 92.5 us here, 93.0 there, 12 heads 138.7, 124.2; 16 selected pages, 4 heads 37.8, 38.5, 16 heads
  // 57.3, 55.6; 512 x 1000, 4 heads 190, 195 (without the look 91.5, 125.8; 36.6, 59.7; 188)
  constexpr bool kLate = NT == 2;
  if (!kLate) look();
  // requests without tokens, and refused ones: no block's range holds them
  for (int b = c; b < a.B; b += n_ctas) {
    const int T = checked_len(a.lens, b, a.max_pages, a.c.ps);
    if (T > 0) continue;
    const float x = T < 0 ? NAN : 0.0f;
    for (int i = threadIdx.x; i < a.Hq * kD; i += kThreads) a.out[(long long)b * a.Hq * kD + i] = x;
    if (a.lse != nullptr)
      for (int i = threadIdx.x; i < a.Hq; i += kThreads) a.lse[(long long)b * a.Hq + i] = T < 0 ? NAN : -INFINITY;
    if (T < 0 && threadIdx.x == 0) flag(a.c, KVQ_PAGED_ERR_LENGTH);
    if (per_unit)
      for (int h = threadIdx.x; h < a.c.H; h += kThreads) recs[b * a.c.H + h].u = -1;
  }
  // ranges: none is empty, so the parts of a unit are those of adjacent groups
  const int sms = groups / kBlocksPerSm;
  const long long most = W <= sms ? W : max((long long)sms, W / kMinTiles);
  const int C = int(most < groups ? most : groups);
  if (group >= C) {
    if (kLate) look();
    return;
  }
  const long long s0 = part_start(group, W, C), e0 = part_start(group + 1, W, C);

  Cursor<SEL, F::kTile> at, ahead;
  long long in_request = s0;
  if (a.B <= 32) {
    at.b = min(__popc(__ballot_sync(0xFFFFFFFFu, up_to <= s0)), a.B - 1);
    if (at.b > 0) in_request -= __shfl_sync(0xFFFFFFFFu, up_to, at.b - 1);
  } else {
    at.b = find_request<kThreads>(S.prefix, a.B, work_of, in_request);
  }
  at.load(a);
  divide(in_request, at.tiles + kUnitCost, at.h, at.tile);
  at.h += h0;
  at.pos = s0;
  if (at.tile >= at.tiles) at.next_unit(a, h0);  // the range begins behind the unit's last tile
  if (at.h >= a.c.H || !at.before(a, e0)) {  // (and may hold no tile)
    if (kLate) look();
    return;
  }
  ahead = at;

  Block<DT, QT, NT, SEL> K(a, S);
  const int row = K.warp * F::kRows + (K.lane & (F::kRows - 1));
  Row entry, page;  // looked up one step, and both
  bool have_entry = false, have_page = false;
  // tile i: its selection entry is looked up at i - kStages - 1, its page at i - kStages, its copies issued at
  // i - kStages + 1
  for (int i = -F::kStages - 1; i < 0 || at.before(a, e0); ++i) {
    if (i >= 0) {
      wait_groups<F::kStages - 2>();
      __syncwarp();  // every lane's copies have landed, and every lane has left the stage that is filled next
    }
    const int filled = i + F::kStages - 1;
    if (filled >= 0) {
      if (have_page) K.issue(filled % F::kStages, page);
      commit();
    }
    have_page = have_entry;
    if (have_entry) {
      page = entry;
      look_up_page<SEL>(a, page);
    }
    have_entry = ahead.before(a, e0);
    if (have_entry) {
      look_up_entry<SEL>(a, ahead, ahead.tile * F::kTile + row, entry);
      ahead.next(a, h0);
    }
    if (i == -1) {  // (the first tiles' copies are on their way)
      if (kLate) look();
      K.load_query(at.b, at.h);
      K.clear();
    }
    if (i < 0) continue;
    __syncwarp();  // the stage's mask
    K.attend(i % F::kStages);
    if (at.tile + 1 < at.tiles && at.pos + 1 < e0) {
      ++at.tile;
      ++at.pos;
      continue;
    }
    const long long us = at.pos - at.tile, ue = us + at.tiles;  // the unit's tiles
    float* slot = nullptr;
    if (us < s0 || ue > e0) {
      slot = slots + size_t(2 * c + (us < s0 ? 0 : 1)) * slot_floats(a.g);
    }
    if (us >= s0 && threadIdx.x == 0) {  // it starts here
      const int u = at.b * a.c.H + at.h;
      if (slot != nullptr) recs[per_unit ? u : c] = Rec{u, c, range_of(ue - 1, W, C) - group + 1, 0};
      else if (per_unit) recs[u].u = -1;
    }
    K.finish(at.b, at.h, slot);
    at.next(a, h0);
    if (at.before(a, e0)) {
      K.load_query(at.b, at.h);
      K.clear();
    }
  }
}

struct Joint {  // shared memory of the combine kernel
  float m[kCombineWarps], l[kCombineWarps];
  float4 x[kCombineWarps][32];
  alignas(16) float q[kD];
};

// Maximum (in log2 units), sum of weights and weighted sum of `per` warps from `warp` on; a lane has four channels of x.
__device__ __forceinline__ void join_warps(const Joint& S, int warp, int per, int lane, float& top, float& l, float4& x) {
  top = S.m[warp];
  for (int w = 1; w < per; ++w) top = fmaxf(top, S.m[warp + w]);
  const float base = top == -INFINITY ? 0.0f : top;
  l = 0.0f;
  x = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  for (int w = 0; w < per; ++w) {
    const float f = exp2f(S.m[warp + w] - base);
    const float4 y = S.x[warp + w][lane];
    l += S.l[warp + w] * f;
    x = make_float4(fmaf(f, y.x, x.x), fmaf(f, y.y, x.y), fmaf(f, y.z, x.z), fmaf(f, y.w, x.w));
  }
}
// x / l, scaled, to out and lse of query head j of KV head h.
__device__ __forceinline__ void put_head(const AttnArgs& a, int b, int h, int j, int lane, float top, float l, float4 x) {
  const long long hq = (long long)b * a.Hq + h * a.g + j;
  const float vs = a.c.v_scale != nullptr ? a.c.v_scale[h] : 1.0f;
  if (l == 0.0f) x = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  else x = make_float4(x.x / l * vs, x.y / l * vs, x.z / l * vs, x.w / l * vs);
  reinterpret_cast<float4*>(a.out + hq * kD)[lane] = x;
  if (a.lse != nullptr && lane == 0) a.lse[hq] = (top + log2f(l)) * kLn2;
}

// The attention of one query head to E4M3 keys by FP32 multiply-adds, by a block: a lane has a token of a warp's 32
// for the scores and four channels for the sums. Rare, and slow beside the tensor cores (see combine_kernel).
template <bool SEL>
__device__ __forceinline__ void attend_plainly(const AttnArgs& a, Joint& S, int u, int j) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  Cursor<SEL, kCombineThreads> at;
  at.b = u / a.c.H;
  at.h = u % a.c.H;
  at.load(a);
  if (at.span == 0) return;  // no tokens, or refused: written by the attention kernel
  const float ks = a.c.k_scale != nullptr ? a.c.k_scale[at.h] : 1.0f;
  const float scale = a.scale * kLog2e;
  __syncthreads();  // nobody reads S of the head before
  if (warp == 0) {
    const char* q = a.q + (long long)at.b * a.q_stride + ((long long)(at.h * a.g + j) * kD + 4 * lane) * 2;
    *reinterpret_cast<float4*>(&S.q[4 * lane]) = load4<kBf16>(q);
  }
  __syncthreads();
  float m = -INFINITY, l = 0.0f;
  float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  for (int v0 = 32 * warp; v0 < at.span; v0 += kCombineThreads) {
    Row r;
    look_up_entry<SEL>(a, at, v0 + lane, r);
    look_up_page<SEL>(a, r);
    const bool in_pool = r.page >= 0 && r.page < a.c.n_pages, live = r.live && in_pool;
    const bool refused = __any_sync(0xFFFFFFFFu, r.bad != 0 || (r.live && !in_pool));  // (flagged by the attention kernel)
    const long long off = live ? (long long)r.page * a.c.page_stride + (long long)r.place * a.c.token_stride +
                                     (long long)r.h * a.c.head_stride
                               : -1;
    float s = 0.0f;
    if (live)
#pragma unroll 4
      for (int c = 0; c < kD; c += 16) {
        const uint4 w = *reinterpret_cast<const uint4*>(a.c.k + off + c);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float4 k = times(load4<kE4m3>(&(&w.x)[i]), ks), q = *reinterpret_cast<const float4*>(&S.q[c + 4 * i]);
          s = fmaf(q.x, k.x, fmaf(q.y, k.y, fmaf(q.z, k.z, fmaf(q.w, k.w, s))));
        }
      }
    float mx = live ? s : -INFINITY;
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, x));
    mx = fmaxf(m, mx * scale);
    const float base = mx == -INFINITY ? 0.0f : mx, alpha = exp2_ftz(m - base);
    const float p = live ? exp2_ftz(fmaf(s, scale, -base)) : 0.0f;
    m = mx;
    l = refused ? NAN : fmaf(l, alpha, p);
    o = times(o, alpha);
#pragma unroll 8
    for (int t = 0; t < 32; ++t) {
      const long long x = __shfl_sync(0xFFFFFFFFu, off, t);
      const float w = __shfl_sync(0xFFFFFFFFu, p, t);
      uint32_t y = 0u;
      if (x >= 0) y = *reinterpret_cast<const uint32_t*>(a.c.v + x + 4 * lane);
      const float4 v = load4<kE4m3>(&y);
      o = make_float4(fmaf(w, v.x, o.x), fmaf(w, v.y, o.y), fmaf(w, v.z, o.z), fmaf(w, v.w, o.w));
    }
  }
#pragma unroll
  for (int x = 16; x > 0; x >>= 1) l += __shfl_xor_sync(0xFFFFFFFFu, l, x);
  if (lane == 0) {
    S.m[warp] = m;
    S.l[warp] = l;
  }
  S.x[warp][lane] = o;
  __syncthreads();
  if (warp != 0) return;
  float top;
  join_warps(S, 0, kCombineWarps, lane, top, l, o);
  put_head(a, at.b, at.h, j, lane, top, l, o);
}

// Joins the parts of a unit that several blocks' ranges share; block (r, y): the
// unit of record r, `most` of its group's query heads. A head has 16 / heads warps,
// each with every so many parts, four channels a lane; a part is read once, with a
// running maximum. NARROW (BF16 queries of E4M3 keys): the heads that FP16 does not
// hold are attended again, by block (r, y) those of the units r, r + gridDim.x, ...
// (44 requests, 84000 tokens in all, 32 heads: 48 us without any, 244 with one of 16000
// tokens, 1470 where all are).
template <bool NARROW, bool SEL>
__global__ void __launch_bounds__(kCombineThreads) combine_kernel(AttnArgs a, int n_ctas, int lanes, int most) {
  __shared__ Joint S;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, units = a.B * a.c.H;
  const int j0 = blockIdx.y * most, heads = min(most, a.g - j0), per = kCombineWarps / heads;  // warps of a head
  const int j = j0 + warp / per, mine = warp % per;
  const float* slots = reinterpret_cast<const float*>(a.ws + slots_offset(n_ctas));
  const size_t stride = slot_floats(a.g);
  const uint8_t* wide = wide_heads(a, n_ctas);
  wait_prior_grid();
  allow_dependents();
  const Rec r = reinterpret_cast<const Rec*>(a.ws)[blockIdx.x];
  // (the bounds hold for every record of the attention kernel; a workspace that something else writes meanwhile
  // must not lead outside of it)
  const bool shared = r.u >= 0 && r.u < units && r.first >= 0 && r.first < n_ctas && r.parts >= 1 && r.parts <= n_ctas &&
                      r.first + (r.parts - 1) * lanes < n_ctas;
  // own units x0, x0 + gridDim.x, ...: of as many as a warp has lanes, which have heads to be attended again
  const int x0 = int(blockIdx.x);
  auto look = [&](int u0) {
    const long long u = u0 + (long long)lane * gridDim.x;
    const uint64_t among = (~0ull >> (64 - 8 * heads)) << (8 * (j0 & 7));  // the block's heads
    const auto word = [&] { return *reinterpret_cast<const uint64_t*>(wide + u * kMaxGroup + (j0 & 8)); };
    return __ballot_sync(0xFFFFFFFFu, u < units && (word() & among) != 0);
  };
  uint32_t again = 0u;
  if constexpr (NARROW) again = look(x0);
  if (!shared && again == 0u && (!NARROW || units <= 32 * int(gridDim.x))) return;
  // (another block attends these heads of this one's unit)
  const bool others = NARROW && shared && r.u != x0 && warp < per * heads && wide[r.u * kMaxGroup + j] != 0;
  const int c = r.first, parts = shared ? r.parts : 0;  // slot 2 c + 1 of the first block c, slot 2 c' of the others
  float m = -INFINITY, l = 0.0f;
  float4 x = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  if (warp < per * heads) {
    constexpr int kUnroll = 4;
    for (int i0 = mine; i0 < parts; i0 += kUnroll * per) {
      float2 ml[kUnroll];
      float4 y[kUnroll];
#pragma unroll
      for (int e = 0; e < kUnroll; ++e) {
        const int i = i0 + e * per;
        ml[e] = make_float2(-INFINITY, 0.0f);
        y[e] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (i < parts) {
          const float* p = slots + size_t(i == 0 ? 2 * c + 1 : 2 * (c + i * lanes)) * stride;
          ml[e] = *reinterpret_cast<const float2*>(p + a.g * kD + 2 * j);
          y[e] = reinterpret_cast<const float4*>(p + j * kD)[lane];
        }
      }
      float top = m;
#pragma unroll
      for (int e = 0; e < kUnroll; ++e) top = fmaxf(top, ml[e].x);
      const float base = top == -INFINITY ? 0.0f : top, f = exp2f(m - base);
      m = top;
      l *= f;
      x = make_float4(x.x * f, x.y * f, x.z * f, x.w * f);
#pragma unroll
      for (int e = 0; e < kUnroll; ++e) {
        const float w = exp2f(ml[e].x - base);
        l += ml[e].y * w;
        x = make_float4(fmaf(w, y[e].x, x.x), fmaf(w, y[e].y, x.y), fmaf(w, y[e].z, x.z), fmaf(w, y[e].w, x.w));
      }
    }
    if (lane == 0) {
      S.m[warp] = m;
      S.l[warp] = l;
    }
    S.x[warp][lane] = x;
  }
  __syncthreads();
  if (shared && mine == 0 && warp < per * heads && !others) {
    float top;
    join_warps(S, warp, per, lane, top, l, x);
    put_head(a, r.u / a.c.H, r.u % a.c.H, j, lane, top, l, x);
  }
  if constexpr (NARROW) {
    for (int u0 = x0;;) {
      for (; again != 0u; again &= again - 1u) {
        const int u = u0 + (__ffs(again) - 1) * int(gridDim.x);
        for (int i = j0; i < j0 + heads; ++i)
          if (wide[u * kMaxGroup + i] != 0) attend_plainly<SEL>(a, S, u, i);
      }
      if (units - u0 <= 32 * int(gridDim.x)) break;
      u0 += 32 * int(gridDim.x);
      again = look(u0);
    }
  }
}

template <int DT, int QT, int NT, bool SEL>
cudaError_t launch_form(const AttnArgs& a, cudaStream_t stream) {
  const int smem = int(sizeof(Smem<DT>)), lanes = a.c.H / a.lane_heads, groups = most_blocks(a.sms) / lanes, n = lanes * groups;
  static std::atomic<uint64_t> configured{0};  // bit: device
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (!((configured.load(std::memory_order_relaxed) >> dev) & 1)) {
    e = cudaFuncSetAttribute(attn_kernel<DT, QT, NT, SEL>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    configured.fetch_or(uint64_t(1) << dev, std::memory_order_relaxed);
  }
  count_launch();
  e = launch_dependent(attn_kernel<DT, QT, NT, SEL>, dim3(lanes, groups), dim3(kThreads), size_t(smem), stream, a);
  if (e != cudaSuccess) return e;
  // one head per block while that leaves an SM a block (parts are many then), up to eight else (one head against
  // eight: 1 x 32768 tokens and eight heads 28.7, 32.1 us; 64 x 1000 and four 54.9, 48.9 us)
  const long long units = (long long)a.B * a.c.H;
  const int recs = rec_per_unit(units, n) ? int(units) : n;
  int most = 1;
  while (most < 8 && (long long)recs * ((a.g + most - 1) / most) > a.sms) most *= 2;
  count_launch();
  return launch_dependent(combine_kernel<kNarrow<DT, QT>, kNarrow<DT, QT> && SEL>,
                          dim3(recs, (a.g + most - 1) / most), dim3(kCombineThreads), 0, stream, a, n, lanes, most);
}

template <int DT, int QT>
cudaError_t launch_types(const AttnArgs& a, cudaStream_t stream) {
  // up to eight heads fill half of a product's rows: the form for 16 would do, but takes 7.4 us instead of 6.7 (one
  // request of 256 tokens), 322 instead of 312 (512 x 1000) and 116 instead of 92 (64 ragged ones of 8-bit keys)
  if (a.sel != nullptr)
    return a.g <= 8 ? launch_form<DT, QT, 1, true>(a, stream) : launch_form<DT, QT, 2, true>(a, stream);
  return a.g <= 8 ? launch_form<DT, QT, 1, false>(a, stream) : launch_form<DT, QT, 2, false>(a, stream);
}

}  // namespace

size_t attn_workspace(int B, int H, int Hq, int sms) {
  return slots_offset(most_blocks(sms)) + 2 * size_t(most_blocks(sms)) * slot_floats(Hq / H) * 4 +
         size_t(B) * H * kMaxGroup;
}

cudaError_t launch_attn(const AttnArgs& args, cudaStream_t stream) {
  AttnArgs a = args;
  // as many lanes as leave at most one block in twenty without one (eight lanes against one: 64 x 4000 tokens of
  // 8-bit keys 94, 102 us; 512 x 1000 of BF16 314, 327 us)
  const int n = most_blocks(a.sms);
  int lanes = 1;
  for (int l = 2; l <= a.c.H && 2 * l <= n; ++l)
    if (a.c.H % l == 0 && 20 * (n / l * l) >= 19 * n) lanes = l;
  a.lane_heads = a.c.H / lanes;
  const bool bf = a.q_dtype == kBf16;
  if (a.dtype == kBf16) return launch_types<kBf16, kBf16>(a, stream);
  if (a.dtype == kFp16) return launch_types<kFp16, kFp16>(a, stream);
  return bf ? launch_types<kE4m3, kBf16>(a, stream) : launch_types<kE4m3, kFp16>(a, stream);
}

}  // namespace paged
}  // namespace kvq
