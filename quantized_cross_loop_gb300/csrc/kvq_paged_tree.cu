// kvq_paged_tree.cu — attention of several queries per request (a tree of drafted
// tokens, a chunk of a prompt, a decode step) over a paged cache.
//
// s_t = scale q.k_t over the cached tokens and the drafted ones that a row's mask
// allows, out = sum_t e^(s_t - m) v_t / l, lse = m + ln l, in one pass with a running
// maximum m and sum l per row.
//
// A unit is a request's KV head and up to 128 x TILES of its rows: row r is query
// head r % g of drafted token r / g, so that a token's keys are read once for all of
// them. Tiles of 128 tokens; the tiles of all units, concatenated, are cut into equal
// ranges, one per block (one block an SM); lengths are read on the device, so a
// captured call follows them. A unit that lies in one block's range is finished
// there; of the others each block leaves (m, l, sum) in one of its two slots, and the
// combine kernel joins them.
//
// Both products run on tcgen05 with 128 rows: S = Q K^T from shared memory, O += P V
// with P in tensor memory, where the softmax warps leave it in the place of S. A
// block's warps:
//   softmax   four per row tile, a thread a row: no shuffles; the sums of a row are
//             rescaled only when its maximum grows by more than 2^8 (its weights then
//             go to at most 1, or 2^15 for FP16, by kShift)
//   producers four: 16-byte asynchronous copies of K and V rows into a ring of
//             operand slots; 8-bit rows by way of a staging ring and a conversion
//   MMA       one, a lane of which issues all products
// Exactness: products of 16-bit values are exact, sums FP32. 8-bit keys become 16-bit
// of the queries' type (exact), 8-bit values BF16 (exact). A weight is one 16-bit
// number (times its value's scale, where tokens have one): BF16, whose range holds
// any scale's product, or FP16 for FP16 caches, down to 2^-31 of the largest weight.
// The result is rounded to 16 bits anyway, and three parts would triple the second
// product, which bounds wide trees.
//
// A drafted token's value that is not finite must not reach rows that do not see it
// (0 x infinity): the producers replace it by 0, and the rows that see it get it back
// at the end (loose).
//
// Every wait is bounded (2 s): a wait that runs out sets an error bit and the block
// leaves, after its products in flight.
#include <atomic>
#include <type_traits>

#include "kvq_attn_common.cuh"
#include "kvq_paged.cuh"

namespace kvq {
namespace paged {
namespace {

constexpr int kTile = 128;       // tokens of a tile, rows of a row tile
constexpr int kProducers = 128;  // threads
constexpr int kUnitCost = 1;     // tiles that the end of a unit takes as long as
constexpr int kSlotBytes = kTile * kD * 2;
constexpr int kRawBytes = kTile * kD;
constexpr uint32_t kTmemCols = 512;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr float kSlack = 8.0f;   // log2 of what a row's weights may exceed 1 by before its sums are rescaled
constexpr long long kWaitNs = 2000000000LL;
enum { kBadPage = 1, kLoose = 2 };  // of a unit

// ---------------------------------------------------------------- forms

template <int DT, int QT, int TILES, bool TS>
struct Form {
  static constexpr bool kNarrow = DT == kE4m3;
  static constexpr bool kKeyBf = DT == kBf16 || (kNarrow && QT == kBf16);  // type of Q and K operands
  static constexpr bool kValBf = DT != kFp16;                              // type of P and V operands
  static constexpr float kShift = kValBf ? -kSlack : 15.0f - kSlack;
  static constexpr int kRows = kTile * TILES;
  static constexpr int kSoftmaxWarps = 4 * TILES;
  static constexpr int kMmaWarp = kSoftmaxWarps + kProducers / 32;
  static constexpr int kThreads = (kMmaWarp + 4) * 32;  // (three idle warps: registers are shared out by four)
  // registers of the softmax, producer and MMA warps; 504 = 3 x 168 and 512 = 4 x 128 of the launch
  static constexpr int kSoftmaxRegs = TILES == 1 ? 224 : 144, kProducerRegs = TILES == 1 ? 152 : 112,
                       kMmaRegs = TILES == 1 ? 128 : 112;
  static constexpr int kSlots = kNarrow ? 3 : (TILES == 1 ? 6 : 5);
  static constexpr int kStages = kNarrow ? (TILES == 1 ? 5 : 3) : 0;  // of raw 8-bit rows
  // slots between a copy and the look at it: 8-bit rows are all converted, of 16-bit ones the drafted values checked
  static constexpr int kLag = kNarrow ? kStages - 1 : 2;
};

template <class F>
struct Smem {
  char q[F::kRows * kD * 2];
  union {
    char slot[F::kSlots][kSlotBytes];
    Prefix<F::kThreads> prefix;  // before the first copy
  };
  char raw[F::kStages > 0 ? F::kStages : 1][F::kStages > 0 ? kRawBytes : 16];
  float scales[F::kSoftmaxWarps / 4][2][2][F::kNarrow ? kTile : 4];  // row tile, parity, K and V, token
  unsigned long long full[F::kSlots], empty[F::kSlots];
  unsigned long long s_full[2], p_ready[2], pv_done[2], q_full, drain;
  uint32_t tmem;
  int flags[8];  // of the unit by its number's last bits
  volatile int abort;
};

// ---------------------------------------------------------------- PTX

__device__ __forceinline__ uint32_t smem_addr(const void* p) { return uint32_t(__cvta_generic_to_shared(p)); }
__device__ __forceinline__ void mbar_init(unsigned long long* bar, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(smem_addr(bar)), "r"(count));
}
__device__ __forceinline__ void mbar_arrive(unsigned long long* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_addr(bar)) : "memory");
}
__device__ __forceinline__ bool mbar_try_wait(unsigned long long* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile("{ .reg .pred p; mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, 200; selp.u32 %0, 1, 0, p; }"
               : "=r"(ok)
               : "r"(smem_addr(bar)), "r"(parity)
               : "memory");
  return ok != 0;
}
__device__ __forceinline__ long long global_ns() {
  long long t;
  asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
  return t;
}
// Waits for the phase of this parity; false when it took kWaitNs, or another wait of the block did.
__device__ __forceinline__ bool mbar_wait_long(unsigned long long* bar, uint32_t parity, volatile int* abort) {
  const long long t0 = global_ns();
  while (!mbar_try_wait(bar, parity)) {
    if (*abort) return false;
    if (global_ns() - t0 > kWaitNs) {
      *abort = 1;
      return false;
    }
  }
  return true;
}
__device__ __forceinline__ bool mbar_wait(unsigned long long* bar, uint32_t parity, volatile int* abort) {
  return mbar_try_wait(bar, parity) || mbar_wait_long(bar, parity, abort);
}

__device__ __forceinline__ void fence_async_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// Shared-memory matrix descriptor of operands with a 128-byte swizzle: 1024 bytes from eight rows (tokens) to the next
// eight; in an MN-major operand `lbo` bytes from 64 channels to the next 64.
__device__ __forceinline__ uint64_t smem_desc(uint32_t addr, uint32_t lbo) {
  return uint64_t((addr & 0x3FFFFu) >> 4) | (uint64_t(lbo >> 4) << 16) | (uint64_t(1024 >> 4) << 32) | (1ull << 46) |
         (2ull << 61);
}
// Instruction descriptor of kind::f16: A and B of one type, FP32 D, 128 x 128; b_mn: B is MN-major.
__host__ __device__ constexpr uint32_t instr_desc(bool bf16, bool b_mn) {
  return (1u << 4) | (uint32_t(bf16) << 7) | (uint32_t(bf16) << 10) | (uint32_t(b_mn) << 16) | ((128u >> 3) << 17) |
         ((128u >> 4) << 24);
}
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{ .reg .pred p; setp.ne.b32 p, %4, 0; tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p; }" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{ .reg .pred p; setp.ne.b32 p, %4, 0; tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p; }" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}
__device__ __forceinline__ void mma_commit(unsigned long long* bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_addr(bar))
               : "memory");
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// A thread's row: 32 columns of tensor memory. The registers are read only behind tmem_wait_ld.
__device__ __forceinline__ void tmem_ld(uint32_t at, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(at)
      : "memory");
}
__device__ __forceinline__ void tmem_wait_ld(uint32_t (&r)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                 "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]),
                 "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]),
                 "+r"(r[23]), "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]),
                 "+r"(r[30]), "+r"(r[31])::"memory");
}
// Registers of further loads that a tmem_wait_ld has waited for, too.
__device__ __forceinline__ void tmem_landed(uint32_t (&r)[32]) {
#pragma unroll
  for (int i = 0; i < 32; i += 8)
    asm volatile("" : "+r"(r[i]), "+r"(r[i + 1]), "+r"(r[i + 2]), "+r"(r[i + 3]), "+r"(r[i + 4]), "+r"(r[i + 5]),
                      "+r"(r[i + 6]), "+r"(r[i + 7])::"memory");
}
// 16 columns, at once and waited for.
__device__ __forceinline__ void tmem_ld16(uint32_t at, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, "
      "[%16];\n\ttcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(at)
      : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t at, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
      "%15, %16};" ::"r"(at),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ void copy16(uint32_t dst, const char* src, bool live) {
  const int n = live ? 16 : 0;  // 0: zeros
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void wait_groups() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
// The barrier counts this thread once its copies so far have landed.
__device__ __forceinline__ void arrive_landed(unsigned long long* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_addr(bar)) : "memory");
}
template <int N>
__device__ __forceinline__ void more_registers() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void fewer_registers() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
__device__ __forceinline__ uint4 lds16(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ void sts16(uint32_t a, const uint4& v) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}

// 2^x; results below 2^-126 are 0.
__device__ __forceinline__ float exp2_ftz(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
template <bool BF>
__device__ __forceinline__ uint32_t pack(float a, float b) {
  if constexpr (BF) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
  } else {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
}
// Four E4M3 values as two pairs of 16-bit numbers (exact).
template <bool BF>
__device__ __forceinline__ uint2 widen(uint32_t w) {
  const uint32_t a = e4m3x2_to_f16x2(w & 0xFFFFu), b = e4m3x2_to_f16x2(w >> 16);
  if constexpr (!BF) return make_uint2(a, b);
  const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&a));
  const float2 y = __half22float2(*reinterpret_cast<const __half2*>(&b));
  return make_uint2(pack<true>(x.x, x.y), pack<true>(y.x, y.y));
}

// ---------------------------------------------------------------- units

// Request b's rows and tokens; n 0 where it has none or is refused.
struct Request {
  int P, n, row0;
  bool refused;
  __device__ __forceinline__ void load(const TreeArgs& a, int b) {
    n = row_range(a.offsets, a.n_rows, b, row0);
    P = n > 0 ? checked_len(a.lens, b, a.max_pages, a.c.ps) : 0;
    refused = n < 0 || (n > 0 && (P < 0 || P + (long long)n > (long long)a.max_pages * a.c.ps.d ||
                                  n > KVQ_PAGED_MAX_DRAFT || (a.mask != nullptr && n > 32 * a.mask_words)));
    if (refused) n = 0;
  }
  // Tokens that row block rb of R rows looks at: without a mask up to its last row's own.
  __device__ __forceinline__ int tokens(const TreeArgs& a, int rb, int R) const {
    return a.mask != nullptr ? P + n : P + (min(n * a.g, (rb + 1) * R) - 1) / a.g + 1;
  }
  __device__ __forceinline__ int blocks(const TreeArgs& a, int R) const { return (n * a.g + R - 1) / R; }
  __device__ __forceinline__ static int tiles(int tokens) { return (tokens + kTile - 1) / kTile; }
  // Work of one KV head.
  __device__ __forceinline__ long long work(const TreeArgs& a, int R) const {
    const int nb = blocks(a, R);
    if (a.mask != nullptr) return (long long)nb * (tiles(P + n) + kUnitCost);
    long long w = 0;
    for (int rb = 0; rb < nb; ++rb) w += tiles(tokens(a, rb, R)) + kUnitCost;
    return w;
  }
};

// The units that a block's range [s0, e0) of the work touches, in order.
template <int R>
struct Walk {
  Request r;
  int b, h, rb;
  int tokens, tiles;      // of the unit
  int begin, end;         // its tiles in the range
  int number;             // of the unit within the range
  long long pos;          // of the unit's first tile
  __device__ __forceinline__ void unit(const TreeArgs& a) {
    tokens = r.tokens(a, rb, R);
    tiles = Request::tiles(tokens);
  }
  __device__ __forceinline__ void clip(long long s0, long long e0) {
    begin = int(max(0LL, min((long long)tiles, s0 - pos)));
    end = int(max(0LL, min((long long)tiles, e0 - pos)));
  }
  // at: position of s0 within request b
  __device__ __forceinline__ bool open(const TreeArgs& a, int bb, long long at, long long s0, long long e0) {
    b = bb;
    rb = h = number = 0;
    r.load(a, b);
    const long long head = max(1LL, r.work(a, R));
    if (at < 0x7FFFFFFF && head < 0x7FFFFFFF) {
      h = int(at) / int(head);
    } else {
      h = int(at / head);
    }
    pos = s0 - at + h * head;
    unit(a);
    while (pos + tiles + kUnitCost <= s0 && rb + 1 < r.blocks(a, R)) {
      pos += tiles + kUnitCost;
      ++rb;
      unit(a);
    }
    clip(s0, e0);
    if (begin < end) return true;
    const bool more = next(a, s0, e0);  // the range begins behind the unit's last tile
    number = 0;
    return more;
  }
  __device__ __forceinline__ bool next(const TreeArgs& a, long long s0, long long e0) {
    pos += tiles + kUnitCost;
    if (pos >= e0) return false;
    ++number;
    if (++rb == r.blocks(a, R)) {
      rb = 0;
      if (++h == a.c.H) {
        h = 0;
        do {
          if (++b >= a.B) return false;
          r.load(a, b);
        } while (r.n == 0);
      }
    }
    unit(a);
    clip(s0, e0);
    return true;
  }
};

// 32 bits of what row i of a request sees, from its drafted token j0 (which may be negative: cached tokens) on.
__device__ __forceinline__ uint32_t seen_word(const uint32_t* mask, int words, int n, int i, int k) {
  if (k < 0) return 0xFFFFFFFFu;
  const int last = mask != nullptr ? n : i + 1;  // tokens from here on are not seen
  const int left = last - 32 * k;
  if (left <= 0) return 0u;
  const uint32_t live = left >= 32 ? 0xFFFFFFFFu : (1u << left) - 1u;
  return mask == nullptr ? live : (k < words ? mask[k] & live : 0u);
}
__device__ __forceinline__ uint32_t seen_bits(const uint32_t* mask, int words, int n, int i, int j0) {
  const int k = j0 >> 5;  // (rounds down)
  const uint32_t lo = seen_word(mask, words, n, i, k);
  if ((j0 & 31) == 0) return lo;
  return __funnelshift_r(lo, seen_word(mask, words, n, i, k + 1), j0 & 31);
}

// Sum of the values that are not finite in channel c of the drafted tokens that row i sees (0: none).
template <int DT>
__device__ __forceinline__ float loose(const TreeArgs& a, const Request& r, int b, int h, int i, int c) {
  const uint32_t* mask = a.mask != nullptr ? a.mask + (long long)(r.row0 + i) * a.mask_words : nullptr;
  float sum = 0.0f;
  for (int j = 0; j < r.n; ++j) {
    if (!((seen_word(mask, a.mask_words, r.n, i, j >> 5) >> (j & 31)) & 1)) continue;
    const int t = r.P + j, e = a.c.ps.div(t), page = a.table[(long long)b * a.max_pages + e];
    const int place = t - e * int(a.c.ps.d);
    if (page < 0 || page >= a.c.n_pages) continue;
    const char* p = a.c.v + (long long)page * a.c.page_stride + (long long)place * a.c.token_stride +
                    (long long)h * a.c.head_stride + (c & ~3) * elem_bytes<DT>();
    const float4 x = load4<DT>(p);
    float v = (&x.x)[c & 3];
    if (DT == kE4m3 && a.c.v_scale != nullptr)
      v *= a.c.v_scale[a.c.token_scales ? ((long long)page * a.c.H + h) * int(a.c.ps.d) + place : h];
    if (!isfinite(v)) sum += v;
  }
  return sum;
}

// Where in an operand slot a 16-byte chunk (eight channels) of a token (or row) lies: 64 channels of all 128 tokens, then
// the other 64, a token's 128 bytes with its chunks swizzled by the token's number. The same for a K-major operand (keys,
// queries) and an MN-major one (values). (Core matrices of 8 x 16 bytes without a swizzle take each of a row's chunks to
// another line of shared memory: the copies' writes then took the products half of their rate.)
__device__ __forceinline__ uint32_t chunk_at(int token, int chunk) {
  return uint32_t((chunk >> 3) * (kSlotBytes / 2) + token * 128 + (((chunk ^ token) & 7) << 4));
}

struct Rec {  // a unit that begins in a block's range and goes on behind it (parts 0: none)
  int32_t b, h, rb, parts;
};
__host__ __device__ constexpr size_t slots_offset(int n) { return size_t(n) * sizeof(Rec); }
// sums [32][rows][4], then m and l by row, then flags
__host__ __device__ constexpr size_t slot_floats(int rows) { return size_t(rows) * (kD + 2) + 4; }

// ---------------------------------------------------------------- softmax warps

// scale ks, whose product may leave FP32's normal range where the logits do not
__device__ __forceinline__ float scaled(float scale, float ks) {
  const float x = scale * ks;
  return isfinite(ks) ? fminf(fmaxf(x, 0x1p-149f), 3.402823466e38f) : ks;
}

template <int DT, int QT, int TILES, bool TS>
struct Softmax {
  using F = Form<DT, QT, TILES, TS>;
  const TreeArgs& a;
  Smem<F>& S;
  const int tile, thread, warp, lane;  // row tile, thread and warp of the tile's 128
  const uint32_t lanes;                // tensor-memory lanes of the warp
  const uint32_t o_at;

  __device__ __forceinline__ Softmax(const TreeArgs& args, Smem<F>& s)
      : a(args), S(s), tile(threadIdx.x / kTile), thread(threadIdx.x % kTile), warp((threadIdx.x >> 5) & 3),
        lane(threadIdx.x & 31), lanes(s.tmem + (uint32_t((threadIdx.x >> 5) & 3) << 21)), o_at(lanes + 128u * (threadIdx.x / kTile)) {}

  __device__ __forceinline__ void sync() const { asm volatile("bar.sync %0, 128;" ::"r"(tile + 1) : "memory"); }

  // The unit's queries of this tile as an operand; the warp's own 32 rows.
  __device__ __forceinline__ void load_queries(const Walk<F::kRows>& w) {
    const int M = w.r.n * a.g, r = w.rb * F::kRows + threadIdx.x;
    long long off = -1;
    if (r < M) {
      const int i = r / a.g, j = r - i * a.g;
      off = (w.r.row0 + i) * a.q_stride + (long long)(w.h * a.g + j) * (kD * 2);
    }
    const uint32_t to = smem_addr(S.q) + tile * kSlotBytes;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const long long x = __shfl_sync(0xFFFFFFFFu, off, 4 * e + (lane >> 3));
#pragma unroll
      for (int f = 0; f < 2; ++f) {
        const int chunk = 8 * f + (lane & 7);
        copy16(to + chunk_at(32 * warp + 4 * e + (lane >> 3), chunk), a.q + (x < 0 ? 0 : x) + chunk * 16, x >= 0);
      }
    }
    commit();
    wait_groups<0>();
    fence_async_smem();
    __syncwarp();
    if (lane == 0) mbar_arrive(&S.q_full);
  }

  // Where token thread's scales of a tile are, or -1.
  __device__ __forceinline__ long long scale_at(const Walk<F::kRows>& w, int t) const {
    if (t >= w.tokens) return -1;
    const int e = a.c.ps.div(t), page = a.table[(long long)w.b * a.max_pages + e];
    if (page < 0 || page >= a.c.n_pages) return -1;
    return ((long long)page * a.c.H + w.h) * int(a.c.ps.d) + (t - e * int(a.c.ps.d));
  }

  __device__ __forceinline__ void run(Walk<F::kRows> w, long long s0, long long e0, long long W, int C) {
    uint32_t count = 0;  // tiles of this thread's row tile so far
    uint32_t units = 0;
    bool more = true;
    while (more) {
      load_queries(w);
      const int M = w.r.n * a.g, r = w.rb * F::kRows + threadIdx.x;
      const bool active = w.rb * F::kRows + tile * kTile < M;  // the row tile has rows
      // (a row tile without work must not arrive for the next unit in the same phase)
      if (!active && !mbar_wait(&S.q_full, units & 1u, &S.abort)) return;
      ++units;
      const bool rows = w.rb * F::kRows + tile * kTile + warp * 32 < M;  // the warp has
      float m = -INFINITY, l = 0.0f;
      const int i = r / a.g;
      const uint32_t* mask = a.mask != nullptr && r < M ? a.mask + (long long)(w.r.row0 + i) * a.mask_words : nullptr;
      float sc = a.scale * kLog2e;
      if constexpr (DT == kE4m3 && !TS)
        if (a.c.k_scale != nullptr) sc = scaled(sc, a.c.k_scale[w.h]);
      long long at_next = -1;
      float ks_next = 0.0f, vs_next = 0.0f;
      [[maybe_unused]] auto fetch = [&](long long at) {
        ks_next = at >= 0 ? a.c.k_scale[at] : 0.0f;
        vs_next = at >= 0 ? a.c.v_scale[at] : 0.0f;
      };
      if constexpr (TS)
        if (active) {
          fetch(scale_at(w, w.begin * kTile + thread));
          at_next = scale_at(w, (w.begin + 1) * kTile + thread);
        }
      for (int k = w.begin; active && k < w.end; ++k, ++count) {
        const int t0 = k * kTile;
        const uint32_t buf = TILES == 1 ? count & 1u : uint32_t(tile), phase = TILES == 1 ? (count >> 1) & 1u : count & 1u;
        const uint32_t s_at = lanes + 256u + 128u * buf;
        const float* kf = S.scales[tile][k & 1][0];
        const float* vf = S.scales[tile][k & 1][1];
        if constexpr (TS) {
          float vs = vs_next;
          if (t0 + thread >= w.r.P && !isfinite(vs)) {
            atomicOr(&S.flags[w.number & 7], kLoose);
            vs = 0.0f;
          }
          S.scales[tile][k & 1][0][thread] = scaled(sc, ks_next);
          S.scales[tile][k & 1][1][thread] = vs;
          sync();
          fetch(at_next);
          at_next = k + 2 < w.end ? scale_at(w, t0 + 2 * kTile + thread) : -1;
        }
        if (!mbar_wait(&S.s_full[buf], phase, &S.abort)) return;
        tc_fence_after();
        if (rows) {
          // Scores 64 columns at a time, twice: for their maximum, and for the weights (held in between they would take
          // 128 registers). TS: in log2 units, else the products' own.
          const bool drafted = t0 + kTile > w.r.P;
          uint32_t x[2][32];
          auto pair = [&](int c, int e) { return make_float2(__uint_as_float(x[c][e]), __uint_as_float(x[c][e + 1])); };
          auto load = [&](int half) {
            tmem_ld(s_at + 64 * half, x[0]);
            tmem_ld(s_at + 64 * half + 32, x[1]);
            if constexpr (TS) {
              // (a row's scales are the same for all lanes: read while the scores are on their way)
#pragma unroll
              for (int c = 0; c < 2; ++c) {
                float4 f[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) f[e] = *reinterpret_cast<const float4*>(&kf[64 * half + 32 * c + 4 * e]);
                if (c == 0) {
                  tmem_wait_ld(x[0]);
                  tmem_landed(x[1]);
                }
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                  const float2 y = __fmul2_rn(pair(c, 4 * e), make_float2(f[e].x, f[e].y));
                  const float2 z = __fmul2_rn(pair(c, 4 * e + 2), make_float2(f[e].z, f[e].w));
                  x[c][4 * e] = __float_as_uint(y.x);
                  x[c][4 * e + 1] = __float_as_uint(y.y);
                  x[c][4 * e + 2] = __float_as_uint(z.x);
                  x[c][4 * e + 3] = __float_as_uint(z.y);
                }
              }
            } else {
              tmem_wait_ld(x[0]);
              tmem_landed(x[1]);
            }
            if (drafted) {
#pragma unroll
              for (int c = 0; c < 2; ++c) {
                const uint32_t see = r < M ? seen_bits(mask, a.mask_words, w.r.n, i, t0 + 64 * half + 32 * c - w.r.P) : 0u;
#pragma unroll
                for (int e = 0; e < 32; ++e)
                  if (!((see >> e) & 1)) x[c][e] = 0xFF800000u;
              }
            }
          };
          float mx = -INFINITY;
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            load(half);
#pragma unroll
            for (int c = 0; c < 2; ++c)
#pragma unroll
              for (int e = 0; e < 32; e += 2) mx = max3(mx, __uint_as_float(x[c][e]), __uint_as_float(x[c][e + 1]));
          }
          if constexpr (!TS) mx *= sc;
          if (k == w.begin) {
            m = mx;
          } else if (__any_sync(0xFFFFFFFFu, mx > m + kSlack)) {
            const float top = fmaxf(m, mx), alpha = exp2_ftz(m - (top == -INFINITY ? 0.0f : top));
            m = top;
            l *= alpha;
            // the sums are at rest behind the product before
            if (!mbar_wait(&S.pv_done[TILES == 1 ? 0 : tile], (count - 1) & 1u, &S.abort)) return;
            tc_fence_after();
#pragma unroll 1
            for (int c = 0; c < 8; ++c) {
              uint32_t y[16];
              tmem_ld16(o_at + 16 * c, y);
#pragma unroll
              for (int e = 0; e < 16; ++e) y[e] = __float_as_uint(__uint_as_float(y[e]) * alpha);
              tmem_st16(o_at + 16 * c, y);
            }
            tmem_wait_st();
          }
          const float base = F::kShift - (m == -INFINITY ? 0.0f : m);
          float2 sum[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            load(half);
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              uint32_t p[16];
              [[maybe_unused]] float4 f[8];
              if constexpr (TS) {
#pragma unroll
                for (int e = 0; e < 8; ++e) f[e] = *reinterpret_cast<const float4*>(&vf[64 * half + 32 * c + 4 * e]);
              }
#pragma unroll
              for (int e = 0; e < 32; e += 2) {
                float2 y;
                if constexpr (TS) y = __fadd2_rn(pair(c, e), make_float2(base, base));
                else y = __ffma2_rn(pair(c, e), make_float2(sc, sc), make_float2(base, base));
                y = make_float2(exp2_ftz(y.x), exp2_ftz(y.y));
                sum[(e >> 1) & 1] = __fadd2_rn(sum[(e >> 1) & 1], y);
                if constexpr (TS) y = __fmul2_rn(y, e & 2 ? make_float2(f[e / 4].z, f[e / 4].w) : make_float2(f[e / 4].x, f[e / 4].y));
                p[e / 2] = pack<F::kValBf>(y.x, y.y);
              }
              tmem_st16(s_at + 32 * half + 16 * c, p);  // (in the place of scores that are read)
            }
          }
          l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
          tmem_wait_st();
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&S.p_ready[buf]);
      }
      if (active) {
        if (!mbar_wait(&S.pv_done[TILES == 1 ? 0 : tile], (count - 1) & 1u, &S.abort)) return;
        tc_fence_after();
      }
      if (threadIdx.x == 0) S.flags[(w.number + 4) & 7] = 0;  // (the producers are at most three units ahead)
      if (active && rows) finish(w, s0, W, C, r, M, i, m, l);
      if (threadIdx.x == 0 && w.begin == 0 && w.end < w.tiles) {
        const long long last = w.pos + w.tiles - 1;
        reinterpret_cast<Rec*>(a.ws)[blockIdx.x] = Rec{w.b, w.h, w.rb, cta_of(last, W, C) - int(blockIdx.x) + 1};
      }
      tc_fence_before();
      more = w.next(a, s0, e0);
    }
  }

  // The unit's rows, or this part of it, to out and lse or to a slot.
  __device__ __forceinline__ void finish(const Walk<F::kRows>& w, long long s0, long long W, int C, int r, int M, int i, float m,
                                         float l) {
    const bool whole = w.begin == 0 && w.end == w.tiles;
    const int flags = *reinterpret_cast<volatile int*>(&S.flags[w.number & 7]);
    if (flags & kBadPage) l = NAN;
    if (whole) {
      float f = l == 0.0f ? 0.0f : 1.0f / l;
      if (DT == kE4m3 && !TS && a.c.v_scale != nullptr) f *= a.c.v_scale[w.h];
      const long long head = (long long)(w.r.row0 + i) * a.Hq + w.h * a.g + (r - i * a.g);
      char* to = a.out + head * (kD * 2);
      if (r < M && a.lse != nullptr) a.lse[head] = (m - F::kShift + log2f(l)) * kLn2;
#pragma unroll 1
      for (int c = 0; c < 4; ++c) {
        uint32_t x[32];
        tmem_ld(o_at + 32 * c, x);
        tmem_wait_ld(x);
        if (r >= M) continue;
#pragma unroll
        for (int e = 0; e < 32; ++e) x[e] = l == 0.0f ? 0u : __float_as_uint(__uint_as_float(x[e]) * f);
        if ((flags & kLoose) && l != 0.0f)
          for (int e = 0; e < 32; ++e) {
            const float y = loose<DT>(a, w.r, w.b, w.h, i, 32 * c + e);
#pragma unroll
            for (int d = 0; d < 32; ++d)
              if (d == e) x[d] = __float_as_uint(__uint_as_float(x[d]) + y);
          }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          uint4 y;
#pragma unroll
          for (int d = 0; d < 4; ++d)
            (&y.x)[d] = pack<QT == kBf16>(__uint_as_float(x[8 * e + 2 * d]), __uint_as_float(x[8 * e + 2 * d + 1]));
          *reinterpret_cast<uint4*>(to + 64 * c + 16 * e) = y;
        }
      }
    } else {
      float* slot = reinterpret_cast<float*>(a.ws + slots_offset(gridDim.x)) +
                    size_t(2 * blockIdx.x + (w.begin > 0 ? 0 : 1)) * slot_floats(F::kRows);
      const int row = threadIdx.x;
#pragma unroll 1
      for (int c = 0; c < 4; ++c) {
        uint32_t x[32];
        tmem_ld(o_at + 32 * c, x);
        tmem_wait_ld(x);
#pragma unroll
        for (int e = 0; e < 8; ++e)
          *reinterpret_cast<uint4*>(slot + (size_t(8 * c + e) * F::kRows + row) * 4) =
              make_uint4(x[4 * e], x[4 * e + 1], x[4 * e + 2], x[4 * e + 3]);
      }
      slot[size_t(F::kRows) * kD + row] = m - F::kShift;
      slot[size_t(F::kRows) * (kD + 1) + row] = l;
      if (row == 0) slot[size_t(F::kRows) * (kD + 2)] = __int_as_float(flags);
    }
  }
};

// ---------------------------------------------------------------- producers

template <int DT, int QT, int TILES, bool TS>
__device__ __forceinline__ void produce(const TreeArgs& a, Smem<Form<DT, QT, TILES, TS>>& S,
                                        Walk<Form<DT, QT, TILES, TS>::kRows> w, long long s0, long long e0) {
  using F = Form<DT, QT, TILES, TS>;
  const int thread = int(threadIdx.x) - F::kSoftmaxWarps * 32, warp = thread >> 5, lane = thread & 31;
  const uint32_t slots = smem_addr(S.slot), raws = smem_addr(S.raw) + thread * 16;
  struct Past {  // a copy in flight: from which of the tile's tokens on values may be replaced, and the unit
    int from, number;
  } past[F::kLag + 1];
#pragma unroll
  for (int i = 0; i <= F::kLag; ++i) past[i] = Past{kTile, 0};
  constexpr int kFirst = F::kLag % 2;  // the half of a tile in which a copy of keys is looked at
  constexpr int kHalves = kD * elem_bytes<DT>() / 128;  // 128-byte pieces of a row

  // Copy number x (K of a tile, then V) has landed: makes it an operand. (Of 16-bit rows only the drafted values come
  // here; the others arrive by themselves.)
  auto land = [&](uint32_t x, const Past& p, auto is_value) -> bool {
    constexpr bool value = decltype(is_value)::value;
    const uint32_t slot = x % F::kSlots;
    const uint32_t to = slots + slot * kSlotBytes;
    if constexpr (F::kNarrow) {
      if (!mbar_wait(&S.empty[slot], (x / F::kSlots + 1) & 1u, &S.abort)) return false;
      const uint32_t from = raws + (x % F::kStages) * kRawBytes;
      uint4 y[8];  // 16 channels of eight tokens
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] = lds16(from + i * (kProducers * 16));
      if (value && p.from < kTile) {  // drafted tokens: NaN is replaced by 0
        uint32_t any = 0u;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          if (32 * warp + 4 * i + (lane >> 3) < p.from) continue;
#pragma unroll
          for (int d = 0; d < 4; ++d) {
            const uint32_t nan = (((&y[i].x)[d] & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;  // bytes of 0x7F or 0xFF
            (&y[i].x)[d] &= ~((nan >> 7) * 255u);
            any |= nan;
          }
        }
        if (any != 0u) atomicOr(&S.flags[p.number & 7], kLoose);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int token = 32 * warp + 4 * i + (lane >> 3), chunk = 2 * (lane & 7);
        uint2 z[4];
#pragma unroll
        for (int d = 0; d < 4; ++d) z[d] = widen<value ? F::kValBf : F::kKeyBf>((&y[i].x)[d]);
        sts16(to + chunk_at(token, chunk), make_uint4(z[0].x, z[0].y, z[1].x, z[1].y));
        sts16(to + chunk_at(token, chunk + 1), make_uint4(z[2].x, z[2].y, z[3].x, z[3].y));
      }
    } else if constexpr (value) {  // drafted ones
      constexpr uint32_t kInf = DT == kBf16 ? 0x7F80u : 0x7C00u;
#pragma unroll 1
      for (int e = 0; e < 16; ++e) {
        const int token = 32 * warp + 4 * (e >> 1) + (lane >> 3), chunk = 8 * (e & 1) + (lane & 7);
        if (token < p.from) continue;
        const uint32_t at = to + chunk_at(token, chunk);
        uint4 y = lds16(at);
        bool any = false;
#pragma unroll
        for (int d = 0; d < 4; ++d) {
          uint32_t& v = (&y.x)[d];
          if ((v & kInf) == kInf) {
            v &= 0xFFFF0000u;
            any = true;
          }
          if (((v >> 16) & kInf) == kInf) {
            v &= 0x0000FFFFu;
            any = true;
          }
        }
        if (any) {
          sts16(at, y);
          atomicOr(&S.flags[p.number & 7], kLoose);
        }
      }
    }
    fence_async_smem();
    mbar_arrive(&S.full[slot]);
    return true;
  };

  // The pool's row of this lane's token (32 warp + lane) of a tile: page of the pool (looked up a tile ahead)
  auto page_of = [&](const Walk<F::kRows>& u, int k) {
    const int t = k * kTile + 32 * warp + lane;
    return t < u.tokens ? a.table[(long long)u.b * a.max_pages + a.c.ps.div(t)] : -2;  // -2: no token
  };
  uint32_t x = 0;
  int page = page_of(w, w.begin);
  for (bool more = true; more;) {
    for (int k = w.begin; k < w.end; ++k) {
      const int t = k * kTile + 32 * warp + lane;
      long long off = -1;
      if (page >= 0 && page < a.c.n_pages) {
        const int place = t - a.c.ps.div(t) * int(a.c.ps.d);
        off = (long long)page * a.c.page_stride + (long long)place * a.c.token_stride + (long long)w.h * a.c.head_stride;
      } else if (page != -2 || t < w.tokens) {
        flag(a.c, KVQ_PAGED_ERR_PAGE);
        atomicOr(&S.flags[w.number & 7], kBadPage);
      }
      if (k + 1 < w.end) page = page_of(w, k + 1);
      const Past now{max(0, min(kTile, w.r.P - k * kTile)), w.number};
#pragma unroll
      for (int half = 0; half < 2; ++half, ++x) {
        const char* pool = half == 0 ? a.c.k : a.c.v;
        uint32_t to = 0;
        if constexpr (!F::kNarrow) {
          if (!mbar_wait(&S.empty[x % F::kSlots], (x / F::kSlots + 1) & 1u, &S.abort)) return;
          to = slots + (x % F::kSlots) * kSlotBytes;
        } else {
          to = raws + (x % F::kStages) * kRawBytes;
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const long long y = __shfl_sync(0xFFFFFFFFu, off, 4 * e + (lane >> 3));
#pragma unroll
          for (int f = 0; f < kHalves; ++f) {
            const int chunk = 8 * f + (lane & 7);
            const uint32_t at = F::kNarrow ? to + e * (kProducers * 16)
                                           : to + chunk_at(32 * warp + 4 * e + (lane >> 3), chunk);
            copy16(at, pool + (y < 0 ? 0 : y) + chunk * 16, y >= 0);
          }
        }
        commit();
#pragma unroll
        for (int i = F::kLag; i > 0; --i) past[i] = past[i - 1];
        past[0] = now;
        if constexpr (!F::kNarrow)
          if (half == 0 || now.from == kTile) {
            arrive_landed(&S.full[x % F::kSlots]);
            past[0].from = kTile;
          }
        if (F::kNarrow ? x >= uint32_t(F::kLag) : past[F::kLag].from < kTile) {
          wait_groups<F::kLag>();
          if (half == kFirst ? !land(x - F::kLag, past[F::kLag], std::false_type{})
                             : !land(x - F::kLag, past[F::kLag], std::true_type{}))
            return;
        }
      }
    }
    more = w.next(a, s0, e0);
    if (more) page = page_of(w, w.begin);
  }
  wait_groups<0>();
#pragma unroll
  for (int i = F::kLag - 1; i >= 0; --i)  // (the last one was of values)
    if (F::kNarrow ? x >= uint32_t(i + 1) : past[i].from < kTile)
      if (i % 2 ? !land(x - 1 - i, past[i], std::false_type{}) : !land(x - 1 - i, past[i], std::true_type{})) return;
}

// ---------------------------------------------------------------- products

template <int DT, int QT, int TILES, bool TS>
__device__ __forceinline__ bool multiply(const TreeArgs& a, Smem<Form<DT, QT, TILES, TS>>& S,
                                         Walk<Form<DT, QT, TILES, TS>::kRows> w, long long s0, long long e0) {
  using F = Form<DT, QT, TILES, TS>;
  const uint32_t tmem = S.tmem, q = smem_addr(S.q), slots = smem_addr(S.slot);
  uint32_t x = 0;             // slots so far
  uint32_t count[2] = {0, 0};  // products of each row tile so far
  uint32_t units = 0;
  auto keys = [&](int tile, uint32_t x, uint32_t buf) {
    const uint64_t qa = smem_desc(q + tile * kSlotBytes, 16), kb = smem_desc(slots + (x % F::kSlots) * kSlotBytes, 16);
#pragma unroll
    for (uint32_t k = 0; k < 8; ++k) {  // 16 channels: 32 bytes on, four times in each half
      const uint32_t on = 2u * (k & 3u) + (kSlotBytes / 32) * (k >> 2);
      mma_ss(tmem + 256u + 128u * buf, qa + on, kb + on, instr_desc(F::kKeyBf, false), k > 0);
    }
    mma_commit(&S.s_full[buf]);
  };
  auto values = [&](int tile, uint32_t x, uint32_t buf, bool first) {
    const uint64_t vb = smem_desc(slots + (x % F::kSlots) * kSlotBytes, kSlotBytes / 2);
#pragma unroll
    for (uint32_t k = 0; k < 8; ++k)  // 16 tokens: 2048 bytes on
      mma_ts(tmem + 128u * tile, tmem + 256u + 128u * buf + 8u * k, vb + 128u * k, instr_desc(F::kValBf, true),
             !first || k > 0);
    mma_commit(&S.pv_done[tile]);
  };
  auto filled = [&](uint32_t x) {
    if (!mbar_wait(&S.full[x % F::kSlots], (x / F::kSlots) & 1u, &S.abort)) return false;
    if constexpr (!F::kNarrow) fence_async_smem();  // (copies that arrive by themselves have no fence behind them)
    tc_fence_after();
    return true;
  };
  auto weights = [&](uint32_t buf, uint32_t phase) {
    if (!mbar_wait(&S.p_ready[buf], phase & 1u, &S.abort)) return false;
    tc_fence_after();
    return true;
  };
  for (bool more = true; more; more = w.next(a, s0, e0)) {
    if (!mbar_wait(&S.q_full, units++ & 1u, &S.abort)) return false;
    tc_fence_after();
    const int n = w.end - w.begin;
    if constexpr (TILES == 1) {
      // scores of tile k + 1 are under way while the softmax warps work on tile k's
      for (int k = 0; k <= n; ++k) {
        if (k < n) {
          if (!filled(x + 2 * k)) return false;
          keys(0, x + 2 * k, (count[0] + k) & 1u);
          mma_commit(&S.empty[(x + 2 * k) % F::kSlots]);
        }
        if (k > 0) {
          const uint32_t c = count[0] + k - 1, y = x + 2 * (k - 1) + 1;
          if (!filled(y) || !weights(c & 1u, c >> 1)) return false;
          values(0, y, c & 1u, k == 1);
          mma_commit(&S.empty[y % F::kSlots]);
        }
      }
      count[0] += n;
    } else {
      const bool both = w.rb * F::kRows + kTile < w.r.n * a.g;  // the second row tile has rows
      for (int k = 0; k <= n; ++k)
        for (int tile = 0; tile < 2; ++tile) {  // a row tile's products while the other's softmax runs
          const bool on = tile == 0 || both, last = tile == 1;
          if (k > 0) {
            const uint32_t y = x + 2 * (k - 1) + 1;
            if (on) {
              if (!filled(y) || !weights(tile, count[tile])) return false;
              values(tile, y, tile, k == 1);
              ++count[tile];
            }
            if (last) mma_commit(&S.empty[y % F::kSlots]);
          }
          if (k < n) {
            if (on) {
              if (!filled(x + 2 * k)) return false;
              keys(tile, x + 2 * k, tile);
            }
            if (last) mma_commit(&S.empty[(x + 2 * k) % F::kSlots]);
          }
        }
    }
    x += 2 * n;
  }
  return true;
}

// ---------------------------------------------------------------- kernels

template <int DT, int QT, int TILES, bool TS>
__global__ void __launch_bounds__(Form<DT, QT, TILES, TS>::kThreads, 1) tree_kernel(const __grid_constant__ TreeArgs a) {
  using F = Form<DT, QT, TILES, TS>;
  constexpr int R = F::kRows;
  extern __shared__ __align__(1024) char smem[];
  Smem<F>& S = *reinterpret_cast<Smem<F>*>(smem);
  wait_prior_grid();
  allow_dependents();
  const int warp = threadIdx.x >> 5;
  if (threadIdx.x == 0) {
    reinterpret_cast<Rec*>(a.ws)[blockIdx.x] = Rec{0, 0, 0, 0};
    for (int i = 0; i < F::kSlots; ++i) {
      mbar_init(&S.full[i], kProducers);
      mbar_init(&S.empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&S.s_full[i], 1);
      mbar_init(&S.p_ready[i], 4);
      mbar_init(&S.pv_done[i], 1);
    }
    mbar_init(&S.q_full, F::kSoftmaxWarps);
    mbar_init(&S.drain, 1);
    for (int i = 0; i < 8; ++i) S.flags[i] = 0;
    S.abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  // requests that are refused: no block's range holds them
  for (int b = blockIdx.x; b < a.B; b += gridDim.x) {
    Request r;
    r.load(a, b);
    if (!r.refused) continue;
    if (threadIdx.x == 0) flag(a.c, KVQ_PAGED_ERR_LENGTH);
    const int n = row_range(a.offsets, a.n_rows, b, r.row0);
    const uint32_t nan = QT == kBf16 ? 0x7FC07FC0u : 0x7E007E00u;
    for (long long i = threadIdx.x; i < (long long)max(n, 0) * a.Hq * (kD / 2); i += F::kThreads)
      reinterpret_cast<uint32_t*>(a.out)[(long long)r.row0 * a.Hq * (kD / 2) + i] = nan;
    if (a.lse != nullptr)
      for (long long i = threadIdx.x; i < (long long)max(n, 0) * a.Hq; i += F::kThreads)
        a.lse[(long long)r.row0 * a.Hq + i] = NAN;
  }
  auto work_of = [&](int b) {
    Request r;
    r.load(a, b);
    return r.n > 0 ? r.work(a, R) * a.c.H : 0LL;
  };
  build_prefix<F::kThreads>(S.prefix, a.B, work_of);
  // ranges: none is empty, so the parts of a unit are those of adjacent blocks
  const long long W = S.prefix.pre[F::kThreads];
  const int C = int(min(W, (long long)gridDim.x)), c = blockIdx.x;
  if (c >= C) return;
  const long long s0 = part_start(c, W, C), e0 = part_start(c + 1, W, C);
  Walk<R> w;
  long long at = s0;
  const int b = find_request<F::kThreads>(S.prefix, a.B, work_of, at);
  if (!w.open(a, b, at, s0, e0)) return;  // (the same for all threads)
  if (warp == F::kMmaWarp) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(&S.tmem)),
                 "n"(kTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();  // (and nobody reads the prefix any more)
  tc_fence_after();

  if (warp < F::kSoftmaxWarps) {
    more_registers<F::kSoftmaxRegs>();
    Softmax<DT, QT, TILES, TS> K(a, S);
    K.run(w, s0, e0, W, C);
  } else if (warp < F::kMmaWarp) {
    fewer_registers<F::kProducerRegs>();
    produce<DT, QT, TILES, TS>(a, S, w, s0, e0);
    wait_groups<0>();
  } else {
    fewer_registers<F::kMmaRegs>();
    if (threadIdx.x == F::kMmaWarp * 32) {
      multiply<DT, QT, TILES, TS>(a, S, w, s0, e0);
      // the products in flight end before the tensor memory is freed
      mma_commit(&S.drain);
      int never = 0;
      mbar_wait(&S.drain, 0, &never);
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (threadIdx.x == 0 && S.abort) flag(a.c, KVQ_PAGED_ERR_WAIT);
  if (warp == F::kMmaWarp) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(S.tmem), "n"(kTmemCols) : "memory");
  }
}

// Joins the parts of a unit that several blocks' ranges share: block (c, y) those of the unit that begins in block c's
// range, its rows 32 y .. 32 y + 31, a lane a row, a warp 16 channels of it (and every other part).
constexpr int kJoinWarps = 16;

template <int DT, int QT, int TILES>
__global__ void __launch_bounds__(kJoinWarps * 32) join_kernel(const __grid_constant__ TreeArgs a) {
  constexpr int R = kTile * TILES;
  __shared__ float s_ml[2][32];
  __shared__ float4 s_x[8][4][32];
  wait_prior_grid();
  allow_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, group = warp & 7, odd = warp >> 3;
  const Rec rec = reinterpret_cast<const Rec*>(a.ws)[blockIdx.x];
  // (the bounds hold for every record of the attention kernel; a workspace that something else writes meanwhile must
  // not lead outside of it)
  const int n = gridDim.x;
  if (rec.parts < 2 || rec.parts > n - int(blockIdx.x) || rec.b < 0 || rec.b >= a.B || rec.h < 0 || rec.h >= a.c.H ||
      rec.rb < 0)
    return;
  Request r;
  r.load(a, rec.b);
  const int M = r.n * a.g, row = 32 * blockIdx.y + lane, at = rec.rb * R + row;
  if (rec.rb * R + 32 * int(blockIdx.y) >= M) return;
  const float* slots = reinterpret_cast<const float*>(a.ws + slots_offset(n));
  float m = -INFINITY, l = 0.0f;
  float4 x[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) x[e] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  int flags = 0;
  for (int i = odd; i < rec.parts; i += 2) {
    const float* p = slots + size_t(i == 0 ? 2 * blockIdx.x + 1 : 2 * (blockIdx.x + i)) * slot_floats(R);
    const float pm = p[size_t(R) * kD + row], pl = p[size_t(R) * (kD + 1) + row];
    flags |= __float_as_int(p[size_t(R) * (kD + 2)]);
    float4 y[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) y[e] = *reinterpret_cast<const float4*>(p + (size_t(4 * group + e) * R + row) * 4);
    const float top = fmaxf(m, pm), base = top == -INFINITY ? 0.0f : top, f = exp2f(m - base), g = exp2f(pm - base);
    m = top;
    l = l * f + pl * g;
#pragma unroll
    for (int e = 0; e < 4; ++e)
      x[e] = make_float4(fmaf(g, y[e].x, x[e].x * f), fmaf(g, y[e].y, x[e].y * f), fmaf(g, y[e].z, x[e].z * f),
                         fmaf(g, y[e].w, x[e].w * f));
  }
  if (odd) {
#pragma unroll
    for (int e = 0; e < 4; ++e) s_x[group][e][lane] = x[e];
    if (group == 0) {
      s_ml[0][lane] = m;
      s_ml[1][lane] = l;
    }
  }
  flags = __syncthreads_or(flags & kLoose);
  if (odd || at >= M) return;
  const float pm = s_ml[0][lane], top = fmaxf(m, pm), base = top == -INFINITY ? 0.0f : top, f = exp2f(m - base),
              g = exp2f(pm - base);
  l = l * f + s_ml[1][lane] * g;
  const int i = at / a.g;
  const long long head = (long long)(r.row0 + i) * a.Hq + rec.h * a.g + (at - i * a.g);
  float inv = l == 0.0f ? 0.0f : 1.0f / l;
  if (DT == kE4m3 && !a.c.token_scales && a.c.v_scale != nullptr) inv *= a.c.v_scale[rec.h];
  uint32_t y[8];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float4 z = s_x[group][e][lane];
    float4 v = make_float4(fmaf(g, z.x, x[e].x * f), fmaf(g, z.y, x[e].y * f), fmaf(g, z.z, x[e].z * f),
                           fmaf(g, z.w, x[e].w * f));
    v = l == 0.0f ? make_float4(0.0f, 0.0f, 0.0f, 0.0f) : times(v, inv);
    if (flags && l != 0.0f) {
      v.x += loose<DT>(a, r, rec.b, rec.h, i, 16 * group + 4 * e);
      v.y += loose<DT>(a, r, rec.b, rec.h, i, 16 * group + 4 * e + 1);
      v.z += loose<DT>(a, r, rec.b, rec.h, i, 16 * group + 4 * e + 2);
      v.w += loose<DT>(a, r, rec.b, rec.h, i, 16 * group + 4 * e + 3);
    }
    y[2 * e] = pack<QT == kBf16>(v.x, v.y);
    y[2 * e + 1] = pack<QT == kBf16>(v.z, v.w);
  }
  uint4* to = reinterpret_cast<uint4*>(a.out + head * (kD * 2) + group * 32);
  to[0] = make_uint4(y[0], y[1], y[2], y[3]);
  to[1] = make_uint4(y[4], y[5], y[6], y[7]);
  if (a.lse != nullptr && group == 0) a.lse[head] = (top + log2f(l)) * kLn2;
}

template <int DT, int QT, int TILES, bool TS>
cudaError_t launch_form(const TreeArgs& a, cudaStream_t stream) {
  using F = Form<DT, QT, TILES, TS>;
  const int smem = int(sizeof(Smem<F>));
  static_assert(sizeof(Smem<F>) <= 232448, "shared memory of a block");
  static std::atomic<uint64_t> configured{0};  // bit: device
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (!((configured.load(std::memory_order_relaxed) >> dev) & 1)) {
    e = cudaFuncSetAttribute(tree_kernel<DT, QT, TILES, TS>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    configured.fetch_or(uint64_t(1) << dev, std::memory_order_relaxed);
  }
  count_launch();
  e = launch_dependent(tree_kernel<DT, QT, TILES, TS>, dim3(a.sms), dim3(F::kThreads), size_t(smem), stream, a);
  if (e != cudaSuccess) return e;
  const long long rows = min((long long)a.n_rows * a.g, (long long)F::kRows);  // of a unit, at most
  count_launch();
  return launch_dependent(join_kernel<DT, QT, TILES>, dim3(a.sms, int((rows + 31) / 32)), dim3(kJoinWarps * 32), 0,
                          stream, a);
}

// Two row tiles per block where the requests' mean rows fill more than one.
int row_tiles(int B, int g, int n_rows) { return ((long long)n_rows + B - 1) / (B > 0 ? B : 1) * g > kTile ? 2 : 1; }

template <int DT, int QT>
cudaError_t launch_types(const TreeArgs& a, cudaStream_t stream) {
  const bool two = row_tiles(a.B, a.g, a.n_rows) == 2;
  if constexpr (DT == kE4m3)
    if (a.c.token_scales) return two ? launch_form<DT, QT, 2, true>(a, stream) : launch_form<DT, QT, 1, true>(a, stream);
  return two ? launch_form<DT, QT, 2, false>(a, stream) : launch_form<DT, QT, 1, false>(a, stream);
}

}  // namespace

size_t tree_workspace(int B, int H, int Hq, int n_rows, int sms) {
  return slots_offset(sms) + 2 * size_t(sms) * slot_floats(kTile * row_tiles(B, Hq / H, n_rows)) * 4;
}

cudaError_t launch_tree(const TreeArgs& a, cudaStream_t stream) {
  const bool bf = a.q_dtype == kBf16;
  if (a.dtype == kBf16) return launch_types<kBf16, kBf16>(a, stream);
  if (a.dtype == kFp16) return launch_types<kFp16, kFp16>(a, stream);
  return bf ? launch_types<kE4m3, kBf16>(a, stream) : launch_types<kE4m3, kFp16>(a, stream);
}

}  // namespace paged
}  // namespace kvq
