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
// joining kernel joins them.
//
// Both products run on tcgen05 with 128 rows: S = Q K^T, the queries in tensor memory
// (one row tile) or in shared memory (two: sums and scores fill tensor memory), and
// O += P V with P in tensor memory, where the softmax warps leave it in the place of
// S. A block's warps:
//   softmax   four per row tile, a thread a row: no shuffles; the sums of a row are
//             rescaled only when its maximum grows by more than 2^8, with scales per
//             token 2^4 (its weights then go to at most 1, or 2^15 for FP16, by
//             kShift). A unit of up to 64 (32)
//             rows is in the row tile twice (four times), each copy for its share of
//             a tile's tokens, else a few rows would leave three warps of four idle
//   producers four: 16-byte asynchronous copies of K and V rows into a ring of
//             operand slots; 8-bit rows into a ring of their own, from which the same
//             threads convert them (one row tile: two groups of four, which take the
//             tiles in turn)
//   MMA       one, which stays together and elects a lane to issue the products: their
//             descriptors are then the warp's and computed once (issued by a lone
//             thread wide trees took 240 us for 235, of E4M3 271 for 251; in a loop that
//             is not unrolled 278: a product's issue is on the rows' critical path)
//   screeners two, for drafted values of 16-bit rows (below); or two that look up the
//             scales of a tile's tokens
// Exactness: products of 16-bit values are exact, sums FP32. 8-bit keys become 16-bit
// numbers of the queries' type, 8-bit values FP16, both exactly. A weight is one
// 16-bit number: of BF16 for BF16 caches (its operand's type is the values'), of FP16
// for the others, there down to 2^-31 of the largest weight with values' scales
// (where tokens have them) multiplied in before the rounding. That adds 4 to 9% to the
// error that the rounding of the result leaves; three parts would triple the second
// product, which bounds wide trees.
//
// A drafted token's value that is not finite must not reach rows that do not see it
// (0 x infinity): the screeners, or the conversion, replace it by 0, and the rows that
// see it get it back at the end (loose).
//
// Every wait is bounded (2 s). When one runs out an error bit is set; producers,
// products and screeners leave, whole warps at a time; the softmax warps, which meet at
// barriers of their own, go through their tiles without waiting; products in flight end
// before the tensor memory is freed. (With waits that have a limit in those barriers'
// place one token each of E4M3 took 205 us for 176.)
//
// Bound: few rows, HBM (each cached row is read once); from about 128 rows a KV head on
// a row tile's chain of product, softmax (128 x 128 exponentials) and product. Measured,
// 8 KV heads, BF16 but where said (from one GPU to another 2-3% less): 64 requests of up
// to 16383 tokens, one new token each, 172 us, 6.1 TB/s (91% of a copy's rate); 512 x 1000
// tokens, four new ones each, 338 us (95%); trees of 16 over 64 requests of up to 4095
// tokens 95 us, 5.2 TB/s; trees of 64, 64 heads, over 8 x 16384 tokens 223 us, 1.23
// PFLOP/s (in a long run of calls 241, 1.14 PFLOP/s); 4 x 65535 tokens of E4M3 with a scale
// per token 176 us, with one per head 132. One token each over E4M3, 64 requests: with a
// scale per token 177 us (3.1 TB/s), with one per head 161; every 8-bit row is widened in
// shared memory for products of 128 rows of which four are real, and
// kvq_paged_decode_attn, which widens in registers, takes 92.5 for the latter.
// The block's roles share an instruction cache, and their code is kept in loops for
// it: unrolled forms stalled on instructions more than on anything else (4 x 65535
// tokens of E4M3 with a scale per token 330 us, 176 now).
#include <atomic>
#include <type_traits>

#include "kvq_attn_common.cuh"
#include "kvq_paged.cuh"

namespace kvq {
namespace paged {
namespace {

constexpr int kTile = 128;       // tokens of a tile, rows of a row tile
constexpr int kScaleRing = 4;    // tiles whose scales are there at a time
constexpr int kUnitCost = 2;     // tiles that the end of a unit takes as long as (64 requests of one token: 1 176 us, 2 170, 3 171)
constexpr int kSlotBytes = kTile * kD * 2;
constexpr int kRawBytes = kTile * kD;
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kColS = 256;  // scores and weights: two buffers of 128 columns; the sums are at 0 (and 128: second row tile)
constexpr uint32_t kColQ = 128;  // one row tile: queries, two buffers of 64
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr float kSlack = 8.0f;   // log2 of what a row's weights may exceed 1 by before its sums are rescaled (Form::kRise)
constexpr int kWaitTries = 1 << 19;  // of a wait, each of up to 4.1 us: 2 s

// ---------------------------------------------------------------- forms

template <int DT, int QT, int TILES, bool TS>
struct Form {
  static constexpr bool kNarrow = DT == kE4m3;
  static constexpr bool kKeyBf = DT == kBf16 || (kNarrow && QT == kBf16);  // type of Q and K operands
  static constexpr bool kValBf = DT == kBf16;                              // type of P and V operands
  // With scales per token the sums are to a bound of the products of weights and scales, which is up to 2^kNear above the
  // largest product: that comes off the slack, so that FP16 holds the largest product at 2^7 or more in any case (its
  // smallest step is 2^-31 of that) and at 2^15 at most. (Scales within 2^kNear spare the look for the largest product:
  // wide trees 324 us, with it 362. Two for four leaves more slack, 323, and more tiles that have to look.)
  static constexpr float kNear = TS ? 4.0f : 0.0f;
  static constexpr float kRise = kSlack - kNear;  // log2 of what the products may grow by before the sums are rescaled
  static constexpr float kShift = kValBf ? -kRise : 15.0f - kRise;
  static constexpr int kRows = kTile * TILES;
  static constexpr int kSoftmaxWarps = 4 * TILES;
  // groups of four producer warps, which take the tiles in turn: 8-bit rows are copied, converted and stored by the same
  // threads, one after the other, and two groups do it side by side (eight warps together were slower: 64 requests of
  // one token, a scale per head, 244 us then, 207 in turn, with a warp of its own for the scales per token)
  static constexpr int kGroups = kNarrow && TILES == 1 ? 2 : 1;
  static constexpr int kProducerWarps = 4 * kGroups;
  static constexpr int kProducers = 128;  // threads of a group
  static constexpr int kMmaWarp = kSoftmaxWarps + kProducerWarps;
  static constexpr int kThreads = (kMmaWarp + 4) * 32;  // (registers are shared out by four warps)
  // registers of the softmax, producer and MMA warps, by four of which they come to 3 x 168 or 4 x 128 of the launch
  static constexpr int kSoftmaxRegs = kThreads == 384 ? 224 : TILES == 1 ? 176 : 144;
  static constexpr int kProducerRegs = kThreads == 384 ? 152 : 112;
  static constexpr int kMmaRegs = kThreads == 384 ? 128 : 112;
  static_assert(kSoftmaxRegs * TILES + kProducerRegs * kProducerWarps / 4 + kMmaRegs == (kThreads == 384 ? 504 : 512));
  // One row tile: the queries are in tensor memory, two units' (A of the products); two fill it with sums and scores.
  static constexpr int kQueries = TILES == 1 ? 0 : kRows;
  static constexpr int kSlots = kNarrow ? (TILES == 1 ? 4 : 3) : TILES == 1 ? 6 : 5;
  static constexpr int kStages = kNarrow ? (TILES == 1 ? 2 : 3) : 0;  // a group's 8-bit rows as they come
  static constexpr int kScreeners = kNarrow ? 0 : 64;  // threads (two warps behind the MMA warp) that check drafted values
};

template <class F>
struct Smem {
  union {
    char slot[F::kSlots][kSlotBytes];
    Prefix<F::kThreads> prefix;  // before the first copy
  };
  char q[F::kQueries > 0 ? F::kQueries * kD * 2 : 16];
  char raw[F::kStages > 0 ? F::kGroups * F::kStages : 1][F::kStages > 0 ? kRawBytes : 16];
  // scales of a tile's tokens: the keys' (into log2 units), the logarithms of the values', the values'; and the smallest
  // and largest of those logarithms
  float scales[F::kNarrow ? kScaleRing : 1][3][F::kNarrow ? kTile : 4];
  float2 range[kScaleRing][2];
  unsigned long long scales_full[kScaleRing], scales_free[kScaleRing];
  // one row tile: what its copies of the rows are joined by
  float part[F::kQueries > 0 ? 1 : kTile][33];
  float part_ml[3][F::kQueries > 0 ? 1 : kTile];
  unsigned long long full[F::kSlots], empty[F::kSlots];
  unsigned long long raw_full[F::kSlots];  // 16-bit drafted values, before they are checked
  unsigned long long s_full[2], p_ready[2], pv_done[2], q_full[2], q_free[2], o_free, drain;
  uint32_t tmem;
  int bad_page[16];  // of the unit by its number's last bits
  int loose;         // some drafted value was replaced
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
// Waits for the phase of this parity; false when it took kWaitTries, or another wait of the block did. (Tries are counted,
// not the time, which goes on while a kernel is set aside.)
__device__ __forceinline__ bool mbar_wait_long(unsigned long long* bar, uint32_t parity, volatile int* abort) {
#pragma unroll 1
  for (int i = 0; i < kWaitTries; ++i) {
    if (*abort) return false;
    if (mbar_try_wait(bar, parity)) return true;
  }
  *abort = 1;
  return false;
}
__device__ __forceinline__ bool mbar_wait(unsigned long long* bar, uint32_t parity, volatile int* abort) {
  return mbar_try_wait(bar, parity) || mbar_wait_long(bar, parity, abort);
}
// The same by a whole warp, with one answer for all lanes: what it does next takes all of them.
__device__ __forceinline__ bool warp_wait(unsigned long long* bar, uint32_t parity, volatile int* abort) {
  return __all_sync(0xFFFFFFFFu, mbar_try_wait(bar, parity)) || __all_sync(0xFFFFFFFFu, mbar_wait_long(bar, parity, abort));
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

// One lane of a warp that is together.
__device__ __forceinline__ bool elect() {
  uint32_t ok;
  asm volatile("{ .reg .pred p; elect.sync _|p, 0xFFFFFFFF; selp.u32 %0, 1, 0, p; }" : "=r"(ok));
  return ok != 0;
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
__device__ __forceinline__ void tmem_st(uint32_t at, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
      "%15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(at),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
      "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
      "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
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
// All of this thread's copies, those that are in no group among them.
__device__ __forceinline__ void wait_copies() { asm volatile("cp.async.wait_all;" ::: "memory"); }
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
__device__ __forceinline__ float4 lds4(uint32_t a) {
  float4 v;
  asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(a) : "memory");
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
    P = checked_len(a.lens, b, a.max_pages, a.c.ps);
    n = row_range(a.offsets, a.n_rows, b, row0);
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
#pragma unroll 1
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
#pragma unroll 1
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
#pragma unroll 1
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

// A unit of few rows has them in the row tile several times, each copy for its own share of a tile's tokens, so that all
// softmax warps have work (the products take 128 rows in any case): the copies of M rows in all.
__device__ __forceinline__ int copies(int M) { return M <= kTile / 4 ? 4 : M <= kTile / 2 ? 2 : 1; }

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
// Workspace: Rec[n], int[n] (a block replaced some drafted value), 2 n slots: sums [32][rows][4], then by row the
// weights' maximum and sum and what the sums are to.
__host__ __device__ constexpr size_t loose_offset(int n) { return size_t(n) * sizeof(Rec); }
__host__ __device__ constexpr size_t slots_offset(int n) { return loose_offset(n) + (size_t(n) * 4 + 15) / 16 * 16; }
__host__ __device__ constexpr size_t slot_floats(int rows) { return size_t(rows) * (kD + 3); }

// ---------------------------------------------------------------- softmax warps

// scale ks, whose product may leave FP32's normal range where the logits do not
__device__ __forceinline__ float scaled(float scale, float ks) {
  const float x = scale * ks;
  return isfinite(ks) ? fminf(fmaxf(x, 0x1p-149f), 3.402823466e38f) : ks;
}

// FP32 numbers as whole numbers in the same order, and back.
__device__ __forceinline__ int in_order(float x) {
  const int i = __float_as_int(x);
  return i ^ ((i >> 31) & 0x7FFFFFFF);
}
__device__ __forceinline__ float in_order(int i) { return __int_as_float(i ^ ((i >> 31) & 0x7FFFFFFF)); }

// 2^x / l as two factors f and g (l or a scale may take either out of FP32's range where the product with a sum stays
// in it): f comes in as 1 / l.
__device__ __forceinline__ void between(float x, float& f, float& g) {
  const float half = rintf(0.5f * x);
  f *= exp2f(fminf(fmaxf(half, -126.0f), 127.0f));
  g = exp2f(fminf(fmaxf(x - half, -126.0f), 127.0f));
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

  // A wait that runs out is noted (S.abort), and the warp goes on with what is there: its reads and writes are in bounds
  // whatever they find, the waits that follow end after a try, and all lanes and warps come to the barriers that they
  // share. (Warps that left would leave others at finish_copies' barriers, which have no limit.)
  __device__ __forceinline__ void wait(unsigned long long* bar, uint32_t phase) const {
    mbar_wait(bar, phase & 1u, &S.abort);
    tc_fence_after();
  }
  __device__ __forceinline__ void sync() const { asm volatile("bar.sync %0, 128;" ::"r"(tile + 1) : "memory"); }

  // Two row tiles: the unit's queries of this tile as an operand; the warp's own 32 rows.
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
    if (lane == 0) mbar_arrive(&S.q_full[0]);
  }

  // Waits for the sums of the row tile's c-th product. (One row tile: that and the one before it may both be under way,
  // and a wait tells only odd phases from even ones: they take turns at two barriers.)
  __device__ __forceinline__ void summed(uint32_t c) const {
    wait(&S.pv_done[TILES == 1 ? c & 1u : tile], TILES == 1 ? c >> 1 : c);
  }

  struct Row {
    int P, n, i;           // the request's cached and drafted tokens, the row's drafted token
    bool live;
    const uint32_t* mask;  // (nullptr: tokens 0 .. i)
    // the weights' running maximum (log2) and sum, times 2^kShift; TS: not shifted, and `to` is the maximum of the weights
    // times the values' scales, to which the sums of values are (else to m)
    float m, l, to;
  };

  // The scores of tile k in 32 n columns, from 32 n copy on, become weights in the place of the first half of them (for
  // the other columns 0), the row's sums follow. The scores are read 32 columns at a time, for their maximum and then,
  // scaled ones (TS) from where the first reading left them, for the weights. (All in loops: unrolled, or with an instance
  // for each n, the code of a block's roles does not stay in the instruction cache beside one another: 4 x 65535 tokens
  // of 8-bit rows with a scale per head 198 us, 143 us so; 512 x 1000 tokens of 16 bits 353 and 339.)
  __device__ __forceinline__ void weigh(Row& row, int k, int begin, uint32_t count, uint32_t all, uint32_t s_at, int copy,
                                        int n, float sc) {
    const bool drafted = (k + 1) * kTile > row.P;
    // the tile's scales: a token's is the same for all lanes
    [[maybe_unused]] const uint32_t kf = smem_addr(S.scales[all % kScaleRing][0]) + 128 * n * copy, lv = kf + 4 * kTile,
                                    vf = lv + 4 * kTile;
    const uint32_t x_at = s_at + 32u * n * copy, p_at = s_at + 16u * n * copy;
    uint32_t x[32];
    auto pair = [](const uint32_t (&z)[32], int e) { return make_float2(__uint_as_float(z[e]), __uint_as_float(z[e + 1])); };
    auto put = [&](int e, float2 y) {
      x[e] = __float_as_uint(y.x);
      x[e + 1] = __float_as_uint(y.y);
    };
    auto mask = [&](int part) {
      const int j0 = k * kTile + 32 * (n * copy + part) - row.P;
      const uint32_t see = row.live ? seen_bits(row.mask, a.mask_words, row.n, row.i, j0) : 0u;
#pragma unroll
      for (int e = 0; e < 32; ++e)
        if (!((see >> e) & 1)) x[e] = 0xFF800000u;
    };
    // Two row tiles and a tile of cached tokens: for the maximum the next columns are on their way while these are worked
    // on (wide trees of 16 bits 235 us, 229 so, chunks 244 and 239; the same for the weights 229 and 237, and registers
    // went to memory).
    constexpr bool kAhead = TILES == 2 && !TS;
    [[maybe_unused]] uint32_t y[32];
    float mx = -INFINITY, nx = -INFINITY;
    // TS: the largest product of a weight and its scale: no more than the largest of each, which will do while the
    // scales are within 2^kNear of one another
    bool far = false;
    float high = -INFINITY;
    if constexpr (TS) {
      const float2 y = S.range[all % kScaleRing][0], z = S.range[all % kScaleRing][1];
      const float low = fminf(y.x, z.x);
      high = fmaxf(y.y, z.y);
      far = high - low > F::kNear;
    }
    auto highest = [&](const uint32_t (&z)[32]) {  // (in two chains: wide trees 230 us by one, 224 so)
      float top = -INFINITY;
#pragma unroll
      for (int e = 0; e < 32; e += 4) {
        mx = max3(mx, __uint_as_float(z[e]), __uint_as_float(z[e + 1]));
        top = max3(top, __uint_as_float(z[e + 2]), __uint_as_float(z[e + 3]));
      }
      mx = fmaxf(mx, top);
    };
    if (kAhead && !drafted) {
      tmem_ld(x_at, x);
#pragma unroll
      for (int part = 0; part < 4; part += 2) {
        tmem_wait_ld(x);
        tmem_ld(x_at + 32 * (part + 1), y);
        highest(x);
        tmem_wait_ld(y);
        if (part == 0) tmem_ld(x_at + 64, x);
        highest(y);
      }
    } else
#pragma unroll 1
    for (int part = 0; part < n; ++part) {
      tmem_ld(x_at + 32 * part, x);
      if constexpr (TS) {  // into log2 units
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          float4 f[4];  // (the first ones are read while the scores are on their way)
#pragma unroll
          for (int e = 0; e < 4; ++e) f[e] = lds4(kf + 4 * (32 * part + 16 * q + 4 * e));
          if (q == 0) tmem_wait_ld(x);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int i = 16 * q + 4 * e;
            put(i, __fmul2_rn(pair(x, i), make_float2(f[e].x, f[e].y)));
            put(i + 2, __fmul2_rn(pair(x, i + 2), make_float2(f[e].z, f[e].w)));
          }
        }
      } else {
        tmem_wait_ld(x);
      }
      if (drafted) mask(part);
      highest(x);
      if constexpr (TS) {
        if (far)
#pragma unroll
          for (int e = 0; e < 32; e += 4) {
            const float4 f = lds4(lv + 4 * (32 * part + e));
            const float2 y = __fadd2_rn(pair(x, e), make_float2(f.x, f.y));
            const float2 z = __fadd2_rn(pair(x, e + 2), make_float2(f.z, f.w));
            nx = max3(max3(nx, y.x, y.y), z.x, z.y);
          }
        tmem_st(x_at + 32 * part, x);
      }
    }
    if constexpr (TS) {
      if (!far) nx = mx + high;
      tmem_wait_st();
    } else {
      nx = mx *= sc;
    }
    float& top = TS ? row.to : row.m;  // what the sums are to
    if (k == begin) {
      row.m = mx;
      row.to = nx;
    } else {
      if (TS && mx > row.m + kSlack) {
        row.l *= exp2_ftz(row.m - mx);
        row.m = mx;
      }
      if (__any_sync(0xFFFFFFFFu, nx > top + F::kRise)) {
        const float to = fmaxf(top, nx), alpha = exp2_ftz(top - (to == -INFINITY ? 0.0f : to));
        top = to;
        if constexpr (!TS) row.l *= alpha;
        // the sums are at rest behind the product before
        summed(count - 1);
#pragma unroll 1
        for (int c = 0; c < 8; ++c) {
          uint32_t y[16];
          tmem_ld16(o_at + 16 * c, y);
#pragma unroll
          for (int e = 0; e < 16; ++e) y[e] = __float_as_uint(__uint_as_float(y[e]) * alpha);
          tmem_st16(o_at + 16 * c, y);
        }
      }
    }
    // TS: the weights themselves are to `to` by 2^on, so that FP16 holds the largest product with a scale, and their own
    // sum is taken back to m; what of `on` might leave FP32's range (scales near its ends) is multiplied in behind the
    // scales (2^rest times a scale may be infinite, that of a token whose weight is 0 among them). Weights below 2^-186
    // of m's are 0 then, or below 2^-66 where the products are 2^71 above it.
    [[maybe_unused]] float on = 0.0f, rest = 0.0f;
    if constexpr (TS) {
      const float x = row.to == -INFINITY ? 0.0f : row.m - row.to + F::kShift;
      on = fminf(fmaxf(x, -60.0f), 60.0f);
      rest = x - on;
    }
    [[maybe_unused]] const bool extreme = TS && __any_sync(0xFFFFFFFFu, rest != 0.0f);
    [[maybe_unused]] const float more = exp2f(rest);
    const float base = (TS ? on : F::kShift) - (row.m == -INFINITY ? 0.0f : row.m);
    float2 sum[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
#pragma unroll 1
    for (int part = 0; part < n; ++part) {
      tmem_ld(x_at + 32 * part, x);
      tmem_wait_ld(x);
      if (!TS && drafted) mask(part);
      uint32_t p[16];
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        [[maybe_unused]] float4 f[4];
        if constexpr (TS) {
#pragma unroll
          for (int e = 0; e < 4; ++e) f[e] = lds4(vf + 4 * (32 * part + 16 * q + 4 * e));
        }
#pragma unroll
        for (int i = 0; i < 16; i += 2) {
          const int e = 16 * q + i;
          float2 y;
          if constexpr (TS) y = __fadd2_rn(pair(x, e), make_float2(base, base));
          else y = __ffma2_rn(pair(x, e), make_float2(sc, sc), make_float2(base, base));
          y = make_float2(exp2_ftz(y.x), exp2_ftz(y.y));
          sum[(i >> 1) & 1] = __fadd2_rn(sum[(i >> 1) & 1], y);
          if constexpr (TS) {
            y = __fmul2_rn(y, i & 2 ? make_float2(f[i / 4].z, f[i / 4].w) : make_float2(f[i / 4].x, f[i / 4].y));
            if (extreme) y = __fmul2_rn(y, make_float2(more, more));
          }
          p[e / 2] = pack<F::kValBf>(y.x, y.y);
        }
      }
      tmem_st16(p_at + 16 * part, p);
    }
    if (n < 4) {
      uint32_t none[16];
#pragma unroll
      for (int e = 0; e < 16; ++e) none[e] = 0u;
#pragma unroll 1
      for (int c = n; c < 4; ++c) tmem_st16(s_at + 16 * ((n * copy + c) & 3), none);
    }
    sum[0] = __fadd2_rn(sum[0], sum[1]);
    row.l += TS ? (sum[0].x + sum[0].y) * exp2_ftz(-on) : sum[0].x + sum[0].y;
    tmem_wait_st();
  }

  __device__ __forceinline__ void run(Walk<F::kRows> w, long long s0, long long e0, long long W, int C) {
    uint32_t count = 0;  // tiles of this thread's row tile so far
    uint32_t units = 0;
    [[maybe_unused]] uint32_t all = 0;  // tiles so far, with those of units without rows for this row tile
    bool more = true;
    while (more) {
      if constexpr (TILES == 2) load_queries(w);
      Walk<F::kRows> next = w;  // (one row tile: looked up while there is work to do)
      if constexpr (TILES == 1) more = next.next(a, s0, e0);
      const int M = w.r.n * a.g, same = TILES == 1 ? copies(M) : 1;
      const int copy = thread / (kTile / same), r = w.rb * F::kRows + tile * kTile + thread % (kTile / same);
      const bool active = w.rb * F::kRows + tile * kTile < M;  // the row tile has rows
      // (a row tile without work must not arrive for the next unit in the same phase)
      if (TILES == 2 && !active) wait(&S.q_full[0], units);
      ++units;
      const bool rows = same > 1 || w.rb * F::kRows + tile * kTile + warp * 32 < M;  // the warp has
      Row row{w.r.P, w.r.n, r / a.g, r < M, nullptr, -INFINITY, 0.0f, -INFINITY};
      if (a.mask != nullptr && r < M) row.mask = a.mask + (long long)(w.r.row0 + row.i) * a.mask_words;
      float sc = a.scale * kLog2e;
      if constexpr (DT == kE4m3 && !TS)
        if (a.c.k_scale != nullptr) sc = scaled(sc, a.c.k_scale[w.h]);
      for (int k = w.begin; active && k < w.end; ++k, ++count) {
        const uint32_t buf = TILES == 1 ? count & 1u : uint32_t(tile), phase = TILES == 1 ? (count >> 1) & 1u : count & 1u;
        const uint32_t s_at = lanes + kColS + 128u * buf;
        if constexpr (TS) mbar_wait(&S.scales_full[all % kScaleRing], (all / kScaleRing) & 1u, &S.abort);
        wait(&S.s_full[buf], phase);
        if (rows) weigh(row, k, w.begin, count, all, s_at, same > 1 ? copy : 0, 4 / same, sc);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&S.p_ready[buf]);
          if constexpr (TS) mbar_arrive(&S.scales_free[all % kScaleRing]);
        }
        if constexpr (TS) ++all;
      }
      if constexpr (TS && TILES == 2)
        if (!active)
          for (int k = w.begin; k < w.end; ++k, ++all) {  // (the ring's places are free when all warps have passed them)
            mbar_wait(&S.scales_full[all % kScaleRing], (all / kScaleRing) & 1u, &S.abort);
            __syncwarp();
            if (lane == 0) mbar_arrive(&S.scales_free[all % kScaleRing]);
          }
      if (active) summed(count - 1);
      if (threadIdx.x == 0) S.bad_page[(w.number + 8) & 15] = 0;  // (the producers are less than eight units ahead)
      if (active) {
        if (same == 4) finish_copies<4>(w, row, r, copy);
        else if (same == 2) finish_copies<2>(w, row, r, copy);
        else if (rows) finish(w, row, r, M);
      }
      if (threadIdx.x == 0 && w.begin == 0 && w.end < w.tiles) {
        const long long last = w.pos + w.tiles - 1;
        reinterpret_cast<Rec*>(a.ws)[blockIdx.x] = Rec{w.b, w.h, w.rb, cta_of(last, W, C) - int(blockIdx.x) + 1};
      }
      tc_fence_before();
      if constexpr (TILES == 1) {
        __syncwarp();
        if (lane == 0) mbar_arrive(&S.o_free);
        w = next;
      } else {
        more = w.next(a, s0, e0);
      }
    }
  }

  // What a whole unit's sums are multiplied by, in two factors (their product may leave FP32's range where the sums times
  // one and then the other do not: 8-bit values' scales are as small as 2^-126).
  __device__ __forceinline__ float2 factors(const Walk<F::kRows>& w, const Row& row) const {
    float2 f = make_float2(row.l == 0.0f ? 0.0f : 1.0f / row.l, 1.0f);
    if (DT == kE4m3 && !TS && a.c.v_scale != nullptr) f.y = a.c.v_scale[w.h];
    if constexpr (TS) between(row.to - F::kShift - row.m, f.x, f.y);
    return f;
  }
  __device__ __forceinline__ bool is_whole(const Walk<F::kRows>& w) const { return w.begin == 0 && w.end == w.tiles; }
  __device__ __forceinline__ bool bad_page(const Walk<F::kRows>& w) const {
    return *reinterpret_cast<volatile int*>(&S.bad_page[w.number & 15]) != 0;
  }
  // Where a whole unit's row goes, in query heads.
  __device__ __forceinline__ long long head_of(const Walk<F::kRows>& w, const Row& row, int r) const {
    return (long long)(w.r.row0 + row.i) * a.Hq + w.h * a.g + (r - row.i * a.g);
  }
  __device__ __forceinline__ float* slot_of(const Walk<F::kRows>& w) const {
    return reinterpret_cast<float*>(a.ws + slots_offset(gridDim.x)) +
           size_t(2 * blockIdx.x + (w.begin > 0 ? 0 : 1)) * slot_floats(F::kRows);
  }
  __device__ __forceinline__ void put_lse(long long head, const Row& row) const {
    if (a.lse != nullptr) a.lse[head] = (row.m - (TS ? 0.0f : F::kShift) + log2f(row.l)) * kLn2;
  }
  __device__ __forceinline__ void put_slot(float* slot, int at, const Row& row) const {
    slot[size_t(F::kRows) * kD + at] = TS ? row.m : row.m - F::kShift;
    slot[size_t(F::kRows) * (kD + 1) + at] = row.l;
    slot[size_t(F::kRows) * (kD + 2) + at] = (TS ? row.to : row.m) - F::kShift;
  }
  // N channels of a whole unit's row from c on, scaled and rounded, to out.
  template <int N>
  __device__ __forceinline__ void put_out(const Row& row, long long head, int c, float (&x)[N], float2 f) const {
#pragma unroll
    for (int e = 0; e < N; ++e) x[e] = row.l == 0.0f ? 0.0f : (DT == kE4m3 ? x[e] * f.x * f.y : x[e] * f.x);
    char* to = a.out + head * (kD * 2) + c * 2;
#pragma unroll
    for (int e = 0; e < N; e += 8)
      *reinterpret_cast<uint4*>(to + 2 * e) =
          make_uint4(pack<QT == kBf16>(x[e], x[e + 1]), pack<QT == kBf16>(x[e + 2], x[e + 3]),
                     pack<QT == kBf16>(x[e + 4], x[e + 5]), pack<QT == kBf16>(x[e + 6], x[e + 7]));
  }

  // The unit's rows, or this part of it, to out and lse or to a slot.
  __device__ __forceinline__ void finish(const Walk<F::kRows>& w, Row& row, int r, int M) {
    if (bad_page(w)) row.l = NAN;
    if (is_whole(w)) {
      const float2 f = factors(w, row);
      const long long head = head_of(w, row, r);
      if (r < M) put_lse(head, row);
#pragma unroll 1
      for (int c = 0; c < 4; ++c) {
        uint32_t x[32];
        __syncwarp();  // (the lanes without a row are back)
        tmem_ld(o_at + 32 * c, x);
        tmem_wait_ld(x);
        if (r >= M) continue;
        float y[32];
#pragma unroll
        for (int e = 0; e < 32; ++e) y[e] = __uint_as_float(x[e]);
        put_out<32>(row, head, 32 * c, y, f);
      }
    } else {
      float* slot = slot_of(w);
      const int at = threadIdx.x;
#pragma unroll 1
      for (int c = 0; c < 4; ++c) {
        uint32_t x[32];
        tmem_ld(o_at + 32 * c, x);
        tmem_wait_ld(x);
#pragma unroll
        for (int e = 0; e < 8; ++e)
          *reinterpret_cast<uint4*>(slot + (size_t(8 * c + e) * F::kRows + at) * 4) =
              make_uint4(x[4 * e], x[4 * e + 1], x[4 * e + 2], x[4 * e + 3]);
      }
      put_slot(slot, at, row);
    }
  }

  // The same for rows in several copies, joined first: a thread's share is 32 / same channels of each 32 of its row.
  template <int SAME>
  __device__ __forceinline__ void finish_copies(const Walk<F::kRows>& w, Row& row, int r, int copy) {
    constexpr int kEach = kTile / SAME, kShare = 32 / SAME;
    const int at = thread % kEach, M = w.r.n * a.g;
    S.part_ml[0][thread] = row.m;
    S.part_ml[1][thread] = row.l;
    if constexpr (TS) S.part_ml[2][thread] = row.to;
    sync();
    const float mine = TS ? row.to : row.m;
    float m[SAME], l[SAME], top = -INFINITY, to = -INFINITY;
#pragma unroll
    for (int i = 0; i < SAME; ++i) {
      m[i] = S.part_ml[0][i * kEach + at];
      l[i] = S.part_ml[1][i * kEach + at];
      top = fmaxf(top, m[i]);
      if constexpr (TS) to = fmaxf(to, S.part_ml[2][i * kEach + at]);
    }
    row.l = 0.0f;
#pragma unroll
    for (int i = 0; i < SAME; ++i) row.l = fmaf(l[i], exp2_ftz(m[i] - (top == -INFINITY ? 0.0f : top)), row.l);
    row.m = top;
    row.to = to;
    if (!TS) to = top;
    if (bad_page(w)) row.l = NAN;
    const float own = exp2_ftz(mine - (to == -INFINITY ? 0.0f : to));
    const bool whole = is_whole(w), live = r < M;
    const float2 f = factors(w, row);
    const long long head = head_of(w, row, r);
    float* slot = slot_of(w);
    if (copy == 0 && live) {
      if (whole) put_lse(head, row);
      else put_slot(slot, at, row);
    }
#pragma unroll 1
    for (int c = 0; c < 4; ++c) {
      uint32_t x[32];
      __syncwarp();  // (the lanes without a row are back)
      tmem_ld(o_at + 32 * c, x);
      tmem_wait_ld(x);
#pragma unroll
      for (int e = 0; e < 32; ++e) S.part[thread][e] = __uint_as_float(x[e]) * own;
      sync();
      float y[kShare];
#pragma unroll
      for (int d = 0; d < kShare; ++d) y[d] = S.part[at][copy * kShare + d];
#pragma unroll
      for (int i = 1; i < SAME; ++i)
#pragma unroll
        for (int d = 0; d < kShare; ++d) y[d] += S.part[i * kEach + at][copy * kShare + d];
      sync();  // the buffer is free again
      if (!live) continue;
      if (whole) {
        put_out<kShare>(row, head, 32 * c + copy * kShare, y, f);
      } else {
#pragma unroll
        for (int d = 0; d < kShare; d += 4)
          *reinterpret_cast<float4*>(slot + (size_t((32 * c + copy * kShare + d) / 4) * F::kRows + at) * 4) =
              make_float4(y[d], y[d + 1], y[d + 2], y[d + 3]);
      }
    }
  }
};

// ---------------------------------------------------------------- producers

// What a group of producer warps goes through: every kGroups-th tile of the range.
template <class F>
struct Tiles {
  const TreeArgs& a;
  Smem<F>& S;
  const long long s0, e0;
  Walk<F::kRows> w;
  const int group, thread, warp, lane;
  uint32_t units = 0;
  int k;
  bool more = true;
  int page;       // of the pool, of the lane's token (32 warp + lane) of the tile (looked up a tile ahead)
  long long off;  // of that token's row in the pools, or -1
  int drafts;     // the first drafted token of the tile

  __device__ __forceinline__ Tiles(const TreeArgs& args, Smem<F>& s, const Walk<F::kRows>& walk, long long from, long long to)
      : a(args), S(s), s0(from), e0(to), w(walk), group((int(threadIdx.x) - F::kSoftmaxWarps * 32) / F::kProducers),
        thread((int(threadIdx.x) - F::kSoftmaxWarps * 32) % F::kProducers), warp(thread >> 5), lane(thread & 31),
        k(walk.begin) {
    if (F::kGroups > 1 && group == 1) step();
    if (!more) return;
    page = page_of(k);
    place();
  }
  __device__ __forceinline__ void step() {
    if (!more || ++k < w.end) return;
    ++units;
    more = w.next(a, s0, e0);
    if (more) k = w.begin;
  }
  __device__ __forceinline__ int page_of(int tile) const {
    const int t = tile * kTile + 32 * warp + lane;
    return t < w.tokens ? a.table[(long long)w.b * a.max_pages + a.c.ps.div(t)] : -2;  // -2: no token
  }
  __device__ __forceinline__ void place() {
    const int t = k * kTile + 32 * warp + lane;
    off = -1;
    if (page >= 0 && page < a.c.n_pages) {
      const int at = t - a.c.ps.div(t) * int(a.c.ps.d);
      off = (long long)page * a.c.page_stride + (long long)at * a.c.token_stride + (long long)w.h * a.c.head_stride;
    } else if (page != -2 || t < w.tokens) {
      flag(a.c, KVQ_PAGED_ERR_PAGE);
      S.bad_page[w.number & 15] = 1;
    }
    if (k + F::kGroups < w.end) page = page_of(k + F::kGroups);
    drafts = max(0, min(kTile, w.r.P - k * kTile));
  }
  // On to the group's next tile.
  __device__ __forceinline__ void next() {
    const uint32_t before = units;
#pragma unroll 1
    for (int i = 0; i < F::kGroups; ++i) step();
    if (!more) return;
    if (before != units) page = page_of(k);
    place();
  }
  // One row tile: the unit's queries to tensor memory, a row by a thread of the group that has its first tile. N words
  // of the row from `at` on.
  template <int N>
  __device__ __forceinline__ void load_queries(uint32_t (&q)[N], int at) const {
    const int M = w.r.n * a.g, r = w.rb * F::kRows + thread % (kTile / copies(M));
    const bool live = r < M;
    const int i = r / a.g;
    const char* from =
        a.q + (live ? (w.r.row0 + i) * a.q_stride + (long long)(w.h * a.g + (r - i * a.g)) * (kD * 2) + 4 * at : 0);
#pragma unroll
    for (int e = 0; e < N; e += 4) {
      uint4 y = make_uint4(0u, 0u, 0u, 0u);
      if (live) y = *reinterpret_cast<const uint4*>(from + 4 * e);
      q[e] = y.x;
      q[e + 1] = y.y;
      q[e + 2] = y.z;
      q[e + 3] = y.w;
    }
  }
  // The buffer's last queries are those of the unit before the last one, multiplied once all its keys are there.
  __device__ __forceinline__ bool wait_queries() const {
    return warp_wait(&S.q_free[units & 1u], ((units >> 1) + 1) & 1u, &S.abort);
  }
  __device__ __forceinline__ uint32_t queries_at() const {
    return S.tmem + (uint32_t(warp) << 21) + kColQ + 64u * (units & 1u);
  }
  __device__ __forceinline__ void queries_stored() const {
    tmem_wait_st();
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(&S.q_full[units & 1u]);
  }
};

// 16-bit rows: asynchronous copies, which arrive by themselves.
template <class F, bool QUERIES>
__device__ __forceinline__ void produce(Tiles<F>& T) {
  const TreeArgs& a = T.a;
  Smem<F>& S = T.S;
  const uint32_t slots = smem_addr(S.slot);
  uint32_t x = 0;  // copies so far: K and V of a tile, then of the next one
  [[maybe_unused]] uint32_t q[2][32];
#pragma unroll 1
  while (T.more) {
    if constexpr (QUERIES)
      if (T.k == T.w.begin) {
        T.load_queries(q[0], 0);
        T.load_queries(q[1], 32);
      }  // (on their way while the tile's copies are issued)
#pragma unroll 1
    for (int half = 0; half < 2; ++half, ++x) {
      const char* pool = half == 0 ? a.c.k : a.c.v;
      const uint32_t slot = x % F::kSlots, to = slots + slot * kSlotBytes;
      if (!warp_wait(&S.empty[slot], (x / F::kSlots + 1) & 1u, &S.abort)) return;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const long long y = __shfl_sync(0xFFFFFFFFu, T.off, 4 * e + (T.lane >> 3));
#pragma unroll
        for (int f = 0; f < 2; ++f) {
          const int chunk = 8 * f + (T.lane & 7);
          copy16(to + chunk_at(32 * T.warp + 4 * e + (T.lane >> 3), chunk), pool + (y < 0 ? 0 : y) + chunk * 16, y >= 0);
        }
      }
      arrive_landed(half == 0 || T.drafts == kTile ? &S.full[slot] : &S.raw_full[slot]);
    }
    if constexpr (QUERIES)
      if (T.k == T.w.begin) {
        if (!T.wait_queries()) return;
        tc_fence_after();
        tmem_st(T.queries_at(), q[0]);
        tmem_st(T.queries_at() + 32, q[1]);
        T.queries_stored();
      }
    T.next();
  }
}

// A lane's share of an 8-bit copy's i-th part: 16 channels of one of eight tokens, the first or the second half of the
// row's, so that eight lanes write to all banks (a whole row by eight lanes: each bank twice).
__device__ __forceinline__ int part_token(int lane, int i) { return 8 * (i >> 1) + (lane >> 2); }
__device__ __forceinline__ int part_chunk(int lane, int i) { return 4 * (i & 1) + (lane & 3); }

// N parts from the i-th on as chunks of an operand.
template <bool BF, int N>
__device__ __forceinline__ void convert(const uint4 (&z)[N], uint32_t to, int token, int lane, int i) {
#pragma unroll
  for (int e = 0; e < N; ++e) {
    uint2 v[4];
#pragma unroll
    for (int d = 0; d < 4; ++d) v[d] = widen<BF>((&z[e].x)[d]);
    const int t = token + part_token(lane, i + e), c = 2 * part_chunk(lane, i + e);
    sts16(to + chunk_at(t, c), make_uint4(v[0].x, v[0].y, v[1].x, v[1].y));
    sts16(to + chunk_at(t, c + 1), make_uint4(v[2].x, v[2].y, v[3].x, v[3].y));
  }
}

// 8-bit rows: asynchronous copies into a ring of their own, each thread's to be converted by itself. (Loaded into
// registers they left room for two slots more, but the fence behind a conversion then waited for the next loads: 64
// requests of one token with scales per token 308 us.)
template <class F, bool QUERIES, int PARTS>
__device__ __forceinline__ void produce_narrow(Tiles<F>& T) {
  const TreeArgs& a = T.a;
  Smem<F>& S = T.S;
  constexpr int kLag = F::kStages - 1;  // copies between a copy and its conversion
  const uint32_t slots = smem_addr(S.slot), raws = smem_addr(S.raw) + T.group * (F::kStages * kRawBytes) + T.thread * 16;
  uint32_t mine = 0;  // the group's copies so far: K and V of a tile, then of its next one
  // Copies not converted yet, the newest one in the lowest bits: for each the first of the tile's tokens whose value may
  // be replaced (kTile: none, as for all keys).
  uint32_t past = 0;
  int pending = 0;
  // The oldest copy has landed and becomes an operand.
  auto land = [&]() -> bool {
    const uint32_t y = mine - pending, x = F::kGroups > 1 ? 4 * (y >> 1) + 2 * T.group + (y & 1u) : y;  // (x: of all)
    const uint32_t slot = x % F::kSlots, to = slots + slot * kSlotBytes, raw = raws + (y % F::kStages) * kRawBytes;
    const int from = int(past >> (8 * (pending - 1))) & 0xFF;
    if (!warp_wait(&S.empty[slot], (x / F::kSlots + 1) & 1u, &S.abort)) return false;
#pragma unroll 1
    for (int i = 0; i < 8; i += PARTS) {
      uint4 z[PARTS];
#pragma unroll
      for (int e = 0; e < PARTS; ++e) z[e] = lds16(raw + (i + e) * (F::kProducers * 16));
      if (from < kTile) {  // drafted values: NaN becomes 0
        uint32_t any = 0u;
#pragma unroll
        for (int e = 0; e < PARTS; ++e) {
          if (32 * T.warp + part_token(T.lane, i + e) < from) continue;
#pragma unroll
          for (int d = 0; d < 4; ++d) {
            uint32_t& v = (&z[e].x)[d];
            const uint32_t nan = ((v & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;  // bytes of 0x7F or 0xFF
            v &= ~((nan >> 7) * 255u);
            any |= nan;
          }
        }
        if (any != 0u) S.loose = 1;
      }
      if (F::kKeyBf && (y & 1u) == 0u) convert<true>(z, to, 32 * T.warp, T.lane, i);
      else convert<false>(z, to, 32 * T.warp, T.lane, i);
    }
    fence_async_smem();
    __syncwarp();
    if (T.lane == 0) mbar_arrive(&S.full[slot]);
    --pending;
    return true;
  };
#pragma unroll 1
  for (;;) {
#pragma unroll 1
    for (int half = 0; half < 2; ++half) {
      if (T.more) {
        const char* pool = half == 0 ? a.c.k : a.c.v;
        const uint32_t to = raws + (mine % F::kStages) * kRawBytes;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const long long y = __shfl_sync(0xFFFFFFFFu, T.off, part_token(T.lane, e));
          copy16(to + e * (F::kProducers * 16), pool + (y < 0 ? 0 : y) + part_chunk(T.lane, e) * 16, y >= 0);
        }
        commit();
        past = past << 8 | uint32_t(half == 0 ? kTile : T.drafts);
        ++mine;
        ++pending;
      }
#pragma unroll 1
      while (pending > (T.more ? kLag : 0)) {
        if (T.more) wait_groups<kLag>();
        else wait_groups<0>();
        if (!land()) return;
      }
    }
    if (!T.more) break;
    if constexpr (QUERIES)
      if (T.k == T.w.begin) {
        if (!T.wait_queries()) return;  // (of the copies before it the group has none left)
        tc_fence_after();
#pragma unroll 1
        for (int i = 0; i < 4; ++i) {  // (not loaded ahead: beside the conversion there are no registers)
          uint32_t q[16];
          T.load_queries(q, 16 * i);
          tmem_st16(T.queries_at() + 16 * i, q);
        }
        T.queries_stored();
      }
    T.next();
  }
}

// Two warps: the scales of the tiles' tokens (8-bit rows with a scale per token), two tokens a lane, looked up in two
// steps one and two tiles ahead.
template <class F>
__device__ __forceinline__ void load_scales(const TreeArgs& a, Smem<F>& S, Walk<F::kRows> w, long long s0, long long e0) {
  const int lane = threadIdx.x & 31, part = int(threadIdx.x >> 5) - F::kMmaWarp - 1, first = 64 * part + 2 * lane;
  const float sc = a.scale * kLog2e;
  struct Tile {
    int t0, P, h;
    bool there;
  };
  int k = w.begin;
  bool more = true;
  int page[2];  // of the pool, -1: no token
  float ks[2], vs[2];
  auto look_up = [&]() -> Tile {
    if (!more) return Tile{0, 0, 0, false};
    const Tile t{k * kTile + first, w.r.P, w.h, true};
#pragma unroll
    for (int i = 0; i < 2; ++i)
      page[i] = t.t0 + i < w.tokens ? a.table[(long long)w.b * a.max_pages + a.c.ps.div(t.t0 + i)] : -1;
    if (++k == w.end) {
      more = w.next(a, s0, e0);
      if (more) k = w.begin;
    }
    return t;
  };
  auto fetch = [&](const Tile& t) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      ks[i] = vs[i] = 0.0f;
      if (!t.there || page[i] < 0 || page[i] >= a.c.n_pages) continue;
      const int at = t.t0 + i;
      const long long x = ((long long)page[i] * a.c.H + t.h) * int(a.c.ps.d) + (at - a.c.ps.div(at) * int(a.c.ps.d));
      ks[i] = a.c.k_scale[x];
      vs[i] = a.c.v_scale[x];
    }
  };
  Tile now{0, 0, 0, false}, next{0, 0, 0, false};
  uint32_t c = 0;
#pragma unroll 1
  for (int turn = 0;; ++turn) {  // (the first two turns only look ahead)
    if (turn >= 2) {
      if (!now.there) return;
      const uint32_t at = c % kScaleRing;
      if (!warp_wait(&S.scales_free[at], (c / kScaleRing + 1) & 1u, &S.abort)) return;
      float2 f, l, v;
      float low = INFINITY, high = -INFINITY;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float x = vs[i];
        if (now.t0 + i >= now.P && !isfinite(x)) {  // a drafted token's: as its values that are not finite
          S.loose = 1;
          x = 0.0f;
        }
        const float y = __log2f(x);  // (decides what the sums are to, not what they are)
        (&f.x)[i] = scaled(sc, ks[i]);
        (&l.x)[i] = y;
        (&v.x)[i] = x;
        // a scale of 0 (no token) does not count; one that is not finite makes the range so
        low = fminf(low, x == 0.0f ? INFINITY : y);
        high = fmaxf(high, y != y ? INFINITY : y);
      }
      *reinterpret_cast<float2*>(&S.scales[at][0][first]) = f;
      *reinterpret_cast<float2*>(&S.scales[at][1][first]) = l;
      *reinterpret_cast<float2*>(&S.scales[at][2][first]) = v;
      low = in_order(__reduce_min_sync(0xFFFFFFFFu, in_order(low)));
      high = in_order(__reduce_max_sync(0xFFFFFFFFu, in_order(high)));
      if (lane == 0) S.range[at][part] = make_float2(low, high);
      __syncwarp();
      if (lane == 0) mbar_arrive(&S.scales_full[at]);
      ++c;
    }
    now = next;
    fetch(now);
    next = look_up();
  }
}

// Two warps: drafted values of 16-bit rows that are not finite become 0 before they are multiplied.
template <int DT, int QT, int TILES, bool TS>
__device__ __forceinline__ void screen_values(const TreeArgs& a, Smem<Form<DT, QT, TILES, TS>>& S,
                                             Walk<Form<DT, QT, TILES, TS>::kRows> w, long long s0, long long e0) {
  using F = Form<DT, QT, TILES, TS>;
  const int thread = int(threadIdx.x) - (F::kMmaWarp + 1) * 32;
  constexpr uint32_t kInf = DT == kBf16 ? 0x7F80u : 0x7C00u;
  uint32_t x = 0, phases = 0;  // copies so far; the parity of each slot's next check
  for (bool more = true; more; more = w.next(a, s0, e0)) {
    const int k0 = max(w.begin, min(w.end, w.r.P / kTile));  // the first tile with drafted tokens
    for (int k = k0; k < w.end; ++k) {
      const uint32_t slot = (x + 2 * (k - w.begin) + 1) % F::kSlots, at = smem_addr(S.slot) + slot * kSlotBytes;
      const int from = max(0, min(kTile, w.r.P - k * kTile)), to = min(kTile, w.tokens - k * kTile);
      if (!warp_wait(&S.raw_full[slot], (phases >> slot) & 1u, &S.abort)) return;
      phases ^= 1u << slot;
      // a token's 16 chunks by 16 threads: two of each 128 bytes, in their swizzled order
#pragma unroll 4
      for (int token = from + thread / 8; token < to; token += F::kScreeners / 8) {
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const uint32_t p = at + half * (kSlotBytes / 2) + token * 128 + (thread & 7) * 16;
          uint4 z = lds16(p);
          bool any = false;
#pragma unroll
          for (int d = 0; d < 4; ++d) {
            uint32_t& v = (&z.x)[d];
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
            sts16(p, z);
            S.loose = 1;
          }
        }
      }
      fence_async_smem();
      asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0], %1;" ::"r"(smem_addr(&S.full[slot])),
                   "r"(F::kProducers / F::kScreeners)
                   : "memory");
    }
    x += 2 * (w.end - w.begin);
  }
}

// ---------------------------------------------------------------- products

template <int DT, int QT, int TILES, bool TS>
__device__ __forceinline__ bool multiply(const TreeArgs& a, Smem<Form<DT, QT, TILES, TS>>& S,
                                         Walk<Form<DT, QT, TILES, TS>::kRows> w, long long s0, long long e0) {
  using F = Form<DT, QT, TILES, TS>;
  auto same = [](uint32_t x) { return __shfl_sync(0xFFFFFFFFu, x, 0); };
  const uint32_t tmem = same(S.tmem), q = smem_addr(S.q), slots = smem_addr(S.slot);
  uint32_t x = 0;             // slots so far
  uint32_t count[2] = {0, 0};  // products of each row tile so far
  uint32_t units = 0;
  auto keys = [&](int tile, uint32_t x, uint32_t buf) {
    const uint32_t slot = same(x % F::kSlots), to = same(tmem + kColS + 128u * buf);
    [[maybe_unused]] const uint32_t qa = same(tmem + kColQ + 64u * (units & 1u));
    const uint64_t kb = smem_desc(slots + slot * kSlotBytes, 16);
    if (!elect()) return;
#pragma unroll
    for (uint32_t k = 0; k < 8; ++k) {  // 16 channels: 32 bytes on, four times in each half
      const uint32_t on = 2u * (k & 3u) + (kSlotBytes / 32) * (k >> 2);
      if constexpr (TILES == 1)
        mma_ts(to, qa + 8u * k, kb + on, instr_desc(F::kKeyBf, false),
               k > 0);
      else
        mma_ss(to, smem_desc(q + tile * kSlotBytes, 16) + on, kb + on,
               instr_desc(F::kKeyBf, false), k > 0);
    }
    mma_commit(&S.s_full[buf]);
  };
  auto values = [&](int tile, uint32_t x, uint32_t buf, bool first) {
    const uint32_t slot = same(x % F::kSlots), from = same(tmem + kColS + 128u * buf);
    const uint64_t vb = smem_desc(slots + slot * kSlotBytes, kSlotBytes / 2);
    if (!elect()) return;
#pragma unroll
    for (uint32_t k = 0; k < 8; ++k)  // 16 tokens: 2048 bytes on
      mma_ts(tmem + 128u * tile, from + 8u * k, vb + 128u * k, instr_desc(F::kValBf, true),
             !first || k > 0);
    mma_commit(&S.pv_done[TILES == 1 ? buf : tile]);
  };
  auto wait = [&](unsigned long long* bar, uint32_t phase) {
    if (!warp_wait(bar, phase & 1u, &S.abort)) return false;
    tc_fence_after();
    return true;
  };
  auto filled = [&](uint32_t x) {
    if (!warp_wait(&S.full[x % F::kSlots], (x / F::kSlots) & 1u, &S.abort)) return false;
    if constexpr (!F::kNarrow) fence_async_smem();  // (copies that arrive by themselves have no fence behind them)
    tc_fence_after();
    return true;
  };
  auto done = [&](unsigned long long* bar) {
    if (elect()) mma_commit(bar);
  };
  for (bool more = true; more; more = w.next(a, s0, e0), ++units) {
    const int n = w.end - w.begin;
    if constexpr (TILES == 1) {
      if (!wait(&S.q_full[units & 1u], units >> 1)) return false;
      // scores of tile k + 1 are under way while the softmax warps work on tile k's
      for (int k = 0; k <= n; ++k) {
        if (k < n) {
          if (!filled(x + 2 * k)) return false;
          keys(0, x + 2 * k, (count[0] + k) & 1u);
          done(&S.empty[(x + 2 * k) % F::kSlots]);
          if (k + 1 == n) done(&S.q_free[units & 1u]);
        }
        if (k > 0) {
          const uint32_t c = count[0] + k - 1, y = x + 2 * (k - 1) + 1;
          if (!filled(y) || !wait(&S.p_ready[c & 1u], c >> 1)) return false;
          if (k == 1 && units > 0 && !wait(&S.o_free, units - 1)) return false;  // the unit's sums before are read
          values(0, y, c & 1u, k == 1);
          done(&S.empty[y % F::kSlots]);
        }
      }
      count[0] += n;
    } else {
      if (!wait(&S.q_full[0], units)) return false;
      const bool both = w.rb * F::kRows + kTile < w.r.n * a.g;  // the second row tile has rows
      for (int k = 0; k <= n; ++k)
        for (int tile = 0; tile < 2; ++tile) {  // a row tile's products while the other's softmax runs
          const bool on = tile == 0 || both, last = tile == 1;
          if (k > 0) {
            const uint32_t y = x + 2 * (k - 1) + 1;
            if (on) {
              if (!filled(y) || !wait(&S.p_ready[tile], count[tile])) return false;
              values(tile, y, tile, k == 1);
              ++count[tile];
            }
            if (last) done(&S.empty[y % F::kSlots]);
          }
          if (k < n) {
            if (on) {
              if (!filled(x + 2 * k)) return false;
              keys(tile, x + 2 * k, tile);
            }
            if (last) done(&S.empty[(x + 2 * k) % F::kSlots]);
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
    reinterpret_cast<int*>(a.ws + loose_offset(gridDim.x))[blockIdx.x] = 0;
    for (int i = 0; i < F::kSlots; ++i) {
      mbar_init(&S.full[i], F::kNarrow ? 4 : F::kProducers);
      mbar_init(&S.raw_full[i], F::kProducers);
      mbar_init(&S.empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&S.s_full[i], 1);
      mbar_init(&S.p_ready[i], 4);
      mbar_init(&S.pv_done[i], 1);
      mbar_init(&S.q_full[i], TILES == 1 ? 4 : F::kSoftmaxWarps);
      mbar_init(&S.q_free[i], 1);
    }
    for (int i = 0; i < kScaleRing; ++i) {
      mbar_init(&S.scales_full[i], 2);
      mbar_init(&S.scales_free[i], F::kSoftmaxWarps);
    }
    mbar_init(&S.o_free, 4);
    mbar_init(&S.drain, 1);
    for (int i = 0; i < 16; ++i) S.bad_page[i] = 0;
    S.loose = 0;
    S.abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  // requests that are refused: no block's range holds them
#pragma unroll 1
  for (int b = blockIdx.x; b < a.B; b += gridDim.x) {
    Request r;
    r.load(a, b);
    if (!r.refused) continue;
    if (threadIdx.x == 0) flag(a.c, KVQ_PAGED_ERR_LENGTH);
    const int n = row_range(a.offsets, a.n_rows, b, r.row0);
    const uint32_t nan = QT == kBf16 ? 0x7FC07FC0u : 0x7E007E00u;
#pragma unroll 1
    for (long long i = threadIdx.x; i < (long long)max(n, 0) * a.Hq * (kD / 2); i += F::kThreads)
      reinterpret_cast<uint32_t*>(a.out)[(long long)r.row0 * a.Hq * (kD / 2) + i] = nan;
    if (a.lse != nullptr)
#pragma unroll 1
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
    Tiles<F> T(a, S, w, s0, e0);
    // of a copy's eight parts those that a thread converts at once: two where the code for BF16 keys and for FP16 values
    // stands beside that for scales per token, else four (the code's size: 64 requests of one token with BF16 queries and
    // scales per token 233 us by four, 177 by two; with FP16 queries 173 and 178; with a scale per head 161 and 166)
    if constexpr (F::kNarrow) produce_narrow<F, TILES == 1, TS && F::kKeyBf ? 2 : 4>(T);
    else produce<F, TILES == 1>(T);
    wait_copies();  // (where a wait has run out some may be under way)
  } else {
    fewer_registers<F::kMmaRegs>();
    if (warp == F::kMmaWarp) {
      multiply<DT, QT, TILES, TS>(a, S, w, s0, e0);
      // the products in flight end before the tensor memory is freed
      if (elect()) mma_commit(&S.drain);
      int never = 0;
      mbar_wait(&S.drain, 0, &never);
    }
    if constexpr (TS)
      if (warp == F::kMmaWarp + 1 || warp == F::kMmaWarp + 2) load_scales<F>(a, S, w, s0, e0);
    if constexpr (F::kScreeners > 0)
      if (warp > F::kMmaWarp && warp <= F::kMmaWarp + F::kScreeners / 32) screen_values<DT, QT, TILES, TS>(a, S, w, s0, e0);
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (threadIdx.x == 0) {
    if (S.abort) flag(a.c, KVQ_PAGED_ERR_WAIT);
    if (S.loose) reinterpret_cast<int*>(a.ws + loose_offset(gridDim.x))[blockIdx.x] = 1;
  }
  if (warp == F::kMmaWarp) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(S.tmem), "n"(kTmemCols) : "memory");
  }
}

// Joins the parts of a unit that several blocks' ranges share: block (c, y) those of the unit that begins in block c's
// range, its rows 32 y .. 32 y + 31, a lane a row, a warp 16 channels of it (and every other part). Where some drafted
// value was replaced by 0 (loose), the blocks add what is not finite to the rows that see it: to those of shared units
// here, to the others behind them.
constexpr int kJoinWarps = 16;

// `top` becomes the larger of top and part; what is to them is to it times f and g.
__device__ __forceinline__ void share(float& top, float part, float& f, float& g) {
  const float to = fmaxf(top, part), base = to == -INFINITY ? 0.0f : to;
  f = exp2f(top - base);
  g = exp2f(part - base);
  top = to;
}
__device__ __forceinline__ void join(float& m, float& l, float pm, float pl) {
  float f, g;
  share(m, pm, f, g);
  l = l * f + pl * g;
}

// Sum of the values that are not finite in channels c .. c + 3 of the drafted tokens that row i sees (0: none).
template <int DT>
__device__ __noinline__ float4 loose(const TreeArgs& a, const Request& r, int b, int h, int i, int c) {
  const uint32_t* mask = a.mask != nullptr ? a.mask + (long long)(r.row0 + i) * a.mask_words : nullptr;
  float4 sum = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  for (int j = 0; j < r.n; ++j) {
    if (!((seen_word(mask, a.mask_words, r.n, i, j >> 5) >> (j & 31)) & 1)) continue;
    const int t = r.P + j, e = a.c.ps.div(t), page = a.table[(long long)b * a.max_pages + e];
    const int place = t - e * int(a.c.ps.d);
    if (page < 0 || page >= a.c.n_pages) continue;
    float4 x = load4<DT>(a.c.v + (long long)page * a.c.page_stride + (long long)place * a.c.token_stride +
                         (long long)h * a.c.head_stride + c * elem_bytes<DT>());
    if (DT == kE4m3 && a.c.v_scale != nullptr)
      x = times(x, a.c.v_scale[a.c.token_scales ? ((long long)page * a.c.H + h) * int(a.c.ps.d) + place : h]);
#pragma unroll
    for (int d = 0; d < 4; ++d)
      if (!isfinite((&x.x)[d])) (&sum.x)[d] += (&x.x)[d];
  }
  return sum;
}

template <int DT, int QT, int TILES>
__global__ void __launch_bounds__(kJoinWarps * 32) join_kernel(const __grid_constant__ TreeArgs a) {
  constexpr int R = kTile * TILES;
  __shared__ float s_ml[3][32];
  __shared__ float4 s_x[8][4][32];
  wait_prior_grid();
  allow_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, group = warp & 7, odd = warp >> 3, n = gridDim.x;
  const Rec* recs = reinterpret_cast<const Rec*>(a.ws);
  const Rec rec = recs[blockIdx.x];
  int some = 0;
  for (int i = threadIdx.x; i < n; i += kJoinWarps * 32) some |= reinterpret_cast<const int*>(a.ws + loose_offset(n))[i];
  // (the bounds hold for every record of the attention kernel; a workspace that something else writes meanwhile must
  // not lead outside of it)
  auto shared = [&](const Rec& x, int c) {
    return x.parts >= 2 && x.parts <= n - c && x.b >= 0 && x.b < a.B && x.h >= 0 && x.h < a.c.H && x.rb >= 0;
  };
  const bool mine = shared(rec, blockIdx.x);
  Request r;
  r.load(a, mine ? rec.b : 0);
  const int row = 32 * blockIdx.y + lane, at = rec.rb * R + row, parts = mine && at - lane < r.n * a.g ? rec.parts : 0;
  const float* slots = reinterpret_cast<const float*>(a.ws + slots_offset(n));
  float m = -INFINITY, l = 0.0f, to = -INFINITY;  // (to: what the sums are to)
  float4 x[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) x[e] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  for (int i = odd; i < parts; i += 2) {
    const float* p = slots + size_t(i == 0 ? 2 * blockIdx.x + 1 : 2 * (blockIdx.x + i)) * slot_floats(R);
    const float pm = p[size_t(R) * kD + row], pl = p[size_t(R) * (kD + 1) + row], pn = p[size_t(R) * (kD + 2) + row];
    float4 y[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) y[e] = *reinterpret_cast<const float4*>(p + (size_t(4 * group + e) * R + row) * 4);
    join(m, l, pm, pl);
    float f, g;
    share(to, pn, f, g);
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
      s_ml[2][lane] = to;
    }
  }
  some = __syncthreads_or(some);
  if (!odd && parts > 0 && at < r.n * a.g) {
    join(m, l, s_ml[0][lane], s_ml[1][lane]);
    float f, g;
    share(to, s_ml[2][lane], f, g);
    const int i = at / a.g;
    const long long head = (long long)(r.row0 + i) * a.Hq + rec.h * a.g + (at - i * a.g);
    float inv = l == 0.0f ? 0.0f : 1.0f / l, inv2 = 1.0f;
    if (DT == kE4m3 && a.c.token_scales) between(to - m, inv, inv2);
    else if (DT == kE4m3 && a.c.v_scale != nullptr) inv2 = a.c.v_scale[rec.h];
    uint4* out = reinterpret_cast<uint4*>(a.out + head * (kD * 2) + group * 32);
    uint32_t y[8];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float4 z = s_x[group][e][lane];
      float4 v = make_float4(fmaf(g, z.x, x[e].x * f), fmaf(g, z.y, x[e].y * f), fmaf(g, z.z, x[e].z * f),
                             fmaf(g, z.w, x[e].w * f));
      v = l == 0.0f ? make_float4(0.0f, 0.0f, 0.0f, 0.0f) : times(times(v, inv), inv2);
      if (some) {
        const float4 u = loose<DT>(a, r, rec.b, rec.h, i, 16 * group + 4 * e);
        v = make_float4(v.x + u.x, v.y + u.y, v.z + u.z, v.w + u.w);
      }
      y[2 * e] = pack<QT == kBf16>(v.x, v.y);
      y[2 * e + 1] = pack<QT == kBf16>(v.z, v.w);
    }
    out[0] = make_uint4(y[0], y[1], y[2], y[3]);
    out[1] = make_uint4(y[4], y[5], y[6], y[7]);
    if (a.lse != nullptr && group == 0) a.lse[head] = (m + log2f(l)) * kLn2;
  }
  if (!some) return;
  // rows of units that are not shared: a warp a query head, a lane four channels
  const int warps = n * gridDim.y * kJoinWarps, me = (blockIdx.y * n + blockIdx.x) * kJoinWarps + warp;
  for (int b = 0; b < a.B; ++b) {
    r.load(a, b);
    for (long long u = me; u < (long long)r.n * a.Hq; u += warps) {
      const int i = int(u / a.Hq), hq = int(u - (long long)i * a.Hq), h = hq / a.g, rb = (i * a.g + hq - h * a.g) / R;
      bool joined = false;
      for (int c = lane; c < n; c += 32) joined |= shared(recs[c], c) && recs[c].b == b && recs[c].h == h && recs[c].rb == rb;
      if (__any_sync(0xFFFFFFFFu, joined)) continue;
      const float4 y = loose<DT>(a, r, b, h, i, 4 * lane);
      if (y.x == 0.0f && y.y == 0.0f && y.z == 0.0f && y.w == 0.0f) continue;
      char* p = a.out + ((long long)(r.row0 + i) * a.Hq + hq) * (kD * 2) + 8 * lane;
      const float4 x = load4<QT>(p);
      store4<QT>(p, make_float4(x.x + y.x, x.y + y.y, x.z + y.z, x.w + y.w));
    }
  }
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

// Two row tiles per block where the requests' mean rows fill more than one. (By the mean, since the host does not see
// the offsets: a chunk of 1000 rows over 8192 tokens among 63 single rows, which then goes by one, took 319 us, the chunk
// alone 143 by two and the single rows 170 by one.)
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

size_t tree_workspace_up_to(int B, int H, int Hq, int n_rows, int sms) {
  return tree_workspace(min(B, 1), H, Hq, n_rows, sms);  // (the fewer the requests the wider are theirs)
}

cudaError_t launch_tree(const TreeArgs& a, cudaStream_t stream) {
  const bool bf = a.q_dtype == kBf16;
  if (a.dtype == kBf16) return launch_types<kBf16, kBf16>(a, stream);
  if (a.dtype == kFp16) return launch_types<kFp16, kFp16>(a, stream);
  return bf ? launch_types<kE4m3, kBf16>(a, stream) : launch_types<kE4m3, kFp16>(a, stream);
}

}  // namespace paged
}  // namespace kvq
