// Attention of query rows over a paged key-value cache (sm_103a).
//
// For a (row, kv head) item with G query heads and tiles of 128 tokens:
//   S   = K Q^T          one tcgen05.mma chain, M = 128 tokens, N = G heads (padded)
//   P   = 2^(c S - m)    c = softmax scale * log2 e
//   O^T += V^T P         one chain, M = head dim, N = heads
// with a running maximum m and sum l per head: one pass over the cache. The
// tokens are the M side, so any G from 1 to 128 fills the tensor core's rows,
// one thread owns one token in the softmax (its mask and, for an E4M3 cache,
// its scales are per-thread constants), and K and V tiles are read by the MMA
// in the layout the cache has: K as a K-major and V as an M-major operand,
// both 128-byte rows per token. m is raised only when a score exceeds it by
// kTau (in log2), which keeps the rescale of O out of the common path; P stays
// below 2^kTau, and sums in fp32 do not mind.
//
// Rounding. Queries, keys and values go to the tensor core as the cache and the
// caller hold them: bf16, and E4M3 codes widened to bf16, which is exact. S, m,
// l and O are fp32. P goes to the tensor core in two bf16 numbers, hi + lo (16
// bits), as one operand of 2 N columns with an accumulator for each half, so V
// is read once for both. One bf16 alone moved results by up to 2^-9 of the
// weights and measured 870 against 893 us on the selected chunk of its day: the
// second number costs little. Over an E4M3 cache the token's key scale
// multiplies its scores, and its value scale multiplies P after l has taken it:
// m follows the scores alone, and a bf16 has the exponents of fp32, so neither
// a token of zeros nor one of large values costs the others' weights any bits.
// (kind::f8f6f4 reads the codes as they are, but wants P and Q in 8 bits too.
// Two E4M3 numbers for each lost what was below 2^-18 of the largest weight
// times scale: a token of zero values, whose scale is 1, beside values of 1
// then took 10 to 60 % of the result. It measured 97 against 127 us on 64 rows
// of 4096 to 32768 tokens, and 60 against 70 us on 256 rows of 2048 selected.)
//
// Split. The tiles of all items form one list, cut into equal ranges, one per
// CTA and SM, whatever the rows' lengths are. A range that starts or ends
// inside an item leaves an unnormalised partial (O, m, l) in the workspace, and
// combine_kernel joins the partials of an item in the order of the list, so
// results do not depend on timing. Joining them in the attention kernel, by
// the last CTAs to arrive, measured 31.4 against 26.5 us on 64 rows of 2048
// selected tokens: the code it adds costs more than the second launch.
//
// Roles: warps 0-3 copy K, V and Q tiles (cp.async), warp 4 cuts the work into
// segments, warps 5 and 7 issue the MMAs, warp 6 looks up addresses, warps 8-15
// are two softmax groups of 128 threads, each with half of the heads. Over an
// E4M3 cache warps 0-3 copy and widen keys and warps 16-19 values. All roles
// run from one instruction cache: loops are kept short and cold parts rolled
// (unrolled copies of the role loops cost 893 against 648 us on the selected
// chunk; widening four pieces at a time instead of two 667 against 653 us on a
// batch of 8-bit contexts).
//
// Bounds (a plain copy reaches 6790 GB/s):
//  - contexts of 4096 to 32768, 64 rows, 8 heads on each of 8 kv heads, bf16:
//    703 to 709 us for 4.83 GB, 6.8 to 6.9 TB/s: DRAM.
//  - 4096 rows of 2048 selected tokens, 64 heads on one kv head, bf16: 588 us.
//    Each tile's 64 KB come from L2 in 256-byte rows: 7.3 TB/s, where a kernel
//    that only copies such rows into shared memory, by four warps, reaches 7.4.
//  - 64 rows of such contexts, E4M3, 64 heads on one kv head: 127 us for 314 MB,
//    2.5 TB/s; with 64 heads on 8 kv heads 676 us for 2.5 GB. A tile costs some
//    7500 warp instructions at half of the issue slots, and the widening alone
//    128 KB of shared-memory traffic; without any loading or widening the rest of
//    the first still took 116 us, of the second 500.
//  - 128 heads on one kv head, the same contexts: 158 us over a bf16 cache, 168
//    over an E4M3 one: the softmax, 64 heads a thread.
//  - small calls: start-up (launch, three dependent loads to the first key, a
//    tile's chain of copy, two products and softmax) and the join, 6 to 25 us.
#include "smq_attn.cuh"
#include "smq_kernels.cuh"
#include "smq_ptx.cuh"

#include <cuda_bf16.h>

#include <type_traits>

namespace smq {

namespace {

constexpr int kLoaders = 128;   // threads; over an E4M3 cache as many again, a group for keys and one for values
constexpr int kSoftmax = 256;
constexpr int kSegRing = 8;     // segments published ahead
constexpr float kUnset = -3.0e38f;           // the running maximum of a partial without tokens
constexpr int kSmemLimit = 232448 - 1024;  // less the static part

// A run of tiles of one (row, kv head) item.
struct AttnSeg {
  int32_t row, kvh;
  int32_t tile0, ntiles;  // ntiles = 0: the end of this CTA's work
  int32_t first, last;    // decode: positions [first, last); selected: entries [0, num_ids)
  int32_t slot;           // partial slot, -1: the whole item, write the result
  int32_t table_row;      // of the block table, -1: out of range
};
static_assert(sizeof(AttnSeg) == 32, "");

// A kernel's shapes. N is the group of query heads rounded up to 16, 32, 64 or 128. Shared memory holds kSlots tiles of
// K or V as the tensor core reads them (16 or 32 KB each), over an E4M3 cache kRaws tiles of codes of each side, Q, P and the
// rings; what is left over after those goes to the tiles in flight.
template <int D, bool kE4m3, int N>
struct Shape {
  static constexpr int kRow = 2 * D;                             // bytes per token, in bf16
  static constexpr int kBlocks = kRow > 128 ? 2 : 1;             // 128-byte columns
  static constexpr int kUnit = kBlocks * 128 * 128;              // bytes of a K or V tile
  static constexpr int kRaw = kE4m3 ? 128 * D : 0;               // bytes of its codes
  static constexpr int kQBytes = kBlocks * N * 128;
  static constexpr int kQBufs = N >= 64 ? 1 : 2;
  static constexpr int kPRow = N * 2 > 128 ? 128 : N * 2;        // bytes of a P row in a block
  static constexpr int kPPart = 128 * N * 2;
  static constexpr int kPBytes = 2 * kPPart;                     // hi and lo of P
  static constexpr int kCols = N / 2;                            // heads per softmax thread
  static constexpr int kThreads = kE4m3 ? 640 : 512;
  // registers of a thread: at launch all of an SM's, then most for the 256 softmax threads (of the widest group, which
  // hold twice the heads: 168 against 152 measured 173 and 230 us on 64 rows of 128 heads on one 8-bit kv head)
  static constexpr int kRegs = kE4m3 ? 96 : 128;
  static constexpr int kSoftmaxRegs = !kE4m3 ? 184 : N == 128 ? 168 : 152;
  static constexpr int kOtherRegs = !kE4m3 ? 72 : N == 128 ? 48 : 56;
  static_assert(kSoftmax * kSoftmaxRegs + (kThreads - kSoftmax) * kOtherRegs <= kThreads * kRegs, "");
  static constexpr int kAddrReaders = (kE4m3 ? 8 : 4) + 8;       // loader and softmax warps
  static constexpr int kSegReaders = kAddrReaders + 2 + 1;       // and MMA and address warps
  static constexpr int kRing = 8;                                // tiles whose addresses, masks and scales may be ahead of the softmax
  static constexpr int kRingBytes = kRing * 128 * (8 + (kE4m3 ? 8 : 0));
  static constexpr int kMisc = kRingBytes + kRing * 16 + kSegRing * 32 + 640 /*barriers*/ + N * 16 /*m, alpha, raise, 1 / l*/ +
                               8 * kCols * 4 /*scratch*/ + 64;
  static constexpr int kFixed = kQBufs * kQBytes + kPBytes + kMisc;
  static constexpr int kFree = kSmemLimit - kFixed;
  // over an E4M3 cache one or two units of each side, so that what is left over goes to the copies ahead
  static constexpr int kFit = kE4m3 ? (kFree >= 4 * kUnit + 4 * kRaw ? 4 : 2) : kFree / kUnit;
  static constexpr int kSlots = kFit > 12 ? 12 : kFit;
  static constexpr int kRawFit = kE4m3 ? (kFree - kSlots * kUnit) / (kE4m3 ? 2 * kRaw : 1) : 0;
  static constexpr int kRaws = kRawFit > 4 ? 4 : kRawFit;        // of each side
  static constexpr int kSmem = kSlots * kUnit + 2 * kRaws * kRaw + kFixed;
  static constexpr int kTmem = 4 * N;                            // O from hi and from lo, two buffers of S
  static_assert((kE4m3 ? kSlots % 2 == 0 && kRaws >= 1 : kSlots >= 3) && kSmem <= kSmemLimit, "");
  static_assert(kBlocks == 2 || kFixed >= 16384, "an M = 128 operand of a 64-wide head reads past its unit");
};
constexpr float kTau = 8.f;  // log2 of the largest P

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float lg2(float x) {
  float y;
  asm("lg2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Two fp32 operations at once: x = x * f + a, and x += y.
__device__ __forceinline__ void fma2(float& x0, float& x1, float f0, float f1, float a0, float a1) {
  asm("{\n .reg .b64 x, f, a;\n mov.b64 x, {%0, %1};\n mov.b64 f, {%2, %3};\n mov.b64 a, {%4, %5};\n"
      " fma.rn.f32x2 x, x, f, a;\n mov.b64 {%0, %1}, x;\n}"
      : "+f"(x0), "+f"(x1)
      : "f"(f0), "f"(f1), "f"(a0), "f"(a1));
}
__device__ __forceinline__ void mul2(float& x0, float& x1, float y0, float y1) {
  asm("{\n .reg .b64 x, y;\n mov.b64 x, {%0, %1};\n mov.b64 y, {%2, %3};\n mul.rn.f32x2 x, x, y;\n mov.b64 {%0, %1}, x;\n}"
      : "+f"(x0), "+f"(x1)
      : "f"(y0), "f"(y1));
}
__device__ __forceinline__ void add2(float& x0, float& x1, float y0, float y1) {
  asm("{\n .reg .b64 x, y;\n mov.b64 x, {%0, %1};\n mov.b64 y, {%2, %3};\n add.rn.f32x2 x, x, y;\n mov.b64 {%0, %1}, x;\n}"
      : "+f"(x0), "+f"(x1)
      : "f"(y0), "f"(y1));
}

// A warp waits for the phase of the given parity; false, for all of it, after limit_ns or once *abort is set. Some
// forty waits a tile share the issue slots with the softmax: each try is suspended by the hardware until the phase
// completes or a system limit passes, the vote keeps the loop's branches uniform, and the clock is read once in 16 tries.
__device__ __forceinline__ bool wait_phase(uint32_t bar, uint32_t parity, const volatile int* abort, uint64_t limit_ns) {
  uint64_t t0 = 0;
  for (uint32_t n = 1; !__all_sync(0xffffffffu, mbar_try_wait(bar, parity)); ++n) {
    if (n % 16 != 0) continue;
    const uint64_t now = global_ns();
    if (t0 == 0) t0 = now;
    if (__any_sync(0xffffffffu, *abort || now - t0 > limit_ns)) return false;
  }
  return true;
}

// One lane's arrival, without a branch.
__device__ __forceinline__ void arrive_one(uint32_t bar, int lane) {
  asm volatile("{\n .reg .pred p;\n setp.eq.s32 p, %1, 0;\n @p mbarrier.arrive.shared::cta.b64 _, [%0];\n}" ::"r"(bar),
               "r"(lane)
               : "memory");
}

// 16-byte asynchronous copies; of the second, `bytes` 0 fills with zeros and reads nothing.
__device__ __forceinline__ void cp16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp16(uint32_t dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int kLeft>
__device__ __forceinline__ void cp_wait() {  // all but the newest kLeft groups
  asm volatile("cp.async.wait_group %0;" ::"n"(kLeft) : "memory");
}
__device__ __forceinline__ void cp_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }
// 4-byte asynchronous copy.
__device__ __forceinline__ void cp4(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
// Arrive on an mbarrier, as one of its expected arrivals, once this thread's copies so far have landed.
__device__ __forceinline__ void cp_arrive(uint32_t bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}

__device__ __forceinline__ void bar_sync(int id, int threads) {
  asm volatile("barrier.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}
// Barrier of `threads` threads that returns whether any of them said `v`.
__device__ __forceinline__ bool bar_or(int id, int threads, bool v) {
  uint32_t r;
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.b32 p, %3, 0;\n barrier.red.or.pred q, %1, %2, p;\n selp.b32 %0, 1, 0, q;\n}"
      : "=r"(r)
      : "r"(id), "r"(threads), "r"(static_cast<uint32_t>(v))
      : "memory");
  return r != 0;
}

__device__ __forceinline__ void sts16(uint32_t a, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}

// kN consecutive columns of this thread's TMEM lane; valid after tmem_wait_ld, behind pin().
template <int kN>
__device__ __forceinline__ void tmem_ld(uint32_t taddr, float* v) {
  static_assert(kN == 8 || kN == 16 || kN == 32, "");
  if (kN == 8)
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7])
                 : "r"(taddr)
                 : "memory");
  if (kN == 16)
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
                 : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]), "=f"(v[8]), "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15])
                 : "r"(taddr)
                 : "memory");
  if (kN == 32)
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
                 : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]), "=f"(v[8]), "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15]), "=f"(v[16]), "=f"(v[17]), "=f"(v[18]), "=f"(v[19]), "=f"(v[20]), "=f"(v[21]), "=f"(v[22]), "=f"(v[23]), "=f"(v[24]), "=f"(v[25]), "=f"(v[26]), "=f"(v[27]), "=f"(v[28]), "=f"(v[29]), "=f"(v[30]), "=f"(v[31])
                 : "r"(taddr)
                 : "memory");
}
// Keeps uses of loaded registers behind the wait that makes them valid.
template <int kN>
__device__ __forceinline__ void pin(float* v) {
#pragma unroll
  for (int i = 0; i < kN; i += 8)
    asm volatile("" : "+f"(v[i]), "+f"(v[i + 1]), "+f"(v[i + 2]), "+f"(v[i + 3]), "+f"(v[i + 4]), "+f"(v[i + 5]), "+f"(v[i + 6]),
                 "+f"(v[i + 7]));
}
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const float* v) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "f"(v[0]),
               "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7])
               : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Shared-memory matrix descriptors, in two words. The high word: K-major with
// 128-byte rows, or M- / N-major where rows of `row` bytes hold consecutive M
// or N of one k; 8 rows are the stride. The low word: the address and, for
// M- / N-major, the distance to the next block of M or N.
__host__ __device__ constexpr uint32_t desc_hi(int row) {
  return ((8 * row) >> 4) | (1u << 14) | (static_cast<uint32_t>(row == 128 ? 2 : row == 64 ? 4 : 6) << 29);
}
__device__ __forceinline__ uint32_t desc_lo(uint32_t saddr, uint32_t lbo) { return (saddr >> 4) | ((lbo >> 4) << 16); }

__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.b32 %0, 1, 0, p;\n}" : "=r"(r));
  return r != 0;
}

// Instruction descriptor of kind::f16: fp32 accumulation, bf16 operands; `mn` for M-major A and N-major B.
__host__ __device__ constexpr uint32_t mma_idesc(bool mn, int n) {
  return (1u << 4) | (1u << 7) | (1u << 10) | ((mn ? 3u : 0u) << 15) | (static_cast<uint32_t>(n >> 3) << 17) |
         ((128u >> 4) << 24);
}

// D[tmem] (+)= A x B; a and b are descriptors' low words.
__device__ __forceinline__ void mma(uint32_t d, uint32_t a, uint32_t a_hi, uint32_t b, uint32_t b_hi, uint32_t idesc,
                                    uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n .reg .b64 x, y;\n mov.b64 x, {%1, %2};\n mov.b64 y, {%3, %4};\n setp.ne.b32 p, %6, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %5, p;\n}" ::"r"(d),
      "r"(a), "r"(a_hi), "r"(b), "r"(b_hi), "r"(idesc), "r"(accumulate)
      : "memory");
}

__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// x0, x1 as two bf16 pairs, hi + lo: hi is x cut to bf16, lo the rest rounded (16 bits together).
__device__ __forceinline__ void split_bf16x2(float x0, float x1, uint32_t& hi, uint32_t& lo) {
  const uint32_t u0 = __float_as_uint(x0), u1 = __float_as_uint(x1);
  hi = __byte_perm(u0, u1, 0x7632);
  float r0 = __uint_as_float(u0 & 0xffff0000u), r1 = __uint_as_float(u1 & 0xffff0000u);
  fma2(r0, r1, -1.f, -1.f, x0, x1);
  lo = bf16x2(r0, r1);
}

// O from its two parts. Where hi's is infinite, as an infinite value makes it, lo's may be NaN (a lo of zero times
// infinity) and has nothing to add.
__device__ __forceinline__ float join_parts(float hi, float lo) { return fabsf(hi) == INFINITY ? hi : hi + lo; }

// Four E4M3 codes as two pairs of bf16. Through fp16 and fp32, all of it exact: a value has 4 bits, NaN stays NaN.
__device__ __forceinline__ void widen4(uint32_t codes, uint32_t& lo, uint32_t& hi) {
  asm("{\n .reg .b16 a, b, c, d;\n .reg .b32 f, g, x, y;\n"
      " mov.b32 {a, b}, %2;\n"
      " cvt.rn.f16x2.e4m3x2 f, a;\n"
      " cvt.rn.f16x2.e4m3x2 g, b;\n"
      " mov.b32 {a, b}, f;\n"
      " mov.b32 {c, d}, g;\n"
      " cvt.f32.f16 x, a;\n"
      " cvt.f32.f16 y, b;\n"
      " prmt.b32 %0, x, y, 0x7632;\n"
      " cvt.f32.f16 x, c;\n"
      " cvt.f32.f16 y, d;\n"
      " prmt.b32 %1, x, y, 0x7632;\n}"
      : "=r"(lo), "=r"(hi)
      : "r"(codes));
}

// Reduce kN values over the 32 lanes of a warp, halving the values a lane
// keeps at every step: lane i ends with value `first` (and the next, for 64).
// Fewer than 32 values end with copies in neighbouring lanes.
template <int kN, bool kMax>
__device__ __forceinline__ int reduce_columns(float (&v)[kN]) {
  const int lane = threadIdx.x & 31;
  int first = 0, n = kN;
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) {
    if (n > 1) {
      n >>= 1;
      const bool upper = lane & off;
#pragma unroll
      for (int i = 0; i < kN / 2; ++i) {
        if (i < n) {
          const float send = upper ? v[i] : v[i + n], keep = upper ? v[i + n] : v[i];
          const float got = __shfl_xor_sync(0xffffffffu, send, off);
          v[i] = kMax ? fmaxf(keep, got) : keep + got;
        }
      }
      if (upper) first += n;
    } else {
      const float got = __shfl_xor_sync(0xffffffffu, v[0], off);
      v[0] = kMax ? fmaxf(v[0], got) : v[0] + got;
    }
  }
  return first;
}

// The tokens of a row: decode positions [first, last), or entries of its ids.
__device__ __forceinline__ void row_range(const AttnParams& p, int row, bool report, int32_t& first, int32_t& last) {
  if (p.token_ids) {
    first = 0;
    last = p.num_ids;
    return;
  }
  const int64_t cap = static_cast<int64_t>(p.bt_stride) * p.page_size;
  const int32_t ke = p.row_ke[row];
  first = p.row_ks ? max(p.row_ks[row], 0) : 0;
  last = ke > cap ? static_cast<int32_t>(cap) : ke;
  if (report && ke > cap && ke > first) atomicOr(p.status, kStatusBounds);
  if (last < first) last = first;
}

__device__ __forceinline__ int64_t row_tiles(int32_t first, int32_t last) {
  const int64_t n = (static_cast<int64_t>(last) - first + kAttnTile - 1) / kAttnTile;
  return n > 0 ? n : 1;  // a row without tokens still has a result to write
}

// Quotients of what is nearly always short: the 64-bit division is a long routine.
__device__ __forceinline__ long long div_of(long long a, long long b) {
  if (((a | b) >> 32) == 0) return static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
  return a / b;
}

}  // namespace

template <int D, bool kE4m3, int N>
__global__ void __launch_bounds__(Shape<D, kE4m3, N>::kThreads, 1) attention_kernel(const __grid_constant__ AttnParams p) {
  using S = Shape<D, kE4m3, N>;
  constexpr int C = S::kCols, kThreads = S::kThreads;
  extern __shared__ __align__(1024) uint8_t smem[];
  // operands first (1024-byte aligned), then rings, state and barriers
  uint8_t* const units = smem;
  uint8_t* const raws = units + S::kSlots * S::kUnit;  // E4M3
  uint8_t* const q_s = raws + 2 * S::kRaws * S::kRaw;
  uint8_t* const p_s = q_s + S::kQBufs * S::kQBytes;
  int64_t* const ring_off = reinterpret_cast<int64_t*>(p_s + S::kPBytes);          // [ring][128]
  float2* const ring_scale = reinterpret_cast<float2*>(ring_off + S::kRing * 128);  // [ring][128], E4M3
  uint32_t* const ring_mask = reinterpret_cast<uint32_t*>(reinterpret_cast<uint8_t*>(ring_off) + S::kRingBytes);
  AttnSeg* const segs = reinterpret_cast<AttnSeg*>(ring_mask + S::kRing * 4);
  float* const nm_s = reinterpret_cast<float*>(segs + kSegRing);  // [N] running maxima, negated
  float* const alpha_s = nm_s + N;                               // [N] rescale factors
  float* const up_s = alpha_s + N;                               // [N] the last raise of each maximum
  float* const inv_s = up_s + N;                                 // [N] 1 / l of the segment being written
  float* const scratch = inv_s + N;                              // [2][4][C]
  uint64_t* const bars = reinterpret_cast<uint64_t*>(scratch + 8 * C);
  // barriers
  constexpr int kFull = 0, kEmpty = kFull + S::kSlots, kSFull = kEmpty + S::kSlots, kSEmpty = kSFull + 2, kPFull = kSEmpty + 2,
                kPvDone = kPFull + 1, kQEmpty = kPvDone + 1, kQFull = kQEmpty + 2, kSegFull = kQFull + 2,
                kSegEmpty = kSegFull + kSegRing,
                kAFull = kSegEmpty + kSegRing, kAEmpty = kAFull + S::kRing, kDrain = kAEmpty + S::kRing, kScFull = kDrain + 2,
                kBars = kScFull + (kE4m3 ? S::kRing : 0);
  static_assert(kBars * 8 <= 640, "");
  auto bar = [&](int i) { return smem_addr(bars + i); };

  __shared__ uint32_t tmem_slot;
  __shared__ int abort_flag;
  __shared__ long long warp_sum[kThreads / 32];
  __shared__ long long start_idx;
  __shared__ int start_row;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint64_t limit = static_cast<uint64_t>(p.wait_ns);
  griddep_launch_dependents();

  if (tid < kBars) {  // a barrier a thread
    const int i = tid;
    const int count = i < kEmpty ? (kE4m3 ? kLoaders / 32 : kLoaders)         // K and V units: loader warps, or each thread's copies
                      : i < kSEmpty ? 1                                       // freed by the MMAs; S
                      : i < kPvDone ? kSoftmax / 32                           // S read, P written: each softmax warp
                      : i < kQFull ? 1                                        // O; queries freed by the MMAs
                      : i < kSegFull ? kLoaders                               // queries over an 8-bit cache: each thread's copies
                      : i < kSegEmpty ? 1 : i < kAFull ? S::kSegReaders          // segments
                      : i < kAEmpty ? 1 : i < kDrain ? S::kAddrReaders           // addresses
                      : i < kScFull ? 1 : 64;                                 // drains; scales: each lane's copies, and its stores
    mbar_init(bar(i), count);
  }
  if (tid == 0) {
    abort_flag = 0;
    start_row = -1;
  }
  if (tid < kBars) mbar_init_fence();
  if (tid < N) nm_s[tid] = 0.f;
  if (warp == 5) tmem_alloc(smem_addr(&tmem_slot), S::kTmem);
  griddep_wait();

  // ---- this CTA's range of the tile list
  tc_fence_before();
  long long total, begin, chunk;
  if (p.token_ids) {  // rows of one length
    total = row_tiles(0, p.num_ids) * p.kv_heads * p.rows;
  } else {  // prefix sums over the rows
    const int per_thread = (p.rows + kThreads - 1) / kThreads;
    long long mine = 0;
    for (int i = 0; i < per_thread; ++i) {
      const int r = tid * per_thread + i;
      if (r >= p.rows) break;
      int32_t first, last;
      row_range(p, r, blockIdx.x == 0, first, last);
      mine += row_tiles(first, last) * p.kv_heads;
    }
    long long incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    if (lane == 31) warp_sum[warp] = incl;
    __syncthreads();
    long long before = incl - mine;
    total = 0;
    for (int w = 0; w < kThreads / 32; ++w) {
      if (w < warp) before += warp_sum[w];
      total += warp_sum[w];
    }
    begin = div_of(total + gridDim.x - 1, gridDim.x) * blockIdx.x;
    if (begin < total && begin >= before && begin < before + mine) {
      long long at = before;
      for (int i = 0; i < per_thread; ++i) {
        const int r = tid * per_thread + i;
        int32_t first, last;
        row_range(p, r, false, first, last);
        const long long t = row_tiles(first, last) * p.kv_heads;
        if (begin < at + t) {
          start_row = r;
          start_idx = begin - at;
          break;
        }
        at += t;
      }
    }
  }
  chunk = div_of(total + gridDim.x - 1, gridDim.x);
  begin = chunk * blockIdx.x;
  const long long work = begin < total ? min(chunk, total - begin) : 0;
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_slot;
  const uint32_t tmem_o = tmem, tmem_sc = tmem + 2 * N;
  const volatile int* const abort = &abort_flag;
  auto fail = [&] { *reinterpret_cast<volatile int*>(&abort_flag) = 1; };  // reported at the end

  // the softmax threads take registers that the others do not need
  if (warp < 8 || warp >= 16) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(S::kOtherRegs));
    if (warp < 4 || warp >= 16) {
      // ------------------------------------------------------------ loaders
      const int stall_tile = blockIdx.x == 0 ? p.stall_tile : -1;  // tests: its keys are not handed over
      const uint32_t units_a = smem_addr(units);
      bool ok = true;
      auto wait = [&](int b, uint32_t parity) {
        ok = wait_phase(bar(b), parity, abort, limit);
        return ok;
      };
      auto fetch_queries = [&](const AttnSeg& sg, int qb) {
        const uint16_t* const qrow = p.q + sg.row * p.q_stride + static_cast<int64_t>(sg.kvh) * p.group * D;
        constexpr int kQChunks = D * 2 / 16, kQTok = 32 / kQChunks;
        const int c = lane % kQChunks;
        for (int i = warp * kQTok + lane / kQChunks; i < N; i += 4 * kQTok)
          cp16(smem_addr(q_s + qb * S::kQBytes) + (c >> 3) * (N * 128) + i * 128 + (((c & 7) ^ (i & 7)) << 4),
               qrow + (i < p.group ? i * D + c * 8 : 0), i < p.group ? 16 : 0);
      };
      if constexpr (kE4m3) {
        // Warps 0-3 bring keys, warps 16-19 values. Each lane copies pieces of 16 codes into a place of its own and widens
        // them later into the unit that the tensor core reads, so the copies need no barrier. Two cursors go over the
        // tiles: one copies, up to kRaws tiles ahead of the one that widens.
        constexpr int kPieces = D / 16;                             // of a token
        constexpr int kTok = 32 / kPieces, kPer = 32 / kTok;        // tokens per warp instruction, pieces per lane and unit
        // Eight lanes have two neighbouring tokens' pieces of one 128-byte column, so that their stores, two 16-byte
        // chunks apart within a token and swizzled by the token, meet every bank once.
        const int piece = (lane & 3) | (kPieces == 8 ? (lane >> 1) & 4 : 0);
        const int sub = kPieces == 8 ? ((lane >> 2) & 1) | ((lane >> 3) & 2) : lane >> 2;
        const bool values = warp >= 16;
        const int w0 = (warp & 3) * 32;                             // the warp's first token
        uint8_t* const mine = raws + (values ? S::kRaws * S::kRaw : 0) + w0 * D + lane * 16;
        const uint8_t* const base = static_cast<const uint8_t*>(values ? p.v_cache : p.k_cache) + piece * 16;
        int ahead = 0;                                              // tiles copied and not yet widened
        int cseg = 0, cleft = 0, ctile = 0, craw = 0, qseg = 0;     // copying; segments whose queries are asked for
        int seg = 0, left = 0, tile = 0, raw = 0;                   // widening
        int slot = values ? 1 : 0;                                  // keys in the even units, values in the odd ones
        uint32_t turn = 1;
        bool more = true;
        auto ready = [&](int b, uint32_t parity) { return __all_sync(0xffffffffu, mbar_test_wait(bar(b), parity)); };
        while (true) {
          if (more && ahead < S::kRaws) {
            // copy the next tile; as long as there is something to widen, only if its segment and addresses are there
            bool there = true;
            if (cleft == 0) {
              const int at = kSegFull + cseg % kSegRing, parity = (cseg / kSegRing) & 1;
              there = ahead > 0 ? ready(at, parity) : wait(at, parity);
              if (there) {
                const AttnSeg& sg = segs[cseg % kSegRing];
                cleft = sg.ntiles;
                more = there = cleft > 0;
                const int qb = cseg % S::kQBufs;
                if (more && !values && qseg == cseg && ready(kQEmpty + qb, (cseg / S::kQBufs + 1) & 1)) {
                  fetch_queries(sg, qb);
                  cp_arrive(bar(kQFull + qb));
                  ++qseg;
                }
                ++cseg;
              }
            }
            if (there) {
              const int at = kAFull + ctile % S::kRing, parity = (ctile / S::kRing) & 1;
              there = ahead > 0 ? ready(at, parity) : wait(at, parity);
            }
            if (!ok) break;
            if (there) {
              const int64_t* const offs = ring_off + ctile % S::kRing * 128 + w0 + sub;
              const uint32_t dst = smem_addr(mine) + craw * S::kRaw;
              const bool whole = ring_mask[ctile % S::kRing * 4 + (warp & 3)] == 0xffffffffu;  // every token is there
              if (__builtin_expect(whole, 1)) {
#pragma unroll
                for (int i0 = 0; i0 < kPer; i0 += 4) {
                  const uint8_t* src[4];
#pragma unroll
                  for (int i = 0; i < 4; ++i) src[i] = base + offs[(i0 + i) * kTok];
#pragma unroll
                  for (int i = 0; i < 4; ++i) cp16(dst + (i0 + i) * 512, src[i]);
                }
              } else {
#pragma unroll 1
                for (int i = 0; i < kPer; ++i) {
                  const int64_t o = offs[i * kTok];
                  cp16(dst + i * 512, base + (o < 0 ? 0 : o), o < 0 ? 0 : 16);
                }
              }
              cp_commit();
              __syncwarp();
              arrive_one(bar(kAEmpty + ctile % S::kRing), lane);
              ++ctile;
              --cleft;
              if (++craw == S::kRaws) craw = 0;
              ++ahead;
              continue;
            }
          }
          if (ahead == 0) break;
          if (left == 0) {
            left = segs[seg % kSegRing].ntiles;
            if (!values && qseg == seg) {
              const int qb = seg % S::kQBufs;
              if (!wait(kQEmpty + qb, (seg / S::kQBufs + 1) & 1)) break;
              fetch_queries(segs[seg % kSegRing], qb);
              cp_arrive(bar(kQFull + qb));
              ++qseg;
            }
            __syncwarp();
            arrive_one(bar(kSegEmpty + seg % kSegRing), lane);
            ++seg;
          }
          if (!wait(kEmpty + slot, turn)) break;
          if (ahead == S::kRaws)
            cp_wait<S::kRaws - 1>();  // the oldest tile has landed
          else
            cp_wait_all();
          const uint8_t* const src = mine + raw * S::kRaw;
          const uint32_t dst = units_a + slot * S::kUnit + (piece >> 2) * 16384 + (w0 + sub) * 128;
#pragma unroll 1
          for (int i0 = 0; i0 < kPer; i0 += 2) {
            uint4 w[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) w[i] = *reinterpret_cast<const uint4*>(src + (i0 + i) * 512);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const uint32_t row = dst + (i0 + i) * (kTok * 128), t = (i * kTok + sub) & 7;  // i0 * kTok is a multiple of 8
              uint32_t x[4];
              widen4(w[i].x, x[0], x[1]);
              widen4(w[i].y, x[2], x[3]);
              sts16(row + (((piece & 3) * 2 ^ t) << 4), x[0], x[1], x[2], x[3]);
              widen4(w[i].z, x[0], x[1]);
              widen4(w[i].w, x[2], x[3]);
              sts16(row + (((piece & 3) * 2 + 1 ^ t) << 4), x[0], x[1], x[2], x[3]);
            }
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (values || stall_tile != tile) arrive_one(bar(kFull + slot), lane);
          slot += 2;
          if (slot >= S::kSlots) {
            slot -= S::kSlots;
            turn ^= 1;
          }
          if (++raw == S::kRaws) raw = 0;
          --ahead;
          ++tile;
          --left;
        }
      } else {
        constexpr int kChunks = S::kRow / 16;         // 16-byte pieces of a token
        constexpr int kTok = 32 / kChunks;            // tokens per warp instruction
        const int piece = lane % kChunks, sub = lane / kChunks;
        // Units: K 0, V 0, K 1, V 1, ... The unit's barrier counts each thread's copies when they land; the MMA warps'
        // proxy fence, after their wait, orders them before the tensor core's reads.
        int slot = 0, seg = 0, left = 0, tile = 0;  // left: tiles of this segment
        uint32_t turn = 1;                          // parity that says that the slot is free
        for (bool values = false; ok; values = !values) {
          if (!values) {
            if (left == 0) {
              if (!wait(kSegFull + seg % kSegRing, (seg / kSegRing) & 1)) break;
              const AttnSeg sg = segs[seg % kSegRing];
              left = sg.ntiles;
              if (left == 0) break;
              // the segment's queries: its first K tile's barrier covers them
              const int qb = seg % S::kQBufs;
              if (!wait(kQEmpty + qb, (seg / S::kQBufs + 1) & 1)) break;
              fetch_queries(sg, qb);
              __syncwarp();
              arrive_one(bar(kSegEmpty + seg % kSegRing), lane);
              ++seg;
            }
            if (!wait(kAFull + tile % S::kRing, (tile / S::kRing) & 1)) break;
          }
          if (!wait(kEmpty + slot, turn)) break;
          const uint8_t* const base = static_cast<const uint8_t*>(values ? p.v_cache : p.k_cache) + piece * 16;
          const uint32_t dst0 = units_a + slot * S::kUnit + (piece >> 3) * 16384;
          const int64_t* const offs = ring_off + tile % S::kRing * 128 + warp * 32 + sub;
          constexpr int kBatch = 32 / kTok < 8 ? 32 / kTok : 8;  // addresses first, so that the copies issue back to back
          const uint32_t dst1 = dst0 + (warp * 32 + sub) * 128;
          const bool whole = ring_mask[tile % S::kRing * 4 + warp] == 0xffffffffu;  // every token of the warp is there
          if (__builtin_expect(whole, 1)) {
#pragma unroll
            for (int i0 = 0; i0 < 32 / kTok; i0 += kBatch) {
              const uint8_t* src[kBatch];
#pragma unroll
              for (int i = 0; i < kBatch; ++i) src[i] = base + offs[(i0 + i) * kTok];
#pragma unroll
              for (int i = 0; i < kBatch; ++i)
                cp16(dst1 + (i0 + i) * kTok * 128 + (((piece & 7) ^ (((i0 + i) * kTok + sub) & 7)) << 4), src[i]);
            }
          } else {
#pragma unroll 1
            for (int i0 = 0; i0 < 32 / kTok; i0 += 4) {
              int64_t o[4];
#pragma unroll
              for (int i = 0; i < 4; ++i) o[i] = offs[(i0 + i) * kTok];
#pragma unroll
              for (int i = 0; i < 4; ++i)
                cp16(dst1 + (i0 + i) * kTok * 128 + (((piece & 7) ^ (((i0 + i) * kTok + sub) & 7)) << 4),
                     base + (o[i] < 0 ? 0 : o[i]), o[i] < 0 ? 0 : 16);
            }
          }
          if (values || stall_tile != tile) cp_arrive(bar(kFull + slot));
          if (++slot == S::kSlots) {
            slot = 0;
            turn ^= 1;
          }
          if (values) {
            __syncwarp();
            arrive_one(bar(kAEmpty + tile % S::kRing), lane);
            ++tile;
            --left;
          }
        }
      }
      if (!ok && lane == 0) fail();
      cp_wait_all();
    } else if (warp == 4) {
      // ---------------------------------------------------------- scheduler
      long long left = work;
      int row = 0;
      long long idx = 0;  // tile of the row, over its kv heads
      if (work > 0 && p.token_ids) {
        const long long per_row = row_tiles(0, p.num_ids) * p.kv_heads;
        row = static_cast<int>(div_of(begin, per_row));
        idx = begin - row * per_row;
      } else if (work > 0) {
        row = start_row;
        idx = start_idx;
      }
      int4 info = make_int4(0, 0, 0, 0);
      int base = -64, seg = 0;
      int32_t first_l = 0, last_l = 0, table_l = 0;
      bool ok = true;
      while (ok) {
        AttnSeg sg;
        sg.ntiles = 0;
        if (left > 0) {
          if (row >= base + 32) {  // the next 32 rows' ranges, one per lane
            base = row;
            if (row + lane < p.rows) {
              table_l = p.row_indices ? p.row_indices[row + lane] : row + lane;
              if (table_l < 0 || table_l >= p.bt_rows) table_l = -1;
              row_range(p, row + lane, false, first_l, last_l);
            }
          }
          sg.table_row = __shfl_sync(0xffffffffu, table_l, row - base);
          sg.first = __shfl_sync(0xffffffffu, first_l, row - base);
          sg.last = __shfl_sync(0xffffffffu, last_l, row - base);
          const long long t = row_tiles(sg.first, sg.last);
          sg.row = row;
          sg.kvh = p.kv_heads == 1 ? 0 : static_cast<int>(div_of(idx, t));
          sg.tile0 = static_cast<int>(idx - sg.kvh * t);
          const long long n = min(t - sg.tile0, left);
          sg.ntiles = static_cast<int>(n);
          const bool starts = sg.tile0 == 0, ends = sg.tile0 + n == t;
          sg.slot = starts && ends ? -1 : 2 * static_cast<int>(blockIdx.x) + (starts ? 1 : 0);
          if (starts && !ends) info = make_int4(row, sg.kvh, static_cast<int>(div_of(t - n + chunk - 1, chunk)), 0);
          left -= n;
          idx += n;
          if (idx == t * p.kv_heads) {
            ++row;
            idx = 0;
          }
        }
        if (seg >= kSegRing) ok = wait_phase(bar(kSegEmpty + seg % kSegRing), (seg / kSegRing - 1) & 1, abort, limit);
        if (!ok) break;
        if (lane == 0) {
          segs[seg % kSegRing] = sg;
          mbar_arrive(bar(kSegFull + seg % kSegRing));
        }
        ++seg;
        if (sg.ntiles == 0) break;
      }
      if (lane == 0) {
        if (!ok) fail();
        p.seg_info[blockIdx.x] = info;
      }
    } else if (warp != 6) {
      // ---------------------------------------------------------------- MMA
      // Warp 5 issues S = K Q^T, warp 7 O += V^T P: apart, so that S runs ahead of the softmax. The whole warp runs
      // the loop, so that descriptors stay in uniform registers, and one elected thread issues.
      constexpr uint32_t kRowHi = desc_hi(128);
      const bool scores = warp == 5;
      bool ok = true;
      auto wait = [&](int b, uint32_t parity) {
        ok = wait_phase(bar(b), parity, abort, limit);
        return ok;
      };
      int slot = scores ? 0 : 1, it = 0;  // the tile's unit: K tiles are the even ones, V tiles the odd ones
      uint32_t turn = 0;
      for (int seg = 0; ok; ++seg) {
        if (!wait(kSegFull + seg % kSegRing, (seg / kSegRing) & 1)) break;
        const int n = segs[seg % kSegRing].ntiles;
        __syncwarp();
        arrive_one(bar(kSegEmpty + seg % kSegRing), lane);
        if (n == 0) break;
        const int qb = seg % S::kQBufs;
        if (kE4m3 && scores && !wait(kQFull + qb, (seg / S::kQBufs) & 1)) break;
        for (int j = 0; j < n; ++j, ++it) {
          // the softmax reads the tile's mask and scales behind S: they are there before S is issued
          if (scores && !wait((kE4m3 ? kScFull : kAFull) + it % S::kRing, (it / S::kRing) & 1)) break;
          if (!wait(kFull + slot, turn)) break;
          if (!wait(scores ? kSEmpty + (it & 1) : kPFull, scores ? ((it >> 1) + 1) & 1 : it & 1)) break;
          fence_proxy_async_smem();
          tc_fence_after();
          const uint32_t unit_a = smem_addr(units) + slot * S::kUnit;
          if (scores) {
            constexpr uint32_t kDesc = mma_idesc(false, N);
            const uint32_t a = desc_lo(unit_a, 16), q = desc_lo(smem_addr(q_s) + qb * S::kQBytes, 16);
            if (elect_one()) {
#pragma unroll
              for (int k = 0; k < S::kRow / 32; ++k)  // 32 bytes of K
                mma(tmem_sc + (it & 1) * N, a + (((k >> 2) * 16384 + (k & 3) * 32) >> 4), kRowHi,
                    q + (((k >> 2) * (N * 128) + (k & 3) * 32) >> 4), kRowHi, kDesc, k > 0);
              mma_commit(bar(kEmpty + slot));
              mma_commit(bar(kSFull + (it & 1)));
              if (j == n - 1) mma_commit(bar(kQEmpty + qb));
            }
          } else {
            constexpr uint32_t kDesc = mma_idesc(true, 2 * N);
            const uint32_t a = desc_lo(unit_a, 16384), q = desc_lo(smem_addr(p_s), 128 * S::kPRow);
            if (elect_one()) {
#pragma unroll
              for (int k = 0; k < 8; ++k)  // 16 tokens
                mma(tmem_o, a + ((k * 16 * 128) >> 4), kRowHi, q + ((k * 16 * S::kPRow) >> 4), desc_hi(S::kPRow), kDesc,
                    j + k > 0);
              mma_commit(bar(kEmpty + slot));
              mma_commit(bar(kPvDone));
            }
          }
          __syncwarp();
          slot += 2;
          if (slot >= S::kSlots) {
            slot -= S::kSlots;
            turn ^= 1;
          }
        }
      }
      if (!ok && lane == 0) fail();
      // The MMAs issued so far read shared memory and write TMEM, which a softmax whose waits ran out would free under
      // them: they end by themselves, so this wait has a limit of its own and not the plan's.
      if (it > 0) {
        const int drain = scores ? kDrain : kDrain + 1;
        if (elect_one()) mma_commit(bar(drain));
        const int never = 0;
        wait_phase(bar(drain), 0, &never, 2000000000ull);
      }
      __syncwarp();
    } else {
      // ---------------------------------------------------------- addresses
      // One warp, four tokens a lane; the next tile's ids are on their way while this tile's pages are looked up.
      const int shift = p.page_shift;
      bool ok = true;
      auto wait = [&](int b, uint32_t parity) {
        ok = wait_phase(bar(b), parity, abort, limit);
        return ok;
      };
      AttnSeg sg;
      sg.ntiles = 0;
      int seg = -1, j = 0;
      int64_t ids_at = 0, head_at = 0;
      const int32_t* table = nullptr;  // the row's block-table row, null if out of range
      // the next tile of the work: its tokens' positions, -1 where there is none; false at the end
      auto next_tile = [&](int32_t(&pos)[4]) {
        if (++j >= sg.ntiles) {
          ++seg;
          j = 0;
          if (!wait(kSegFull + seg % kSegRing, (seg / kSegRing) & 1)) return false;
          sg = segs[seg % kSegRing];
          __syncwarp();
          arrive_one(bar(kSegEmpty + seg % kSegRing), lane);
          if (sg.ntiles == 0) return false;
          table = sg.table_row >= 0 ? p.block_table + static_cast<int64_t>(sg.table_row) * p.bt_stride : nullptr;
          ids_at = static_cast<int64_t>(sg.row) * p.ids_ld;
          head_at = static_cast<int64_t>(sg.kvh) * p.page_size;
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int64_t e = static_cast<int64_t>(sg.tile0 + j) * kAttnTile + k * 32 + lane;
          pos[k] = -1;
          if (p.token_ids) {
            if (e < sg.last) pos[k] = p.token_ids[ids_at + e];
          } else if (sg.first + e < sg.last) {
            pos[k] = static_cast<int32_t>(sg.first + e);
          }
        }
        return true;
      };
      int32_t ahead[4];
      bool more = next_tile(ahead);
      for (int it = 0; more; ++it) {
        const int a = it % S::kRing;
        const int64_t head = head_at;
        int32_t in_page[4], page[4];
        bool asked[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          asked[k] = ahead[k] >= 0;
          page[k] = -1;
          in_page[k] = 0;
          if (asked[k]) {
            const int32_t col = shift >= 0 ? ahead[k] >> shift : ahead[k] / p.page_size;
            in_page[k] = ahead[k] - col * p.page_size;
            if (table && col < p.bt_stride) page[k] = table[col];
          }
        }
        more = next_tile(ahead);
        if (!ok || !wait(kAEmpty + a, (it / S::kRing + 1) & 1)) break;
        bool bad = false;
        int64_t off[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          off[k] = -1;
          float2* const scale = ring_scale + a * 128 + k * 32 + lane;
          if (page[k] >= 0 && page[k] < p.num_pages) {
            const int64_t vec = head + in_page[k];
            off[k] = (page[k] * p.page_stride + vec * D) * (kE4m3 ? 1 : 2);
            if (kE4m3) {
              const int64_t at = page[k] * p.scale_page_stride + vec;
              cp4(smem_addr(&scale->x), p.k_scales + at);
              cp4(smem_addr(&scale->y), p.v_scales + at);
            }
          } else {
            if (kE4m3) *scale = make_float2(1.f, 1.f);
            bad |= asked[k];
          }
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          ring_off[a * 128 + k * 32 + lane] = off[k];
          const uint32_t mask = __ballot_sync(0xffffffffu, off[k] >= 0);
          if (lane == 0) ring_mask[a * 4 + k] = mask;
        }
        if (kE4m3) {
          cp_arrive(bar(kScFull + a));
          mbar_arrive(bar(kScFull + a));
        }
        if (bad) atomicOr(p.status, kStatusBounds);
        __syncwarp();
        arrive_one(bar(kAFull + a), lane);
      }
      if (!ok && lane == 0) fail();
      cp_wait_all();
    }
  } else {
    // ------------------------------------------------------------ softmax
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(S::kSoftmaxRegs));
    const int wg = (warp - 8) >> 2, quarter = warp & 3;
    const int t = quarter * 32 + lane;          // this thread's token, and its row of O^T
    const int c0 = wg * C;                      // its first head
    const int bar_id = 1 + wg, wt = tid & 127;
    const uint32_t lanes = static_cast<uint32_t>(quarter * 32) << 16;
    const uint32_t o_col = tmem_o + lanes + c0;
    float* const red = scratch + wg * 4 * C;
    // this thread's row of P: the 16-byte pieces of its heads, swizzled (its first piece is a multiple of their number)
    constexpr int kWords = C / 2;
    constexpr bool kWide = N == 128;  // a block of 64 heads for each group
    const int p_swz = (S::kPRow == 128 ? (t & 7) : S::kPRow == 64 ? ((t >> 1) & 3) : ((t >> 2) & 1)) ^
                      (kWide ? 0 : wg * (kWords / 4));
    const uint32_t p_row = smem_addr(p_s) + t * S::kPRow + (kWide ? wg * 128 * S::kPRow : 0);
    bool failed = false, leave = false;
    int it = 0;
    auto wait = [&](int b, uint32_t parity) {
      if (!failed) failed = !wait_phase(bar(b), parity, abort, limit);
    };
    // Write the result of segment w, whose O is final: normalised by inv_s, or as a partial.
    auto write_out = [&](const AttnSeg& w) {
      tc_fence_after();
      constexpr int kStep = C <= 32 && C >= 16 ? 16 : 8;
#pragma unroll (C > 32 ? 1 : 2)
      for (int c = 0; c < C; c += kStep) {
        if (c0 + c >= p.group) break;
        float o[kStep], o2[kStep];
        tmem_ld<kStep>(o_col + c, o);
        tmem_ld<kStep>(o_col + N + c, o2);
        tmem_wait_ld();
        pin<kStep>(o);
        pin<kStep>(o2);
        if (t >= D) continue;  // whole warps
        if (w.slot >= 0) {
          float* const dst = p.part_o + (w.slot * p.group + c0 + c) * D + t;
#pragma unroll
          for (int i = 0; i < kStep; ++i)
            if (c0 + c + i < p.group) dst[i * D] = join_parts(o[i], o2[i]);
        } else {
          // lanes 2 i and 2 i + 1 exchange, so that each writes two elements of every other head
          uint16_t* const dst = p.out +
                                ((static_cast<int64_t>(w.row) * p.kv_heads + w.kvh) * p.group + c0 + c + (lane & 1)) * D +
                                (t & ~1);
#pragma unroll
          for (int i = 0; i < kStep; i += 2) {
            const float x = join_parts(o[i], o2[i]) * inv_s[c0 + c + i];
            const float y = join_parts(o[i + 1], o2[i + 1]) * inv_s[c0 + c + i + 1];
            const float got = __shfl_xor_sync(0xffffffffu, lane & 1 ? x : y, 1);
            if (c0 + c + i + (lane & 1) < p.group)
              *reinterpret_cast<uint32_t*>(dst + i * D) = lane & 1 ? bf16x2(got, y) : bf16x2(x, got);
          }
        }
      }
      tc_fence_before();
    };
    float l[C];
    bool s_ready = false;
    AttnSeg done;  // the segment whose O is still to be written: behind the next one's first tile
    done.ntiles = 0;
    for (int seg = 0;; ++seg) {
      wait(kSegFull + seg % kSegRing, (seg / kSegRing) & 1);
      // a group leaves together: a failed wait anywhere in it ends all of it
      if (bar_or(bar_id, 128, failed)) break;
      const AttnSeg sg = segs[seg % kSegRing];
      __syncwarp();
      arrive_one(bar(kSegEmpty + seg % kSegRing), lane);
      if (sg.ntiles == 0) {
        if (done.ntiles > 0) {
          wait(kPvDone, (it - 1) & 1);
          if (!failed) write_out(done);
        }
        break;
      }
#pragma unroll
      for (int c = 0; c < C; ++c) l[c] = 0.f;
      bool fresh = true;  // some head has had no score above minus infinity so far
      bool mine = wt < C && c0 + wt < p.group;  // the head that this thread keeps the maximum of is one of them
      for (int j = 0; j < sg.ntiles; ++j, ++it) {
        const int a = it % S::kRing;
        if (__builtin_expect(!s_ready, 0)) wait(kSFull + (it & 1), (it >> 1) & 1);
        float s[C];  // scores, less the running maxima, then P
        bool over = failed;
        tc_fence_after();  // (after a failed wait the scores are of no use, and do no harm)
        const uint32_t s_col = tmem_sc + lanes + (it & 1) * N + c0;
        constexpr int kLd = C > 32 ? 32 : C;
#pragma unroll
        for (int c = 0; c < C; c += kLd) tmem_ld<kLd>(s_col + c, s + c);
        float mul = p.scale_log2, vs = 1.f;
        const uint4 mask = *reinterpret_cast<const uint4*>(ring_mask + a * 4);
        const bool valid = ((quarter == 0 ? mask.x : quarter == 1 ? mask.y : quarter == 2 ? mask.z : mask.w) >> lane) & 1;
        const bool first = fresh && (mask.x | mask.y | mask.z | mask.w) != 0;
        if (kE4m3) {
          const float2 sc = ring_scale[a * 128 + t];
          mul *= sc.x;
          vs = sc.y;
        }
        tmem_wait_ld();
        pin<C>(s);
        tc_fence_before();
        __syncwarp();
        arrive_one(bar(kSEmpty + (it & 1)), lane);
        arrive_one(bar(kAEmpty + a), lane);
        float most = -INFINITY;
#pragma unroll
        for (int c = 0; c < C; c += 4) {
          const float4 a4 = *reinterpret_cast<const float4*>(nm_s + c0 + c);
          fma2(s[c], s[c + 1], mul, mul, a4.x, a4.y);
          fma2(s[c + 2], s[c + 3], mul, mul, a4.z, a4.w);
          most = fmaxf(fmaxf(most, fmaxf(s[c], s[c + 1])), fmaxf(s[c + 2], s[c + 3]));
        }
        if (!valid) {
#pragma unroll
          for (int c = 0; c < C; ++c) s[c] = -INFINITY;
          most = -INFINITY;
        }
        over |= most > kTau || first;
        const bool raise = bar_or(bar_id, 128, over);
        // asked early, as an answer takes its time behind the copies in the load-store queue
        const bool pv_ready = it == 0 || __all_sync(0xffffffffu, mbar_test_wait(bar(kPvDone), (it - 1) & 1));
        if (__builtin_expect(raise, 0)) {
          // raise this group's maxima to the tile's, or set them at the row's first tokens
          constexpr int kHalf = C > 32 ? 32 : C;
#pragma unroll
          for (int h = 0; h < C; h += kHalf) {
            float v[kHalf];
#pragma unroll
            for (int c = 0; c < kHalf; ++c) v[c] = s[h + c];
            const int col = reduce_columns<kHalf, true>(v);
            red[quarter * C + h + col] = v[0];
          }
          if (bar_or(bar_id, 128, failed)) {
            leave = true;
            break;
          }
          if (wt < C) {
            const float top = fmaxf(fmaxf(red[wt], red[C + wt]), fmaxf(red[2 * C + wt], red[3 * C + wt]));
            const float up = top == -INFINITY ? 0.f : mine ? top : fmaxf(top, 0.f);
            nm_s[c0 + wt] -= up;
            up_s[c0 + wt] = up;
            alpha_s[c0 + wt] = mine ? 1.f : ex2(-up);  // nothing to rescale at a head's first scores
            mine = mine && top == -INFINITY;
          }
          fresh = bar_or(bar_id, 128, mine);
#pragma unroll
          for (int c = 0; c < C; c += 4) {
            const float4 a4 = *reinterpret_cast<const float4*>(alpha_s + c0 + c);
            const float4 u4 = *reinterpret_cast<const float4*>(up_s + c0 + c);
            l[c] *= a4.x, l[c + 1] *= a4.y, l[c + 2] *= a4.z, l[c + 3] *= a4.w;
            s[c] -= u4.x, s[c + 1] -= u4.y, s[c + 2] -= u4.z, s[c + 3] -= u4.w;
          }
        }
        // this thread's row of P: C heads of token t, in two parts
        uint32_t hi[kWords], lo[kWords];
#pragma unroll
        for (int c = 0; c < C; ++c) s[c] = ex2(s[c]);
#pragma unroll
        for (int i = 0; i < kWords; ++i) {
          add2(l[2 * i], l[2 * i + 1], s[2 * i], s[2 * i + 1]);
          if (kE4m3) mul2(s[2 * i], s[2 * i + 1], vs, vs);
          split_bf16x2(s[2 * i], s[2 * i + 1], hi[i], lo[i]);
        }
        // computed here, not behind the wait, where the compiler would move it
#pragma unroll
        for (int i = 0; i < kWords; ++i) asm volatile("" : "+r"(hi[i]), "+r"(lo[i]));
        s_ready = __all_sync(0xffffffffu, mbar_test_wait(bar(kSFull + ((it + 1) & 1)), ((it + 1) >> 1) & 1));
        if (__builtin_expect(!pv_ready, 0)) wait(kPvDone, (it - 1) & 1);  // O is final up to the previous tile, and P is free
        if (__builtin_expect(j == 0 && done.ntiles > 0, 0)) write_out(done);
        if (__builtin_expect(raise && j > 0, 0)) {
          tc_fence_after();
#pragma unroll
          for (int part = 0; part < 2; ++part)
#pragma unroll
            for (int c = 0; c < C; c += 8) {
              float o[8];
              tmem_ld<8>(o_col + part * N + c, o);
              tmem_wait_ld();
              pin<8>(o);
#pragma unroll
              for (int i = 0; i < 8; ++i) o[i] *= alpha_s[c0 + c + i];
              tmem_st8(o_col + part * N + c, o);
            }
          tmem_wait_st();
          tc_fence_before();
        }
#pragma unroll
        for (int i = 0; i < kWords; i += 4) {
          const uint32_t at = p_row + ((i / 4 ^ p_swz) << 4);
          sts16(at, hi[i], hi[i + 1], hi[i + 2], hi[i + 3]);
          sts16(at + S::kPPart, lo[i], lo[i + 1], lo[i + 2], lo[i + 3]);
        }
        fence_proxy_async_smem();
        __syncwarp();
        arrive_one(bar(kPFull), lane);
      }
      if (leave) break;
      // ---- the segment's sums; its O follows behind the next tile's scores
      const int col = reduce_columns<C, false>(l);
#pragma unroll
      for (int i = 0; i < (C > 32 ? C / 32 : 1); ++i) red[quarter * C + col + i] = l[i];
      bar_sync(bar_id, 128);
      if (wt < C) {
        const int h = c0 + wt;
        const float sum = red[wt] + red[C + wt] + red[2 * C + wt] + red[3 * C + wt];
        const float m = mine ? kUnset : -nm_s[h];
        nm_s[h] = 0.f;
        inv_s[h] = sum == 0.f ? 0.f : __fdividef(1.f, sum);
        if (h < p.group) {
          if (sg.slot >= 0)
            p.part_ml[sg.slot * p.group + h] = make_float2(m, sum);
          else if (p.lse)
            p.lse[static_cast<int64_t>(sg.row) * p.kv_heads * p.group + sg.kvh * p.group + h] =
                (m + lg2(sum)) * 0.69314718055994531f;
        }
      }
      done = sg;
    }
    if (failed) fail();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (tid == 0 && abort_flag) atomicOr(p.status, kStatusTimeout);
  if (warp == 5) tmem_dealloc(tmem, S::kTmem);
}

// Join the partials of an item that CTA `first` of the attention kernel began
// and others continued: out = sum_i w_i O_i / sum_i w_i l_i with
// w_i = 2^(m_i - max m). Bound by latency, of its instructions too (a call runs
// them once), so the two forms are compiled apart. kFew, for few items, whose
// partials are many: a block per item and head, which looks for the item's
// first CTA and shares the partials among its eight warps. Otherwise a block
// per CTA and eight heads, a warp each. The first partial outputs are loaded
// along with the maxima.
template <int D, bool kFew>
__global__ void __launch_bounds__(256) combine_kernel(const __grid_constant__ AttnParams p, int ctas) {
  constexpr int kPer = D / 32, kBatch = kFew ? 8 : 4;
  griddep_launch_dependents();
  griddep_wait();
  __shared__ float acc_s[kFew ? 8 : 1][D], sum_s[8], max_s[8];
  __shared__ int first_s;
  int first = blockIdx.x;
  if (kFew) {
    if (threadIdx.x == 0) first_s = -1;
    __syncthreads();
    for (int c = threadIdx.x; c < ctas; c += 256) {
      const int4 i = p.seg_info[c];
      if (i.z > 0 && static_cast<int64_t>(i.x) * p.kv_heads + i.y == blockIdx.x) first_s = c;
    }
    __syncthreads();
    first = first_s;
    if (first < 0) return;
  }
  const int4 info = p.seg_info[first];
  const int parts = info.z + 1;
  if (parts == 1) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  constexpr int shares = kFew ? 8 : 1;  // warps per head
  const int h = kFew ? blockIdx.y : blockIdx.y * 8 + warp;
  const int i0 = kFew ? warp : 0;
  const int n = h < p.group && i0 < parts ? (parts - i0 + shares - 1) / shares : 0;  // partials of this warp
  auto slot = [&](int k) {
    const int i = i0 + k * shares;
    return (i == 0 ? 2 * first + 1 : 2 * (first + i)) * p.group + h;  // below 2^20: two partials an SM, 128 heads
  };
  float m = kUnset, l = 0.f, acc[kPer];
#pragma unroll
  for (int j = 0; j < kPer; ++j) acc[j] = 0.f;
#pragma unroll 1
  for (int base = 0; base < n; base += 32) {
    const int count = min(32, n - base);
    float2 ml = make_float2(kUnset, 0.f);
    if (lane < count) ml = p.part_ml[slot(base + lane)];
    float w = 0.f;
#pragma unroll 1
    for (int k0 = 0; k0 < count; k0 += kBatch) {
      using Vec = typename std::conditional<kPer == 4, float4, float2>::type;
      union {
        Vec v;
        float f[kPer];
      } x[kBatch];
#pragma unroll
      for (int k = 0; k < kBatch; ++k)
        if (k0 + k < count) x[k].v = *reinterpret_cast<const Vec*>(p.part_o + slot(base + k0 + k) * D + lane * kPer);
      if (k0 == 0) {
        float top = ml.x;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        const float now = fmaxf(m, top), old = ex2(m - now);
        w = ex2(ml.x - now);
        float sum = lane < count ? w * ml.y : 0.f;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        l = fmaf(l, old, sum);
#pragma unroll
        for (int j = 0; j < kPer; ++j) acc[j] *= old;
        m = now;
      }
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        const float wk = __shfl_sync(0xffffffffu, w, k0 + k);
        if (k0 + k < count)
#pragma unroll
          for (int j = 0; j < kPer; ++j) acc[j] = fmaf(x[k].f[j], wk, acc[j]);
      }
    }
  }
  if (kFew) {
#pragma unroll
    for (int j = 0; j < kPer; ++j) acc_s[warp][lane * kPer + j] = acc[j];
    if (lane == 0) {
      sum_s[warp] = l;
      max_s[warp] = m;
    }
    __syncthreads();
    if (warp != 0) return;
    m = max_s[0];
    for (int w = 1; w < 8; ++w) m = fmaxf(m, max_s[w]);
    l = 0.f;
#pragma unroll
    for (int j = 0; j < kPer; ++j) acc[j] = 0.f;
    for (int w = 0; w < 8; ++w) {
      const float wk = ex2(max_s[w] - m);
      l = fmaf(sum_s[w], wk, l);
#pragma unroll
      for (int j = 0; j < kPer; ++j) acc[j] = fmaf(acc_s[w][lane * kPer + j], wk, acc[j]);
    }
  }
  if (h >= p.group) return;
  const float inv = l == 0.f ? 0.f : __fdividef(1.f, l);
  const int64_t out_row = (static_cast<int64_t>(info.x) * p.kv_heads + info.y) * p.group + h;
#pragma unroll
  for (int j = 0; j < kPer; j += 2)
    *reinterpret_cast<uint32_t*>(p.out + out_row * D + lane * kPer + j) = bf16x2(acc[j] * inv, acc[j + 1] * inv);
  if (p.lse && lane == 0) p.lse[out_row] = (m + lg2(l)) * 0.69314718055994531f;
}

namespace {

template <typename K, typename... A>
cudaError_t launch(K kernel, dim3 grid, int threads, size_t smem, cudaStream_t stream, A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// Calls f with the kernel of a geometry and its shape.
template <typename F>
cudaError_t with_kernel(int head_dim, bool e4m3, int group, F f) {
#define SMQ_ATTN(D, E, N) return f(attention_kernel<D, E, N>, Shape<D, E, N>())
#define SMQ_ATTN_GROUPS(D, E)         \
  if (group <= 16) SMQ_ATTN(D, E, 16); \
  if (group <= 32) SMQ_ATTN(D, E, 32); \
  if (group <= 64) SMQ_ATTN(D, E, 64); \
  SMQ_ATTN(D, E, 128)
  if (head_dim == 128) {
    if (e4m3) {
      SMQ_ATTN_GROUPS(128, true);
    }
    SMQ_ATTN_GROUPS(128, false);
  }
  if (e4m3) {
    SMQ_ATTN_GROUPS(64, true);
  }
  SMQ_ATTN_GROUPS(64, false);
#undef SMQ_ATTN_GROUPS
#undef SMQ_ATTN
}

}  // namespace

cudaError_t prepare_attention(int head_dim, bool e4m3, int group) {
  return with_kernel(head_dim, e4m3, group, [](auto kernel, auto shape) {
    // the register split waits for ever on a launch with fewer registers than it hands out
    cudaFuncAttributes a;
    const cudaError_t rc = cudaFuncGetAttributes(&a, kernel);
    if (rc != cudaSuccess) return rc;
    if (a.numRegs != decltype(shape)::kRegs) return cudaErrorInvalidKernelImage;
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, decltype(shape)::kSmem);
  });
}

cudaError_t launch_attention(const AttnParams& p, bool e4m3, int grid, cudaStream_t stream) {
  cudaError_t rc = with_kernel(p.head_dim, e4m3, p.group, [&](auto kernel, auto shape) {
    return launch(kernel, dim3(grid), decltype(shape)::kThreads, decltype(shape)::kSmem, stream, p);
  });
  if (rc != cudaSuccess) return rc;
  // no row is shared where the tile list is cut between items only
  const int64_t tiles = ((p.token_ids ? p.num_ids : static_cast<int64_t>(p.bt_stride) * p.page_size) + kAttnTile - 1) / kAttnTile;
  const int64_t chunk = (tiles * p.rows * p.kv_heads + grid - 1) / grid;
  if (tiles == 1 || (p.token_ids && chunk % tiles == 0)) return cudaSuccess;
  // few items: an item has many partials, shared by a CTA per head
  const int64_t items = static_cast<int64_t>(p.rows) * p.kv_heads;
  if (items * 4 < grid)
    return launch(p.head_dim == 128 ? combine_kernel<128, true> : combine_kernel<64, true>,
                  dim3(static_cast<unsigned>(items), p.group), 256, 0, stream, p, grid);
  return launch(p.head_dim == 128 ? combine_kernel<128, false> : combine_kernel<64, false>, dim3(grid, (p.group + 7) / 8), 256,
                0, stream, p, grid);
}

}  // namespace smq
