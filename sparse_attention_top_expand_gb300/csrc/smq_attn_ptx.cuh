// Arithmetic, copies, barriers and tcgen05 helpers that the attention kernels
// share (smq_attn.cu, smq_seq_attn.cu). Device code only.
#pragma once

#include "smq_ptx.cuh"

#include <cuda_bf16.h>

#include <cstdint>

namespace smq {

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

__device__ __forceinline__ void lds16(uint32_t a, uint32_t* v) {
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]) : "r"(a) : "memory");
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

// Quotients of what is nearly always short: the 64-bit division is a long routine.
__device__ __forceinline__ long long div_of(long long a, long long b) {
  if (((a | b) >> 32) == 0) return static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
  return a / b;
}

}  // namespace smq
