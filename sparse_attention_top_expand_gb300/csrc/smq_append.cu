// Rotate a step's queries and keys by their positions and write keys and
// values into the paged cache (sm_103a).
//
// One thread holds 16 elements of a head: the two halves of eight rotation
// pairs, or 16 consecutive elements where the head does not rotate, so a
// 128-wide head is 8 neighbouring lanes and its amax is three shuffles. A
// warp's lanes keep the cosines and sines of their pairs in registers and walk
// over the heads of one token (queries, then keys, then values): the table
// row is read once per warp, not once per head.
//
// The kernel moves bytes only (about 3 operations for every 4 bytes), so it is
// bound by DRAM for a chunk and by launch and load latency for a step: 4096
// tokens of 64 + 16 heads of 128 in bf16 take 32.6 us, 5.2 TB/s; 4093 tokens of
// 32 + 8 heads of 64 into an E4M3 cache 9.6 us (10.9 before the loads streamed;
// 14.5 with the next pass loaded ahead); 64 tokens 3.7 us; one token's call is
// the host's launch, 2.8 us.
// Rounding: products and sums round to fp32 one by one (no fused
// multiply-add), so a result does not depend on how the compiler contracts
// them; then once to bf16, or to E4M3 with scale amax / 448.
#include "smq_attn.cuh"
#include "smq_kernels.cuh"
#include "smq_ptx.cuh"

#include <cuda_bf16.h>

namespace smq {

namespace {

constexpr int kAppendThreads = 128;

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  uint16_t lo, hi;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
  return static_cast<uint32_t>(lo) | (static_cast<uint32_t>(hi) << 16);
}

}  // namespace

// Warps of token `t`: `parts` of them, each taking every parts-th group of
// 32 / kLanes heads.
template <int D, bool kE4m3>
__global__ void __launch_bounds__(kAppendThreads) append_kernel(const __grid_constant__ AppendParams p, int parts) {
  constexpr int kLanes = D / 16;           // lanes per head
  constexpr int kHeads = 32 / kLanes;      // heads per warp pass
  griddep_launch_dependents();
  griddep_wait();
  const int lane = threadIdx.x & 31, j = lane % kLanes, sub = lane / kLanes;
  const int64_t warp = (static_cast<int64_t>(blockIdx.x) * kAppendThreads + threadIdx.x) >> 5;
  const int64_t t = warp / parts;
  if (t >= p.rows) return;
  const int part = static_cast<int>(warp % parts);
  const int half = p.rot_dim / 2;
  const bool turns = j < p.rot_dim / 16;
  // first elements of this lane's two groups of eight
  const int e0 = turns && !p.interleaved ? 8 * j : 16 * j;
  const int e1 = turns && !p.interleaved ? half + 8 * j : 16 * j + 8;
  float c[8], s[8];
  if (p.rot_dim > 0) {
    const int64_t pos = p.positions[t];
    if (pos < 0 || pos >= p.num_positions) {
      if (lane == 0) atomicOr(p.status, kStatusBounds);
      return;
    }
    if (turns) {
      const float4* row = reinterpret_cast<const float4*>(p.cos_sin + pos * p.rot_dim + 8 * j);
      const float4* srow = reinterpret_cast<const float4*>(p.cos_sin + pos * p.rot_dim + half + 8 * j);
      const float4 c0 = row[0], c1 = row[1], s0 = srow[0], s1 = srow[1];
      c[0] = c0.x, c[1] = c0.y, c[2] = c0.z, c[3] = c0.w, c[4] = c1.x, c[5] = c1.y, c[6] = c1.z, c[7] = c1.w;
      s[0] = s0.x, s[1] = s0.y, s[2] = s0.z, s[3] = s0.w, s[4] = s1.x, s[5] = s1.y, s[6] = s1.z, s[7] = s1.w;
    }
  }
  int64_t slot = p.slot_mapping[t];
  int64_t page = 0;
  int32_t off = 0;
  if (slot >= 0) {
    page = slot / p.page_size;
    off = static_cast<int32_t>(slot - page * p.page_size);
    if (page >= p.num_pages) {
      if (lane == 0) atomicOr(p.status, kStatusBounds);
      slot = -1;
    }
  }
  const int nq = p.q ? p.heads : 0;
  const int total = nq + 2 * p.kv_heads;
  // every lane of the warp takes every pass, so that the shuffles are whole
  for (int h0 = part * kHeads; h0 < total; h0 += parts * kHeads) {
    const int vec = h0 + sub;
    const bool is_q = vec < nq, is_v = vec >= nq + p.kv_heads;
    const int head = is_q ? vec : is_v ? vec - nq - p.kv_heads : vec - nq;
    const bool live = vec < total && (is_q || slot >= 0);
    uint4 a = make_uint4(0, 0, 0, 0), b = a;
    if (live) {
      const uint16_t* src = (is_q ? p.q + t * p.q_stride : is_v ? p.v + t * p.v_stride : p.k + t * p.k_stride) +
                            static_cast<int64_t>(head) * D;
      a = __ldcs(reinterpret_cast<const uint4*>(src + e0));
      b = __ldcs(reinterpret_cast<const uint4*>(src + e1));
    }
    const uint32_t wa[4] = {a.x, a.y, a.z, a.w}, wb[4] = {b.x, b.y, b.z, b.w};
    float x[8], y[8];  // elements e0 .. e0 + 7 and e1 .. e1 + 7
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = bf16_lo(wa[i]), x[2 * i + 1] = bf16_hi(wa[i]);
      y[2 * i] = bf16_lo(wb[i]), y[2 * i + 1] = bf16_hi(wb[i]);
    }
    if (turns && !is_v) {
      if (p.interleaved) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float u = x[2 * i], w = x[2 * i + 1];
          x[2 * i] = __fsub_rn(__fmul_rn(u, c[i]), __fmul_rn(w, s[i]));
          x[2 * i + 1] = __fadd_rn(__fmul_rn(w, c[i]), __fmul_rn(u, s[i]));
          u = y[2 * i], w = y[2 * i + 1];
          y[2 * i] = __fsub_rn(__fmul_rn(u, c[i + 4]), __fmul_rn(w, s[i + 4]));
          y[2 * i + 1] = __fadd_rn(__fmul_rn(w, c[i + 4]), __fmul_rn(u, s[i + 4]));
        }
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float u = x[i], w = y[i];
          x[i] = __fsub_rn(__fmul_rn(u, c[i]), __fmul_rn(w, s[i]));
          y[i] = __fadd_rn(__fmul_rn(w, c[i]), __fmul_rn(u, s[i]));
        }
      }
    }
    if (!kE4m3 || is_q) {
      uint4 oa, ob;
      oa = make_uint4(bf16x2(x[0], x[1]), bf16x2(x[2], x[3]), bf16x2(x[4], x[5]), bf16x2(x[6], x[7]));
      ob = make_uint4(bf16x2(y[0], y[1]), bf16x2(y[2], y[3]), bf16x2(y[4], y[5]), bf16x2(y[6], y[7]));
      if (live) {
        uint16_t* dst;
        if (is_q) {
          dst = p.q_out + (t * p.heads + head) * D;
        } else {
          dst = static_cast<uint16_t*>(is_v ? p.v_cache : p.k_cache) + page * p.page_stride +
                (static_cast<int64_t>(head) * p.page_size + off) * D;
        }
        *reinterpret_cast<uint4*>(dst + e0) = oa;
        *reinterpret_cast<uint4*>(dst + e1) = ob;
      }
    }
    if (kE4m3) {
      float amax = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) amax = fmaxf(amax, fmaxf(fabsf(x[i]), fabsf(y[i])));
#pragma unroll
      for (int o = kLanes / 2; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
      if (live && !is_q) {
        const float scale = amax > 0.f ? __fdiv_rn(amax, 448.f) : 1.f;
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          w[i] = e4m3x4(__fdiv_rn(x[4 * i], scale), __fdiv_rn(x[4 * i + 1], scale), __fdiv_rn(x[4 * i + 2], scale),
                        __fdiv_rn(x[4 * i + 3], scale));
          w[i + 2] = e4m3x4(__fdiv_rn(y[4 * i], scale), __fdiv_rn(y[4 * i + 1], scale), __fdiv_rn(y[4 * i + 2], scale),
                            __fdiv_rn(y[4 * i + 3], scale));
        }
        uint8_t* dst = static_cast<uint8_t*>(is_v ? p.v_cache : p.k_cache) + page * p.page_stride +
                       (static_cast<int64_t>(head) * p.page_size + off) * D;
        *reinterpret_cast<uint2*>(dst + e0) = make_uint2(w[0], w[1]);
        *reinterpret_cast<uint2*>(dst + e1) = make_uint2(w[2], w[3]);
        if (j == 0)
          (is_v ? p.v_scales : p.k_scales)[page * p.scale_page_stride + static_cast<int64_t>(head) * p.page_size + off] =
              scale;
      }
    }
  }
}

cudaError_t launch_append(const AppendParams& p, int head_dim, bool e4m3, int num_sms, cudaStream_t stream) {
  const int per_pass = 32 / (head_dim / 16);
  const int passes = ((p.q ? p.heads : 0) + 2 * p.kv_heads + per_pass - 1) / per_pass;
  // A warp keeps the token's table row over its passes; with too few tokens to
  // fill the SMs the passes are spread over more warps instead, up to 16 warps
  // an SM (48 measured 31.6 against 32.3 us on the bf16 chunk, but 13.0 against
  // 10.9 on the 8-bit one, whose 72 registers let an SM hold 28 warps: it then
  // ran in two waves).
  int64_t parts = (static_cast<int64_t>(num_sms) * 16 + p.rows - 1) / p.rows;
  parts = parts < 1 ? 1 : parts > passes ? passes : parts;
  const int64_t warps = static_cast<int64_t>(p.rows) * parts;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>((warps + kAppendThreads / 32 - 1) / (kAppendThreads / 32)));
  cfg.blockDim = dim3(kAppendThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  auto kernel = head_dim == 128 ? (e4m3 ? append_kernel<128, true> : append_kernel<128, false>)
                                : (e4m3 ? append_kernel<64, true> : append_kernel<64, false>);
  return cudaLaunchKernelEx(&cfg, kernel, p, static_cast<int>(parts));
}

}  // namespace smq
