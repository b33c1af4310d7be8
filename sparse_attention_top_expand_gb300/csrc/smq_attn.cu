// Attention of query rows over a paged key-value cache (sm_103a).
#include "smq_attn.cuh"
#include "smq_kernels.cuh"
#include "smq_ptx.cuh"

#include <cuda_bf16.h>
#include <cuda_fp8.h>

namespace smq {

namespace {

constexpr int kAttnThreads = 128;

template <bool kE4m3>
__device__ __forceinline__ float load_element(const void* base, int64_t at) {
  if (kE4m3) {
    __nv_fp8_e4m3 v;
    v.__x = static_cast<const uint8_t*>(base)[at];
    return static_cast<float>(v);
  }
  return __uint_as_float(static_cast<uint32_t>(static_cast<const uint16_t*>(base)[at]) << 16);
}

// Position `pos` of the row's sequence as a page and an offset in it; false
// (and the status bit) where it has none.
__device__ __forceinline__ bool place_of(const AttnParams& p, int64_t table_row, int64_t pos, int64_t* page, int* off) {
  if (table_row < 0 || table_row >= p.bt_rows || pos / p.page_size >= p.bt_stride) {
    atomicOr(p.status, kStatusBounds);
    return false;
  }
  *page = p.block_table[table_row * p.bt_stride + pos / p.page_size];
  *off = static_cast<int>(pos % p.page_size);
  if (*page < 0 || *page >= p.num_pages) {
    atomicOr(p.status, kStatusBounds);
    return false;
  }
  return true;
}

}  // namespace

// One CTA per (row, query head). Each warp takes every fourth token with a
// running maximum and sum; the four joined at the end.
template <int D, bool kE4m3>
__global__ void __launch_bounds__(kAttnThreads) attention_kernel(const __grid_constant__ AttnParams p) {
  constexpr int kPer = D / 32;
  constexpr int kWarps = kAttnThreads / 32;
  griddep_launch_dependents();
  griddep_wait();
  __shared__ float acc_s[kWarps][D];
  __shared__ float max_s[kWarps], sum_s[kWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int row = blockIdx.x, head = blockIdx.y, kv = head / p.group, heads = p.kv_heads * p.group;
  const int64_t table_row = p.row_indices ? p.row_indices[row] : row;
  float q[kPer], acc[kPer];
  for (int i = 0; i < kPer; ++i) {
    q[i] = load_element<false>(p.q, row * p.q_stride + static_cast<int64_t>(head) * D + lane + 32 * i);
    acc[i] = 0.f;
  }
  int64_t first = 0, last = p.num_ids;
  if (!p.token_ids) {
    first = p.row_ks ? max(p.row_ks[row], 0) : 0;
    last = p.row_ke[row];
  }
  float m = -INFINITY, l = 0.f;
  for (int64_t t = first + warp; t < last; t += kWarps) {
    const int64_t pos = p.token_ids ? p.token_ids[static_cast<int64_t>(row) * p.ids_ld + t] : t;
    if (pos < 0) continue;
    int64_t page;
    int off;
    if (!place_of(p, table_row, pos, &page, &off)) continue;
    const int64_t in_page = static_cast<int64_t>(kv) * p.page_size + off;
    const int64_t at = page * p.page_stride + in_page * D + lane;
    float dot = 0.f;
    for (int i = 0; i < kPer; ++i) dot = fmaf(q[i], load_element<kE4m3>(p.k_cache, at + 32 * i), dot);
    for (int o = 16; o > 0; o >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
    if (kE4m3) dot *= p.k_scales[page * p.scale_page_stride + in_page];
    const float s = dot * p.scale_log2;
    const float m_new = fmaxf(m, s);
    const float old = exp2f(m - m_new), w = exp2f(s - m_new);
    l = l * old + w;
    const float wv = kE4m3 ? w * p.v_scales[page * p.scale_page_stride + in_page] : w;
    for (int i = 0; i < kPer; ++i) acc[i] = fmaf(acc[i], old, wv * load_element<kE4m3>(p.v_cache, at + 32 * i));
    m = m_new;
  }
  for (int i = 0; i < kPer; ++i) acc_s[warp][lane + 32 * i] = acc[i];
  if (lane == 0) max_s[warp] = m, sum_s[warp] = l;
  __syncthreads();
  float most = -INFINITY, total = 0.f;
  for (int w = 0; w < kWarps; ++w) most = fmaxf(most, max_s[w]);
  for (int w = 0; w < kWarps; ++w) total += sum_s[w] > 0.f || sum_s[w] != sum_s[w] ? sum_s[w] * exp2f(max_s[w] - most) : 0.f;
  const int64_t out_row = static_cast<int64_t>(row) * heads + head;
  for (int d = threadIdx.x; d < D; d += kAttnThreads) {
    float o = 0.f;
    for (int w = 0; w < kWarps; ++w)
      if (max_s[w] != -INFINITY) o += acc_s[w][d] * exp2f(max_s[w] - most);
    p.out[out_row * D + d] = __bfloat16_as_ushort(__float2bfloat16_rn(total != 0.f ? o / total : 0.f));
  }
  if (p.lse && threadIdx.x == 0) p.lse[out_row] = (most + log2f(total)) * 0.69314718055994531f;
}

cudaError_t launch_attention(const AttnParams& p, bool e4m3, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(p.rows, p.kv_heads * p.group);
  cfg.blockDim = dim3(kAttnThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  auto kernel = p.head_dim == 128 ? (e4m3 ? attention_kernel<128, true> : attention_kernel<128, false>)
                                  : (e4m3 ? attention_kernel<64, true> : attention_kernel<64, false>);
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

}  // namespace smq
