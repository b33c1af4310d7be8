// Attention of sequences' query rows over a paged key-value cache (sm_103a): a
// sliding window with sinks, or a tree of drafted tokens.
//
// The simplest form: a block per (sequence, row, kv head), a warp per query
// head, one token after another with a running maximum and sum. Each lane holds
// D / 32 elements of the query, the token's key and value, and the result.
#include "smq_attn.cuh"
#include "smq_attn_ptx.cuh"
#include "smq_kernels.cuh"
#include "smq_ptx.cuh"

namespace smq {

namespace {

constexpr int kSimpleThreads = 128;

template <bool kE4m3>
__device__ __forceinline__ float element(const void* base, int64_t at) {
  if (kE4m3) {
    uint32_t lo, hi;
    widen4(static_cast<const uint8_t*>(base)[at], lo, hi);
    return __uint_as_float(lo << 16);
  }
  return __uint_as_float(static_cast<uint32_t>(static_cast<const uint16_t*>(base)[at]) << 16);
}

}  // namespace

template <int D, bool kE4m3>
__global__ void __launch_bounds__(kSimpleThreads) seq_attention_kernel(const __grid_constant__ SeqAttnParams p) {
  constexpr int kPer = D / 32;
  griddep_launch_dependents();
  griddep_wait();
  const int b = blockIdx.z, i = blockIdx.x, g = blockIdx.y;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int first = p.cu_rows[b], last = p.cu_rows[b + 1], n = last - first;
  if (first < 0 || last < first || last > p.rows || n > p.max_seq_rows) {
    if (threadIdx.x == 0) atomicOr(p.status, kStatusBounds);
    return;
  }
  if (i >= n) return;
  const int64_t length = p.seq_len[b], base = length - n, row = first + i;
  int table_row = p.seq_indices ? p.seq_indices[b] : b;
  if (table_row < 0 || table_row >= p.bt_rows) table_row = -1;
  // visible: [0, sinks) and [from, to), or the context and the mask's tokens
  const int64_t to = p.tree_mask ? length : base + i + 1;
  const int64_t from = p.tree_mask ? 0 : max(static_cast<int64_t>(0), to - p.window);
  for (int h = warp; h < p.group; h += kSimpleThreads / 32) {
    const int64_t head = static_cast<int64_t>(g) * p.group + h;
    float q[kPer], acc[kPer], m = -INFINITY, l = 0.f;
    for (int k = 0; k < kPer; ++k) {
      q[k] = element<false>(p.q + row * p.q_stride + head * D, lane * kPer + k);
      acc[k] = 0.f;
    }
    for (int64_t t = 0; t < to; ++t) {
      if (t >= p.sinks && t < from) t = from;
      if (p.tree_mask && t >= base) {
        const int j = static_cast<int>(t - base);
        if (!(p.tree_mask[row * p.mask_words + j / 32] >> (j % 32) & 1)) continue;
      }
      const int64_t col = t / p.page_size;
      int64_t page = -1;
      if (table_row >= 0 && col < p.bt_stride) page = p.block_table[static_cast<int64_t>(table_row) * p.bt_stride + col];
      if (page < 0 || page >= p.num_pages) {
        if (lane == 0) atomicOr(p.status, kStatusBounds);
        if (table_row < 0 || col >= p.bt_stride) break;
        continue;
      }
      const int64_t vec = static_cast<int64_t>(g) * p.page_size + t % p.page_size;
      const int64_t at = page * p.page_stride + vec * D + lane * kPer;
      float s = 0.f, v[kPer];
      for (int k = 0; k < kPer; ++k) s = fmaf(q[k], element<kE4m3>(p.k_cache, at + k), s);
      for (int k = 0; k < kPer; ++k) v[k] = element<kE4m3>(p.v_cache, at + k);
      for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
      if (kE4m3) {
        s *= p.k_scales[page * p.scale_page_stride + vec];
        const float vs = p.v_scales[page * p.scale_page_stride + vec];
        for (int k = 0; k < kPer; ++k) v[k] *= vs;
      }
      s *= p.scale_log2;
      const float now = fmaxf(m, s), ref = now == -INFINITY ? 0.f : now;
      const float old = ex2(m - ref), w = ex2(s - ref);
      m = now;
      l = l * old + w;
      for (int k = 0; k < kPer; ++k) acc[k] = acc[k] * old + w * v[k];
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
    for (int k = 0; k < kPer; k += 2)
      *reinterpret_cast<uint32_t*>(p.out + (row * p.kv_heads * p.group + head) * D + lane * kPer + k) =
          bf16x2(acc[k] * inv, acc[k + 1] * inv);
    if (p.lse && lane == 0) p.lse[row * p.kv_heads * p.group + head] = l == 0.f ? -INFINITY : (m + lg2(l)) * 0.69314718055994531f;
  }
}

cudaError_t launch_seq_attention(const SeqAttnParams& p, bool e4m3, int grid, cudaStream_t stream) {
  (void)grid;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(p.max_seq_rows, p.kv_heads, p.num_seqs);
  cfg.blockDim = dim3(kSimpleThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  auto kernel = p.head_dim == 128 ? (e4m3 ? seq_attention_kernel<128, true> : seq_attention_kernel<128, false>)
                                  : (e4m3 ? seq_attention_kernel<64, true> : seq_attention_kernel<64, false>);
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

}  // namespace smq
