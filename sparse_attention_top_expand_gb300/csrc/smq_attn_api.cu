// Host side of the attention operators declared in include/smq.h: the plan,
// argument validation and the launches. Nothing here allocates device memory.
#include "smq.h"
#include "smq_attn.cuh"
#include "smq_kernels.cuh"

#include <cuda_runtime.h>

#include <cmath>
#include <cstddef>
#include <cstdint>
#include <cstring>
#include <new>

struct smq_attn_plan {
  smq_attn_plan_desc desc;
  int64_t wait_ns;     // every pipeline wait gives up after this
  int32_t stall_tile;  // failure-path tests: a withheld hand-off, -1: none
  int32_t num_sms;
  float scale;
  bool prepared;
};

namespace {

constexpr size_t kStatusBytes = 256;

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// Workspace: [status word, 256 B][one int4 per CTA][maxima and sums][partial outputs], two partials per CTA.
struct Scratch {
  size_t info, ml, o, end;
};

Scratch scratch_of(const smq_attn_plan* p) {
  auto up = [](size_t x) { return (x + 255) / 256 * 256; };
  const size_t slots = 2 * static_cast<size_t>(p->num_sms);
  const size_t group = p->desc.num_heads / p->desc.num_kv_heads;
  Scratch s;
  s.info = kStatusBytes;
  s.ml = s.info + up(p->num_sms * sizeof(int4));
  s.o = s.ml + up(slots * group * sizeof(float2));
  s.end = s.o + slots * group * p->desc.head_dim * sizeof(float);
  return s;
}

int check_device(smq_attn_plan* p) {
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess) return SMQ_ERR_CUDA;
  if (dev != p->desc.device) return SMQ_ERR_INVALID_ARG;
  if (!p->prepared) {
    if (smq::prepare_attention(p->desc.head_dim, p->desc.cache_type == SMQ_CACHE_E4M3,
                               p->desc.num_heads / p->desc.num_kv_heads) != cudaSuccess)
      return SMQ_ERR_CUDA;
    p->prepared = true;
  }
  return SMQ_OK;
}

struct CacheArgs {
  const void* k;
  const void* v;
  const float* ks;
  const float* vs;
  int64_t num_pages, page_stride, scale_page_stride;
};

int check_cache(const smq_attn_plan* p, const CacheArgs& c) {
  const smq_attn_plan_desc& d = p->desc;
  const int64_t vectors = static_cast<int64_t>(d.num_kv_heads) * d.page_size;
  if (!c.k || !c.v || c.num_pages <= 0 || c.num_pages > INT32_MAX) return SMQ_ERR_INVALID_ARG;
  if (!aligned(c.k, 16) || !aligned(c.v, 16) || c.page_stride < vectors * d.head_dim || c.page_stride % 16 != 0)
    return SMQ_ERR_INVALID_ARG;
  if (d.cache_type == SMQ_CACHE_E4M3) {
    if (!c.ks || !c.vs || !aligned(c.ks, 4) || !aligned(c.vs, 4) || c.scale_page_stride < vectors)
      return SMQ_ERR_INVALID_ARG;
  } else if (c.ks || c.vs) {
    return SMQ_ERR_INVALID_ARG;  // a bfloat16 cache has no scales
  }
  return SMQ_OK;
}

bool strided_ok(const void* p, int64_t stride, int64_t row) { return p && aligned(p, 16) && stride % 8 == 0 && stride >= row; }

int run_attention(const smq_attn_plan* plan, const smq_attention_args* args, bool selected, void* stream) {
  if (!plan || !args || args->struct_size < sizeof(smq_attention_args)) return SMQ_ERR_INVALID_ARG;
  const smq_attention_args& a = *args;
  const smq_attn_plan_desc& d = plan->desc;
  if (a.rows < 0 || a.rows > d.max_rows) return SMQ_ERR_INVALID_ARG;
  if (a.rows == 0) return SMQ_OK;
  if (!strided_ok(a.q, a.q_stride, static_cast<int64_t>(d.num_heads) * d.head_dim)) return SMQ_ERR_INVALID_ARG;
  int rc = check_cache(plan, {a.k_cache, a.v_cache, a.k_scales, a.v_scales, a.num_pages, a.page_stride, a.scale_page_stride});
  if (rc != SMQ_OK) return rc;
  if (!a.block_table || !aligned(a.block_table, 4) || a.bt_rows <= 0 || a.bt_stride <= 0 || !aligned(a.row_indices, 4))
    return SMQ_ERR_INVALID_ARG;
  if (selected) {
    if (!a.token_ids || !aligned(a.token_ids, 4) || a.num_ids <= 0 || a.num_ids > (1 << 20) || a.ids_ld < a.num_ids ||
        a.row_ks || a.row_ke)
      return SMQ_ERR_INVALID_ARG;
  } else if (a.token_ids || !a.row_ke || !aligned(a.row_ke, 4) || !aligned(a.row_ks, 4)) {
    return SMQ_ERR_INVALID_ARG;
  }
  if (!a.out || !aligned(a.out, 16) || !aligned(a.lse, 4) || !a.workspace || !aligned(a.workspace, 16))
    return SMQ_ERR_INVALID_ARG;
  if (a.workspace_bytes < scratch_of(plan).end) return SMQ_ERR_WORKSPACE_TOO_SMALL;
  rc = check_device(const_cast<smq_attn_plan*>(plan));
  if (rc != SMQ_OK) return rc;
  smq::AttnParams p;
  std::memset(&p, 0, sizeof p);
  p.rows = a.rows;
  p.kv_heads = d.num_kv_heads;
  p.group = d.num_heads / d.num_kv_heads;
  p.head_dim = d.head_dim;
  p.page_size = d.page_size;
  p.page_shift = -1;
  for (int i = 0; i <= 16; ++i)
    if (d.page_size == 1 << i) p.page_shift = i;
  p.scale_log2 = plan->scale * 1.4426950408889634f;
  p.q = a.q;
  p.q_stride = a.q_stride;
  p.k_cache = a.k_cache;
  p.v_cache = a.v_cache;
  p.k_scales = a.k_scales;
  p.v_scales = a.v_scales;
  p.num_pages = a.num_pages;
  p.page_stride = a.page_stride;
  p.scale_page_stride = a.scale_page_stride;
  p.block_table = a.block_table;
  p.bt_rows = a.bt_rows;
  p.bt_stride = a.bt_stride;
  p.row_indices = a.row_indices;
  p.row_ks = a.row_ks;
  p.row_ke = a.row_ke;
  p.token_ids = a.token_ids;
  p.num_ids = a.num_ids;
  p.ids_ld = a.ids_ld;
  p.out = a.out;
  p.lse = a.lse;
  const Scratch w = scratch_of(plan);
  uint8_t* ws = static_cast<uint8_t*>(a.workspace);
  p.seg_info = reinterpret_cast<int4*>(ws + w.info);
  p.part_ml = reinterpret_cast<float2*>(ws + w.ml);
  p.part_o = reinterpret_cast<float*>(ws + w.o);
  p.status = static_cast<int32_t*>(a.workspace);
  p.wait_ns = plan->wait_ns;
  p.stall_tile = plan->stall_tile;
  return smq::launch_attention(p, d.cache_type == SMQ_CACHE_E4M3, plan->num_sms, static_cast<cudaStream_t>(stream)) == cudaSuccess
             ? SMQ_OK
             : SMQ_ERR_CUDA;
}

}  // namespace

extern "C" {

SMQ_API int smq_attn_plan_create(const smq_attn_plan_desc* desc, smq_attn_plan** plan) {
  if (!desc || !plan || desc->struct_size < sizeof(smq_attn_plan_desc)) return SMQ_ERR_INVALID_ARG;
  *plan = nullptr;
  const smq_attn_plan_desc& d = *desc;
  if (d.num_heads <= 0 || d.num_kv_heads <= 0 || d.num_heads % d.num_kv_heads != 0 || d.page_size <= 0 ||
      d.max_rows <= 0 || d.device < 0 || !std::isfinite(d.softmax_scale))
    return SMQ_ERR_INVALID_ARG;
  if (d.cache_type != SMQ_CACHE_BF16 && d.cache_type != SMQ_CACHE_E4M3) return SMQ_ERR_INVALID_ARG;
  if ((d.head_dim != 64 && d.head_dim != 128) || d.num_heads > 1024 || d.num_kv_heads > 128 ||
      d.num_heads / d.num_kv_heads > 128 || d.page_size > 65536 || d.max_rows > smq::kMaxRowsPerCall)
    return SMQ_ERR_UNSUPPORTED;
  int count = 0;
  if (cudaGetDeviceCount(&count) != cudaSuccess || d.device >= count) return SMQ_ERR_CUDA;
  int major = 0, minor = 0, sms = 0;
  if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, d.device) != cudaSuccess ||
      cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, d.device) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, d.device) != cudaSuccess)
    return SMQ_ERR_CUDA;
  if (major != 10 || minor != 3) return SMQ_ERR_UNSUPPORTED;  // built for sm_103a only
  smq_attn_plan* p = new (std::nothrow) smq_attn_plan;
  if (!p) return SMQ_ERR_INVALID_ARG;
  p->desc = d;
  p->wait_ns = 2000000000ll;  // 2 s: far beyond any legitimate wait
  p->stall_tile = -1;
  p->num_sms = sms;
  p->prepared = false;
  p->scale = d.softmax_scale != 0.f ? d.softmax_scale : 1.f / std::sqrt(static_cast<float>(d.head_dim));
  *plan = p;
  return SMQ_OK;
}

SMQ_API int smq_attn_plan_destroy(smq_attn_plan* plan) {
  delete plan;
  return SMQ_OK;
}

SMQ_API int smq_attn_plan_set_wait_limit(smq_attn_plan* plan, int64_t ns) {
  if (!plan || ns <= 0) return SMQ_ERR_INVALID_ARG;
  plan->wait_ns = ns;
  return SMQ_OK;
}

SMQ_API int smq_attn_plan_inject_stall(smq_attn_plan* plan, int32_t tile) {
  if (!plan || tile < -1) return SMQ_ERR_INVALID_ARG;
  plan->stall_tile = tile;
  return SMQ_OK;
}

SMQ_API int smq_attn_workspace_size(const smq_attn_plan* plan, size_t* bytes) {
  if (!plan || !bytes) return SMQ_ERR_INVALID_ARG;
  *bytes = scratch_of(plan).end;
  return SMQ_OK;
}

SMQ_API int smq_attn_workspace_init(const smq_attn_plan* plan, void* workspace, size_t workspace_bytes, void* stream) {
  if (!plan || !workspace || workspace_bytes < kStatusBytes) return SMQ_ERR_INVALID_ARG;
  return cudaMemsetAsync(workspace, 0, kStatusBytes, static_cast<cudaStream_t>(stream)) == cudaSuccess ? SMQ_OK
                                                                                                       : SMQ_ERR_CUDA;
}

SMQ_API int sparse_mqa_append_kv(const smq_attn_plan* plan, const smq_append_args* args, void* stream) {
  if (!plan || !args || args->struct_size < sizeof(smq_append_args)) return SMQ_ERR_INVALID_ARG;
  const smq_append_args& a = *args;
  const smq_attn_plan_desc& d = plan->desc;
  if (a.rows < 0 || a.rows > d.max_rows) return SMQ_ERR_INVALID_ARG;
  if (a.rows == 0) return SMQ_OK;
  const int64_t kv_row = static_cast<int64_t>(d.num_kv_heads) * d.head_dim;
  if (!strided_ok(a.k, a.k_stride, kv_row) || !strided_ok(a.v, a.v_stride, kv_row)) return SMQ_ERR_INVALID_ARG;
  if ((a.q == nullptr) != (a.q_out == nullptr)) return SMQ_ERR_INVALID_ARG;
  if (a.q && (!strided_ok(a.q, a.q_stride, static_cast<int64_t>(d.num_heads) * d.head_dim) || !aligned(a.q_out, 16)))
    return SMQ_ERR_INVALID_ARG;
  if (a.rot_dim < 0 || a.rot_dim > d.head_dim || a.rot_dim % 16 != 0) return SMQ_ERR_INVALID_ARG;
  if (a.rot_dim > 0 &&
      (!a.positions || !a.cos_sin || !aligned(a.positions, 8) || !aligned(a.cos_sin, 16) || a.num_positions <= 0))
    return SMQ_ERR_INVALID_ARG;
  if (!a.slot_mapping || !aligned(a.slot_mapping, 8)) return SMQ_ERR_INVALID_ARG;
  int rc = check_cache(plan, {a.k_cache, a.v_cache, a.k_scales, a.v_scales, a.num_pages, a.page_stride, a.scale_page_stride});
  if (rc != SMQ_OK) return rc;
  if (!a.workspace || !aligned(a.workspace, 16)) return SMQ_ERR_INVALID_ARG;
  if (a.workspace_bytes < kStatusBytes) return SMQ_ERR_WORKSPACE_TOO_SMALL;
  rc = check_device(const_cast<smq_attn_plan*>(plan));
  if (rc != SMQ_OK) return rc;
  smq::AppendParams p;
  std::memset(&p, 0, sizeof p);
  p.rows = a.rows;
  p.heads = d.num_heads;
  p.kv_heads = d.num_kv_heads;
  p.page_size = d.page_size;
  p.rot_dim = a.rot_dim;
  p.interleaved = a.interleaved ? 1 : 0;
  p.num_positions = a.num_positions;
  p.num_pages = a.num_pages;
  p.page_stride = a.page_stride;
  p.scale_page_stride = a.scale_page_stride;
  p.q = a.q;
  p.k = a.k;
  p.v = a.v;
  p.q_stride = a.q_stride;
  p.k_stride = a.k_stride;
  p.v_stride = a.v_stride;
  p.positions = a.positions;
  p.cos_sin = a.cos_sin;
  p.slot_mapping = a.slot_mapping;
  p.q_out = a.q_out;
  p.k_cache = a.k_cache;
  p.v_cache = a.v_cache;
  p.k_scales = a.k_scales;
  p.v_scales = a.v_scales;
  p.status = static_cast<int32_t*>(a.workspace);
  return smq::launch_append(p, d.head_dim, d.cache_type == SMQ_CACHE_E4M3, plan->num_sms,
                            static_cast<cudaStream_t>(stream)) == cudaSuccess
             ? SMQ_OK
             : SMQ_ERR_CUDA;
}

SMQ_API int sparse_mqa_attention_decode(const smq_attn_plan* plan, const smq_attention_args* args, void* stream) {
  return run_attention(plan, args, false, stream);
}

SMQ_API int sparse_mqa_attention_selected(const smq_attn_plan* plan, const smq_attention_args* args, void* stream) {
  return run_attention(plan, args, true, stream);
}

}  // extern "C"
