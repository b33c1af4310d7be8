// Host side of the page operators declared in include/smq.h: the plan, argument
// validation and the launches. Nothing here allocates device memory.
#include "smq.h"
#include "smq_kernels.cuh"
#include "smq_pages.cuh"

#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>
#include <cstring>
#include <new>

struct smq_page_plan {
  smq_page_plan_desc desc;
  int32_t num_sms;
};

namespace {

constexpr size_t kStatusBytes = 256;
constexpr int kMaxVectors = 1024;

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// Workspace: [status word, 256 B][free pages of each segment][takes or counts][free list][its
// pages as bits][sources' entries of a fork].
struct Scratch {
  size_t free_counts, takes, free_list, free_bits, snapshot, end;
  int64_t segment, segments;
};

Scratch scratch_of(const smq_page_plan* p) {
  auto up = [](size_t x) { return (x + 255) / 256 * 256; };
  const int64_t entries = static_cast<int64_t>(p->desc.table_rows) * p->desc.table_columns;
  Scratch s;
  // Segments of 4096 pages, or longer ones so that there are no more than kMaxSegments. A batch of 512 rows that turns over in a
  // pool of 524288 pages takes 22 us, and two calls that fill and empty its table 33; with 2048 pages a segment 23 and 30, with
  // 8192 the two calls 37, with 16384 42.
  const int64_t units = (p->desc.num_pages + smq::kSegmentUnit - 1) / smq::kSegmentUnit;
  const int64_t per = (units + smq::kMaxSegments - 1) / smq::kMaxSegments;
  s.segment = (per < 2 ? 2 : per) * smq::kSegmentUnit;
  s.segments = (p->desc.num_pages + s.segment - 1) / s.segment;
  s.free_counts = kStatusBytes;
  s.takes = s.free_counts + up(smq::kMaxSegments * sizeof(int32_t));
  s.free_list = s.takes + up(p->desc.table_rows * sizeof(int32_t));
  s.free_bits = s.free_list + up(s.segments * s.segment * sizeof(int32_t));
  s.snapshot = s.free_bits + up(s.segments * s.segment / 8);
  s.end = s.snapshot + entries * sizeof(int32_t);
  return s;
}

int check_call(const smq_page_plan* p, int32_t num_rows, const void* workspace, size_t workspace_bytes) {
  if (num_rows < 0 || num_rows > p->desc.table_rows) return SMQ_ERR_INVALID_ARG;
  if (!workspace || !aligned(workspace, 16)) return SMQ_ERR_INVALID_ARG;
  return workspace_bytes < scratch_of(p).end ? SMQ_ERR_WORKSPACE_TOO_SMALL : SMQ_OK;
}

int check_device(const smq_page_plan* p) {
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess) return SMQ_ERR_CUDA;
  return dev == p->desc.device ? SMQ_OK : SMQ_ERR_INVALID_ARG;
}

int take_planes(const smq_page_plan* p, const smq_page_plane* from, int32_t count, smq::Planes* to) {
  if (count < 0 || count > SMQ_MAX_PLANES || (count > 0 && !from)) return SMQ_ERR_INVALID_ARG;
  std::memset(to, 0, sizeof *to);
  to->count = count;
  for (int i = 0; i < count; ++i) {
    const smq_page_plane& q = from[i];
    if (!q.base || !aligned(q.base, 4) || q.vectors <= 0 || q.token_bytes <= 0 || q.token_bytes % 4 != 0 || q.page_stride % 4 != 0)
      return SMQ_ERR_INVALID_ARG;
    if (q.vectors > kMaxVectors || q.token_bytes > smq::kMaxTokenBytes) return SMQ_ERR_UNSUPPORTED;
    if (q.page_stride < static_cast<int64_t>(q.vectors) * p->desc.page_size * q.token_bytes) return SMQ_ERR_INVALID_ARG;
    to->plane[i] = q;
  }
  return SMQ_OK;
}

// Whether two planes share bytes of some page: one thing listed twice, or slices that overlap. Views of one allocation have one
// page stride.
bool share_bytes(const smq_page_plan* p, const smq_page_plane& x, const smq_page_plane& y) {
  const bool first = reinterpret_cast<uintptr_t>(x.base) <= reinterpret_cast<uintptr_t>(y.base);
  const smq_page_plane &a = first ? x : y, &b = first ? y : x;
  const uint64_t apart = reinterpret_cast<uintptr_t>(b.base) - reinterpret_cast<uintptr_t>(a.base);
  if (a.page_stride != b.page_stride) return apart == 0;
  auto size = [&](const smq_page_plane& q) { return static_cast<uint64_t>(q.vectors) * p->desc.page_size * q.token_bytes; };
  const uint64_t stride = a.page_stride, at = apart % stride;
  if (apart >= stride * (p->desc.num_pages - 1) + size(a)) return false;  // b begins behind a's last page
  return at < size(a) || at + size(b) > stride;
}

smq::PagesParams params_of(const smq_page_plan* plan, int32_t num_rows, int32_t* table, int32_t* refs, void* workspace) {
  const smq_page_plan_desc& d = plan->desc;
  const Scratch w = scratch_of(plan);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  smq::PagesParams p;
  std::memset(&p, 0, sizeof p);
  p.num_rows = num_rows;
  p.table_rows = d.table_rows;
  p.columns = d.table_columns;
  p.page_size = d.page_size;
  p.num_pages = static_cast<int32_t>(d.num_pages);
  p.table = table;
  p.refs = refs;
  p.status = reinterpret_cast<int32_t*>(ws);
  p.segment = static_cast<int32_t>(w.segment);
  p.segments = static_cast<int32_t>(w.segments);
  p.free_counts = reinterpret_cast<int32_t*>(ws + w.free_counts);
  p.takes = reinterpret_cast<int32_t*>(ws + w.takes);
  p.free_list = reinterpret_cast<int32_t*>(ws + w.free_list);
  p.free_bits = reinterpret_cast<uint32_t*>(ws + w.free_bits);
  p.snapshot = reinterpret_cast<int32_t*>(ws + w.snapshot);
  return p;
}

}  // namespace

extern "C" {

SMQ_API int smq_page_plan_create(const smq_page_plan_desc* desc, smq_page_plan** plan) {
  if (!desc || !plan || desc->struct_size < sizeof(smq_page_plan_desc)) return SMQ_ERR_INVALID_ARG;
  *plan = nullptr;
  const smq_page_plan_desc& d = *desc;
  if (d.page_size <= 0 || d.num_pages <= 0 || d.table_rows <= 0 || d.table_columns <= 0 || d.device < 0)
    return SMQ_ERR_INVALID_ARG;
  if (d.page_size > 65536 || d.num_pages > INT32_MAX || d.table_rows > smq::kMaxRowsPerCall || d.table_columns > (1 << 20) ||
      static_cast<int64_t>(d.table_rows) * d.table_columns > INT32_MAX)
    return SMQ_ERR_UNSUPPORTED;
  int count = 0;
  if (cudaGetDeviceCount(&count) != cudaSuccess || d.device >= count) return SMQ_ERR_CUDA;
  int major = 0, minor = 0, sms = 0;
  if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, d.device) != cudaSuccess ||
      cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, d.device) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, d.device) != cudaSuccess)
    return SMQ_ERR_CUDA;
  if (major != 10 || minor != 3) return SMQ_ERR_UNSUPPORTED;  // built for sm_103a only
  smq_page_plan* p = new (std::nothrow) smq_page_plan;
  if (!p) return SMQ_ERR_INVALID_ARG;
  p->desc = d;
  p->num_sms = sms;
  *plan = p;
  return SMQ_OK;
}

SMQ_API int smq_page_plan_destroy(smq_page_plan* plan) {
  delete plan;
  return SMQ_OK;
}

SMQ_API int smq_page_workspace_size(const smq_page_plan* plan, size_t* bytes) {
  if (!plan || !bytes) return SMQ_ERR_INVALID_ARG;
  *bytes = scratch_of(plan).end;
  return SMQ_OK;
}

SMQ_API int smq_page_workspace_init(const smq_page_plan* plan, void* workspace, size_t workspace_bytes, void* stream) {
  if (!plan || !workspace || workspace_bytes < kStatusBytes) return SMQ_ERR_INVALID_ARG;
  return cudaMemsetAsync(workspace, 0, kStatusBytes, static_cast<cudaStream_t>(stream)) == cudaSuccess ? SMQ_OK
                                                                                                       : SMQ_ERR_CUDA;
}

SMQ_API int sparse_mqa_pages_resize(const smq_page_plan* plan, const smq_pages_resize_args* args, void* stream) {
  if (!plan || !args || args->struct_size < sizeof(smq_pages_resize_args)) return SMQ_ERR_INVALID_ARG;
  const smq_pages_resize_args& a = *args;
  int rc = check_call(plan, a.num_rows, a.workspace, a.workspace_bytes);
  if (rc != SMQ_OK) return rc;
  if (a.num_rows == 0) return SMQ_OK;
  if (!a.block_table || !a.page_refs || !a.row_end || a.keep_first < 0 || !aligned(a.block_table, 4) ||
      !aligned(a.page_refs, 4) || !aligned(a.rows, 4) || !aligned(a.row_begin, 4) || !aligned(a.row_end, 4))
    return SMQ_ERR_INVALID_ARG;
  rc = check_device(plan);
  if (rc != SMQ_OK) return rc;
  smq::PagesParams p = params_of(plan, a.num_rows, a.block_table, a.page_refs, a.workspace);
  p.rows = a.rows;
  p.row_begin = a.row_begin;
  p.row_end = a.row_end;
  p.keep_first = a.keep_first;
  smq::Planes none = {};
  return smq::launch_pages(p, none, static_cast<cudaStream_t>(stream)) == cudaSuccess ? SMQ_OK : SMQ_ERR_CUDA;
}

SMQ_API int sparse_mqa_pages_fork(const smq_page_plan* plan, const smq_pages_fork_args* args, void* stream) {
  if (!plan || !args || args->struct_size < sizeof(smq_pages_fork_args)) return SMQ_ERR_INVALID_ARG;
  const smq_pages_fork_args& a = *args;
  int rc = check_call(plan, a.num_rows, a.workspace, a.workspace_bytes);
  if (rc != SMQ_OK) return rc;
  smq::Planes planes;
  rc = take_planes(plan, a.planes, a.num_planes, &planes);
  if (rc != SMQ_OK) return rc;
  if (a.num_rows == 0) return SMQ_OK;
  if (!a.block_table || !a.page_refs || !a.src_rows || !a.dst_rows || !a.row_len || !aligned(a.block_table, 4) ||
      !aligned(a.page_refs, 4) || !aligned(a.src_rows, 4) || !aligned(a.dst_rows, 4) || !aligned(a.row_len, 4))
    return SMQ_ERR_INVALID_ARG;
  rc = check_device(plan);
  if (rc != SMQ_OK) return rc;
  smq::PagesParams p = params_of(plan, a.num_rows, a.block_table, a.page_refs, a.workspace);
  p.rows = a.dst_rows;
  p.row_end = a.row_len;
  p.src_rows = a.src_rows;
  return smq::launch_pages(p, planes, static_cast<cudaStream_t>(stream)) == cudaSuccess ? SMQ_OK : SMQ_ERR_CUDA;
}

SMQ_API int sparse_mqa_cache_compact(const smq_page_plan* plan, const smq_cache_compact_args* args, void* stream) {
  if (!plan || !args || args->struct_size < sizeof(smq_cache_compact_args)) return SMQ_ERR_INVALID_ARG;
  const smq_cache_compact_args& a = *args;
  int rc = check_call(plan, a.num_rows, a.workspace, a.workspace_bytes);
  if (rc != SMQ_OK) return rc;
  smq::Planes planes;
  rc = take_planes(plan, a.planes, a.num_planes, &planes);
  if (rc != SMQ_OK) return rc;
  if (a.num_planes == 0 || a.num_keep <= 0 || a.num_keep > (1 << 20) || a.keep_ld < a.num_keep) return SMQ_ERR_INVALID_ARG;
  for (int i = 0; i < planes.count; ++i)
    for (int j = 0; j < i; ++j)
      if (share_bytes(plan, planes.plane[i], planes.plane[j])) return SMQ_ERR_INVALID_ARG;  // their tokens would move twice
  if (a.num_rows == 0) return SMQ_OK;
  if (!a.block_table || !a.page_refs || !a.row_start || !a.keep_ids || !aligned(a.block_table, 4) ||
      !aligned(a.page_refs, 4) || !aligned(a.rows, 4) || !aligned(a.row_start, 4) || !aligned(a.keep_ids, 4))
    return SMQ_ERR_INVALID_ARG;
  rc = check_device(plan);
  if (rc != SMQ_OK) return rc;
  const smq_page_plan_desc& d = plan->desc;
  smq::CompactParams p;
  std::memset(&p, 0, sizeof p);
  p.num_rows = a.num_rows;
  p.table_rows = d.table_rows;
  p.columns = d.table_columns;
  p.page_size = d.page_size;
  p.num_pages = static_cast<int32_t>(d.num_pages);
  p.num_keep = a.num_keep;
  p.keep_ld = a.keep_ld;
  p.table = a.block_table;
  p.refs = a.page_refs;
  p.rows = a.rows;
  p.row_start = a.row_start;
  p.keep_ids = a.keep_ids;
  p.status = static_cast<int32_t*>(a.workspace);
  p.counts = reinterpret_cast<int32_t*>(static_cast<uint8_t*>(a.workspace) + scratch_of(plan).takes);
  return smq::launch_compact(p, planes, plan->num_sms, static_cast<cudaStream_t>(stream)) == cudaSuccess ? SMQ_OK
                                                                                                         : SMQ_ERR_CUDA;
}

}  // extern "C"
