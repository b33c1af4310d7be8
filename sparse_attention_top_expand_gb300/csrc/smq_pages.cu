// Pages of the paged caches (sm_103a): rows of the block table that take, share
// and give back pages, and the tokens that move between pages.
//
// State and result are counts and ids, so a call must not depend on timing. A
// call is two launches: pages_plan_kernel only reads (which pages are free, what
// each listed row takes), pages_apply_kernel writes. Ranks come from prefix
// sums in the order of rows and columns; counts change by atomic additions,
// whose order does not matter.
#include "smq_pages.cuh"

#include "smq_kernels.cuh"
#include "smq_ptx.cuh"

namespace smq {

namespace {

constexpr int kPlanThreads = 512;
constexpr int kScanCtas = 8;  // the cluster that looks for free pages
constexpr int kApplyThreads = 256;
constexpr int kCopyBytes = 16384;  // a fork's copy: vectors of a page that one block takes

// What row i of a resize is to hold: columns [lo, hi) and, below hi, [0, first).
struct Want {
  int32_t lo, hi, first;
  __device__ bool operator()(int32_t c) const { return c < hi && (c >= lo || c < first); }
};

__device__ __forceinline__ Want want_of(const PagesParams& p, int i, bool* past) {
  const int64_t cap = static_cast<int64_t>(p.columns) * p.page_size;
  int64_t begin = p.row_begin ? p.row_begin[i] : 0, end = p.row_end[i];
  *past = begin > cap || end > cap;
  begin = begin < 0 ? 0 : begin > cap ? cap : begin;
  end = end < 0 ? 0 : end > cap ? cap : end;
  const int64_t first = p.keep_first < end ? p.keep_first : end;
  Want w;
  w.lo = static_cast<int32_t>(begin / p.page_size);
  w.hi = static_cast<int32_t>((end + p.page_size - 1) / p.page_size);
  w.first = static_cast<int32_t>((first + p.page_size - 1) / p.page_size);
  return w;
}

// The length of fork i: whole pages, and tokens of the next one.
struct Length {
  int32_t full, rest;
};
__device__ __forceinline__ Length length_of(const PagesParams& p, int i, bool* past) {
  const int64_t cap = static_cast<int64_t>(p.columns) * p.page_size;
  int64_t n = p.row_end[i];
  *past = n > cap;
  n = n < 0 ? 0 : n > cap ? cap : n;
  Length l;
  l.full = static_cast<int32_t>(n / p.page_size);
  l.rest = static_cast<int32_t>(n % p.page_size);
  return l;
}

// Row i as listed is a row of the table that was not listed before. A warp's call.
__device__ __forceinline__ bool row_is_new(const int32_t* rows, int i, int32_t table_rows, int lane) {
  if (!rows) return i < table_rows;
  const int32_t row = rows[i];
  bool bad = row < 0 || row >= table_rows;
  for (int j = lane; j < i; j += 32) bad |= rows[j] == row;
  return !__any_sync(0xffffffffu, bad);
}

// Bits of the free ones among pages i .. i + 3.
__device__ __forceinline__ uint32_t free_bits(const PagesParams& p, bool wide, int64_t i) {
  uint32_t m = 0;
  if (wide && i + 4 <= p.num_pages) {
    const int4 v = *reinterpret_cast<const int4*>(p.refs + i);
    m = (v.x == 0) | (v.y == 0) << 1 | (v.z == 0) << 2 | (v.w == 0) << 3;
  } else {
    for (int k = 0; k < 4; ++k)
      if (i + k < p.num_pages && p.refs[i + k] == 0) m |= 1u << k;
  }
  return m;
}

// The free list: each warp of the cluster has a range of pages, counts the free
// ones, and writes them behind those of the warps before it.
__device__ __forceinline__ void list_free_pages(const PagesParams& p) {
  constexpr int kWarps = kPlanThreads / 32;
  __shared__ uint32_t warp_count[kWarps], cta_count;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, rank = static_cast<int>(cluster_ctarank());
  const int64_t per = ((static_cast<int64_t>(p.num_pages) + kScanCtas * kWarps - 1) / (kScanCtas * kWarps) + 127) / 128 * 128;
  const int64_t begin = (rank * kWarps + warp) * per;
  const int64_t end = begin + per < p.num_pages ? begin + per : p.num_pages;
  const bool wide = reinterpret_cast<uintptr_t>(p.refs) % 16 == 0;
  uint32_t n = 0;
#pragma unroll 8
  for (int64_t i = begin + lane * 4; i < end; i += 128) n += __popc(free_bits(p, wide, i));
  n = __reduce_add_sync(0xffffffffu, n);
  if (lane == 0) warp_count[warp] = n;
  __syncthreads();
  if (threadIdx.x == 0) {
    uint32_t all = 0;
    for (int w = 0; w < kWarps; ++w) all += warp_count[w];
    cta_count = all;
  }
  cluster_sync();
  int64_t at = 0, total = 0;
  for (int c = 0; c < kScanCtas; ++c) {
    const uint32_t v = ld_dsmem_u32(smem_addr(&cta_count), c);
    if (c < rank) at += v;
    total += v;
  }
  cluster_sync();  // the counts have been read before a CTA leaves
  for (int w = 0; w < warp; ++w) at += warp_count[w];
  if (rank == 0 && threadIdx.x == 0) *p.free_count = static_cast<int32_t>(total < p.free_cap ? total : p.free_cap);
#pragma unroll 4
  for (int64_t i0 = begin; i0 < end && at < p.free_cap; i0 += 128) {
    const int64_t i = i0 + lane * 4;
    uint32_t m = i < end ? free_bits(p, wide, i) : 0;
    uint32_t incl = __popc(m);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    int64_t to = at + incl - __popc(m);
    at += __shfl_sync(0xffffffffu, incl, 31);
    while (m) {
      if (to < p.free_cap) p.free_list[to] = static_cast<int32_t>(i + __ffs(m) - 1);
      ++to;
      m &= m - 1;
    }
  }
}

}  // namespace

// Reads only: the free pages (the first cluster), and for each listed row how
// many pages it takes (a warp each). A fork's sources are also copied, as its
// destinations may be sources of others.
template <bool kFork>
__global__ void __cluster_dims__(kScanCtas, 1, 1) __launch_bounds__(kPlanThreads)
    pages_plan_kernel(const __grid_constant__ PagesParams p) {
  griddep_launch_dependents();
  griddep_wait();
  if (blockIdx.x < kScanCtas) {
    list_free_pages(p);
    return;
  }
  const int lane = threadIdx.x & 31;
  const int i = (blockIdx.x - kScanCtas) * (kPlanThreads / 32) + (threadIdx.x >> 5);
  if (i >= p.num_rows) return;
  bool bad = !row_is_new(p.rows, i, p.table_rows, lane), past;
  const int32_t row = p.rows ? p.rows[i] : i;
  int takes = 0;
  if (kFork) {
    const int32_t src = p.src_rows[i];
    bad |= src < 0 || src >= p.table_rows;
    if (bad || src == row) {
      takes = -1;
    } else {
      const Length n = length_of(p, i, &past);
      bad = past;
      const int32_t* from = p.table + static_cast<int64_t>(src) * p.columns;
      int32_t* to = p.snapshot + static_cast<int64_t>(i) * p.columns;
      const int32_t cols = n.full + (n.rest > 0);
#pragma unroll 4
      for (int32_t c = lane; c < cols; c += 32) {
        int32_t page = from[c];
        if (page >= 0 && (page >= p.num_pages || p.refs[page] <= 0)) {
          bad = true;
          page = -1;
        }
        to[c] = page < 0 ? -1 : page;
        if (c == n.full && page >= 0) takes = 1;
      }
      takes = __any_sync(0xffffffffu, takes);
    }
  } else if (bad) {
    takes = -1;
  } else {
    const Want want = want_of(p, i, &past);
    bad = past;
    const int32_t* from = p.table + static_cast<int64_t>(row) * p.columns;
#pragma unroll 4
    for (int32_t c = lane; c < want.hi; c += 32) takes += want(c) && from[c] < 0;
    takes = __reduce_add_sync(0xffffffffu, takes);
  }
  if (lane == 0) p.takes[i] = takes;
  if (bad) atomicOr(p.status, kStatusBounds);
}

namespace {

__device__ __forceinline__ void give_back(const PagesParams& p, int32_t page) {
  bool bad = page >= p.num_pages;
  if (!bad && atomicSub(p.refs + page, 1) <= 0) {
    atomicAdd(p.refs + page, 1);
    bad = true;
  }
  if (bad) atomicOr(p.status, kStatusBounds);
}

// Tokens [0, rest) of a page to another, one plane's vectors [v0, v1); a block's call.
template <typename T>
__device__ __forceinline__ void copy_tokens(const smq_page_plane& q, int32_t from, int32_t to, int page_size, int rest, int v0,
                                            int v1) {
  const int64_t run = static_cast<int64_t>(page_size) * q.token_bytes;
  const int n = static_cast<int>(static_cast<int64_t>(rest) * q.token_bytes / sizeof(T));
  const uint8_t* src = static_cast<const uint8_t*>(q.base) + from * q.page_stride + v0 * run;
  uint8_t* dst = static_cast<uint8_t*>(q.base) + to * q.page_stride + v0 * run;
  for (int v = v0; v < v1; ++v, src += run, dst += run) {
#pragma unroll 4
    for (int i = threadIdx.x; i < n; i += kApplyThreads) reinterpret_cast<T*>(dst)[i] = reinterpret_cast<const T*>(src)[i];
  }
}

struct CopyItems {
  int32_t first[SMQ_MAX_PLANES + 1];  // blocks of a fork's copy before each plane's
  int32_t vectors[SMQ_MAX_PLANES];    // vectors that a block takes
  bool wide[SMQ_MAX_PLANES];          // in pieces of 16 bytes
};

}  // namespace

// Blocks [0, row_blocks): a warp per listed row changes the table and the
// counts. The others copy the pages that forks have begun: a block per fork,
// plane and group of vectors.
template <bool kFork>
__global__ void __launch_bounds__(kApplyThreads)
    pages_apply_kernel(const __grid_constant__ PagesParams p, const __grid_constant__ Planes planes,
                       const __grid_constant__ CopyItems items, int row_blocks) {
  griddep_launch_dependents();
  griddep_wait();
  const int lane = threadIdx.x & 31;
  const int32_t nfree = *p.free_count;
  bool past;
  if (kFork && static_cast<int>(blockIdx.x) >= row_blocks) {
    const int per = items.first[planes.count];
    const int i = (blockIdx.x - row_blocks) / per, item = (blockIdx.x - row_blocks) % per;
    if (p.takes[i] <= 0) return;
    __shared__ int32_t warp_sum[kApplyThreads / 32];
    int32_t rank = 0;
    for (int j = threadIdx.x; j < i; j += kApplyThreads) rank += p.takes[j] > 0;
    rank = __reduce_add_sync(0xffffffffu, rank);
    if (lane == 0) warp_sum[threadIdx.x >> 5] = rank;
    __syncthreads();
    rank = 0;
    for (int w = 0; w < kApplyThreads / 32; ++w) rank += warp_sum[w];
    if (rank >= nfree) return;
    const Length n = length_of(p, i, &past);
    int k = 0;
    while (item >= items.first[k + 1]) ++k;
    const smq_page_plane& q = planes.plane[k];
    const int v0 = (item - items.first[k]) * items.vectors[k];
    const int v1 = v0 + items.vectors[k] < q.vectors ? v0 + items.vectors[k] : q.vectors;
    const int32_t from = p.snapshot[static_cast<int64_t>(i) * p.columns + n.full], to = p.free_list[rank];
    if (items.wide[k])
      copy_tokens<uint4>(q, from, to, p.page_size, n.rest, v0, v1);
    else
      copy_tokens<uint32_t>(q, from, to, p.page_size, n.rest, v0, v1);
    return;
  }
  const int i = blockIdx.x * (kApplyThreads / 32) + (threadIdx.x >> 5);
  if (i >= p.num_rows || p.takes[i] < 0) return;
  const int32_t row = p.rows ? p.rows[i] : i;
  int32_t base = 0;  // rank of the next page that this row takes
  for (int j = lane; j < i; j += 32) base += p.takes[j] > 0 ? p.takes[j] : 0;
  base = __reduce_add_sync(0xffffffffu, base);
  int32_t* const entries = p.table + static_cast<int64_t>(row) * p.columns;
  bool none = false;
  if (kFork) {
    const Length n = length_of(p, i, &past);
    const int32_t* const from = p.snapshot + static_cast<int64_t>(i) * p.columns;
#pragma unroll 4
    for (int32_t c = lane; c < p.columns; c += 32) {
      const int32_t old = entries[c];
      int32_t page = c < n.full || (c == n.full && n.rest > 0) ? from[c] : -1;
      if (c == n.full && page >= 0) {
        none = base >= nfree;
        page = none ? -1 : p.free_list[base];
      }
      entries[c] = page;
      if (page >= 0) atomicAdd(p.refs + page, 1);
      if (old >= 0) give_back(p, old);
    }
  } else {
    const Want want = want_of(p, i, &past);
#pragma unroll 4
    for (int32_t c0 = 0; c0 < p.columns; c0 += 32) {
      const int32_t c = c0 + lane;
      const int32_t old = c < p.columns ? entries[c] : -1;
      const bool take = want(c) && old < 0 && c < p.columns;
      const uint32_t ballot = __ballot_sync(0xffffffffu, take);
      if (take) {
        const int32_t r = base + __popc(ballot & ((1u << lane) - 1));
        if (r < nfree) {
          const int32_t page = p.free_list[r];
          entries[c] = page;
          atomicAdd(p.refs + page, 1);
        } else {
          none = true;
        }
      } else if (old >= 0 && !want(c)) {
        entries[c] = -1;
        give_back(p, old);
      }
      base += __popc(ballot);
    }
  }
  if (none) atomicOr(p.status, kStatusNoPages);
}

// ------------------------------------------------------------------- compact
//
// Tokens move in place towards the front: the j-th kept one, id k_j, to s + j,
// with k ascending and k_0 >= s, so k_j >= s + j. Chunks of consecutive j are
// moved in order, each read whole before it is written: place s + j can be the
// source of a k_i = s + j only with i <= j, so what a chunk overwrites belongs to
// itself or to chunks before it.

namespace {

constexpr int kMoveThreads = 256;
constexpr int kMovePieces = 8;        // of 16 or 4 bytes, per thread and chunk
constexpr int kMoveTokens = 256;      // most of a chunk
constexpr int kCheckThreads = 1024;
constexpr int kFusedKeep = 1024;      // longest list that every block checks for itself

struct MoveItems {
  int32_t first[SMQ_MAX_PLANES + 1];  // blocks of a row before each plane's
  int32_t vectors[SMQ_MAX_PLANES];    // vectors that a block takes
  bool wide[SMQ_MAX_PLANES];
};

// How many tokens row i moves, 0 where the list, a page or a count refuses it. All threads of a block.
template <int kThreads>
__device__ __forceinline__ int check_row(const CompactParams& p, int i) {
  __shared__ int first_end, first_bad;
  if (threadIdx.x == 0) {
    first_end = p.num_keep;
    first_bad = INT32_MAX;
  }
  __syncthreads();
  const int32_t row = p.rows ? p.rows[i] : i;
  bool bad_row = row < 0 || row >= p.table_rows;
  if (p.rows)
    for (int j = threadIdx.x; j < i; j += kThreads) bad_row |= p.rows[j] == row;
  bad_row = __syncthreads_or(bad_row);
  const int32_t start = p.row_start[i];
  if (!bad_row) {
    const int32_t* const ids = p.keep_ids + static_cast<int64_t>(i) * p.keep_ld;
    const int32_t* const entries = p.table + static_cast<int64_t>(row) * p.columns;
    int end = INT32_MAX, bad = INT32_MAX;
    for (int j = threadIdx.x; j < p.num_keep; j += kThreads) {
      const int32_t id = ids[j];
      if (id < 0) {
        end = min(end, j);
        break;
      }
      bool ok = start >= 0 && id - start >= j && (j == 0 || id > ids[j - 1]) && id / p.page_size < p.columns;
      if (ok) {  // (the place it moves to is not behind it)
        const int32_t a = entries[id / p.page_size], b = entries[(start + j) / p.page_size];
        ok = a >= 0 && a < p.num_pages && b >= 0 && b < p.num_pages && (id == start + j || p.refs[b] <= 1);
      }
      if (!ok) {
        bad = min(bad, j);
        break;
      }
    }
    if (end != INT32_MAX) atomicMin(&first_end, end);
    if (bad != INT32_MAX) atomicMin(&first_bad, bad);
  }
  __syncthreads();
  const bool refused = bad_row || first_bad < first_end;
  if (refused && threadIdx.x == 0) atomicOr(p.status, kStatusBounds);
  return refused ? 0 : first_end;
}

}  // namespace

__global__ void __launch_bounds__(kCheckThreads) compact_check_kernel(const __grid_constant__ CompactParams p) {
  griddep_launch_dependents();
  griddep_wait();
  const int n = check_row<kCheckThreads>(p, blockIdx.x);
  if (threadIdx.x == 0) p.counts[blockIdx.x] = n;
}

namespace {

template <typename T>
__device__ __forceinline__ void move_tokens(const CompactParams& p, const smq_page_plane& q, int i, int count, int v0, int v1,
                                            int64_t* src_s, int64_t* dst_s) {
  const int row = p.rows ? p.rows[i] : i;
  const int32_t start = p.row_start[i];
  const int32_t* const ids = p.keep_ids + static_cast<int64_t>(i) * p.keep_ld;
  const int32_t* const entries = p.table + static_cast<int64_t>(row) * p.columns;
  const int64_t run = static_cast<int64_t>(p.page_size) * q.token_bytes;
  const int per_vec = q.token_bytes / static_cast<int>(sizeof(T)), per_tok = per_vec * (v1 - v0);
  int chunk = kMoveThreads * kMovePieces / per_tok;
  chunk = chunk > kMoveTokens ? kMoveTokens : chunk;
  uint8_t* const base = static_cast<uint8_t*>(q.base) + v0 * run;
  for (int j0 = 0; j0 < count; j0 += chunk) {
    const int n = min(chunk, count - j0);
    if (static_cast<int>(threadIdx.x) < n) {
      const int32_t from = ids[j0 + threadIdx.x], to = start + j0 + static_cast<int>(threadIdx.x);
      const int32_t a = entries[from / p.page_size], b = entries[to / p.page_size];
      src_s[threadIdx.x] = from == to ? -1 : a * q.page_stride + static_cast<int64_t>(from % p.page_size) * q.token_bytes;
      dst_s[threadIdx.x] = b * q.page_stride + static_cast<int64_t>(to % p.page_size) * q.token_bytes;
    }
    __syncthreads();
    T got[kMovePieces];
    int64_t dst[kMovePieces];
#pragma unroll
    for (int k = 0; k < kMovePieces; ++k) {
      const int e = k * kMoveThreads + threadIdx.x;
      const int t = e / per_tok, w = e - t * per_tok;
      dst[k] = -1;
      if (t < n && src_s[t] >= 0) {
        const int v = w / per_vec;
        const int64_t at = v * run + static_cast<int64_t>(w - v * per_vec) * sizeof(T);
        got[k] = *reinterpret_cast<const T*>(base + src_s[t] + at);
        dst[k] = dst_s[t] + at;
      }
    }
    __syncthreads();  // the chunk has been read
#pragma unroll
    for (int k = 0; k < kMovePieces; ++k)
      if (dst[k] >= 0) *reinterpret_cast<T*>(base + dst[k]) = got[k];
  }
}

}  // namespace

// A block per listed row, plane and group of vectors.
template <bool kFused>
__global__ void __launch_bounds__(kMoveThreads)
    compact_kernel(const __grid_constant__ CompactParams p, const __grid_constant__ Planes planes,
                   const __grid_constant__ MoveItems items) {
  griddep_launch_dependents();
  griddep_wait();
  __shared__ int64_t src_s[kMoveTokens], dst_s[kMoveTokens];
  const int per = items.first[planes.count];
  const int i = blockIdx.x / per, item = blockIdx.x % per;
  const int count = kFused ? check_row<kMoveThreads>(p, i) : p.counts[i];
  if (count == 0) return;
  int k = 0;
  while (item >= items.first[k + 1]) ++k;
  const smq_page_plane& q = planes.plane[k];
  const int v0 = (item - items.first[k]) * items.vectors[k];
  const int v1 = v0 + items.vectors[k] < q.vectors ? v0 + items.vectors[k] : q.vectors;
  if (items.wide[k])
    move_tokens<uint4>(p, q, i, count, v0, v1, src_s, dst_s);
  else
    move_tokens<uint32_t>(p, q, i, count, v0, v1, src_s, dst_s);
}

namespace {

template <typename K, typename... A>
cudaError_t launch(K kernel, int64_t grid, int threads, cudaStream_t stream, A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(grid));
  cfg.blockDim = dim3(threads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

bool in_16(const smq_page_plane& q, int64_t a) {
  return reinterpret_cast<uintptr_t>(q.base) % 16 == 0 && q.page_stride % 16 == 0 && a % 16 == 0;
}

}  // namespace

cudaError_t launch_pages(const PagesParams& p, const Planes& planes, cudaStream_t stream) {
  const bool fork = p.src_rows != nullptr;
  const int per_cluster = kScanCtas * (kPlanThreads / 32);
  const int64_t plan_blocks = kScanCtas * (1 + (static_cast<int64_t>(p.num_rows) + per_cluster - 1) / per_cluster);
  cudaError_t rc = launch(fork ? pages_plan_kernel<true> : pages_plan_kernel<false>, plan_blocks, kPlanThreads, stream, p);
  if (rc != cudaSuccess) return rc;
  CopyItems items = {};
  for (int k = 0; k < planes.count; ++k) {
    const smq_page_plane& q = planes.plane[k];
    const int64_t run = static_cast<int64_t>(p.page_size) * q.token_bytes;
    int64_t v = kCopyBytes / run;
    v = v < 1 ? 1 : v > q.vectors ? q.vectors : v;
    items.vectors[k] = static_cast<int32_t>(v);
    items.first[k + 1] = items.first[k] + static_cast<int32_t>((q.vectors + v - 1) / v);
    items.wide[k] = in_16(q, q.token_bytes);
  }
  const int row_blocks = (p.num_rows + kApplyThreads / 32 - 1) / (kApplyThreads / 32);
  const int64_t blocks = row_blocks + static_cast<int64_t>(p.num_rows) * items.first[planes.count];
  return launch(fork ? pages_apply_kernel<true> : pages_apply_kernel<false>, blocks, kApplyThreads, stream, p, planes, items,
                row_blocks);
}

cudaError_t launch_compact(const CompactParams& p, const Planes& planes, int num_sms, cudaStream_t stream) {
  (void)num_sms;
  MoveItems items = {};
  for (int k = 0; k < planes.count; ++k) {
    const smq_page_plane& q = planes.plane[k];
    items.wide[k] = in_16(q, q.token_bytes);
    const int piece = items.wide[k] ? 16 : 4;
    // as many vectors as give a thread two pieces of the longest chunk
    int64_t v = 2ll * kMoveThreads * piece / (static_cast<int64_t>(kMoveTokens) * q.token_bytes);
    v = v < 1 ? 1 : v > q.vectors ? q.vectors : v;
    items.vectors[k] = static_cast<int32_t>(v);
    items.first[k + 1] = items.first[k] + static_cast<int32_t>((q.vectors + v - 1) / v);
  }
  const int64_t blocks = static_cast<int64_t>(p.num_rows) * items.first[planes.count];
  if (p.num_keep <= kFusedKeep) return launch(compact_kernel<true>, blocks, kMoveThreads, stream, p, planes, items);
  cudaError_t rc = launch(compact_check_kernel, p.num_rows, kCheckThreads, stream, p);
  if (rc != cudaSuccess) return rc;
  return launch(compact_kernel<false>, blocks, kMoveThreads, stream, p, planes, items);
}

}  // namespace smq
