// Pages of the paged caches (sm_103a): rows of the block table that take, share
// and give back pages, and the tokens that move between pages.
//
// State and result are counts and ids, so a call must not depend on timing, also
// where a table and its counts do not agree. A call is two launches.
// pages_plan_kernel finds which pages are free, as a list and as bits, and what
// each listed row takes, and counts the pages that forks share: a count above zero
// grows, so what is free does not change. pages_apply_kernel writes the rest. Ranks
// come from prefix sums in the order of rows and columns. Counts change by atomic
// operations whose order does not matter: pages that are taken were free, and a
// free page is not given back (its bit says so); of the others all additions
// come before all subtractions, which stop at zero. A row is a block's work in
// both: with a warp a row 512 rows of 2048 columns over 524288 pages took 74 us, so
// 21 to 22. Small calls are two launches, some 9 us.
#include "smq_pages.cuh"

#include "smq_kernels.cuh"
#include "smq_ptx.cuh"

namespace smq {

namespace {

constexpr int kPlanThreads = 512;
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

// The sum of v over a block of kThreads, to all of them. `scratch` holds a word a warp.
template <int kThreads>
__device__ __forceinline__ int block_sum(int v, int* scratch) {
  v = __reduce_add_sync(0xffffffffu, v);
  __syncthreads();  // the scratch of an earlier sum has been read
  if ((threadIdx.x & 31) == 0) scratch[threadIdx.x >> 5] = v;
  __syncthreads();
  v = 0;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) v += scratch[w];
  return v;
}

// The sum of v over the threads before this one, and over all of them.
template <int kThreads>
__device__ __forceinline__ int block_before(int v, int* scratch, int* total) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int incl = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += x;
  }
  __syncthreads();
  if (lane == 31) scratch[warp] = incl;
  __syncthreads();
  int before = incl - v;
  *total = 0;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) {
    if (w < warp) before += scratch[w];
    *total += scratch[w];
  }
  return before;
}

// Bits of the free ones among pages i .. i + 3, below end.
__device__ __forceinline__ uint32_t free_bits(const PagesParams& p, bool wide, int64_t i, int64_t end) {
  uint32_t m = 0;
  if (wide && i + 4 <= end) {
    const int4 v = *reinterpret_cast<const int4*>(p.refs + i);
    m = (v.x == 0) | (v.y == 0) << 1 | (v.z == 0) << 2 | (v.w == 0) << 3;
  } else {
    for (int k = 0; k < 4; ++k)
      if (i + k < end && p.refs[i + k] == 0) m |= 1u << k;
  }
  return m;
}

// The free pages of segment k of the pool, listed in order at the segment's place in the free list: each warp has a range,
// counts, and writes behind the warps before it.
__device__ __forceinline__ void list_free_pages(const PagesParams& p, int k) {
  constexpr int kWarps = kPlanThreads / 32;
  __shared__ int scratch[kWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t first = static_cast<int64_t>(k) * p.segment, per = p.segment / kWarps;  // a multiple of 128
  const int64_t limit = first + p.segment < p.num_pages ? first + p.segment : p.num_pages;
  const int64_t begin = first + warp * per, end = begin + per < limit ? begin + per : limit;
  const bool wide = reinterpret_cast<uintptr_t>(p.refs) % 16 == 0;
  int n = 0;
#pragma unroll 4
  for (int64_t i = begin + lane * 4; i < end; i += 128) n += __popc(free_bits(p, wide, i, end));
  n = __reduce_add_sync(0xffffffffu, n);
  if (lane == 0) scratch[warp] = n;
  __syncthreads();
  int32_t* to = p.free_list + first;
  int total = 0;
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) to += scratch[w];
    total += scratch[w];
  }
  if (threadIdx.x == 0) p.free_counts[k] = total;
  for (int64_t i0 = begin; i0 < end; i0 += 128) {
    const int64_t i = i0 + lane * 4;
    uint32_t m = i < end ? free_bits(p, wide, i, end) : 0;
    uint32_t word = m << (lane % 8 * 4);  // of eight lanes
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) word |= __shfl_xor_sync(0xffffffffu, word, o);
    if (lane % 8 == 0) p.free_bits[i / 32] = word;
    int incl = __popc(m);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    int32_t* at = to + incl - __popc(m);
    to += __shfl_sync(0xffffffffu, incl, 31);
    for (; m; m &= m - 1) *at++ = static_cast<int32_t>(i + __ffs(m) - 1);
  }
}

// The free list as one: pages by rank, over the segments' counts. All threads of a block make it.
struct FreeList {
  int32_t* before;  // [kMaxSegments] in shared memory: free pages of the segments before
  int segments, total;
  __device__ FreeList(const PagesParams& p, int32_t* smem, int* scratch) : before(smem), segments(p.segments) {
    int mine[kMaxSegments / kApplyThreads], sum = 0;
#pragma unroll
    for (int j = 0; j < kMaxSegments / kApplyThreads; ++j) {
      const int k = threadIdx.x * (kMaxSegments / kApplyThreads) + j;
      mine[j] = k < segments ? p.free_counts[k] : 0;
      sum += mine[j];
    }
    int at = block_before<kApplyThreads>(sum, scratch, &total);
#pragma unroll
    for (int j = 0; j < kMaxSegments / kApplyThreads; ++j) {
      before[threadIdx.x * (kMaxSegments / kApplyThreads) + j] = at;
      at += mine[j];
    }
    __syncthreads();
  }
  // the page of rank r, -1: there are not so many
  __device__ int32_t page(const PagesParams& p, int64_t r) const {
    if (r >= total) return -1;
    int lo = 0, hi = segments;  // before[lo] <= r < before[hi]
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (before[mid] <= r)
        lo = mid;
      else
        hi = mid;
    }
    return p.free_list[static_cast<int64_t>(lo) * p.segment + (r - before[lo])];
  }
};

}  // namespace

// Blocks [0, segments) list the free pages, the others say for a listed row each
// how many pages it takes. A fork's sources are also copied, as its destinations
// may be sources of others, and the whole pages that it shares are counted.
template <bool kFork>
__global__ void __launch_bounds__(kPlanThreads) pages_plan_kernel(const __grid_constant__ PagesParams p) {
  griddep_launch_dependents();
  griddep_wait();
  if (static_cast<int>(blockIdx.x) < p.segments) {
    list_free_pages(p, blockIdx.x);
    return;
  }
  const int i = blockIdx.x - p.segments;
  const int32_t row = p.rows ? p.rows[i] : i;
  bool bad = row < 0 || row >= p.table_rows, past;
  if (p.rows)
    for (int j = threadIdx.x; j < i; j += kPlanThreads) bad |= p.rows[j] == row;
  int32_t src = 0;
  if (kFork) {
    src = p.src_rows[i];
    bad |= src < 0 || src >= p.table_rows;
  }
  bad = __syncthreads_or(bad);
  int takes = 0;
  if (bad || (kFork && src == row)) {
    takes = -1;
  } else if (kFork) {
    const Length n = length_of(p, i, &past);
    bad = past;
    const int32_t* from = p.table + static_cast<int64_t>(src) * p.columns;
    int32_t* to = p.snapshot + static_cast<int64_t>(i) * p.columns;
    const int32_t cols = n.full + (n.rest > 0);
    bool take = false;
#pragma unroll 2
    for (int32_t c = threadIdx.x; c < cols; c += kPlanThreads) {
      int32_t page = from[c];
      if (page >= 0 && (page >= p.num_pages || p.refs[page] <= 0)) {
        bad = true;
        page = -1;
      }
      to[c] = page < 0 ? -1 : page;
      take |= c == n.full && page >= 0;
      if (c < n.full && page >= 0) atomicAdd(p.refs + page, 1);
    }
    takes = __syncthreads_or(take) ? 1 : 0;
  } else {
    __shared__ int scratch[kPlanThreads / 32];
    const Want want = want_of(p, i, &past);
    bad = past;
    const int32_t* from = p.table + static_cast<int64_t>(row) * p.columns;
#pragma unroll 4
    for (int32_t c = threadIdx.x; c < want.hi; c += kPlanThreads) takes += want(c) && from[c] < 0;
    takes = block_sum<kPlanThreads>(takes, scratch);
  }
  if (threadIdx.x == 0) p.takes[i] = takes;
  if (bad) atomicOr(p.status, kStatusBounds);
}

namespace {

__device__ __forceinline__ void give_back(const PagesParams& p, int32_t page) {
  bool bad = page >= p.num_pages || ((p.free_bits[page / 32] >> (page % 32)) & 1);  // nobody's page, that another row may take
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

// Blocks [0, num_rows) change the table and the counts, a listed row each. The
// others copy the pages that forks have begun: a block per fork, plane and group
// of vectors.
template <bool kFork>
__global__ void __launch_bounds__(kApplyThreads)
    pages_apply_kernel(const __grid_constant__ PagesParams p, const __grid_constant__ Planes planes,
                       const __grid_constant__ CopyItems items) {
  griddep_launch_dependents();
  griddep_wait();
  __shared__ int32_t before_s[kMaxSegments];
  __shared__ int scratch[kApplyThreads / 32];
  bool past;
  const int extra = static_cast<int>(blockIdx.x) - p.num_rows;  // of the copies
  const int per = kFork ? items.first[planes.count] : 0;
  const int i = kFork && extra >= 0 ? extra / per : blockIdx.x;
  const int takes = p.takes[i];
  if (takes < 0 || (kFork && extra >= 0 && takes == 0)) return;
  int64_t base = 0;  // rank of the row's first page
  int32_t fresh = -1;
  if (takes > 0) {
    int sum = 0;
    for (int j = threadIdx.x; j < i; j += kApplyThreads) sum += max(p.takes[j], 0);
    base = block_sum<kApplyThreads>(sum, scratch);
  }
  if (!kFork) {
    const FreeList list(p, before_s, scratch);
    const Want want = want_of(p, i, &past);
    int32_t* const entries = p.table + static_cast<int64_t>(p.rows ? p.rows[i] : i) * p.columns;
    bool none = false, bad = false;
    constexpr int kPer = 4;  // columns of a thread, next to each other so that ranks follow them
    for (int32_t c0 = 0; c0 < p.columns; c0 += kApplyThreads * kPer) {
      int32_t old[kPer];
      int n = 0;
#pragma unroll
      for (int k = 0; k < kPer; ++k) {
        const int32_t c = c0 + threadIdx.x * kPer + k;
        old[k] = c < p.columns ? entries[c] : -1;
        n += old[k] < 0 && c < p.columns && want(c);
      }
      int64_t r = base;
      if (takes > 0) {
        int all;
        r += block_before<kApplyThreads>(n, scratch, &all);
        base += all;
      }
#pragma unroll
      for (int k = 0; k < kPer; ++k) {
        const int32_t c = c0 + threadIdx.x * kPer + k;
        if (c >= p.columns) break;
        if (want(c)) {
          bad |= old[k] >= p.num_pages;
          if (old[k] >= 0) continue;
          const int32_t page = list.page(p, r++);
          none |= page < 0;
          if (page < 0) continue;
          entries[c] = page;
          atomicAdd(p.refs + page, 1);
        } else if (old[k] >= 0) {
          entries[c] = -1;
          give_back(p, old[k]);
        }
      }
    }
    if (none) atomicOr(p.status, kStatusNoPages);
    if (bad) atomicOr(p.status, kStatusBounds);
    return;
  }
  const Length n = length_of(p, i, &past);
  if (takes > 0) {
    const FreeList list(p, before_s, scratch);
    fresh = list.page(p, base);
  }
  const int32_t* const from = p.snapshot + static_cast<int64_t>(i) * p.columns;
  if (extra < 0) {
    int32_t* const entries = p.table + static_cast<int64_t>(p.rows[i]) * p.columns;
#pragma unroll 4
    for (int32_t c = threadIdx.x; c < p.columns; c += kApplyThreads) {
      const int32_t old = entries[c];
      int32_t page = c < n.full ? from[c] : -1;
      if (c == n.full && takes > 0) page = fresh;
      entries[c] = page;
      if (c == n.full && page >= 0) atomicAdd(p.refs + page, 1);  // (the others' counts: pages_plan_kernel)
      if (old >= 0) give_back(p, old);
    }
    if (threadIdx.x == 0 && takes > 0 && fresh < 0) atomicOr(p.status, kStatusNoPages);
  } else if (fresh >= 0) {
    const int item = extra % per;
    int k = 0;
    while (item >= items.first[k + 1]) ++k;
    const smq_page_plane& q = planes.plane[k];
    const int v0 = (item - items.first[k]) * items.vectors[k];
    const int v1 = v0 + items.vectors[k] < q.vectors ? v0 + items.vectors[k] : q.vectors;
    if (items.wide[k])
      copy_tokens<uint4>(q, from[n.full], fresh, p.page_size, n.rest, v0, v1);
    else
      copy_tokens<uint32_t>(q, from[n.full], fresh, p.page_size, n.rest, v0, v1);
  }
}

// ------------------------------------------------------------------- compact
//
// Tokens move in place towards the front: the j-th kept one, id k_j, to s + j,
// with k ascending and k_0 >= s, so k_j >= s + j. Rounds of consecutive j are
// moved in order, each read whole before it is written: place s + j can be the
// source of a k_i = s + j only with i <= j, so what a round overwrites belongs to
// itself or to rounds before it. Where an item (a row's vectors of one plane) has a cluster, its
// CTAs share each round and meet in between; where no place is the source of
// another, as when the newer part of a context moves forward, they need not.
//
// Bound by DRAM, half reads, half writes: 604 MB of 16 contexts, 256-byte tokens,
// 238 to 242 us, 5.0 to 5.1 TB/s of both together. Two 16-byte pieces a thread and
// eight CTAs an SM; four pieces measured 265, eight with the next round in flight 319.
// 64 rows of up to eight tokens take 5.4 us.

namespace {

constexpr int kMoveThreads = 256;
constexpr int kMovePieces = 2;        // of 16 or 4 bytes, per thread and round
constexpr int kMoveTokens = 256;      // most of a CTA's part of a round
static_assert(kMaxTokenBytes / 4 <= kMoveThreads * kMovePieces, "a CTA's part of a round holds a token");
constexpr int kCheckThreads = 1024;
constexpr int kFusedKeep = 1024;      // longest list that every block checks for itself
constexpr int kApart = 1 << 30;       // in a count: no place is the source of another

struct MoveItems {
  int32_t first[SMQ_MAX_PLANES + 1];  // items of a row before each plane's
  int32_t vectors[SMQ_MAX_PLANES];    // vectors of an item
  bool wide[SMQ_MAX_PLANES];
  int32_t ctas;                       // CTAs of an item: its cluster
};

// How many tokens row i moves, 0 where the list, a page or a count refuses it. All threads of a block.
template <int kThreads>
__device__ __forceinline__ int check_row(const CompactParams& p, int i) {
  __shared__ int first_end, first_bad, first_move;
  if (threadIdx.x == 0) {
    first_end = p.num_keep;
    first_bad = first_move = INT32_MAX;
  }
  __syncthreads();
  const int32_t row = p.rows ? p.rows[i] : i;
  bool bad_row = row < 0 || row >= p.table_rows;
  if (p.rows)
    for (int j = threadIdx.x; j < i; j += kThreads) bad_row |= p.rows[j] == row;
  bad_row = __syncthreads_or(bad_row);
  const int32_t start = p.row_start[i];
  const int32_t* const ids = p.keep_ids + static_cast<int64_t>(i) * p.keep_ld;
  if (!bad_row) {
    const int32_t* const entries = p.table + static_cast<int64_t>(row) * p.columns;
    int end = INT32_MAX, bad = INT32_MAX, move = INT32_MAX;
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
      if (id != start + j) move = min(move, j);
    }
    if (end != INT32_MAX) atomicMin(&first_end, end);
    if (bad != INT32_MAX) atomicMin(&first_bad, bad);
    if (move != INT32_MAX) atomicMin(&first_move, move);
  }
  __syncthreads();
  const bool refused = bad_row || first_bad < first_end;
  if (refused && threadIdx.x == 0) atomicOr(p.status, kStatusBounds);
  if (refused) return 0;
  const int n = first_end, m = first_move;
  return n | (n > 0 && (m >= n || ids[m] - start >= n) ? kApart : 0);
}

}  // namespace

__global__ void __launch_bounds__(kCheckThreads) compact_check_kernel(const __grid_constant__ CompactParams p) {
  griddep_launch_dependents();
  griddep_wait();
  const int n = check_row<kCheckThreads>(p, blockIdx.x);
  if (threadIdx.x == 0) p.counts[blockIdx.x] = n;
}

namespace {

// A thread's pieces of a round, and where they go (-1: nowhere).
template <typename T>
struct Pieces {
  T got[kMovePieces];
  int64_t dst[kMovePieces];
};

// The part of CTA `part` of `ctas` in moving `count` tokens of row i, vectors [v0, v1) of a plane.
template <typename T>
__device__ __forceinline__ void move_tokens(const CompactParams& p, const smq_page_plane& q, int i, int count, bool apart, int v0,
                                            int v1, int part, int ctas, int64_t (*src_s)[kMoveTokens],
                                            int64_t (*dst_s)[kMoveTokens]) {
  const int row = p.rows ? p.rows[i] : i, tid = threadIdx.x;
  const int32_t start = p.row_start[i];
  const int32_t* const ids = p.keep_ids + static_cast<int64_t>(i) * p.keep_ld;
  const int32_t* const entries = p.table + static_cast<int64_t>(row) * p.columns;
  const int64_t run = static_cast<int64_t>(p.page_size) * q.token_bytes;
  const int per_vec = q.token_bytes / static_cast<int>(sizeof(T)), per_tok = per_vec * (v1 - v0);
  int chunk = kMoveThreads * kMovePieces / per_tok;
  chunk = chunk > kMoveTokens ? kMoveTokens : chunk;
  uint8_t* const base = static_cast<uint8_t*>(q.base) + v0 * run;
  const int rounds = (count + chunk * ctas - 1) / (chunk * ctas);
  auto first_of = [&](int r) { return (r * ctas + part) * chunk; };
  auto addresses = [&](int r) {  // of round r's tokens, in one of two places
    const int j = first_of(r) + tid;
    if (tid < chunk && j < count) {
      const int32_t from = ids[j], to = start + j;
      const int32_t a = entries[from / p.page_size], b = entries[to / p.page_size];
      src_s[r % 2][tid] = from == to ? -1 : a * q.page_stride + static_cast<int64_t>(from % p.page_size) * q.token_bytes;
      dst_s[r % 2][tid] = b * q.page_stride + static_cast<int64_t>(to % p.page_size) * q.token_bytes;
    }
  };
  // piece tid of a round is of token t0; where a token's pieces divide the block's threads, so that the thread's next ones
  // are at the same place in a token, nothing has to be divided again
  const int step = kMoveThreads / per_tok, t0 = tid / per_tok;
  const bool even_split = step * per_tok == kMoveThreads;
  auto place = [&](int w) {  // of piece w of a token
    const int v = w / per_vec;
    return v * run + static_cast<int64_t>(w - v * per_vec) * sizeof(T);
  };
  const int64_t at0 = place(tid - t0 * per_tok);
  auto load = [&](int r, Pieces<T>& x) {
    const int n = min(chunk, count - first_of(r));
#pragma unroll
    for (int k = 0; k < kMovePieces; ++k) {
      const int e = k * kMoveThreads + tid;
      const int t = even_split ? t0 + k * step : e / per_tok;
      x.dst[k] = -1;
      if (t < n && src_s[r % 2][t] >= 0) {
        const int64_t at = even_split ? at0 : place(e - t * per_tok);
        x.got[k] = __ldcg(reinterpret_cast<const T*>(base + src_s[r % 2][t] + at));
        x.dst[k] = dst_s[r % 2][t] + at;
      }
    }
  };
  auto store = [&](const Pieces<T>& x) {
#pragma unroll
    for (int k = 0; k < kMovePieces; ++k)
      if (x.dst[k] >= 0) *reinterpret_cast<T*>(base + x.dst[k]) = x.got[k];
  };
  addresses(0);
  __syncthreads();
  for (int r = 0; r < rounds; ++r) {
    Pieces<T> x;
    load(r, x);
    addresses(r + 1);
    // every thread has asked for round r, and the next one's addresses are there
    if (ctas > 1 && !apart)
      cluster_sync();
    else
      __syncthreads();
    store(x);
  }
}

}  // namespace

// A cluster (of one CTA or more) per listed row, plane and group of vectors.
template <bool kFused>
__global__ void __launch_bounds__(kMoveThreads, 8)
    compact_kernel(const __grid_constant__ CompactParams p, const __grid_constant__ Planes planes,
                   const __grid_constant__ MoveItems items) {
  griddep_launch_dependents();
  griddep_wait();
  __shared__ int64_t src_s[2][kMoveTokens], dst_s[2][kMoveTokens];
  const int per = items.first[planes.count], part = blockIdx.x % items.ctas, unit = blockIdx.x / items.ctas;
  const int i = unit / per, item = unit % per;
  const int count = kFused ? check_row<kMoveThreads>(p, i) : p.counts[i];
  if (count == 0) return;  // the same in all CTAs of the cluster
  int k = 0;
  while (item >= items.first[k + 1]) ++k;
  const smq_page_plane& q = planes.plane[k];
  const int v0 = (item - items.first[k]) * items.vectors[k];
  const int v1 = v0 + items.vectors[k] < q.vectors ? v0 + items.vectors[k] : q.vectors;
  const int n = count & (kApart - 1);
  const bool apart = (count & kApart) != 0;
  if (items.wide[k])
    move_tokens<uint4>(p, q, i, n, apart, v0, v1, part, items.ctas, src_s, dst_s);
  else
    move_tokens<uint32_t>(p, q, i, n, apart, v0, v1, part, items.ctas, src_s, dst_s);
}

namespace {

template <typename K, typename... A>
cudaError_t launch(K kernel, int64_t grid, int threads, int cluster, cudaStream_t stream, A... args) {
  if (grid > INT32_MAX) return cudaErrorInvalidConfiguration;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(grid));
  cfg.blockDim = dim3(threads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

bool in_16(const smq_page_plane& q) {
  return reinterpret_cast<uintptr_t>(q.base) % 16 == 0 && q.page_stride % 16 == 0 && q.token_bytes % 16 == 0;
}

}  // namespace

cudaError_t launch_pages(const PagesParams& p, const Planes& planes, cudaStream_t stream) {
  const bool fork = p.src_rows != nullptr;
  cudaError_t rc = launch(fork ? pages_plan_kernel<true> : pages_plan_kernel<false>, static_cast<int64_t>(p.segments) + p.num_rows,
                          kPlanThreads, 1, stream, p);
  if (rc != cudaSuccess) return rc;
  CopyItems items = {};
  for (int k = 0; k < planes.count; ++k) {
    const smq_page_plane& q = planes.plane[k];
    const int64_t run = static_cast<int64_t>(p.page_size) * q.token_bytes;
    int64_t v = kCopyBytes / run;
    v = v < 1 ? 1 : v > q.vectors ? q.vectors : v;
    items.vectors[k] = static_cast<int32_t>(v);
    items.first[k + 1] = items.first[k] + static_cast<int32_t>((q.vectors + v - 1) / v);
    items.wide[k] = in_16(q);
  }
  const int64_t blocks = static_cast<int64_t>(p.num_rows) * (1 + items.first[planes.count]);
  return launch(fork ? pages_apply_kernel<true> : pages_apply_kernel<false>, blocks, kApplyThreads, 1, stream, p, planes, items);
}

cudaError_t launch_compact(const CompactParams& p, const Planes& planes, int num_sms, cudaStream_t stream) {
  MoveItems items = {};
  for (int k = 0; k < planes.count; ++k) {
    const smq_page_plane& q = planes.plane[k];
    items.wide[k] = in_16(q);
    const int piece = items.wide[k] ? 16 : 4;
    // as many vectors as give a thread two pieces of the longest round
    int64_t v = 2ll * kMoveThreads * piece / (static_cast<int64_t>(kMoveTokens) * q.token_bytes);
    v = v < 1 ? 1 : v > q.vectors ? q.vectors : v;
    items.vectors[k] = static_cast<int32_t>(v);
    items.first[k + 1] = items.first[k] + static_cast<int32_t>((q.vectors + v - 1) / v);
  }
  const int64_t blocks = static_cast<int64_t>(p.num_rows) * items.first[planes.count];
  items.ctas = 1;
  if (p.num_keep <= kFusedKeep) return launch(compact_kernel<true>, blocks, kMoveThreads, 1, stream, p, planes, items);
  // Few items: a cluster each, until there are twelve CTAs an SM or clusters of eight. One context of 32768 tokens, 8 kv heads,
  // 113 us, without clusters 676; 16 of them 362 and 801, 64 of 16384 tokens 685 and 697; until 6 or 24 an SM: the same within 2 %.
  while (items.ctas < 8 && blocks * items.ctas < 12ll * num_sms) items.ctas *= 2;
  cudaError_t rc = launch(compact_check_kernel, p.num_rows, kCheckThreads, 1, stream, p);
  if (rc != cudaSuccess) return rc;
  return launch(compact_kernel<false>, blocks * items.ctas, kMoveThreads, items.ctas, stream, p, planes, items);
}

}  // namespace smq
