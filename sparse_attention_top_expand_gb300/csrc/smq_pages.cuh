// Parameter blocks and launchers of the page operators (smq_pages.cu), shared
// with their host side (smq_pages_api.cu).
#pragma once

#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

#include "smq.h"

namespace smq {

constexpr int kStatusNoPages = 32;  // SMQ_ERR_NO_PAGES
constexpr int kSegmentUnit = 2048;  // pages: a segment's are shared by 16 warps in pieces of 128
constexpr int kMaxSegments = 1024;
constexpr int kMaxTokenBytes = 2048;  // of a plane

struct Planes {
  smq_page_plane plane[SMQ_MAX_PLANES];
  int32_t count;
};

// Rows of the block table, as listed, and what the plan kernel leaves for the
// apply kernel. Row i is the i-th listed one.
struct PagesParams {
  int32_t num_rows;
  int32_t table_rows;
  int32_t columns;
  int32_t page_size;
  int32_t num_pages;
  int32_t keep_first;
  int32_t* table;
  int32_t* refs;
  const int32_t* rows;       // resize: may be null; fork: destinations
  const int32_t* row_begin;  // resize, may be null
  const int32_t* row_end;    // resize: end; fork: length
  const int32_t* src_rows;   // fork: sources, else null
  int32_t* takes;            // [num_rows] pages that row i takes, -1: the row is skipped
  // The pool in `segments` runs of `segment` pages: the free ones of run k, in order, at free_list + k * segment, and
  // their number.
  int32_t segments;
  int32_t segment;           // a multiple of kSegmentUnit
  int32_t* free_counts;      // [segments]
  int32_t* free_list;        // [segments * segment]
  uint32_t* free_bits;       // [segments * segment / 32] a bit a page
  int32_t* snapshot;         // fork: [num_rows][columns] the sources' entries
  int32_t* status;
};

struct CompactParams {
  int32_t num_rows;
  int32_t table_rows;
  int32_t columns;
  int32_t page_size;
  int32_t num_pages;
  int32_t num_keep;
  int32_t keep_ld;
  const int32_t* table;
  const int32_t* refs;
  const int32_t* rows;  // may be null
  const int32_t* row_start;
  const int32_t* keep_ids;
  int32_t* counts;      // [num_rows] tokens that row i moves, 0: none
  int32_t* status;
};

cudaError_t launch_pages(const PagesParams& p, const Planes& planes, cudaStream_t stream);
cudaError_t launch_compact(const CompactParams& p, const Planes& planes, int num_sms, cudaStream_t stream);

}  // namespace smq
