// mx_pages.hpp - arguments of the page bookkeeping and page copy kernels.
#pragma once

#include "mx.hpp"

namespace nvfp4 {

// Sequences in slots and the pages they hold: entries [0, ceil(len / page_size)) of a slot's row.
struct MxPages {
  int32_t* table;   // [slots, max_pages]
  int32_t* lens;    // [slots]
  int32_t* refs;    // [num_pages] entries that hold each page; below 1: free
  int64_t stride, num_pages;
  int slots, max_pages, page_shift;
};

constexpr int64_t kMxMostListed = 1 << 16;

// workspace of a reserve: by slot its first place in the list; by listed slot where its pages start among
// the new ones and twice their number (one more if its last page is copied, -1: not served); the new pages
struct MxReserveWork {
  int32_t* mark;
  int2* plan;
  int32_t* found;
  int32_t* fresh;
};

// workspaces
int64_t mx_reserve_bytes(int64_t n, int64_t slots, int64_t max_pages, int64_t num_pages);
int64_t mx_compact_bytes(int64_t num_pages);

hipError_t launch_mx_pages_free(const MxPages& p, const int32_t* slots, const int32_t* keep, int n, hipStream_t stream);
hipError_t launch_mx_pages_fork(const MxPages& p, const int32_t* parents, const int32_t* children, int n, int32_t* done,
                                hipStream_t stream);
hipError_t launch_mx_pages_reserve(const MxPages& p, const int32_t* slots, const int32_t* lens, int n, int32_t* done,
                                   int32_t* src, int32_t* dst, void* workspace, hipStream_t stream);
hipError_t launch_mx_pages_compact(const MxPages& p, int32_t* table_out, int64_t stride_out, int32_t* refs_out,
                                   int32_t* src, int32_t* dst, int32_t* used, void* workspace, hipStream_t stream);
hipError_t launch_mx_cache_copy(const MxCache& from, int64_t from_pages, const MxCache& to, int64_t to_pages,
                                int page_size, const int32_t* src, const int32_t* dst, int64_t n, hipStream_t stream);

}  // namespace nvfp4
