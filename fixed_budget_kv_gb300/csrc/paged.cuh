// The paged key/value cache that the kvpop_paged_* calls share: a sequence's slot t lies
// at place t % page of page table[i, t / page], for every KV head.
#pragma once

#include "common.cuh"

namespace kvpop {

struct Paged {
  const int32_t* cu;     // [n + 1] rows of each sequence, or NULL: one each
  const int32_t* lens;   // [n] slots held, the new tokens included
  const int32_t* table;  // [n, max_pages]
  int* status;
  int T, n, H, D, pages, max_pages, log_page;

  __device__ __forceinline__ int lo(int i) const { return cu ? max(0, min(cu[i], T)) : i; }
  // rows [lo, hi) of sequence i
  __device__ __forceinline__ int hi(int i, int lo) const { return cu ? max(lo, min(cu[i + 1], T)) : i + 1; }
  __device__ __forceinline__ int len(int i) const { return max(0, min(lens[i], max_pages << log_page)); }
  // the page of slot t < len(i), or -1 where the table names none
  __device__ __forceinline__ int page_of(int i, int t) const {
    const int p = table[(size_t)i * max_pages + (t >> log_page)];
    return p >= 0 && p < pages ? p : -1;
  }
  // (page, head, place) as a row of [pages, H, page]
  __device__ __forceinline__ size_t slot_row(int pg, int h, int t) const {
    return (((size_t)pg * H + h) << log_page) + (t & ((1 << log_page) - 1));
  }
};

// A table entry that names no page: the slots behind it are skipped.
__device__ __forceinline__ void report_page(int* status, int entry) {
  report_error(status, KVPOP_ERR_INVALID_ARG, SITE_PAGED_TABLE, entry);
}

constexpr int kMinPage = 16, kMaxPage = 65536;

// Host checks that every call makes; fills `p` (T = n, cu = NULL for calls without rows).
kvpop_status paged_check(const char* name, int T, int n, int H, int D, const int32_t* cu, const int32_t* lens,
                         const int32_t* table, int max_pages, int pages, int page, Paged* p);
// ... of calls with query rows, without pointers
kvpop_status paged_check_rows(const char* name, int T, int n, int Hq, int H, int D, int max_pages, int page);
// ... and of one of the caches
kvpop_status paged_check_cache(const char* name, const char* which, const void* x, int64_t stride, int H, int D, int pages,
                               int page);

}  // namespace kvpop
