// The checks that the kvpop_paged_* calls share, and kvpop_paged_append: new tokens' keys
// and values into the pages.
//
// Row r of a sequence with c new tokens goes to slot len - c + r.  A warp takes a token's k and v
// of up to kHeads (D = 128) or twice as many heads: all 16-byte pieces are on their way before the
// slot is looked up.  Bound by memory: 8 D bytes a token and head.  16 384 tokens of 8 heads of
// D = 128: 24 us, 83% of the copy rate.
#include <string.h>

#include "paged.cuh"

namespace kvpop {

kvpop_status paged_check(const char* name, int T, int n, int H, int D, const int32_t* cu, const int32_t* lens,
                         const int32_t* table, int max_pages, int pages, int page, Paged* p) {
  if (!lens || !table) {
    set_last_error("%s: lens and table must be non-NULL", name);
    return KVPOP_ERR_INVALID_ARG;
  }
  if (T <= 0 || n <= 0 || H <= 0 || max_pages <= 0 || pages <= 0 || page <= 0) {
    set_last_error("%s: bad shape T=%d n=%d H=%d pages=%d page=%d max_pages=%d", name, T, n, H, pages, page, max_pages);
    return KVPOP_ERR_INVALID_ARG;
  }
  if (!cu && T != n) {
    set_last_error("%s: cu is needed with %d rows of %d sequences", name, T, n);
    return KVPOP_ERR_INVALID_ARG;
  }
  if (D != 64 && D != 128) {
    set_last_error("%s: D=%d unsupported (64 or 128)", name, D);
    return KVPOP_ERR_UNSUPPORTED;
  }
  if (page < kMinPage || page > kMaxPage || (page & (page - 1))) {
    set_last_error("%s: page=%d unsupported (a power of two from %d to %d)", name, page, kMinPage, kMaxPage);
    return KVPOP_ERR_UNSUPPORTED;
  }
  if (H > 65535 || n > 65535 || T > (1 << 24) || (long long)max_pages * page > (1 << 30)) {
    set_last_error("%s: at most 65535 heads and sequences, 2^24 rows and 2^30 slots a sequence", name);
    return KVPOP_ERR_UNSUPPORTED;
  }
  if ((reinterpret_cast<uintptr_t>(cu) | reinterpret_cast<uintptr_t>(lens) | reinterpret_cast<uintptr_t>(table)) & 3) {
    set_last_error("%s: cu, lens and table must be 4-byte aligned", name);
    return KVPOP_ERR_UNSUPPORTED;
  }
  memset(p, 0, sizeof(*p));
  p->cu = cu;
  p->lens = lens;
  p->table = table;
  p->T = T;
  p->n = n;
  p->H = H;
  p->D = D;
  p->pages = pages;
  p->max_pages = max_pages;
  while ((1 << p->log_page) < page) ++p->log_page;
  p->status = device_status_ptr();
  return KVPOP_OK;
}

kvpop_status paged_check_rows(const char* name, int T, int n, int Hq, int H, int D, int max_pages, int page) {
  if (T <= 0 || n <= 0 || H <= 0 || Hq <= 0 || max_pages <= 0 || page <= 0 || Hq % H != 0) {
    set_last_error("%s: bad shape T=%d n=%d Hq=%d H=%d max_pages=%d page=%d", name, T, n, Hq, H, max_pages, page);
    return KVPOP_ERR_INVALID_ARG;
  }
  if ((D != 64 && D != 128) || 128 % (Hq / H) != 0) {
    set_last_error("%s: D=%d (64 or 128), G=%d (dividing 128) unsupported", name, D, Hq / H);
    return KVPOP_ERR_UNSUPPORTED;
  }
  if (page < kMinPage || page > kMaxPage || (page & (page - 1))) {
    set_last_error("%s: page=%d unsupported (a power of two from %d to %d)", name, page, kMinPage, kMaxPage);
    return KVPOP_ERR_UNSUPPORTED;
  }
  const long long slots = (long long)max_pages * page;
  if (H > 65535 || Hq > 65535 || n > 65535 || T > (1 << 24) || (long long)T * Hq > 0x7fffffffll || slots > (1 << 30)) {
    set_last_error("%s: at most 65535 heads and sequences, 2^24 tokens, 2^31 - 1 rows and 2^30 slots a sequence", name);
    return KVPOP_ERR_UNSUPPORTED;
  }
  // the kernels number their units of work in 32 bits: up to three for a tile of rows and keys, and
  // setting a tile of rows up counts as eight more
  if ((n + (long long)T * (Hq / H) / 128) * H > 0x7fffffffll / (3 * ((slots + 127) / 128 + 8))) {
    set_last_error("%s: more than 7 * 10^8 tiles of rows and keys", name);
    return KVPOP_ERR_UNSUPPORTED;
  }
  return KVPOP_OK;
}

kvpop_status paged_check_cache(const char* name, const char* which, const void* x, int64_t stride, int H, int D, int pages,
                               int page) {
  if (!x) {
    set_last_error("%s: %s must be non-NULL", name, which);
    return KVPOP_ERR_INVALID_ARG;
  }
  if (stride < (int64_t)H * page * D) {
    set_last_error("%s: pages of %s overlap (%lld elements apart)", name, which, (long long)stride);
    return KVPOP_ERR_INVALID_ARG;
  }
  if ((stride & 7) || (reinterpret_cast<uintptr_t>(x) & 15) || stride >= (1ll << 38)) {
    set_last_error("%s: %s must be 16-byte aligned, its pages a multiple of 8 elements apart, below 2^38", name, which);
    return KVPOP_ERR_UNSUPPORTED;
  }
  return KVPOP_OK;
}

namespace {

constexpr int kThreads = 256;
constexpr int kHeads = 8;  // rows of k or v that a lane has in flight

struct AppendParams {
  Paged c;
  const uint4 *k_new, *v_new;
  int64_t k_new_stride, v_new_stride;  // 16-byte pieces between tokens
  uint4 *k, *v;
  int64_t k_stride, v_stride;  // 16-byte pieces between pages
  float* scores;
};

// The sequence that row `row` is in: the last whose rows begin at or before it.  -1 where none is.
__device__ __forceinline__ int sequence_of(const Paged& c, int row) {
  if (!c.cu) return row;
  int a = 0, b = c.n;  // cu[a] <= row < cu[b], if cu is non-decreasing
  if (row < c.cu[0] || row >= c.cu[c.n]) return -1;
  while (b - a > 1) {
    const int m = (a + b) >> 1;
    if (c.cu[m] <= row) a = m;
    else b = m;
  }
  return a;
}

__global__ void __launch_bounds__(kThreads) append_kernel(const __grid_constant__ AppendParams p) {
  grid_dep_wait();
  grid_dep_launch();
  const Paged& c = p.c;
  const int ch = c.D / 8, lane = lane_id();  // pieces of a row
  // D = 128: half of the lanes take a row of k, half one of v; D = 64: two rows of each
  const int x = lane % ch, sub = lane / ch % (16 / ch);
  const bool is_v = lane >= 16;
  const uint4* from = is_v ? p.v_new : p.k_new;
  uint4* to = is_v ? p.v : p.k;
  const int64_t from_stride = is_v ? p.v_new_stride : p.k_new_stride, to_stride = is_v ? p.v_stride : p.k_stride;
  const int rows = 16 / ch, heads = kHeads * rows, groups = (c.H + heads - 1) / heads;
  const long long items = (long long)c.T * groups;
  for (long long w = (long long)blockIdx.x * (kThreads / 32) + warp_id(); w < items;
       w += (long long)gridDim.x * (kThreads / 32)) {
    const int row = (int)(w / groups), h0 = (int)(w - (long long)row * groups) * heads + sub;
    // the new rows do not depend on where they go
    uint4 y[kHeads];
#pragma unroll
    for (int u = 0; u < kHeads; ++u)
      if (h0 + u * rows < c.H) y[u] = from[row * from_stride + (size_t)(h0 + u * rows) * ch + x];
    const int i = sequence_of(c, row);
    if (i < 0) continue;
    const int lo = c.lo(i), hi = c.hi(i, lo);
    const int len = c.len(i), t = len - (hi - row);
    if (t < 0 || t >= len) continue;  // more new tokens than slots: the first of them have none
    const int pg = c.page_of(i, t);
    if (pg < 0) {
      if (lane == 0) report_page(c.status, i);
      continue;
    }
#pragma unroll
    for (int u = 0; u < kHeads; ++u) {
      const int h = h0 + u * rows;
      if (h < c.H) {
        to[pg * to_stride + (((size_t)h << c.log_page) + (t & ((1 << c.log_page) - 1))) * ch + x] = y[u];
        if (p.scores && !is_v && x == 0) p.scores[c.slot_row(pg, h, t)] = 0.0f;
      }
    }
  }
}

}  // namespace
}  // namespace kvpop

using namespace kvpop;

extern "C" kvpop_status kvpop_paged_append(const void* k_new, int64_t k_new_stride, const void* v_new, int64_t v_new_stride,
                                           int T, int n, int H, int D, const int32_t* cu, const int32_t* lens,
                                           const int32_t* table, int max_pages, void* kp, int64_t kp_stride, void* vp,
                                           int64_t vp_stride, int pages, int page, float* scores, kvpop_stream stream) {
  const char* name = "kvpop_paged_append";
  if (!k_new || !v_new) {
    set_last_error("%s: k_new and v_new must be non-NULL", name);
    return KVPOP_ERR_INVALID_ARG;
  }
  AppendParams prm;
  kvpop_status st = paged_check(name, T, n, H, D, cu, lens, table, max_pages, pages, page, &prm.c);
  if (st == KVPOP_OK) st = paged_check_cache(name, "kp", kp, kp_stride, H, D, pages, page);
  if (st == KVPOP_OK) st = paged_check_cache(name, "vp", vp, vp_stride, H, D, pages, page);
  if (st != KVPOP_OK) return st;
  if (k_new_stride < (int64_t)H * D || v_new_stride < (int64_t)H * D) {
    set_last_error("%s: tokens overlap (k %lld, v %lld elements apart)", name, (long long)k_new_stride,
                   (long long)v_new_stride);
    return KVPOP_ERR_INVALID_ARG;
  }
  if (((k_new_stride | v_new_stride) & 7) || ((reinterpret_cast<uintptr_t>(k_new) | reinterpret_cast<uintptr_t>(v_new)) & 15) ||
      (reinterpret_cast<uintptr_t>(scores) & 3)) {
    set_last_error("%s: k_new and v_new must be 16-byte aligned with strides that are multiples of 8", name);
    return KVPOP_ERR_UNSUPPORTED;
  }
  prm.k_new = (const uint4*)k_new;
  prm.v_new = (const uint4*)v_new;
  prm.k_new_stride = k_new_stride / 8;
  prm.v_new_stride = v_new_stride / 8;
  prm.k = (uint4*)kp;
  prm.v = (uint4*)vp;
  prm.k_stride = kp_stride / 8;
  prm.v_stride = vp_stride / 8;
  prm.scores = scores;
  const int heads = kHeads * (128 / D);
  const long long items = (long long)T * ((H + heads - 1) / heads);
  const int blocks = (int)min((items + kThreads / 32 - 1) / (kThreads / 32), 8ll * num_sms());
  return cuda_check(launch_pdl(append_kernel, dim3(blocks), dim3(kThreads), 0, reinterpret_cast<cudaStream_t>(stream), prm),
                    "kvpop_paged_append: launch");
}
