// kvpop_paged_mass: the attention weight that each key of a paged cache receives from a chunk's rows.
//
// One thread takes one slot of one head and walks the rows that see it.
#include <string.h>

#include "paged.cuh"

namespace kvpop {
namespace {

constexpr int kThreads = 256;

struct MassParams {
  Paged c;
  const __nv_bfloat16 *q, *k;
  const float* lse;
  int64_t k_stride;  // elements between pages
  float* scores;
  int Hq, G;
  float scale, decay;
};

template <int D>
__global__ void __launch_bounds__(kThreads) mass_simple(const __grid_constant__ MassParams p) {
  grid_dep_wait();
  grid_dep_launch();
  const Paged& c = p.c;
  const int i = blockIdx.y / c.H, h = blockIdx.y - i * c.H;
  const int lo = c.lo(i), hi = c.hi(i, lo), len = c.len(i);
  for (int t = blockIdx.x * kThreads + threadIdx.x; t < len; t += gridDim.x * kThreads) {
    const int pg = c.page_of(i, t);
    if (pg < 0) {
      report_page(c.status, i);
      continue;
    }
    const __nv_bfloat16* k = p.k + pg * p.k_stride + (((size_t)h << c.log_page) + (t & ((1 << c.log_page) - 1))) * D;
    float sum = 0.0f;
    for (int row = max(lo, hi - (len - t)); row < hi; ++row)
      for (int g = 0; g < p.G; ++g) {
        const size_t at = (size_t)row * p.Hq + h * p.G + g;
        float s = 0.0f;
        for (int d = 0; d < D; ++d) s += __bfloat162float(p.q[at * D + d]) * __bfloat162float(k[d]);
        sum += p.lse[at] == __int_as_float(0xff800000) ? 0.0f : expf(s * p.scale - p.lse[at]);
      }
    float* out = p.scores + c.slot_row(pg, h, t);
    *out = p.decay == 0.0f ? sum : p.decay * *out + sum;
  }
}

}  // namespace
}  // namespace kvpop

using namespace kvpop;

extern "C" kvpop_status kvpop_paged_mass_workspace_size(int T, int n, int Hq, int H, int D, int max_pages, int page,
                                                        size_t* bytes) {
  const char* name = "kvpop_paged_mass_workspace_size";
  if (!bytes) {
    set_last_error("%s: bytes must be non-NULL", name);
    return KVPOP_ERR_INVALID_ARG;
  }
  kvpop_status st = paged_check_rows(name, T, n, Hq, H, D, max_pages, page);
  if (st != KVPOP_OK) return st;
  *bytes = 256;
  return KVPOP_OK;
}

extern "C" kvpop_status kvpop_paged_mass(const void* q, const float* lse, int T, int n, int Hq, int H, int D, float scale,
                                         float decay, const int32_t* cu, const int32_t* lens, const int32_t* table,
                                         int max_pages, const void* kp, int64_t kp_stride, int pages, int page,
                                         float* scores, void* workspace, size_t workspace_bytes, kvpop_stream stream) {
  const char* name = "kvpop_paged_mass";
  if (!q || !lse || !scores || !workspace) {
    set_last_error("%s: q, lse, scores and workspace must be non-NULL", name);
    return KVPOP_ERR_INVALID_ARG;
  }
  if (!(decay >= 0.0f && decay <= 1.0f)) {
    set_last_error("%s: decay=%g outside [0, 1]", name, (double)decay);
    return KVPOP_ERR_INVALID_ARG;
  }
  MassParams prm;
  size_t need = 0;
  kvpop_status st = paged_check(name, T, n, H, D, cu, lens, table, max_pages, pages, page, &prm.c);
  if (st == KVPOP_OK) st = paged_check_cache(name, "kp", kp, kp_stride, H, D, pages, page);
  if (st == KVPOP_OK) st = kvpop_paged_mass_workspace_size(T, n, Hq, H, D, max_pages, page, &need);
  if (st != KVPOP_OK) return st;
  if (workspace_bytes < need) {
    set_last_error("%s: workspace of %zu bytes, %zu needed", name, workspace_bytes, need);
    return KVPOP_ERR_INVALID_ARG;
  }
  if ((reinterpret_cast<uintptr_t>(q) & 15) || ((reinterpret_cast<uintptr_t>(lse) | reinterpret_cast<uintptr_t>(scores)) & 3) ||
      (reinterpret_cast<uintptr_t>(workspace) & 255)) {
    set_last_error("%s: q must be 16-byte, lse and scores 4-byte, workspace 256-byte aligned", name);
    return KVPOP_ERR_UNSUPPORTED;
  }
  prm.q = (const __nv_bfloat16*)q;
  prm.k = (const __nv_bfloat16*)kp;
  prm.lse = lse;
  prm.k_stride = kp_stride;
  prm.scores = scores;
  prm.Hq = Hq;
  prm.G = Hq / H;
  prm.scale = scale > 0.0f ? scale : 1.0f / sqrtf((float)D);
  prm.decay = decay;
  if ((long long)n * H > 65535) {
    set_last_error("%s: n * H above 65535", name);
    return KVPOP_ERR_UNSUPPORTED;
  }
  const dim3 grid((unsigned)min(1024ll, ((long long)max_pages * page + kThreads - 1) / kThreads), n * H);
  cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
  return cuda_check(D == 128 ? launch_pdl(mass_simple<128>, grid, dim3(kThreads), 0, cs, prm)
                             : launch_pdl(mass_simple<64>, grid, dim3(kThreads), 0, cs, prm),
                    "kvpop_paged_mass: launch");
}
