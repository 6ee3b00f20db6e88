// kvpop_paged_attn: attention of ragged chunks of new tokens over a paged cache.
//
// One warp takes one row (token and query head): 32 slots at a time, a lane each, with a running
// maximum and sum; then the lanes share out the columns of V.
#include <string.h>

#include "paged.cuh"

namespace kvpop {
namespace {

constexpr int kThreads = 256;

struct AttnParams {
  Paged c;
  const __nv_bfloat16 *q, *k, *v;
  int64_t k_stride, v_stride;  // elements between pages
  __nv_bfloat16* O;
  float* lse;
  int Hq, G;
  float scale;
};

template <int D>
__global__ void __launch_bounds__(kThreads) attn_simple(const __grid_constant__ AttnParams p) {
  grid_dep_wait();
  grid_dep_launch();
  const Paged& c = p.c;
  const int lane = lane_id();
  __shared__ float q_s[kThreads / 32][D];
  float* q = q_s[warp_id()];
  const int rows = c.cu ? c.T : c.n;
  for (long long w = (long long)blockIdx.x * (kThreads / 32) + warp_id(); w < (long long)rows * p.Hq;
       w += (long long)gridDim.x * (kThreads / 32)) {
    const int row = (int)(w / p.Hq), hq = (int)(w - (long long)row * p.Hq), h = hq / p.G;
    int i = row;
    if (c.cu) {
      for (i = 0; i < c.n; ++i)
        if (row >= c.lo(i) && row < c.hi(i, c.lo(i))) break;
      if (i == c.n) continue;
    }
    const int lo = c.lo(i), hi = c.hi(i, lo);
    const int sees = max(0, c.len(i) - (hi - row) + 1);
    __syncwarp();
    for (int d = lane; d < D; d += 32) q[d] = __bfloat162float(p.q[((size_t)row * p.Hq + hq) * D + d]);
    __syncwarp();
    float m = __int_as_float(0xff800000), l = 0.0f, o[D / 32] = {};
    for (int t0 = 0; t0 < sees; t0 += 32) {
      const int t = t0 + lane;
      float s = __int_as_float(0xff800000);
      int pg = -1;
      if (t < sees) {
        pg = c.page_of(i, t);
        if (pg < 0) report_page(c.status, i);
        s = 0.0f;
        if (pg >= 0) {
          const __nv_bfloat16* k = p.k + pg * p.k_stride + (((size_t)h << c.log_page) + (t & ((1 << c.log_page) - 1))) * D;
          for (int d = 0; d < D; ++d) s += q[d] * __bfloat162float(k[d]);
        }
        s *= p.scale;
      }
      float mt = s;
      for (int x = 16; x; x >>= 1) mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, x));
      const float mn = fmaxf(m, mt), f = m == __int_as_float(0xff800000) ? 0.0f : expf(m - mn);
      const float e = t < sees ? expf(s - mn) : 0.0f;
      l *= f;
      for (int u = 0; u < D / 32; ++u) o[u] *= f;
      m = mn;
      for (int x = 0; x < 32 && t0 + x < sees; ++x) {
        const float ex = __shfl_sync(0xffffffffu, e, x);
        const int px = __shfl_sync(0xffffffffu, pg, x);
        l += ex;
        if (px < 0) continue;
        const __nv_bfloat16* v =
            p.v + px * p.v_stride + (((size_t)h << c.log_page) + ((t0 + x) & ((1 << c.log_page) - 1))) * D;
        for (int u = 0; u < D / 32; ++u) o[u] += ex * __bfloat162float(v[lane + 32 * u]);
      }
    }
    const size_t at = (size_t)row * p.Hq + hq;
    for (int u = 0; u < D / 32; ++u) p.O[at * D + lane + 32 * u] = __float2bfloat16(sees > 0 ? o[u] / l : 0.0f);
    if (lane == 0) p.lse[at] = sees > 0 ? m + logf(l) : __int_as_float(0xff800000);
  }
}

}  // namespace
}  // namespace kvpop

using namespace kvpop;

extern "C" kvpop_status kvpop_paged_attn_workspace_size(int T, int n, int Hq, int H, int D, int max_pages, int page,
                                                        size_t* bytes) {
  const char* name = "kvpop_paged_attn_workspace_size";
  if (!bytes) {
    set_last_error("%s: bytes must be non-NULL", name);
    return KVPOP_ERR_INVALID_ARG;
  }
  kvpop_status st = paged_check_rows(name, T, n, Hq, H, D, max_pages, page);
  if (st != KVPOP_OK) return st;
  *bytes = 256;
  return KVPOP_OK;
}

extern "C" kvpop_status kvpop_paged_attn(const void* q, int T, int n, int Hq, int H, int D, float scale, const int32_t* cu,
                                         const int32_t* lens, const int32_t* table, int max_pages, const void* kp,
                                         int64_t kp_stride, const void* vp, int64_t vp_stride, int pages, int page, void* O,
                                         float* lse, void* workspace, size_t workspace_bytes, kvpop_stream stream) {
  const char* name = "kvpop_paged_attn";
  if (!q || !O || !lse || !workspace) {
    set_last_error("%s: q, O, lse and workspace must be non-NULL", name);
    return KVPOP_ERR_INVALID_ARG;
  }
  AttnParams prm;
  size_t need = 0;
  kvpop_status st = paged_check(name, T, n, H, D, cu, lens, table, max_pages, pages, page, &prm.c);
  if (st == KVPOP_OK) st = paged_check_cache(name, "kp", kp, kp_stride, H, D, pages, page);
  if (st == KVPOP_OK) st = paged_check_cache(name, "vp", vp, vp_stride, H, D, pages, page);
  if (st == KVPOP_OK) st = kvpop_paged_attn_workspace_size(T, n, Hq, H, D, max_pages, page, &need);
  if (st != KVPOP_OK) return st;
  if (workspace_bytes < need) {
    set_last_error("%s: workspace of %zu bytes, %zu needed", name, workspace_bytes, need);
    return KVPOP_ERR_INVALID_ARG;
  }
  if (((reinterpret_cast<uintptr_t>(q) | reinterpret_cast<uintptr_t>(O)) & 15) || (reinterpret_cast<uintptr_t>(lse) & 3) ||
      (reinterpret_cast<uintptr_t>(workspace) & 255)) {
    set_last_error("%s: q and O must be 16-byte, lse 4-byte, workspace 256-byte aligned", name);
    return KVPOP_ERR_UNSUPPORTED;
  }
  prm.q = (const __nv_bfloat16*)q;
  prm.k = (const __nv_bfloat16*)kp;
  prm.v = (const __nv_bfloat16*)vp;
  prm.k_stride = kp_stride;
  prm.v_stride = vp_stride;
  prm.O = (__nv_bfloat16*)O;
  prm.lse = lse;
  prm.Hq = Hq;
  prm.G = Hq / H;
  prm.scale = scale > 0.0f ? scale : 1.0f / sqrtf((float)D);
  const dim3 grid(8 * num_sms());
  cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
  return cuda_check(D == 128 ? launch_pdl(attn_simple<128>, grid, dim3(kThreads), 0, cs, prm)
                             : launch_pdl(attn_simple<64>, grid, dim3(kThreads), 0, cs, prm),
                    "kvpop_paged_attn: launch");
}
