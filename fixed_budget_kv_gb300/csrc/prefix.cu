// kvpop_prefix_attn: decode rows over key/value prefixes that groups of sequences
// share, joined with another attention result of the same rows.
#include "common.cuh"

namespace kvpop {
namespace {

constexpr int kThreads = 256;

struct PrefixParams {
  const __nv_bfloat16* q;
  const __nv_bfloat16* k;
  const __nv_bfloat16* v;
  const int32_t* cu;
  const int32_t* lens;
  const __nv_bfloat16* o2;
  const float* lse2;
  __nv_bfloat16* O;
  float* lse;
  int n, m, P, Hq, H, G;
  float scale_log2;
};

// One CTA per (sequence, query head): each warp takes every 8th key with a running
// maximum and sum, then the warps' results are joined.
template <int D>
__global__ void __launch_bounds__(kThreads) prefix_simple(const PrefixParams p) {
  constexpr int E = D / 32;
  __shared__ float m_s[8], l_s[8], o_s[8][D];
  const int i = blockIdx.x, hq = blockIdx.y, h = hq / p.G;
  const int lane = lane_id(), warp = warp_id();
  grid_dep_launch();
  grid_dep_wait();
  int g = -1;
  if (!p.cu) {
    g = 0;
  } else {
    int seen = 0;
    for (int j = 0; j < p.m; ++j) {
      const int lo = max(seen, min(p.cu[j], p.n)), hi = max(lo, min(p.cu[j + 1], p.n));
      if (i >= lo && i < hi) g = j;
      seen = hi;
    }
  }
  if (g < 0) return;
  const int len = p.lens ? max(0, min(p.lens[g], p.P)) : p.P;
  const size_t row = (size_t)i * p.Hq + hq;
  float qr[E], o[E] = {};
  for (int e = 0; e < E; ++e) qr[e] = __bfloat162float(p.q[row * D + lane * E + e]) * p.scale_log2;
  const float ninf = __int_as_float(0xff800000);
  float mx = ninf, l = 0.f;
  for (int t = warp; t < len; t += 8) {
    const size_t at = (((size_t)g * p.P + t) * p.H + h) * D + lane * E;
    float s = 0.f;
    for (int e = 0; e < E; ++e) s += qr[e] * __bfloat162float(p.k[at + e]);
    for (int x = 16; x > 0; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
    const float mn = fmaxf(mx, s);
    const float a = mn == ninf ? 1.f : exp2f(mx - mn), w = mn == ninf ? 0.f : exp2f(s - mn);
    l = l * a + w;
    for (int e = 0; e < E; ++e) o[e] = o[e] * a + w * __bfloat162float(p.v[at + e]);
    mx = mn;
  }
  if (lane == 0) m_s[warp] = mx, l_s[warp] = l;
  for (int e = 0; e < E; ++e) o_s[warp][lane * E + e] = o[e];
  const float j2 = p.o2 ? p.lse2[row] * 1.4426950408889634f : ninf;  // read before lse, which may be lse2, is written
  __syncthreads();
  if (threadIdx.x < D) {
    const int d = threadIdx.x;
    float M = j2, L = 0.f, O = 0.f;
    for (int w = 0; w < 8; ++w) M = fmaxf(M, m_s[w]);
    for (int w = 0; w < 8; ++w)
      if (m_s[w] != ninf) {
        const float f = exp2f(m_s[w] - M);
        L += f * l_s[w];
        O += f * o_s[w][d];
      }
    if (j2 != ninf) {
      const float f = exp2f(j2 - M);
      L += f;
      O += f * __bfloat162float(p.o2[row * D + d]);
    }
    p.O[row * D + d] = __float2bfloat16_rn(L > 0.f ? O / L : 0.f);
    __syncwarp();
    if (d == 0) p.lse[row] = L > 0.f ? (M + log2f(L)) * 0.69314718055994531f : ninf;
  }
}

}  // namespace
}  // namespace kvpop

using namespace kvpop;

extern "C" kvpop_status kvpop_prefix_attn_workspace_size(int n, int m, int P, int Hq, int H, int D, size_t* bytes) {
  if (!bytes || n <= 0 || m <= 0 || P <= 0 || H <= 0 || Hq <= 0 || Hq % H != 0) {
    set_last_error("kvpop_prefix_attn_workspace_size: bad arguments");
    return KVPOP_ERR_INVALID_ARG;
  }
  if ((D != 64 && D != 128) || 128 % (Hq / H) != 0) {
    set_last_error("kvpop_prefix_attn_workspace_size: D=%d (64 or 128), G=%d (dividing 128) unsupported", D, Hq / H);
    return KVPOP_ERR_UNSUPPORTED;
  }
  *bytes = 256;
  return KVPOP_OK;
}

extern "C" kvpop_status kvpop_prefix_attn(const void* q, const void* pk, const void* pv, int n, int m, int P, int Hq,
                                          int H, int D, float scale, const int32_t* cu, const int32_t* lens,
                                          const void* O2, const float* lse2, void* O, float* lse, void* workspace,
                                          size_t workspace_bytes, kvpop_stream stream) {
  if (!q || !pk || !pv || !O || !lse || !workspace) {
    set_last_error("kvpop_prefix_attn: q, pk, pv, O, lse and workspace must be non-NULL");
    return KVPOP_ERR_INVALID_ARG;
  }
  if ((O2 == nullptr) != (lse2 == nullptr)) {
    set_last_error("kvpop_prefix_attn: O2 and lse2 go together");
    return KVPOP_ERR_INVALID_ARG;
  }
  size_t need = 0;
  kvpop_status st = kvpop_prefix_attn_workspace_size(n, m, P, Hq, H, D, &need);
  if (st != KVPOP_OK) return st;
  if (!cu && m != 1) {
    set_last_error("kvpop_prefix_attn: cu is needed with m=%d prefixes", m);
    return KVPOP_ERR_INVALID_ARG;
  }
  if (workspace_bytes < need) {
    set_last_error("kvpop_prefix_attn: workspace of %zu bytes, %zu needed", workspace_bytes, need);
    return KVPOP_ERR_INVALID_ARG;
  }
  const uintptr_t am = reinterpret_cast<uintptr_t>(q) | reinterpret_cast<uintptr_t>(pk) |
                       reinterpret_cast<uintptr_t>(pv) | reinterpret_cast<uintptr_t>(O) |
                       reinterpret_cast<uintptr_t>(O2);
  if ((am & 15) || (reinterpret_cast<uintptr_t>(workspace) & 255)) {
    set_last_error("kvpop_prefix_attn: q, pk, pv, O, O2 must be 16-byte, workspace 256-byte aligned");
    return KVPOP_ERR_UNSUPPORTED;
  }
  if (H > 65535 || Hq > 65535 || m > 65535 || n > (1 << 24)) {
    set_last_error("kvpop_prefix_attn: at most 65535 heads and prefixes and 2^24 sequences");
    return KVPOP_ERR_UNSUPPORTED;
  }
  PrefixParams prm = {};
  prm.q = (const __nv_bfloat16*)q;
  prm.k = (const __nv_bfloat16*)pk;
  prm.v = (const __nv_bfloat16*)pv;
  prm.cu = cu;
  prm.lens = lens;
  prm.o2 = (const __nv_bfloat16*)O2;
  prm.lse2 = lse2;
  prm.O = (__nv_bfloat16*)O;
  prm.lse = lse;
  prm.n = n;
  prm.m = m;
  prm.P = P;
  prm.Hq = Hq;
  prm.H = H;
  prm.G = Hq / H;
  prm.scale_log2 = (scale > 0.0f ? scale : 1.0f / sqrtf((float)D)) * 1.4426950408889634f;
  auto kern = D == 128 ? prefix_simple<128> : prefix_simple<64>;
  return cuda_check(launch_pdl(kern, dim3(n, Hq), dim3(kThreads), 0, reinterpret_cast<cudaStream_t>(stream), prm),
                    "kvpop_prefix_attn: launch");
}
