// kvpop_qk_norm_rope and its gradient: the RMS norm of every query and key head
// and the position rotation, in one pass over the projections.
//
// For a head row x (D values), weights w, frequencies f_i and position t:
//   r = (mean x^2 + eps)^(-1/2),  y = r x w,
//   (z_a, z_b) = (y_a cos - y_b sin, y_b cos + y_a sin) at the angle t f_i
// for the pairs (i, i + R/2) or (2i, 2i + 1), i < R/2; dims >= R keep y.
// Backward, g = dL/dz: dy turns g back by the same angle, e = dy w,
//   dx = r (e - x r^2 mean(e x)),  dw = sum over rows of dy x r.
//
// Layout: a lane holds both members of its pairs -- two 16-byte pieces of a
// row, D/16 lanes to a row -- so the rotation needs no exchange and a row's sum
// takes log2(D/16) shuffles.  A warp takes one token: its lanes compute the
// token's R/2 angles once (shared out over the row groups) and use them for
// every head; with few tokens, or to fill the last round, several warps share one.
// HBM-bound: 4 bytes a value forward, 8 backward.  Measured (Hq 32, H 8, D 128, q and k
// from a packed projection, one GB300): 16 384 tokens 57 us forward (87% of the copy rate)
// and 111 us backward (89%), 131 072 tokens 402 us forward (98%).  Angles and weights stay
// in shared memory, in the order in which the lanes read them: the registers that this
// frees are worth more as further warps (421 -> 402 us, 118 -> 111 us).
//
// Angles: f / 2 pi becomes a 64-bit fixed-point fraction of a turn, so the
// product with an integer position wraps at whole turns without any loss; the
// top 32 bits, as a signed number, go to sincospif.  The fraction is off by less
// than 2 units of 2^-64 for any finite f, 2^-32 of a turn at position 2^31, and
// as much again goes with the low half: 2^-28 rad.  What counts is the conversion
// of the top half to fp32, at most 2^-25 of a half turn or 2^-23 rad, and
// sincospif's own rounding: 2^-22 rad in all.
#include "common.cuh"

namespace kvpop {
namespace {

constexpr int kWarps = 4;          // per CTA
// Resident CTAs an SM, the grid's limit: as many warps as the registers allow without
// spills.  16 384 tokens forward (loads two passes ahead): 58.7 us with 5, 56.8 with 6, 57.0
// with 7; backward (no loads ahead, more warps instead): 111 us with 5, 132 with 6, and 115
// with 4 and loads one pass ahead.
constexpr int kCtasPerSm = 6;
constexpr int kBwdWarps = 4;
constexpr int kBwdCtasPerSm = 5;
constexpr int kBwdMaxCtas = 1024;  // rows of the weight gradients' workspace

struct QkParams {
  const __nv_bfloat16* q;
  const __nv_bfloat16* k;
  long long q_stride, k_stride;  // elements between tokens
  const float* wq;
  const float* wk;
  const float* inv_freq;
  const int32_t* pos;
  __nv_bfloat16* q_out;
  __nv_bfloat16* k_out;
  long long qo_stride, ko_stride;
  const float* dq;  // backward only: [T, Hq, D], [T, H, D]
  const float* dk;
  float* part;      // backward only: [CTAs, D] partial weight gradients
  int T, S, Hq, H, nrot;  // nrot = R / 16: lanes of a row that rotate
  int slices;             // warps that share a token's heads (backward: its query heads)
  int slices_k;           // backward only: warps that share a token's key heads
  int ctas_q;             // backward only: CTAs that take query heads
  float eps;
};

// Which two 8-column pieces of a row lane j holds: the two members of its eight
// pairs, or two neighbours where it does not rotate.
template <bool INTER>
__device__ __forceinline__ void pieces(int j, int nrot, int& a, int& b) {
  if (!INTER && j < nrot) {
    a = j;
    b = j + nrot;
  } else {
    a = 2 * j;
    b = 2 * j + 1;
  }
}

__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

// Eight bf16 values as four pairs of fp32, and back with one rounding.
__device__ __forceinline__ void unpack8(const uint4& v, uint64_t (&x)[4]) {
  const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) x[i] = pack2(__uint_as_float(u[i] << 16), __uint_as_float(u[i] & 0xffff0000u));
}

__device__ __forceinline__ uint4 pack8(const uint64_t (&x)[4]) {
  uint32_t u[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float lo, hi;
    unpack2(x[i], lo, hi);
    u[i] = pack_bf16x2(lo, hi);
  }
  return make_uint4(u[0], u[1], u[2], u[3]);
}

__device__ __forceinline__ float sum2(uint64_t v) {
  float lo, hi;
  unpack2(v, lo, hi);
  return lo + hi;
}

// Eight floats of lane j: float4 j of two consecutive rows of LPR float4 (no bank conflicts).
template <int LPR>
__device__ __forceinline__ void lds8(const float4* s, int j, uint64_t (&x)[4]) {
  const float4 u = s[j], v = s[LPR + j];
  x[0] = pack2(u.x, u.y);
  x[1] = pack2(u.z, u.w);
  x[2] = pack2(v.x, v.y);
  x[3] = pack2(v.z, v.w);
}

// 0, or NaN for a column that turns by a frequency that is not finite (whose angle is a NaN).
template <bool INTER>
__device__ __forceinline__ float no_angle(const float* inv_freq, int nrot, int col) {
  if (col >= 16 * nrot) return 0.0f;
  return fabsf(inv_freq[INTER ? col / 2 : col < 8 * nrot ? col : col - 8 * nrot]) * 0.0f;
}

// Weights in that order: rows 0, 1 for piece a of each lane, 2, 3 for piece b.  A column
// without an angle gets a NaN, which reaches both members of its pair.
template <int D, bool INTER>
__device__ __forceinline__ void stage_weights(float4* dst, const float* w, const float* inv_freq, int nrot, int thread,
                                              int threads) {
  constexpr int LPR = D / 16;
  for (int i = thread; i < 16 * LPR; i += threads) {
    int a, b;
    pieces<INTER>(i / 4 % LPR, nrot, a, b);
    const int col = 8 * (i < 8 * LPR ? a : b) + 4 * (i / 4 / LPR & 1) + (i & 3);
    reinterpret_cast<float*>(dst)[i] = (w ? w[col] : 1.0f) + no_angle<INTER>(inv_freq, nrot, col);
  }
}

// Turns per position as a fraction of 2^64, whole turns dropped: the 24-bit significand times
// 1 / 2 pi, moved to the exponent's place (the reduction of Payne and Hanek, 1983).  A large
// exponent moves leading bits of 1 / 2 pi out as whole turns: 256 bits leave 128 for the largest.
__device__ __forceinline__ unsigned long long turns64(float f) {
  const unsigned long long c0 = 0x28be60db9391054aull, c1 = 0x7f09d5f47d4d3770ull, c2 = 0x36d8a5664f10e410ull,
                           c3 = 0x7f9458eaf7aef158ull;  // 2^256 / (2 pi)
  const uint32_t u = __float_as_uint(f);
  const int exp = (int)(u >> 23 & 255), sh = 150 - exp;  // |f| = sig 2^-sh
  const unsigned long long sig = exp ? (u & 0x7fffffu) | 0x800000u : 0ull;
  unsigned long long hi = c0, lo = c1, r;
  if (sh < 0) {
    const bool w = sh <= -64;
    const int up = -sh & 63;
    const unsigned long long a = w ? c1 : c0, b = w ? c2 : c1, d = w ? c3 : c2;
    hi = up ? a << up | b >> (64 - up) : a;
    lo = up ? b << up | d >> (64 - up) : b;
  }
  const unsigned long long carry = __umul64hi(sig, lo), p0 = sig * hi + carry;
  const unsigned long long p1 = __umul64hi(sig, hi) + (p0 < carry);
  if (sh <= 0) r = p0;
  else if (sh < 64) r = p0 >> sh | p1 << (64 - sh);
  else r = sh < 128 ? p1 >> (sh - 64) : 0ull;
  return u >> 31 ? 0ull - r : r;
}

// The eight angles of each lane j = lane % LPR: the 32 / LPR row groups compute a share
// each, into the warp's shared memory -- cos in rows 0, 1, sin in rows 2, 3 of LPR float4.
template <int LPR>
struct Angles {
  static constexpr int RPP = 32 / LPR, MINE = 8 / RPP;
  unsigned long long turn[MINE];
  float4* s;

  __device__ __forceinline__ void init(float4* smem, const float* inv_freq, int j, int rg, int nrot) {
    s = smem;
#pragma unroll
    for (int i = 0; i < MINE; ++i) turn[i] = j < nrot ? turns64(inv_freq[8 * j + rg * MINE + i]) : 0ull;
  }
  __device__ __forceinline__ void at(int pos, int j, int rg) {
    __syncwarp();  // every lane has read the angles of the token before
#pragma unroll
    for (int i = 0; i < MINE; ++i) {
      const unsigned long long a = turn[i] * (unsigned long long)(long long)pos;
      float sn, cs;
      sincospif((float)(int)(a >> 32) * 4.656612873077393e-10f, &sn, &cs);  // half turns in [-1, 1]
      const int e = rg * MINE + i;
      float* dst = reinterpret_cast<float*>(s + (e >> 2) * LPR + j) + (e & 3);
      dst[0] = cs;
      dst[8 * LPR] = sn;
    }
    __syncwarp();
  }
  // Half-split pairs sit at the same place of the two pieces, adjacent pairs next to each
  // other in one of them.  BACK turns the other way.
  template <bool INTER, bool BACK>
  __device__ __forceinline__ void rotate(uint64_t (&a)[4], uint64_t (&b)[4], int j) const {
    uint64_t c[4], sn[4];
    lds8<LPR>(s, j, c);
    lds8<LPR>(s + 2 * LPR, j, sn);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (!INTER) {
        const uint64_t ns = sn[i] ^ 0x8000000080000000ull;
        const uint64_t u = fma2(b[i], BACK ? sn[i] : ns, mul2(a[i], c[i]));
        b[i] = fma2(a[i], BACK ? ns : sn[i], mul2(b[i], c[i]));
        a[i] = u;
      } else {
#pragma unroll
        for (int h = 0; h < 2; ++h) {  // angle e = 2 i + h: pair e of a, or e - 4 of b
          const int e = 2 * i + h;
          uint64_t& y = e < 4 ? a[e & 3] : b[e & 3];
          float u, v, c0, c1, s0, s1;
          unpack2(y, u, v);
          unpack2(c[i], c0, c1);
          unpack2(sn[i], s0, s1);
          const float cs = h ? c1 : c0, sg = BACK ? -(h ? s1 : s0) : (h ? s1 : s0);
          y = pack2(u * cs - v * sg, v * cs + u * sg);
        }
      }
    }
  }
};

// The passes of a warp's tasks, one after the other: pass ps of token t takes head
// rows ps * RPP .. of the token.  The forward's loads run ahead, into the next task.
struct Passes {
  uint32_t task, ntask, step;
  int t, ps, p1;

  __device__ __forceinline__ void enter(int slices, int passes) {
    if (task >= ntask) return;
    int sl = 0;
    t = (int)task;
    if (slices > 1) {
      t = (int)(task / (uint32_t)slices);
      sl = (int)task - t * slices;
    }
    ps = passes * sl / slices;
    p1 = passes * (sl + 1) / slices;
  }
  __device__ __forceinline__ bool live() const { return task < ntask; }
  __device__ __forceinline__ bool next(int slices, int passes) {  // true: entered another task
    if (++ps < p1) return false;
    task += step;
    enter(slices, passes);
    return true;
  }
};

template <int D, bool INTER>
__global__ void __launch_bounds__(kWarps * 32, kCtasPerSm) qk_norm_fwd(const QkParams p) {
  constexpr int LPR = D / 16, RPP = 32 / LPR;
  __shared__ float4 w_s[2 * 4 * LPR];  // q, k
  __shared__ float4 ang_s[kWarps][4 * LPR];
  const int lane = lane_id(), j = lane % LPR, rg = lane / LPR;
  grid_dep_launch();
  grid_dep_wait();  // the projections, positions and weights come from earlier kernels
  int pa, pb;
  pieces<INTER>(j, p.nrot, pa, pb);
  const int rows = p.Hq + p.H, passes = (rows + RPP - 1) / RPP;
  // two cursors over this warp's passes: the one being computed and the next one to load
  Passes cur, ahead;
  cur.task = blockIdx.x * kWarps + warp_id();
  cur.ntask = (uint32_t)p.T * p.slices;
  cur.step = gridDim.x * kWarps;
  cur.enter(p.slices, passes);
  ahead = cur;
  const uint4 *q_t, *k_t;  // row 0 of the token being loaded; key rows count on from the query rows
  auto token = [&]() {
    q_t = reinterpret_cast<const uint4*>(p.q + ahead.t * p.q_stride);
    k_t = reinterpret_cast<const uint4*>(p.k + ahead.t * p.k_stride) - (long long)p.Hq * (D / 8);
  };
  if (cur.live()) token();
  auto load = [&](uint4& a, uint4& b) {
    if (!ahead.live()) return;
    const int row = ahead.ps * RPP + rg;
    if (row < rows) {
      const uint4* src = (row >= p.Hq ? k_t : q_t) + row * (D / 8);
      a = src[pa];
      b = src[pb];
    }
    if (ahead.next(p.slices, passes) && ahead.live()) token();
  };
  uint4 r0[2], r1[2];
  r0[0] = r0[1] = r1[0] = r1[1] = make_uint4(0, 0, 0, 0);
  load(r0[0], r0[1]);
  load(r1[0], r1[1]);
  stage_weights<D, INTER>(w_s, p.wq, p.inv_freq, p.nrot, threadIdx.x, kWarps * 32);
  stage_weights<D, INTER>(w_s + 4 * LPR, p.wk, p.inv_freq, p.nrot, threadIdx.x, kWarps * 32);
  Angles<LPR> ang;
  if (p.nrot) ang.init(ang_s[warp_id()], p.inv_freq, j, rg, p.nrot);
  __syncthreads();
  uint4 *qo_t, *ko_t;
  bool fresh = true;
  auto pass = [&](uint4 (&raw)[2]) {
    uint64_t a[4], b[4], wt[4];
    unpack8(raw[0], a);
    unpack8(raw[1], b);
    load(raw[0], raw[1]);  // two passes ahead
    if (fresh) {
      qo_t = reinterpret_cast<uint4*>(p.q_out + cur.t * p.qo_stride);
      ko_t = reinterpret_cast<uint4*>(p.k_out + cur.t * p.ko_stride) - (long long)p.Hq * (D / 8);
      if (p.nrot) ang.at(p.pos ? p.pos[cur.t] : cur.t % p.S, j, rg);
    }
    const int row = cur.ps * RPP + rg;
    const bool is_k = row >= p.Hq;
    uint64_t sq = mul2(a[0], a[0]);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (i) sq = fma2(a[i], a[i], sq);
      sq = fma2(b[i], b[i], sq);
    }
    float ss = sum2(sq);
#pragma unroll
    for (int o = 1; o < LPR; o <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    const float r = rsqrtf(ss * (1.0f / D) + p.eps);
    const uint64_t r2 = pack2(r, r);
    const float4* w = w_s + (is_k ? 4 * LPR : 0);
    lds8<LPR>(w, j, wt);
#pragma unroll
    for (int i = 0; i < 4; ++i) a[i] = mul2(mul2(a[i], r2), wt[i]);
    lds8<LPR>(w + 2 * LPR, j, wt);
#pragma unroll
    for (int i = 0; i < 4; ++i) b[i] = mul2(mul2(b[i], r2), wt[i]);
    if (j < p.nrot) ang.template rotate<INTER, false>(a, b, j);
    if (row < rows) {
      uint4* dst = (is_k ? ko_t : qo_t) + row * (D / 8);
      dst[pa] = pack8(a);
      dst[pb] = pack8(b);
    }
    fresh = cur.next(p.slices, passes);
  };
#pragma unroll 1
  while (cur.live()) {
    pass(r0);
    if (!cur.live()) break;
    pass(r1);
  }
}

// CTAs [0, ctas_q) take the query heads, the others the key heads, so that a lane
// keeps the weight gradient of its 16 columns in registers.
template <int D, bool INTER>
__global__ void __launch_bounds__(kBwdWarps * 32, kBwdCtasPerSm) qk_norm_bwd(const QkParams p) {
  constexpr int LPR = D / 16, RPP = 32 / LPR;
  __shared__ float red[kBwdWarps][D];
  __shared__ float4 w_s[4 * LPR];
  __shared__ float4 ang_s[kBwdWarps][4 * LPR];
  const int lane = lane_id(), warp = warp_id(), j = lane % LPR, rg = lane / LPR;
  grid_dep_launch();
  grid_dep_wait();
  const bool is_k = (int)blockIdx.x >= p.ctas_q;
  const int cta = is_k ? blockIdx.x - p.ctas_q : blockIdx.x;
  const int ctas = is_k ? gridDim.x - p.ctas_q : p.ctas_q;
  const int heads = is_k ? p.H : p.Hq;
  const __nv_bfloat16* x_base = is_k ? p.k : p.q;
  const long long x_stride = is_k ? p.k_stride : p.q_stride, o_stride = is_k ? p.ko_stride : p.qo_stride;
  const float* g_base = is_k ? p.dk : p.dq;
  __nv_bfloat16* o_base = is_k ? p.k_out : p.q_out;
  const float* w = is_k ? p.wk : p.wq;
  int pa, pb;
  pieces<INTER>(j, p.nrot, pa, pb);
  const int passes = (heads + RPP - 1) / RPP, slices = is_k ? p.slices_k : p.slices;
  Passes cur;
  cur.task = cta * kBwdWarps + warp;
  cur.ntask = (uint32_t)p.T * slices;
  cur.step = ctas * kBwdWarps;
  cur.enter(slices, passes);
  uint64_t da[4] = {}, db[4] = {};
  stage_weights<D, INTER>(w_s, w, p.inv_freq, p.nrot, threadIdx.x, kBwdWarps * 32);
  Angles<LPR> ang;
  if (p.nrot) ang.init(ang_s[warp], p.inv_freq, j, rg, p.nrot);
  __syncthreads();
  bool fresh = true;
#pragma unroll 1
  while (cur.live()) {
    const int row = cur.ps * RPP + rg;
    uint4 xa = make_uint4(0, 0, 0, 0), xb = xa;
    float4 g0 = make_float4(0.f, 0.f, 0.f, 0.f), g1 = g0, g2 = g0, g3 = g0;
    if (row < heads) {
      const uint4* x = reinterpret_cast<const uint4*>(x_base + cur.t * x_stride + (size_t)row * D);
      const float4* g = reinterpret_cast<const float4*>(g_base + ((size_t)cur.t * heads + row) * D);
      xa = x[pa];
      xb = x[pb];
      g0 = g[2 * pa];
      g1 = g[2 * pa + 1];
      g2 = g[2 * pb];
      g3 = g[2 * pb + 1];
    }
    if (fresh && p.nrot) ang.at(p.pos ? p.pos[cur.t] : cur.t % p.S, j, rg);
    uint64_t a[4], b[4], wt[4];
    uint64_t ga[4] = {pack2(g0.x, g0.y), pack2(g0.z, g0.w), pack2(g1.x, g1.y), pack2(g1.z, g1.w)};
    uint64_t gb[4] = {pack2(g2.x, g2.y), pack2(g2.z, g2.w), pack2(g3.x, g3.y), pack2(g3.z, g3.w)};
    unpack8(xa, a);
    unpack8(xb, b);
    if (j < p.nrot) ang.template rotate<INTER, true>(ga, gb, j);  // g is now dL/dy
    uint64_t sq = 0, ex = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      sq = fma2(a[i], a[i], sq);
      sq = fma2(b[i], b[i], sq);
    }
    // a weight piece at a time, twice: the registers are short
    lds8<LPR>(w_s, j, wt);
#pragma unroll
    for (int i = 0; i < 4; ++i) ex = fma2(mul2(ga[i], wt[i]), a[i], ex);
    lds8<LPR>(w_s + 2 * LPR, j, wt);
#pragma unroll
    for (int i = 0; i < 4; ++i) ex = fma2(mul2(gb[i], wt[i]), b[i], ex);
    float ss = sum2(sq), es = sum2(ex);
#pragma unroll
    for (int o = 1; o < LPR; o <<= 1) {
      ss += __shfl_xor_sync(0xffffffffu, ss, o);
      es += __shfl_xor_sync(0xffffffffu, es, o);
    }
    const float r = rsqrtf(ss * (1.0f / D) + p.eps);
    const float back = -r * r * (es * (1.0f / D));
    const uint64_t r2 = pack2(r, r), back2 = pack2(back, back);
    if (row < heads) {
      __nv_bfloat16* dst = o_base + cur.t * o_stride + (size_t)row * D;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        da[i] = fma2(ga[i], mul2(a[i], r2), da[i]);
        db[i] = fma2(gb[i], mul2(b[i], r2), db[i]);
      }
      lds8<LPR>(w_s + 2 * LPR, j, wt);
#pragma unroll
      for (int i = 0; i < 4; ++i) b[i] = mul2(fma2(b[i], back2, mul2(gb[i], wt[i])), r2);
      reinterpret_cast<uint4*>(dst)[pb] = pack8(b);
      lds8<LPR>(w_s, j, wt);
#pragma unroll
      for (int i = 0; i < 4; ++i) a[i] = mul2(fma2(a[i], back2, mul2(ga[i], wt[i])), r2);
      reinterpret_cast<uint4*>(dst)[pa] = pack8(a);
    }
    fresh = cur.next(slices, passes);
  }
  // this CTA's sums over its rows, in a fixed order
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    float lo, hi, va, vb;
    unpack2(da[e >> 1], lo, hi);
    va = e & 1 ? hi : lo;
    unpack2(db[e >> 1], lo, hi);
    vb = e & 1 ? hi : lo;
#pragma unroll
    for (int o = LPR; o < 32; o <<= 1) {
      va += __shfl_xor_sync(0xffffffffu, va, o);
      vb += __shfl_xor_sync(0xffffffffu, vb, o);
    }
    if (rg == 0) {
      red[warp][8 * pa + e] = va;
      red[warp][8 * pb + e] = vb;
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < D; i += kBwdWarps * 32) {
    float v = 0.f;
    for (int u = 0; u < kBwdWarps; ++u) v += red[u][i];
    p.part[(size_t)blockIdx.x * D + i] = v + no_angle<INTER>(p.inv_freq, p.nrot, i);
  }
}

// dwq / dwk from the CTAs' sums: CTA = 32 columns of one of the two, 32 warps over the rows.
__global__ void __launch_bounds__(1024)
    qk_norm_dw(const float* part, int D, int ctas_q, int ctas, float* dwq, float* dwk) {
  __shared__ float red[32][33];
  grid_dep_launch();
  grid_dep_wait();
  const int nc = D / 32;
  const bool is_k = (int)blockIdx.x >= nc;
  const int col = (blockIdx.x % nc) * 32 + lane_id();
  const int lo = is_k ? ctas_q : 0, hi = is_k ? ctas : ctas_q;
  float v = 0.f;
#pragma unroll 4
  for (int i = lo + warp_id(); i < hi; i += 32) v += part[(size_t)i * D + col];
  red[warp_id()][lane_id()] = v;
  __syncthreads();
  // warp u sums column u
  v = red[lane_id()][warp_id()];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  float* dw = is_k ? dwk : dwq;
  if (dw && lane_id() == 0) dw[(blockIdx.x % nc) * 32 + warp_id()] = v;
}

kvpop_status check_common(const char* what, const void* q, long long q_stride, const void* k, long long k_stride, int b,
                          int S, int Hq, int H, int D, float eps, const float* inv_freq, int R, const void* qo,
                          long long qo_stride, const void* ko, long long ko_stride) {
  if (!q || !k || !qo || !ko) {
    set_last_error("%s: q, k and the outputs must be non-NULL", what);
    return KVPOP_ERR_INVALID_ARG;
  }
  if (b <= 0 || S <= 0 || Hq <= 0 || H <= 0) {
    set_last_error("%s: bad shape b=%d S=%d Hq=%d H=%d", what, b, S, Hq, H);
    return KVPOP_ERR_INVALID_ARG;
  }
  if (D != 64 && D != 128) {
    set_last_error("%s: D=%d unsupported (64 or 128)", what, D);
    return KVPOP_ERR_UNSUPPORTED;
  }
  if ((long long)b * S > 0x7fffffffll || Hq > 65535 || H > 65535) {
    set_last_error("%s: at most 2^31 - 1 tokens and 65535 heads", what);
    return KVPOP_ERR_UNSUPPORTED;
  }
  if (!(eps >= 0.0f) || eps > 3.0e38f) {
    set_last_error("%s: eps must be finite and >= 0", what);
    return KVPOP_ERR_INVALID_ARG;
  }
  if (R < 0 || R > D || (R > 0 && !inv_freq)) {
    set_last_error("%s: R=%d must be in [0, D], with inv_freq when R > 0", what, R);
    return KVPOP_ERR_INVALID_ARG;
  }
  if (R % 16 != 0) {
    set_last_error("%s: R=%d must be a multiple of 16", what, R);
    return KVPOP_ERR_UNSUPPORTED;
  }
  const long long strides[4] = {q_stride, qo_stride, k_stride, ko_stride};
  for (int i = 0; i < 4; ++i) {
    const long long row = (long long)(i < 2 ? Hq : H) * D;
    if (strides[i] < row && (long long)b * S > 1) {
      set_last_error("%s: a token stride of %lld is less than the heads' %lld values", what, strides[i], row);
      return KVPOP_ERR_INVALID_ARG;
    }
  }
  const uintptr_t am = reinterpret_cast<uintptr_t>(q) | reinterpret_cast<uintptr_t>(k) |
                       reinterpret_cast<uintptr_t>(qo) | reinterpret_cast<uintptr_t>(ko);
  if ((am & 15) || ((q_stride | k_stride | qo_stride | ko_stride) & 7)) {
    set_last_error("%s: q, k and the outputs must be 16-byte aligned with token strides that are multiples of 8", what);
    return KVPOP_ERR_UNSUPPORTED;
  }
  return KVPOP_OK;
}

// Warps that share one token.  A warp's time is its rounds times (passes of a task + the
// token's angles, worth about kAngleCost passes); shares of a token fill the last round
// and, with few tokens, the SMs.
constexpr float kAngleCost = 1.4f;
int pick_slices(long long T, int passes, long long warps) {
  int best = 1;
  float best_cost = 3.0e38f;
  for (int s = 1; s <= passes; ++s) {
    const float cost = (float)((T * s + warps - 1) / warps) * ((passes + s - 1) / s + kAngleCost);
    if (cost < best_cost) {
      best_cost = cost;
      best = s;
    }
    if (T * s > 16 * warps) break;  // more than 16 rounds: the last one hardly counts
  }
  return best;
}

}  // namespace
}  // namespace kvpop

using namespace kvpop;

extern "C" kvpop_status kvpop_qk_norm_rope(const void* q, int64_t q_stride, const void* k, int64_t k_stride, int b,
                                           int S, int Hq, int H, int D, const float* wq, const float* wk, float eps,
                                           const float* inv_freq, int R, int interleaved, const int32_t* pos,
                                           void* q_out, void* k_out, kvpop_stream stream) {
  const long long qo = (long long)Hq * D, ko = (long long)H * D;
  kvpop_status st = check_common("kvpop_qk_norm_rope", q, q_stride, k, k_stride, b, S, Hq, H, D, eps, inv_freq, R,
                                 q_out, qo, k_out, ko);
  if (st != KVPOP_OK) return st;
  QkParams p = {};
  p.q = (const __nv_bfloat16*)q;
  p.k = (const __nv_bfloat16*)k;
  p.q_stride = q_stride;
  p.k_stride = k_stride;
  p.wq = wq;
  p.wk = wk;
  p.inv_freq = inv_freq;
  p.pos = pos;
  p.q_out = (__nv_bfloat16*)q_out;
  p.k_out = (__nv_bfloat16*)k_out;
  p.qo_stride = qo;
  p.ko_stride = ko;
  p.T = b * S;
  p.S = S;
  p.Hq = Hq;
  p.H = H;
  p.nrot = R / 16;
  p.eps = eps;
  const int rpp = 512 / D, passes = (Hq + H + rpp - 1) / rpp;
  const int max_ctas = num_sms() * kCtasPerSm;
  p.slices = pick_slices(p.T, passes, (long long)max_ctas * kWarps);
  const long long ntask = (long long)p.T * p.slices;
  const long long ctas = (ntask + kWarps - 1) / kWarps;
  const dim3 grid((unsigned)(ctas < max_ctas ? ctas : max_ctas));
  auto kern = D == 128 ? (interleaved ? qk_norm_fwd<128, true> : qk_norm_fwd<128, false>)
                       : (interleaved ? qk_norm_fwd<64, true> : qk_norm_fwd<64, false>);
  return cuda_check(launch_pdl(kern, grid, dim3(kWarps * 32), 0, reinterpret_cast<cudaStream_t>(stream), p),
                    "kvpop_qk_norm_rope: launch");
}

extern "C" kvpop_status kvpop_qk_norm_rope_bwd_workspace_size(int D, size_t* bytes) {
  if (!bytes) {
    set_last_error("kvpop_qk_norm_rope_bwd_workspace_size: bytes is NULL");
    return KVPOP_ERR_INVALID_ARG;
  }
  if (D != 64 && D != 128) {
    set_last_error("kvpop_qk_norm_rope_bwd_workspace_size: D=%d unsupported (64 or 128)", D);
    return KVPOP_ERR_UNSUPPORTED;
  }
  *bytes = (size_t)kBwdMaxCtas * D * 4;
  return KVPOP_OK;
}

extern "C" kvpop_status kvpop_qk_norm_rope_bwd(const void* q, int64_t q_stride, const void* k, int64_t k_stride,
                                               const float* dq, const float* dk, int b, int S, int Hq, int H, int D,
                                               const float* wq, const float* wk, float eps, const float* inv_freq,
                                               int R, int interleaved, const int32_t* pos, void* dq_in,
                                               int64_t dq_stride, void* dk_in, int64_t dk_stride, float* dwq,
                                               float* dwk, void* workspace, size_t workspace_bytes,
                                               kvpop_stream stream) {
  kvpop_status st = check_common("kvpop_qk_norm_rope_bwd", q, q_stride, k, k_stride, b, S, Hq, H, D, eps, inv_freq, R,
                                 dq_in, dq_stride, dk_in, dk_stride);
  if (st != KVPOP_OK) return st;
  if (!dq || !dk || !workspace) {
    set_last_error("kvpop_qk_norm_rope_bwd: dq, dk and workspace must be non-NULL");
    return KVPOP_ERR_INVALID_ARG;
  }
  size_t need = 0;
  st = kvpop_qk_norm_rope_bwd_workspace_size(D, &need);
  if (st != KVPOP_OK) return st;
  if (workspace_bytes < need) {
    set_last_error("kvpop_qk_norm_rope_bwd: workspace of %zu bytes, %zu needed", workspace_bytes, need);
    return KVPOP_ERR_INVALID_ARG;
  }
  if (((reinterpret_cast<uintptr_t>(dq) | reinterpret_cast<uintptr_t>(dk)) & 15) ||
      (reinterpret_cast<uintptr_t>(workspace) & 255)) {
    set_last_error("kvpop_qk_norm_rope_bwd: dq and dk must be 16-byte, workspace 256-byte aligned");
    return KVPOP_ERR_UNSUPPORTED;
  }
  QkParams p = {};
  p.q = (const __nv_bfloat16*)q;
  p.k = (const __nv_bfloat16*)k;
  p.q_stride = q_stride;
  p.k_stride = k_stride;
  p.wq = wq;
  p.wk = wk;
  p.inv_freq = inv_freq;
  p.pos = pos;
  p.q_out = (__nv_bfloat16*)dq_in;
  p.k_out = (__nv_bfloat16*)dk_in;
  p.qo_stride = dq_stride;
  p.ko_stride = dk_stride;
  p.dq = dq;
  p.dk = dk;
  p.part = (float*)workspace;
  p.T = b * S;
  p.S = S;
  p.Hq = Hq;
  p.H = H;
  p.nrot = R / 16;
  p.eps = eps;
  const int rpp = 512 / D, pq = (Hq + rpp - 1) / rpp, pk = (H + rpp - 1) / rpp;
  const int max_ctas = min(num_sms() * kBwdCtasPerSm, kBwdMaxCtas);
  // the two kinds of CTAs in proportion to their passes
  const int share_q = max(1, min(max_ctas - 1, (int)(((long long)max_ctas * pq + (pq + pk) / 2) / (pq + pk))));
  const int share_k = max_ctas - share_q;
  p.slices = pick_slices(p.T, pq, (long long)share_q * kBwdWarps);
  p.slices_k = pick_slices(p.T, pk, (long long)share_k * kBwdWarps);
  const int ctas_q = (int)min((long long)share_q, ((long long)p.T * p.slices + kBwdWarps - 1) / kBwdWarps);
  const int ctas_k = (int)min((long long)share_k, ((long long)p.T * p.slices_k + kBwdWarps - 1) / kBwdWarps);
  p.ctas_q = ctas_q;
  cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
  auto kern = D == 128 ? (interleaved ? qk_norm_bwd<128, true> : qk_norm_bwd<128, false>)
                       : (interleaved ? qk_norm_bwd<64, true> : qk_norm_bwd<64, false>);
  st = cuda_check(launch_pdl(kern, dim3(ctas_q + ctas_k), dim3(kBwdWarps * 32), 0, cs, p),
                  "kvpop_qk_norm_rope_bwd: launch");
  if (st != KVPOP_OK || (!dwq && !dwk)) return st;
  return cuda_check(launch_pdl(qk_norm_dw, dim3(2 * D / 32), dim3(1024), 0, cs, (const float*)workspace, D, ctas_q,
                               ctas_q + ctas_k, dwq, dwk),
                    "kvpop_qk_norm_rope_bwd: weight gradient launch");
}
