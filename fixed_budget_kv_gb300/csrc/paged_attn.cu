// kvpop_paged_attn: causal attention of ragged chunks of new tokens over a paged cache.
//
// For query head h G + g of row r of a sequence with c new tokens and len slots:
// s_t = scale q . k_{t,h}, t < len - c + r + 1; lse = log sum exp s_t,
// O = sum exp(s_t - lse) v_t.
//
// A block of up to 256 rows (256 / G tokens of the G query heads of one KV head) meets each
// 128-slot tile of K and V that its last row sees once; the tiles come out of the pages by TMA
// boxes of a page, or of 128 slots of one.  Decode rows are bound by memory (one flop a byte a
// row), chunks by the tensor core and the softmax.
//
// Work split: an item is one (sequence, row block, KV head), in that order, and has units of
// setup and then for each tile, by what these take.  CTA c takes the c-th part of all units, one
// CTA an SM, however ragged the chunks and lengths, which only the device knows.  A CTA's tiles
// fall into segments of one item each, of at most kRunTiles, whose running maximum, sum and
// unnormalised O are added up in a slot of the workspace.  An item whose tiles are all a CTA's
// is finished by it; of the others a CTA has at most two (it begins inside one and ends inside
// another), in a slot each, and paged_merge joins the slots of an item in the order of the
// CTAs.  No atomics: the same call gives the same bits.
//
// Warp roles of paged_kernel (384 threads):
//   warp 0      TMA producer: one ring of K and V tiles in the order of their use
//   warp 1      TMEM allocation; issues tcgen05.mma
//   warp 2      query tiles of each segment
//   warp 3      the CTA's share of the units, handed to the others segment by segment
//   warps 4-7, 8-11  softmax, one thread a row (TMEM lane)
// The two softmax warpgroups are two streams that alternate, so that the tensor core works on
// one while the other is in its softmax.  A segment of more than 128 rows gives each its own row
// tile; a smaller one gives both the same rows and every other slot tile, and joins the two in
// the epilogue.  S = Q K^T lands in TMEM (fp32), becomes bf16 P in place, and O += P V reads P
// from TMEM.  Running maxima are moved lazily, when they grow by more than 2^8 (the weights'
// precision does not depend on their size).  P is rounded to bf16 for its product, as the tensor
// core wants the type of V: each weight by up to 2^-8 of itself, independently, which leaves O
// off by about 1.3e-3 of its size beside the 1.7e-3 of its own rounding.  The row sum is not
// rounded.
//
// The exponentials are ex2.approx.ftz and the logarithm of lse is __log2f: a few units of 2^-22 each,
// small beside the rounded weights, and beside the products' own fp32 roundings in lse.
//
// Measured (8 KV heads, G = 4, D = 128, one GB300, calls in a chain): one row each of 64 sequences
// of 500 .. 16 001 slots 185 us, 96% of the copy rate; 4096 tokens at the end of 32 768 slots
// 1.46-1.49 ms in a continuous run, at the power cap's 1.93 GHz, 1380-1410 TFLOP/s (72-73% of the burst
// rate; 1.35 ms in the first 50 ms, at 2.07 GHz), bound by the issue of products (1.26 ms without
// the softmax) and the hand-overs S -> softmax -> P V; a step of 12 sequences, two long chunks
// among ten short ones and decode rows, 181-185 us, 1050-1070 TFLOP/s (the chunks' rate, 15 us of
// merge, start and switches).  At D = 64 an event costs more than half as much: 4096 tokens over
// 32 768 slots 1.21 ms, 854 TFLOP/s.
#include <string.h>

#include <atomic>

#include "paged.cuh"
#include "segments.cuh"

namespace kvpop {
namespace {

constexpr int kThreads = 384;
constexpr int kKeys = 128;
constexpr int kBlockRows = 256;
constexpr int kBlockBytes = 128 * 128;  // 128 rows x 128 bytes
constexpr float kRescaleLog2 = 8.0f;
constexpr int kMergeThreads = 256;
// Units of a tile, and of setup, the time between the last tile of a segment and the first of the
// next.  A tile takes 1.9 us with two row tiles (bound by products and softmax) and 1.3 with one (by
// its way from memory): the mixed step of 12 sequences took 228 us with 2 : 1, 213 with 1 : 1, 200
// with 3 : 2.
__host__ __device__ constexpr int tile_units(int two) { return 2 + two; }
__host__ __device__ constexpr int setup_units(int two) { return 4 * tile_units(two); }
constexpr int kSegs = 4;  // segments between the walker and the last reader
// Tiles of a segment at most: the tensor core truncates what it adds to an accumulator, so sums of
// more than 2^15 keys are added up outside of it, in fp32 with rounding (prefix.cu has the figures).
// It also keeps the waits that last a segment far below their limit.
constexpr int kRunTiles = 256;
// Register split: warps 0-3 drop to kRegsIo, the softmax warpgroups rise to kRegsSoftmax.
constexpr int kRegsIo = 64;
constexpr int kRegsSoftmax = 216;
constexpr int kRegsNeeded = (128 * kRegsIo + 256 * kRegsSoftmax + kThreads - 1) / kThreads;

// An item that several CTAs share: its first row, head and rows, and the last of its CTAs.
// nrow = 0: none.
struct __align__(16) Split {
  int row0, h, nrow, c1;
};

struct AttnParams {
  CUtensorMap tq, tk, tv;
  Paged c;
  __nv_bfloat16* O;
  float* lse;
  Split* split;     // [CTA] the item that the CTA is the second to work on
  float2* part_ml;  // [CTA, 2 slots, 256 rows] (maximum in log2 units, sum)
  float4* part_o;   // [CTA, 2 slots, 2 row tiles, D / 4, 128 rows]: a warp's store is contiguous
  int Hq, G, log_g, toks;  // toks = 256 / G tokens of a row block
  float scale_log2;
};

// A sequence: rows [lo, lo + c), slots, row blocks and units (the host bounds the sum of all
// units by 2^31).  Blocks 0 .. nb - 2 are whole: block b sees slots below a + toks (b + 1),
// a = len - c; the last sees all.  A block that sees nothing has one tile all the same, for the
// rows' results.
struct Seq {
  int lo, c, len, nb, units;
};
// Tiles of the blocks before block m < nb.
__device__ __forceinline__ int tiles_before(int a, int log_t, int m) {
  int t = 0;
  if (a < 0) {
    // blocks that lie before slot 0: those with toks (b + 1) <= -a
    const int none = min(m, -a >> log_t);
    t = none;
    m -= none;
    a += none << log_t;  // > -toks, or m = 0
  }
  if (m == 0) return t;
  // sum over b < m of floor((a + toks (b + 1) + 127) / 128)
  const long long x = a + (1 << log_t) + 127;
  if (log_t >= 7) return t + m * (int)(x >> 7) + (int)((long long)m * (m - 1) / 2 << (log_t - 7));
  // floor((x + toks b) / 128) = floor((x / toks + b) / p), p = 128 / toks; sums of floor(j / p)
  const int log_p = 7 - log_t;
  auto sum = [&](long long n) {
    const long long q = n >> log_p;
    return (q * (q - 1) / 2 << log_p) + q * (n - (q << log_p));
  };
  const long long j = x >> log_t;
  return t + (int)(sum(j + m) - sum(j));
}
__device__ __forceinline__ int units_before(const AttnParams& p, const Seq& s, int m) {
  return tile_units(1) * tiles_before(s.len - s.c, 8 - p.log_g, m) + m * setup_units(1);
}
// Whether block b has two row tiles; all but the last do.
__device__ __forceinline__ int two_tiles(const AttnParams& p, const Seq& s, int b) {
  return (s.c - b * p.toks) << p.log_g > 128;
}
__device__ __forceinline__ Seq sequence(const AttnParams& p, int i) {
  Seq s;
  s.lo = p.c.lo(i);
  s.c = p.c.hi(i, s.lo) - s.lo;
  s.len = p.c.len(i);
  s.nb = (s.c + p.toks - 1) / p.toks;
  const int two = two_tiles(p, s, s.nb - 1);
  s.units = s.nb ? (units_before(p, s, s.nb - 1) + max(1, (s.len + kKeys - 1) / kKeys) * tile_units(two) + setup_units(two)) * p.c.H : 0;
  return s;
}

// One segment: tiles [kt0, kt0 + NT) of a row block of sequence i, head h.
struct __align__(16) Seg {
  int i, h, row0, nrow;  // first row of q and rows (up to 256, G for each token) of the block
  int kt0, NT, len, flags;
  int sees, pad[3];  // slots that the block's first row sees; less than 1: none
  // two row tiles, one a stream; otherwise one, its slot tiles alternating
  __device__ __forceinline__ bool two() const { return flags & 1; }
  // the last of the block's tiles, and this CTA had all the others
  __device__ __forceinline__ bool whole() const { return flags & 2; }
  // otherwise: 0 when an earlier CTA began the block, 1 when this one did
  __device__ __forceinline__ int slot() const { return flags >> 2 & 1; }
  // this CTA had the tiles before these: their result is in the slot
  __device__ __forceinline__ bool cont() const { return flags & 8; }
};

template <int NS>
struct Bars {
  uint64_t q_full, q_empty;
  uint64_t kv_full[NS], kv_empty[NS];
  uint64_t s_full[2], p_full[2];
  uint64_t o_full, o_empty;
  uint64_t ml_full;
  uint64_t seg_full[kSegs], seg_empty[kSegs];
  uint64_t drain;
};

template <int D>
struct Layout {
  static constexpr int DH = D / 64;
  static constexpr int NS = D == 128 ? 5 : 10;  // 32 KB or 16 KB tiles
  static constexpr int kTile = DH * kBlockBytes;
  static constexpr int q_off = 0;
  static constexpr int kv_off = q_off + 2 * kTile;
  static constexpr int bar_off = kv_off + NS * kTile;
  static constexpr int seg_off = bar_off + ((int)sizeof(Bars<NS>) + 15) / 16 * 16;
  static constexpr int ml_off = seg_off + kSegs * (int)sizeof(Seg);  // [stream][row] (maximum, sum)
  static constexpr int misc_off = ml_off + 2 * 128 * 8;
  static constexpr int total = misc_off + 16;
  static_assert(total <= 232448, "shared memory of one CTA");
};

template <int D>
__global__ void __launch_bounds__(kThreads, 1) paged_kernel(const __grid_constant__ AttnParams p) {
  using L = Layout<D>;
  constexpr int DH = L::DH, NS = L::NS;
  extern __shared__ __align__(1024) uint8_t smem[];  // no slack left to align by hand: the walker checks
  Bars<NS>* bars = reinterpret_cast<Bars<NS>*>(smem + L::bar_off);
  Seg* segs = reinterpret_cast<Seg*>(smem + L::seg_off);
  float2* ml_s = reinterpret_cast<float2*>(smem + L::ml_off);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::misc_off);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::misc_off + 4);
  const uint32_t sbase = smem_u32(smem);
  const int warp = warp_id(), lane = lane_id();

  if (threadIdx.x == 0) {
    mbar_init(&bars->q_full, 1);
    mbar_init(&bars->q_empty, 1);
    for (int i = 0; i < NS; ++i) {
      mbar_init(&bars->kv_full[i], 1);
      mbar_init(&bars->kv_empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bars->s_full[i], 1);
      mbar_init(&bars->p_full[i], 4);
    }
    mbar_init(&bars->o_full, 1);
    mbar_init(&bars->o_empty, 8);
    mbar_init(&bars->ml_full, 8);
    for (int i = 0; i < kSegs; ++i) {
      mbar_init(&bars->seg_full[i], 1);
      mbar_init(&bars->seg_empty[i], 11);  // producer, query tiles, MMA, 8 softmax warps
    }
    mbar_init(&bars->drain, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = *tmem_slot;
  // the previous kernel of the stream may still be running (programmatic launch):
  // wait for it before any global access; this CTA already holds its tensor memory
  grid_dep_wait();
  grid_dep_launch();

  auto fail = [&](int site, int detail) { give_up(p.c.status, site, detail, abort_flag); };
  // segment n, once the walker has written it; false at the end of the work
  auto get_seg = [&](int n, Seg& s) -> bool {
    if (!bar_wait(&bars->seg_full[n % kSegs], (n / kSegs) & 1, abort_flag)) {
      fail(SITE_PAGED_PRODUCER, 3);
      return false;
    }
    s = segs[n % kSegs];
    mbar_arrive(&bars->seg_empty[n % kSegs]);
    return s.NT > 0;
  };

  if (warp < 4) {
    setmaxnreg_dec<kRegsIo>();
    if (warp == 0) {
      // ------------------------------------------------------------ K / V producer
      // Lane (box, half) issues its part of a tile: boxes of a page, or of 128 slots of one, of
      // 64 columns.  Table entries are read three tiles ahead of their first use.
      if (lane == 0) {
        tma_prefetch_desc(&p.tk);
        tma_prefetch_desc(&p.tv);
      }
      const int log_box = min(p.c.log_page, 7), boxes = kKeys >> log_box;
      const int box = lane / DH, dh = lane - box * DH;
      const bool mine = box < boxes;
      const uint32_t dst = dh * kBlockBytes + (box << log_box) * 128;
      Seg s = {};
      Ring<NS> r;
      int loads = 0;
      bool ok = true;
      // the page of this lane's box of tile t; one past the last page (zeros) where there is none
      auto page_at = [&](int t) -> int {
        const int slot = (s.kt0 + t) * kKeys + (box << log_box);
        if (!mine || t >= s.NT || slot >= s.len) return p.c.pages;
        const int pg = p.c.page_of(s.i, slot);
        if (pg >= 0) return pg;
        if (dh == 0) report_page(p.c.status, s.i);
        return p.c.pages;
      };
      auto load = [&](const CUtensorMap* map, int t, int pg) {
        if (!bar_wait_warp(&bars->kv_empty[r.st], r.ph ^ 1, abort_flag)) {
          if (lane == 0) fail(SITE_PAGED_PRODUCER, 1);
          ok = false;
          return;
        }
        if (lane == 0) mbar_arrive_expect_tx(&bars->kv_full[r.st], L::kTile);
        __syncwarp();
        if (mine)
          tma_load_4d(smem + L::kv_off + r.st * L::kTile + dst, map, &bars->kv_full[r.st], dh * 64,
                      ((s.kt0 + t) * kKeys + (box << log_box)) & ((1 << p.c.log_page) - 1), s.h, pg);
        r.skip(1);
        ++loads;
      };
      for (int n = 0; ok; ++n) {
        if (!bar_wait_warp(&bars->seg_full[n % kSegs], (n / kSegs) & 1, abort_flag)) {
          if (lane == 0) fail(SITE_PAGED_PRODUCER, 3);
          break;
        }
        s = segs[n % kSegs];
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars->seg_empty[n % kSegs]);
        if (s.NT == 0) break;
        const bool one = !s.two();  // K runs two tiles ahead of V, with two row tiles one
        int pg[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) pg[u] = page_at(u);
        load(&p.tk, 0, pg[0]);
        if (ok && one && s.NT > 1) load(&p.tk, 1, pg[1]);
        for (int t = 0; ok && t < s.NT; ++t) {
          load(&p.tv, t, pg[0]);
          const int ahead = t + (one ? 2 : 1);
          if (ok && ahead < s.NT) load(&p.tk, ahead, one ? pg[2] : pg[1]);
          pg[0] = pg[1];
          pg[1] = pg[2];
          pg[2] = pg[3];
          pg[3] = page_at(t + 4);
        }
      }
      if (*abort_flag && lane == 0) {
        // given up: nobody has waited for the last loads, which must land before the CTA ends
        for (int i = 0; i < min(loads, NS); ++i) {
          const int seq = loads - 1 - i;
          bar_wait(&bars->kv_full[seq % NS], (seq / NS) & 1, nullptr);
        }
      }
    } else if (warp == 1) {
      // ------------------------------------------------------------ MMA issuer
      // A segment's events alternate between the streams: event e takes key tile e, or with
      // two row tiles row tile e & 1 and key tile e / 2.  S runs two events ahead of P V, into
      // the next segment, so S of a stream always follows P V of the stream's event before.
      // TMEM: S / P of stream w at column 128 w, O at 256 + 128 w.
      // The bookkeeping is in the way of every MMA.  The whole warp runs it, in step, and one
      // elected lane issues: the operands then live in uniform registers.  Places in the rings are
      // counted on.
      constexpr uint32_t idesc_qk = idesc_bf16(128, 128, 0);
      constexpr uint32_t idesc_pv = idesc_bf16(128, D, 1);
      const uint32_t q_lo = desc_lo(sbase + L::q_off, 16), k_lo = desc_lo(sbase + L::kv_off, 16),
                     v_lo = desc_lo(sbase + L::kv_off, DH > 1 ? kBlockBytes : 16);
      Ring<NS> k, v, base;  // the next K and V tile; the first load of the segment that K is in
      int an = 0, a_left = 0, a_NT = 0, bn = 0, b_left = 0;  // segment and events left of it, for S and for P V
      int b_rem = 0;                                         // key tiles left of b's segment
      bool a_two = false, b_two = false;
      uint32_t a_sub = 0, b_sub = 0, aw = 0, bw = 0;  // row tile; stream
      uint32_t a_new = 1, b_new = 2;                  // first event of a segment; first event of each stream in it
      uint32_t np = 0;                                // bit w: parity of stream w's next P
      bool ok = true;
      auto wait_bar = [&](uint64_t* bar, uint32_t ph, int detail) -> bool {
        if (!bar_wait_warp(bar, ph, abort_flag)) {
          if (lane == 0) fail(SITE_PAGED_MMA, detail);
          ok = false;
          return false;
        }
        return true;
      };
      // key tiles and mode of segment n; none at the end of the work
      auto fetch = [&](int n, int& NT, int& left, bool& two, bool last_reader) {
        left = 0;
        if (!wait_bar(&bars->seg_full[n % kSegs], (n / kSegs) & 1, 6)) return;
        // warp reductions of equal values: the results are known to be uniform
        NT = __reduce_max_sync(0xffffffffu, segs[n % kSegs].NT);
        two = __reduce_max_sync(0xffffffffu, segs[n % kSegs].flags) & 1;
        left = two ? 2 * NT : NT;
        if (last_reader && lane == 0) mbar_arrive(&bars->seg_empty[n % kSegs]);
      };
      // V of a segment comes after its first K tiles
      auto enter_v = [&](Ring<NS> at) {
        v = at;
        v.skip(b_two ? 1 : min(b_rem, 2));
      };
      auto issue_s = [&]() {
        if (a_new) {
          if (!wait_bar(&bars->q_full, an & 1, 1)) return;
          a_new = 0;
        }
        if (!a_sub && !wait_bar(&bars->kv_full[k.st], k.ph, 2)) return;
        tc_fence_after();
        const uint32_t d = tbase + 128 * aw, a0 = q_lo + a_sub * (L::kTile / 16), b0 = k_lo + k.st * (L::kTile / 16);
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
          const uint32_t off = ((ks >> 2) * kBlockBytes + (ks & 3) * 32) / 16;
          mma_ss_elect(d, a0 + off, b0 + off, idesc_qk, ks > 0 ? 1u : 0u);
        }
        mma_commit_elect(&bars->s_full[aw]);
        if (!a_two || a_sub) {
          mma_commit_elect(&bars->kv_empty[k.st]);
          k.skip(!a_two && a_left == a_NT ? 1 : 2);
        }
        if (a_two) a_sub ^= 1;
        aw ^= 1;
        if (--a_left == 0) {
          mma_commit_elect(&bars->q_empty);
          a_new = 1;
          base.jump(2 * a_NT);
          k = base;
          fetch(++an, a_NT, a_left, a_two, false);
        }
      };
      Ring<NS> b_base;
      int b_NT = 0;
      fetch(0, a_NT, a_left, a_two, false);
      fetch(0, b_NT, b_left, b_two, true);
      b_rem = b_NT;
      enter_v(b_base);
      for (int i = 0; i < 2 && ok && a_left; ++i) issue_s();
      while (ok && b_left) {
        if (!wait_bar(&bars->p_full[bw], (np >> bw) & 1, 3)) break;
        np ^= 1u << bw;
        if (!b_sub && !wait_bar(&bars->kv_full[v.st], v.ph, 4)) break;
        if (b_new == 2 && !wait_bar(&bars->o_empty, (bn & 1) ^ 1, 5)) break;
        tc_fence_after();
        const uint32_t d = tbase + 256 + 128 * bw, a0 = tbase + 128 * bw, b0 = v_lo + v.st * (L::kTile / 16);
#pragma unroll
        for (int ks = 0; ks < kKeys / 16; ++ks)
          mma_ts_elect(d, a0 + ks * 8, b0 + ks * (2048 / 16), idesc_pv, (b_new == 0 || ks > 0) ? 1u : 0u);
        if (!b_two || b_sub) {
          mma_commit_elect(&bars->kv_empty[v.st]);
          --b_rem;
          v.skip(b_two || b_rem >= 2 ? 2 : 1);
        }
        if (b_new) --b_new;
        if (b_two) b_sub ^= 1;
        bw ^= 1;
        if (--b_left == 0) {
          mma_commit_elect(&bars->o_full);
          b_new = 2;
          b_base.jump(2 * b_NT);
          fetch(++bn, b_NT, b_left, b_two, true);
          b_rem = b_NT;
          enter_v(b_base);
        }
        if (a_left && ok) issue_s();
      }
      // drain every issued MMA before teardown
      mma_commit_elect(&bars->drain);
      bar_wait_warp(&bars->drain, 0, nullptr);
    } else if (warp == 2 && lane == 0) {
      // ------------------------------------------------------------ query tiles
      tma_prefetch_desc(&p.tq);
      Seg s;
      int n = 0;
      for (; get_seg(n, s); ++n) {
        if (!bar_wait(&bars->q_empty, (n & 1) ^ 1, abort_flag)) {
          fail(SITE_PAGED_PRODUCER, 2);
          break;
        }
        const int tiles = s.two() ? 2 : 1;
        mbar_arrive_expect_tx(&bars->q_full, tiles * L::kTile);
        for (int i = 0; i < tiles; ++i)
          for (int dh = 0; dh < DH; ++dh)
            tma_load_4d(smem + L::q_off + i * L::kTile + dh * kBlockBytes, &p.tq, &bars->q_full, dh * 64, s.h * p.G,
                        s.row0 + i * (p.toks / 2), 0);
      }
      if (*abort_flag && n > 0) bar_wait(&bars->q_full, (n - 1) & 1, nullptr);  // as for K and V
    } else if (warp == 3) {
      // ------------------------------------------------------------ the CTA's share
      // lane l holds sequence j0 + l of a window of 32, and its first unit
      int U = 0, members = 0, j0 = 0, base = 0;
      Seq g;
      auto window = [&](int w0, int at) {  // sequences w0 .., the first of them at unit `at`; returns the unit after
        g = w0 + lane < p.c.n ? sequence(p, w0 + lane) : Seq{0, 0, 0, 0, 0};
        const int incl = scan_incl(g.units);
        j0 = w0;
        base = at + incl - g.units;
        return at + __shfl_sync(0xffffffffu, incl, 31);
      };
#pragma unroll 1
      for (int w0 = 0; w0 < p.c.n; w0 += 32) {
        U = window(w0, U);
        members = min(members, p.c.T + 1) + __reduce_add_sync(0xffffffffu, min(g.c, p.c.T));
      }
      Split split = {0, 0, 0, 0};
      if (members > p.c.T) {
        // sequences that overlap, which the interface rules out, could pass the host's bound on U: no work
        U = 0;
        if (blockIdx.x == 0 && lane == 0) report_error(p.c.status, KVPOP_ERR_INVALID_ARG, SITE_PAGED_ROWS, 5);
      }
      if (sbase & 1023) {
        // the tiles would miss their swizzle.  No work either: an early return would leave the
        // merge whatever the workspace held for this CTA's item
        U = 0;
        if (lane == 0) report_error(p.c.status, KVPOP_ERR_INTERNAL, SITE_INTERNAL_CHECK, 60);
      }
      const int C = min((int)gridDim.x, (U + 2) / 3);  // three units each: none has a part of a tile only
      const Share sh(U, max(C, 1));
      int u = 0, end = 0;
      if ((int)blockIdx.x < C) {
        u = sh.first(blockIdx.x);
        end = sh.first(blockIdx.x + 1);
      }
      if (p.c.n > 32 && u < end) {  // back to the window in which the share begins
        int at = 0;
#pragma unroll 1
        for (int w0 = 0; w0 < p.c.n; w0 += 32) {
          at = window(w0, at);
          if (u < at) break;
        }
      }
      bool own = false;  // this CTA began the item that u is in
      // the sequence, row block and head of the item that holds unit u, the item's units, and the
      // first of them; looked up once and counted on
      Seq q = {};
      int seq = 0, rb = 0, h = 0, per = 0, at = 0, two = 0, setup = 0;
      bool known = false;
      auto enter_block = [&]() {
        // slots that its last row sees
        const int sees = rb == q.nb - 1 ? q.len : q.len - q.c + (rb + 1) * p.toks;
        two = two_tiles(p, q, rb);
        setup = setup_units(two);
        per = max(1, (sees + kKeys - 1) / kKeys) * tile_units(two) + setup;
      };
      for (int n = 0;; ++n) {
        Seg s = {0, 0, 0, 0, 0, 0, 0, 0, 0, {0, 0, 0}};  // NT = 0 ends the work
        while (u < end && s.NT == 0) {
          if (!known) {
            // the sequence: the one of the window whose units these are
            const unsigned hit = __ballot_sync(0xffffffffu, g.units > 0 && base <= u && u < base + g.units);
            if (hit == 0) {
              if (j0 + 32 < p.c.n) window(j0 + 32, u);  // u is the window's end
              else end = u;  // only where lens or cu change under the call
              continue;
            }
            const int l = __ffs(hit) - 1, b = __shfl_sync(0xffffffffu, base, l);
            seq = j0 + l;
            q.lo = __shfl_sync(0xffffffffu, g.lo, l);
            q.c = __shfl_sync(0xffffffffu, g.c, l);
            q.len = __shfl_sync(0xffffffffu, g.len, l);
            q.nb = __shfl_sync(0xffffffffu, g.nb, l);
            // the row block: the last that begins at or before the unit
            int over = q.nb;
            rb = 0;
            while (over - rb > 1) {
              const int mid = (rb + over) >> 1;
              if ((long long)units_before(p, q, mid) * p.c.H <= u - b) rb = mid;
              else over = mid;
            }
            enter_block();
            at = b + units_before(p, q, rb) * p.c.H;
            h = (u - at) / per;
            at += h * per;
            known = true;
          }
          // this CTA's units of the item from here on, up to a run of tiles: [off, stop)
          const int off = u - at, stop = min(min(per, off + (end - u)), max(off, setup) + kRunTiles * tile_units(two));
          auto tile = [&](int x) { return two ? max(x - setup, 0) / tile_units(1) : max(x - setup, 0) / tile_units(0); };
          s.kt0 = tile(off);
          s.NT = tile(stop) - s.kt0;
          s.i = seq;
          s.h = h;
          s.row0 = q.lo + rb * p.toks;
          s.nrow = min(p.toks, q.c - rb * p.toks) * p.G;
          s.len = q.len;
          s.sees = q.len - q.c + rb * p.toks + 1;
          const bool cont = s.kt0 > 0 && n > 0;
          own = s.kt0 == 0 || (cont && own);
          s.flags = (s.nrow > 128 ? 1 : 0) | (own && stop == per ? 2 : 0) | (own ? 4 : 0) | (cont ? 8 : 0);
          if (n == 0 && s.kt0 > 0) {
            // the work begins inside an item; the second of its CTAs leaves word of it
            split = {s.row0, h, sh.cta_of(at + setup + tile_units(two) - 1) + 1 == (int)blockIdx.x ? s.nrow : 0, sh.cta_of(at + per - 1)};
          }
          u += stop - off;
          if (stop == per) {  // on to the next item
            at += per;
            if (++h == p.c.H) {
              h = 0;
              if (++rb == q.nb) known = false;
              else enter_block();
            }
          }
        }
        if (n == 0 && lane == 0) p.split[blockIdx.x] = split;
        if (!bar_wait_warp(&bars->seg_empty[n % kSegs], ((n / kSegs) & 1) ^ 1, abort_flag)) {
          if (lane == 0) fail(SITE_PAGED_PRODUCER, 4);
          break;
        }
        if (lane == 0) {
          segs[n % kSegs] = s;
          mbar_arrive(&bars->seg_full[n % kSegs]);
        }
        if (s.NT == 0) break;
      }
    }
  } else {
    setmaxnreg_inc<kRegsSoftmax>();
    // in line: a call leaves too few registers here
    auto fail_here = [&](int site, int detail) {
      report_error(p.c.status, KVPOP_ERR_TIMEOUT, site, detail);
      *abort_flag = 1;
    };
    // ------------------------------------------------------------ softmax
    const int w = (warp - 4) >> 2;  // stream
    const int quarter = warp & 3;
    const int row = quarter * 32 + lane;
    const uint32_t tl = tbase + ((uint32_t)(quarter * 32) << 16);
    const uint32_t s_col = 128 * w, o_col = 256 + 128 * w, o_oth = 256 + 128 * (w ^ 1);
    const float sl2 = p.scale_log2;
    const uint64_t s2 = pack2(sl2, sl2);
    uint32_t cnt = 0, par = 0, nml = 0;
    int sb = 0;
    float m_run = neg_inf(), l_run = 0.0f;  // of the key tiles in the slot
    bool ok = true;
    for (int n = 0; ok; ++n) {
      if (!warp_wait(&bars->seg_full[n % kSegs], (n / kSegs) & 1, abort_flag)) {
        if (lane == 0) fail_here(SITE_PAGED_SOFTMAX, 3);
        break;
      }
      const Seg& s = segs[n % kSegs];
      if (s.NT == 0) break;
      const bool two = s.two();
      const int a = w ^ par;  // row tile, or first key tile
      const int steps = two ? s.NT : (s.NT - a + 1) / 2;
      const int rrow = two ? 128 * a + row : row;  // row within the block
      const bool warp_on = rrow - lane < s.nrow, row_on = rrow < s.nrow;
      // slots that this row sees, and that the warp's first one does
      const int sees = s.sees + (rrow >> p.log_g), sees_w = s.sees + ((rrow - lane) >> p.log_g);
      float m_ref = neg_inf(), l = 0.0f;
      for (int i = 0; i < steps; ++i, ++cnt) {
        const int t = two ? i : 2 * i + a;
        if (!warp_wait(&bars->s_full[w], cnt & 1, abort_flag)) {
          if (lane == 0) fail_here(SITE_PAGED_SOFTMAX, 1);
          ok = false;
          break;
        }
        tc_fence_after();
        const int slot0 = (s.kt0 + t) * kKeys;
        if (warp_on) {
          // the whole S row of this thread (128 fp32) in registers; slots that the row does not see -> -inf
          uint32_t sr[4][32];
#pragma unroll
          for (int ch = 0; ch < 4; ++ch) tmem_ld32(tl + s_col + ch * 32, sr[ch]);
#pragma unroll
          for (int ch = 0; ch < 4; ++ch) tmem_wait_ld_dep(sr[ch]);
          if (sees_w < slot0 + kKeys) {
#pragma unroll
            for (int ch = 0; ch < 4; ++ch)
              if (sees_w < slot0 + ch * 32 + 32) {
#pragma unroll
                for (int c = 0; c < 32; ++c)
                  if (slot0 + ch * 32 + c >= sees) sr[ch][c] = 0xff800000u;
              }
          }
          // P = exp2(s * scale_log2 - m) as bf16, written over S.  Returns the row's sum
          auto weights = [&]() -> float {
            const float nm = (m_ref == neg_inf()) ? 0.0f : -m_ref * sl2;
            const uint64_t n2 = pack2(nm, nm);
            uint64_t lacc = 0;
#pragma unroll
            for (int ch = 0; ch < 4; ++ch) {
              uint32_t pk[16];
#pragma unroll
              for (int c = 0; c < 32; c += 2) {
                const uint64_t xx = fma2(pack2(__uint_as_float(sr[ch][c]), __uint_as_float(sr[ch][c + 1])), s2, n2);
                float e0, e1;
                unpack2(xx, e0, e1);
                const float p0 = ex2_approx(e0), p1 = ex2_approx(e1);
                lacc = add2(lacc, pack2(p0, p1));
                pk[c >> 1] = pack_bf16x2(p0, p1);
              }
              tmem_st16(tl + s_col + ch * 16, pk);
            }
            float l0, l1;
            unpack2(lacc, l0, l1);
            return l0 + l1;
          };
          // The running reference serves as long as no row's weights sum up to more than 2^8: then none of
          // them is larger, which is what moves it.  So most tiles need no maximum (a chunk of 4096 tokens
          // over 32 768 slots 1.46 ms against 1.54); the others are done again from the registers.
          float lt = 0.0f;
          bool known = __all_sync(0xffffffffu, m_ref != neg_inf()), last = false;
#pragma unroll 1
          while (true) {
            if (known) {
              lt = weights();
              if (last || !__any_sync(0xffffffffu, lt > 256.0f)) break;
              // these weights are written over: stores to the same columns are in order only behind a wait
              tmem_wait_st();
            }
            float mt = neg_inf();
#pragma unroll
            for (int ch = 0; ch < 4; ++ch) mt = fmaxf(mt, max32(sr[ch]));
            const float m_new = fmaxf(m_ref, mt);
            const bool need = (m_new - m_ref) * sl2 > kRescaleLog2;  // true when m_ref == -inf and mt finite
            float alpha = 1.0f;
            if (need) {
              alpha = ex2_approx((m_ref - m_new) * sl2);
              l *= alpha;
              m_ref = m_new;
            }
            if (__any_sync(0xffffffffu, need) && i > 0) {
              // O of this stream's last event is complete: S of this one was issued after it
#pragma unroll 1
              for (int cd = 0; cd < D / 32; ++cd) {
                uint32_t r[32];
                tmem_ld32(tl + o_col + cd * 32, r);
                tmem_wait_ld_dep(r);
#pragma unroll
                for (int c = 0; c < 32; ++c) r[c] = __float_as_uint(__uint_as_float(r[c]) * alpha);
                tmem_st32(tl + o_col + cd * 32, r);
              }
            }
            known = last = true;
          }
          l += lt;
          tmem_wait_st();
        }
        const int left = s.len - slot0;  // slots of this tile within the length
        if (left < kKeys) {
          // V rows behind the length hold anything, and 0 * NaN would be NaN: zero them
          const int seq = sb + pos_v(two, s.NT, t), st = seq % NS;
          if (!warp_wait(&bars->kv_full[st], (seq / NS) & 1, abort_flag)) {
            if (lane == 0) fail_here(SITE_PAGED_SOFTMAX, 2);
            ok = false;
            break;
          }
          if (row >= left) {
#pragma unroll
            for (int dh = 0; dh < DH; ++dh) {
              uint4* r = reinterpret_cast<uint4*>(smem + L::kv_off + st * L::kTile + dh * kBlockBytes + row * 128);
#pragma unroll
              for (int u = 0; u < 8; ++u) r[u] = make_uint4(0, 0, 0, 0);
            }
          }
          fence_proxy_async_smem();
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars->p_full[w]);
      }
      if (!ok) break;
      // ---------------------------------------------------------- epilogue
      const size_t orow = (size_t)(s.row0 + (rrow >> p.log_g)) * p.Hq + s.h * p.G + (rrow & (p.G - 1));
      float w_own = 1.0f, w_oth = 0.0f;
      // no weight: -inf; a NaN among the scores keeps a finite maximum and travels in l
      float m2 = l == 0.0f ? neg_inf() : (m_ref == neg_inf() ? 0.0f : m_ref * sl2);
      if (!warp_wait(&bars->o_full, n & 1, abort_flag)) {
        if (lane == 0) fail_here(SITE_PAGED_EPILOGUE, 1);
        break;
      }
      tc_fence_after();
      if (!two) {
        // join the two streams.  O of this segment is complete, so every warp has left the
        // segment before (o_empty) and has read its exchange: one buffer is enough.
        ml_s[w * 128 + row] = make_float2(m2, l);
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars->ml_full);
        if (!warp_wait(&bars->ml_full, nml & 1, abort_flag)) {
          if (lane == 0) fail_here(SITE_PAGED_EPILOGUE, 2);
          break;
        }
        ++nml;
        const float2 o = ml_s[(w ^ 1) * 128 + row];
        const float M = fmaxf(m2, o.x);
        w_own = m2 != neg_inf() ? ex2_approx(m2 - M) : 0.0f;
        w_oth = o.x != neg_inf() ? ex2_approx(o.x - M) : 0.0f;
        l = l * w_own + o.y * w_oth;
        m2 = M;
      }
      // a single-tile segment's columns are shared out between the two streams
      const int c_lo = two ? 0 : w * (D / 2), c_n = two ? D : D / 2;
      const bool both = !two && s.NT > 1, mine = two || steps > 0;
      float w_run = 0.0f;
      if (s.cont()) {
        const float M = fmaxf(m_run, m2);
        const float f = m2 != neg_inf() ? ex2_approx(m2 - M) : 0.0f;
        w_run = m_run != neg_inf() ? ex2_approx(m_run - M) : 0.0f;
        w_own *= f;
        w_oth *= f;
        l = l * f + l_run * w_run;
        m2 = M;
      }
      m_run = m2;
      l_run = l;
      const bool adds = w_run != 0.0f;
      if (s.whole()) {
        const float inv = l != 0.0f ? 1.0f / l : 0.0f;
        w_own *= inv;
        w_oth *= inv;
        w_run *= inv;
      }
      if (warp_on) {
        const size_t slot = (size_t)blockIdx.x * 2 + s.slot();
        float4* po = p.part_o + (slot * 2 + (two ? a : 0)) * (D / 4) * 128 + row;
#pragma unroll 1
        for (int c0 = c_lo; c0 < c_lo + c_n; c0 += 32) {
          uint32_t r[32];
          tmem_ld32(tl + (mine ? o_col : o_oth) + c0, r);
          tmem_wait_ld_dep(r);
          float v[32];
#pragma unroll
          for (int c = 0; c < 32; ++c) v[c] = __uint_as_float(r[c]) * (mine ? w_own : w_oth);
          if (both) {
            tmem_ld32(tl + o_oth + c0, r);
            tmem_wait_ld_dep(r);
#pragma unroll
            for (int c = 0; c < 32; ++c) v[c] += __uint_as_float(r[c]) * w_oth;
          }
          if (row_on && adds) {
#pragma unroll
            for (int u = 0; u < 8; ++u) {
              const float4 y = po[(size_t)(c0 / 4 + u) * 128];
              v[4 * u] += w_run * y.x;
              v[4 * u + 1] += w_run * y.y;
              v[4 * u + 2] += w_run * y.z;
              v[4 * u + 3] += w_run * y.w;
            }
          }
          if (row_on && s.whole()) {
            uint4* dst = reinterpret_cast<uint4*>(p.O + orow * D + c0);
#pragma unroll
            for (int u = 0; u < 4; ++u)
              dst[u] = make_uint4(pack_bf16x2(v[8 * u], v[8 * u + 1]), pack_bf16x2(v[8 * u + 2], v[8 * u + 3]),
                                  pack_bf16x2(v[8 * u + 4], v[8 * u + 5]), pack_bf16x2(v[8 * u + 6], v[8 * u + 7]));
          } else if (row_on) {
#pragma unroll
            for (int u = 0; u < 8; ++u)
              po[(size_t)(c0 / 4 + u) * 128] = make_float4(v[4 * u], v[4 * u + 1], v[4 * u + 2], v[4 * u + 3]);
          }
          __syncwarp();
        }
        if (row_on && c_lo == 0) {
          if (s.whole())
            p.lse[orow] = l != 0.0f ? (m2 + __log2f(l)) * 0.69314718055994531f : neg_inf();
          else
            p.part_ml[slot * kBlockRows + rrow] = make_float2(m2, l);
        }
      }
      tc_fence_before();
      par ^= (two ? 2 * s.NT : s.NT) & 1;
      sb += 2 * s.NT;
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&bars->o_empty);
        mbar_arrive(&bars->seg_empty[n % kSegs]);
      }
    }
  }

  // ------------------------------------------------------------ teardown
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tbase, 512);
  }
}

// The items that several of paged_kernel's CTAs shared, each joined from the slots of its CTAs in
// their order: CTA (x, y) takes rows y of those whose second CTA is in the x-th part of the CTAs.
// Thread (part, c4, row) takes four columns of ROWS rows and every parts-th slot, SLOTS of them at a
// time; the parts are joined through shared memory.  Decode rows have many slots of few rows, blocks
// of a chunk two or three slots of 256: with one row a thread the mixed step of 12
// sequences spent 22 us here, with four 15.
template <int D, int ROWS, int SLOTS>
__global__ void __launch_bounds__(kMergeThreads, ROWS == 1 ? 4 : 2) paged_merge(const __grid_constant__ AttnParams p, int ctas, int parts) {
  __shared__ float2 ml_s[kMergeThreads];
  __shared__ float4 o_s[kMergeThreads];
  static_assert(ROWS == 1 || SLOTS <= 2, "registers");
  grid_dep_launch();
  grid_dep_wait();
  const int wide = kMergeThreads / parts, rows = wide / (D / 4);
  const int part = threadIdx.x / wide, x = threadIdx.x - part * wide, c4 = x / rows;
  const int r0 = blockIdx.y * rows * ROWS + x - c4 * rows;  // and every rows-th after it
  const int lo = (int)((long long)ctas * blockIdx.x / gridDim.x), hi = (int)((long long)ctas * (blockIdx.x + 1) / gridDim.x);
  for (int w0 = lo; w0 < hi; w0 += 32) {
    const Split mine = w0 + lane_id() < hi ? p.split[w0 + lane_id()] : Split{0, 0, 0, 0};
    unsigned todo = __ballot_sync(0xffffffffu, (int)blockIdx.y * rows * ROWS < mine.nrow);
    while (todo) {  // the same in every warp
      const int src = __ffs(todo) - 1;
      todo &= todo - 1;
      const int row0 = __shfl_sync(0xffffffffu, mine.row0, src), h = __shfl_sync(0xffffffffu, mine.h, src),
                nrow = __shfl_sync(0xffffffffu, mine.nrow, src), c1 = __shfl_sync(0xffffffffu, mine.c1, src);
      const int c0 = w0 + src - 1;
      float M[ROWS], l[ROWS];
      float4 o[ROWS];
#pragma unroll
      for (int u = 0; u < ROWS; ++u) {
        M[u] = neg_inf();
        l[u] = 0.0f;
        o[u] = make_float4(0.f, 0.f, 0.f, 0.f);
      }
      auto add = [](const float2& ml, const float4& y, float m, float& l, float4& o) {
        const float f = ml.x != neg_inf() ? ex2_approx(ml.x - m) : 0.0f;
        l += f * ml.y;
        if (ml.x != neg_inf()) {
          o.x += f * y.x;
          o.y += f * y.y;
          o.z += f * y.z;
          o.w += f * y.w;
        }
      };
      for (int c = c0 + part; c <= c1; c += SLOTS * parts) {
        float2 ml[ROWS][SLOTS];
        float4 y[ROWS][SLOTS];
#pragma unroll
        for (int u = 0; u < ROWS; ++u)
#pragma unroll
          for (int k = 0; k < SLOTS; ++k) {
            const int cc = c + k * parts, r = r0 + u * rows;
            ml[u][k] = make_float2(neg_inf(), 0.0f);
            y[u][k] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (cc <= c1 && r < nrow) {
              const size_t slot = (size_t)cc * 2 + (cc == c0 ? 1 : 0);  // the item begins in c0's share
              ml[u][k] = p.part_ml[slot * kBlockRows + r];
              y[u][k] = p.part_o[((slot * 2 + (r >> 7)) * (D / 4) + c4) * 128 + (r & 127)];
            }
          }
#pragma unroll
        for (int u = 0; u < ROWS; ++u) {
          float m = M[u];
#pragma unroll
          for (int k = 0; k < SLOTS; ++k) m = fmaxf(m, ml[u][k].x);
          if (m != neg_inf()) {
            const float f = M[u] != neg_inf() ? ex2_approx(M[u] - m) : 0.0f;
            l[u] *= f;
            o[u].x *= f, o[u].y *= f, o[u].z *= f, o[u].w *= f;
            M[u] = m;
#pragma unroll
            for (int k = 0; k < SLOTS; ++k) add(ml[u][k], y[u][k], m, l[u], o[u]);
          }
        }
      }
      if (parts > 1) {  // ROWS = 1
        ml_s[threadIdx.x] = make_float2(M[0], l[0]);
        o_s[threadIdx.x] = o[0];
        __syncthreads();
        if (part == 0) {
          for (int k = 1; k < parts; ++k) M[0] = fmaxf(M[0], ml_s[x + k * wide].x);
          l[0] = 0.0f;
          o[0] = make_float4(0.f, 0.f, 0.f, 0.f);
          for (int k = 0; M[0] != neg_inf() && k < parts; ++k) add(ml_s[x + k * wide], o_s[x + k * wide], M[0], l[0], o[0]);
        }
      }
#pragma unroll
      for (int u = 0; u < ROWS; ++u) {
        const int r = r0 + u * rows;
        if (part == 0 && r < nrow) {
          const size_t orow = (size_t)(row0 + (r >> p.log_g)) * p.Hq + h * p.G + (r & (p.G - 1));
          const float inv = l[u] != 0.0f ? 1.0f / l[u] : 0.0f;
          *reinterpret_cast<uint2*>(p.O + orow * D + 4 * c4) =
              make_uint2(pack_bf16x2(o[u].x * inv, o[u].y * inv), pack_bf16x2(o[u].z * inv, o[u].w * inv));
          if (c4 == 0) p.lse[orow] = l[u] != 0.0f ? (M[u] + __log2f(l[u])) * 0.69314718055994531f : neg_inf();
        }
      }
      if (parts > 1) __syncthreads();
    }
  }
}

// A bound on the units of a call, and the CTAs of paged_kernel.
int max_ctas(int T, int n, int G, int H, long long slots) {
  const long long tiles = (n + (long long)T * G / kBlockRows) * H * ((slots + kKeys - 1) / kKeys);
  return (int)min((long long)num_sms(), 4 * tiles);  // at least three units a CTA
}
size_t round256(size_t x) { return (x + 255) / 256 * 256; }
size_t ml_offset(int ctas) { return round256((size_t)ctas * sizeof(Split)); }
size_t o_offset(int ctas) { return ml_offset(ctas) + (size_t)ctas * 2 * kBlockRows * 8; }

template <int D>
kvpop_status launch(AttnParams& prm, int ctas, cudaStream_t cs) {
  using L = Layout<D>;
  auto kern = paged_kernel<D>;
  kvpop_status st = KVPOP_OK;
  static std::atomic<uint64_t> ready{0};  // bit d: the kernel is set up on device d
  const int dev = current_device();
  if (dev >= 64 || !(ready.load(std::memory_order_acquire) >> dev & 1)) {
    st = cuda_check(cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, L::total),
                    "kvpop_paged_attn: smem attribute");
    if (st != KVPOP_OK) return st;
    // the register re-split must fit in the launch allocation (granule: 8 per thread)
    cudaFuncAttributes fa;
    st = cuda_check(cudaFuncGetAttributes(&fa, kern), "kvpop_paged_attn: attributes");
    if (st != KVPOP_OK) return st;
    if (((fa.numRegs + 7) / 8) * 8 < kRegsNeeded) {
      set_last_error("kvpop_paged_attn: kernel built with %d registers per thread, %d needed", fa.numRegs, kRegsNeeded);
      return KVPOP_ERR_INTERNAL;
    }
    if (dev < 64) ready.fetch_or(1ull << dev, std::memory_order_release);
  }
  st = cuda_check(launch_pdl(kern, dim3(ctas), dim3(kThreads), L::total, cs, prm), "kvpop_paged_attn: launch");
  if (st != KVPOP_OK) return st;
  // There are at most `items` items, of at most `most` rows, and at most one a CTA that several CTAs share.
  // With few items for the CTAs a thread takes about four slots of a row, and its CTA at least four rows
  // (two sectors of a slot's columns); otherwise four rows, of all slots.
  const long long rows_all = (long long)prm.c.T * prm.G;
  const long long items = prm.c.H * (prm.c.n + rows_all / kBlockRows);
  const int most = prm.c.cu ? (int)min((long long)kBlockRows, rows_all) : prm.G;
  int parts = 1;
  while (kMergeThreads / (D / 4) / parts > 4 && ctas > 4 * parts * items) parts *= 2;
  const bool few = ctas > 4 * items || most <= kMergeThreads / (D / 4);
  const int rows = kMergeThreads / (D / 4) / parts * (few ? 1 : 4);
  const dim3 grid((unsigned)min((long long)ctas, items), (most + rows - 1) / rows);
  return cuda_check(launch_pdl(few ? paged_merge<D, 1, 4> : paged_merge<D, 4, 2>, grid, dim3(kMergeThreads), 0, cs, prm, ctas, parts),
                    "kvpop_paged_attn: merge launch");
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
  const int ctas = max_ctas(T, n, Hq / H, H, (long long)max_pages * page);
  *bytes = o_offset(ctas) + (size_t)ctas * 2 * kBlockRows * D * 4;
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
  const int G = Hq / H, box = min(page, kKeys);
  const uint64_t dq[4] = {(uint64_t)D, (uint64_t)Hq, (uint64_t)T, 1};
  const uint64_t sq[3] = {(uint64_t)D * 2, (uint64_t)Hq * D * 2, (uint64_t)T * Hq * D * 2};
  const uint32_t bq[4] = {64, (uint32_t)G, (uint32_t)(128 / G), 1};
  const uint64_t dk[4] = {(uint64_t)D, (uint64_t)page, (uint64_t)H, (uint64_t)pages};
  const uint64_t sk[3] = {(uint64_t)D * 2, (uint64_t)page * D * 2, (uint64_t)kp_stride * 2};
  const uint64_t sv[3] = {(uint64_t)D * 2, (uint64_t)page * D * 2, (uint64_t)vp_stride * 2};
  const uint32_t bk[4] = {64, (uint32_t)box, 1, 1};
  if (!make_tmap_4d(&prm.tq, q, dq, sq, bq) || !make_tmap_4d(&prm.tk, kp, dk, sk, bk) ||
      !make_tmap_4d(&prm.tv, vp, dk, sv, bk))
    return KVPOP_ERR_CUDA;
  const int ctas = max_ctas(T, n, G, H, (long long)max_pages * page);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  prm.O = (__nv_bfloat16*)O;
  prm.lse = lse;
  prm.split = reinterpret_cast<Split*>(ws);
  prm.part_ml = reinterpret_cast<float2*>(ws + ml_offset(ctas));
  prm.part_o = reinterpret_cast<float4*>(ws + o_offset(ctas));
  prm.Hq = Hq;
  prm.G = G;
  prm.log_g = 0;
  while ((1 << prm.log_g) < G) ++prm.log_g;
  prm.toks = kBlockRows / G;
  prm.scale_log2 = (scale > 0.0f ? scale : 1.0f / sqrtf((float)D)) * 1.4426950408889634f;
  cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
  return D == 128 ? launch<128>(prm, ctas, cs) : launch<64>(prm, ctas, cs);
}
