// kvpop_paged_mass: the attention weight that each key of a paged cache receives from a chunk's
// rows: scores_t = decay scores_t + sum over rows r >= t - (len - c), heads g < G of
// exp(scale q_{r,hG+g} . k_t - lse_{r,hG+g}).
//
// The transposed product S' = K Q^T has a key in each TMEM lane, so that a warp sums its own keys'
// rows and exchanges nothing but four threads' parts at an item's end; every term is a probability,
// so a plain fp32 sum needs no running maximum.  A CTA holds a block of a head's slots, four 128-slot tiles of K (narrow) or two
// (wide), while query tiles of 128 (256) columns, tokens by the G heads, stream past.  Chunks are
// bound by the tensor core beside one exponential a (row, slot); decode rows and observation
// windows by reading K.
//
// Work split: an item is one (sequence, block of slots, KV head), in that order, and has kSetup
// units of setup and one for each query tile that sees the block.  CTA c takes the c-th part of
// all units, one CTA an SM.  An item whose query tiles are all a CTA's is finished by it; of the
// others a CTA has at most two, in a slot of the workspace each, and mass_merge adds the slots of
// an item up in the order of the CTAs.  No atomics: the same call gives the same bits.
//
// Warp roles of mass_kernel (640 threads):
//   warp 0       TMA producer of K
//   warp 1       TMEM allocation; issues tcgen05.mma
//   warp 2       query tiles and their -lse, in log2 units
//   warp 3       the CTA's share of the units and its table entries, handed to the others
//                segment by segment
//   warps 4-19   four warpgroups that sum 128 columns each
// TMEM columns are handed back as soon as they are in registers, and the tensor core works on the
// other tiles meanwhile.  A thread sums a tile's columns by themselves before it adds them to its total:
// long chunks would lose digits in one running sum.  A tile with masked columns is taken 32 columns
// at a time: those before a warp's first key are not read, and what a key does not see becomes -inf
// before the same sum (512 tokens, G = 8, over 16 384 slots 130 us with a conditional sum, 115 so).
// Where such a tile has a row whose lse is NaN, that -inf alone would not keep it from the slots that the
// row does not see: a path of its own masks the lse too (104 us for the decode rows below without it).
// The exponentials are ex2.approx.ftz, within a few units of 2^-22 of themselves.
//
// Measured (8 KV heads, G = 4, D = 128, one GB300, calls in a chain): one row each of 64 sequences
// of 500 .. 16 001 slots 106 us, 86% of the copy rate; 32 rows over 131 072 slots 52 us, 78%;
// 4096 tokens over 32 768 slots 0.70-0.73 ms in a continuous run, at the power cap's 1.93 GHz, 1410-1470
// TFLOP/s (73-76% of the burst rate; 0.65 ms in the first 50 ms, at 2.07 GHz), bound by
// the products beside the exponentials (a step before, at 0.69: 0.62 without the exponentials, 0.56
// without the loads of lse either).  At D = 64 0.58 ms, 882 TFLOP/s.
#include <string.h>

#include <atomic>

#include "paged.cuh"
#include "segments.cuh"

namespace kvpop {
namespace {

constexpr int kThreads = 640;
constexpr int kKeys = 128;
// Two forms of the kernel.  Narrow: a block of four tiles of K against query tiles of up to 128
// columns, one summing warpgroup a tile.  Wide: two tiles against 256 columns, two warpgroups a tile.
// The issuing thread takes about 85 cycles for a product's instruction and 300 between two tiles, the
// tensor core 65 for 128 columns and 130 for 256: wide keeps it busy (4096 tokens over 32 768 slots
// 742 us against 800), narrow has twice the keys on their way from memory (decode rows).
template <bool WIDE>
struct Form {
  static constexpr int kTiles = WIDE ? 2 : 4;
  static constexpr int kCols = WIDE ? 256 : 128;
  static constexpr int kBlockKeys = kTiles * kKeys;
};
constexpr int kBlockBytes = 128 * 128;  // 128 rows x 128 bytes
constexpr int kBoxes = kKeys / kMinPage;  // of a tile, at most
static_assert(Form<false>::kTiles * kBoxes == 32, "one table entry a lane");
// Loading a block of K and changing over to it, in query tiles.
constexpr int kSetup = 2;
constexpr int kSegs = 4;
// Query tiles of a segment at most: keeps the waits that last one far below their limit.
constexpr int kRunTiles = 256;
constexpr int kLseStages = 3;

// An item that several CTAs share, and the last of them.  h = -1: none.
struct __align__(16) Split {
  int i, h, block, c1;
};

struct MassParams {
  CUtensorMap tq, tk;
  Paged c;
  const float* lse;
  float* scores;
  Split* split;  // [CTA] the item that the CTA is the second to work on
  float* part;   // [CTA, 2 slots, keys of a block]
  int Hq, G, log_g, log_p;  // query tiles of 2^log_p tokens
  int q_bytes;              // of a query tile's box and 64 columns
  int block_keys;
  int own_tiles;  // query tiles as long as a block of slots; 0 in the narrow form
  float scale_log2, decay;
  float limit;  // a product up to it stays finite when it is scaled
};

// A sequence: rows [lo, lo + c), slots, blocks of slots, query tiles and units.  A sequence without
// rows has one query tile all the same, without columns: its scores fade.
struct Seq {
  int lo, c, len, nb, nq, units;
};
// The first query tile that sees slot t.
__device__ __forceinline__ int first_tile(int a, int log_p, int t) { return max(0, t - a) >> log_p; }
// Units of setup of block b of slots.  A block with the chunk's own slots has masked query tiles, which
// take half as long again or more in the wide form (2048 tokens, G = 16, over 8192 slots 207 us without
// this, 176 with, 180 with a whole tile each; the narrow form loses by any).
__device__ __forceinline__ int setup_units(const MassParams& p, const Seq& s, int b) {
  return kSetup + ((b + 1) * p.block_keys > s.len - s.c ? min(p.own_tiles, s.nq) / 2 : 0);
}
// Units of blocks 0 .. m - 1 for one head.
__device__ __forceinline__ int units_before(const MassParams& p, const Seq& s, int m) {
  const int a = s.len - s.c;
  // blocks that begin at or behind slot a, from b0 on, are not seen by the first tokens: by
  // f0, f0 + block_keys / tokens, ... query tiles
  const int b0 = a > 0 ? (a + p.block_keys - 1) / p.block_keys : 0;
  const int n = max(0, m - b0);
  const long long f0 = first_tile(a, p.log_p, b0 * p.block_keys);
  const int own = max(0, m - max(0, a) / p.block_keys);  // blocks with slots of the chunk
  return (int)((long long)m * (s.nq + kSetup) - (n * f0 + (long long)n * (n - 1) / 2 * (p.block_keys >> p.log_p)) +
               (long long)own * (setup_units(p, s, s.nb) - kSetup));
}
__device__ __forceinline__ Seq sequence(const MassParams& p, int i) {
  Seq s;
  s.lo = p.c.lo(i);
  s.c = p.c.hi(i, s.lo) - s.lo;
  s.len = p.c.len(i);
  s.nb = (s.len + p.block_keys - 1) / p.block_keys;
  s.nq = max(1, (s.c + (1 << p.log_p) - 1) >> p.log_p);
  s.units = s.nb ? units_before(p, s, s.nb) * p.c.H : 0;
  return s;
}

// One segment: query tiles [q0, q0 + NQ) over a block of slots of sequence i, head h.
struct __align__(16) Seg {
  int i, h, slot0, len;
  int q0, NQ, lo, c;
  int tiles, flags, cmd, pad;  // tiles of K, all of which each of these query tiles sees
  // [tile][box] pages, as the table has them: a box is a page, or 128 slots of one.  One past the
  // last page where there is no slot
  int pages[32];
  // the first of the block's query tiles here; the last of them here
  __device__ __forceinline__ bool begins() const { return flags & 1; }
  __device__ __forceinline__ bool ends() const { return flags & 2; }
  // this CTA has all of the block's query tiles
  __device__ __forceinline__ bool whole() const { return flags & 4; }
  // otherwise: 0 when an earlier CTA began the block, 1 when this one did
  __device__ __forceinline__ int slot() const { return flags >> 3 & 1; }
  // NQ, tiles and the last query tile's columns in units of 32 in one word, for the issuer
  __device__ __forceinline__ void pack(int log_p, int log_g) {
    cmd = NQ | tiles << 10 | max(1, (columns(q0 + NQ - 1, log_p, log_g) + 31) >> 5) << 13;
  }
  // the columns of query tile q
  __device__ __forceinline__ int columns(int q, int log_p, int log_g) const {
    return max(0, min(1 << log_p, c - (q << log_p))) << log_g;
  }
};

template <int NK, int NQS>
struct Bars {
  uint64_t k_full[NK], k_empty[NK];
  uint64_t q_full[NQS], q_empty[NQS];
  uint64_t s_full[4], s_empty[4];
  uint64_t x_full[2][2];  // [tile][buffer]
  uint64_t l_full[kLseStages], l_empty[kLseStages];
  uint64_t seg_full[kSegs], seg_empty[kSegs];
  uint64_t drain;
};

template <int D, bool WIDE>
struct Layout : Form<WIDE> {
  using F = Form<WIDE>;
  static constexpr int DH = D / 64;
  static constexpr int KB = D == 128 ? 1 : 2;  // blocks of K: tile rt of one has a place of its own
  static constexpr int NK = KB * F::kTiles;
  static constexpr int NQ = WIDE ? (D == 128 ? 2 : 4) : (D == 128 ? 3 : 5);  // query tiles
  static constexpr int kTile = DH * kBlockBytes;          // of K
  static constexpr int kHalf = F::kCols * 128;            // 64 columns of a query tile
  static constexpr int kQuery = DH * kHalf;
  static constexpr int k_off = 0;
  static constexpr int q_off = k_off + NK * kTile;
  static constexpr int lse_off = q_off + NQ * kQuery;     // [stage][kCols]
  static constexpr int x_off = lse_off + kLseStages * F::kCols * 4;  // [2][tile][key] sums of the second warpgroup
  static constexpr int bar_off = x_off + (WIDE ? 2 * F::kBlockKeys * 4 : 0);
  static constexpr int seg_off = bar_off + ((int)sizeof(Bars<NK, NQ>) + 15) / 16 * 16;
  static constexpr int misc_off = seg_off + kSegs * (int)sizeof(Seg);  // TMEM address, abort flag, a flag a stage
  static constexpr int total = misc_off + 8 + 4 * kLseStages;
  static_assert(total <= 232448, "shared memory of one CTA");
};

// 32 columns of a warp's 32 TMEM lanes.  Registers keys_reg(k, j) and the next hold lane id / 4 + 8 k,
// columns 8 j + 2 (id mod 4) and the next.
__host__ __device__ constexpr int keys_reg(int k, int j) { return 16 * (k >> 1) + 4 * j + 2 * (k & 1); }
__device__ __forceinline__ void tmem_ld_keys(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
        "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr + (16u << 16)));
}

// ... and 8 columns: registers 2 k and the next hold lane id / 4 + 8 k
__device__ __forceinline__ void tmem_ld_keys8(uint32_t taddr, uint32_t (&r)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.16x256b.x1.b32 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(taddr));
  asm volatile("tcgen05.ld.sync.aligned.16x256b.x1.b32 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(taddr + (16u << 16)));
}

template <int D, bool WIDE>
__global__ void __launch_bounds__(kThreads, 1) mass_kernel(const __grid_constant__ MassParams p) {
  using L = Layout<D, WIDE>;
  constexpr int DH = L::DH, NK = L::NK, NQS = L::NQ, kTiles = L::kTiles, kCols = L::kCols, kBlockKeys = L::kBlockKeys;
  constexpr int kGroups = 4 / kTiles;  // summing warpgroups a tile
  extern __shared__ __align__(1024) uint8_t smem[];  // no slack left to align by hand: the walker checks
  Bars<NK, NQS>* bars = reinterpret_cast<Bars<NK, NQS>*>(smem + L::bar_off);
  Seg* segs = reinterpret_cast<Seg*>(smem + L::seg_off);
  float* lse_s = reinterpret_cast<float*>(smem + L::lse_off);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::misc_off);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::misc_off + 4);
  int* none_s = reinterpret_cast<int*>(smem + L::misc_off + 8);  // [stage] bit 0: a row of it has lse = -inf; bit 1: NaN
  const uint32_t sbase = smem_u32(smem);
  const int warp = warp_id(), lane = lane_id();

  if (threadIdx.x == 0) {
    for (int i = 0; i < NK; ++i) {
      mbar_init(&bars->k_full[i], 1);
      mbar_init(&bars->k_empty[i], 1);
    }
    for (int i = 0; i < NQS; ++i) {
      mbar_init(&bars->q_full[i], 1);
      mbar_init(&bars->q_empty[i], 1);
    }
    for (int i = 0; i < kTiles; ++i) {
      mbar_init(&bars->s_full[i], 1);
      mbar_init(&bars->s_empty[i], 4 * kGroups);
    }
    for (int i = 0; i < 4; ++i) mbar_init(&bars->x_full[i >> 1][i & 1], 4);
    for (int i = 0; i < kLseStages; ++i) {
      mbar_init(&bars->l_full[i], 1);
      mbar_init(&bars->l_empty[i], 16);
    }
    for (int i = 0; i < kSegs; ++i) {
      mbar_init(&bars->seg_full[i], 1);
      mbar_init(&bars->seg_empty[i], 3 + 16);  // K, query tiles, MMA, summing warps
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

  auto fail = [&](int site, int detail) {
    give_up(p.c.status, site, detail, abort_flag);
  };
  // for a whole warp: false where the wait was given up
  auto wait_bar = [&](uint64_t* bar, uint32_t ph, int site, int detail) -> bool {
    if (bar_wait_warp(bar, ph, abort_flag)) return true;
    if (lane == 0) fail(site, detail);
    return false;
  };

  if (warp < 4) {
    if (warp == 0) {
      // ------------------------------------------------------------ K producer
      // Lane (box, half) issues its part of a tile: 64 columns of a box.
      if (lane == 0) tma_prefetch_desc(&p.tk);
      const int log_box = min(p.c.log_page, 7), boxes = kKeys >> log_box;
      const int box = lane / DH, dh = lane - box * DH;
      const bool mine = box < boxes;
      const uint32_t dst = dh * kBlockBytes + (box << log_box) * 128;
      uint32_t used = 0, ph = 0;  // places that hold a tile; parity of each place's next use
      int kb = 0;
      bool ok = true;
      for (int n = 0; ok; ++n) {
        if (!wait_bar(&bars->seg_full[n % kSegs], (n / kSegs) & 1, SITE_PAGED_PRODUCER, 9)) break;
        const Seg& s = segs[n % kSegs];
        if (s.NQ == 0) break;
        for (int t = 0; t < s.tiles; ++t) {
          const int pg = mine ? s.pages[t * kBoxes + box] : 0, at = kb + t;
          if (!(ok = wait_bar(&bars->k_empty[at], (ph >> at & 1) ^ 1, SITE_PAGED_PRODUCER, 1))) break;
          if (lane == 0) mbar_arrive_expect_tx(&bars->k_full[at], L::kTile);
          __syncwarp();
          if (mine)
            tma_load_4d(smem + L::k_off + at * L::kTile + dst, &p.tk, &bars->k_full[at], dh * 64,
                        (s.slot0 + t * kKeys + (box << log_box)) & ((1 << p.c.log_page) - 1), s.h, pg);
          ph ^= 1u << at;
          used |= 1u << at;
        }
        if (L::KB > 1) kb ^= kTiles;
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars->seg_empty[n % kSegs]);
      }
      if (*abort_flag && lane == 0) {
        // given up: nobody has waited for the last loads, which must land before the CTA ends
        for (int i = 0; i < NK; ++i)
          if (used >> i & 1) bar_wait(&bars->k_full[i], (ph >> i & 1) ^ 1, nullptr);
      }
    } else if (warp == 1) {
      // ------------------------------------------------------------ MMA issuer
      // One thread issues (a whole warp in step, as in paged_attn.cu: decode rows 139 us against 119,
      // a window 61 against 53).  Tile rt of a block has TMEM columns kCols rt .. and places of its own;
      // the products cover as many columns as the query tile has.
      const uint32_t k_lo = desc_lo(sbase + L::k_off, 16), q_lo = desc_lo(sbase + L::q_off, 16);
      if (lane == 0) {
        // It waits for the tensor core wherever the short queue is full, so whatever it does between
        // products counts: a segment is one word, read while the first product of the one before runs.
        Ring<NQS> q;
        uint32_t ns = 0, ph = 0;  // bit: parity of a tile's next product, and of a place's next tile of K
        int kb = 0;
        bool ok = true;
        auto wait = [&](uint64_t* bar, uint32_t parity, int detail) -> bool {
          if (bar_wait(bar, parity, abort_flag)) return true;
          fail(SITE_PAGED_MMA, detail);
          return ok = false;
        };
        auto fetch = [&](int n) -> uint32_t {
          if (!wait(&bars->seg_full[n % kSegs], (n / kSegs) & 1, 9)) return 0;
          const uint32_t cmd = segs[n % kSegs].cmd;
          mbar_arrive(&bars->seg_empty[n % kSegs]);
          return cmd;
        };
        uint32_t cmd = fetch(0);
        int n = 1;
        while (ok && cmd != 0) {
          int left = cmd & 1023;
          const int tiles = cmd >> 10 & 7;
          const uint32_t last = cmd >> 13 & 15;
          bool fresh = true;  // the tiles of K may not have landed
          // one query tile against the tiles of K
          auto products = [&](uint32_t idesc) {
            const uint32_t b0 = q_lo + q.st * (L::kQuery / 16);
            if (!wait(&bars->q_full[q.st], q.ph, 1)) return;
#pragma unroll
            for (int rt = 0; rt < kTiles; ++rt) {
              if (rt < tiles) {
                if (fresh) {
                  if (!wait(&bars->k_full[kb + rt], ph >> (kb + rt) & 1, 2)) return;
                  ph ^= 1u << (kb + rt);
                }
                if (!wait(&bars->s_empty[rt], (ns >> rt & 1) ^ 1, 3)) return;
                ns ^= 1u << rt;
                tc_fence_after();
                const uint32_t a0 = k_lo + (kb + rt) * (L::kTile / 16);
#pragma unroll
                for (int ks = 0; ks < D / 16; ++ks) {
                  const uint32_t in = (ks & 3) * 32;
                  mma_ss_lo(tbase + kCols * rt, a0 + ((ks >> 2) * kBlockBytes + in) / 16, b0 + ((ks >> 2) * L::kHalf + in) / 16,
                            idesc, ks > 0 ? 1u : 0u);
                }
                mma_commit(&bars->s_full[rt]);
                if (left == 1) mma_commit(&bars->k_empty[kb + rt]);
                if (rt == 0 && fresh) cmd = fetch(n);
              }
            }
            mma_commit(&bars->q_empty[q.st]);
            q.skip(1);
            fresh = false;
          };
          // only a chunk's last query tile has fewer columns
          for (; ok && left > 1; --left) products(idesc_bf16(128, kCols, 0));
          if (ok) products(idesc_bf16(128, 0, 0) | last << 19);
          if (L::KB > 1) kb ^= kTiles;
          ++n;
        }
        mma_commit(&bars->drain);
        bar_wait(&bars->drain, 0, nullptr);
      }
      __syncwarp();
    } else if (warp == 2) {
      // ------------------------------------------------------------ query tiles and their lse
      if (lane == 0) tma_prefetch_desc(&p.tq);
      Ring<NQS> q;
      Ring<kLseStages> r;
      int loads = 0;
      bool ok = true;
      for (int n = 0; ok; ++n) {
        if (!wait_bar(&bars->seg_full[n % kSegs], (n / kSegs) & 1, SITE_PAGED_PRODUCER, 9)) break;
        const Seg& s = segs[n % kSegs];
        if (s.NQ == 0) break;
        // rows 4 lane .. 4 lane + 3 (and 128 further on) of query tile c: -lse in log2 units; -inf adds nothing
        float x[kCols / 32];
        auto read = [&](int c) {
          const int cols = s.columns(c, p.log_p, p.log_g);
#pragma unroll
          for (int u = 0; u < kCols / 32; ++u) {
            const int col = (u >> 2) * 128 + 4 * lane + (u & 3);
            x[u] = col < cols ? p.lse[(size_t)(s.lo + (c << p.log_p) + (col >> p.log_g)) * p.Hq + s.h * p.G + (col & (p.G - 1))]
                              : __int_as_float(0x7f800000);
          }
        };
        read(s.q0);
        for (int c = s.q0; c < s.q0 + s.NQ; ++c) {
          if (!(ok = wait_bar(&bars->q_empty[q.st], q.ph ^ 1, SITE_PAGED_PRODUCER, 2))) break;
          if (lane == 0) {
            mbar_arrive_expect_tx(&bars->q_full[q.st], DH * p.q_bytes);
            for (int dh = 0; dh < DH; ++dh)
              tma_load_4d(smem + L::q_off + q.st * L::kQuery + dh * L::kHalf, &p.tq, &bars->q_full[q.st], dh * 64, s.h * p.G,
                          s.lo + (c << p.log_p), 0);
          }
          __syncwarp();
          q.skip(1);
          ++loads;
          float y[kCols / 32];
          bool none = false, nan = false;
#pragma unroll
          for (int u = 0; u < kCols / 32; ++u) {
            none |= x[u] == neg_inf();
            nan |= x[u] != x[u];
            y[u] = x[u] == neg_inf() ? neg_inf() : -x[u] * 1.4426950408889634f;
          }
          if (c + 1 < s.q0 + s.NQ) read(c + 1);
          none = __any_sync(0xffffffffu, none);
          nan = __any_sync(0xffffffffu, nan);
          if (!(ok = wait_bar(&bars->l_empty[r.st], r.ph ^ 1, SITE_PAGED_PRODUCER, 3))) break;
#pragma unroll
          for (int u = 0; u < kCols / 32; u += 4)
            reinterpret_cast<float4*>(lse_s)[(r.st * kCols + u * 32) / 4 + lane] = make_float4(y[u], y[u + 1], y[u + 2], y[u + 3]);
          if (lane == 0) none_s[r.st] = none | nan << 1;
          __syncwarp();
          if (lane == 0) mbar_arrive(&bars->l_full[r.st]);
          r.skip(1);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars->seg_empty[n % kSegs]);
      }
      if (*abort_flag && lane == 0) {  // as for K
        for (int i = 0; i < min(loads, NQS); ++i) {
          const int seq = loads - 1 - i;
          bar_wait(&bars->q_full[seq % NQS], (seq / NQS) & 1, nullptr);
        }
      }
    } else {
      // ------------------------------------------------------------ the CTA's share
      // lane l holds sequence j0 + l of a window of 32, and its first unit.  The walker also reads the
      // table, segments ahead of the others
      const int log_box = min(p.c.log_page, 7);
      int U = 0, members = 0, j0 = 0, base = 0;
      Seq g;
      auto window = [&](int w0, int at) {  // sequences w0 .., the first of them at unit `at`; returns the unit after
        g = w0 + lane < p.c.n ? sequence(p, w0 + lane) : Seq{0, 0, 0, 0, 0, 0};
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
      Split split = {0, -1, 0, 0};
      if (members > p.c.T) {
        // sequences that overlap, which the interface rules out, could pass the host's bound on U: no work
        U = 0;
        if (blockIdx.x == 0 && lane == 0) report_error(p.c.status, KVPOP_ERR_INVALID_ARG, SITE_PAGED_ROWS, 6);
      }
      if (sbase & 1023) {
        // the tiles would miss their swizzle.  No work either: an early return would leave the
        // merge whatever the workspace held for this CTA's item
        U = 0;
        if (lane == 0) report_error(p.c.status, KVPOP_ERR_INTERNAL, SITE_INTERNAL_CHECK, 61);
      }
      const int C = min((int)gridDim.x, U);
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
      // the sequence, block of slots and head of the item that holds unit u, the block's units for
      // one head, and the first of the item's; looked up once and counted on
      Seq q = {};
      int seq = 0, kb = 0, h = 0, per = 0, at = 0, setup = 0, pg = 0, seg_pg = 0;
      bool known = false;
      auto enter_block = [&]() {  // lane l reads a table entry of the block, for all of its heads
        per = q.nq - first_tile(q.len - q.c, p.log_p, kb * kBlockKeys) + (setup = setup_units(p, q, kb));
        const int slot = kb * kBlockKeys + lane / kBoxes * kKeys + (lane % kBoxes << log_box);
        pg = p.c.pages;
        if (lane / kBoxes < kTiles && lane % kBoxes < kKeys >> log_box && slot < q.len) {
          pg = p.c.page_of(seq, slot);
          if (pg < 0) {
            report_page(p.c.status, seq);
            pg = p.c.pages;
          }
        }
      };
      for (int n = 0;; ++n) {
        Seg s = {};  // NQ = 0 ends the work
        while (u < end && s.NQ == 0) {
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
            q.nq = __shfl_sync(0xffffffffu, g.nq, l);
            // the block: the last that begins at or before the unit
            int over = q.nb;
            kb = 0;
            while (over - kb > 1) {
              const int mid = (kb + over) >> 1;
              if ((long long)units_before(p, q, mid) * p.c.H <= u - b) kb = mid;
              else over = mid;
            }
            enter_block();
            at = b + units_before(p, q, kb) * p.c.H;
            h = (u - at) / per;
            at += h * per;
            known = true;
          }
          s.i = seq;
          s.h = h;
          s.slot0 = kb * kBlockKeys;
          s.len = q.len;
          s.lo = q.lo;
          s.c = q.c;
          const int a = q.len - q.c, q_lo = first_tile(a, p.log_p, s.slot0), off = u - at;
          // this CTA's units of the item from here on, as long as the same tiles are seen, up to a run
          // of query tiles: [off, stop)
          const int t0 = max(off - setup, 0);
          int stop = min(min(per, off + (end - u)), max(off, setup) + kRunTiles);
          s.tiles = 0;
          for (int rt = 0; rt < kTiles && s.slot0 + rt * kKeys < s.len; ++rt) {
            const int f = first_tile(a, p.log_p, s.slot0 + rt * kKeys) - q_lo;
            if (f <= t0) ++s.tiles;
            else stop = min(stop, f + setup);
          }
          const int t1 = max(stop - setup, 0);
          s.q0 = q_lo + t0;
          s.NQ = t1 - t0;
          seg_pg = pg;
          if (s.NQ) s.pack(p.log_p, p.log_g);
          const bool cont = t0 > 0 && n > 0;
          own = t0 == 0 || (cont && own);
          s.flags = (cont ? 0 : 1) | (stop == per || u + (stop - off) == end ? 2 : 0) | (own && stop == per ? 4 : 0) |
                    (own ? 8 : 0);
          if (n == 0 && t0 > 0) {
            // the work begins inside an item; the second of its CTAs leaves word of it
            const int first = at + setup;
            split = {seq, sh.cta_of(first) + 1 == (int)blockIdx.x ? h : -1, kb, sh.cta_of(at + per - 1)};
          }
          u += stop - off;
          if (stop == per) {  // on to the next item
            at += per;
            if (++h == p.c.H) {
              h = 0;
              if (++kb == q.nb) known = false;
              else if (u < end) enter_block();
            }
          }
        }
        if (n == 0 && lane == 0) p.split[blockIdx.x] = split;
        if (!wait_bar(&bars->seg_empty[n % kSegs], ((n / kSegs) & 1) ^ 1, SITE_PAGED_PRODUCER, 4)) break;
        segs[n % kSegs].pages[lane] = seg_pg;
        if (lane == 0) {
          Seg& to = segs[n % kSegs];
          to.i = s.i, to.h = s.h, to.slot0 = s.slot0, to.len = s.len;
          to.q0 = s.q0, to.NQ = s.NQ, to.lo = s.lo, to.c = s.c;
          to.tiles = s.tiles, to.flags = s.flags, to.cmd = s.cmd;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars->seg_full[n % kSegs]);
        if (s.NQ == 0) break;
      }
    }
  } else {
    // ------------------------------------------------------------ sums
    const int rt = (warp - 4) / (4 * kGroups), half = (warp - 4) / 4 % kGroups;  // tile of the block, columns of it
    const int quarter = warp & 3;
    // Narrow: a thread sums the columns of one key.  Wide: of four of the warp's 32 keys, lane / 4 + 8 k, a
    // quarter of the columns, two of each eight, so that it needs a quarter of the rows' lse (a load for
    // a whole warp counts for two or three of shared memory's cycles, beside what the tensor core reads:
    // 4096 tokens over 32 768 slots 688 us with one key, 652 with four; the narrow form is 2-4% slower with
    // four).  In the end key lane / 4 + 8 (lane mod 4) is its own.
    constexpr int kOwn = WIDE ? 4 : 1;
    const int sub = lane >> 2, pair = 2 * (lane & 3);
    const int row = rt * kKeys + quarter * 32 + (WIDE ? sub + 4 * pair : lane);  // of the block
    const uint32_t tl = tbase + ((uint32_t)(quarter * 32) << 16) + kCols * rt + 128 * half;
    const uint64_t s2 = pack2(p.scale_log2, p.scale_log2);
    float totals[kOwn] = {};
    uint32_t ns = 0;  // parity of this tile's next product
    uint32_t nx = 0;  // sums joined
    Ring<kLseStages> r;
    bool ok = true;
    for (int n = 0; ok; ++n) {
      if (!wait_bar(&bars->seg_full[n % kSegs], (n / kSegs) & 1, SITE_PAGED_SOFTMAX, 9)) break;
      const Seg& s = segs[n % kSegs];
      if (s.NQ == 0) break;
      if (s.begins()) {
#pragma unroll
        for (int k = 0; k < kOwn; ++k) totals[k] = 0.0f;
      }
      const int t = s.slot0 + row, a = s.len - s.c;
      const bool on = t < s.len, finish = on && half == 0 && s.ends() && s.whole();
      // the slot's old score, on its way while the products run
      float* out = nullptr;
      float old = 0.0f;
      if (finish) {
        const int pg = segs[n % kSegs].pages[rt * kBoxes + ((row & (kKeys - 1)) >> min(p.c.log_page, 7))];
        if (pg < p.c.pages) {
          out = p.scores + p.c.slot_row(pg, s.h, t);
          if (p.decay != 0.0f) old = *out;
        }
      }
      // query tiles from `clear` on have no column of a token before the key's tile ends; `part` is
      // the one with fewer columns than the others.  In registers: the barriers make shared memory anew
      const bool seen = rt < s.tiles;
      const int q0 = s.q0, q1 = q0 + s.NQ, clear = (max(0, s.slot0 + rt * kKeys + kKeys - 1 - a) + (1 << p.log_p) - 1) >> p.log_p;
      const int part = s.c & ((1 << p.log_p) - 1) || s.c == 0 ? s.c >> p.log_p : 0x7fffffff;
      for (int c = q0; c < q1; ++c) {
        if (!(ok = wait_bar(&bars->l_full[r.st], r.ph, SITE_PAGED_SOFTMAX, 1))) break;
        if (seen) {
          const float* l2 = lse_s + r.st * kCols + 128 * half;
          const bool masked = c < clear || c >= part || none_s[r.st];
          if (!(ok = wait_bar(&bars->s_full[rt], ns, SITE_PAGED_SOFTMAX, 2))) break;
          ns ^= 1;
          tc_fence_after();
          uint64_t acc[WIDE ? 4 : 2] = {};  // packed fp32 pairs
          uint32_t ra[32], rb[32];
          auto load = [](uint32_t addr, uint32_t(&x)[32]) {
            if constexpr (WIDE) tmem_ld_keys(addr, x);
            else tmem_ld32(addr, x);
          };
          auto add_pair = [&](uint64_t& to, uint32_t x0, uint32_t x1, float l0, float l1) {
            float e0, e1;
            unpack2(fma2(pack2(__uint_as_float(x0), __uint_as_float(x1)), s2, pack2(l0, l1)), e0, e1);
            to = add2(to, pack2(ex2_approx(e0), ex2_approx(e1)));
          };
          auto add_chunk = [&](const uint32_t(&x)[32], const float* lse2) {
            if constexpr (WIDE) {
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                const float2 lv = *reinterpret_cast<const float2*>(lse2 + 8 * j + pair);
#pragma unroll
                for (int k = 0; k < 4; ++k) add_pair(acc[k], x[keys_reg(k, j)], x[keys_reg(k, j) + 1], lv.x, lv.y);
              }
            } else {
#pragma unroll
              for (int cc = 0; cc < 32; cc += 4) {
                const float4 lv = *reinterpret_cast<const float4*>(lse2 + cc);
                add_pair(acc[0], x[cc], x[cc + 1], lv.x, lv.y);
                add_pair(acc[1], x[cc + 2], x[cc + 3], lv.z, lv.w);
              }
            }
          };
          auto hand_back = [&]() {  // all of the tile's columns are in registers
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars->s_empty[rt]);
          };
          if (!masked) {
            load(tl, ra);
#pragma unroll
            for (int ch = 0; ch < 4; ++ch) {
              uint32_t(&x)[32] = (ch & 1) ? rb : ra;
              uint32_t(&nxt)[32] = (ch & 1) ? ra : rb;
              tmem_wait_ld_dep(x);
              if (ch < 3) load(tl + (ch + 1) * 32, nxt);
              else hand_back();
              add_chunk(x, l2 + ch * 32);
            }
          } else {
            // Columns below lo are of tokens before the key's own, from cols on of other sequences
            const int cols = s.columns(c, p.log_p, p.log_g) - 128 * half;
            const int first = s.slot0 + rt * kKeys + quarter * 32 - a - (c << p.log_p);
            auto lo = [&](int key) { return (max(0, first + key) << p.log_g) - 128 * half; };
            const int ch1 = min(4, (cols + 31) >> 5);
            const int none = none_s[r.st];
            const bool foreign = c >= part || none;
            int ch = max(0, lo(0) >> 5);
            if (none & 2) {
              // a NaN lse, which the -inf of a product would not hide from the slots behind its row: the lse is
              // masked too, eight columns at a time in the same order
#pragma unroll 1
              for (int at = 0; at < ch1 * 32; at += 8) {
                uint32_t x[8];
                if constexpr (WIDE) tmem_ld_keys8(tl + at, x);
                else tmem_ld8(tl + at, x);
                tmem_wait_ld_dep8(x);
#pragma unroll
                for (int u = 0; u < 8; u += 2) {
                  const int key = WIDE ? sub + 4 * u : lane, col = at + (WIDE ? pair : u);
                  float v[2], l[2];
#pragma unroll
                  for (int e = 0; e < 2; ++e) {
                    const bool hidden = col + e < lo(key);
                    v[e] = hidden ? neg_inf() : fminf(__uint_as_float(x[u + e]), p.limit);
                    l[e] = hidden ? neg_inf() : l2[col + e];
                  }
                  add_pair(acc[WIDE ? u / 2 : u / 2 & 1], __float_as_uint(v[0]), __float_as_uint(v[1]), l[0], l[1]);
                }
              }
              ch = ch1;
            }
            if (ch < ch1) load(tl + ch * 32, ra);
            else hand_back();
#pragma unroll 1
            for (; ch < ch1; ++ch) {
              tmem_wait_ld_dep(ra);
              if (ch + 1 == ch1) hand_back();
              if (ch * 32 < lo(31)) {
                if constexpr (WIDE) {
#pragma unroll
                  for (int k = 0; k < 4; ++k) {
                    const int below = lo(sub + 8 * k) - ch * 32 - pair;
#pragma unroll
                    for (int j = 0; j < 4; ++j)
#pragma unroll
                      for (int e = 0; e < 2; ++e)
                        ra[keys_reg(k, j) + e] = 8 * j + e < below ? 0xff800000u : ra[keys_reg(k, j) + e];
                  }
                } else {
                  const int below = lo(lane) - ch * 32;
#pragma unroll
                  for (int cc = 0; cc < 32; ++cc) ra[cc] = cc < below ? 0xff800000u : ra[cc];
                }
              }
              if (foreign) {
                // their -lse is -inf, and a finite product with it adds nothing; a NaN becomes the limit
#pragma unroll
                for (int cc = 0; cc < 32; ++cc) ra[cc] = __float_as_uint(fminf(__uint_as_float(ra[cc]), p.limit));
              }
              add_chunk(ra, l2 + ch * 32);
              if (ch + 1 < ch1) load(tl + (ch + 1) * 32, ra);
            }
          }
#pragma unroll
          for (int k = 0; k < kOwn; ++k) {
            float y0, y1;
            unpack2(WIDE ? acc[k] : add2(acc[0], acc[1]), y0, y1);
            totals[k] += y0 + y1;
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars->l_empty[r.st]);
        r.skip(1);
      }
      if (!ok) break;
      float total = totals[0];
      if constexpr (WIDE) {
        if (s.ends()) {  // of the key, from the four threads that have a part of it
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            float y = totals[k];
            y += __shfl_xor_sync(0xffffffffu, y, 1);
            y += __shfl_xor_sync(0xffffffffu, y, 2);
            if (pair == 2 * k) total = y;
          }
        }
      }
      if (WIDE && s.ends() && seen) {
        // The second warpgroup's sums join the first's, unless no row has seen the tile: both are 0
        // then.  Of the tiles that were seen it is at most one ahead, as TMEM is handed back by both:
        // two buffers, each with a barrier of its own
        float* x_s = reinterpret_cast<float*>(smem + L::x_off) + (nx & 1) * kBlockKeys;
        if (half == 1) {
          x_s[row] = total;
          __syncwarp();
          if (lane == 0) mbar_arrive(&bars->x_full[rt][nx & 1]);
        } else {
          if (!(ok = wait_bar(&bars->x_full[rt][nx & 1], nx >> 1 & 1, SITE_PAGED_SOFTMAX, 3))) break;
          total += x_s[row];
        }
        ++nx;
      }
      if (finish) {
        if (out) *out = p.decay != 0.0f ? fmaf(p.decay, old, total) : total;
      } else if (on && half == 0 && s.ends()) {
        p.part[((size_t)blockIdx.x * 2 + s.slot()) * kBlockKeys + row] = total;
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars->seg_empty[n % kSegs]);
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

// The items that several of mass_kernel's CTAs shared: CTA x adds up the slots of the one whose
// second CTA it names, in the order of the CTAs.
__global__ void __launch_bounds__(kKeys) mass_merge(const __grid_constant__ MassParams p) {
  grid_dep_launch();
  grid_dep_wait();
  const Split s = p.split[blockIdx.x];
  if (s.h < 0) return;
  const int row = blockIdx.y * kKeys + threadIdx.x, t = s.block * p.block_keys + row;
  if (t >= p.c.len(s.i)) return;
  const int pg = p.c.page_of(s.i, t);
  if (pg < 0) return;
  float* out = p.scores + p.c.slot_row(pg, s.h, t);
  const float old = p.decay != 0.0f ? *out : 0.0f;
  const int c0 = blockIdx.x - 1;
  float total = 0.0f;
#pragma unroll 8
  for (int c = c0; c <= s.c1; ++c)  // the item begins in c0's share
    total += p.part[((size_t)c * 2 + (c == c0 ? 1 : 0)) * p.block_keys + row];
  *out = p.decay != 0.0f ? fmaf(p.decay, old, total) : total;
}

// A bound on the units of a call, and the CTAs of mass_kernel: as many for both forms, so that
// the workspace does not depend on which is taken.
int max_ctas(int T, int n, int G, int H, long long slots) {
  constexpr int kBlock = Form<true>::kBlockKeys;
  const long long units = ((long long)T * G / 128 + (long long)n * (1 + kSetup)) * H * ((slots + kBlock - 1) / kBlock);
  return (int)min((long long)num_sms(), units);
}
size_t part_offset(int ctas) { return ((size_t)ctas * sizeof(Split) + 255) / 256 * 256; }

template <int D, bool WIDE>
kvpop_status launch(MassParams& prm, int ctas, cudaStream_t cs) {
  using L = Layout<D, WIDE>;
  auto kern = mass_kernel<D, WIDE>;
  kvpop_status st = KVPOP_OK;
  static std::atomic<uint64_t> ready{0};  // bit d: the kernel is set up on device d
  const int dev = current_device();
  if (dev >= 64 || !(ready.load(std::memory_order_acquire) >> dev & 1)) {
    st = cuda_check(cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, L::total),
                    "kvpop_paged_mass: smem attribute");
    if (st != KVPOP_OK) return st;
    if (dev < 64) ready.fetch_or(1ull << dev, std::memory_order_release);
  }
  st = cuda_check(launch_pdl(kern, dim3(ctas), dim3(kThreads), L::total, cs, prm), "kvpop_paged_mass: launch");
  if (st != KVPOP_OK) return st;
  return cuda_check(launch_pdl(mass_merge, dim3(ctas, L::kTiles), dim3(kKeys), 0, cs, prm), "kvpop_paged_mass: merge launch");
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
  const int ctas = max_ctas(T, n, Hq / H, H, (long long)max_pages * page);
  *bytes = part_offset(ctas) + (size_t)ctas * 2 * Form<false>::kBlockKeys * 4;
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
  const int G = Hq / H, box = min(page, kKeys);
  // Wide from 512 rows a sequence and head on, and 32 G tokens (their mean: only the device knows each).
  // Wide against narrow, one sequence, D = 128, us: over 16 384 slots of 8 heads 64 tokens of G = 4 17.5
  // against 19, 96 27 against 23, 128 25 against 27, 1024 99 against 113; over 8192 slots of 4 heads G = 16
  // 256 tokens 46 against 39, 512 61 against 64, 2048 176 against 194.
  const bool wide = (long long)T * G >= 512ll * n && T >= 32ll * G * n;
  const int cols = wide ? Form<true>::kCols : Form<false>::kCols;
  // a decode step's rows lie alone: their boxes take no other sequence's along
  const int tokens = cu ? cols / G : 1;
  const uint64_t dq[4] = {(uint64_t)D, (uint64_t)Hq, (uint64_t)T, 1};
  const uint64_t sq[3] = {(uint64_t)D * 2, (uint64_t)Hq * D * 2, (uint64_t)T * Hq * D * 2};
  const uint32_t bq[4] = {64, (uint32_t)G, (uint32_t)tokens, 1};
  const uint64_t dk[4] = {(uint64_t)D, (uint64_t)page, (uint64_t)H, (uint64_t)pages};
  const uint64_t sk[3] = {(uint64_t)D * 2, (uint64_t)page * D * 2, (uint64_t)kp_stride * 2};
  const uint32_t bk[4] = {64, (uint32_t)box, 1, 1};
  if (!make_tmap_4d(&prm.tq, q, dq, sq, bq) || !make_tmap_4d(&prm.tk, kp, dk, sk, bk)) return KVPOP_ERR_CUDA;
  const int ctas = max_ctas(T, n, G, H, (long long)max_pages * page);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  prm.lse = lse;
  prm.scores = scores;
  prm.split = reinterpret_cast<Split*>(ws);
  prm.part = reinterpret_cast<float*>(ws + part_offset(ctas));
  prm.Hq = Hq;
  prm.G = G;
  prm.log_g = 0;
  while ((1 << prm.log_g) < G) ++prm.log_g;
  prm.log_p = (wide ? 8 : 7) - prm.log_g;
  prm.block_keys = wide ? Form<true>::kBlockKeys : Form<false>::kBlockKeys;
  prm.own_tiles = wide ? prm.block_keys >> prm.log_p : 0;
  prm.q_bytes = tokens * G * 128;
  prm.scale_log2 = (scale > 0.0f ? scale : 1.0f / sqrtf((float)D)) * 1.4426950408889634f;
  prm.limit = 1e38f / fmaxf(1.0f, prm.scale_log2);
  prm.decay = decay;
  cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
  if (D == 128) return wide ? launch<128, true>(prm, ctas, cs) : launch<128, false>(prm, ctas, cs);
  return wide ? launch<64, true>(prm, ctas, cs) : launch<64, false>(prm, ctas, cs);
}
