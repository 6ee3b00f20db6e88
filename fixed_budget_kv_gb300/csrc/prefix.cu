// kvpop_prefix_attn: decode rows over key/value prefixes that groups of sequences
// share, joined with another attention result of the same rows.
//
// For query head h G + g of sequence i in group j: s_t = scale q . k_{j,t,h},
// t < lens[j]; lse = log sum exp s_t, O = sum exp(s_t - lse) v_t; a join adds the
// keys behind (O2, lse2) by their log-sum-exp.
//
// The rows of one (prefix, KV head) are the G query heads of the group's
// sequences.  A block of up to 256 of them meets each 128-key tile of K and V
// once, so a prefix is read from memory once per 256 rows; the arithmetic is
// rows flop a byte, memory-bound up to about that many rows.
//
// Work split: an item is one (group, 256-row block, KV head), in that order, and has
// kSetup units of setup and then a unit for each 128-key tile.  CTA c takes the c-th
// part of all units, one CTA an SM, so that every SM has the same work however ragged
// the groups and lengths.  A CTA's key tiles fall into segments of one item each, of at most
// kRunTiles, whose running maximum, sum and unnormalised O are added up in a slot of the
// workspace.  An item whose key tiles are all a CTA's is finished by it; of the others a CTA
// has at most two (it begins inside one and ends inside another), in a slot each, and
// prefix_merge joins the slots of an item in the order of the CTAs.  No atomics:
// the same call gives the same bits.
//
// Warp roles of prefix_kernel (384 threads):
//   warp 0      TMA producer: one ring of K and V tiles in the order of their use
//   warp 1      TMEM allocation; issues tcgen05.mma
//   warp 2      query tiles of each segment
//   warp 3      the CTA's share of the units, handed to the others segment by segment
//   warps 4-7, 8-11  softmax, one thread a row (TMEM lane)
// The two softmax warpgroups are two streams that alternate, so that the tensor
// core works on one while the other is in its softmax.  A segment of more than
// 128 rows gives each its own row tile; a smaller one gives both the same rows
// and every other key tile, and joins the two in the epilogue.  S = Q K^T lands in
// TMEM (fp32), becomes bf16 P in place, and O += P V reads P from TMEM.  Running
// maxima are moved lazily, when they grow by more than 2^8 (the weights' precision does
// not depend on their size).  P is rounded to bf16 for its product, as the tensor core wants the
// type of V: each weight by up to 2^-8 of itself, independently, which leaves O off by about
// 1.3e-3 of its size beside the 1.7e-3 of its own rounding.  The row sum is not rounded.
//
// Measured (8 KV heads, G = 4, D = 128, one GB300, calls in a chain): 16 rows a head
// over 131 072 keys 94 us, 84% of the copy rate (the kernel alone 91-93%, 85-87 us under ncu;
// the merge the rest); 64 over 16 384 keys 29.4 us; 2 x 256 over 8192 keys
// 75 us, 900 TFLOP/s, bound by the hand-overs S -> softmax -> P V of the two streams.
#include <string.h>

#include <atomic>

#include "segments.cuh"

namespace kvpop {
namespace {

constexpr int kThreads = 384;
constexpr int kKeys = 128;
constexpr int kBlockRows = 256;
constexpr int kBlockBytes = 128 * 128;  // 128 rows x 128 bytes
constexpr float kRescaleLog2 = 8.0f;
// When chosen, 64 rows a head over 16k keys took 33.6 us with 256 and 36.8 with 512 (29.4 now).
constexpr int kMergeThreads = 256;
// Time between the last tile of a segment and the first of the next, in key tiles: when chosen, eight
// ragged groups took 61 us with 0, 46 with 1, 41 with 2, 33 with 4, 34 with 6 (29.4 now, with 4).
constexpr int kSetup = 4;
constexpr int kSegs = 4;  // segments between the walker and the last reader
// Key tiles of a segment at most.  The tensor core truncates what it adds to an accumulator, so a
// long sum loses part of itself: O of 2^17 / 2^20 / 2^24 keys in one run came out 4e-4 / 6e-3 /
// 1e-1 too small.  Runs of 2^15 keys (1e-4) are added up outside of it, in fp32 with rounding,
// for 2-3% of a long item's time (2^20 keys, 256 rows a CTA, D = 64 / 128: 13.1 / 14.6 ms against
// 12.8 / 14.2 in one run; runs of 2^14 13.2 / 14.8, of 2^16 13.05 / 14.5).  It also keeps the
// waits that last a segment (query tiles, the walker) far below their limit.
constexpr int kRunTiles = 256;
// Register split: warps 0-3 drop to kRegsIo, the softmax warpgroups rise to kRegsSoftmax.
constexpr int kRegsIo = 64;
constexpr int kRegsSoftmax = 216;
constexpr int kRegsNeeded = (128 * kRegsIo + 256 * kRegsSoftmax + kThreads - 1) / kThreads;

// An item that several CTAs share: rows, and its CTAs c0 .. c1.  nrow = 0: none.
// CTA 0 is nobody's second: its c1 is -1 when the call is refused, otherwise 0.
struct __align__(16) Split {
  int seq0, h, nrow, c1;
};

struct PrefixParams {
  CUtensorMap tq, tk, tv;
  const int32_t* cu;
  const int32_t* lens;
  const __nv_bfloat16* o2;
  const float* lse2;
  __nv_bfloat16* O;
  float* lse;
  Split* split;      // [CTA] the item that the CTA is the second to work on
  float2* part_ml;   // [CTA, 2 slots, 256 rows] (maximum in log2 units, sum)
  float4* part_o;    // [CTA, 2 slots, 2 row tiles, D / 4, 128 rows]: a warp's store is contiguous
  int* status;
  int n, m, P, Hq, H, G, seqs;  // seqs = 256 / G sequences of a row block
  float scale_log2;
};

// Group j: its sequences [lo, hi), keys, key tiles and units (the host bounds the sum
// of all units by 2^31).
struct Group {
  int lo, hi, len, nt, units;
};
__device__ __forceinline__ Group group_of(const PrefixParams& p, int j) {
  Group g;
  g.lo = p.cu ? max(0, min(p.cu[j], p.n)) : 0;
  g.hi = p.cu ? max(g.lo, min(p.cu[j + 1], p.n)) : p.n;
  g.len = p.lens ? max(0, min(p.lens[j], p.P)) : p.P;
  g.nt = (g.len + kKeys - 1) / kKeys;
  g.units = g.nt ? (g.hi - g.lo + p.seqs - 1) / p.seqs * p.H * (g.nt + kSetup) : 0;
  return g;
}

// One segment: key tiles [kt0, kt0 + NT) of an item of group j, head h.
struct __align__(16) Seg {
  int j, h, seq0, nrow;  // first sequence and rows (up to 256) of the block
  int kt0, NT, len, flags;
  // two row tiles, one a stream; otherwise one, its key tiles alternating
  __device__ __forceinline__ bool two() const { return flags & 1; }
  // the last of the block's key tiles, and this CTA had all the others
  __device__ __forceinline__ bool whole() const { return flags & 2; }
  // otherwise: 0 when an earlier CTA began the block, 1 when this one did
  __device__ __forceinline__ int slot() const { return flags >> 2 & 1; }
  // this CTA had the key tiles before these: their result is in the slot
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
__global__ void __launch_bounds__(kThreads, 1) prefix_kernel(const __grid_constant__ PrefixParams p) {
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

  auto fail = [&](int site, int detail) {
    report_error(p.status, KVPOP_ERR_TIMEOUT, site, detail);
    *abort_flag = 1;
  };
  // segment n, once the walker has written it; false at the end of the work
  auto get_seg = [&](int n, Seg& s) -> bool {
    if (!mbar_wait(&bars->seg_full[n % kSegs], (n / kSegs) & 1, abort_flag)) {
      fail(SITE_PREFIX_PRODUCER, 3);
      return false;
    }
    s = segs[n % kSegs];
    mbar_arrive(&bars->seg_empty[n % kSegs]);
    return s.NT > 0;
  };

  if (warp < 4) {
    setmaxnreg_dec<kRegsIo>();
    if (warp == 0 && lane == 0) {
      // ------------------------------------------------------------ K / V producer
      tma_prefetch_desc(&p.tk);
      tma_prefetch_desc(&p.tv);
      Seg s;
      Ring<NS> r;
      int loads = 0;
      bool ok = true;
      auto load = [&](const CUtensorMap* map, int t) {
        if (!mbar_wait(&bars->kv_empty[r.st], r.ph ^ 1, abort_flag)) {
          fail(SITE_PREFIX_PRODUCER, 1);
          ok = false;
          return;
        }
        mbar_arrive_expect_tx(&bars->kv_full[r.st], L::kTile);
        for (int dh = 0; dh < DH; ++dh)
          tma_load_4d(smem + L::kv_off + r.st * L::kTile + dh * kBlockBytes, map, &bars->kv_full[r.st], dh * 64, s.h,
                      (s.kt0 + t) * kKeys, s.j);
        r.skip(1);
        ++loads;
      };
      for (int n = 0; ok && get_seg(n, s); ++n) {
        const int ahead = s.two() ? 1 : 2;  // K tiles before the first V
        for (int t = 0; ok && t < min(ahead, s.NT); ++t) load(&p.tk, t);
        for (int t = 0; ok && t < s.NT; ++t) {
          load(&p.tv, t);
          if (ok && t + ahead < s.NT) load(&p.tk, t + ahead);
        }
      }
      if (*abort_flag) {
        // given up: nobody has waited for the last loads, which must land before the CTA ends
        for (int i = 0; i < min(loads, NS); ++i) {
          const int seq = loads - 1 - i;
          mbar_wait(&bars->kv_full[seq % NS], (seq / NS) & 1, nullptr);
        }
      }
    } else if (warp == 1) {
      // ------------------------------------------------------------ MMA issuer
      // A segment's events alternate between the streams: event e takes key tile e, or with
      // two row tiles row tile e & 1 and key tile e / 2.  S runs two events ahead of P V, into
      // the next segment, so S of a stream always follows P V of the stream's event before.
      // TMEM: S / P of stream w at column 128 w, O at 256 + 128 w.
      // The bookkeeping is in the way of every MMA.  The whole warp runs it, in step, and one
      // elected lane issues: the operands then live in uniform registers (256 x 8k keys: 77 us
      // against 84 with a single thread here).  Places in the rings are counted on.
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
        if (!warp_wait(bar, ph, abort_flag)) {
          if (lane == 0) fail(SITE_PREFIX_MMA, detail);
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
      warp_wait(&bars->drain, 0, nullptr);
    } else if (warp == 2 && lane == 0) {
      // ------------------------------------------------------------ query tiles
      tma_prefetch_desc(&p.tq);
      Seg s;
      int n = 0;
      for (; get_seg(n, s); ++n) {
        if (!mbar_wait(&bars->q_empty, (n & 1) ^ 1, abort_flag)) {
          fail(SITE_PREFIX_PRODUCER, 2);
          break;
        }
        const int tiles = s.two() ? 2 : 1;
        mbar_arrive_expect_tx(&bars->q_full, tiles * L::kTile);
        for (int i = 0; i < tiles; ++i)
          for (int dh = 0; dh < DH; ++dh)
            tma_load_4d(smem + L::q_off + i * L::kTile + dh * kBlockBytes, &p.tq, &bars->q_full, dh * 64, s.h * p.G,
                        s.seq0 + i * (p.seqs / 2), 0);
      }
      if (*abort_flag && n > 0) mbar_wait(&bars->q_full, (n - 1) & 1, nullptr);  // as for K and V
    } else if (warp == 3) {
      // ------------------------------------------------------------ the CTA's share
      // lane l holds group j0 + l of a window of 32 groups, and its first unit
      int U = 0, members = 0, j0 = 0, base = 0;
      Group g;
      auto window = [&](int w0, int at) {  // groups w0 .., the first of them at unit `at`; returns the unit after
        g = w0 + lane < p.m ? group_of(p, w0 + lane) : Group{0, 0, 0, 0, 0};
        const int incl = scan_incl(g.units);
        j0 = w0;
        base = at + incl - g.units;
        return at + __shfl_sync(0xffffffffu, incl, 31);
      };
#pragma unroll 1
      for (int w0 = 0; w0 < p.m; w0 += 32) {
        U = window(w0, U);
        members = min(members, p.n + 1) + __reduce_add_sync(0xffffffffu, min(g.hi - g.lo, p.n));
      }
      Split split = {0, 0, 0, 0};
      if (members > p.n) {
        // groups that overlap, which the interface rules out, could pass the host's bound on U: no work
        U = 0;
        split.c1 = -1;
        if (blockIdx.x == 0 && lane == 0) report_error(p.status, KVPOP_ERR_INVALID_ARG, SITE_PREFIX_PRODUCER, 5);
      }
      if (sbase & 1023) {
        // the tiles would miss their swizzle.  No work either: an early return would leave the
        // merge whatever the workspace held for this CTA's item
        U = 0;
        split.c1 = -1;
        if (lane == 0) report_error(p.status, KVPOP_ERR_INTERNAL, SITE_INTERNAL_CHECK, 50);
      }
      const int C = min((int)gridDim.x, U);
      const Share sh(U, max(C, 1));
      int u = 0, end = 0;
      if ((int)blockIdx.x < C) {
        u = sh.first(blockIdx.x);
        end = sh.first(blockIdx.x + 1);
      }
      if (p.m > 32 && u < end) {  // back to the window in which the share begins
        int at = 0;
#pragma unroll 1
        for (int w0 = 0;; w0 += 32) {
          at = window(w0, at);
          if (u < at) break;
        }
      }
      bool own = false;  // this CTA began the item that u is in
      for (int n = 0;; ++n) {
        Seg s = {0, 0, 0, 0, 0, 0, 0, 0};  // NT = 0 ends the work
        while (u < end && s.NT == 0) {
          // the group that holds unit u: the last of the window that begins at or before it
          unsigned at = __ballot_sync(0xffffffffu, g.units > 0 && base <= u && u < base + g.units);
          if (at == 0) {
            window(j0 + 32, u);  // u is the window's end
            continue;
          }
          const int l = __ffs(at) - 1;
          const int b = __shfl_sync(0xffffffffu, base, l), lo = __shfl_sync(0xffffffffu, g.lo, l),
                    hi = __shfl_sync(0xffffffffu, g.hi, l), nt = __shfl_sync(0xffffffffu, g.nt, l);
          s.len = __shfl_sync(0xffffffffu, g.len, l);
          const int per = nt + kSetup, item = (u - b) / per, off = (u - b) - item * per;
          // this CTA's units of the item from here on, up to a run of key tiles: [off, stop)
          const int stop = min(min(per, off + (end - u)), max(off, kSetup) + kRunTiles);
          s.kt0 = max(off - kSetup, 0);
          s.NT = max(stop - kSetup, 0) - s.kt0;
          const int rb = item / p.H;
          s.j = j0 + l;
          s.h = item - rb * p.H;
          s.seq0 = lo + rb * p.seqs;
          s.nrow = min(p.seqs, hi - s.seq0) * p.G;
          const bool cont = s.kt0 > 0 && n > 0;
          own = s.kt0 == 0 || (cont && own);
          s.flags = (s.nrow > 128 ? 1 : 0) | (own && stop == per ? 2 : 0) | (own ? 4 : 0) | (cont ? 8 : 0);
          if (n == 0 && s.kt0 > 0) {
            // the work begins inside an item; the second of its CTAs leaves word of it
            const int first = b + item * per + kSetup;
            split = {s.seq0, s.h, sh.cta_of(first) + 1 == (int)blockIdx.x ? s.nrow : 0, sh.cta_of(first + nt - 1)};
          }
          u += stop - off;
        }
        if (n == 0 && lane == 0) p.split[blockIdx.x] = split;
        if (!warp_wait(&bars->seg_empty[n % kSegs], ((n / kSegs) & 1) ^ 1, abort_flag)) {
          if (lane == 0) fail(SITE_PREFIX_PRODUCER, 4);
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
        if (lane == 0) fail(SITE_PREFIX_SOFTMAX, 3);
        break;
      }
      const Seg& s = segs[n % kSegs];
      if (s.NT == 0) break;
      const bool two = s.two();
      const int a = w ^ par;  // row tile, or first key tile
      const int steps = two ? s.NT : (s.NT - a + 1) / 2;
      const int rrow = two ? 128 * a + row : row;  // row within the block
      const bool warp_on = rrow - lane < s.nrow, row_on = rrow < s.nrow;
      float m_ref = neg_inf(), l = 0.0f;
      for (int i = 0; i < steps; ++i, ++cnt) {
        const int t = two ? i : 2 * i + a;
        if (!warp_wait(&bars->s_full[w], cnt & 1, abort_flag)) {
          if (lane == 0) fail(SITE_PREFIX_SOFTMAX, 1);
          ok = false;
          break;
        }
        tc_fence_after();
        const int left = s.len - (s.kt0 + t) * kKeys;  // keys of this tile within the length
        if (warp_on) {
          // the whole S row of this thread (128 fp32) in registers; keys past the length -> -inf
          uint32_t sr[4][32];
#pragma unroll
          for (int ch = 0; ch < 4; ++ch) tmem_ld32(tl + s_col + ch * 32, sr[ch]);
#pragma unroll
          for (int ch = 0; ch < 4; ++ch) tmem_wait_ld_dep(sr[ch]);
          float mt = neg_inf();
#pragma unroll
          for (int ch = 0; ch < 4; ++ch) {
            if (left < ch * 32 + 32) {
#pragma unroll
              for (int c = 0; c < 32; ++c)
                if (ch * 32 + c >= left) sr[ch][c] = 0xff800000u;
            }
            mt = fmaxf(mt, max32(sr[ch]));
          }
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
          // P = exp2(s * scale_log2 - m) as bf16, written over S
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
          l += l0 + l1;
          tmem_wait_st();
        }
        if (left < kKeys && s.len < p.P) {
          // V rows past the length hold anything, and 0 * NaN would be NaN: zero them
          const int seq = sb + pos_v(two, s.NT, t), st = seq % NS;
          if (!warp_wait(&bars->kv_full[st], (seq / NS) & 1, abort_flag)) {
            if (lane == 0) fail(SITE_PREFIX_SOFTMAX, 2);
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
      const size_t orow = (size_t)(s.seq0 + rrow / p.G) * p.Hq + s.h * p.G + rrow % p.G;
      // read before lse, which may be lse2, is written
      const float j2 = s.whole() && p.o2 != nullptr && row_on ? p.lse2[orow] * 1.4426950408889634f : neg_inf();
      float w_own = 1.0f, w_oth = 0.0f;
      // no weight: -inf; a NaN among the scores keeps a finite maximum and travels in l
      float m2 = l == 0.0f ? neg_inf() : (m_ref == neg_inf() ? 0.0f : m_ref * sl2);
      if (!warp_wait(&bars->o_full, n & 1, abort_flag)) {
        if (lane == 0) fail(SITE_PREFIX_EPILOGUE, 1);
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
          if (lane == 0) fail(SITE_PREFIX_EPILOGUE, 2);
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
      float w_run = 0.0f, w_j = 0.0f;
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
      bool joins = false;
      if (s.whole()) {
        const float T = fmaxf(m2, j2);
        const float w_p = m2 != neg_inf() ? ex2_approx(m2 - T) : 0.0f;
        w_j = j2 != neg_inf() ? ex2_approx(j2 - T) : 0.0f;
        l = l * w_p + w_j;
        joins = w_j != 0.0f;  // before 1 / l, which may be NaN: o2 need not be there
        const float inv = l != 0.0f ? 1.0f / l : 0.0f;
        w_own *= w_p * inv;
        w_oth *= w_p * inv;
        w_run *= w_p * inv;
        w_j *= inv;
        m2 = T;
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
            if (joins) {
              const uint4* j = reinterpret_cast<const uint4*>(p.o2 + orow * D + c0);
#pragma unroll
              for (int u = 0; u < 4; ++u) {
                const uint4 y = j[u];
                const uint32_t yy[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                  v[8 * u + 2 * c] += w_j * __uint_as_float(yy[c] << 16);
                  v[8 * u + 2 * c + 1] += w_j * __uint_as_float(yy[c] & 0xffff0000u);
                }
              }
            }
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

// A row's result from (maximum, sum, unnormalised O) of its four columns and the join.
template <int D>
__device__ __forceinline__ void finish_row(const PrefixParams& p, size_t orow, int c4, float j2, float M, float l,
                                           float4 o) {
  const float T = fmaxf(M, j2);
  const float w = M != neg_inf() ? ex2_approx(M - T) : 0.0f, wj = j2 != neg_inf() ? ex2_approx(j2 - T) : 0.0f;
  l = l * w + wj;
  o = M != neg_inf() ? make_float4(o.x * w, o.y * w, o.z * w, o.w * w) : make_float4(0.f, 0.f, 0.f, 0.f);
  if (wj != 0.0f) {
    const uint2 y = *reinterpret_cast<const uint2*>(p.o2 + orow * D + 4 * c4);
    o.x += wj * __uint_as_float(y.x << 16);
    o.y += wj * __uint_as_float(y.x & 0xffff0000u);
    o.z += wj * __uint_as_float(y.y << 16);
    o.w += wj * __uint_as_float(y.y & 0xffff0000u);
  }
  const float inv = l != 0.0f ? 1.0f / l : 0.0f;
  *reinterpret_cast<uint2*>(p.O + orow * D + 4 * c4) =
      make_uint2(pack_bf16x2(o.x * inv, o.y * inv), pack_bf16x2(o.z * inv, o.w * inv));
  if (c4 == 0) p.lse[orow] = l != 0.0f ? (T + __log2f(l)) * 0.69314718055994531f : neg_inf();
}

// The items that several of prefix_kernel's CTAs shared, each joined from the slots of its
// CTAs in their order: CTA (x, y < chunks) takes rows y of those whose second CTA is in the
// x-th part of the CTAs.  Thread (part, c4, row) takes four columns and every parts-th slot;
// the parts are joined through shared memory.
// CTAs (x, y >= chunks): the rows of groups without keys, which get what they join or nothing.
// 512 sequences of 32 heads, joined: the call takes 20 us, as with 128 keys each (885 us when
// each such group was one CTA's).  Last in the grid, so that the merge's CTAs are not in their
// way: in front of them they cost 1 us (eight ragged groups: 30.4 us against 29.2).
template <int D>
__global__ void __launch_bounds__(kMergeThreads, 4) prefix_merge(const __grid_constant__ PrefixParams p, int ctas, int parts,
                                                              int chunks) {
  constexpr int kBatch = 4;
  __shared__ float2 ml_s[kMergeThreads];
  __shared__ float4 o_s[kMergeThreads];
  grid_dep_launch();
  grid_dep_wait();
  if ((int)blockIdx.y >= chunks) {
    const bool refused = p.split[0].c1 < 0;  // these rows stay as they were too
    // a window of groups at a time: their sequences without keys in a line, rows of it shared
    // out over these CTAs
    __shared__ int ends_s[kMergeThreads], shift_s[kMergeThreads], warp_s[kMergeThreads / 32];
    const int block = (blockIdx.y - chunks) * gridDim.x + blockIdx.x, blocks = (gridDim.y - chunks) * gridDim.x;
    constexpr int kRows = kMergeThreads / (D / 4);
    const int c4 = threadIdx.x % (D / 4);
    for (int w0 = 0; w0 < p.m; w0 += kMergeThreads) {
      Group g = w0 + (int)threadIdx.x < p.m ? group_of(p, w0 + threadIdx.x) : Group{0, 0, 0, 0, 0};
      if (refused) return;
      if (!__syncthreads_or(g.nt == 0 && g.hi > g.lo)) continue;
      int end = scan_incl(g.nt == 0 ? g.hi - g.lo : 0);
      if (lane_id() == 31) warp_s[warp_id()] = end;
      __syncthreads();
      for (int w = 0; w < warp_id(); ++w) end += warp_s[w];
      ends_s[threadIdx.x] = end;          // in the line
      shift_s[threadIdx.x] = g.hi - end;  // from the line to the sequence
      __syncthreads();
      const long long all = (long long)ends_s[kMergeThreads - 1] * p.Hq;
      for (long long r0 = (long long)block * kRows; r0 < all; r0 += (long long)blocks * kRows) {
        const long long r = r0 + threadIdx.x / (D / 4);
        const bool on = r < all;
        const int at = on ? (int)(r / p.Hq) : 0;
        int l = 0;  // the first group that ends behind it
#pragma unroll
        for (int step = kMergeThreads / 2; step > 0; step >>= 1)
          if (ends_s[l + step - 1] <= at) l += step;
        const size_t orow = on ? (size_t)(at + shift_s[l]) * p.Hq + (r - (long long)at * p.Hq) : 0;
        const float j2 = on && p.o2 ? p.lse2[orow] * 1.4426950408889634f : neg_inf();
        __syncwarp();  // lse, which may be lse2, is written after the row's lanes, of one warp, have read it
        if (on) finish_row<D>(p, orow, c4, j2, neg_inf(), 0.0f, make_float4(0.f, 0.f, 0.f, 0.f));
      }
      __syncthreads();
    }
    return;
  }
  const int wide = kMergeThreads / parts, rows = wide / (D / 4);
  const int part = threadIdx.x / wide, x = threadIdx.x - part * wide, c4 = x / rows, r = blockIdx.y * rows + x - c4 * rows;
  const int lo = (int)((long long)ctas * blockIdx.x / gridDim.x), hi = (int)((long long)ctas * (blockIdx.x + 1) / gridDim.x);
  for (int w0 = lo; w0 < hi; w0 += 32) {
    const Split mine = w0 + lane_id() < hi ? p.split[w0 + lane_id()] : Split{0, 0, 0, 0};
    unsigned todo = __ballot_sync(0xffffffffu, (int)blockIdx.y * rows < mine.nrow);
    while (todo) {  // the same in every warp
      const int src = __ffs(todo) - 1;
      todo &= todo - 1;
      const int seq0 = __shfl_sync(0xffffffffu, mine.seq0, src), h = __shfl_sync(0xffffffffu, mine.h, src),
                nrow = __shfl_sync(0xffffffffu, mine.nrow, src), c1 = __shfl_sync(0xffffffffu, mine.c1, src);
      const int c0 = w0 + src - 1;
      const bool on = r < nrow;
      const size_t orow = on ? (size_t)(seq0 + r / p.G) * p.Hq + h * p.G + r % p.G : 0;
      const float j2 = on && p.o2 ? p.lse2[orow] * 1.4426950408889634f : neg_inf();
      float M = neg_inf(), l = 0.0f;
      float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
      auto add = [&](const float2& ml, const float4& y, float m) {
        const float f = ml.x != neg_inf() ? ex2_approx(ml.x - m) : 0.0f;
        l += f * ml.y;
        if (ml.x != neg_inf()) {
          o.x += f * y.x;
          o.y += f * y.y;
          o.z += f * y.z;
          o.w += f * y.w;
        }
      };
      for (int c = c0 + part; on && c <= c1; c += kBatch * parts) {
        float2 ml[kBatch];
        float4 y[kBatch];
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
          const int cc = c + k * parts;
          ml[k] = make_float2(neg_inf(), 0.0f);
          y[k] = make_float4(0.f, 0.f, 0.f, 0.f);
          if (cc <= c1) {
            const size_t slot = (size_t)cc * 2 + (cc == c0 ? 1 : 0);  // the item begins in c0's share
            ml[k] = p.part_ml[slot * kBlockRows + r];
            y[k] = p.part_o[((slot * 2 + (r >> 7)) * (D / 4) + c4) * 128 + (r & 127)];
          }
        }
        float m = M;
#pragma unroll
        for (int k = 0; k < kBatch; ++k) m = fmaxf(m, ml[k].x);
        if (m != neg_inf()) {
          const float f = M != neg_inf() ? ex2_approx(M - m) : 0.0f;
          l *= f;
          o.x *= f, o.y *= f, o.z *= f, o.w *= f;
          M = m;
#pragma unroll
          for (int k = 0; k < kBatch; ++k) add(ml[k], y[k], m);
        }
      }
      ml_s[threadIdx.x] = make_float2(M, l);
      o_s[threadIdx.x] = o;
      __syncthreads();  // also: lse, which may be lse2, is written after every thread has read it
      if (on && part == 0) {
        if (parts > 1) {
          for (int k = 1; k < parts; ++k) M = fmaxf(M, ml_s[x + k * wide].x);
          l = 0.0f;
          o = make_float4(0.f, 0.f, 0.f, 0.f);
          for (int k = 0; M != neg_inf() && k < parts; ++k) add(ml_s[x + k * wide], o_s[x + k * wide], M);
        }
        finish_row<D>(p, orow, c4, j2, M, l, o);
      }
      __syncthreads();
    }
  }
}

// A bound on the units of a call, and the CTAs of prefix_kernel.
long long max_units(int n, int m, int P, int H, int G) {
  return (m + (long long)n * G / kBlockRows) * H * ((P + kKeys - 1ll) / kKeys + kSetup);
}
int max_ctas(int n, int m, int P, int H, int G) {
  return (int)min((long long)num_sms(), max_units(n, m, P, H, G));
}
size_t round256(size_t x) { return (x + 255) / 256 * 256; }
size_t ml_offset(int ctas) { return round256((size_t)ctas * sizeof(Split)); }
size_t o_offset(int ctas) { return ml_offset(ctas) + (size_t)ctas * 2 * kBlockRows * 8; }

template <int D>
kvpop_status launch(PrefixParams& prm, int ctas, cudaStream_t cs) {
  using L = Layout<D>;
  auto kern = prefix_kernel<D>;
  kvpop_status st = KVPOP_OK;
  static std::atomic<uint64_t> ready{0};  // bit d: the kernel is set up on device d
  const int dev = current_device();
  if (dev >= 64 || !(ready.load(std::memory_order_acquire) >> dev & 1)) {
    st = cuda_check(cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, L::total),
                    "kvpop_prefix_attn: smem attribute");
    if (st != KVPOP_OK) return st;
    // the register re-split must fit in the launch allocation (granule: 8 per thread)
    cudaFuncAttributes fa;
    st = cuda_check(cudaFuncGetAttributes(&fa, kern), "kvpop_prefix_attn: attributes");
    if (st != KVPOP_OK) return st;
    if (((fa.numRegs + 7) / 8) * 8 < kRegsNeeded) {
      set_last_error("kvpop_prefix_attn: kernel built with %d registers per thread, %d needed", fa.numRegs, kRegsNeeded);
      return KVPOP_ERR_INTERNAL;
    }
    if (dev < 64) ready.fetch_or(1ull << dev, std::memory_order_release);
  }
  st = cuda_check(launch_pdl(kern, dim3(ctas), dim3(kThreads), L::total, cs, prm), "kvpop_prefix_attn: launch");
  if (st != KVPOP_OK) return st;
  // A thread of the merge takes about four slots of a row, a CTA at least four rows (two
  // sectors of a slot's columns).  There are at most `items` items, and at most one a CTA
  // that several CTAs share.
  const long long rows_all = (long long)prm.n * prm.G;
  const int items = prm.H * (prm.m == 1 ? (int)((rows_all + kBlockRows - 1) / kBlockRows)
                                        : prm.m + (int)(rows_all / kBlockRows));
  int parts = 1;
  while (kMergeThreads / (D / 4) / parts > 4 && ctas / items > 4 * parts) parts *= 2;
  const int rows = kMergeThreads / (D / 4) / parts;
  const int chunks = ((int)min((long long)kBlockRows, rows_all) + rows - 1) / rows;
  const int across = min(ctas, items);
  // groups without keys need lens.  Up to four CTAs an SM, all that fit (64 registers): with one an
  // SM 8192 such sequences take 293 us, with four 94
  const long long passes = (prm.n * (long long)prm.Hq + kMergeThreads / (D / 4) - 1) / (kMergeThreads / (D / 4));
  const int empties = prm.lens ? (int)min(passes, 4ll * num_sms()) : 0;
  const dim3 grid(across, chunks + (empties + across - 1) / across);
  return cuda_check(launch_pdl(prefix_merge<D>, grid, dim3(kMergeThreads), 0, cs, prm, ctas, parts, chunks),
                    "kvpop_prefix_attn: merge launch");
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
  // these first: they keep max_units within 64 bits
  if (H > 65535 || Hq > 65535 || m > 65535 || n > (1 << 24) || (long long)n * Hq > 0x7fffffffll) {
    set_last_error("kvpop_prefix_attn: at most 65535 heads and prefixes, 2^24 sequences and 2^31 - 1 rows");
    return KVPOP_ERR_UNSUPPORTED;
  }
  if (P > (1 << 30) || max_units(n, m, P, H, Hq / H) > 0x7fffffffll) {
    set_last_error("kvpop_prefix_attn_workspace_size: more than 2^30 keys or 2^31 - 1 tiles of rows and keys");
    return KVPOP_ERR_UNSUPPORTED;
  }
  const int ctas = max_ctas(n, m, P, H, Hq / H);
  *bytes = o_offset(ctas) + (size_t)ctas * 2 * kBlockRows * D * 4;
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
  const int G = Hq / H;
  PrefixParams prm;
  memset(&prm, 0, sizeof(prm));
  const uint64_t dq[4] = {(uint64_t)D, (uint64_t)Hq, (uint64_t)n, 1};
  const uint64_t sq[3] = {(uint64_t)D * 2, (uint64_t)Hq * D * 2, (uint64_t)n * Hq * D * 2};
  const uint32_t bq[4] = {64, (uint32_t)G, (uint32_t)(128 / G), 1};
  const uint64_t dk[4] = {(uint64_t)D, (uint64_t)H, (uint64_t)P, (uint64_t)m};
  const uint64_t sk[3] = {(uint64_t)D * 2, (uint64_t)H * D * 2, (uint64_t)P * H * D * 2};
  const uint32_t bk[4] = {64, 1, kKeys, 1};
  if (!make_tmap_4d(&prm.tq, q, dq, sq, bq) || !make_tmap_4d(&prm.tk, pk, dk, sk, bk) ||
      !make_tmap_4d(&prm.tv, pv, dk, sk, bk))
    return KVPOP_ERR_CUDA;
  const int ctas = max_ctas(n, m, P, H, G);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  prm.cu = cu;
  prm.lens = lens;
  prm.o2 = (const __nv_bfloat16*)O2;
  prm.lse2 = lse2;
  prm.O = (__nv_bfloat16*)O;
  prm.lse = lse;
  prm.split = reinterpret_cast<Split*>(ws);
  prm.part_ml = reinterpret_cast<float2*>(ws + ml_offset(ctas));
  prm.part_o = reinterpret_cast<float4*>(ws + o_offset(ctas));
  prm.status = device_status_ptr();
  prm.n = n;
  prm.m = m;
  prm.P = P;
  prm.Hq = Hq;
  prm.H = H;
  prm.G = G;
  prm.seqs = kBlockRows / G;
  prm.scale_log2 = (scale > 0.0f ? scale : 1.0f / sqrtf((float)D)) * 1.4426950408889634f;
  cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
  return D == 128 ? launch<128>(prm, ctas, cs) : launch<64>(prm, ctas, cs);
}
