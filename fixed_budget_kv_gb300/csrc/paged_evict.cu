// kvpop_paged_evict: each head of a paged cache down to B = s + w + k slots by the attention
// weight that its keys have received.
//
// Of a sequence with len > B slots, a head keeps slots [0, s), [len - w, len) and the k best of
// [s, len - w) in the order (score falling, slot rising), NaN counting as -inf and -0 as +0.
//
// evict_select, one cluster a (sequence, head), its CTAs a part of the slots each: the k-th best
// score by a radix select (11 + 11 + 10 bits of an order-preserving key, the CTAs' histograms
// added up through distributed shared memory; the keys that share the first digit are set aside
// for the others), then the kept slots in their order: a thread has consecutive slots, so one scan
// gives every thread its place.  Bound by its chain of barriers.
// evict_move: kept slot j goes from kept[j] >= j to j.  A CTA, or a cluster of them where there are few
// heads, moves K (with the scores) or V of a head in rising order, a batch of rows at a time: loads,
// barrier, stores.  The next batch's sources lie at or above its own slots, so behind everything stored
// before: nothing is lost and no second copy is needed.  Bound by memory.
//
// Measured (8 KV heads, D = 128, one GB300): 64 sequences of 1700 .. 4099 slots to 2048, 845 MB: select
// 19 us, move 134 us (5.8 TB/s), in a chain of calls 180 us; one of 131 072 slots to 4096: 18 us
// (the barriers of eight clusters) and 7-16 us (rows in and out of 128 SMs), in a chain 30-32 us.
#include <atomic>

#include "paged.cuh"
#include "segments.cuh"

namespace kvpop {
namespace {

constexpr int kBins = 2048;
// Keys with the first digit of the k-th best that are set aside, at most: by a CTA, and of a cluster
constexpr int kSet = 2048, kTied = 8192;
constexpr int kCacheBytes = 163840;  // for the keys of a CTA's part, at most
constexpr int kMaxCluster = 8;
constexpr int kMoveBatch = 8;  // pieces that a thread has in flight
// Threads of a CTA with few heads and with many (64 sequences to 2048 slots, a first pass on cold
// caches: 128 threads 216 us, 256 199, 512 185, 1024 198).
constexpr int kMoveFew = 1024, kMoveMany = 512;

struct EvictParams {
  Paged c;
  float* scores;
  uint4 *k, *v;
  int64_t k_stride, v_stride;  // 16-byte pieces between pages
  int32_t *kept, *new_lens;
  int s, w, top, B;
  int held;  // groups of four keys that the select's shared memory has room for
};

// fp32 -> uint32 of the same order; NaN as -inf, -0 as +0
__device__ __forceinline__ uint32_t order_key(float x) {
  if (x != x) x = __int_as_float(0xff800000);
  if (x == 0.0f) x = 0.0f;
  const uint32_t u = __float_as_uint(x);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

__device__ __forceinline__ uint32_t ld_cluster_u32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ void st_cluster_u32(uint32_t addr, uint32_t v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}

// Exclusive sums of two values over the block.  Two barriers.
template <int THREADS>
__device__ __forceinline__ uint2 block_scan(uint2 x, uint2* warp_s) {
  uint2 y = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t a = __shfl_up_sync(0xffffffffu, y.x, o), b = __shfl_up_sync(0xffffffffu, y.y, o);
    if (lane_id() >= o) y.x += a, y.y += b;
  }
  __syncthreads();  // the sums of the scan before have been read
  if (lane_id() == 31) warp_s[warp_id()] = y;
  __syncthreads();
  const uint2 before = lane_id() < warp_id() ? warp_s[lane_id()] : make_uint2(0, 0);
  return make_uint2(__reduce_add_sync(0xffffffffu, before.x) + y.x - x.x, __reduce_add_sync(0xffffffffu, before.y) + y.y - x.y);
}

template <int THREADS>
__global__ void __launch_bounds__(THREADS, THREADS == 512 ? 4 : 1) evict_select(const __grid_constant__ EvictParams p) {
  static_assert(THREADS / 32 <= 32 && 1024 % THREADS == 0, "one warp holds the warps' sums; whole bins a thread");
  extern __shared__ __align__(16) uint32_t keys_s[];  // the part's keys, if they fit, and the tied ones
  __shared__ uint32_t hists[2][kBins], total[kBins];  // a pass counts in one while the next one's is cleared
  uint32_t* tied = keys_s + (p.held + p.held / 8) * 4;  // keys that share the first digit of the k-th best
  __shared__ uint2 warp_s[THREADS / 32];
  __shared__ uint32_t found[2];   // the bin of the k-th best, and how many of it stay
  __shared__ uint32_t counts[2];  // keys of this part above the k-th best, and equal to it
  __shared__ uint32_t ntied;
  const int tid = threadIdx.x;
  for (int b = tid; b < kBins; b += THREADS) hists[0][b] = 0;
  if (tid == 0) ntied = 0;
  grid_dep_wait();
  grid_dep_launch();
  const Paged& c = p.c;
  const int CS = gridDim.x, rank = blockIdx.x;  // one cluster along x
  const int i = blockIdx.y / c.H, h = blockIdx.y - i * c.H;
  const int len = c.len(i);
  int32_t* kept = p.kept + (size_t)blockIdx.y * p.B;
  if (len <= p.B) {
    for (int j = rank * THREADS + tid; j < p.B; j += CS * THREADS) kept[j] = j < len ? j : -1;
    return;  // the whole cluster
  }
  for (int j = rank * THREADS + tid; j < p.s; j += CS * THREADS) kept[j] = j;
  for (int j = rank * THREADS + tid; j < p.w; j += CS * THREADS) kept[p.s + p.top + j] = len - p.w + j;
  if (p.top == 0) return;
  // the slots that may go, [s, end), in groups of four: this CTA has groups [g0, g1)
  const int end = len - p.w, first = p.s & ~3, groups = (end - first + 3) / 4;
  const int g0 = (int)((long long)groups * rank / CS), g1 = (int)((long long)groups * (rank + 1) / CS);
  const bool held = g1 - g0 <= p.held;
  const int32_t* table = c.table + (size_t)i * c.max_pages;
  // group g's keys; a table entry that names no page: the worst
  auto keys_at = [&](int g, int pg) -> uint4 {
    float4 x = make_float4(neg_inf(), neg_inf(), neg_inf(), neg_inf());
    if ((unsigned)pg < (unsigned)c.pages) x = *reinterpret_cast<const float4*>(p.scores + c.slot_row(pg, h, first + 4 * g));
    return make_uint4(order_key(x.x), order_key(x.y), order_key(x.z), order_key(x.w));
  };
  // a gap after eight groups: consecutive groups of a thread then lie in different banks from its neighbours'
  auto place = [](int g) { return g + (g >> 3); };
  auto keys_of = [&](int g) -> uint4 {
    return held ? reinterpret_cast<const uint4*>(keys_s)[place(g - g0)] : keys_at(g, table[(first + 4 * g) >> c.log_page]);
  };
  // bit u: slot u of group g may go
  auto free_slots = [&](int g) -> uint32_t {
    const int t = first + 4 * g;
    uint32_t m = 15;
    if (t < p.s) m &= 15u << (p.s - t);
    if (t + 4 > end) m &= 15u >> (t + 4 - end);
    return m;
  };
  // one warp's keys into a histogram, m: which of them
  auto count = [&](uint32_t* hist, uint32_t m, const uint4& x, int shift, int bins) {
    const uint32_t bin[4] = {x.x >> shift & bins - 1, x.y >> shift & bins - 1, x.z >> shift & bins - 1, x.w >> shift & bins - 1};
    // many equal scores (nothing received yet): one addition for the whole warp
    const uint32_t ref = __shfl_sync(0xffffffffu, bin[1], 16);
    const bool same = m == 15 && bin[0] == ref && bin[1] == ref && bin[2] == ref && bin[3] == ref;
    if (__all_sync(0xffffffffu, same)) {
      if (lane_id() == 0) atomicAdd(&hist[ref], 128u);
      return;
    }
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (m >> u & 1) atomicAdd(&hist[bin[u]], 1u);
  };
  uint32_t prefix = 0, need = p.top;
  // the bin of the k-th best from the counts of a pass, over the cluster or those of this CTA
  auto find = [&](const uint32_t* hist, int shift, int bins, bool over_all) {
    if (over_all) {
      // CTA r adds up its share of the bins over the cluster and hands the sums to all
      cluster_sync();
      const int per = bins / CS;
      for (int b = rank * per + tid; b < (rank + 1) * per; b += THREADS) {
        uint32_t x[kMaxCluster], sum = 0;
#pragma unroll
        for (int r = 0; r < kMaxCluster; ++r) x[r] = r < CS ? ld_cluster_u32(cluster_addr(smem_u32(&hist[b]), r)) : 0;
#pragma unroll
        for (int r = 0; r < kMaxCluster; ++r) sum += x[r];
#pragma unroll
        for (int r = 0; r < kMaxCluster; ++r)
          if (r < CS) st_cluster_u32(cluster_addr(smem_u32(&total[b]), r), sum);
      }
      cluster_sync();
    } else {
      __syncthreads();
    }
    const uint32_t* sums = over_all ? total : hist;
    // from the best bin down: thread `tid` has bins [top - per, top) of them
    const int per = bins / THREADS, top = bins - tid * per;
    uint32_t mine = 0;
    for (int b = 1; b <= per; ++b) mine += sums[top - b];
    const uint32_t before = block_scan<THREADS>(make_uint2(mine, 0), warp_s).x;
    if (before < need && need <= before + mine) {
      uint32_t at = before;
      for (int b = 1; b <= per; ++b) {
        const uint32_t x = sums[top - b];
        if (need <= at + x) {
          found[0] = top - b;
          found[1] = need - at;
          break;
        }
        at += x;
      }
    }
    __syncthreads();
    prefix |= found[0] << shift;
    need = found[1];
  };
  __syncthreads();
  // first digit.  Four groups a thread on their way at a time
  for (int base = g0; base < g1; base += 4 * THREADS) {
    int pg[4];
    uint4 x[4];
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      const int g = base + v * THREADS + tid;
      pg[v] = g < g1 ? table[(first + 4 * g) >> c.log_page] : -1;
    }
#pragma unroll
    for (int v = 0; v < 4; ++v) x[v] = keys_at(base + v * THREADS + tid, pg[v]);
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      const int g = base + v * THREADS + tid;
      if (base + v * THREADS + (tid & ~31) >= g1) break;  // nothing for this warp
      if (g < g1) {
        if ((unsigned)pg[v] >= (unsigned)c.pages) report_page(c.status, i);
        if (held) reinterpret_cast<uint4*>(keys_s)[place(g - g0)] = x[v];
      }
      count(hists[0], g < g1 ? free_slots(g) : 0, x[v], 21, 2048);
    }
  }
  for (int b = tid; b < kBins; b += THREADS) hists[1][b] = 0;
  find(hists[0], 21, 2048, CS > 1);
  // the keys that share it, by themselves if they are not too many
  auto ties = [&](int g, const uint4& x, int shift) -> uint32_t {
    const uint32_t d = prefix >> shift;
    return ((x.x >> shift == d) | (x.y >> shift == d) << 1 | (x.z >> shift == d) << 2 | (x.w >> shift == d) << 3) & free_slots(g);
  };
  for (int base = g0; base < g1; base += THREADS) {
    const int g = base + tid;
    const uint4 x = g < g1 ? keys_of(g) : make_uint4(0, 0, 0, 0);
    const uint32_t m = g < g1 ? ties(g, x, 21) : 0, key[4] = {x.x, x.y, x.z, x.w};
    // one addition a warp
    uint32_t n = 0, mine[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const unsigned b = __ballot_sync(0xffffffffu, m >> u & 1);
      mine[u] = n + __popc(b & ((1u << lane_id()) - 1));
      n += __popc(b);
    }
    if (n == 0) continue;
    uint32_t at = lane_id() == 0 ? atomicAdd(&ntied, n) : 0;
    at = __shfl_sync(0xffffffffu, at, 0);
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if ((m >> u & 1) && at + mine[u] < kSet) tied[at + mine[u]] = key[u];
  }
  for (int b = tid; b < kBins; b += THREADS) hists[0][b] = 0;
  // In a cluster every CTA takes the others' sets to its own, and the other digits need no more of it
  __syncthreads();
  bool few = ntied <= kSet;
  uint32_t n = ntied;
  if (CS > 1) {
    // threads / 8 to each of the others
    cluster_sync();
    const int r = tid * kMaxCluster / THREADS, k0 = tid % (THREADS / kMaxCluster);
    uint32_t to = n, of = 0, sum = 0, most = 0;
#pragma unroll
    for (int x = 0; x < kMaxCluster; ++x) {
      const uint32_t y = x < CS ? ld_cluster_u32(cluster_addr(smem_u32(&ntied), x)) : 0;
      sum += y;
      most = max(most, y);
      if (x == r) of = y;
      if (x < r && x != rank) to += y;
    }
    few = most <= kSet && sum <= kTied;
    if (few && r < CS && r != rank) {
#pragma unroll 4
      for (uint32_t k = k0; k < of; k += THREADS / kMaxCluster)
        tied[to + k] = ld_cluster_u32(cluster_addr(smem_u32(&tied[k]), r));
    }
    n = sum;
    cluster_sync();
  }
#pragma unroll 1
  for (int pass = 1; pass < 3; ++pass) {
    const int above = pass == 1 ? 21 : 10, shift = pass == 1 ? 10 : 0, bins = pass == 1 ? 2048 : 1024;
    uint32_t* hist = hists[pass & 1];
    if (few) {
      for (uint32_t k = tid; k < n; k += THREADS)
        if (tied[k] >> above == prefix >> above) atomicAdd(&hist[tied[k] >> shift & bins - 1], 1u);
    } else {
      for (int base = g0; base < g1; base += THREADS) {
        const int g = base + tid;
        const uint4 x = g < g1 ? keys_of(g) : make_uint4(0, 0, 0, 0);
        count(hist, g < g1 ? ties(g, x, above) : 0, x, shift, bins);
      }
    }
    find(hist, shift, bins, CS > 1 && !few);
  }
  // prefix is the k-th best key, and `need` of its slots stay, the lowest ones.  A thread has `per`
  // consecutive groups; bits: slots of the first eight above the k-th best, and equal to it
  const int per = (g1 - g0 + THREADS - 1) / THREADS, ga = min(g1, g0 + tid * per), gb = min(g1, ga + per);
  uint32_t above = 0, equal = 0, bits_a = 0, bits_e = 0;
  for (int g = ga; g < gb; ++g) {
    const uint4 x = keys_of(g);
    const uint32_t m = free_slots(g);
    const uint32_t a = ((x.x > prefix) | (x.y > prefix) << 1 | (x.z > prefix) << 2 | (x.w > prefix) << 3) & m;
    const uint32_t e = ((x.x == prefix) | (x.y == prefix) << 1 | (x.z == prefix) << 2 | (x.w == prefix) << 3) & m;
    above += __popc(a);
    equal += __popc(e);
    if (g - ga < 8) {
      bits_a |= a << 4 * (g - ga);
      bits_e |= e << 4 * (g - ga);
    }
  }
  const uint32_t mine_above = above, mine_equal = equal;
  const uint2 sums = block_scan<THREADS>(make_uint2(above, equal), warp_s);
  above = sums.x;
  equal = sums.y;
  if (CS > 1) {
    if (tid == THREADS - 1) {
      counts[0] = above + mine_above;
      counts[1] = equal + mine_equal;
    }
    cluster_sync();
    uint32_t a[kMaxCluster], e[kMaxCluster];
#pragma unroll
    for (int r = 0; r < kMaxCluster; ++r) {
      a[r] = r < rank ? ld_cluster_u32(cluster_addr(smem_u32(&counts[0]), r)) : 0;
      e[r] = r < rank ? ld_cluster_u32(cluster_addr(smem_u32(&counts[1]), r)) : 0;
    }
#pragma unroll
    for (int r = 0; r < kMaxCluster; ++r) {
      above += a[r];
      equal += e[r];
    }
    // Both sums go through the barrier, so that the others' counts have been read when it is reached;
    // what this CTA still writes is no business of the cluster's
    asm volatile("barrier.cluster.arrive.relaxed.aligned;" : "+r"(above), "+r"(equal)::"memory");
  }
  auto keep = [&](bool is_above, int t) {
    if (is_above || equal < need) kept[p.s + above + min(equal, need)] = t;
    above += is_above;
    equal += !is_above;
  };
  if (per <= 8) {
    for (uint32_t m = bits_a | bits_e; m; m &= m - 1) {
      const int u = __ffs(m) - 1;
      keep(bits_a >> u & 1, first + 4 * ga + u);
    }
  } else if (mine_above + mine_equal > 0) {
    for (int g = ga; g < gb; ++g) {
      const uint4 x = keys_of(g);
      const uint32_t key[4] = {x.x, x.y, x.z, x.w}, m = free_slots(g);
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if ((m >> u & 1) && key[u] >= prefix) keep(key[u] > prefix, first + 4 * g + u);
    }
  }
  if (CS > 1) asm volatile("barrier.cluster.wait.aligned;" ::: "memory");  // nobody leaves while its counts are read
}

template <int THREADS>
__global__ void __launch_bounds__(THREADS, 1024 / THREADS) evict_move(const __grid_constant__ EvictParams p) {
  constexpr int kRows = THREADS;  // of a batch, at most (D = 64)
  // Pages that a batch's rows come from and go to, and their slots; -1: nothing to move.  Three batches:
  // the one that is looked up, the one that is loaded, and the one before, which slower warps may
  // still be storing.
  __shared__ int from_s[3][kRows], to_s[3][kRows], slot_s[3][kRows];
  grid_dep_wait();
  grid_dep_launch();
  const Paged& c = p.c;
  const int CS = gridDim.x / 2, rank = blockIdx.x % CS;
  const bool is_v = (int)blockIdx.x >= CS;
  const int i = blockIdx.y / c.H, h = blockIdx.y - i * c.H;
  const int32_t* kept = p.kept + (size_t)blockIdx.y * p.B;
  const int32_t* table = c.table + (size_t)i * c.max_pages;
  // new_lens may be lens: nothing else here reads it
  if (blockIdx.x == 0 && h == 0 && threadIdx.x == 0) p.new_lens[i] = min(c.len(i), p.B);
  uint4* base = is_v ? p.v : p.k;
  const int64_t stride = is_v ? p.v_stride : p.k_stride;
  const int ch = c.D / 8, rows = THREADS / ch, mine = rows * kMoveBatch;  // pieces of a row; rows at a time, and of a batch
  const int r = threadIdx.x / ch, x = threadIdx.x - r * ch, in_page = (1 << c.log_page) - 1;
  auto piece = [&](int pg, int t) { return base + pg * stride + (int64_t)(((size_t)h << c.log_page) + (t & in_page)) * ch + x; };
  // one row a thread: the rows of this CTA's part of the batch at j0
  auto look_up = [&](int j0, int buf) {
    const int k = threadIdx.x, j = j0 + rank * mine + k;
    if (k >= mine) return;
    const int t = j < p.B ? kept[j] : -1;
    int from = -1, to = -1;
    if (t > j) {
      from = table[t >> c.log_page];
      to = table[j >> c.log_page];
      if ((unsigned)from >= (unsigned)c.pages || (unsigned)to >= (unsigned)c.pages) {
        report_page(c.status, i);
        from = to = -1;
      }
    }
    from_s[buf][k] = from;
    to_s[buf][k] = to;
    slot_s[buf][k] = t;
  };
  look_up(0, 0);
  __syncthreads();
  const int batch = CS * mine;
  for (int j0 = 0, buf = 0, next = 1; j0 < p.B; j0 += batch, buf = next, next = next == 2 ? 0 : next + 1) {
    uint4 y[kMoveBatch];
    float w[kMoveBatch];
#pragma unroll
    for (int u = 0; u < kMoveBatch; ++u) {
      const int k = u * rows + r, pg = from_s[buf][k], t = slot_s[buf][k];
      if (pg >= 0) {
        y[u] = *piece(pg, t);
        if (!is_v && x == 0) w[u] = p.scores[c.slot_row(pg, h, t)];
      }
    }
    if (j0 + batch < p.B) look_up(j0 + batch, next);
    // the whole batch has been read
    if (CS > 1) cluster_sync();
    else __syncthreads();
#pragma unroll
    for (int u = 0; u < kMoveBatch; ++u) {
      const int k = u * rows + r, pg = to_s[buf][k], j = j0 + rank * mine + k;
      if (pg >= 0) {
        *piece(pg, j) = y[u];
        if (!is_v && x == 0) p.scores[c.slot_row(pg, h, j)] = w[u];
      }
    }
  }
}

}  // namespace
}  // namespace kvpop

using namespace kvpop;

extern "C" kvpop_status kvpop_paged_evict(void* kp, int64_t kp_stride, void* vp, int64_t vp_stride, float* scores, int n,
                                          int H, int D, kvpop_budget budget, const int32_t* lens, const int32_t* table,
                                          int max_pages, int pages, int page, int32_t* kept, int32_t* new_lens,
                                          kvpop_stream stream) {
  const char* name = "kvpop_paged_evict";
  if (!scores || !kept || !new_lens) {
    set_last_error("%s: scores, kept and new_lens must be non-NULL", name);
    return KVPOP_ERR_INVALID_ARG;
  }
  const long long B = (long long)budget.s + budget.w + budget.k;
  if (budget.s < 0 || budget.w < 0 || budget.k < 0 || B < 1 || B > (1 << 30)) {
    set_last_error("%s: bad budget s=%d w=%d k=%d", name, budget.s, budget.w, budget.k);
    return KVPOP_ERR_INVALID_ARG;
  }
  EvictParams prm;
  kvpop_status st = paged_check(name, n, n, H, D, nullptr, lens, table, max_pages, pages, page, &prm.c);
  if (st == KVPOP_OK) st = paged_check_cache(name, "kp", kp, kp_stride, H, D, pages, page);
  if (st == KVPOP_OK) st = paged_check_cache(name, "vp", vp, vp_stride, H, D, pages, page);
  if (st != KVPOP_OK) return st;
  if (((long long)n * H) > 65535) {
    set_last_error("%s: n * H = %lld above 65535", name, (long long)n * H);
    return KVPOP_ERR_UNSUPPORTED;
  }
  if ((reinterpret_cast<uintptr_t>(scores) & 15) ||
      ((reinterpret_cast<uintptr_t>(kept) | reinterpret_cast<uintptr_t>(new_lens)) & 3)) {
    set_last_error("%s: scores must be 16-byte aligned, kept and new_lens 4-byte", name);
    return KVPOP_ERR_UNSUPPORTED;
  }
  prm.scores = scores;
  prm.k = (uint4*)kp;
  prm.v = (uint4*)vp;
  prm.k_stride = kp_stride / 8;
  prm.v_stride = vp_stride / 8;
  prm.kept = kept;
  prm.new_lens = new_lens;
  prm.s = budget.s;
  prm.w = budget.w;
  prm.top = budget.k;
  prm.B = (int)B;
  cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
  // CTAs a (sequence, head): as many as fill the SMs, with 2048 slots each at least
  const long long heads = (long long)n * H, most = (long long)max_pages * page;
  int CS = 1;
  while (CS < kMaxCluster && heads * CS * 2 <= 2ll * num_sms() && most / (CS * 2) >= 2048) CS *= 2;
  // The host knows the table's width, not the lengths.  A table for more slots than the sequences have
  // leaves fewer CTAs an SM: 64 sequences of 1700 .. 4099 slots to 2048 take 180 us with a tight table
  // and 160 with one for 131 072 slots (252 and 232 of 8000 .. 16 001), 200 of 1000 .. 3001 with 2 heads
  // of D = 64 31 and 39.  Room for four CTAs an SM at any width: 180, 262 and 34, but 328 instead of
  // 272 for 64 sequences of 16 000 .. 32 001, whose keys are then read again.
  prm.held = (int)min((long long)(kCacheBytes / 16 * 8 / 9), most / CS / 4 + 4);
  auto select = CS > 1 ? evict_select<1024> : evict_select<512>;
  static std::atomic<uint64_t> ready{0};  // bit d: the kernels are set up on device d
  const int dev = current_device();
  if (dev >= 64 || !(ready.load(std::memory_order_acquire) >> dev & 1)) {
    for (auto kern : {evict_select<1024>, evict_select<512>}) {
      st = cuda_check(cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kCacheBytes + kTied * 4),
                      "kvpop_paged_evict: smem attribute");
      if (st != KVPOP_OK) return st;
    }
    if (dev < 64) ready.fetch_or(1ull << dev, std::memory_order_release);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(CS, (unsigned)heads);
  cfg.blockDim = dim3(CS > 1 ? 1024 : 512);
  cfg.dynamicSmemBytes = ((size_t)prm.held + prm.held / 8) * 16 + (CS > 1 ? kTied : kSet) * 4;
  cfg.stream = cs;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = CS;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  st = cuda_check(cudaLaunchKernelEx(&cfg, select, prm), "kvpop_paged_evict: launch");
  if (st != KVPOP_OK) return st;
  // CTAs a head's K (and as many its V): one an SM as long as there are few heads, and rows for them
  const bool few = heads * 2 <= num_sms();
  int CM = 1;
  while (CM < kMaxCluster && heads * 4 * CM <= num_sms() && (long long)CM * kMoveFew / (D / 8) * kMoveBatch < B) CM *= 2;
  cfg.gridDim = dim3(2 * CM, (unsigned)heads);
  cfg.blockDim = dim3(few ? kMoveFew : kMoveMany);
  cfg.dynamicSmemBytes = 0;
  attr[1].val.clusterDim.x = CM;
  return cuda_check(cudaLaunchKernelEx(&cfg, few ? evict_move<kMoveFew> : evict_move<kMoveMany>, prm),
                    "kvpop_paged_evict: move launch");
}
