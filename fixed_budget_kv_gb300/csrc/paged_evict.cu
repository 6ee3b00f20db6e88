// kvpop_paged_evict: each head of a paged cache down to B = s + w + k slots by the attention
// weight that its keys have received.
//
// Of a sequence with len > B slots, a head keeps slots [0, s), [len - w, len) and the k best of
// [s, len - w) in the order (score falling, slot rising), NaN counting as -inf and -0 as +0.
//
// evict_select, one cluster a (sequence, head), its CTAs a part of the slots each: the k-th best
// score by a radix select (11 + 11 + 10 bits of an order-preserving key, the CTAs' histograms
// added up through distributed shared memory), then the kept slots in their order: a thread has
// consecutive slots, so one scan gives every thread its place.  Bound by its chain of barriers.
// evict_move: kept slot j goes from kept[j] >= j to j.  One CTA moves one column slice of K or V
// (or the scores) of a head in rising order, a batch at a time: loads, barrier, stores.  The next
// batch's sources lie at or above its own slots, so behind everything stored before: nothing is
// lost and no second copy is needed.  Bound by memory.
#include <atomic>

#include "paged.cuh"
#include "segments.cuh"

namespace kvpop {
namespace {

constexpr int kBins = 2048;
constexpr int kCacheKeys = 49152;  // keys of a CTA's part held in shared memory, at most
constexpr int kMaxCluster = 8;
constexpr int kMoveThreads = 256;
constexpr int kMoveBatch = 8;  // pieces that a thread has in flight
constexpr int kMoveRows = kMoveThreads * kMoveBatch / 2;  // rows of a batch, at most (32-byte slices)

struct EvictParams {
  Paged c;
  float* scores;
  uint4 *k, *v;
  int64_t k_stride, v_stride;  // 16-byte pieces between pages
  int32_t *kept, *new_lens;
  int s, w, top, B, slices;
  int held;  // keys that the select's shared memory has room for
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

// Exclusive sum over the block.  Two barriers.
template <int THREADS>
__device__ __forceinline__ uint32_t block_scan(uint32_t x, uint32_t* warp_s) {
  uint32_t y = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t z = __shfl_up_sync(0xffffffffu, y, o);
    if (lane_id() >= o) y += z;
  }
  __syncthreads();  // the sums of the scan before have been read
  if (lane_id() == 31) warp_s[warp_id()] = y;
  __syncthreads();
  uint32_t before = lane_id() < warp_id() ? warp_s[lane_id()] : 0;
  return __reduce_add_sync(0xffffffffu, before) + y - x;
}

template <int THREADS>
__global__ void __launch_bounds__(THREADS) evict_select(const __grid_constant__ EvictParams p) {
  static_assert(THREADS / 32 <= 32 && kBins % THREADS == 0, "one warp holds the warps' sums");
  extern __shared__ __align__(16) uint32_t keys_s[];  // the part's keys, if they fit
  __shared__ uint32_t hist[kBins], total[kBins];
  __shared__ uint32_t warp_s[THREADS / 32];
  __shared__ uint32_t found[2];   // the bin of the k-th best, and how many of it stay
  __shared__ uint32_t counts[2];  // keys of this part above the k-th best, and equal to it
  const int tid = threadIdx.x;
  for (int b = tid; b < kBins; b += THREADS) hist[b] = 0;
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
  const bool held = (g1 - g0) * 4 <= p.held;
  // the page of group g < g1; 0 and a report where the table names none
  auto page_at = [&](int g, bool& bad) -> int {
    const int pg = g < g1 ? c.table[(size_t)i * c.max_pages + ((first + 4 * g) >> c.log_page)] : 0;
    bad = pg < 0 || pg >= c.pages;
    return bad ? 0 : pg;
  };
  auto keys_at = [&](int g, int pg, bool bad) -> uint4 {
    float4 x = make_float4(neg_inf(), neg_inf(), neg_inf(), neg_inf());
    if (g < g1 && !bad) x = *reinterpret_cast<const float4*>(p.scores + c.slot_row(pg, h, first + 4 * g));
    return make_uint4(order_key(x.x), order_key(x.y), order_key(x.z), order_key(x.w));
  };
  auto keys_of = [&](int g) -> uint4 {
    if (held) return reinterpret_cast<const uint4*>(keys_s)[g - g0];
    bool bad;
    const int pg = page_at(g, bad);
    return keys_at(g, pg, bad);
  };
  auto free_slot = [&](int t) { return t >= p.s && t < end; };
  uint32_t prefix = 0, mask = 0, need = p.top;
  // one warp's groups into the histogram
  auto count = [&](int g, const uint4& x, int shift, int bins) {
    const uint32_t key[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const bool on = g < g1 && free_slot(first + 4 * g + u) && (key[u] & mask) == prefix;
      const uint32_t bin = (key[u] >> shift) & (bins - 1);
      // many equal scores (nothing received yet): one addition for the whole warp
      const unsigned act = __ballot_sync(0xffffffffu, on);
      if (act == 0) continue;
      const int lead = __ffs(act) - 1;
      const uint32_t ref = __shfl_sync(0xffffffffu, bin, lead);
      if (__all_sync(0xffffffffu, !on || bin == ref)) {
        if (lane_id() == lead) atomicAdd(&hist[bin], (uint32_t)__popc(act));
      } else if (on) {
        atomicAdd(&hist[bin], 1u);
      }
    }
  };
  __syncthreads();
  for (int pass = 0; pass < 3; ++pass) {
    const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, bins = pass == 2 ? 1024 : 2048;
    if (pass == 0) {
      // four groups a thread on their way at a time
      for (int base = g0; base < g1; base += 4 * THREADS) {
        int pg[4];
        bool bad[4];
        uint4 x[4];
#pragma unroll
        for (int v = 0; v < 4; ++v) pg[v] = page_at(base + v * THREADS + tid, bad[v]);
#pragma unroll
        for (int v = 0; v < 4; ++v) x[v] = keys_at(base + v * THREADS + tid, pg[v], bad[v]);
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          const int g = base + v * THREADS + tid;
          if (bad[v]) report_page(c.status, i);
          if (held && g < g1) reinterpret_cast<uint4*>(keys_s)[g - g0] = x[v];
          count(g, x[v], shift, bins);
        }
      }
    } else {
      for (int base = g0; base < g1; base += THREADS) {
        const int g = base + tid;
        count(g, g < g1 ? keys_of(g) : make_uint4(0, 0, 0, 0), shift, bins);
      }
    }
    if (CS > 1) {
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
    const uint32_t* sums = CS > 1 ? total : hist;
    // from the best bin down: thread `tid` has bins [top - per, top) of them
    const int per = bins / THREADS, top = bins - tid * per;
    uint32_t mine = 0;
    for (int b = 1; b <= per; ++b) mine += sums[top - b];
    const uint32_t before = block_scan<THREADS>(mine, warp_s);
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
    mask |= (uint32_t)(bins - 1) << shift;
    need = found[1];
    if (pass < 2) {
      // in a cluster every CTA has read it: the sums are out
      for (int b = tid; b < kBins; b += THREADS) hist[b] = 0;
      __syncthreads();
    }
  }
  // prefix is the k-th best key, and `need` of its slots stay, the lowest ones
  const int per = (g1 - g0 + THREADS - 1) / THREADS, ga = min(g1, g0 + tid * per), gb = min(g1, ga + per);
  uint32_t above = 0, equal = 0;
  for (int g = ga; g < gb; ++g) {
    const uint4 x = keys_of(g);
    const uint32_t key[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (free_slot(first + 4 * g + u)) {
        above += key[u] > prefix;
        equal += key[u] == prefix;
      }
  }
  const uint32_t mine_above = above, mine_equal = equal;
  above = block_scan<THREADS>(above, warp_s);
  equal = block_scan<THREADS>(equal, warp_s);
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
  }
  if (mine_above + mine_equal > 0) {
    for (int g = ga; g < gb; ++g) {
      const uint4 x = keys_of(g);
      const uint32_t key[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if (free_slot(first + 4 * g + u)) {
          const bool stays = key[u] > prefix || (key[u] == prefix && equal < need);
          if (stays) kept[p.s + above + min(equal, need)] = first + 4 * g + u;
          above += key[u] > prefix;
          equal += key[u] == prefix;
        }
    }
  }
  if (CS > 1) cluster_sync();  // nobody leaves while its counts are read
}

// Where a batch's rows come from and go to; -1: nothing to move.  Three batches: of the one that is
// looked up, the one that is loaded, and the one before, which slower warps may still be storing.
struct Moves {
  int64_t src[3][kMoveRows], dst[3][kMoveRows];
};

// Kept rows j -> their slots, BATCH pieces of type V a thread and batch, `per` pieces a row.
// at(page, place) is the row's first piece.
template <int BATCH, typename V, typename At>
__device__ __forceinline__ void move_rows(const EvictParams& p, Moves& m, const int32_t* kept, int i, int per, V* base, At at) {
  const Paged& c = p.c;
  const int rows = kMoveThreads / per, batch = rows * BATCH, r = threadIdx.x / per, x = threadIdx.x - r * per;
  auto resolve = [&](int j0, int buf) {
    for (int k = threadIdx.x; k < batch; k += kMoveThreads) {
      const int j = j0 + k, t = j < p.B ? kept[j] : -1;
      int64_t src = -1, dst = -1;
      if (t > j) {
        const int a = c.page_of(i, t), b = c.page_of(i, j);
        if (a >= 0 && b >= 0) {
          src = at(a, t);
          dst = at(b, j);
        } else {
          report_page(c.status, i);
        }
      }
      m.src[buf][k] = src;
      m.dst[buf][k] = dst;
    }
  };
  resolve(0, 0);
  __syncthreads();
  for (int j0 = 0, buf = 0, next = 1; j0 < p.B; j0 += batch, buf = next, next = next == 2 ? 0 : next + 1) {
    V y[BATCH];
#pragma unroll
    for (int u = 0; u < BATCH; ++u) {
      const int64_t src = m.src[buf][u * rows + r];
      if (src >= 0) y[u] = base[src + x];
    }
    if (j0 + batch < p.B) resolve(j0 + batch, next);
    __syncthreads();  // the whole batch has been read
#pragma unroll
    for (int u = 0; u < BATCH; ++u) {
      const int64_t dst = m.dst[buf][u * rows + r];
      if (dst >= 0) base[dst + x] = y[u];
    }
  }
}

__global__ void __launch_bounds__(kMoveThreads, 4) evict_move(const __grid_constant__ EvictParams p) {
  __shared__ Moves moves;
  grid_dep_wait();
  grid_dep_launch();
  const Paged& c = p.c;
  const int i = blockIdx.y / c.H, h = blockIdx.y - i * c.H, part = blockIdx.x;
  const int32_t* kept = p.kept + (size_t)blockIdx.y * p.B;
  const int ch = c.D / 8, per = ch / p.slices;  // pieces of a row, and of a slice
  if (part == 2 * p.slices) {
    // new_lens may be lens: nothing else here reads it
    if (h == 0 && threadIdx.x == 0) p.new_lens[i] = min(c.len(i), p.B);
    move_rows<kMoveRows / kMoveThreads>(p, moves, kept, i, 1, p.scores, [&](int pg, int t) { return (int64_t)c.slot_row(pg, h, t); });
    return;
  }
  const bool is_v = part >= p.slices;
  const int64_t stride = is_v ? p.v_stride : p.k_stride;
  const int x0 = (part - (is_v ? p.slices : 0)) * per;
  move_rows<kMoveBatch>(p, moves, kept, i, per, is_v ? p.v : p.k, [&](int pg, int t) {
    return pg * stride + (int64_t)(((size_t)h << c.log_page) + (t & ((1 << c.log_page) - 1))) * ch + x0;
  });
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
  prm.held = (int)min((long long)kCacheKeys, (most / CS + 16) / 4 * 4);
  auto select = CS > 1 ? evict_select<1024> : evict_select<512>;
  static std::atomic<uint64_t> ready{0};  // bit d: the kernels are set up on device d
  const int dev = current_device();
  if (dev >= 64 || !(ready.load(std::memory_order_acquire) >> dev & 1)) {
    for (auto kern : {evict_select<1024>, evict_select<512>}) {
      st = cuda_check(cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kCacheKeys * 4),
                      "kvpop_paged_evict: smem attribute");
      if (st != KVPOP_OK) return st;
    }
    if (dev < 64) ready.fetch_or(1ull << dev, std::memory_order_release);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(CS, (unsigned)heads);
  cfg.blockDim = dim3(CS > 1 ? 1024 : 512);
  cfg.dynamicSmemBytes = (size_t)prm.held * 4;
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
  // column slices of a head's K and V: down to 32 bytes, until there are four CTAs an SM
  prm.slices = 1;
  while (prm.slices < D / 16 && heads * 2 * prm.slices < 4ll * num_sms()) prm.slices *= 2;
  return cuda_check(launch_pdl(evict_move, dim3(2 * prm.slices + 1, (unsigned)heads), dim3(kMoveThreads), 0, cs, prm),
                    "kvpop_paged_evict: move launch");
}
