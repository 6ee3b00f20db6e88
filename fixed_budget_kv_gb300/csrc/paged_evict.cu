// kvpop_paged_evict: each head of a paged cache down to B = s + w + k slots by the attention
// weight that its keys have received.
//
// Of a sequence with len > B slots, a head keeps slots [0, s), [len - w, len) and the k best of
// [s, len - w) in the order (score falling, slot rising), NaN counting as -inf and -0 as +0.
//
// evict_select, one cluster a (sequence, head), its CTAs a part of the slots each: the k-th best
// score by a radix select (11 + 11 + 10 bits of an order-preserving key, the CTAs' histograms
// added up through distributed shared memory), then the kept slots in their order by a scan.
// evict_move: kept slot j goes from kept[j] >= j to j.  One CTA moves one column slice of K or V
// (or the scores) of a head in rising order, a batch at a time: loads, barrier, stores.  The next
// batch's sources lie at or above its own slots, so behind everything stored before: nothing is
// lost and no second copy is needed.
#include <atomic>

#include "paged.cuh"

namespace kvpop {
namespace {

constexpr int kThreads = 512;
constexpr int kBins = 2048;
constexpr int kCacheKeys = 24576;  // keys of a CTA's part held in shared memory
constexpr int kMaxCluster = 8;
constexpr int kMoveThreads = 512;
constexpr int kMoveBatch = 8;  // rows that a thread has in flight

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

// Exclusive sum over the block; `all` is the block's sum.  Two barriers.
__device__ __forceinline__ uint32_t block_scan(uint32_t x, uint32_t* warp_s, uint32_t& all) {
  uint32_t y = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t z = __shfl_up_sync(0xffffffffu, y, o);
    if (lane_id() >= o) y += z;
  }
  __syncthreads();  // the sums of the scan before have been read
  if (lane_id() == 31) warp_s[warp_id()] = y;
  __syncthreads();
  uint32_t before = 0, sum = 0;
#pragma unroll
  for (int i = 0; i < kThreads / 32; ++i) {
    const uint32_t z = warp_s[i];
    if (i < warp_id()) before += z;
    sum += z;
  }
  all = sum;
  return before + y - x;
}

__global__ void __launch_bounds__(kThreads) evict_select(const __grid_constant__ EvictParams p) {
  extern __shared__ __align__(16) uint32_t keys_s[];  // the part's keys, if they fit
  __shared__ uint32_t hist[kBins], total[kBins];
  __shared__ uint32_t warp_s[kThreads / 32];
  __shared__ uint32_t found[2];      // the bin of the k-th best, and how many of it stay
  __shared__ uint32_t counts[2];     // keys of this part above the k-th best, and equal to it
  grid_dep_wait();
  grid_dep_launch();
  const Paged& c = p.c;
  const int CS = gridDim.x, rank = blockIdx.x;  // one cluster along x
  const int i = blockIdx.y / c.H, h = blockIdx.y - i * c.H;
  const int tid = threadIdx.x, len = c.len(i);
  int32_t* kept = p.kept + (size_t)blockIdx.y * p.B;
  if (len <= p.B) {
    for (int j = rank * kThreads + tid; j < p.B; j += CS * kThreads) kept[j] = j < len ? j : -1;
    return;  // the whole cluster
  }
  for (int j = rank * kThreads + tid; j < p.s; j += CS * kThreads) kept[j] = j;
  for (int j = rank * kThreads + tid; j < p.w; j += CS * kThreads) kept[p.s + p.top + j] = len - p.w + j;
  if (p.top == 0) return;
  // the slots that may go, [s, end), in groups of four: this CTA has groups [g0, g1)
  const int end = len - p.w, first = p.s & ~3, groups = (end - first + 3) / 4;
  const int g0 = (int)((long long)groups * rank / CS), g1 = (int)((long long)groups * (rank + 1) / CS);
  const bool held = (g1 - g0) * 4 <= p.held;
  auto from_memory = [&](int g) -> uint4 {
    const int t = first + 4 * g, pg = c.page_of(i, t);
    if (pg < 0) {
      report_page(c.status, i);
      const uint32_t low = order_key(__int_as_float(0xff800000));
      return make_uint4(low, low, low, low);
    }
    const float4 x = *reinterpret_cast<const float4*>(p.scores + c.slot_row(pg, h, t));
    return make_uint4(order_key(x.x), order_key(x.y), order_key(x.z), order_key(x.w));
  };
  auto keys_of = [&](int g) { return held ? reinterpret_cast<const uint4*>(keys_s)[g - g0] : from_memory(g); };
  if (held) {
#pragma unroll 4
    for (int g = g0 + tid; g < g1; g += kThreads) reinterpret_cast<uint4*>(keys_s)[g - g0] = from_memory(g);
  }
  auto free_slot = [&](int t) { return t >= p.s && t < end; };
  uint32_t prefix = 0, mask = 0, need = p.top;
  for (int pass = 0; pass < 3; ++pass) {
    const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, bits = pass == 2 ? 10 : 11, bins = 1 << bits;
    for (int b = tid; b < bins; b += kThreads) hist[b] = 0;
    __syncthreads();
    for (int base = g0; base < g1; base += kThreads) {
      const int g = base + tid;
      const uint4 x = g < g1 ? keys_of(g) : make_uint4(0, 0, 0, 0);
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
    }
    if (CS > 1) {
      // CTA r adds up its share of the bins over the cluster and hands the sums to all
      cluster_sync();
      const int per = bins / CS;
      for (int b = rank * per + tid; b < (rank + 1) * per; b += kThreads) {
        uint32_t sum = 0;
        for (int r = 0; r < CS; ++r) sum += ld_cluster_u32(cluster_addr(smem_u32(&hist[b]), r));
        for (int r = 0; r < CS; ++r) st_cluster_u32(cluster_addr(smem_u32(&total[b]), r), sum);
      }
      cluster_sync();
    } else {
      __syncthreads();
    }
    const uint32_t* sums = CS > 1 ? total : hist;
    // from the best bin down: thread `tid` has bins [top - per, top) of them
    const int per = bins / kThreads, top = bins - tid * per;
    uint32_t mine = 0;
    for (int b = 1; b <= per; ++b) mine += sums[top - b];
    uint32_t all;
    const uint32_t before = block_scan(mine, warp_s, all);
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
  }
  // prefix is the k-th best key, and `need` of its slots stay, the lowest ones
  uint32_t above = 0, equal = 0;
  if (CS > 1) {
    for (int g = g0 + tid; g < g1; g += kThreads) {
      const uint4 x = keys_of(g);
      const uint32_t key[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if (free_slot(first + 4 * g + u)) {
          above += key[u] > prefix;
          equal += key[u] == prefix;
        }
    }
    above = __reduce_add_sync(0xffffffffu, above);
    equal = __reduce_add_sync(0xffffffffu, equal);
    if (tid < 2) counts[tid] = 0;
    __syncthreads();
    if (lane_id() == 0) {
      atomicAdd(&counts[0], above);
      atomicAdd(&counts[1], equal);
    }
    cluster_sync();
    above = equal = 0;
    for (int r = 0; r < rank; ++r) {
      above += ld_cluster_u32(cluster_addr(smem_u32(&counts[0]), r));
      equal += ld_cluster_u32(cluster_addr(smem_u32(&counts[1]), r));
    }
  }
  for (int base = g0; base < g1; base += kThreads) {
    const int g = base + tid;
    uint32_t key[4] = {0, 0, 0, 0}, n = 0;  // slots above in the low half, equal ones in the high half
    bool on[4] = {false, false, false, false};
    if (g < g1) {
      const uint4 x = keys_of(g);
      key[0] = x.x, key[1] = x.y, key[2] = x.z, key[3] = x.w;
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        on[u] = free_slot(first + 4 * g + u);
        if (on[u]) n += key[u] > prefix ? 1u : key[u] == prefix ? 0x10000u : 0u;
      }
    }
    uint32_t all;
    const uint32_t before = block_scan(n, warp_s, all);
    uint32_t a = above + (before & 0xffffu), e = equal + (before >> 16);
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (on[u]) {
        const bool stays = key[u] > prefix || (key[u] == prefix && e < need);
        if (stays) kept[p.s + a + min(e, need)] = first + 4 * g + u;
        a += key[u] > prefix;
        e += key[u] == prefix;
      }
    above += all & 0xffffu;
    equal += all >> 16;
  }
  if (CS > 1) cluster_sync();  // nobody leaves while its counts are read
}

// Rows kept[j] -> j of one slice; `row` gives a slot's address.
template <typename V, typename Row>
__device__ __forceinline__ void move_rows(const EvictParams& p, const int32_t* kept, int i, int per_row, Row row) {
  const Paged& c = p.c;
  const int rows = kMoveThreads / per_row, r = threadIdx.x / per_row;
  for (int base = 0; base < p.B; base += rows * kMoveBatch) {
    V x[kMoveBatch];
    V* to[kMoveBatch];
#pragma unroll
    for (int u = 0; u < kMoveBatch; ++u) {
      const int j = base + u * rows + r, t = j < p.B ? kept[j] : -1;
      to[u] = nullptr;
      if (t > j) {
        const int a = c.page_of(i, t), b = c.page_of(i, j);
        if (a >= 0 && b >= 0) {
          x[u] = *row(a, t);
          to[u] = row(b, j);
        } else {
          report_page(c.status, i);
        }
      }
    }
    __syncthreads();
#pragma unroll
    for (int u = 0; u < kMoveBatch; ++u)
      if (to[u]) *to[u] = x[u];
  }
}

__global__ void __launch_bounds__(kMoveThreads) evict_move(const __grid_constant__ EvictParams p) {
  grid_dep_wait();
  grid_dep_launch();
  const Paged& c = p.c;
  const int i = blockIdx.y / c.H, h = blockIdx.y - i * c.H, part = blockIdx.x;
  const int32_t* kept = p.kept + (size_t)blockIdx.y * p.B;
  if (part == 2 * p.slices) {
    // new_lens may be lens: nothing else here reads it
    if (h == 0 && threadIdx.x == 0) p.new_lens[i] = min(c.len(i), p.B);
    move_rows<float>(p, kept, i, 1, [&](int pg, int t) { return p.scores + c.slot_row(pg, h, t); });
    return;
  }
  const bool is_v = part >= p.slices;
  const int ch = c.D / 8, per = ch / p.slices;  // pieces of a row, and of a slice
  uint4* base = is_v ? p.v : p.k;
  const int64_t stride = is_v ? p.v_stride : p.k_stride;
  const int x = (part - (is_v ? p.slices : 0)) * per + threadIdx.x % per;
  move_rows<uint4>(p, kept, i, per, [&](int pg, int t) {
    return base + pg * stride + (((size_t)h << c.log_page) + (t & ((1 << c.log_page) - 1))) * ch + x;
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
  static std::atomic<uint64_t> ready{0};  // bit d: the kernel is set up on device d
  const int dev = current_device();
  if (dev >= 64 || !(ready.load(std::memory_order_acquire) >> dev & 1)) {
    st = cuda_check(cudaFuncSetAttribute(evict_select, cudaFuncAttributeMaxDynamicSharedMemorySize, kCacheKeys * 4),
                    "kvpop_paged_evict: smem attribute");
    if (st != KVPOP_OK) return st;
    if (dev < 64) ready.fetch_or(1ull << dev, std::memory_order_release);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(CS, (unsigned)heads);
  cfg.blockDim = dim3(kThreads);
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
  st = cuda_check(cudaLaunchKernelEx(&cfg, evict_select, prm), "kvpop_paged_evict: launch");
  if (st != KVPOP_OK) return st;
  // column slices of a head's K and V: down to 32 bytes, until there are two CTAs an SM
  prm.slices = 1;
  while (prm.slices < D / 16 && heads * 2 * prm.slices < 2ll * num_sms()) prm.slices *= 2;
  return cuda_check(launch_pdl(evict_move, dim3(2 * prm.slices + 1, (unsigned)heads), dim3(kMoveThreads), 0, cs, prm),
                    "kvpop_paged_evict: move launch");
}
