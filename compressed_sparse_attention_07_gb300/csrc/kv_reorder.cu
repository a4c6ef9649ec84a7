// The beams' cached states in the order of a selection.
//
// Full pages are shared through the block table; of the last pages, written in part,
// the groups' beams have as many as there are beams, and the pages of beams without
// children are what the second children of others need: E = D, as (children that keep
// a page) = (beams with children).  So a reordering is two kernels: kv_tails_kernel
// copies the written slots of E last pages a group, in every layer, which is bound by
// HBM (2 x the slots' bytes) or, for a few beams, by the latency of parents -> page ids ->
// slots; kv_table_kernel then permutes the table's columns in place, which the first
// still reads.  A warp of each CTA works its group's permutation out by ballots.
#include <algorithm>

#include "kv.cuh"

namespace csa2 {
namespace {

constexpr int kMaxBeams = 64, kThreads = 256, kCols = 64;

struct Layer {
  uint8_t *k, *ks, *v, *vs;
};
template <int kLayers>
struct ReorderArgs {
  int beams, layers, max_pages, num_pages;
  // a page's data in units of 16 bytes, its scales in units of 4; slots 0 .. 63 fill each run
  // of so many of them (a kv head's codes or scales, a 16-byte chunk of its bf16 channels)
  int units, run, sunits, srun;
  int32_t* table;
  const int32_t* parents;
  const int32_t* kv_len;
  int32_t* status;
  Layer layer[kLayers];
};

// What becomes of a group: lane l has its beams l and 32 + l.
struct Plan {
  int n, rest;               // full pages, slots written in the last one
  int parent[2], tail[2];    // of the lane's beams: the parent (-1), and whose last page it has
  bool extra[2];
};
__device__ __forceinline__ int nth_set(uint64_t mask, int r) {  // r < the bits set
  for (; r > 0; --r) mask &= mask - 1;
  return __ffsll((long long)mask) - 1;
}
// The whole warp; false (status set) when the group's parents or lengths are wrong.
__device__ __forceinline__ bool plan_of(int g, int beams, int max_pages, const int32_t* parents, const int32_t* kv_len,
                                        int32_t* status, Plan& p) {
  constexpr uint32_t kAll = 0xffffffffu;
  const int lane = threadIdx.x & 31, first = g * beams;
  const int len0 = __ldg(kv_len + first);
  bool ok = len0 >= 0 && len0 <= (int64_t)max_pages * kPage;
  bool there[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int i = 32 * h + lane;
    there[h] = i < beams;
    p.parent[h] = -1;
    if (there[h]) {
      const int q = __ldg(parents + first + i);
      ok = ok && (q == -1 || (q >= first && q < first + beams)) && __ldg(kv_len + first + i) == len0;
      p.parent[h] = q == -1 ? -1 : q - first;
    }
  }
  if (!__all_sync(kAll, ok)) {
    if (lane == 0) report(status, CSA2_ERR_BAD_INDEX);
    return false;
  }
  p.n = len0 / kPage, p.rest = len0 % kPage;
  uint64_t alive[2], stays = 0, extra = 0;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint64_t bit = p.parent[h] >= 0 ? 1ull << p.parent[h] : 0;
    alive[h] = __reduce_or_sync(kAll, (uint32_t)bit) | (uint64_t)__reduce_or_sync(kAll, (uint32_t)(bit >> 32)) << 32;
    stays |= (uint64_t)__ballot_sync(kAll, p.parent[h] == 32 * h + lane) << (32 * h);
  }
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint32_t same = __match_any_sync(kAll, p.parent[h]);
    const int q = p.parent[h];
    bool keeps = q >= 0;
    if (keeps && (stays >> q & 1)) keeps = q == 32 * h + lane;
    else if (keeps) keeps = __ffs(same) - 1 == lane && !(h == 1 && (alive[0] >> q & 1));
    p.extra[h] = there[h] && !keeps;
    extra |= (uint64_t)__ballot_sync(kAll, p.extra[h]) << (32 * h);
  }
  const uint64_t all = beams == 64 ? ~0ull : (1ull << beams) - 1, dead = all & ~(alive[0] | alive[1]);
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int i = 32 * h + lane;
    p.tail[h] = p.extra[h] ? nth_set(dead, __popcll(extra & ((1ull << i) - 1))) : p.parent[h];
  }
  return true;
}

// The first n of every `run` units (a power of two up to kThreads) of a page of `units`, all
// threads, kDeep units of each on their way.
template <typename V, int kDeep>
__device__ __forceinline__ void copy_page(uint8_t* to, const uint8_t* from, int units, int run, int n) {
  if ((int)(threadIdx.x & (run - 1)) >= n) return;
  const V* src = reinterpret_cast<const V*>(from) + threadIdx.x;
  V* dst = reinterpret_cast<V*>(to) + threadIdx.x;
  for (int u = threadIdx.x; u < units; u += kDeep * kThreads, src += kDeep * kThreads, dst += kDeep * kThreads) {
    V v[kDeep];
#pragma unroll
    for (int i = 0; i < kDeep; ++i)
      if (u + i * kThreads < units) v[i] = src[i * kThreads];
#pragma unroll
    for (int i = 0; i < kDeep; ++i)
      if (u + i * kThreads < units) dst[i * kThreads] = v[i];
  }
}

// Some of a group's copies: job e's last page, its keys (even x) or values in layer x / 2,
// is number e + jobs x.
template <int kLayers>
__global__ void __launch_bounds__(kThreads, 3) kv_tails_kernel(const __grid_constant__ ReorderArgs<kLayers> a) {
  __shared__ int from[kMaxBeams], to[kMaxBeams], jobs, slots;
  griddep_wait();    // every input may be the previous kernel's output
  griddep_launch();  // (kv_table_kernel waits for this one, and lets its own successor start at its end)
  const int g = blockIdx.x, lane = threadIdx.x & 31;
  if (threadIdx.x < 32) {
    Plan p;
    int n = 0;
    if (plan_of(g, a.beams, a.max_pages, a.parents, a.kv_len, a.status, p) && p.rest) {
      const int32_t* column = a.table + (int64_t)g * a.beams * a.max_pages + p.n;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        bool job = p.extra[h] && p.parent[h] >= 0;
        int src = 0, dst = 0;
        if (job) {
          src = column[(int64_t)p.parent[h] * a.max_pages], dst = column[(int64_t)p.tail[h] * a.max_pages];
          if (src < 0 || src >= a.num_pages || dst < 0 || dst >= a.num_pages) {
            report(a.status, CSA2_ERR_BAD_PAGE);
            job = false;
          }
        }
        const uint32_t who = __ballot_sync(0xffffffffu, job);
        const int at = n + __popc(who & ((1u << lane) - 1));
        if (job) from[at] = src, to[at] = dst;
        n += __popc(who);
      }
    }
    if (lane == 0) jobs = n, slots = n ? p.rest : 0;
  }
  __syncthreads();
  const int n = jobs, rest = slots;
  const int64_t page = (int64_t)a.units * 16, spage = (int64_t)a.sunits * 4;
  for (int i = blockIdx.y; i < n * 2 * a.layers; i += gridDim.y) {
    const int x = i / n, src = from[i - x * n], dst = to[i - x * n];
    const Layer& l = a.layer[x / 2];
    uint8_t* data = x & 1 ? l.v : l.k;
    copy_page<uint4, 8>(data + dst * page, data + src * page, a.units, a.run, rest * a.run / kPage);
    if (a.sunits) {
      uint8_t* scales = x & 1 ? l.vs : l.ks;
      copy_page<uint32_t, 4>(scales + dst * spage, scales + src * spage, a.sunits, a.srun, rest * a.srun / kPage);
    }
  }
}

// A group's rows of the table, kCols columns at a time.
__global__ void __launch_bounds__(kThreads) kv_table_kernel(int beams, int max_pages, int32_t* table, const int32_t* parents,
                                                            const int32_t* kv_len, int32_t* status) {
  __shared__ int32_t was[kMaxBeams][kCols];
  __shared__ int source[2][kMaxBeams];  // of the full pages, of the last
  griddep_wait();
  const int g = blockIdx.x, tid = threadIdx.x, lane = tid & 31;
  Plan p;
  if (!plan_of(g, beams, max_pages, parents, kv_len, status, p)) return;
  const int last = p.n + (p.rest ? 1 : 0);  // columns to permute
  if (tid < 32)
    for (int h = 0; h < 2; ++h)
      if (32 * h + lane < beams) {
        source[0][32 * h + lane] = p.parent[h] < 0 ? 32 * h + lane : p.parent[h];
        source[1][32 * h + lane] = p.tail[h];
      }
  int32_t* rows = table + (int64_t)g * beams * max_pages;
  for (int64_t c0 = (int64_t)blockIdx.y * kCols; c0 < last; c0 += (int64_t)gridDim.y * kCols) {
    const int cols = (int)min((int64_t)kCols, last - c0);
    __syncthreads();
    for (int x = tid; x < beams * kCols; x += kThreads)
      if (x % kCols < cols) was[x / kCols][x % kCols] = rows[(int64_t)(x / kCols) * max_pages + c0 + x % kCols];
    __syncthreads();
    for (int x = tid; x < beams * kCols; x += kThreads)
      if (x % kCols < cols)
        rows[(int64_t)(x / kCols) * max_pages + c0 + x % kCols] = was[source[c0 + x % kCols == p.n][x / kCols]][x % kCols];
  }
}

template <int kLayers>
cudaError_t tails_of(const csa2_kv_cfg& cfg, int layers, const csa2_kv_cache* caches, int groups, int beams,
                     const int32_t* parents, const int32_t* kv_len, int32_t* status, cudaStream_t stream) {
  const bool fp4 = cfg.cache_dtype == CSA2_CACHE_FP4;
  const int d = cfg.head_dim;
  ReorderArgs<kLayers> a = {};
  a.beams = beams, a.layers = layers, a.max_pages = caches[0].max_pages, a.num_pages = caches[0].num_pages;
  a.units = cfg.kv_heads * kv_block_bytes(d, fp4) / 16, a.run = fp4 ? kv_block_bytes(d, true) / 16 : kPage;
  if (fp4) a.sunits = cfg.kv_heads * kv_scale_bytes(d) / 4, a.srun = kv_scale_bytes(d) / 4;
  a.table = const_cast<int32_t*>(caches[0].block_table), a.parents = parents, a.kv_len = kv_len, a.status = status;
  for (int i = 0; i < layers; ++i)
    a.layer[i] = Layer{static_cast<uint8_t*>(caches[i].k_data), static_cast<uint8_t*>(caches[i].k_scales),
                       static_cast<uint8_t*>(caches[i].v_data), static_cast<uint8_t*>(caches[i].v_scales)};
  // twelve CTAs an SM in all: with three, groups of 63 slots to copy end late beside groups of
  // few (16 groups of 8 beams in 16 layers of 4 heads of 128 in bf16: 26.0 us; so 24.5)
  const int64_t across = std::max<int64_t>(1, 12 * (int64_t)num_sms() / groups);
  return launch_k(kv_tails_kernel<kLayers>, dim3(groups, (unsigned)std::min<int64_t>(2 * layers * beams, across)), dim3(kThreads),
                  0, stream, 0, a);
}

}  // namespace

cudaError_t launch_kv_reorder(const csa2_kv_cfg& cfg, int layers, const csa2_kv_cache* caches, int groups, int beams,
                              const int32_t* parents, const int32_t* kv_len, int32_t* status, cudaStream_t stream) {
  const cudaError_t e = layers <= 16
                            ? tails_of<16>(cfg, layers, caches, groups, beams, parents, kv_len, status, stream)
                            : tails_of<CSA2_MAX_LAYERS>(cfg, layers, caches, groups, beams, parents, kv_len, status, stream);
  if (e != cudaSuccess) return e;
  const int max_pages = caches[0].max_pages;
  return launch_k(kv_table_kernel, dim3(groups, std::min(64, (max_pages + kCols - 1) / kCols)), dim3(kThreads), 0, stream, 0, beams,
                  max_pages, const_cast<int32_t*>(caches[0].block_table), parents, kv_len, status);
}

}  // namespace csa2
