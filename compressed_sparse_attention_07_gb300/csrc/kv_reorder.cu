// The beams' cached states in the order of a selection.
//
// Full pages are shared through the block table; of the last pages, written in part,
// the groups' beams have as many as there are beams, and the pages of beams without
// children are what the second children of others need: E = D, as (children that keep
// a page) = (beams with children).  So a reordering is two kernels: kv_tails_kernel
// copies the written slots of E last pages a group, in every layer, which is bound by
// HBM (2 x the slots' bytes) or, for a few beams, by the latency of parents -> page ids ->
// slots; kv_table_kernel then permutes the table's columns in place, which the first
// still reads.  Each warp works out its group's permutation by itself, by ballots: a few
// dozen instructions, against a barrier and a pass through memory.
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
  int beams, max_pages, num_pages;
  int runs, run_step, slot_bytes, sruns, srun_step, sslot_bytes;  // data, scales of a page
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

// Runs of `bytes` bytes, `step` apart, of one page into another, by the warps of the CTA.
template <typename V>
__device__ __forceinline__ void copy_runs(uint8_t* dst, const uint8_t* src, int runs, int step, int bytes) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, n = bytes / (int)sizeof(V);
  for (int r = warp; r < runs; r += kThreads / 32) {
    const V* s = reinterpret_cast<const V*>(src + (int64_t)r * step);
    V* d = reinterpret_cast<V*>(dst + (int64_t)r * step);
#pragma unroll 4
    for (int i = lane; i < n; i += 32) d[i] = s[i];
  }
}

// One beam's last page in one layer: keys (blockIdx.z even) or values.
template <int kLayers>
__global__ void __launch_bounds__(kThreads) kv_tails_kernel(const __grid_constant__ ReorderArgs<kLayers> a) {
  griddep_wait();  // every input may be the previous kernel's output
  const int g = blockIdx.x / a.beams, i = blockIdx.x % a.beams;
  Plan p;
  if (!plan_of(g, a.beams, a.max_pages, a.parents, a.kv_len, a.status, p) || p.rest == 0) return;
  const int h = i >> 5, from = i & 31;
  const bool extra = __shfl_sync(0xffffffffu, h ? p.extra[1] : p.extra[0], from);
  const int parent = __shfl_sync(0xffffffffu, h ? p.parent[1] : p.parent[0], from);
  const int tail = __shfl_sync(0xffffffffu, h ? p.tail[1] : p.tail[0], from);
  if (!extra || parent < 0) return;
  const int64_t row = (int64_t)g * a.beams;
  const int src = a.table[(row + parent) * a.max_pages + p.n], dst = a.table[(row + tail) * a.max_pages + p.n];
  if (src < 0 || src >= a.num_pages || dst < 0 || dst >= a.num_pages) {
    if (threadIdx.x == 0) report(a.status, CSA2_ERR_BAD_PAGE);
    return;
  }
  const Layer& l = a.layer[blockIdx.y];
  uint8_t* data = blockIdx.z ? l.v : l.k;
  const int64_t page = (int64_t)a.runs * a.run_step;
  copy_runs<uint4>(data + dst * page, data + src * page, a.runs, a.run_step, p.rest * a.slot_bytes);
  if (a.sruns) {
    uint8_t* scales = blockIdx.z ? l.vs : l.ks;
    const int64_t spage = (int64_t)a.sruns * a.srun_step;
    copy_runs<uint32_t>(scales + dst * spage, scales + src * spage, a.sruns, a.srun_step, p.rest * a.sslot_bytes);
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
  a.beams = beams, a.max_pages = caches[0].max_pages, a.num_pages = caches[0].num_pages;
  a.runs = fp4 ? cfg.kv_heads : cfg.kv_heads * (d / 8);
  a.run_step = fp4 ? kv_block_bytes(d, true) : kPage * 16, a.slot_bytes = fp4 ? d / 2 : 16;
  if (fp4) a.sruns = cfg.kv_heads, a.srun_step = kv_scale_bytes(d), a.sslot_bytes = d / 16;
  a.table = const_cast<int32_t*>(caches[0].block_table), a.parents = parents, a.kv_len = kv_len, a.status = status;
  for (int i = 0; i < layers; ++i)
    a.layer[i] = Layer{static_cast<uint8_t*>(caches[i].k_data), static_cast<uint8_t*>(caches[i].k_scales),
                       static_cast<uint8_t*>(caches[i].v_data), static_cast<uint8_t*>(caches[i].v_scales)};
  return launch_k(kv_tails_kernel<kLayers>, dim3(groups * beams, layers, 2), dim3(kThreads), 0, stream, 0, a);
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
