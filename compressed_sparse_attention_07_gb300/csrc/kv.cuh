// Shared by the paged key / value operators (kv_append, kv_attend,
// kv_cross_attend): the cache view, a ragged batch's sequence bounds and the
// range of keys that a tile of query rows sees.
#pragma once

#include <atomic>

#include "internal.h"

namespace csa2 {

struct KvView {
  uint8_t* k;
  uint8_t* ks;
  uint8_t* v;
  uint8_t* vs;
  const int32_t* table;
  int32_t max_pages;
  int32_t num_pages;
};

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t mul2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}
// Two E4M3 bytes -> f16 pair (exact).
__device__ __forceinline__ uint32_t scales2(uint32_t pair) {
  uint32_t r;
  const uint16_t p = (uint16_t)pair;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(p));
  return r;
}
// Eight E2M1 codes -> four f16 pairs.
__device__ __forceinline__ void codes8(uint32_t w, uint32_t (&r)[4]) {
  asm("{\n .reg .b8 b0, b1, b2, b3;\n mov.b32 {b0, b1, b2, b3}, %4;\n"
      " cvt.rn.f16x2.e2m1x2 %0, b0;\n cvt.rn.f16x2.e2m1x2 %1, b1;\n"
      " cvt.rn.f16x2.e2m1x2 %2, b2;\n cvt.rn.f16x2.e2m1x2 %3, b3;\n}\n"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
      : "r"(w));
}
// E4M3 code nearest to y >= 0, saturating.
__device__ __forceinline__ uint32_t e4m3_code(float y) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(0.0f), "f"(y));
  return r & 0xFFu;
}
// Codes of x / s (0 < s), ties to the even code, saturating: eight nibbles, channel
// 0 lowest.  |x| may pass 6 s, up to 9 s at the smallest scales, whose steps are
// wide, and without bound at the largest: the conversion saturates.  The quotient is
// rounded correctly from the reciprocal by one step with the remainder
// (Markstein), so that a value half way between two codes is seen as such; where
// the remainder underflows, the code is 0 either way.  The sign of a value that
// rounds to zero is dropped.
__device__ __forceinline__ uint32_t e2m1x8(const float (&x)[8], float s) {
  const float inv = __frcp_rn(s);
  float y[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float q = __fmul_rn(x[i], inv);
    y[i] = __fmaf_rn(__fmaf_rn(-q, s, x[i]), inv, q);
  }
  uint32_t w;
  asm("{\n .reg .b8 b0, b1, b2, b3;\n"
      " cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n"
      " cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n"
      " mov.b32 %0, {b0, b1, b2, b3};\n}\n"
      : "=r"(w)
      : "f"(y[0]), "f"(y[1]), "f"(y[2]), "f"(y[3]), "f"(y[4]), "f"(y[5]), "f"(y[6]), "f"(y[7]));
  const uint32_t m = w & 0x77777777u;
  const uint32_t nz = (m | (m >> 1) | (m >> 2)) & 0x11111111u;
  return m | (w & (nz << 3));
}
// Pairs of fp32 for the packed arithmetic.
__device__ __forceinline__ uint64_t pack2(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void unpack2(uint64_t x, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(x));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
// Bytes of one (page, kv head) block of keys or of values.
__host__ __device__ constexpr int kv_block_bytes(int dim, bool fp4) { return fp4 ? kPage * dim / 2 : kPage * dim * 2; }
__host__ __device__ constexpr int kv_scale_bytes(int dim) { return kPage * dim / 16; }

// n / d for 0 <= n < 2^31 without a division (several hundred cycles at a CTA's
// start): with s = ceil(log2 d) and m = floor(2^(31 + s) / d) + 1 the error of
// n m / 2^(31 + s) is below n / 2^(31 + s) < 1 / d.
struct Divisor {
  uint32_t mul, shift;
};
inline Divisor divisor(int d) {
  uint32_t s = 0;
  while ((1ll << s) < d) ++s;
  return {(uint32_t)((1ull << (31 + s)) / d + 1), 31 + s};
}
__device__ __forceinline__ int quotient(int n, const Divisor& d) {
  return (int)(((uint64_t)(uint32_t)n * d.mul) >> d.shift);
}

// Arguments of an attention call.
struct KvAtt {
  int B, T, n_heads, kv_heads, group, window, causal, max_q;
  Divisor by_group, by_heads, by_parts, by_pages;  // group, kv_heads, n_parts, part_pages
  int max_kv;
  const uint16_t* q;
  int64_t q_stride;
  const int32_t* cu;
  KvView c;
  const int32_t* kv_len;
  float scale;  // softmax scale
  uint16_t* out;
  int64_t out_stride;
  float* lse;
  // division of the keys: parts of `part_pages` pages; with n_parts > 1 the
  // partial outputs go to part_o [n_parts][part_step][dim] and their log2-sum-exp2 to
  // part_l [n_parts][part_step] (kv_part_row)
  int n_parts, part_pages;
  int64_t part_step;  // T * n_heads, or (tile kernel) the divided tiles times part_rows
  int part_rows;      // most rows of a tile; 0: by row and head
  int cluster;  // the parts of a head join in a cluster instead
  // (tile kernel) most row tiles, of all kv heads; how many, in the order of their
  // CTAs, are not divided
  int tiles, whole;
  float* part_o;
  float* part_l;
  // FP4 pages decoded for this call: page p of sequence b and a kv head as f16 in a
  // BF16 page's order, at block (b * plain_pages + p) * kv_heads + kv head
  uint8_t* plain_k;  // null: none
  uint8_t* plain_v;
  int plain_pages;
  int32_t* status;
};

__device__ __forceinline__ int group_of(const KvAtt& a, int n) { return quotient(n, a.by_group); }

// Where row r of the id-th row tile (its first is tile0; row and head number `at` of the
// batch) has its partial outputs, in each part.
__device__ __forceinline__ int64_t kv_part_row(const KvAtt& a, int id, int r, int tile0, int64_t at) {
  return a.part_rows ? (int64_t)(id - a.whole) * a.part_rows + r - tile0 : at;
}

// Rows and keys of sequence b; false (status set) when they are out of bounds.
__device__ __forceinline__ bool kv_sequence(const KvAtt& a, int b, int& row0, int& rows, int& keys) {
  const int lo = __ldg(a.cu + b), hi = __ldg(a.cu + b + 1), n = __ldg(a.kv_len + b);
  if (lo < 0 || hi < lo || hi > a.T || hi - lo > a.max_q || n < 0 || n > a.max_kv) {
    report(a.status, CSA2_ERR_BAD_INDEX);
    return false;
  }
  row0 = lo;
  rows = hi - lo;
  keys = n;
  return true;
}

// The id-th row tile of the call: sequences in order, their kv heads, of each the
// tiles from the last (the longest) on.  Sequences have what tiles their rows fill, so
// that a batch of one prompt and many single tokens is not a grid of empty CTAs (4096
// tokens and 63 single ones, 64 over 8 heads of 128: 792 us with the longest's tiles
// for each, 376 so; four prompts of 700 .. 1500: 132 and 132).  The whole warp; false
// behind the last tile; sequences out of bounds have none (status set).
__device__ __forceinline__ bool kv_tile(const KvAtt& a, int tile_rows, int id, int& b, int& kh, int& tile) {
  const int lane = threadIdx.x & 31, want = quotient(id, a.by_heads);
  int before = 0;  // tiles of a kv head so far
  for (int b0 = 0; b0 < a.B; b0 += 128) {  // four sequences a lane
    int n[4], lo = 0;
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      const int s = b0 + 4 * lane + x;
      n[x] = 0;
      if (s < a.B) {
        if (x == 0) lo = __ldg(a.cu + s);
        const int hi = __ldg(a.cu + s + 1), keys = __ldg(a.kv_len + s);
        if (lo < 0 || hi < lo || hi > a.T || hi - lo > a.max_q || keys < 0 || keys > a.max_kv)
          report(a.status, CSA2_ERR_BAD_INDEX);
        else n[x] = ((hi - lo) * a.group + tile_rows - 1) / tile_rows;
        lo = hi;
      }
    }
    const int own = n[0] + n[1] + n[2] + n[3];
    int upto = own;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, upto, d);
      if (lane >= d) upto += v;
    }
    upto += before;
    const uint32_t past = __ballot_sync(0xffffffffu, upto > want);
    if (past) {
      int first = upto - own, s = b0 + 4 * lane, count = n[0];
#pragma unroll
      for (int x = 1; x < 4; ++x)
        if (want >= first + count) first += count, count = n[x], ++s;
      // from the first lane past it; a reduction, so that the compiler knows the
      // numbers as the warp's, not the lanes'
      const bool own_it = lane == __ffs(past) - 1;
      b = __reduce_max_sync(0xffffffffu, own_it ? s : 0), first = __reduce_max_sync(0xffffffffu, own_it ? first : 0);
      count = __reduce_max_sync(0xffffffffu, own_it ? count : 0);
      const int at = id - first * a.kv_heads;
      if ((unsigned)at >= (unsigned)(count * a.kv_heads)) return false;  // rows counted twice (bad cu) past 2^31
      kh = (int)__fdividef((float)at, (float)count);  // at / count, off by one at most
      int rest = at - kh * count;
      if (rest < 0) --kh, rest += count;
      if (rest >= count) ++kh, rest -= count;
      tile = count - 1 - rest;
      return true;
    }
    before = __shfl_sync(0xffffffffu, upto, 31);
  }
  return false;
}

// Position up to which (exclusive) row `i` of `rows` sees keys, and from which.
__device__ __forceinline__ int kv_hi(const KvAtt& a, int i, int rows, int keys) {
  if (!a.causal) return keys;
  const int h = keys - rows + i + 1;
  return h < 0 ? 0 : h;
}
__device__ __forceinline__ int kv_lo(const KvAtt& a, int i, int rows, int keys) {
  if (!a.causal || a.window == 0) return 0;
  const int l = keys - rows + i + 1 - a.window;
  return l < 0 ? 0 : l;
}

// Pages [p0, p1) that rows i0 .. i1 (inclusive) see.
__device__ __forceinline__ void kv_pages(const KvAtt& a, int i0, int i1, int rows, int keys, int& p0, int& p1) {
  const int lo = kv_lo(a, i0, rows, keys), hi = kv_hi(a, i1, rows, keys);
  p0 = lo / kPage;
  p1 = hi > lo ? (hi + kPage - 1) / kPage : p0;
}

// Parts of pages [p0, p1).
__device__ __forceinline__ int kv_parts(const KvAtt& a, int p0, int p1) {
  return quotient(p1 - p0 + a.part_pages - 1, a.by_pages);
}

// csa2_attend reads queries and window rows before it waits for the kernel ahead of it,
// so a kernel that writes a call's outputs lets its successor start only when its CTAs
// have ended; started early, csa2_attend read what stood there before.  It costs a call
// the overlap with the next one's start: single-sequence decode 7.33 -> 7.74 us in a graph
// of such calls, drafts 147 -> 149 us; appends take 2.46 -> 2.36 us.  What is sound is
// kv_join_kernel's early start, as that kernel writes the outputs and waits before.
__device__ __forceinline__ bool kv_joined(const KvAtt& a) { return a.n_parts > 1 && !a.cluster; }

// Rotary positions of several axes: pos [T][n] (null: the running position), of [pairs].
struct KvAxes {
  const int32_t* pos;
  int n;
  const uint8_t* of;
};
cudaError_t launch_kv_append(const csa2_kv_cfg& cfg, int B, int T, const uint16_t* q, int64_t q_stride,
                             const uint16_t* k, int64_t k_stride, const uint16_t* v, int64_t v_stride,
                             const int32_t* cu, const int64_t* pos0, const KvAxes& axes, const float* rope,
                             int64_t rope_rows, const KvView& c, uint16_t* q_out, int64_t q_out_stride, uint16_t* k_out,
                             uint16_t* v_out, int32_t* status, cudaStream_t stream);
// The beams' tables and last pages (kv_reorder.cu).
cudaError_t launch_kv_reorder(const csa2_kv_cfg& cfg, int layers, const csa2_kv_cache* caches, int groups, int beams,
                              const int32_t* parents, const int32_t* kv_len, int32_t* status, cudaStream_t stream);

// How a call divides the keys, from sizes alone, with no more than `room` bytes of
// partial outputs.
struct KvPlan {
  int n_parts, part_pages;
  bool cluster;  // the parts join in a cluster, without workspace
  int64_t tiles, whole;  // (tile kernel) row tiles of all kv heads, those that are not divided
  int64_t ctas;          // (tile kernel) of it or of the joining kernel, whichever has more
  int64_t part_step;     // as in KvAtt
  int part_rows;
  size_t bytes;  // of the partial outputs
};
KvPlan kv_plan(const csa2_kv_cfg& cfg, int B, int T, int max_q, int max_kv, bool cross, size_t room);

// Let `kern` use `bytes` of dynamic shared memory: set once on each device, as setting it
// takes the host a microsecond (one token on 4095: 9.4 us a call so, 10.3 set at every
// call).  Threads may make their first calls at once: `done` is atomic, and setting it
// twice does no harm.
template <typename K>
cudaError_t allow_smem(K kern, int bytes, std::atomic<bool> (&done)[64]) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess || (dev < 64 && done[dev].load(std::memory_order_acquire))) return e;
  e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess && dev < 64) done[dev].store(true, std::memory_order_release);
  return e;
}

// The plan of the tile kernel, which takes more rows of a kv head than kMostRows;
// its launch, and the rows of its CTA.
constexpr int kMostRows = 32;
KvPlan kv_tiles_plan(const csa2_kv_cfg& cfg, int B, int T, int max_q, int64_t max_kv, bool cross, size_t room);
cudaError_t launch_kv_tiles(const csa2_kv_cfg& cfg, int B, const KvAtt& a, cudaStream_t stream);
// Bytes of the keys decoded for a call, or 0 where they are decoded in passing.
size_t kv_plain_bytes(const csa2_kv_cfg& cfg, int B, int T, int max_q, int64_t max_kv, bool cross);
int kv_tiles_rows();

cudaError_t launch_kv_attend(const csa2_kv_cfg& cfg, int B, KvAtt& a, cudaStream_t stream);

}  // namespace csa2
