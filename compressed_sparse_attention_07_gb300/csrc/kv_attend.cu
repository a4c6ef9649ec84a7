// Attention over the paged key / value cache: out = softmax(scale q K^T) V.
//
// One warp per query row and head: the keys it sees are taken 32 at a time,
// one a lane for the scores, then 32 values for the output's channels, with
// the running maximum and sum of the softmax in fp32.
#include "kv.cuh"

namespace csa2 {
namespace {

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

template <int D, bool kFp4>
__device__ float kv_value(const uint8_t* data, const uint8_t* scales, int slot, int c) {
  if (kFp4) {
    const uint32_t w = data[slot * (D / 2) + c / 2];
    return e2m1_to_float((c & 1) ? w >> 4 : w & 15u) * e4m3_to_float(scales[slot * (D / 16) + c / 16]);
  }
  return bf16_bits_to_float(reinterpret_cast<const uint16_t*>(data)[((c / 8) * kPage + slot) * 8 + c % 8]);
}

template <int D, bool kFp4>
__global__ void __launch_bounds__(256) kv_plain_kernel(KvAtt a) {
  griddep_wait();
  griddep_launch();
  const int b = blockIdx.y, warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  int row0, rows, keys;
  if (!kv_sequence(a, b, row0, rows, keys)) return;
  const int64_t r = (int64_t)blockIdx.x * 8 + warp;
  if (r >= (int64_t)rows * a.n_heads) return;
  const int i = (int)(r / a.n_heads), h = (int)(r % a.n_heads), kh = h / a.group;
  const uint16_t* q = a.q + (int64_t)(row0 + i) * a.q_stride + h * D;
  const int lo = kv_lo(a, i, rows, keys), hi = kv_hi(a, i, rows, keys);
  float m = -INFINITY, l = 0.0f, o[D / 32] = {};
  for (int j0 = lo / 32 * 32; j0 < hi; j0 += 32) {
    const int32_t page = __ldg(a.c.table + (int64_t)b * a.c.max_pages + j0 / kPage);
    if (page < 0 || page >= a.c.num_pages) {
      report(a.status, CSA2_ERR_BAD_PAGE);
      continue;
    }
    const int64_t block = (int64_t)page * a.kv_heads + kh;
    const uint8_t* kd = a.c.k + block * kv_block_bytes(D, kFp4);
    const uint8_t* vd = a.c.v + block * kv_block_bytes(D, kFp4);
    const uint8_t* ks = kFp4 ? a.c.ks + block * kv_scale_bytes(D) : nullptr;
    const uint8_t* vs = kFp4 ? a.c.vs + block * kv_scale_bytes(D) : nullptr;
    const int j = j0 + lane;
    float s = -INFINITY;
    if (j >= lo && j < hi) {
      s = 0.0f;
      for (int c = 0; c < D; ++c) s = fmaf(bf16_bits_to_float(__ldg(q + c)), kv_value<D, kFp4>(kd, ks, j % kPage, c), s);
      s *= a.scale * kLog2e;
    }
    float top = s;
#pragma unroll
    for (int d = 16; d; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
    const float m2 = fmaxf(m, top);
    const float f = exp2f(m - m2);
    const float p = s == -INFINITY ? 0.0f : exp2f(s - m2);
    m = m2;
    l = l * f + p;
#pragma unroll
    for (int x = 0; x < D / 32; ++x) o[x] *= f;
    for (int t = 0; t < 32; ++t) {
      const float pt = __shfl_sync(0xffffffffu, p, t);
      if (j0 + t < lo || j0 + t >= hi) continue;
#pragma unroll
      for (int x = 0; x < D / 32; ++x) o[x] = fmaf(pt, kv_value<D, kFp4>(vd, vs, (j0 + t) % kPage, x * 32 + lane), o[x]);
    }
  }
#pragma unroll
  for (int d = 16; d; d >>= 1) l += __shfl_xor_sync(0xffffffffu, l, d);
  const float inv = l > 0.0f ? 1.0f / l : 0.0f;
  uint16_t* out = a.out + (int64_t)(row0 + i) * a.out_stride + h * D;
#pragma unroll
  for (int x = 0; x < D / 32; ++x) out[x * 32 + lane] = __bfloat16_as_ushort(__float2bfloat16_rn(o[x] * inv));
  if (a.lse && lane == 0) a.lse[(int64_t)(row0 + i) * a.n_heads + h] = l > 0.0f ? (m + log2f(l)) * kLn2 : -INFINITY;
}

}  // namespace

void kv_plan(const csa2_kv_cfg&, int, int, int max_kv, bool, int, int* n_parts, int* part_pages) {
  *n_parts = 1;
  *part_pages = (max_kv + kPage - 1) / kPage;
}

cudaError_t launch_kv_attend(const csa2_kv_cfg& cfg, int B, KvAtt& a, cudaStream_t stream) {
  const dim3 grid((unsigned)(((int64_t)a.max_q * a.n_heads + 7) / 8), B);
  const bool fp4 = cfg.cache_dtype == CSA2_CACHE_FP4;
  if (cfg.head_dim == 128)
    return fp4 ? launch_k(kv_plain_kernel<128, true>, grid, dim3(256), 0, stream, 0, a)
               : launch_k(kv_plain_kernel<128, false>, grid, dim3(256), 0, stream, 0, a);
  return fp4 ? launch_k(kv_plain_kernel<64, true>, grid, dim3(256), 0, stream, 0, a)
             : launch_k(kv_plain_kernel<64, false>, grid, dim3(256), 0, stream, 0, a);
}

}  // namespace csa2
