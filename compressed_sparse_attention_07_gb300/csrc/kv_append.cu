// Keys and values of new tokens into the paged cache, queries beside them.
//
// A token's rows (n_heads queries, kv_heads keys, kv_heads values) are read
// once as bf16, 8 channels a thread; queries and keys are rotated,
//   (a, b) -> (a cos - b sin, a sin + b cos),
// with (cos, sin) from the caller's table, products and sums each rounded to
// fp32 (so that a code near a rounding border does not depend on how the
// compiler contracts them); keys and values are encoded (FP4: scale = E4M3
// nearest to amax / 6 of 16 channels, i.e. of two neighbouring threads, code =
// E2M1 nearest to x / scale) and stored in the token's page.
// The call moves 2 B a channel in and 2 B (queries) or 0.5625 B (FP4) out and
// computes a few operations on each: bound by HBM for long prompts, by latency
// for a decode step, which is why a token's rows are spread over CTAs there.
#include "kv.cuh"

namespace csa2 {
namespace {

constexpr int kThreads = 256, kMostPasses = 4;

struct AppendArgs {
  int B, T, n_q, n_kv, rope_dims, half;
  const uint16_t *q, *k, *v;
  int64_t q_stride, k_stride, v_stride;
  const int32_t* cu;
  const int64_t* pos0;
  const float* rope;
  int64_t rope_rows;
  KvView c;
  uint16_t* q_out;
  int64_t q_out_stride;
  uint16_t *k_out, *v_out;
  int32_t* status;
};

__device__ __forceinline__ void unpack8(uint4 w, float (&x)[8]) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(u[i] << 16);
    x[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
  return make_uint4(bf16x2(x[0], x[1]), bf16x2(x[2], x[3]), bf16x2(x[4], x[5]), bf16x2(x[6], x[7]));
}

// E4M3 code nearest to y >= 0, saturating.
__device__ __forceinline__ uint32_t e4m3_code(float y) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(0.0f), "f"(y));
  return r & 0xFFu;
}
// Codes of x / s, ties to the even code, saturating: eight nibbles, channel 0
// lowest.  The sign of a value that rounds to zero is dropped.
__device__ __forceinline__ uint32_t e2m1x8(const float (&x)[8], float s) {
  float y[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) y[i] = __fdiv_rn(x[i], s);
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

template <int kDim_, bool kFp4, int kPasses>
__global__ void __launch_bounds__(kThreads) kv_append_kernel(AppendArgs a) {
  constexpr int kLanes = kDim_ / 8;              // threads of a row
  constexpr int kRows = kThreads / kLanes;       // rows of a pass
  griddep_wait();  // every input may be the previous kernel's output
  griddep_launch();
  const int n = blockIdx.x, tid = threadIdx.x;
  const int col = tid % kLanes, c0 = 8 * col;  // this thread's channels in every row
  const int n_rows = a.n_q + 2 * a.n_kv;
  const int first = (blockIdx.y * kPasses) * kRows + tid / kLanes;
  // the rows first: their way from HBM covers the look-ups below
  uint4 raw[kPasses];
#pragma unroll
  for (int p = 0; p < kPasses; ++p) {
    const int r = first + p * kRows;
    raw[p] = make_uint4(0, 0, 0, 0);
    if (r < n_rows) {
      const uint16_t* src = r < a.n_q            ? a.q + (int64_t)n * a.q_stride + r * kDim_
                            : r < a.n_q + a.n_kv ? a.k + (int64_t)n * a.k_stride + (r - a.n_q) * kDim_
                                                 : a.v + (int64_t)n * a.v_stride + (r - a.n_q - a.n_kv) * kDim_;
      raw[p] = *reinterpret_cast<const uint4*>(src + c0);
    }
  }
  // the token's sequence: how many sequences end at or before it
  int b = 0;
  for (int i0 = 0; i0 < a.B; i0 += kThreads) {
    const int i = i0 + tid;
    b += __syncthreads_count(i < a.B && __ldg(a.cu + i + 1) <= n);
  }
  if (b >= a.B) return;  // behind the last sequence
  const int lo = __ldg(a.cu + b), hi = __ldg(a.cu + b + 1);
  if (n < lo && b == 0 && lo <= a.T) return;  // ahead of the first
  const int64_t pos = __ldg(a.pos0 + b) + (n - lo);
  if (lo < 0 || n < lo || n >= hi || hi > a.T || pos < 0 || pos >= (int64_t)a.c.max_pages * kPage ||
      (a.rope_dims && pos >= a.rope_rows)) {
    if (tid == 0) report(a.status, CSA2_ERR_BAD_INDEX);
    return;
  }
  const int32_t page = __ldg(a.c.table + (int64_t)b * a.c.max_pages + pos / kPage);
  const int slot = (int)(pos % kPage);
  const bool page_ok = page >= 0 && page < a.c.num_pages;
  if (!page_ok && tid == 0) report(a.status, CSA2_ERR_BAD_PAGE);

  const int pairs = a.rope_dims / 2;
  const bool turned = c0 < a.rope_dims;
  const bool second = a.half && c0 >= pairs;  // holds the b's of its pairs
  float cs[8], sn[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) cs[i] = 1.0f, sn[i] = 0.0f;
  if (turned) {
    const float4* t = reinterpret_cast<const float4*>(a.rope + pos * a.rope_dims);
    if (a.half) {
      const int p = second ? c0 - pairs : c0;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float4 f = __ldg(t + p / 2 + i);
        cs[2 * i] = f.x, sn[2 * i] = f.y, cs[2 * i + 1] = f.z, sn[2 * i + 1] = f.w;
      }
    } else {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float4 f = __ldg(t + c0 / 4 + i);
        cs[2 * i] = f.x, sn[2 * i] = f.y, cs[2 * i + 1] = f.z, sn[2 * i + 1] = f.w;
      }
    }
  }
  const int mate = second ? (tid & 31) - pairs / 8 : (tid & 31) + pairs / 8;

#pragma unroll
  for (int p = 0; p < kPasses; ++p) {
    const int r = first + p * kRows;
    const bool live = r < n_rows;
    const bool is_q = r < a.n_q, is_v = r >= a.n_q + a.n_kv;
    const int h = is_q ? r : is_v ? r - a.n_q - a.n_kv : r - a.n_q;
    float x[8];
    unpack8(raw[p], x);
    if (a.half) {  // uniform: the pair's other member is in another thread of the row
      float y[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] = __shfl_sync(0xffffffffu, x[i], mate & 31);
      if (turned && !is_v) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          x[i] = second ? __fadd_rn(__fmul_rn(y[i], sn[i]), __fmul_rn(x[i], cs[i]))
                        : __fsub_rn(__fmul_rn(x[i], cs[i]), __fmul_rn(y[i], sn[i]));
      }
    } else if (turned && !is_v) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float u = x[2 * i], w = x[2 * i + 1];
        x[2 * i] = __fsub_rn(__fmul_rn(u, cs[i]), __fmul_rn(w, sn[i]));
        x[2 * i + 1] = __fadd_rn(__fmul_rn(u, sn[i]), __fmul_rn(w, cs[i]));
      }
    }
    if (!is_q) {
      constexpr float kMost = 3.3895313892515355e38f;  // largest bf16
      bool bad = false;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if (!(fabsf(x[i]) <= kMost)) {
          bad = true;
          x[i] = x[i] != x[i] ? 0.0f : copysignf(kMost, x[i]);
        }
      }
      if (bad && live) report(a.status, CSA2_ERR_RANGE);
    }
    float amax = 0.0f;
    if (kFp4) {
#pragma unroll
      for (int i = 0; i < 8; ++i) amax = fmaxf(amax, fabsf(x[i]));
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
    }
    if (!live) continue;
    if (is_q) {
      *reinterpret_cast<uint4*>(a.q_out + (int64_t)n * a.q_out_stride + h * kDim_ + c0) = pack8(x);
      continue;
    }
    uint16_t* plain = is_v ? a.v_out : a.k_out;
    const int64_t block = (int64_t)page * a.n_kv + h;
    if (kFp4) {
      const uint32_t sc = e4m3_code(__fdiv_rn(amax, 6.0f));
      const float s = e4m3_to_float(sc);
      const uint32_t w = sc ? e2m1x8(x, s) : 0u;
      if (page_ok) {
        uint8_t* data = (is_v ? a.c.v : a.c.k) + block * kv_block_bytes(kDim_, true);
        *reinterpret_cast<uint32_t*>(data + slot * (kDim_ / 2) + c0 / 2) = w;
        if ((col & 1) == 0)
          ((is_v ? a.c.vs : a.c.ks) + block * kv_scale_bytes(kDim_))[slot * (kDim_ / 16) + col / 2] = (uint8_t)sc;
      }
      if (plain) {
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = e2m1_to_float((w >> (4 * i)) & 15u) * s;
      }
    } else if (page_ok) {
      uint8_t* data = (is_v ? a.c.v : a.c.k) + block * kv_block_bytes(kDim_, false);
      *reinterpret_cast<uint4*>(data + (col * kPage + slot) * 16) = pack8(x);
    }
    if (plain) *reinterpret_cast<uint4*>(plain + ((int64_t)n * a.n_kv + h) * kDim_ + c0) = pack8(x);
  }
}

}  // namespace

cudaError_t launch_kv_append(const csa2_kv_cfg& cfg, int B, int T, const uint16_t* q, int64_t q_stride,
                             const uint16_t* k, int64_t k_stride, const uint16_t* v, int64_t v_stride,
                             const int32_t* cu, const int64_t* pos0, const float* rope, int64_t rope_rows,
                             const KvView& c, uint16_t* q_out, int64_t q_out_stride, uint16_t* k_out, uint16_t* v_out,
                             int32_t* status, cudaStream_t stream) {
  AppendArgs a{B, T, q ? cfg.n_heads : 0, cfg.kv_heads, cfg.rope_dims, cfg.rope_style == CSA2_ROPE_HALF ? 1 : 0,
               q, k, v, q_stride, k_stride, v_stride, cu, pos0, rope, rope_rows, c, q_out, q_out_stride, k_out, v_out,
               status};
  const int rows = kThreads / (cfg.head_dim / 8);
  const int passes = (a.n_q + 2 * a.n_kv + rows - 1) / rows;
  // a CTA for each of a token's passes while these do not fill the GPU, then a
  // CTA for four
  const bool few = (int64_t)T * passes <= 8 * num_sms();
  const dim3 grid(T, few ? passes : (passes + kMostPasses - 1) / kMostPasses), block(kThreads);
  const bool fp4 = cfg.cache_dtype == CSA2_CACHE_FP4;
#define CSA2_APPEND(D, F)                                                                      \
  (few ? launch_k(kv_append_kernel<D, F, 1>, grid, block, 0, stream, 0, a)                     \
       : launch_k(kv_append_kernel<D, F, kMostPasses>, grid, block, 0, stream, 0, a))
  if (cfg.head_dim == 128) return fp4 ? CSA2_APPEND(128, true) : CSA2_APPEND(128, false);
  return fp4 ? CSA2_APPEND(64, true) : CSA2_APPEND(64, false);
#undef CSA2_APPEND
}

}  // namespace csa2
