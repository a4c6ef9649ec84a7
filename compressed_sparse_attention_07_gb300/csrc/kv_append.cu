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
// for a decode step.  So there are two kernels:
//  - kv_append_few_kernel: a CTA for 32 or 16 rows of a token (16 a pass), which
//    reads its rows while it looks up the token's sequence, page and angles:
//    2.3 us for 8 tokens of 64 + 2 x 8 heads of 128 in FP4;
//  - kv_append_stream_kernel, from kFewItems pieces an SM on: two CTAs an SM
//    take pieces of up to 24 KB (a token, four small ones or a part of a large
//    one) in turn; one warp looks up 32 tokens at a time and keeps four pieces on
//    their way by bulk copies, eight warps rotate, encode and store.  8 prompts
//    of 37 .. 2021 tokens, 64 + 2 x 8 heads of 128, in FP4 take 66 us, 5.3 TB/s
//    (107 us with a CTA for each piece, which waits for its look-ups).
#include <algorithm>

#include "kv.cuh"
#include "tc.cuh"

namespace csa2 {
namespace {

constexpr int kThreads = 256;
// Pieces an SM from which the stream kernel is the faster: 1000 tokens of 64 + 2 x 8
// heads of 128 in FP4 take 13.0 us in the first kernel and 13.7 us in it, 1300 take
// 16.6 and 15.8 us; 1000 of 32 + 2 x 4 heads of 64 in bf16 5.4 and 5.8 us, 2000 9.0
// and 8.5 (GPU time in graphs of calls on rows of their own, as below).
constexpr int kFewItems = 8;

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

__device__ __forceinline__ void widen(const uint32_t (&u)[4], float (&x)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(u[i] << 16);
    x[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
  }
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

// What a thread keeps for its eight channels of every row of a token: the
// cosines, and the sines with the sign they have in that channel.
struct Turn {
  float c[8], s[8];
  // table: the token's row of angles (global or shared memory)
  __device__ __forceinline__ void load(const float4* table, int c0, int pairs, bool half) {
    if (half) {  // eight pairs, of which this thread holds the a's or the b's
      const bool second = c0 >= pairs;
      const float4* t = table + (second ? c0 - pairs : c0) / 2;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float4 f = t[i];
        c[2 * i] = f.x, c[2 * i + 1] = f.z;
        s[2 * i] = second ? f.y : -f.y, s[2 * i + 1] = second ? f.w : -f.w;
      }
    } else {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float4 f = table[c0 / 4 + i];
        c[4 * i] = c[4 * i + 1] = f.x, c[4 * i + 2] = c[4 * i + 3] = f.z;
        s[4 * i] = -f.y, s[4 * i + 1] = f.y, s[4 * i + 2] = -f.w, s[4 * i + 3] = f.w;
      }
    }
  }
};

struct Place {
  int n;         // token
  int32_t page;  // -1: not there
  int slot;
};

// Eight channels w (column col) of row r of a token's queries, keys and values
// -> rotated, encoded and stored.  The whole warp calls it; `mate`: the lane
// with the other members of this thread's pairs (half style), `turned`: whether
// its channels are rotated at all.
template <int kDim_, bool kFp4>
__device__ __forceinline__ void put_row(const AppendArgs& a, const Place& at, int r, bool live, int col, const Turn& turn,
                                        bool turned, int mate, uint4 w) {
  const int c0 = 8 * col;
  const bool is_q = r < a.n_q, is_v = r >= a.n_q + a.n_kv;
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
  float v[8];
  widen(u, v);
  if (a.rope_dims) {
    // v c + y s, y the other member: each product and the sum rounded by itself
    // (the packed fp32 operations do not keep the products apart)
    uint32_t o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = a.half ? __shfl_sync(0xffffffffu, u[i], mate) : __byte_perm(u[i], 0, 0x1032);
    if (turned && !is_v) {
      float y[8];
      widen(o, y);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = __fadd_rn(__fmul_rn(v[i], turn.c[i]), __fmul_rn(y[i], turn.s[i]));
    }
  }
  if (is_q && live)
    *reinterpret_cast<uint4*>(a.q_out + (int64_t)at.n * a.q_out_stride + r * kDim_ + c0) =
        make_uint4(bf16x2(v[0], v[1]), bf16x2(v[2], v[3]), bf16x2(v[4], v[5]), bf16x2(v[6], v[7]));
  const bool mine = live && !is_q;
  if (!__any_sync(0xffffffffu, mine)) return;
  float amax = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) amax = fmaxf(amax, fabsf(v[i]));
  constexpr float kMost = 3.3895313892515355e38f;  // largest bf16
  float sum = 0.0f;  // NaN if any is
#pragma unroll
  for (int i = 0; i < 8; ++i) sum = fmaf(v[i], 0.0f, sum);
  if (mine && (!(amax <= kMost) || sum != 0.0f)) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (!(fabsf(v[i]) <= kMost)) v[i] = v[i] != v[i] ? 0.0f : copysignf(kMost, v[i]);
    amax = fminf(amax, kMost);
    report(a.status, CSA2_ERR_RANGE);
  }
  uint16_t* plain = is_v ? a.v_out : a.k_out;
  const int h = is_v ? r - a.n_q - a.n_kv : r - a.n_q;
  const int64_t block = (int64_t)at.page * a.n_kv + h;
  uint4 stored;
  if constexpr (kFp4) {
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
    if (!mine) return;
    const uint32_t sc = e4m3_code(__fdiv_rn(amax, 6.0f));
    const float s = e4m3_to_float(sc);
    const uint32_t codes = sc ? e2m1x8(v, s) : 0u;
    if (at.page >= 0) {
      uint8_t* data = (is_v ? a.c.v : a.c.k) + block * kv_block_bytes(kDim_, true);
      *reinterpret_cast<uint32_t*>(data + at.slot * (kDim_ / 2) + c0 / 2) = codes;
      if ((col & 1) == 0)
        ((is_v ? a.c.vs : a.c.ks) + block * kv_scale_bytes(kDim_))[at.slot * (kDim_ / 16) + col / 2] = (uint8_t)sc;
    }
    if (!plain) return;
    uint32_t d[4];
    codes8(codes, d);
#pragma unroll
    for (int i = 0; i < 4; ++i) {  // E2M1 x E4M3: exact in fp32 and in bf16
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&d[i]));
      d[i] = bf16x2(f.x * s, f.y * s);
    }
    stored = make_uint4(d[0], d[1], d[2], d[3]);
  } else {
    if (!mine) return;
    stored = make_uint4(bf16x2(v[0], v[1]), bf16x2(v[2], v[3]), bf16x2(v[4], v[5]), bf16x2(v[6], v[7]));
    if (at.page >= 0)
      *reinterpret_cast<uint4*>((is_v ? a.c.v : a.c.k) + block * kv_block_bytes(kDim_, false) +
                                (col * kPage + at.slot) * 16) = stored;
    if (!plain) return;
  }
  *reinterpret_cast<uint4*>(plain + ((int64_t)at.n * a.n_kv + h) * kDim_ + c0) = stored;
}

template <int kDim_, bool kFp4, int kPasses>
__global__ void __launch_bounds__(kThreads) kv_append_few_kernel(AppendArgs a) {
  constexpr int kLanes = kDim_ / 8;              // threads of a row
  constexpr int kRows = kThreads / kLanes;       // rows of a pass
  griddep_wait();  // every input may be the previous kernel's output
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
  const bool page_ok = page >= 0 && page < a.c.num_pages;
  if (!page_ok && tid == 0) report(a.status, CSA2_ERR_BAD_PAGE);
  const Place at{n, page_ok ? page : -1, (int)(pos % kPage)};

  const int pairs = a.rope_dims / 2;
  const bool turned = c0 < a.rope_dims;
  Turn turn = {};
  if (turned) turn.load(reinterpret_cast<const float4*>(a.rope + pos * a.rope_dims), c0, pairs, a.half);
  const int mate = ((tid & 31) + (c0 >= pairs ? -pairs : pairs) / 8) & 31;
#pragma unroll
  for (int p = 0; p < kPasses; ++p) {
    const int r = first + p * kRows;
    put_row<kDim_, kFp4>(a, at, r, r < n_rows, col, turn, turned, mate, raw[p]);
  }
}

// ---- many tokens
constexpr int kSlots = 4, kWorkWarps = 8, kStreamThreads = 32 * (kWorkWarps + 1);
template <int kDim_>
constexpr int kPieceRows = 24576 / (2 * kDim_);  // at most, of one token

constexpr int kSmall = 4;  // small tokens stand this many in a piece
template <int kTokens>
struct StreamPiece {   // what the workers need to know of a piece
  Place at[kTokens];   // n < 0: no token
  int row0, rows;      // of each token; no rows: the end
};

// Sequence of token n by bisection over cu (the first that ends behind n), and
// its place; false when it has none.
__device__ __forceinline__ bool find_place(const AppendArgs& a, int n, Place& at, int64_t& pos) {
  int lo_b = 0, hi_b = a.B;
  while (lo_b < hi_b) {
    const int mid = (lo_b + hi_b) / 2;
    if (__ldg(a.cu + mid + 1) <= n) lo_b = mid + 1;
    else hi_b = mid;
  }
  if (lo_b >= a.B) return false;  // behind the last sequence
  const int lo = __ldg(a.cu + lo_b), hi = __ldg(a.cu + lo_b + 1);
  if (n < lo && lo_b == 0 && lo <= a.T) return false;  // ahead of the first
  pos = __ldg(a.pos0 + lo_b) + (n - lo);
  if (lo < 0 || n < lo || n >= hi || hi > a.T || pos < 0 || pos >= (int64_t)a.c.max_pages * kPage ||
      (a.rope_dims && pos >= a.rope_rows)) {
    report(a.status, CSA2_ERR_BAD_INDEX);
    return false;
  }
  const int32_t page = __ldg(a.c.table + (int64_t)lo_b * a.c.max_pages + pos / kPage);
  const bool there = page >= 0 && page < a.c.num_pages;
  if (!there) report(a.status, CSA2_ERR_BAD_PAGE);
  at = Place{n, there ? page : -1, (int)(pos % kPage)};
  return true;
}

template <int kDim_>
constexpr int slot_bytes() { return kPieceRows<kDim_> * kDim_ * 2 + kDim_ * 4; }  // each token's rows, then its angles

template <int kDim_, bool kFp4, int kTokens>
__global__ void __launch_bounds__(kStreamThreads, 2) kv_append_stream_kernel(AppendArgs a) {
  constexpr int kLanes = kDim_ / 8, kWarpRows = 32 / kLanes;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ __align__(8) uint64_t full[kSlots], empty[kSlots];
  __shared__ StreamPiece<kTokens> piece[kSlots];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    for (int s = 0; s < kSlots; ++s) {
      tc::mbar_init(&full[s], kTokens);
      tc::mbar_init(&empty[s], kWorkWarps);
    }
    tc::fence_mbar_init();
  }
  __syncthreads();
  griddep_wait();  // every input may be the previous kernel's output
  // A piece holds kTokens whole tokens, or (per > 1) one of the parts of a token.
  const int n_rows = a.n_q + 2 * a.n_kv;
  const int per = kTokens > 1 ? 1 : (n_rows + kPieceRows<kDim_> - 1) / kPieceRows<kDim_>;
  const int most = ((n_rows + per - 1) / per + 15) / 16 * 16;  // rows of a part
  const int64_t pieces = per > 1 ? (int64_t)a.T * per : (a.T + kTokens - 1) / kTokens;
  const int angles = (per > 1 ? most : n_rows) * kDim_ * 2, token_bytes = angles + a.rope_dims * 4;
  bool ok = true;
  if (warp == kWorkWarps) {
    int count = 0;  // pieces sent so far
    const int k = lane % kTokens, groups = 32 / kTokens;
    for (int64_t base = blockIdx.x; base < pieces && ok; base += groups * (int64_t)gridDim.x) {
      // each lane looks up one token
      const int64_t i = base + lane / kTokens * (int64_t)gridDim.x;
      const int64_t n = per > 1 ? i / per : i * kTokens + k;
      const int row0 = per > 1 ? (int)(i % per) * most : 0;
      Place at{-1, -1, 0};
      int64_t pos = 0;
      // (parts are whole passes: a token's last may be empty)
      const bool there = i < pieces && n < a.T && row0 < n_rows && find_place(a, (int)n, at, pos);
      const uint32_t found = __ballot_sync(0xffffffffu, there);
      for (int g = 0; g < groups && ok; ++g) {
        if (!((found >> (g * kTokens)) & ((2u << (kTokens - 1)) - 1u))) continue;
        const int s = count % kSlots;
        if (count >= kSlots) ok = __all_sync(0xffffffffu, tc::mbar_wait(&empty[s], ((count / kSlots) & 1) ^ 1));
        if (!ok) break;
        ++count;
        if (lane / kTokens == g) {
          const int rows = min(per > 1 ? most : n_rows, n_rows - row0);
          piece[s].at[k] = at;
          if (k == 0) piece[s].row0 = row0, piece[s].rows = rows;
          uint8_t* dst = smem + s * slot_bytes<kDim_>() + k * token_bytes;
          tc::mbar_arrive_expect_tx(&full[s], there ? rows * kDim_ * 2 + a.rope_dims * 4 : 0);
          if (there) {
            // queries, keys and values: up to three runs
            const int q1 = min(row0 + rows, a.n_q), k1 = min(row0 + rows, a.n_q + a.n_kv);
            if (row0 < q1) tc::bulk_g2s(dst, a.q + n * a.q_stride + row0 * kDim_, (q1 - row0) * kDim_ * 2, &full[s]);
            const int k0 = max(row0, a.n_q);
            if (k0 < k1)
              tc::bulk_g2s(dst + (k0 - row0) * kDim_ * 2, a.k + n * a.k_stride + (k0 - a.n_q) * kDim_,
                           (k1 - k0) * kDim_ * 2, &full[s]);
            const int v0 = max(row0, a.n_q + a.n_kv), v1 = row0 + rows;
            if (v0 < v1)
              tc::bulk_g2s(dst + (v0 - row0) * kDim_ * 2, a.v + n * a.v_stride + (v0 - a.n_q - a.n_kv) * kDim_,
                           (v1 - v0) * kDim_ * 2, &full[s]);
            if (a.rope_dims)
              tc::bulk_g2s(dst + angles, a.rope + pos * a.rope_dims, a.rope_dims * 4, &full[s]);
          }
        }
        __syncwarp();
      }
    }
    // the end: a piece without rows
    const int s = count % kSlots;
    if (ok && count >= kSlots) ok = __all_sync(0xffffffffu, tc::mbar_wait(&empty[s], ((count / kSlots) & 1) ^ 1));
    if (!ok && lane == 0) report(a.status, CSA2_ERR_TIMEOUT);
    if (ok && lane < kTokens) {
      if (lane == 0) piece[s].rows = 0;
      tc::mbar_arrive(&full[s]);
    }
    // nothing may land in shared memory after the CTA has left
    for (int i = max(0, count - kSlots + (ok ? 1 : 0)); i < count; ++i) tc::mbar_wait(&full[i % kSlots], (i / kSlots) & 1);
  } else {
    const int col = tid % kLanes, c0 = 8 * col, pairs = a.rope_dims / 2;
    const bool turned = c0 < a.rope_dims;
    const int mate = (lane + (c0 >= pairs ? -pairs : pairs) / 8) & 31;
    // each token's share of the warps
    constexpr int kShare = kWorkWarps / kTokens;
    const int k = warp / kShare;
    for (int count = 0;; ++count) {
      const int s = count % kSlots;
      if (!__all_sync(0xffffffffu, tc::mbar_wait(&full[s], (count / kSlots) & 1))) {
        if (lane == 0) report(a.status, CSA2_ERR_TIMEOUT);
        break;
      }
      const int rows = piece[s].rows, row0 = piece[s].row0;
      if (rows == 0) break;
      const Place at = piece[s].at[k];
      if (at.n >= 0) {
        const uint8_t* src = smem + s * slot_bytes<kDim_>() + k * token_bytes;
        Turn turn = {};
        if (turned) turn.load(reinterpret_cast<const float4*>(src + angles), c0, pairs, a.half);
#pragma unroll 2
        for (int r0 = warp % kShare * kWarpRows; r0 < rows; r0 += kShare * kWarpRows) {
          const int r = r0 + lane / kLanes;
          const bool live = r < rows;
          put_row<kDim_, kFp4>(a, at, row0 + r, live, col, turn, turned, mate,
                               live ? *reinterpret_cast<const uint4*>(src + (r * kDim_ + c0) * 2) : make_uint4(0, 0, 0, 0));
        }
      }
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&empty[s]);
    }
  }
}

template <int kDim_, bool kFp4, int kTokens>
cudaError_t stream_of(const AppendArgs& a, int64_t pieces, cudaStream_t stream) {
  auto kern = kv_append_stream_kernel<kDim_, kFp4, kTokens>;
  constexpr int kSmem = kSlots * slot_bytes<kDim_>();
  static std::atomic<bool> done[64];
  const cudaError_t e = allow_smem(kern, kSmem, done);
  if (e != cudaSuccess) return e;
  const int64_t ctas = std::min<int64_t>(pieces, 2 * num_sms());
  return launch_k(kern, dim3((unsigned)ctas), dim3(kStreamThreads), kSmem, stream, 0, a);
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
  const int rows = a.n_q + 2 * a.n_kv;
  const bool fp4 = cfg.cache_dtype == CSA2_CACHE_FP4;
  const int piece_rows = 24576 / (2 * cfg.head_dim);
  const int64_t pieces = (int64_t)T * ((rows + piece_rows - 1) / piece_rows);
  if (pieces >= kFewItems * num_sms()) {
    // four small tokens to a piece where they fit: 4096 tokens of 24 + 2 x 8 heads of
    // 64 in FP4 take 14.0 us so and 19.9 us one by one, 16000 take 37.5 and 65.2 us
    const bool small = kSmall * (rows + 2) <= piece_rows + 2;
#define CSA2_STREAM(D, F)                                                     \
  (small ? stream_of<D, F, kSmall>(a, (T + kSmall - 1) / kSmall, stream)      \
         : stream_of<D, F, 1>(a, pieces, stream))
    if (cfg.head_dim == 128) return fp4 ? CSA2_STREAM(128, true) : CSA2_STREAM(128, false);
    return fp4 ? CSA2_STREAM(64, true) : CSA2_STREAM(64, false);
#undef CSA2_STREAM
  }
  const int per_pass = kThreads / (cfg.head_dim / 8), passes = (rows + per_pass - 1) / per_pass;
  // one pass a CTA while the passes do not fill the GPU, two beyond: 32 tokens of 128 +
  // 2 x 16 heads of 128 (320 passes) take 2.6 us by one and 3.1 by two, 200 tokens of 64
  // + 2 x 8 heads of 128 (1000 passes) 5.1 and 4.4
  const bool few = (int64_t)T * passes <= 3 * num_sms();
  const dim3 grid(T, few ? passes : (passes + 1) / 2), block(kThreads);
#define CSA2_APPEND(D, F)                                                          \
  (few ? launch_k(kv_append_few_kernel<D, F, 1>, grid, block, 0, stream, 0, a)     \
       : launch_k(kv_append_few_kernel<D, F, 2>, grid, block, 0, stream, 0, a))
  if (cfg.head_dim == 128) return fp4 ? CSA2_APPEND(128, true) : CSA2_APPEND(128, false);
  return fp4 ? CSA2_APPEND(64, true) : CSA2_APPEND(64, false);
#undef CSA2_APPEND
}

}  // namespace csa2
