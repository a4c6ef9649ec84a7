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
// With positions of three axes the same calls take 3.8 us (all of an append's GPU time in a
// graph) and 67 us.
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
  // positions of several axes (kAxes), [T][n_axes], and the axis of each pair, two bits
  const int32_t* axes;
  int n_axes;
  uint32_t axis_of[4];
};

__device__ __forceinline__ int axis_of(const AppendArgs& a, int pair) {
  const int w = pair >> 4;
  const uint32_t bits = w == 0 ? a.axis_of[0] : w == 1 ? a.axis_of[1] : w == 2 ? a.axis_of[2] : a.axis_of[3];
  return (int)(bits >> (2 * (pair & 15))) & 3;
}

__device__ __forceinline__ void widen(const uint32_t (&u)[4], float (&x)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(u[i] << 16);
    x[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
  }
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
  // angle(i): that of the thread's i-th pair
  template <typename Angle>
  __device__ __forceinline__ void load_axes(Angle angle, bool second, bool half) {
    if (half) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float2 f = angle(i);
        c[i] = f.x, s[i] = second ? f.y : -f.y;
      }
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 f = angle(i);
        c[2 * i] = c[2 * i + 1] = f.x;
        s[2 * i] = -f.y, s[2 * i + 1] = f.y;
      }
    }
  }
};
// The first pair of a thread's eight channels (eight pairs' a's or b's, or four pairs).
__device__ __forceinline__ int first_pair(int c0, int pairs, bool half) { return half ? (c0 >= pairs ? c0 - pairs : c0) : c0 / 2; }

// A token's positions on the axes; false when one is outside the table.
__device__ __forceinline__ bool load_axes(const AppendArgs& a, int n, int (&at)[4]) {
  bool ok = true;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    at[i] = i < a.n_axes ? __ldg(a.axes + (int64_t)n * a.n_axes + i) : 0;
    ok = ok && at[i] >= 0 && at[i] < a.rope_rows;
  }
  return ok;
}

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

template <int kDim_, bool kFp4, int kPasses, bool kAxes>
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
  int axes[4];
  const bool on_table = kAxes ? load_axes(a, n, axes) : !a.rope_dims || pos < a.rope_rows;
  if (lo < 0 || n < lo || n >= hi || hi > a.T || pos < 0 || pos >= (int64_t)a.c.max_pages * kPage || !on_table) {
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
  if constexpr (kAxes) {
    const int p0 = first_pair(c0, pairs, a.half);
    if (turned)
      turn.load_axes([&](int i) {
        const int axis = axis_of(a, p0 + i);
        const int at = axis == 0 ? axes[0] : axis == 1 ? axes[1] : axis == 2 ? axes[2] : axes[3];
        return reinterpret_cast<const float2*>(a.rope + (int64_t)at * a.rope_dims)[p0 + i];
      }, c0 >= pairs, a.half);
  } else if (turned) {
    turn.load(reinterpret_cast<const float4*>(a.rope + pos * a.rope_dims), c0, pairs, a.half);
  }
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
template <bool kAxes>
__device__ __forceinline__ bool find_place(const AppendArgs& a, int n, Place& at, int64_t& pos, int (&axes)[4]) {
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
  const bool on_table = kAxes ? load_axes(a, n, axes) : !a.rope_dims || pos < a.rope_rows;
  if (lo < 0 || n < lo || n >= hi || hi > a.T || pos < 0 || pos >= (int64_t)a.c.max_pages * kPage || !on_table) {
    report(a.status, CSA2_ERR_BAD_INDEX);
    return false;
  }
  const int32_t page = __ldg(a.c.table + (int64_t)lo_b * a.c.max_pages + pos / kPage);
  const bool there = page >= 0 && page < a.c.num_pages;
  if (!there) report(a.status, CSA2_ERR_BAD_PAGE);
  at = Place{n, there ? page : -1, (int)(pos % kPage)};
  return true;
}

// Each token's rows, then its angles (of every axis: 4 slots of two CTAs still fit an SM).
template <int kDim_, bool kAxes>
constexpr int slot_bytes() { return kPieceRows<kDim_> * kDim_ * 2 + kDim_ * 4 * (kAxes ? 4 : 1); }

template <int kDim_, bool kFp4, int kTokens, bool kAxes>
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
  const int angles = (per > 1 ? most : n_rows) * kDim_ * 2, token_bytes = angles + a.rope_dims * 4 * (kAxes ? a.n_axes : 1);
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
      int axes[4];
      // (parts are whole passes: a token's last may be empty)
      const bool there = i < pieces && n < a.T && row0 < n_rows && find_place<kAxes>(a, (int)n, at, pos, axes);
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
          uint8_t* dst = smem + s * slot_bytes<kDim_, kAxes>() + k * token_bytes;
          tc::mbar_arrive_expect_tx(&full[s], there ? rows * kDim_ * 2 + token_bytes - angles : 0);
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
            if constexpr (kAxes) {
              for (int x = 0; x < a.n_axes; ++x)
                tc::bulk_g2s(dst + angles + x * a.rope_dims * 4,
                             a.rope + (int64_t)(x == 0 ? axes[0] : x == 1 ? axes[1] : x == 2 ? axes[2] : axes[3]) * a.rope_dims,
                             a.rope_dims * 4, &full[s]);
            } else if (a.rope_dims)
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
    // where the thread's pairs have their angles among a token's (found for each token, 86 us
    // for 8 prompts of 37 .. 2021 tokens of 64 + 2 x 8 heads of 128 in FP4)
    int of[8] = {};
    if (kAxes && turned)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int p = first_pair(c0, pairs, a.half) + (a.half ? i : i & 3);
        of[i] = axis_of(a, p) * a.rope_dims * 4 + p * 8;
      }
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
        const uint8_t* src = smem + s * slot_bytes<kDim_, kAxes>() + k * token_bytes;
        Turn turn = {};
        if constexpr (kAxes) {
          if (turned)
            turn.load_axes([&](int i) { return *reinterpret_cast<const float2*>(src + angles + of[i]); }, c0 >= pairs, a.half);
        } else if (turned) {
          turn.load(reinterpret_cast<const float4*>(src + angles), c0, pairs, a.half);
        }
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

template <int kDim_, bool kFp4, int kTokens, bool kAxes>
cudaError_t stream_of(const AppendArgs& a, int64_t pieces, cudaStream_t stream) {
  auto kern = kv_append_stream_kernel<kDim_, kFp4, kTokens, kAxes>;
  constexpr int kSmem = kSlots * slot_bytes<kDim_, kAxes>();
  static std::atomic<bool> done[64];
  const cudaError_t e = allow_smem(kern, kSmem, done);
  if (e != cudaSuccess) return e;
  const int64_t ctas = std::min<int64_t>(pieces, 2 * num_sms());
  return launch_k(kern, dim3((unsigned)ctas), dim3(kStreamThreads), kSmem, stream, 0, a);
}

template <bool kAxes>
cudaError_t launch_of(const csa2_kv_cfg& cfg, const AppendArgs& a, cudaStream_t stream) {
  const int rows = a.n_q + 2 * a.n_kv, T = a.T;
  const bool fp4 = cfg.cache_dtype == CSA2_CACHE_FP4;
  const int piece_rows = 24576 / (2 * cfg.head_dim);
  const int64_t pieces = (int64_t)T * ((rows + piece_rows - 1) / piece_rows);
  if (pieces >= kFewItems * num_sms()) {
    // four small tokens to a piece where they fit: 4096 tokens of 24 + 2 x 8 heads of
    // 64 in FP4 take 14.0 us so and 19.9 us one by one, 16000 take 37.5 and 65.2 us
    // (a slot has room for four rows of angles, each two rows' worth, with kAxes)
    const bool small = kAxes ? kSmall * (rows + 2 * a.n_axes) <= piece_rows + 8 : kSmall * (rows + 2) <= piece_rows + 2;
#define CSA2_STREAM(D, F)                                                             \
  (small ? stream_of<D, F, kSmall, kAxes>(a, (T + kSmall - 1) / kSmall, stream)       \
         : stream_of<D, F, 1, kAxes>(a, pieces, stream))
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
#define CSA2_APPEND(D, F)                                                                 \
  (few ? launch_k(kv_append_few_kernel<D, F, 1, kAxes>, grid, block, 0, stream, 0, a)     \
       : launch_k(kv_append_few_kernel<D, F, 2, kAxes>, grid, block, 0, stream, 0, a))
  if (cfg.head_dim == 128) return fp4 ? CSA2_APPEND(128, true) : CSA2_APPEND(128, false);
  return fp4 ? CSA2_APPEND(64, true) : CSA2_APPEND(64, false);
#undef CSA2_APPEND
}

}  // namespace

cudaError_t launch_kv_append(const csa2_kv_cfg& cfg, int B, int T, const uint16_t* q, int64_t q_stride,
                             const uint16_t* k, int64_t k_stride, const uint16_t* v, int64_t v_stride,
                             const int32_t* cu, const int64_t* pos0, const KvAxes& axes, const float* rope,
                             int64_t rope_rows, const KvView& c, uint16_t* q_out, int64_t q_out_stride, uint16_t* k_out,
                             uint16_t* v_out, int32_t* status, cudaStream_t stream) {
  AppendArgs a{B, T, q ? cfg.n_heads : 0, cfg.kv_heads, cfg.rope_dims, cfg.rope_style == CSA2_ROPE_HALF ? 1 : 0,
               q, k, v, q_stride, k_stride, v_stride, cu, pos0, rope, rope_rows, c, q_out, q_out_stride, k_out, v_out,
               status, axes.pos, axes.n, {}};
  for (int i = 0; axes.pos && i < cfg.rope_dims / 2; ++i) a.axis_of[i / 16] |= (uint32_t)axes.of[i] << (2 * (i % 16));
  return axes.pos ? launch_of<true>(cfg, a, stream) : launch_of<false>(cfg, a, stream);
}

}  // namespace csa2
