// Best continuations over beams and vocabulary.
//
// Within a beam the order of scores is that of its logits, so the best `take` of a group
// are among the best `take` logits of each beam; their scores need the beam's log-sum-
// exp, a shift.  So one pass over the logits, which bounds the call (HBM for a serving
// batch, latency for one user's beams):
//  - beam_part_kernel: a CTA holds a part of up to 16384 logits of a row in registers and
//    forms the part's maximum m, the sum of exp(x - m) (32 in fp32, these in fp64), and its best `take` logits in
//    order: the `take`-th largest of 64 groups' maxima is a lower bound of the take-th
//    largest logit, the few logits that reach it go to a list, and the list is ranked by
//    counting.  Where ties make the list too long, the best are found one by one.
//  - beam_join_kernel: a CTA a group adds the parts' sums in fp64, forms the candidates'
//    scores in fp64 and ranks them in the same way, by (score, beam, token).
#include <algorithm>

#include "kv.cuh"

namespace csa2 {
namespace {

constexpr int kThreads = 512, kWarps = kThreads / 32, kList = 1024;
constexpr int kPart = 16384, kPer = kPart / kThreads;  // logits of a CTA, of a thread
constexpr int kMost = 64;                               // take, beams

struct PartSum {
  double sum;  // of exp(x - most)
  float most, pad;
};
struct BeamArgs {
  int groups, beams, vocab, take, parts;
  const void* logits;
  int64_t stride;
  const float* cum;
  const uint8_t* done;
  int end_token;
  float* scores;
  int32_t* parents;
  int32_t* tokens;
  float* lse;
  PartSum* part_sum;  // [rows][parts]
  uint2* part_best;   // [rows][parts][take] logit bits, token
  int32_t* status;
};

// fp32 -> unsigned in the same order; -inf -> 0x007FFFFF.
__device__ __forceinline__ uint32_t key_of(float x) {
  const uint32_t u = __float_as_uint(x + 0.0f);  // -0 -> +0: equal logits are equal
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float of_key(uint32_t k) { return __uint_as_float(k & 0x80000000u ? k & 0x7FFFFFFFu : ~k); }
constexpr uint32_t kNone = 0x007FFFFFu;  // of -inf

__device__ __forceinline__ float clean(float x, bool& bad) {
  if (!(x < INFINITY)) {
    bad = true;
    return -INFINITY;
  }
  return x;
}

template <bool kBf16>
__global__ void __launch_bounds__(kThreads) beam_part_kernel(const BeamArgs a) {
  __shared__ double sums[kWarps];
  __shared__ float most;
  __shared__ uint32_t best[64];
  __shared__ uint32_t bound, count;
  __shared__ uint2 list[kList];
  griddep_wait();  // every input may be the previous kernel's output
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int part = blockIdx.x;
  const int64_t row = blockIdx.y + (int64_t)blockIdx.z * 65535;
  if (row >= (int64_t)a.groups * a.beams) return;
  const int64_t at = row * a.parts + part;
  if (a.done && a.done[row]) return;
  const int v0 = part * kPart, n = min(kPart, a.vocab - v0);
  // element j of a thread: v0 + (j / 8) * 8 * kThreads + 8 * tid + j % 8
  float x[kPer];
  bool bad = false;
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    const int i = (j / 8) * (8 * kThreads) + 8 * tid + (j & 7);
    x[j] = -INFINITY;
    if (i < n) {
      const int64_t e = row * a.stride + v0 + i;
      x[j] = clean(kBf16 ? bf16_bits_to_float(__ldg(static_cast<const uint16_t*>(a.logits) + e))
                         : __ldg(static_cast<const float*>(a.logits) + e), bad);
    }
  }
  if (bad) report(a.status, CSA2_ERR_RANGE);
  float m = -INFINITY;
#pragma unroll
  for (int j = 0; j < kPer; ++j) m = fmaxf(m, x[j]);
  // maxima of 64 groups of 8 threads
  uint32_t mine = key_of(m);
  uint32_t group = mine;
#pragma unroll
  for (int d = 1; d < 8; d <<= 1) group = max(group, __shfl_xor_sync(0xffffffffu, group, d));
  if ((tid & 7) == 0) best[tid >> 3] = group;
  if (tid == 0) count = 0;
  __syncthreads();
  if (tid < 64) {
    const uint32_t k = best[tid];
    int rank = 0;
    for (int j = 0; j < 64; ++j) rank += best[j] > k || (best[j] == k && j < tid);
    if (rank == a.take - 1) bound = max(k, kNone + 1);
    if (rank == 0) most = of_key(k);
  }
  __syncthreads();
  const uint32_t least = bound;
  const float top = most;
  // the sum, and what reaches the bound
  float sum = 0.0f;
  constexpr float kHi = 1.44269502f, kLo = 1.92596299e-8f;  // log2 e
  if (top > -INFINITY) {
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      const float d = x[j] - top;
      sum += ex2(fmaf(d, kHi, d * kLo));
    }
  }
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    const uint32_t k = key_of(x[j]);
    if (k >= least) {
      const uint32_t p = atomicAdd(&count, 1u);
      if (p < kList) list[p] = make_uint2(k, v0 + (j / 8) * (8 * kThreads) + 8 * tid + (j & 7));
    }
  }
  double wide = sum;
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) wide += __shfl_xor_sync(0xffffffffu, wide, d);
  if (lane == 0) sums[warp] = wide;
  __syncthreads();
  if (tid == 0) {
    double s = 0.0;
    for (int w = 0; w < kWarps; ++w) s += sums[w];
    a.part_sum[at] = PartSum{s, top, 0.0f};
  }
  uint2* out = a.part_best + at * a.take;
  const int c = (int)count;
  if (c <= kList) {
    for (int p = tid; p < c; p += kThreads) {
      const uint2 e = list[p];
      int rank = 0;
      for (int q = 0; q < c; ++q) {
        const uint2 f = list[q];
        rank += f.x > e.x || (f.x == e.x && f.y < e.y);
      }
      if (rank < a.take) out[rank] = e;
    }
    for (int p = c + tid; p < a.take; p += kThreads) out[p] = make_uint2(kNone, 0);
  } else {
    // one by one: the best behind the last, (key, place) as one number
    __shared__ unsigned long long next[kWarps];
    unsigned long long last = ~0ull;
    for (int r = 0; r < a.take; ++r) {
      unsigned long long b = 0;
#pragma unroll
      for (int j = 0; j < kPer; ++j) {
        const uint32_t i = v0 + (j / 8) * (8 * kThreads) + 8 * tid + (j & 7);
        const unsigned long long e = (unsigned long long)key_of(x[j]) << 32 | (0xffffffffu - i);
        if (e < last && e > b) b = e;
      }
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) {
        const unsigned long long o = __shfl_xor_sync(0xffffffffu, b, d);
        b = o > b ? o : b;
      }
      __syncthreads();
      if (lane == 0) next[warp] = b;
      __syncthreads();
      for (int w = 0; w < kWarps; ++w) b = next[w] > b ? next[w] : b;
      last = b;
      if (tid == 0) out[r] = make_uint2((uint32_t)(b >> 32), 0xffffffffu - (uint32_t)b);
    }
  }
}

// fp64 -> unsigned in the same order.
__device__ __forceinline__ uint64_t key_of(double x) {
  const uint64_t u = (uint64_t)__double_as_longlong(x + 0.0);
  return u >> 63 ? ~u : u | 1ull << 63;
}
constexpr uint64_t kNone64 = 0x000FFFFFFFFFFFFFull;  // of -inf

__global__ void __launch_bounds__(kThreads) beam_join_kernel(const BeamArgs a) {
  __shared__ double shift[kMost];  // cum - lse
  __shared__ uint64_t best[64];
  __shared__ uint64_t bound;
  __shared__ uint32_t count;
  __shared__ uint64_t lkey[kList];
  __shared__ uint2 lplace[kList];  // beam, token
  __shared__ unsigned long long wkey[kWarps], wplace[kWarps];
  griddep_wait();
  const int g = blockIdx.x, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int64_t row0 = (int64_t)g * a.beams;
  for (int k = warp; k < a.beams; k += kWarps) {
    const int64_t row = row0 + k;
    const bool over = a.done && a.done[row];
    double lse = 0.0;
    if (!over) {
      float m = -INFINITY;
      for (int p = lane; p < a.parts; p += 32) m = fmaxf(m, a.part_sum[row * a.parts + p].most);
      m = of_key(__reduce_max_sync(0xffffffffu, key_of(m)));
      double s = 0.0;
      for (int p = lane; p < a.parts; p += 32) {
        const PartSum e = a.part_sum[row * a.parts + p];
        if (e.most > -INFINITY) s += e.sum * exp((double)e.most - (double)m);
      }
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
      lse = m > -INFINITY ? (double)m + log(s) : -INFINITY;
    }
    if (lane == 0) {
      bool bad = false;
      const float c = clean(a.cum[row], bad);
      if (bad) report(a.status, CSA2_ERR_RANGE);
      shift[k] = lse > -INFINITY ? (double)c - lse : -INFINITY;
      if (a.lse) a.lse[row] = (float)lse;
    }
  }
  if (tid == 0) count = 0;
  __syncthreads();
  // candidate c: beam c / per, then part, then rank in it; a done beam has its first alone
  const int per = a.parts * a.take, total = a.beams * per;
  auto score_of = [&](int c, int& beam, int& token) {
    beam = c / per;
    const int64_t row = row0 + beam;
    if (a.done && a.done[row]) {
      token = a.end_token;
      return c % per == 0 ? shift[beam] : -(double)INFINITY;
    }
    const uint2 e = a.part_best[row * per + c % per];
    token = (int)e.y;
    return e.x > kNone ? (double)of_key(e.x) + shift[beam] : -(double)INFINITY;
  };
  uint64_t top = kNone64;
  for (int c = tid; c < total; c += kThreads) {
    int b, t;
    top = max(top, key_of(score_of(c, b, t)));
  }
#pragma unroll
  for (int d = 1; d < 8; d <<= 1) top = max(top, (uint64_t)__shfl_xor_sync(0xffffffffu, (unsigned long long)top, d));
  if ((tid & 7) == 0) best[tid >> 3] = top;
  __syncthreads();
  if (tid < 64) {
    const uint64_t k = best[tid];
    int rank = 0;
    for (int j = 0; j < 64; ++j) rank += best[j] > k || (best[j] == k && j < tid);
    if (rank == a.take - 1) bound = max(k, kNone64 + 1);
  }
  __syncthreads();
  for (int c = tid; c < total; c += kThreads) {
    int b, t;
    const uint64_t k = key_of(score_of(c, b, t));
    if (k >= bound) {
      const uint32_t p = atomicAdd(&count, 1u);
      if (p < kList) lkey[p] = k, lplace[p] = make_uint2(b, t);
    }
  }
  __syncthreads();
  auto put = [&](int r, uint64_t k, uint32_t beam, uint32_t token) {
    const double s = __longlong_as_double((long long)(k >> 63 ? k & 0x7FFFFFFFFFFFFFFFull : ~k));
    const int64_t o = (int64_t)g * a.take + r;
    a.scores[o] = (float)s, a.parents[o] = (int32_t)(row0 + beam), a.tokens[o] = (int32_t)token;
  };
  auto none = [&](int r) {
    const int64_t o = (int64_t)g * a.take + r;
    a.scores[o] = -INFINITY, a.parents[o] = -1, a.tokens[o] = -1;
  };
  const int n = (int)count;
  if (n <= kList) {
    for (int p = tid; p < n; p += kThreads) {
      const uint64_t k = lkey[p];
      const uint2 e = lplace[p];
      int rank = 0;
      for (int q = 0; q < n; ++q) {
        const uint2 f = lplace[q];
        rank += lkey[q] > k || (lkey[q] == k && (f.x < e.x || (f.x == e.x && f.y < e.y)));
      }
      if (rank < a.take) put(rank, k, e.x, e.y);
    }
    for (int r = n + tid; r < a.take; r += kThreads) none(r);
    return;
  }
  // more than the list holds have the same scores: one by one
  unsigned long long last_k = ~0ull, last_p = 0;
  for (int r = 0; r < a.take; ++r) {
    unsigned long long bk = kNone64, bp = ~0ull;  // place: the smaller first
    for (int c = tid; c < total; c += kThreads) {
      int b, t;
      const unsigned long long k = key_of(score_of(c, b, t)), p = (unsigned long long)b << 32 | (uint32_t)t;
      const bool behind = k < last_k || (k == last_k && p > last_p);
      if (behind && (k > bk || (k == bk && p < bp))) bk = k, bp = p;
    }
    for (int d = 16; d > 0; d >>= 1) {
      const unsigned long long ok = __shfl_xor_sync(0xffffffffu, bk, d), op = __shfl_xor_sync(0xffffffffu, bp, d);
      if (ok > bk || (ok == bk && op < bp)) bk = ok, bp = op;
    }
    __syncthreads();
    if (lane == 0) wkey[warp] = bk, wplace[warp] = bp;
    __syncthreads();
    for (int w = 0; w < kWarps; ++w)
      if (wkey[w] > bk || (wkey[w] == bk && wplace[w] < bp)) bk = wkey[w], bp = wplace[w];
    last_k = bk, last_p = bp;
    if (tid == 0) {
      if (bk > kNone64) put(r, bk, (uint32_t)(bp >> 32), (uint32_t)bp);
      else none(r);
    }
  }
}

int parts_of(int vocab) { return (int)(((int64_t)vocab + kPart - 1) / kPart); }
bool sizes_ok(int32_t groups, int32_t beams, int32_t vocab, int32_t take) {
  return groups >= 0 && beams >= 1 && vocab >= 1 && take >= 1;
}
bool sizes_fit(int32_t groups, int32_t beams, int32_t vocab, int32_t take) {
  return beams <= kMost && take <= kMost && (int64_t)groups * beams * parts_of(vocab) <= INT32_MAX &&
         (int64_t)parts_of(vocab) * beams * take <= INT32_MAX / 2;
}
size_t sums_bytes(int64_t groups, int beams, int vocab) {
  return (size_t)((groups * beams * parts_of(vocab) * sizeof(PartSum) + 255) / 256 * 256);
}
bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

}  // namespace
}  // namespace csa2

using namespace csa2;

extern "C" {

size_t csa2_beam_workspace_bytes(int32_t groups, int32_t beams, int32_t vocab, int32_t take) {
  if (!sizes_ok(groups, beams, vocab, take) || !sizes_fit(groups, beams, vocab, take)) return 0;
  return sums_bytes(groups, beams, vocab) + (size_t)groups * beams * parts_of(vocab) * take * sizeof(uint2);
}

int32_t csa2_beam_select(int32_t groups, int32_t beams, int32_t vocab, int32_t take, const void* logits,
                         int32_t logits_dtype, int64_t stride, const float* cum, const uint8_t* done, int32_t end_token,
                         float* scores, int32_t* parents, int32_t* tokens, float* lse, void* workspace,
                         size_t workspace_bytes, int32_t* status, void* stream) {
  if (!sizes_ok(groups, beams, vocab, take) || (logits_dtype != CSA2_BF16 && logits_dtype != CSA2_F32))
    return CSA2_ERR_INVALID_ARG;
  if (!sizes_fit(groups, beams, vocab, take)) return CSA2_ERR_UNSUPPORTED;
  if (groups == 0) return CSA2_OK;
  if (!logits || !cum || !scores || !parents || !tokens || !aligned(logits, 16) || stride < vocab || !aligned(cum, 4) ||
      !aligned(scores, 4) || !aligned(parents, 4) || !aligned(tokens, 4) || !aligned(lse, 4) || !aligned(status, 4) ||
      (done && (end_token < 0 || end_token >= vocab)) || !aligned(workspace, 256))
    return CSA2_ERR_INVALID_ARG;
  if (!workspace || workspace_bytes < csa2_beam_workspace_bytes(groups, beams, vocab, take)) return CSA2_ERR_CAPACITY;
  BeamArgs a{groups, beams, vocab, take, parts_of(vocab), logits, stride, cum, done, end_token, scores, parents, tokens, lse,
             static_cast<PartSum*>(workspace),
             reinterpret_cast<uint2*>(static_cast<uint8_t*>(workspace) + sums_bytes(groups, beams, vocab)), status};
  const int64_t rows = (int64_t)groups * beams;
  const dim3 grid(a.parts, (unsigned)std::min<int64_t>(rows, 65535), (unsigned)((rows + 65534) / 65535));
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e = logits_dtype == CSA2_BF16 ? launch_k(beam_part_kernel<true>, grid, dim3(kThreads), 0, s, 0, a)
                                            : launch_k(beam_part_kernel<false>, grid, dim3(kThreads), 0, s, 0, a);
  if (e == cudaSuccess) e = launch_k(beam_join_kernel, dim3(groups), dim3(kThreads), 0, s, 0, a);
  return e == cudaSuccess ? CSA2_OK : CSA2_ERR_CUDA;
}

}  // extern "C"
