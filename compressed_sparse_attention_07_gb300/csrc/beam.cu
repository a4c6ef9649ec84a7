// Best continuations over beams and vocabulary.
//
// Within a beam the order of scores is that of its logits, so the best `take` of a group
// are among the best `take` logits of each beam; their scores need the beam's log-sum-
// exp, a shift.  So one pass over the logits, which bounds the call (HBM for a serving
// batch, latency for one user's beams):
//  - beam_part_kernel: a warp streams a part of a row through registers, 2048 bf16 or 1024
//    fp32 logits (a window) at a time, so nothing waits on another warp (with 16384
//    logits a CTA and five barriers, 512 beams of 128001 took 84 us).  It keeps the
//    largest so far, the sum of exp(x - it), and a list of the logits that may be among the
//    best: of the lanes' maxima so far the `take`-th largest, to 16 bits, is a lower
//    bound of the take-th largest logit; the few 16-byte vectors of the window whose
//    maximum reaches it are read again, and the logits that do are listed.  In the end
//    those that reach the last bound are ranked by counting.  Where ties make the list
//    too long, the best are found one by one.
//  - beam_join_kernel: a CTA a group adds the parts' sums as sums of two fp32, forms the
//    candidates' scores in fp64 and ranks them in the same way, by (score, beam, token).
#include <algorithm>

#include "kv.cuh"

namespace csa2 {
namespace {

constexpr int kMost = 64;  // take, beams
// part: warps of a CTA, 16-byte vectors of a lane in a window, list of a warp, windows of a warp
constexpr int kPartWarps = 4, kN = 8, kPartList = 512;
__host__ __device__ constexpr int most_windows(int take) { return take > 32 ? 4 : 8; }  // (what they list fits kPartList)
// join
constexpr int kThreads = 512, kWarps = kThreads / 32, kList = 2048;

struct PartSum {
  float sum, low;  // of exp(x - most), as the sum of two fp32
  float most, pad;
};
struct BeamArgs {
  int groups, beams, vocab, take, parts, part;  // part: logits of one
  Divisor by_parts;
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
  int bf16;
};

// fp32 -> unsigned in the same order; -inf -> 0x007FFFFF.
__device__ __forceinline__ uint32_t key_of(float x) {
  const uint32_t u = __float_as_uint(x + 0.0f);  // -0 -> +0: equal logits are equal
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float of_key(uint32_t k) { return __uint_as_float(k & 0x80000000u ? k & 0x7FFFFFFFu : ~k); }
constexpr uint32_t kNone = 0x007FFFFFu;  // of -inf
constexpr uint32_t kDone = 0xFFFFFFFFu;  // of no number: what a beam that is done proposes

__device__ __forceinline__ float counts_as(float x) { return x < INFINITY ? x : -INFINITY; }
__device__ __forceinline__ float clean(float x, bool& bad) {
  bad = bad || !(x < INFINITY);
  return counts_as(x);
}
// The larger, NaN if one is.
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ uint32_t max_nan2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ float low(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float high(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// A lane's logits of a window as they come, vectors of 16 bytes, 32 apart.
template <bool kBf16>
struct Held {
  static constexpr int kVec = kBf16 ? 8 : 4;
  uint4 v[kN];
  static __device__ __forceinline__ float get(const uint4& u, int i) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
    if constexpr (kBf16) return i & 1 ? high(w[i / 2]) : low(w[i / 2]);
    else return __uint_as_float(w[i]);
  }
  // what is no number, or +inf, as -inf
  static __device__ __forceinline__ uint32_t clean_word(uint32_t w) {
    if constexpr (kBf16) {
      if (!(low(w) < INFINITY)) w = (w & 0xFFFF0000u) | 0xFF80u;
      if (!(high(w) < INFINITY)) w = (w & 0xFFFFu) | 0xFF800000u;
      return w;
    } else {
      return __uint_as_float(w) < INFINITY ? w : 0xFF800000u;
    }
  }
  static __device__ __forceinline__ void clean_vector(uint4& u) {
    u = make_uint4(clean_word(u.x), clean_word(u.y), clean_word(u.z), clean_word(u.w));
  }
  // the largest of vector j, NaN if one is
  __device__ __forceinline__ float most(int j) const {
    const uint4 u = v[j];
    if constexpr (kBf16) {
      const uint32_t m = max_nan2(max_nan2(u.x, u.y), max_nan2(u.z, u.w));
      return max_nan(low(m), high(m));
    } else {
      return max_nan(max_nan(get(u, 0), get(u, 1)), max_nan(get(u, 2), get(u, 3)));
    }
  }
};

// kMany: more than 32 to take.
template <bool kBf16, bool kMany>
__global__ void __launch_bounds__(32 * kPartWarps, kMany ? 6 : 7) beam_part_kernel(const BeamArgs a) {
  using H = Held<kBf16>;
  constexpr int kVec = H::kVec;
  constexpr uint32_t kAll = 0xffffffffu;
  __shared__ uint2 lists[kPartWarps][kPartList];
  __shared__ int counts[kPartWarps];
  griddep_wait();    // every input may be the previous kernel's output
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int at = blockIdx.x * kPartWarps + warp, row = quotient(at, a.by_parts);
  if (row >= a.groups * a.beams) return;  // (whole warps)
  if (a.done && a.done[row]) {            // one candidate, at cum: of lse 0 and a key of its own
    const bool has = at == row * a.parts;
    for (int r = lane; r < a.take; r += 32)
      a.part_best[(int64_t)at * a.take + r] = make_uint2(has && r == 0 ? kDone : kNone, (uint32_t)a.end_token);
    if (lane == 0) a.part_sum[at] = has ? PartSum{1.0f, 0.0f, 0.0f, 0.0f} : PartSum{0.0f, 0.0f, -INFINITY, 0.0f};
    return;
  }
  // Values [v0, v1) of the row: whole 16 bytes of memory from v0 + head on, and what is
  // before and behind them (rows of an odd size begin anywhere), a value a lane.
  const int v0 = (at - row * a.parts) * a.part, v1 = min(v0 + a.part, a.vocab), n = max(0, v1 - v0);
  const int64_t e0 = row * a.stride + v0;
  const int head = min(n, (int)(-e0 & (kVec - 1))), vectors = (n - head) / kVec, tail = n - head - vectors * kVec;
  const uint8_t* first = static_cast<const uint8_t*>(a.logits) + e0 * (kBf16 ? 2 : 4);
  const uint4* window = reinterpret_cast<const uint4*>(first + head * (kBf16 ? 2 : 4)) + lane;
  const uint32_t none = kBf16 ? 0xFF80FF80u : 0xFF800000u;
  H x;
  auto load = [&](int from) {
#pragma unroll
    for (int j = 0; j < kN; ++j) {
      x.v[j] = make_uint4(none, none, none, none);
      if (from + 32 * j + lane < vectors) x.v[j] = __ldg(window + from + 32 * j);
    }
  };
  load(0);
  const int odd = lane < head ? lane : lane - head < tail ? n - tail + lane - head : -1;  // its place in the part
  float alone = -INFINITY;
  bool bad = false;
  if (odd >= 0)
    alone = clean(kBf16 ? bf16_bits_to_float(__ldg(reinterpret_cast<const uint16_t*>(first) + odd))
                        : __ldg(reinterpret_cast<const float*>(first) + odd), bad);
  uint2* list = lists[warp];
  if (lane == 0) counts[warp] = 0;
  __syncwarp();
  auto take_in = [&](float value, int place) {
    const int c = atomicAdd(&counts[warp], 1);
    if (c < kPartList) list[c] = make_uint2(key_of(value), v0 + place);
  };

  float run0 = alone, run1 = -INFINITY;  // the lane's largest so far, of each half of its vectors
  float top = -INFINITY;                 // the warp's
  double sum = 0.0;                      // of exp(x - top), the lane's
  uint32_t bound = kNone + 1;            // of keys
  for (int from = 0; from == 0 || from < vectors; from += 32 * kN) {
    float vm[kN], m0 = -INFINITY, m1 = -INFINITY;
#pragma unroll
    for (int j = 0; j < kN; ++j) {
      vm[j] = x.most(j);
      float& m = j < kN / 2 ? m0 : m1;
      m = max_nan(m, vm[j]);
    }
    const bool odd_ones = !__all_sync(kAll, max_nan(m0, m1) < INFINITY);  // NaN or +inf
    if (odd_ones) {
      bad = bad || !(max_nan(m0, m1) < INFINITY);
      m0 = m1 = -INFINITY;
#pragma unroll
      for (int j = 0; j < kN; ++j) {
        H::clean_vector(x.v[j]);
        vm[j] = x.most(j);
        float& m = j < kN / 2 ? m0 : m1;
        m = fmaxf(m, vm[j]);
      }
    }
    run0 = fmaxf(run0, m0), run1 = fmaxf(run1, m1);
    const uint32_t k0 = key_of(a.take > 16 ? run0 : fmaxf(run0, run1)), k1 = key_of(run1);
    const float most = of_key(__reduce_max_sync(kAll, max(k0, k1)));
    uint32_t hits = 0;
    if (most > -INFINITY) {
      if (most > top) {
        if (top > -INFINITY) sum *= (double)ex2((top - most) * kLog2e);
        top = most;
      }
      // the largest multiple of 2^16 that `take` of the maxima reach: of 32 up to 16 (of
      // which 22 logits are expected to reach it), else of 64
      uint32_t b = 0;
      if (a.take <= 16) {
#pragma unroll
        for (int i = 31; i >= 16; --i)
          if (__popc(__ballot_sync(kAll, k0 >= (b | 1u << i))) >= a.take) b |= 1u << i;
      } else {
#pragma unroll
        for (int i = 31; i >= 16; --i)
          if (__popc(__ballot_sync(kAll, k0 >= (b | 1u << i))) + __popc(__ballot_sync(kAll, k1 >= (b | 1u << i))) >= a.take)
            b |= 1u << i;
      }
      if constexpr (kMany) {
        // the last of 64 maxima is a weak bound (of 2048 logits 250 reach it, at times more than
        // the list holds, and one such warp took 500 us): of 128, the window's alone, 87
        uint32_t k[kN / 2], w = 0;
#pragma unroll
        for (int j = 0; j < kN / 2; ++j) k[j] = key_of(fmaxf(vm[2 * j], vm[2 * j + 1]));
#pragma unroll 1
        for (int i = 31; i >= 16; --i) {
          int reach = 0;
#pragma unroll
          for (int j = 0; j < kN / 2; ++j) reach += __popc(__ballot_sync(kAll, k[j] >= (w | 1u << i)));
          if (reach >= a.take) w |= 1u << i;
        }
        b = max(b, w);
      }
      bound = max(bound, b);
      const float least = of_key(bound);
#pragma unroll
      for (int j = 0; j < kN; ++j) hits |= (vm[j] >= least ? 1u : 0u) << j;
      if (from == 0 && alone >= least) take_in(alone, odd);
      const float odd_one = from == 0 ? ex2((alone - top) * kLog2e) : 0.0f;
      // The largest, 1 here, is counted apart where it stands alone: added in fp32 to what is beside it,
      // it would leave that to 2^-24, and of two beams with one likely word the better is the one
      // with less beside it.  Where another lane has a logit within 3 of it (nearly always of usual
      // rows) what is beside it is 0.05 at least.  64 x 8 beams of 128001 take 39.9 us so, 39.3 without
      // (within 2: 40.7).
      if (__popc(__ballot_sync(kAll, fmaxf(run0, run1) >= top - 3.0f)) == 1) {
        float ones = odd_one == 1.0f ? 1.0f : 0.0f, beside = odd_one == 1.0f ? 0.0f : odd_one;
#pragma unroll
        for (int j = 0; j < kN; ++j)
#pragma unroll
          for (int i = 0; i < kVec; ++i) {
            const float d = H::get(x.v[j], i) - top, e = ex2(d * kLog2e);
            if (d == 0.0f) ones += 1.0f;
            else beside += e;
          }
        sum += (double)ones;
        sum += (double)beside;
      } else {
        // two at a time, in fp32 for a window
        uint64_t both = pack2(odd_one, 0.0f);
        const uint64_t minus = pack2(-top, -top), scale = pack2(kLog2e, kLog2e);
#pragma unroll
        for (int j = 0; j < kN; ++j)
#pragma unroll
          for (int i = 0; i < kVec; i += 2) {
            float p, q;
            unpack2(fma2(add2(pack2(H::get(x.v[j], i), H::get(x.v[j], i + 1)), minus), scale, 0), p, q);
            both = add2(both, pack2(ex2(p), ex2(q)));
          }
        float p, q;
        unpack2(both, p, q);
        sum += (double)(p + q);
      }
    }
    // the next window's loads, before what this one has to list
    load(from + 32 * kN);
    while (hits) {
      const int j = __ffs(hits) - 1;
      hits &= hits - 1;
      uint4 u = __ldg(window + from + 32 * j);
      if (odd_ones) H::clean_vector(u);
      uint32_t which = 0;
      const float least = of_key(bound);
#pragma unroll
      for (int i = 0; i < kVec; ++i) which |= (H::get(u, i) >= least ? 1u : 0u) << i;
      while (which) {
        const int i = __ffs(which) - 1;
        which &= which - 1;
        uint32_t w = i / (kVec / 4) == 0 ? u.x : i / (kVec / 4) == 1 ? u.y : i / (kVec / 4) == 2 ? u.z : u.w;
        if (kBf16) w = i & 1 ? w & 0xFFFF0000u : w << 16;
        take_in(__uint_as_float(w), head + (from + 32 * j + lane) * kVec + i);
      }
    }
    __syncwarp();
  }
  // (the join waits for this kernel, and alone writes a call's outputs; let in at the beginning, its
  // CTAs gather on the SMs that have room first: 16 x 5 beams of 51865 in fp32 17.0 us, 13.4 so)
  griddep_launch();
  if (bad) report(a.status, CSA2_ERR_RANGE);
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(kAll, sum, d);
  if (lane == 0) a.part_sum[at] = PartSum{(float)sum, (float)(sum - (double)(float)sum), top, 0.0f};
  uint2* out = a.part_best + (int64_t)at * a.take;
  int c = counts[warp];
  __syncwarp();
  if (c <= kPartList) {
    // those that reach the last bound
    int kept = 0;
    for (int p0 = 0; p0 < c; p0 += 32) {
      const uint2 e = p0 + lane < c ? list[p0 + lane] : make_uint2(0, 0);
      const uint32_t stay = __ballot_sync(kAll, e.x >= bound);
      if (e.x >= bound) list[kept + __popc(stay & ((1u << lane) - 1))] = e;
      kept += __popc(stay);
      __syncwarp();
    }
    c = kept;
    for (int p = lane; p < c; p += 32) {
      const uint2 e = list[p];
      int rank = 0;
#pragma unroll 4
      for (int q = 0; q < c; ++q) {
        const uint2 f = list[q];
        rank += f.x > e.x || (f.x == e.x && f.y < e.y);
      }
      if (rank < a.take) out[rank] = e;
    }
    for (int p = c + lane; p < a.take; p += 32) out[p] = make_uint2(kNone, 0);
    return;
  }
  // one by one: the best behind the last, (key, place) as one number
  unsigned long long last = ~0ull;
  for (int r = 0; r < a.take; ++r) {
    unsigned long long b = 0;
    auto look = [&](float value, int place) {
      const unsigned long long e = (unsigned long long)key_of(value) << 32 | (0xffffffffu - (uint32_t)(v0 + place));
      if (e < last && e > b) b = e;
    };
    if (odd >= 0) look(alone, odd);
#pragma unroll 1
    for (int j = lane; j < vectors; j += 32) {
      uint4 u = __ldg(window - lane + j);
      H::clean_vector(u);
#pragma unroll
      for (int i = 0; i < kVec; ++i) look(H::get(u, i), head + j * kVec + i);
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) {
      const unsigned long long o = __shfl_xor_sync(kAll, b, d);
      b = o > b ? o : b;
    }
    last = b;
    if (lane == 0) out[r] = make_uint2((uint32_t)(b >> 32), 0xffffffffu - (uint32_t)b);
  }
}

// s + low times f, and the sum of two, as sums of two fp32 (Dekker, Knuth).  An addition in fp64
// takes longer here than these six.
__device__ __forceinline__ void scale2(float& s, float& low, float f) {
  const float p = __fmul_rn(s, f);
  low = fmaf(low, f, fmaf(s, f, -p)), s = p;
}
__device__ __forceinline__ void sum2(float& s, float& low, float t, float t_low) {
  const float r = __fadd_rn(s, t), u = __fsub_rn(r, s);
  const float e = __fadd_rn(__fsub_rn(s, __fsub_rn(r, u)), __fsub_rn(t, u)) + (low + t_low);
  s = __fadd_rn(r, e), low = __fsub_rn(e, __fsub_rn(s, r));
}

// Natural logarithm of h + l >= 1/2 as e log 2 + z + rest, off by 2^-28 at most (the
// library's in fp64 took 3000 cycles): h = 2^e m, m in [2/3, 4/3); log m = 2 (z + z^3 / 3 +
// z^5 / 5 ..) with z = (m - 1) / (m + 1), |z| <= 1/5, as a sum of two fp32, and what there is
// beside h.
struct Log {
  float e, z, rest;
  __device__ __forceinline__ double exact() const { return fma((double)e, 0.693147180559945309, (double)z) + (double)rest; }
};
__device__ __forceinline__ Log log_of(float h, float l) {
  const int bits = __float_as_int(h), e = (bits - 0x3F2AAAAB) >> 23;
  const float m = __int_as_float(bits - (e << 23));
  const float f = m - 1.0f, g = m + 1.0f, gl = m - (g - 1.0f);  // g + gl = m + 1
  const float z = f / g;
  const float zl = (fmaf(-z, g, f) - z * gl) / g;
  const float w = z * z;
  const float tail = z * w * fmaf(w, fmaf(w, fmaf(w, fmaf(w, fmaf(w, 1.0f / 13, 1.0f / 11), 1.0f / 9), 1.0f / 7), 1.0f / 5), 1.0f / 3);
  return Log{(float)e, 2.0f * z, 2.0f * (zl + tail) + l / h};
}

// fp64 -> unsigned in the same order (no -0 comes here).
__device__ __forceinline__ uint64_t key_of(double x) {
  const uint64_t u = (uint64_t)__double_as_longlong(x);
  return u >> 63 ? ~u : u | 1ull << 63;
}
constexpr uint64_t kNone64 = 0x000FFFFFFFFFFFFFull;  // of -inf

struct Likes {
  uint32_t marks[kMost];
  int of[kMost];  // whose sum a beam has: its own number, -1 without candidates
  uint32_t set[2][2], differ[2][2];
};
// Of the beams in `set` those whose logits are beam b's; all threads.
template <bool kBf16>
__device__ __forceinline__ uint64_t same_rows(const BeamArgs& a, int64_t row0, int b, uint64_t set, Likes& likes) {
  constexpr int kEach = 16;
  const uint8_t* first = static_cast<const uint8_t*>(a.logits);
  auto load = [&](int beam, int v0, float (&x)[kEach]) {
    const uint8_t* row = first + (row0 + beam) * a.stride * (kBf16 ? 2 : 4);
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      const int v = min(v0 + i * kThreads + (int)threadIdx.x, a.vocab - 1);
      x[i] = kBf16 ? bf16_bits_to_float(__ldg(reinterpret_cast<const uint16_t*>(row) + v)) : __ldg(reinterpret_cast<const float*>(row) + v);
    }
  };
  for (int v0 = 0, c = 0; v0 < a.vocab; v0 += kEach * kThreads, c ^= 1) {
    float x[kEach], y[kEach];
    uint64_t differ = 0;
    load(b, v0, x);
    for (uint64_t m = set; m; m &= m - 1) {
      const int k = __ffsll((long long)m) - 1;
      bool no = false;
      load(k, v0, y);
#pragma unroll
      for (int i = 0; i < kEach; ++i) no |= counts_as(x[i]) != counts_as(y[i]);
      if (no) differ |= 1ull << k;
    }
    if (differ) atomicOr(&likes.differ[c][0], (uint32_t)differ), atomicOr(&likes.differ[c][1], (uint32_t)(differ >> 32));
    __syncthreads();
    set &= ~((uint64_t)likes.differ[c][1] << 32 | likes.differ[c][0]);
    if (!set) break;
  }
  return set;
}
// Beams whose logits are the same are given the same sum, so that their scores are ties.  Rows that
// begin equally far from 16 bytes are summed alike to the last bit; this is for those that do not
// (kUneven), whose sums differ by 2^-16 at most: twice 33 additions of a window in fp32 (2^-19), and
// exponents off by 2^-23 of themselves, of which those up to log 2^30 count (2^-18.6), in the terms and
// where a larger logit rescales them.  Sums that near with the same largest logit are common (one likely
// word: 1 and a little), so the rows themselves are compared, after a mark of each part's best (key,
// token), which rarely agrees where rows differ.  All threads; `live`: beam tid has candidates.
// Where all rows are the same, 64 x 8 of 128001 in bf16 take 175 us in place of 40.8, 16 x 5 of 51865 in
// fp32 39 in place of 12.6; where sums are near and rows differ 45.4 and 15.6.
__device__ __forceinline__ bool near_sums(int b, int k, const float* sums, const float* lows, const float* most) {
  return most[b] == most[k] && fabsf((sums[b] - sums[k]) + (lows[b] - lows[k])) <= 0x1p-15f * sums[k];
}
// Whether beam tid's sum is near a lower one's; the first kMost threads.
__device__ __forceinline__ bool may_share(bool live, const float* sums, const float* lows, const float* most) {
  const int tid = threadIdx.x, lane = tid & 31;
  uint32_t same = __match_any_sync(0xffffffffu, __float_as_uint(live ? most[tid] + 0.0f : INFINITY)) & ((1u << lane) - 1);
  bool some = false;
  if (live) {
    for (; same; same &= same - 1) some |= near_sums(tid - lane + __ffs(same) - 1, tid, sums, lows, most);
    for (int b = 0; b < tid - lane; ++b) some |= near_sums(b, tid, sums, lows, most);
  }
  return some;
}
// (Not inlined, so that what is common stays small: 16 x 5 of 51865 12.9 -> 12.7 us.)
__device__ __noinline__ void share_sums(const BeamArgs& a, int64_t row0, bool live, float* sums, float* lows, const float* most,
                                           Likes& likes) {
  const int tid = threadIdx.x;
  auto near = [&](int b, int k) { return likes.of[b] == b && near_sums(b, k, sums, lows, most); };
  if (tid < kMost) likes.of[tid] = live ? tid : -1;
  {  // eight threads a beam
    const int k = tid >> 3;
    uint32_t mark = 0;
    if (k < a.beams)
      for (int p = tid & 7; p < a.parts; p += 8) {
        const uint2 e = a.part_best[((row0 + k) * a.parts + p) * a.take];
        mark += (e.x ^ __funnelshift_l(e.y, e.y, 13)) * (0x9E3779B1u * (2 * p + 1));
      }
#pragma unroll
    for (int d = 1; d < 8; d <<= 1) mark += __shfl_xor_sync(0xffffffffu, mark, d);
    if ((tid & 7) == 0) likes.marks[k] = mark;
  }
  __syncthreads();
  auto next = [&](int b) {  // the first from b on that may be beam tid's like
    while (b < tid && !(near(b, tid) && likes.marks[b] == likes.marks[tid])) ++b;
    return b < tid ? b : -1;
  };
  int like = live ? next(0) : -1;
  for (int b = 0; b < a.beams - 1; ++b) {
    if (tid < 64) {
      const uint32_t m = __ballot_sync(0xffffffffu, like == b);
      if ((tid & 31) == 0) likes.set[b & 1][tid >> 5] = m;
    } else if (tid < 68) {
      likes.differ[tid >> 1 & 1][tid & 1] = 0;
    }
    __syncthreads();
    uint64_t set = (uint64_t)likes.set[b & 1][1] << 32 | likes.set[b & 1][0];
    if (!set) continue;
    set = a.bf16 ? same_rows<true>(a, row0, b, set, likes) : same_rows<false>(a, row0, b, set, likes);
    const bool same = like == b && (set >> tid & 1);
    if (same) sums[tid] = sums[b], lows[tid] = lows[b], likes.of[tid] = b;
    __syncthreads();
    if (like == b) like = same ? -1 : next(b + 1);
  }
  __syncthreads();
}

// kUneven: a group's rows may begin differently far from 16 bytes.
template <bool kUneven>
__global__ void __launch_bounds__(kThreads, 2) beam_join_kernel(const BeamArgs a) {
  __shared__ float sums[kMost], lows[kMost];  // of exp(x - most)
  __shared__ Log logs[kMost];
  __shared__ float most[kMost], cums[kMost], logs32[kMost];
  __shared__ uint32_t best[64];
  __shared__ uint32_t bound, far, count;
  __shared__ uint64_t lkey[kList];
  __shared__ uint64_t lplace[kList];  // beam, token
  __shared__ unsigned long long wkey[kWarps], wplace[kWarps];
  griddep_wait();
  const int g = blockIdx.x, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int64_t row0 = (int64_t)g * a.beams;
  // A list is what a part has, in order; list c is beam c / parts's.  Of the lists'
  // beginnings, 64 candidates at least where there are as many, the `take`-th largest of 64
  // groups' maxima is a bound, and few candidates reach it: found in fp32, up to what that
  // may be off by, as an fp64 instruction of a warp takes an SM 16 cycles here.
  const int lists = a.beams * a.parts, depth = min(a.take, max(1, max((63 + lists) / lists, kThreads / lists))), samples = lists * depth;
  const uint2* mine = a.part_best + row0 * a.parts * a.take;
  auto score_of = [&](uint2 e, int beam) {
    // relative to the beam's largest (beside logits near fp32's lowest the rest would be
    // lost), what fp64 adds exactly first
    const double x = e.x == kDone ? 0.0 : (double)of_key(e.x) - (double)most[beam];
    return e.x <= kNone ? -(double)INFINITY : x + (double)cums[beam] - logs[beam].exact();
  };
  auto near_of = [&](uint2 e, int beam) {
    return e.x <= kNone ? -INFINITY : (e.x == kDone ? 0.0f : of_key(e.x) - most[beam]) + cums[beam] - logs32[beam];
  };
  auto beam_of = [&](int list) { return quotient(list, a.by_parts); };
  // (asked for ahead of the beams' sums; neighbouring samples in different groups)
  const int sample0 = (tid & 7) * 64 + (tid >> 3);
  uint2 raw0 = make_uint2(0, 0);
  if (sample0 < samples) raw0 = mine[(sample0 % lists) * a.take + sample0 / lists];
  float cum = tid < a.beams ? a.cum[row0 + tid] : 0.0f;
  const bool ended = kUneven && tid < a.beams && a.done && a.done[row0 + tid];
  {  // the beams' sums: eight threads a beam
    const int k = tid >> 3;
    float m = -INFINITY, s = 0.0f, low = 0.0f;
    if (k < a.beams)
      for (int p = tid & 7; p < a.parts; p += 8) {
        const PartSum e = a.part_sum[(row0 + k) * a.parts + p];
        if (e.most > m) scale2(s, low, ex2((m - e.most) * kLog2e)), m = e.most;
        if (e.most > -INFINITY) {
          float t = e.sum, t_low = e.low;
          scale2(t, t_low, ex2((e.most - m) * kLog2e));
          sum2(s, low, t, t_low);
        }
      }
    float all = m;
#pragma unroll
    for (int d = 1; d < 8; d <<= 1) all = fmaxf(all, __shfl_xor_sync(0xffffffffu, all, d));
    if (all > -INFINITY) scale2(s, low, ex2((m - all) * kLog2e));
#pragma unroll
    for (int d = 1; d < 8; d <<= 1) {
      const float t = __shfl_xor_sync(0xffffffffu, s, d), t_low = __shfl_xor_sync(0xffffffffu, low, d);
      sum2(s, low, t, t_low);
    }
    if ((tid & 7) == 0) sums[k] = s, lows[k] = low, most[k] = all;
  }
  if (tid == 0) count = 0, far = 0;
  __syncthreads();
  bool bad = false;
  cum = clean(cum, bad);
  if (bad) report(a.status, CSA2_ERR_RANGE);
  auto take_log = [&]() {
    // (as fp64 holds the sum: up to 2^-53 of it, what is beside 1 makes no difference)
    const bool some = most[tid] > -INFINITY;
    const float low = fabsf(lows[tid]) <= 0x1p-53f * sums[tid] ? 0.0f : lows[tid];
    const Log l = some ? log_of(sums[tid], low) : Log{0.0f, 0.0f, 0.0f};
    const float near = fmaf(l.e, 0.693147181f, l.z) + l.rest;
    logs[tid] = l, logs32[tid] = near;
    cums[tid] = some ? cum + 0.0f : -INFINITY;
    if (some && cum > -INFINITY) atomicMax(&far, __float_as_uint(fabsf(cum) + near + 1.0f));  // (sums are 1 at least)
  };
  if (tid < a.beams) take_log();
  if constexpr (kUneven) {
    __shared__ Likes likes;
    const bool live = tid < a.beams && !ended && cum > -INFINITY && most[tid] > -INFINITY;
    if (__syncthreads_or(tid < kMost && may_share(live, sums, lows, most))) {
      share_sums(a, row0, live, sums, lows, most, likes);
      if (tid < a.beams) take_log();
      __syncthreads();
    }
  } else {
    __syncthreads();
  }
  uint32_t top = sample0 < samples ? key_of(near_of(raw0, beam_of(sample0 % lists))) : kNone;
  for (int i = sample0 + kThreads; i < samples; i += kThreads)
    top = max(top, key_of(near_of(mine[(i % lists) * a.take + i / lists], beam_of(i % lists))));
  if (a.take <= 16) {
#pragma unroll
    for (int d = 1; d < 8; d <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, d));
    if ((tid & 7) == 0) best[tid >> 3] = top;
    __syncthreads();
    {  // eight threads rank a maximum
      const int i = tid >> 3, j0 = (tid & 7) * 8;
      int rank = 0;
#pragma unroll
      for (int j = 0; j < 8; ++j) rank += best[j0 + j] > top || (best[j0 + j] == top && j0 + j < i);
#pragma unroll
      for (int d = 1; d < 8; d <<= 1) rank += __shfl_xor_sync(0xffffffffu, rank, d);
      if ((tid & 7) == 0 && rank == a.take - 1) bound = top;
    }
    __syncthreads();
  } else {
    // (of 64 maxima the last few are weak bounds: of all threads', to 20 bits)
    uint32_t b = 0;
    for (int i = 31; i >= 12; --i)
      if (__syncthreads_count(top >= (b | 1u << i)) >= a.take) b |= 1u << i;
    if (tid == 0) bound = b;
    __syncthreads();
  }
  // Three roundings, and the logarithm's three: of terms that are no larger than the score, cum
  // and the logarithm together, each 2^-24 of it; twice, for the bound's and a candidate's.
  const float reach = of_key(bound);
  const float least = bound <= kNone ? -INFINITY : reach - 0x1p-20f * (fabsf(reach) + __uint_as_float(far));
  for (int i = sample0; i < samples; i += kThreads) {
    const int c = i % lists, b = beam_of(c);
    uint2 e = i == sample0 ? raw0 : mine[c * a.take + i / lists];
    // the last sample of a list goes on with the rest of it
    for (int r = i / lists; e.x > kNone && near_of(e, b) >= least; e = mine[c * a.take + r]) {
      const uint64_t k = key_of(score_of(e, b));
      if (k > kNone64) {
        const uint32_t p = atomicAdd(&count, 1u);
        if (p < kList) lkey[p] = k, lplace[p] = (uint64_t)b << 32 | e.y;
      }
      if (++r < depth || r == a.take) break;
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
  // (by the last warps, which have less to do in what follows)
  if (a.lse && tid >= kThreads - kMost && tid - (kThreads - kMost) < a.beams) {
    const int k = tid - (kThreads - kMost);
    a.lse[row0 + k] = most[k] > -INFINITY ? (float)((double)most[k] + logs[k].exact()) : -INFINITY;
  }
  if (n <= kList) {
    for (int p0 = 0; p0 < n; p0 += kThreads / 8) {  // eight threads rank a candidate
      const int p = p0 + (tid >> 3);
      const uint64_t k = lkey[min(p, n - 1)], e = lplace[min(p, n - 1)];
      int rank = 0;
#pragma unroll 4
      for (int q = tid & 7; q < n; q += 8) rank += (int)(lkey[q] > k) | ((int)(lkey[q] == k) & (int)(lplace[q] < e));
#pragma unroll
      for (int d = 1; d < 8; d <<= 1) rank += __shfl_xor_sync(0xffffffffu, rank, d);
      if ((tid & 7) == 0 && p < n && rank < a.take) put(rank, k, (uint32_t)(e >> 32), (uint32_t)e);
    }
    for (int r = n + tid; r < a.take; r += kThreads) none(r);
    return;
  }
  // more than the list holds have the same scores: one by one
  unsigned long long last_k = ~0ull, last_p = 0;
  for (int r = 0; r < a.take; ++r) {
    unsigned long long bk = kNone64, bp = ~0ull;  // place: the smaller first
    for (int c = tid; c < lists * a.take; c += kThreads) {
      const uint2 e = mine[c];
      const int b = beam_of(c / a.take);
      const unsigned long long k = key_of(score_of(e, b)), p = (unsigned long long)b << 32 | e.y;
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

// Parts of a row, all of like size, of 1 to most_windows() windows: those of least time, of
// which a window takes a warp 5 parts alone and 9 more with the SM full (28 warps; 1.25 and
// 2.25 us), and its start a window.  512 rows of 128001 in bf16 take 36.7 us in 8 parts,
// one wave of 27 warps an SM, and 42.9 in 9, which begin a second one.  (152 SMs by number, and
// no more partial results than most_results has, as that has to hold for every call that
// is no larger in any size.)
struct Parts {
  int n, size;
};
int windows_of(int vocab, bool bf16) { return (vocab - 1) / (kN * 32 * (bf16 ? 8 : 4)) + 1; }
int64_t most_results(int64_t rows, int vocab, int take) {
  const int64_t windows = windows_of(vocab, false);
  const int each = most_windows(take);
  return std::max(rows * ((windows + each - 1) / each), std::min<int64_t>(rows * windows, 8192));
}
Parts parts_of(int64_t rows, int vocab, int take, bool bf16) {
  constexpr int64_t kWave = 152 * 28;
  const int vec = bf16 ? 8 : 4, windows = windows_of(vocab, bf16);
  const int64_t most = most_results(rows, vocab, take);
  int n = 0;
  double least = INFINITY;
  for (int each = 1; each <= most_windows(take); ++each) {
    const int64_t parts = (windows + each - 1) / each, warps = rows * parts;
    if (warps > most) continue;
    const double time = (each + 1) * (5.0 * (double)((warps + kWave - 1) / kWave) + 9.0 * (double)warps / (double)kWave);
    if (time < least) least = time, n = (int)parts;
  }
  return {n, ((vocab - 1) / n / vec + 1) * vec};
}
bool sizes_ok(int32_t groups, int32_t beams, int32_t vocab, int32_t take) {
  return groups >= 0 && beams >= 1 && vocab >= 1 && take >= 1;
}
bool sizes_fit(int32_t groups, int32_t beams, int32_t vocab, int32_t take) {
  // (a part's end is its beginning and its size, in 32 bits)
  if (beams > kMost || take > kMost || vocab > (1 << 30) || (int64_t)groups * beams > INT32_MAX) return false;
  // (a group's lists, times take, are numbered in 32 bits too)
  return most_results((int64_t)groups * beams, vocab, take) <= INT32_MAX - kPartWarps &&
         most_results(beams, vocab, take) * take <= INT32_MAX / 2;
}
size_t sums_bytes(int64_t results) { return (size_t)((results * sizeof(PartSum) + 255) / 256 * 256); }
bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

}  // namespace
}  // namespace csa2

using namespace csa2;

extern "C" {

size_t csa2_beam_workspace_bytes(int32_t groups, int32_t beams, int32_t vocab, int32_t take) {
  if (!sizes_ok(groups, beams, vocab, take) || !sizes_fit(groups, beams, vocab, take)) return 0;
  const int64_t results = most_results((int64_t)groups * beams, vocab, take);
  return sums_bytes(results) + (size_t)(results * take) * sizeof(uint2);
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
  const int64_t rows = (int64_t)groups * beams;
  const bool bf16 = logits_dtype == CSA2_BF16;
  const Parts parts = parts_of(rows, vocab, take, bf16);
  BeamArgs a{groups, beams, vocab, take, parts.n, parts.size, divisor(parts.n), logits, stride, cum, done, end_token, scores,
             parents, tokens, lse, static_cast<PartSum*>(workspace),
             reinterpret_cast<uint2*>(static_cast<uint8_t*>(workspace) + sums_bytes(rows * parts.n)), status, bf16};
  const dim3 grid((unsigned)((rows * parts.n + kPartWarps - 1) / kPartWarps)), block(32 * kPartWarps);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e = take > 32 ? (bf16 ? launch_k(beam_part_kernel<true, true>, grid, block, 0, s, 0, a)
                                    : launch_k(beam_part_kernel<false, true>, grid, block, 0, s, 0, a))
                            : (bf16 ? launch_k(beam_part_kernel<true, false>, grid, block, 0, s, 0, a)
                                    : launch_k(beam_part_kernel<false, false>, grid, block, 0, s, 0, a));
  const bool uneven = beams > 1 && stride % (bf16 ? 8 : 4) != 0;
  if (e == cudaSuccess) e = launch_k(uneven ? beam_join_kernel<true> : beam_join_kernel<false>, dim3(groups), dim3(kThreads), 0, s, 0, a);
  return e == cudaSuccess ? CSA2_OK : CSA2_ERR_CUDA;
}

}  // extern "C"
