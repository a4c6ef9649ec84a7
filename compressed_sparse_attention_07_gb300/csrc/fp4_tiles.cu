// Projections with 4-bit weights for more than a few rows of x: tcgen05 over tiles of
// 128 rows of W x 16 .. 256 rows of x.
//
// D[128][rows of x] = W x^T accumulates in tensor memory over steps of 128 channels.  A
// step's packed weights (9 KB) come by one bulk copy, its rows of x by two tensor copies
// (64 channels each, 128-byte swizzle; rows and channels outside are zeros); four
// or six sets of four warps, a step each, decode the weights, a row a lane, into tensor memory,
// from where the products take their left operand; one warp issues the eight products of
// 128 x rows x 16.  Few rows are bound by the weights' bytes and their decoding, many by
// the products (256 rows: 1024 cycles a step) and shared memory beside them: x goes in and
// is read once a step, 1024 cycles at 128 bytes a cycle; with the left operand in shared
// memory too they were 1570, and took 1690.  A CTA takes tile after tile, up to 128 rows
// of x with two accumulators, so that the sums of one are stored while the next is
// formed.  Each tile of the last wave is divided among a cluster, along k, where that ends sooner
// (512 rows of 4096 -> 10240, 160 tiles: 46.6 -> 35.3 us, 40 rows of 4096 -> 20480 26.7 -> 20.2);
// its CTAs join their sums through distributed shared memory in rank order.
// The accumulator's additions cut off, so for fp32 outputs an accumulator takes 1024 channels and
// the storing warps add such sums in fp32 (kApart; launch_fp4_tiles has the figures).
// In graphs 64 rows over 128001 words take 78.5 us, 40 rows of 4096 -> 10240 14.3, 4096 rows 203 to 214 (power).
#include <cuda.h>

#include <algorithm>
#include <cmath>

#include "fp4.cuh"
#include "tc.cuh"

namespace csa2 {
namespace {

constexpr int kSmemMost = 227 * 1024 - 1024;

// Places of the rings for kTok rows of x: kS steps of decoded weights in tensor memory,
// 64 columns each beside kD accumulators; kX places of kBoxes boxes of x; kP packed steps.
// Four decoding warps, a set, have every kSets-th step (six sets where registers and columns
// allow), so a set does not see every phase of every place, and must not take the phase before the last (of the same parity) for
// the last.  Packed steps may land out of order: with kP a multiple of kSets a set sees
// every phase of its own places.  Decoded steps become free in order: a set that passed
// step n - kSets knows step n - kSets - kS to be free, hence step n - 2 kS if kS >= kSets.
// kApart: an accumulator takes kSpan steps, which the storing warps add to sums of their own.  Those stand in
// registers, kTok of a thread, so that what the CTA starts with is dealt out anew (kSplit); 64 rows leave out
// a set of decoding warps for it (over 128001 words, in sums of 2048 channels, six sets of 56 registers take
// 83.8 us, five of 64 82.4).
template <int kTok, bool kApart>
struct Rings {
  static constexpr int kSpan = kApart ? 8 : 1 << 30;
  static constexpr int kSets = kTok >= 128 ? 4 : kApart && kTok == 64 ? 5 : 6, kThreads = 32 * (8 + 4 * kSets);
  static constexpr int kD = kTok == 256 ? 1 : 2, kS = kSets;
  static constexpr int kBoxes = kTok == 256 ? 1 : 2, kX = kTok == 256 ? 5 : kSets;
  // a step's decoded weights and rows of x come and go by the same barriers: full_a, empty_a
  static constexpr bool kJoint = kTok < 256;
  static constexpr int kBoxBytes = kTok * 128, kXBytes = kBoxes * kBoxBytes;
  static constexpr int kP = kTok == 256 ? 4 : kTok == 128 ? 8 : kTok == 64 ? 2 * kSets : 18;
  static constexpr int kSmem = 1024 + kX * kXBytes + kP * kTileBytes;
  static constexpr int kA = kD * kTok;  // first column of the decoded weights
  static constexpr int kCols = 512;
  static constexpr bool kSplit = kApart && kTok >= 32;
  static constexpr int kLaunchRegs = 65536 / kThreads / 8 * 8, kIssueRegs = 40, kDecodeRegs = 64;
  static constexpr int kSumRegs = (2 + kSets) * kLaunchRegs - kIssueRegs - kSets * kDecodeRegs;
  static_assert((kSpan & (kSpan - 1)) == 0 && (!kSplit || (kSumRegs % 8 == 0 && kSumRegs <= 256 && kSumRegs > kTok)), "");
  static_assert((!kJoint || kX == kS) && kP % kSets == 0 && kS >= kSets && kA + 64 * kS <= kCols && kSmem <= kSmemMost &&
                    kX * kXBytes >= kTok * kTileRows * 4, "");
};

// A place of a ring and the parity of its next phase.
template <int kSlots>
struct Place {
  int s = 0;
  uint32_t phase = 0;
  __device__ __forceinline__ void next() {
    if (++s == kSlots) s = 0, phase ^= 1;
  }
};

// A CTA's work: `whole` tiles to itself, every gridDim.x-th; then, in a cluster, its share of the
// steps of one tile that the cluster's CTAs divide, if there is one for it.
struct TileArgs {
  Fp4Linear l;
  int row_tiles, tiles;  // of W, in all
  int size;              // CTAs of a cluster
  int whole;
  // what sums are short of (fp4_bf16's weights), where alpha times it would pass fp32's largest; else 1,
  // and l.alpha has it (a product more in every store: 40 rows of 4096 -> 10240 14.2 -> 14.9 us)
  float unit;
  Divisor by_rows, by_size;  // row_tiles, size
};
struct Run {
  int tile, s0, s1;  // steps [s0, s1)
};
constexpr int kMostCluster = 8;

__device__ __forceinline__ void tensor_g2s(uint32_t dst, const CUtensorMap* map, int x, int y, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cta.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
      "l"(map), "r"(x), "r"(y), "r"(tc::smem_u32(bar))
      : "memory");
}

__device__ __forceinline__ void put(float* o, float y) { *o = y; }
__device__ __forceinline__ void put(__nv_bfloat16* o, float y) { *o = __float2bfloat16_rn(y); }
// A lane's sums of `most` rows of x, one of each row of out.
template <typename T, int kCols>
__device__ __forceinline__ void store_columns(T* o, const uint32_t (&v)[kCols], int most, const Fp4Linear& l, float bias) {
  if (most == kCols) {
#pragma unroll
    for (int j = 0; j < kCols; ++j, o += l.out_stride) put(o, fmaf(__uint_as_float(v[j]), l.alpha, bias));
  } else {
#pragma unroll
    for (int j = 0; j < kCols; ++j, o += l.out_stride)
      if (j < most) put(o, fmaf(__uint_as_float(v[j]), l.alpha, bias));
  }
}

template <int N>
__device__ __forceinline__ void regs_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

template <int kI>
struct Number {
  __device__ constexpr int operator()() const { return kI; }
};

// A value that is the same in all lanes, in a register that is known to be.  What a run's loops
// of copies and products start from goes through it: found a lane in its own register, 64 rows
// over 128001 words took 82.0 us instead of 79.0, 300 rows of 8192 -> 8192 46.4 instead of 44.2.
__device__ __forceinline__ uint32_t uniform(uint32_t v) { return __reduce_max_sync(0xffffffffu, v); }

template <int kTok, bool kApart>
__global__ void __launch_bounds__(Rings<kTok, kApart>::kThreads, 1) fp4_tiles_kernel(const __grid_constant__ CUtensorMap map, const TileArgs a) {
  using R = Rings<kTok, kApart>;
  extern __shared__ uint8_t raw[];
  uint8_t* smem = raw + ((1024 - (tc::smem_u32(raw) & 1023)) & 1023);
  uint8_t *xs = smem, *ps = xs + R::kX * R::kXBytes;
  __shared__ __align__(8) uint64_t full_p[R::kP], empty_p[R::kP], full_x[R::kX], empty_x[R::kX], full_a[R::kS],
      empty_a[R::kS], full_d[R::kD], empty_d[R::kD], drained;
  __shared__ uint32_t tmem;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    for (int i = 0; i < R::kP; ++i) tc::mbar_init(&full_p[i], 1), tc::mbar_init(&empty_p[i], 4);
    for (int i = 0; i < R::kX; ++i) tc::mbar_init(&full_x[i], 1), tc::mbar_init(&empty_x[i], 1);
    for (int i = 0; i < R::kS; ++i) tc::mbar_init(&full_a[i], R::kJoint ? 5 : 4), tc::mbar_init(&empty_a[i], 1);
    for (int i = 0; i < R::kD; ++i) tc::mbar_init(&full_d[i], 1), tc::mbar_init(&empty_d[i], 4);
    tc::mbar_init(&drained, 1);
    tc::fence_mbar_init();
  }
  const int k_blocks = a.l.k_blocks, rank = a.size > 1 ? (int)tc::cluster_rank() : 0;
  const int wholes = a.whole + (a.size == 1 && (int)blockIdx.x < a.tiles - a.whole * (int)gridDim.x ? 1 : 0);
  const int divided = a.whole * (int)gridDim.x + quotient(blockIdx.x, a.by_size);  // the cluster's tile
  const bool shares = a.size > 1 && divided < a.tiles;
  const int p0 = shares ? quotient(rank * k_blocks, a.by_size) : 0, p1 = shares ? quotient((rank + 1) * k_blocks, a.by_size) : 0;
  const int runs = wholes + (shares ? 1 : 0);
  auto run_of = [&](int i) {
    return i < wholes ? Run{(int)(blockIdx.x + i * gridDim.x), 0, k_blocks} : Run{divided, p0, p1};
  };
  auto x_tile = [&](int tile) { return quotient(tile, a.by_rows); };
  auto w_tile = [&](int tile) { return tile - quotient(tile, a.by_rows) * a.row_tiles; };
  auto weights = [&](int tile) { return a.l.w + (int64_t)w_tile(tile) * k_blocks * kTileBytes; };
  // blocks of 16 rows that a tile has (what it decodes beyond them is not stored)
  auto blocks = [&](int tile) { return min(kTileBlocks, (a.l.n + kBlockRows - 1) / kBlockRows - w_tile(tile) * kTileBlocks); };
  if (tid == 0) {
    const Run r = run_of(0);
    tc::bulk_prefetch_l2(weights(r.tile) + (int64_t)r.s0 * kTileBytes, min(R::kP, r.s1 - r.s0) * kTileBytes);
  }
  griddep_wait();  // every input may be the previous kernel's output
  if (warp == 3) {
    tc::tmem_alloc(&tmem, R::kCols);
    tc::tmem_relinquish();
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  // Every wait gives up after a second; its thread then goes on with what is there (all
  // addresses stay inside the rings), but starts no copy, and reports.
  bool ok = true;

  // (Warps that issue copies or products stay together, and one lane issues.)
  auto copy_weights = [&]() {
    int n = 0;
    Place<R::kP> at;
    for (int i = 0; i < runs && ok; ++i) {
      const Run r = run_of(i);
      const uint64_t first = reinterpret_cast<uint64_t>(weights(r.tile) + (int64_t)r.s0 * kTileBytes);
      const uint8_t* src = reinterpret_cast<const uint8_t*>((uint64_t)uniform((uint32_t)(first >> 32)) << 32 | uniform((uint32_t)first));
      const int bytes = (int)uniform(blocks(r.tile) * kBlockBytes), steps = (int)uniform(r.s1 - r.s0);
      for (int step = 0; step < steps; ++step, ++n, at.next(), src += kTileBytes) {
        if (n >= R::kP) tc::mbar_wait_or(&empty_p[at.s], at.phase ^ 1, ok);
        if (!__all_sync(0xffffffffu, ok)) break;
        if (tc::elect_one()) {
          tc::mbar_arrive_expect_tx(&full_p[at.s], bytes);
          tc::bulk_g2s(ps + at.s * kTileBytes, src, bytes, &full_p[at.s]);
        }
        __syncwarp();
      }
      ok = __all_sync(0xffffffffu, ok);  // (a wait may run out for some lanes alone; voted on in each step, 64 rows 2 % slower)
    }
    // nothing may land in shared memory after the CTA has left
    for (int i = max(0, n - R::kP); i < n && tc::mbar_wait(&full_p[i % R::kP], (i / R::kP) & 1); ++i) {}
  };
  auto copy_rows = [&]() {
    int n = 0;
    Place<R::kX> at;
    uint64_t *const full = R::kJoint ? full_a : full_x, *const empty = R::kJoint ? empty_a : empty_x;
    for (int i = 0; i < runs && ok; ++i) {
      const Run r = run_of(i);
      const int row = (int)uniform(x_tile(r.tile) * kTok), end = (int)uniform(2 * r.s1);
      for (int box = (int)uniform(2 * r.s0); box < end; box += R::kBoxes, ++n, at.next()) {
        if (n >= R::kX) tc::mbar_wait_or(&empty[at.s], at.phase ^ 1, ok);
        if (!__all_sync(0xffffffffu, ok)) break;
        if (tc::elect_one()) {
          tc::mbar_arrive_expect_tx(&full[at.s], R::kXBytes);
#pragma unroll
          for (int i = 0; i < R::kBoxes; ++i)
            tensor_g2s(tc::smem_u32(xs + at.s * R::kXBytes + i * R::kBoxBytes), &map, (box + i) * 64, row, &full[at.s]);
        }
        __syncwarp();
      }
      ok = __all_sync(0xffffffffu, ok);  // (a wait may run out for some lanes alone; voted on in each step, 64 rows 2 % slower)
    }
    for (int i = max(0, n - R::kX); i < n && tc::mbar_wait(&full[i % R::kX], (i / R::kX) & 1); ++i) {}
  };
  auto products = [&]() {
    constexpr uint32_t kIdesc = tc::idesc_f16(kTileRows, kTok, true, true, false, false);
    constexpr uint32_t kHi = tc::sdesc_hi(1024) | 2u << 29;  // 128-byte swizzle
    const uint32_t tb = uniform(tmem), x_lo = uniform(tc::sdesc_lo(tc::smem_u32(xs), 16));
    Place<R::kS> pa;
    Place<R::kX> px;
    Place<R::kD> pd;
    int sums = 0;  // begun so far
    for (int i = 0; i < runs; ++i, ++sums, pd.next()) {
      const Run run = run_of(i);
      const int steps = (int)uniform(run.s1 - run.s0);
      if ((kApart ? sums : i) >= R::kD) tc::mbar_wait_or(&empty_d[pd.s], pd.phase ^ 1, ok);
      if constexpr (R::kJoint) {
        // two steps at a time where there are two
        for (int step = 0; step < steps; step += 2) {
          const bool two = step + 1 < steps, fresh = kApart ? (step & (R::kSpan - 1)) == 0 : step == 0;
          if (kApart && fresh && step > 0) {  // the next accumulator
            if (tc::elect_one()) tc::mma_commit(&full_d[pd.s]);
            __syncwarp();
            pd.next();
            if (++sums >= R::kD) tc::mbar_wait_or(&empty_d[pd.s], pd.phase ^ 1, ok);
          }
          const int s = pa.s;
          tc::mbar_wait_or(&full_a[s], pa.phase, ok);
          pa.next();
          const int s2 = pa.s;
          if (two) {
            tc::mbar_wait_or(&full_a[s2], pa.phase, ok);
            pa.next();
          }
          __syncwarp();
          tc::fence_after_sync();
          if (tc::elect_one()) {
#pragma unroll
            for (int k = 0; k < 8; ++k)
              tc::mma_ts_lo(tb + pd.s * kTok, tb + R::kA + 64 * s + 8 * k,
                            x_lo + s * (R::kXBytes / 16) + (k / 4) * (R::kBoxBytes / 16) + (k % 4) * 2, kHi, kIdesc,
                            k > 0 || !fresh);
            tc::mma_commit(&empty_a[s]);
            if (two) {
#pragma unroll
              for (int k = 0; k < 8; ++k)
                tc::mma_ts_lo(tb + pd.s * kTok, tb + R::kA + 64 * s2 + 8 * k,
                              x_lo + s2 * (R::kXBytes / 16) + (k / 4) * (R::kBoxBytes / 16) + (k % 4) * 2, kHi, kIdesc, 1);
              tc::mma_commit(&empty_a[s2]);
            }
          }
          __syncwarp();
        }
      } else {
        for (int step = 0; step < steps; ++step, pa.next()) {
          tc::mbar_wait_or(&full_a[pa.s], pa.phase, ok);
#pragma unroll
          for (int half = 0; half < 2; ++half, px.next()) {
            tc::mbar_wait_or(&full_x[px.s], px.phase, ok);
            __syncwarp();
            tc::fence_after_sync();
            if (tc::elect_one()) {
#pragma unroll
              for (int k = 0; k < 4; ++k)
                tc::mma_ts_lo(tb + pd.s * kTok, tb + R::kA + 64 * pa.s + 8 * (4 * half + k),
                              x_lo + px.s * (R::kXBytes / 16) + k * 2, kHi, kIdesc, half > 0 || k > 0 || step > 0);
              tc::mma_commit(&empty_x[px.s]);
              if (half == 1) tc::mma_commit(&empty_a[pa.s]);
            }
            __syncwarp();
          }
        }
      }
      if (tc::elect_one()) tc::mma_commit(&full_d[pd.s]);
      __syncwarp();
    }
    if (tc::elect_one()) tc::mma_commit(&drained);
    __syncwarp();
    tc::mbar_wait(&drained, 0);
  };
  auto decode_steps = [&]() {
    const int set = (warp - 8) >> 2, q = warp & 3, r = lane & 15;  // rows 32 q .. of every kSets-th step
    const uint8_t* const src = ps + (2 * q + (lane >> 4)) * kBlockBytes;
    const uint32_t dst0 = tc::taddr(tmem, 32 * q, R::kA);
    const int mine = wholes * k_blocks + p1 - p0;  // steps of all runs
    int p = set % R::kP, s = set % R::kS;
    uint32_t p_phase = 0, s_phase = set / R::kS & 1;
    for (int n = set; n < mine; n += R::kSets) {
      tc::mbar_wait_or(&full_p[p], p_phase, ok);
      __syncwarp();
      const uint8_t* b = src + p * kTileBytes;
      uint4 u[4];
#pragma unroll
      for (int t = 0; t < 4; ++t) u[t] = *reinterpret_cast<const uint4*>(b + fp4_unit(r, t));
      const uint4 sc = *reinterpret_cast<const uint4*>(b + kBlockCodes + (r & 7) * 16);
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&empty_p[p]);
      const uint32_t scales[4] = {sc.x, sc.y, sc.z, sc.w};
      const uint32_t dst = dst0 + 64 * s;
      auto decode = [&](auto t, uint32_t (&c)[16]) {
        const uint32_t words[4] = {u[t()].x, u[t()].y, u[t()].z, u[t()].w};
        const uint32_t two = scales[t()] >> (r & 8 ? 16 : 0);
        const uint32_t f[2] = {fp4_scale(two, 0), fp4_scale(two, 1)};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint32_t v[4];
          fp4_bf16(words[i], f[i / 2], v);
#pragma unroll
          for (int j = 0; j < 4; ++j) c[(i ^ t()) * 4 + j] = v[j];
        }
      };
      // a unit or two ahead of the wait, so that a place is not held while they are decoded
      uint32_t c0[16], c1[16];
      decode(Number<0>(), c0);
      if constexpr (R::kSets == 4) decode(Number<1>(), c1);
      if (n >= R::kS) tc::mbar_wait_or(&empty_a[s], s_phase ^ 1, ok);
      __syncwarp();
      tc::fence_after_sync();
      tc::tmem_st16(dst, c0);
      if constexpr (R::kSets != 4) decode(Number<1>(), c1);
      tc::tmem_st16(dst + 16, c1);
      decode(Number<2>(), c0);
      tc::tmem_st16(dst + 32, c0);
      decode(Number<3>(), c1);
      tc::tmem_st16(dst + 48, c1);
      tc::tmem_wait_st();
      tc::fence_before_sync();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&full_a[s]);
      if ((p += R::kSets) >= R::kP) p -= R::kP, p_phase ^= 1;
      if ((s += R::kSets) >= R::kS) s -= R::kS, s_phase ^= 1;
    }
  };
  auto store_sums = [&]() {  // a lane has a row of W
    const int lane0 = 32 * (warp & 3);
    constexpr int kCols = kApart ? (kTok < 32 || kTok == 128 ? 16 : 32) : kTok < 32 ? kTok : 32;
    Place<R::kD> at;
    for (int n = 0; n < runs; ++n) {
      const int tile = run_of(n).tile;
      const int i = w_tile(tile) * kTileRows + lane0 + lane, t0 = x_tile(tile) * kTok;
      const bool there = i < a.l.n;
      const float bias = there ? fp4_bias(a.l, i) : 0.0f;
      if constexpr (kApart) {
        // (the last run: nothing fills x's ring or reads it any more)
        uint32_t* const piece = n < wholes ? nullptr : reinterpret_cast<uint32_t*>(xs);
        float sum[kTok / kCols][kCols] = {};
        const Run run = run_of(n);
        for (int left = run.s1 - run.s0; left > 0; left -= R::kSpan, at.next()) {
          tc::mbar_wait_or(&full_d[at.s], at.phase, ok);
          __syncwarp();
          tc::fence_after_sync();
#pragma unroll
          for (int c = 0; c < kTok / kCols; ++c) {
            uint32_t v[kCols];
            if constexpr (kCols == 32) tc::tmem_ld32(tc::taddr(tmem, lane0, at.s * kTok + c * kCols), v);
            else tc::tmem_ld_n<kCols>(tc::taddr(tmem, lane0, at.s * kTok + c * kCols), v);
            tc::tmem_wait_ld();
#pragma unroll
            for (int j = 0; j < kCols; ++j) sum[c][j] += __uint_as_float(v[j]);
          }
          tc::fence_before_sync();
          __syncwarp();
          if (lane == 0) tc::mbar_arrive(&empty_d[at.s]);
        }
#pragma unroll
        for (int c = 0; c < kTok; c += kCols) {
          uint32_t v[kCols];
#pragma unroll
          for (int j = 0; j < kCols; ++j) v[j] = __float_as_uint(sum[c / kCols][j]);
          if (a.unit != 1.0f) {
#pragma unroll
            for (int j = 0; j < kCols; ++j) v[j] = __float_as_uint(__uint_as_float(v[j]) * a.unit);
          }
          if (piece) {  // [row of x][row of W]
#pragma unroll
            for (int j = 0; j < kCols; ++j) piece[(c + j) * kTileRows + lane0 + lane] = v[j];
          } else if (there) {
            const int most = min(kCols, a.l.T - t0 - c);
            const int64_t at0 = (int64_t)(t0 + c) * a.l.out_stride + i;
            if (a.l.f32) store_columns(static_cast<float*>(a.l.out) + at0, v, most, a.l, bias);
            else store_columns(static_cast<__nv_bfloat16*>(a.l.out) + at0, v, most, a.l, bias);
          }
        }
      } else {
        tc::mbar_wait_or(&full_d[at.s], at.phase, ok);
        // (the last run: nothing fills x's ring or reads it any more)
        uint32_t* const piece = n < wholes ? nullptr : reinterpret_cast<uint32_t*>(xs);
        __syncwarp();
        tc::fence_after_sync();
#pragma unroll 1
        for (int c = 0; c < kTok; c += kCols) {
          uint32_t v[kCols];
          __syncwarp();
          if constexpr (kCols == 32) tc::tmem_ld32(tc::taddr(tmem, lane0, at.s * kTok + c), v);
          else tc::tmem_ld16(tc::taddr(tmem, lane0, at.s * kTok + c), v);
          tc::tmem_wait_ld();
          if (piece) {  // [row of x][row of W]
#pragma unroll
            for (int j = 0; j < kCols; ++j) piece[(c + j) * kTileRows + lane0 + lane] = v[j];
          } else if (there) {
            const int most = min(kCols, a.l.T - t0 - c);
            const int64_t at0 = (int64_t)(t0 + c) * a.l.out_stride + i;
            if (a.l.f32) store_columns(static_cast<float*>(a.l.out) + at0, v, most, a.l, bias);
            else store_columns(static_cast<__nv_bfloat16*>(a.l.out) + at0, v, most, a.l, bias);
          }
        }
        __syncwarp();
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&empty_d[at.s]);
        at.next();
      }
    }
  };
  // (kSplit: the issuing warps under one condition, as what they run is then fitted to their registers.
  // The order counts: 1024 rows of 4096 -> 10240 take 59.1 us with the issuing warps first, 58.1 so,
  // and where sums are held 128 rows 18.8 with them first, 19.8 with the others)
  if constexpr (R::kSplit) {
    if (warp < 4) {
      regs_dec<R::kIssueRegs>();
      if (warp == 0) copy_weights();
      else if (warp == 1) copy_rows();
      else if (warp == 2) products();
    } else if (warp < 8) {
      regs_inc<R::kSumRegs>();
      store_sums();
    } else {
      if constexpr (R::kDecodeRegs < R::kLaunchRegs) regs_dec<R::kDecodeRegs>();
      decode_steps();
    }
  } else {
    if (warp >= 8) decode_steps();
    else if (warp >= 4) store_sums();
    else if (warp == 0) copy_weights();
    else if (warp == 1) copy_rows();
    else if (warp == 2) products();
  }
  if (!ok) report(a.l.status, CSA2_ERR_TIMEOUT);
  __syncwarp();
  __syncthreads();
  if (warp == 3) tc::tmem_dealloc(tmem, R::kCols);
  if (a.size > 1) {
    tc::cluster_sync();
    // this CTA's share of the divided tile's rows of x
    const int t0 = x_tile(divided) * kTok, i = w_tile(divided) * kTileRows + tid % kTileRows;
    const uint32_t mine = tc::smem_u32(xs);
    if (shares && i < a.l.n) {
      const float bias = fp4_bias(a.l, i);
      for (int t = rank + a.size * (tid / kTileRows); t < kTok && t0 + t < a.l.T; t += a.size * (R::kThreads / kTileRows)) {
        const uint32_t at = mine + (t * kTileRows + tid % kTileRows) * 4;
        float v[kMostCluster], sum = 0.0f;
#pragma unroll
        for (int r = 0; r < kMostCluster; ++r) v[r] = r < a.size ? tc::ld_dsmem(tc::map_rank(at, r)) : 0.0f;
#pragma unroll
        for (int r = 0; r < kMostCluster; ++r) sum += v[r];
        fp4_store(a.l, t0 + t, i, sum, a.l.alpha, bias);
      }
    }
    __syncwarp();
    tc::cluster_sync();
  }
}

using Encode = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                            const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                            CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
Encode encoder() {
  static std::atomic<Encode> known{nullptr};
  Encode f = known.load(std::memory_order_acquire);
  if (f) return f;
  void* p = nullptr;
  cudaDriverEntryPointQueryResult r;
  if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &r) != cudaSuccess ||
      r != cudaDriverEntryPointSuccess)
    return nullptr;
  f = reinterpret_cast<Encode>(p);
  known.store(f, std::memory_order_release);
  return f;
}

// Clusters of c CTAs that the device runs at once.
template <int kTok, bool kApart>
int clusters_of(int c) {
  using R = Rings<kTok, kApart>;
  static std::atomic<int> known[64][kMostCluster + 1];  // and 1
  int device = 0;
  if (cudaGetDevice(&device) != cudaSuccess || device < 0 || device >= 64) return 0;
  int n = known[device][c].load(std::memory_order_relaxed);
  if (n) return n - 1;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr = {};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = c, attr.val.clusterDim.y = 1, attr.val.clusterDim.z = 1;
  cfg.gridDim = dim3(c), cfg.blockDim = dim3(R::kThreads), cfg.dynamicSmemBytes = R::kSmem;
  cfg.attrs = &attr, cfg.numAttrs = 1;
  if (cudaOccupancyMaxActiveClusters(&n, fp4_tiles_kernel<kTok, kApart>, &cfg) != cudaSuccess) {
    (void)cudaGetLastError();
    n = 0;
  }
  n = std::min(n, num_sms() / c);
  known[device][c].store(n + 1, std::memory_order_relaxed);
  return n;
}

template <int kTok, bool kApart>
cudaError_t launch_of(const Fp4Linear& l, cudaStream_t stream) {
  using R = Rings<kTok, kApart>;
  auto kern = fp4_tiles_kernel<kTok, kApart>;
  static std::atomic<bool> done[64];
  const cudaError_t e = allow_smem(kern, R::kSmem, done);
  if (e != cudaSuccess) return e;
  if constexpr (R::kSplit) {  // (shares beyond what the CTA starts with would be waited for without end)
    static std::atomic<int> regs{0};
    if (!regs.load(std::memory_order_relaxed)) {
      cudaFuncAttributes at;
      const cudaError_t e = cudaFuncGetAttributes(&at, kern);
      if (e != cudaSuccess) return e;
      regs.store(at.numRegs, std::memory_order_relaxed);
    }
    if ((regs.load(std::memory_order_relaxed) + 7) / 8 * 8 < R::kLaunchRegs) return cudaErrorInvalidConfiguration;
  }
  const Encode encode = encoder();
  if (!encode) return cudaErrorNotSupported;
  CUtensorMap map;
  const cuuint64_t dims[2] = {(cuuint64_t)l.k, (cuuint64_t)l.T}, strides[1] = {(cuuint64_t)(l.T > 1 ? l.x_stride : l.k) * 2};
  const cuuint32_t box[2] = {64, kTok}, unit[2] = {1, 1};
  if (encode(&map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<uint16_t*>(l.x), dims, strides, box, unit,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
    return cudaErrorInvalidValue;
  TileArgs a{l, fp4_row_tiles(l.n), 0, 1, 0, 1.0f, {}, {}};
  if (std::isfinite(l.alpha * kFp4Unit)) a.l.alpha *= kFp4Unit;
  else a.unit = kFp4Unit;
  const int64_t tiles = (int64_t)a.row_tiles * ((l.T + kTok - 1) / kTok);
  if (tiles > INT32_MAX / 8) return cudaErrorInvalidValue;
  a.tiles = (int)tiles;
  // Whole tiles as long as every CTA has one; a cluster divides each tile of the last wave where that
  // ends sooner by a tenth, in steps, of which the join of so many sums takes about kJoin.
  constexpr int kJoin = kTok / 8 < 12 ? kTok / 8 : 12;
  const int sms = num_sms();
  int ctas = std::min(a.tiles, sms);
  int64_t least = (int64_t)((a.tiles + sms - 1) / sms) * l.k_blocks * 10 / 11;
  for (int c = 2; c <= std::min(kMostCluster, l.k_blocks); ++c) {
    const int n = clusters_of<kTok, kApart>(c), whole = n ? a.tiles / (n * c) : 0, rest = n ? a.tiles % (n * c) : 0;
    const int64_t steps = (int64_t)whole * l.k_blocks + (l.k_blocks + c - 1) / c + kJoin;
    if (rest == 0 || rest > n || steps > least) continue;
    least = steps, a.size = c, a.whole = whole, ctas = (whole ? n : rest) * c;
  }
  if (a.size == 1) a.whole = a.tiles / ctas;
  a.by_rows = divisor(a.row_tiles), a.by_size = divisor(a.size);
  return launch_k(kern, dim3(ctas), dim3(R::kThreads), R::kSmem, stream, a.size > 1 ? a.size : 0, map, a);
}

}  // namespace

cudaError_t launch_fp4_tiles(const Fp4Linear& l, cudaStream_t stream) {
  // The accumulator's additions cut off: what it sums over 1024 channels is 1.9e-7 of its norm off for
  // normal weights (a plain product in fp32: 2e-7) and 4.2e-7 for codes drawn evenly, over 4096 9.6e-7 and
  // 2.0e-6, over 16384 6.2e-6.  fp32 outputs are therefore summed 1024 channels at a time (17 rows of 4096 ->
  // 10240 13.7 -> 14.4 us, 40 14.4 -> 15.2, 64 over 128001 words 78.2 -> 82.8, 128 rows 17.3 -> 18.8); beyond 128
  // rows, where that takes the narrower tile, from 4096 channels on (1024 rows 58.5 us, 73 so; 256 rows of
  // 16384 -> 4096 28.7 -> 35.0).  bf16 outputs, rounded by 2^-9 and more, from 32768 on.
  const int most = !l.f32 ? 256 : l.T > 128 ? 32 : 8;
  if (l.k_blocks > most || !std::isfinite(l.alpha * kFp4Unit)) {
    if (l.T <= 16) return launch_of<16, true>(l, stream);
    if (l.T <= 32) return launch_of<32, true>(l, stream);
    if (l.T <= 64) return launch_of<64, true>(l, stream);
    return launch_of<128, true>(l, stream);
  }
  if (l.T <= 16) return launch_of<16, false>(l, stream);
  if (l.T <= 32) return launch_of<32, false>(l, stream);
  if (l.T <= 64) return launch_of<64, false>(l, stream);
  if (l.T <= 128) return launch_of<128, false>(l, stream);
  return launch_of<256, false>(l, stream);
}

}  // namespace csa2
