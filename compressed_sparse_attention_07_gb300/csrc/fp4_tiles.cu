// Projections with 4-bit weights for more than a few rows of x: tcgen05 over tiles of
// 128 rows of W x 16 .. 256 rows of x.
//
// D[128][rows of x] = W x^T accumulates in tensor memory over steps of 128 channels.  A
// step's packed weights (9 KB) come by bulk copies, its rows of x by tensor copies (two
// boxes of 64 channels, 128-byte swizzle; rows and channels outside are zeros);
// sixteen warps decode the weights, 32 of a row a lane, into the left operand's tile
// in shared memory, whose 8-row columns of 16 bytes stand 2080 bytes apart so that
// lanes of one phase write different banks; one warp issues the eight products of
// 128 x rows x 16.  Few rows are bound by the weights' bytes and their decoding, many
// by the products (256 rows: 512 cycles a step, of which decoding takes 320 issue slots
// of each scheduler).  A CTA takes tile after tile, with two accumulators, so that the
// sums of one are stored while the next is formed.  Where the tiles fill less than
// half the SMs, a cluster divides k, and its CTAs join their sums through distributed
// shared memory in rank order.
#include <cuda.h>

#include <algorithm>

#include "fp4.cuh"
#include "tc.cuh"

namespace csa2 {
namespace {

constexpr int kDecoders = 16, kWarps = 8 + kDecoders, kThreads = 32 * kWarps;
constexpr int kRows = 128;                      // of W a tile
constexpr int kStepBytes = 8 * kBlockBytes;     // packed
constexpr int kChunk = kRows * 16 + 32;         // 16 bytes of every row
constexpr int kABytes = 16 * kChunk;
constexpr int kSmemMost = 227 * 1024 - 1024;

// Places of the rings for kTok rows of x.
template <int kTok>
struct Rings {
  static constexpr int kXBytes = kTok * 2 * kBlockK;
  static constexpr int kX = kTok == 256 ? 2 : kTok == 128 ? 3 : 4;
  static constexpr int kA = kTok == 256 ? 2 : 3;
  static constexpr int kP = kTok >= 128 ? 3 : kTok == 64 ? 6 : 9;
  static constexpr int kSmem = 1024 + kX * kXBytes + kA * kABytes + kP * kStepBytes;
};

struct TileArgs {
  Fp4Linear l;
  int row_tiles, tiles;  // of W, in all
  int split;             // CTAs of a cluster that divide k
};

__device__ __forceinline__ void tensor_g2s(uint32_t dst, const CUtensorMap* map, int x, int y, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cta.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
      "l"(map), "r"(x), "r"(y), "r"(tc::smem_u32(bar))
      : "memory");
}

template <int kTok>
__global__ void __launch_bounds__(kThreads, 1) fp4_tiles_kernel(const __grid_constant__ CUtensorMap map, const TileArgs a) {
  using R = Rings<kTok>;
  extern __shared__ uint8_t raw[];
  uint8_t* smem = raw + ((1024 - (tc::smem_u32(raw) & 1023)) & 1023);
  uint8_t *xs = smem, *as = xs + R::kX * R::kXBytes, *ps = as + R::kA * kABytes;
  __shared__ __align__(8) uint64_t full_p[R::kP], empty_p[R::kP], full_x[R::kX], empty_x[R::kX], full_a[R::kA],
      empty_a[R::kA], full_d[2], empty_d[2], drained;
  __shared__ uint32_t tmem;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    for (int i = 0; i < R::kP; ++i) tc::mbar_init(&full_p[i], 1), tc::mbar_init(&empty_p[i], kDecoders);
    for (int i = 0; i < R::kX; ++i) tc::mbar_init(&full_x[i], 1), tc::mbar_init(&empty_x[i], 1);
    for (int i = 0; i < R::kA; ++i) tc::mbar_init(&full_a[i], kDecoders), tc::mbar_init(&empty_a[i], 1);
    for (int i = 0; i < 2; ++i) tc::mbar_init(&full_d[i], 1), tc::mbar_init(&empty_d[i], 4);
    tc::mbar_init(&drained, 1);
    tc::fence_mbar_init();
  }
  // a CTA's tiles: first, first + stride ..; its steps of each: [s0, s1)
  const int rank = a.split > 1 ? (int)tc::cluster_rank() : 0;
  const int first = blockIdx.x / a.split, stride = gridDim.x / a.split;
  const int s0 = (int)((int64_t)rank * a.l.k_blocks / a.split), s1 = (int)((int64_t)(rank + 1) * a.l.k_blocks / a.split);
  const int groups = (a.l.n + kBlockRows - 1) / kBlockRows;  // of 16 rows
  auto weights = [&](int tile, int step, int g) {
    return a.l.w + (((int64_t)(tile % a.row_tiles) * 8 + g) * a.l.k_blocks + step) * kBlockBytes;
  };
  if (warp == 0 && lane < 8 && first < a.tiles && first % a.row_tiles * 8 + lane < groups)
    for (int i = s0; i < min(s1, s0 + R::kP); ++i) tc::bulk_prefetch_l2(weights(first, i, lane), kBlockBytes);
  griddep_wait();  // every input may be the previous kernel's output
  if (warp == 3) {
    tc::tmem_alloc(&tmem, 2 * kTok);
    tc::tmem_relinquish();
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  bool ok = true;

  if (warp == 0) {  // packed weights
    int n = 0;
    for (int tile = first; tile < a.tiles && ok; tile += stride) {
      const int there = min(8, groups - tile % a.row_tiles * 8);
      for (int step = s0; step < s1 && ok; ++step, ++n) {
        const int s = n % R::kP;
        if (n >= R::kP) ok = __all_sync(0xffffffffu, tc::mbar_wait(&empty_p[s], ((n / R::kP) & 1) ^ 1));
        if (!ok) break;
        if (lane == 0) tc::mbar_arrive_expect_tx(&full_p[s], there * kBlockBytes);
        __syncwarp();
        if (lane < there) tc::bulk_g2s(ps + s * kStepBytes + lane * kBlockBytes, weights(tile, step, lane), kBlockBytes, &full_p[s]);
      }
    }
    // nothing may land in shared memory after the CTA has left
    for (int i = max(0, n - R::kP); i < n; ++i) tc::mbar_wait(&full_p[i % R::kP], (i / R::kP) & 1);
  } else if (warp == 1) {  // rows of x
    int n = 0;
    for (int tile = first; tile < a.tiles && ok; tile += stride) {
      const int row = tile / a.row_tiles * kTok;
      for (int step = s0; step < s1 && ok; ++step, ++n) {
        const int s = n % R::kX;
        if (n >= R::kX) ok = __all_sync(0xffffffffu, tc::mbar_wait(&empty_x[s], ((n / R::kX) & 1) ^ 1));
        if (!ok) break;
        if (lane == 0) {
          tc::mbar_arrive_expect_tx(&full_x[s], R::kXBytes);
          const uint32_t dst = tc::smem_u32(xs + s * R::kXBytes);
          tensor_g2s(dst, &map, step * kBlockK, row, &full_x[s]);
          tensor_g2s(dst + R::kXBytes / 2, &map, step * kBlockK + 64, row, &full_x[s]);
        }
        __syncwarp();
      }
    }
    for (int i = max(0, n - R::kX); i < n; ++i) tc::mbar_wait(&full_x[i % R::kX], (i / R::kX) & 1);
  } else if (warp == 2) {  // products
    constexpr uint32_t kIdesc = tc::idesc_f16(kRows, kTok, true, true, false, false);
    constexpr uint32_t kAHi = tc::sdesc_hi(128), kBHi = tc::sdesc_hi(1024) | 2u << 29;  // B: 128-byte swizzle
    int n = 0, it = 0;
    for (int tile = first; tile < a.tiles && ok; tile += stride, ++it) {
      const int d = it & 1;
      if (it >= 2) ok = __all_sync(0xffffffffu, tc::mbar_wait(&empty_d[d], ((it / 2) & 1) ^ 1));
      for (int step = s0; step < s1 && ok; ++step, ++n) {
        const int sa = n % R::kA, sx = n % R::kX;
        ok = __all_sync(0xffffffffu, tc::mbar_wait(&full_x[sx], (n / R::kX) & 1));
        ok = ok && __all_sync(0xffffffffu, tc::mbar_wait(&full_a[sa], (n / R::kA) & 1));
        if (!ok) break;
        tc::fence_after_sync();
        const uint32_t a_lo = tc::sdesc_lo(tc::smem_u32(as + sa * kABytes), kChunk);
        const uint32_t b_lo = tc::sdesc_lo(tc::smem_u32(xs + sx * R::kXBytes), 16);
        if (tc::elect_one()) {
#pragma unroll
          for (int k = 0; k < 8; ++k)
            tc::mma_ss_lo(tmem + d * kTok, a_lo + k * (2 * kChunk / 16),
                          b_lo + (k / 4) * (R::kXBytes / 2 / 16) + (k % 4) * 2, kAHi, kBHi, kIdesc, step > s0 || k > 0);
          tc::mma_commit(&empty_x[sx]);
          tc::mma_commit(&empty_a[sa]);
          if (step + 1 == s1) tc::mma_commit(&full_d[d]);
        }
        __syncwarp();
      }
    }
    if (tc::elect_one()) tc::mma_commit(&drained);
    __syncwarp();
    tc::mbar_wait(&drained, 0);
  } else if (warp >= 8) {  // decoding
    const int d = warp - 8, group = d >> 1, half = d & 1, g = lane >> 2, t = lane & 3;
    int n = 0;
    for (int tile = first; tile < a.tiles && ok; tile += stride)
      for (int step = s0; step < s1 && ok; ++step, ++n) {
        const int sp = n % R::kP, sa = n % R::kA;
        ok = __all_sync(0xffffffffu, tc::mbar_wait(&full_p[sp], (n / R::kP) & 1));
        if (!ok) break;
        const uint8_t* b = ps + sp * kStepBytes + group * kBlockBytes;
        const uint4 w = *reinterpret_cast<const uint4*>(b + half * 512 + lane * 16);
        const uint32_t sc = *reinterpret_cast<const uint32_t*>(b + kBlockCodes + lane * 4) >> (16 * half);
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&empty_p[sp]);
        if (n >= R::kA) ok = __all_sync(0xffffffffu, tc::mbar_wait(&empty_a[sa], ((n / R::kA) & 1) ^ 1));
        if (!ok) break;
        uint8_t* dst = as + sa * kABytes + d * 128 + g * 16;
        const uint32_t s[2] = {fp4_scale(sc, 0), fp4_scale(sc, 1)};
        const uint32_t words[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          uint32_t r[4];
          fp4_weights(words[j], s[j / 2], r);
          *reinterpret_cast<uint4*>(dst + (4 * t + (j ^ t)) * kChunk) = make_uint4(r[0], r[1], r[2], r[3]);
        }
        tc::fence_async_smem();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&full_a[sa]);
      }
  } else if (warp >= 4) {  // sums out: a lane has a row of W
    const int lane0 = 32 * (warp & 3);
    constexpr int kCols = kTok < 32 ? kTok : 32;
    int it = 0;
    for (int tile = first; tile < a.tiles && ok; tile += stride, ++it) {
      const int d = it & 1, i = tile % a.row_tiles * kRows + lane0 + lane, t0 = tile / a.row_tiles * kTok;
      const bool there = i < a.l.n;
      const float bias = there && rank == 0 ? fp4_bias(a.l, i) : 0.0f;
      ok = __all_sync(0xffffffffu, tc::mbar_wait(&full_d[d], (it / 2) & 1));
      if (!ok) break;
      tc::fence_after_sync();
#pragma unroll 1
      for (int c = 0; c < kTok; c += kCols) {
        uint32_t v[kCols];
        if constexpr (kCols == 32) tc::tmem_ld32(tc::taddr(tmem, lane0, d * kTok + c), v);
        else tc::tmem_ld16(tc::taddr(tmem, lane0, d * kTok + c), v);
        tc::tmem_wait_ld();
        if (a.split > 1) {  // [row of x][row of W], in the rings, which nothing fills any more
#pragma unroll
          for (int j = 0; j < kCols; ++j) reinterpret_cast<uint32_t*>(xs)[(c + j) * kRows + lane0 + lane] = v[j];
        } else if (there) {
          const int most = a.l.T - t0 - c;
          if (a.l.f32) {
            float* o = static_cast<float*>(a.l.out) + (int64_t)(t0 + c) * a.l.out_stride + i;
#pragma unroll
            for (int j = 0; j < kCols; ++j)
              if (j < most) o[j * a.l.out_stride] = fmaf(__uint_as_float(v[j]), a.l.alpha, bias);
          } else {
            __nv_bfloat16* o = static_cast<__nv_bfloat16*>(a.l.out) + (int64_t)(t0 + c) * a.l.out_stride + i;
#pragma unroll
            for (int j = 0; j < kCols; ++j)
              if (j < most) o[j * a.l.out_stride] = __float2bfloat16_rn(fmaf(__uint_as_float(v[j]), a.l.alpha, bias));
          }
        }
      }
      tc::fence_before_sync();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&empty_d[d]);
    }
  }
  if (!ok && lane == 0) report(a.l.status, CSA2_ERR_TIMEOUT);
  __syncwarp();
  __syncthreads();
  if (warp == 3) tc::tmem_dealloc(tmem, 2 * kTok);
  if (a.split > 1) {
    tc::cluster_sync();
    // this CTA's share of the tile's rows of x
    const int t0 = first / a.row_tiles * kTok, i = first % a.row_tiles * kRows + tid % kRows;
    const uint32_t mine = tc::smem_u32(xs);
    for (int t = rank + a.split * (tid / kRows); t < kTok && t0 + t < a.l.T; t += a.split * (kThreads / kRows)) {
      const uint32_t at = mine + (t * kRows + tid % kRows) * 4;
      float sum = 0.0f;
      for (int r = 0; r < a.split; ++r) sum += tc::ld_dsmem(tc::map_rank(at, r));
      if (i < a.l.n) fp4_store(a.l, t0 + t, i, sum, fp4_bias(a.l, i));
    }
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

template <int kTok>
cudaError_t launch_of(const Fp4Linear& l, cudaStream_t stream) {
  using R = Rings<kTok>;
  static_assert(R::kSmem <= kSmemMost && R::kX * R::kXBytes + R::kA * kABytes >= kTok * kRows * 4, "");
  auto kern = fp4_tiles_kernel<kTok>;
  static std::atomic<bool> done[64];
  const cudaError_t e = allow_smem(kern, R::kSmem, done);
  if (e != cudaSuccess) return e;
  const Encode encode = encoder();
  if (!encode) return cudaErrorNotSupported;
  CUtensorMap map;
  const cuuint64_t dims[2] = {(cuuint64_t)l.k, (cuuint64_t)l.T}, strides[1] = {(cuuint64_t)l.x_stride * 2};
  const cuuint32_t box[2] = {64, kTok}, unit[2] = {1, 1};
  if (encode(&map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<uint16_t*>(l.x), dims, strides, box, unit,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
    return cudaErrorInvalidValue;
  TileArgs a{l, (l.n + kRows - 1) / kRows, 0, 1};
  const int64_t tiles = (int64_t)a.row_tiles * ((l.T + kTok - 1) / kTok);
  if (tiles > INT32_MAX / 8) return cudaErrorInvalidValue;
  a.tiles = (int)tiles;
  const int sms = num_sms();
  if (2 * tiles <= sms) a.split = (int)std::max<int64_t>(1, std::min<int64_t>({8, sms / tiles, l.k_blocks}));
  const int ctas = a.split > 1 ? a.tiles * a.split : std::min(a.tiles, sms);
  return launch_k(kern, dim3(ctas), dim3(kThreads), R::kSmem, stream, a.split > 1 ? a.split : 0, map, a);
}

}  // namespace

cudaError_t launch_fp4_tiles(const Fp4Linear& l, cudaStream_t stream) {
  if (l.T <= 16) return launch_of<16>(l, stream);
  if (l.T <= 32) return launch_of<32>(l, stream);
  if (l.T <= 64) return launch_of<64>(l, stream);
  if (l.T <= 128) return launch_of<128>(l, stream);
  return launch_of<256>(l, stream);
}

}  // namespace csa2
