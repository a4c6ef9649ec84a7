// Projections with 4-bit weights for a few rows of x (single tokens, small batches).
//
// y = x W^T reads every weight once, 9/16 of a byte each, for 2 operations a row of x:
// bound by the weights' bytes.  The products run transposed, D[16 rows of W][8 rows of
// x], so that up to 8 rows of x fill a 16x8x16 instruction; the weights are decoded in
// registers, as the left operand, with about 18 instructions for 8 of a lane.  tcgen05
// has nothing to add here: its 128 rows of W would want the decoded weights in shared
// memory, for 8 columns.
// A CTA, one an SM, takes an equal run of tiles (16 or 32 rows of W over all of k), and
// its 16 warps take equal runs of the tiles' blocks laid end to end, whatever tile
// they are of: a warp streams its blocks through a ring of bulk copies of its own and
// stores the sums of whole tiles itself; pieces of tiles that several warps share
// are joined in their order through shared memory, so sums do not depend on timing.
// x stands in shared memory for the whole call.
#include <algorithm>

#include "fp4.cuh"
#include "tc.cuh"

namespace csa2 {
namespace {

constexpr int kWarps = 16, kThreads = 32 * kWarps, kMostSlots = 8;
constexpr int kSmemMost = 227 * 1024 - 2048;  // beside the barriers
// x rows stand an odd multiple of 64 bytes apart (two rows' chunks in different banks).
__host__ __device__ __forceinline__ int x_pitch(int k_blocks) { return k_blocks * 256 + 64; }

struct Shape {
  int slots;  // of a warp's ring
  int smem;
};
// (16 lg) rows a tile; slots 0: does not fit
Shape shape_of(const Fp4Linear& a, int lg) {
  const int64_t fixed = (int64_t)a.T * x_pitch(a.k_blocks) + 2 * kWarps * lg * 512;
  const int64_t ring = (int64_t)kWarps * lg * kBlockBytes;
  const int64_t n = std::min<int64_t>(kMostSlots, (kSmemMost - fixed) / ring);
  if (fixed > kSmemMost || n < 2) return {0, 0};
  return {(int)n, (int)(fixed + n * ring)};
}

__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// A lane's sums of 16 rows of W: rows g and g + 8, rows 2 t and 2 t + 1 of x.
__device__ __forceinline__ void store_group(const Fp4Linear& a, int row0, int lane, float4 d) {
  const int g = lane >> 2, t = 2 * (lane & 3);
  if (t >= a.T) return;
  const float v[4] = {d.x, d.y, d.z, d.w};
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int i = row0 + g + 8 * h;
    if (i >= a.n) return;
    const float b = fp4_bias(a, i);
    fp4_store(a, t, i, v[2 * h], b);
    if (t + 1 < a.T) fp4_store(a, t + 1, i, v[2 * h + 1], b);
  }
}

template <int kGroups>
__global__ void __launch_bounds__(kThreads, 1) fp4_rows_kernel(const Fp4Linear a, int tiles, int slots) {
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ __align__(8) uint64_t full[kWarps][kMostSlots];
  __shared__ int piece_tile[2 * kWarps];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  const int pitch = x_pitch(a.k_blocks);
  uint8_t* ring = smem + warp * slots * (kGroups * kBlockBytes);
  float4* pieces = reinterpret_cast<float4*>(smem + kWarps * slots * (kGroups * kBlockBytes));
  uint8_t* xs = reinterpret_cast<uint8_t*>(pieces + 2 * kWarps * kGroups * 32);

  const int tile0 = (int)((int64_t)blockIdx.x * tiles / gridDim.x);
  const int units = ((int)((int64_t)(blockIdx.x + 1) * tiles / gridDim.x) - tile0) * a.k_blocks;
  const int u0 = (int)((int64_t)warp * units / kWarps), u1 = (int)((int64_t)(warp + 1) * units / kWarps);
  // the next unit to fetch: its blocks, its place in k and in the ring (no division in
  // the loop: with u / k_blocks and u % slots in it a unit of 32 rows took 512
  // instructions, and takes 340)
  const int kb0 = units ? u0 % a.k_blocks : 0, first = units ? u0 / a.k_blocks : 0;
  constexpr int kParts = kTileBlocks / kGroups;  // tiles of this kernel in 128 rows
  const int64_t far = (int64_t)(a.k_blocks - 1) * kTileBytes;
  int src_tile = tile0 + first, src_kb = kb0, src_slot = 0;
  const uint8_t* src = a.w + ((int64_t)(src_tile / kParts) * a.k_blocks + kb0) * kTileBytes +
                       src_tile % kParts * (kGroups * kBlockBytes);
  auto fetch = [&]() {
    tc::mbar_arrive_expect_tx(&full[warp][src_slot], kGroups * kBlockBytes);
    tc::bulk_g2s(ring + src_slot * (kGroups * kBlockBytes), src, kGroups * kBlockBytes, &full[warp][src_slot]);
    src += kTileBytes;
    if (++src_kb == a.k_blocks) {  // the next tile's first block: beside this one's, or at the next 128 rows
      src_kb = 0, ++src_tile;
      src += kGroups * kBlockBytes - (src_tile % kParts ? far + kTileBytes : kTileBytes);
    }
    if (++src_slot == slots) src_slot = 0;
  };
  if (lane == 0) {
    if (u0 < u1) tc::bulk_prefetch_l2(src, kGroups * kBlockBytes);
    for (int s = 0; s < slots; ++s) tc::mbar_init(&full[warp][s], 1);
    tc::fence_mbar_init();
    piece_tile[2 * warp] = piece_tile[2 * warp + 1] = -1;
  }
  __syncwarp();
  griddep_wait();  // every input may be the previous kernel's output
  if (lane == 0)
    for (int u = u0; u < min(u1, u0 + slots); ++u) fetch();
  {  // x, zeros from channel k on
    const int chunks = a.k_blocks * 16;
    for (int r = 0; r < a.T; ++r)
      for (int c = tid; c < chunks; c += kThreads) {
        uint4 v = make_uint4(0, 0, 0, 0);
        if (8 * c < a.k) v = __ldg(reinterpret_cast<const uint4*>(a.x + r * a.x_stride) + c);
        *reinterpret_cast<uint4*>(xs + r * pitch + c * 16) = v;
      }
  }
  __syncthreads();
  const uint8_t* xr = xs + min(g, a.T - 1) * pitch + t * 64;  // (columns from T on are dropped)

  float acc[kGroups][4] = {};
  int kb = kb0, tile = first, piece = 0, s = 0;
  uint32_t phase = 0;
  bool whole = kb == 0, ok = true;
  for (int u = u0; u < u1; ++u) {
    tc::mbar_wait_or(&full[warp][s], phase, ok);  // (sums of what stands there, and a status, where it gives up)
    __syncwarp();
    uint4 lo[kGroups], hi[kGroups];
    uint32_t sc[kGroups];
#pragma unroll
    for (int i = 0; i < kGroups; ++i) {
      const uint8_t* b = ring + (s * kGroups + i) * kBlockBytes;
      lo[i] = *reinterpret_cast<const uint4*>(b + fp4_unit(g, t));
      hi[i] = *reinterpret_cast<const uint4*>(b + fp4_unit(g + 8, t));
      sc[i] = *reinterpret_cast<const uint32_t*>(b + kBlockCodes + 4 * lane);
    }
    __syncwarp();
    if (lane == 0 && u + slots < u1) fetch();
    if (++s == slots) s = 0, phase ^= 1;
    const uint8_t* xk = xr + kb * 256;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint4 x = *reinterpret_cast<const uint4*>(xk + (j ^ t) * 16);
#pragma unroll
      for (int i = 0; i < kGroups; ++i) {
        const uint32_t wl = j == 0 ? lo[i].x : j == 1 ? lo[i].y : j == 2 ? lo[i].z : lo[i].w;
        const uint32_t wh = j == 0 ? hi[i].x : j == 1 ? hi[i].y : j == 2 ? hi[i].z : hi[i].w;
        uint32_t l[4], h[4];
        fp4_weights(wl, fp4_scale(sc[i], j / 2), l);
        fp4_weights(wh, fp4_scale(sc[i], 2 + j / 2), h);
        mma(acc[i], l[0], h[0], l[1], h[1], x.x, x.y);
        mma(acc[i], l[2], h[2], l[3], h[3], x.z, x.w);
      }
    }
    if (++kb == a.k_blocks || u + 1 == u1) {  // the end of the tile, or of the warp's part of it
#pragma unroll
      for (int i = 0; i < kGroups; ++i) {
        const float4 d = make_float4(acc[i][0], acc[i][1], acc[i][2], acc[i][3]);
        if (whole && kb == a.k_blocks) store_group(a, ((tile0 + tile) * kGroups + i) * kBlockRows, lane, d);
        else pieces[((2 * warp + piece) * kGroups + i) * 32 + lane] = d;
        acc[i][0] = acc[i][1] = acc[i][2] = acc[i][3] = 0.0f;
      }
      if (!(whole && kb == a.k_blocks)) {
        if (lane == 0) piece_tile[2 * warp + piece] = tile;
        ++piece;
      }
      if (kb == a.k_blocks) kb = 0, ++tile;
      whole = true;
    }
  }
  if (!ok) {
    report(a.status, CSA2_ERR_TIMEOUT);
    // nothing may land in shared memory after the CTA has left
    for (int u = max(u0, u1 - slots); u < u1; ++u) tc::mbar_wait(&full[warp][(u - u0) % slots], ((u - u0) / slots) & 1);
  }
  __syncthreads();
  // a shared tile's pieces stand in the order of its channels, two places a warp: the
  // warp with the first of them joins them
  for (int p = warp; p < 2 * kWarps; p += kWarps) {
    const int at = piece_tile[p];
    if (at < 0) continue;
    bool first = true;
    for (int q = 0; q < p; ++q) first = first && piece_tile[q] != at;
    if (!first) continue;
#pragma unroll
    for (int i = 0; i < kGroups; ++i) {
      float4 d = pieces[(p * kGroups + i) * 32 + lane];
      for (int q = p + 1; q < 2 * kWarps; ++q) {
        if (piece_tile[q] != at) continue;
        const float4 e = pieces[(q * kGroups + i) * 32 + lane];
        d.x += e.x, d.y += e.y, d.z += e.z, d.w += e.w;
      }
      store_group(a, ((tile0 + at) * kGroups + i) * kBlockRows, lane, d);
    }
  }
}

template <int kGroups>
cudaError_t launch_of(const Fp4Linear& a, const Shape& s, cudaStream_t stream) {
  auto kern = fp4_rows_kernel<kGroups>;
  static std::atomic<bool> done[64];
  const cudaError_t e = allow_smem(kern, kSmemMost, done);
  if (e != cudaSuccess) return e;
  const int tiles = (a.n + 16 * kGroups - 1) / (16 * kGroups);
  return launch_k(kern, dim3((unsigned)std::min(tiles, num_sms())), dim3(kThreads), s.smem, stream, 0, a, tiles, s.slots);
}

}  // namespace

bool fp4_rows_ok(const Fp4Linear& a) { return a.T <= kFp4FewRows && shape_of(a, 1).slots != 0; }

cudaError_t launch_fp4_rows(const Fp4Linear& a, cudaStream_t stream) {
  // 32 rows a tile, which halve x's way through shared memory, where the SMs have
  // several each and the rings stay deep
  const Shape two = shape_of(a, 2);
  if (a.n >= 32 * 8 * num_sms() && two.slots >= 3) return launch_of<2>(a, two, stream);
  return launch_of<1>(a, shape_of(a, 1), stream);
}

}  // namespace csa2
