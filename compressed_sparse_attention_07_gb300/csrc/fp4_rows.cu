// Projections with 4-bit weights for a few rows of x (single tokens, small batches).
//
// y = x W^T reads every weight once, 9/16 of a byte each, for 2 operations a row of x:
// bound by the weights' bytes.  The products run transposed, D[16 rows of W][8 rows of
// x], so that few rows of x fill a 16x8x16 instruction; the weights are decoded to f16 in
// registers, as the left operand.  (To bf16, which x would not have to be brought
// from, decoding bound the kernel: 8 rows of 4096 -> 128001 took 65 us.)  tcgen05
// has nothing to add here: its 128 rows of W would want the decoded weights in tensor
// memory, for 8 or 16 columns.
// A CTA, one an SM, takes an equal run of tiles (16 or 32 rows of W over all of k), and
// its 16 warps take equal runs of the tiles' blocks laid end to end, whatever tile
// they are of: a warp streams its blocks through a ring of bulk copies of its own and
// stores the sums of whole tiles itself; pieces of tiles that several warps share
// are joined in their order through shared memory, so sums do not depend on timing.
// x stands in shared memory for the whole call, as f16 relative to a power of two of its
// row that brings the row's largest to [2^14, 2^15): exact down to 2^-31 of the largest,
// and off by 2^-39 of it at most below.
// In graphs 8 rows over 128001 words of 4096 channels take 50.9 us, 87 % of measured bandwidth; 16
// rows 74 us, bound by issue; 1 row of 1280 -> 4096 4.5 us.
#include <algorithm>

#include "fp4.cuh"
#include "tc.cuh"

namespace csa2 {
namespace {

constexpr int kWarps = 16, kThreads = 32 * kWarps, kMostSlots = 8;
constexpr int kSmemMost = 224 * 1024;  // beside the barriers
// x rows stand an odd multiple of 64 bytes apart (two rows' chunks in different banks).
__host__ __device__ __forceinline__ int x_pitch(int k_blocks) { return k_blocks * 256 + 64; }

struct Shape {
  int slots;  // of a warp's ring
  int smem;
};
// groups x 16 rows of W a tile; slots 0: does not fit
Shape shape_of(const Fp4Linear& a, int groups) {
  const int64_t fixed = (int64_t)a.T * x_pitch(a.k_blocks) + (int64_t)kWarps * groups * 512 * ((a.T + 7) / 8);
  const int64_t ring = (int64_t)kWarps * groups * kBlockBytes;
  const int64_t n = std::min<int64_t>(kMostSlots, (kSmemMost - fixed) / ring);
  if (fixed > kSmemMost || n < 2) return {0, 0};
  return {(int)n, (int)(fixed + n * ring)};
}

__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// A lane's sums of 16 rows of W: rows g and g + 8, rows t and t + 1 of x; what of them is there.
__device__ __forceinline__ void store_group(const Fp4Linear& a, int row0, int t, const float* unscale, float4 d) {
  const float v[4] = {d.x, d.y, d.z, d.w};
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    if (t + c >= a.T) return;
    // the smaller factor first: what fp32 holds in the end is not lost on the way
    const float u = unscale[t + c], first = u > 1.0f ? a.alpha : u, second = u > 1.0f ? u : a.alpha;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int i = row0 + 8 * h;
      if (i < a.n) fp4_store(a, t + c, i, v[2 * h + c] * first, second, fp4_bias(a, i));
    }
  }
}

// x into shared memory as f16 in the order of channels that fp4_f16 has, zeros from channel k
// on, all threads: a power of two of warps for each row, whose largest it takes first.
// `then` is called once the first loads are on their way (behind the rings' copies they took
// up to 3000 cycles more).
template <int kBatch, typename Then>
__device__ __forceinline__ void stage_x(const Fp4Linear& a, uint8_t* xs, int pitch, uint32_t* most, float* unscale, Then then) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, chunks = a.k / 8, all = a.k_blocks * 16;
  const int share = a.T <= 1 ? 16 : a.T <= 2 ? 8 : a.T <= 4 ? 4 : a.T <= 8 ? 2 : 1;
  const int r = warp / share, first = (warp & (share - 1)) * 32 + lane, step = share * 32;
  uint8_t* row = xs + r * pitch;
  const uint4* src = reinterpret_cast<const uint4*>(a.x + r * a.x_stride);
  uint4 v[kBatch];
  auto load = [&](int c0) {
#pragma unroll
    for (int i = 0; i < kBatch; ++i)
      v[i] = r < a.T && c0 + i * step < chunks ? __ldg(src + c0 + i * step) : make_uint4(0, 0, 0, 0);
  };
  load(first);
  __syncthreads();
  then();
  if (r < a.T) {
    uint32_t m = 0;  // largest magnitudes, as bf16 bits, two at a time
    for (int c0 = first; c0 < all; c0 += kBatch * step) {
      if (c0 != first) load(c0);
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
        for (int j = 0; j < 4; ++j) m = __vmaxu2(m, w[j] & 0x7FFF7FFFu);
        if (c0 + i * step < all) *reinterpret_cast<uint4*>(row + (c0 + i * step) * 16) = v[i];
      }
    }
    m = max(m & 0xFFFFu, m >> 16);
    if (__any_sync(0xffffffffu, m >= 0x7F80u)) {  // the largest finite one
      m = 0;
      for (int c = first; c < chunks; c += step) {
        const uint4 v = *reinterpret_cast<const uint4*>(row + c * 16);
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
        for (int j = 0; j < 8; ++j) {
          const uint32_t h = (w[j / 2] >> (j & 1 ? 16 : 0)) & 0x7FFFu;
          if (h < 0x7F80u) m = max(m, h);
        }
      }
    }
    m = __reduce_max_sync(0xffffffffu, m);
    if (lane == 0) atomicMax(&most[r], m);
  }
  __syncthreads();
  if (r < a.T) {
    // 2^e brings the largest, of exponent field f, to [2^14, 2^15)
    const uint32_t m = most[r];
    const int e = m ? min(14 + 127 - (int)(m >> 7), 126) : 0;
    if (first == 0) unscale[r] = __int_as_float((127 - e) << 23);
    const float scale = __int_as_float((e + 127) << 23);
    const uint64_t both = pack2(scale, scale);
#pragma unroll 2
    for (int c = first; c < all; c += step) {
      uint4* p = reinterpret_cast<uint4*>(row + c * 16);
      const uint4 v = *p;
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
      float x[8];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        unpack2(fma2(pack2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u)), both, 0), x[2 * i], x[2 * i + 1]);
      *p = make_uint4(f16x2(x[0], x[2]), f16x2(x[4], x[6]), f16x2(x[1], x[3]), f16x2(x[5], x[7]));
    }
  }
  __syncthreads();
}

// kGroups x 16 rows of W a tile, up to kNt x 8 rows of x.
template <int kGroups, int kNt>
__global__ void __launch_bounds__(kThreads, 1) fp4_rows_kernel(const Fp4Linear a, int tiles, int slots) {
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ __align__(8) uint64_t full[kWarps][kMostSlots];
  __shared__ int piece_tile[2 * kWarps];
  __shared__ uint32_t most[kFp4FewRows];
  __shared__ float unscale[kFp4FewRows];
  constexpr int kUnit = kGroups * kBlockBytes, kPiece = kGroups * kNt * 32;  // bytes; float4
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  const int pitch = x_pitch(a.k_blocks);
  uint8_t* ring = smem + warp * slots * kUnit;
  float4* firsts = reinterpret_cast<float4*>(smem + kWarps * slots * kUnit);  // a warp's first piece
  uint8_t* xs = reinterpret_cast<uint8_t*>(firsts + kWarps * kPiece);

  const uint32_t tile0 = blockIdx.x * tiles / gridDim.x, tile1 = (blockIdx.x + 1) * tiles / gridDim.x;  // (2^20 x SMs)
  const uint32_t units = (tile1 - tile0) * a.k_blocks;
  const int u0 = (int)((uint64_t)warp * units / kWarps), u1 = (int)((uint64_t)(warp + 1) * units / kWarps);
  constexpr int kParts = kTileBlocks / kGroups;  // tiles of this kernel in 128 rows
  auto source = [&](uint32_t tile, uint32_t kb) {
    return a.w + ((int64_t)(tile / kParts) * a.k_blocks + kb) * kTileBytes + tile % kParts * kUnit;
  };
  const int first = u0 / a.k_blocks, kb0 = u0 - first * a.k_blocks;
  if (lane < slots) tc::mbar_init(&full[warp][lane], 1);
  tc::fence_mbar_init();
  if (lane < 2) piece_tile[2 * warp + lane] = -1;
  if (lane == 0) {
    if (u0 < u1) tc::bulk_prefetch_l2(source(tile0 + first, kb0), kUnit);
    most[warp] = 0;
  }
  __syncwarp();
  griddep_wait();  // every input may be the previous kernel's output
  // the next unit to fetch: its blocks, its place in k and in the ring (no division in
  // the loop: with u / k_blocks and u % slots in it a unit took 170 instructions more)
  uint32_t src_tile = tile0 + (u0 + slots) / a.k_blocks;
  int src_kb = (u0 + slots) % a.k_blocks, src_slot = 0;
  const uint8_t* src = source(src_tile, src_kb);
  auto fetch = [&]() {
    tc::mbar_arrive_expect_tx(&full[warp][src_slot], kUnit);
    tc::bulk_g2s(ring + src_slot * kUnit, src, kUnit, &full[warp][src_slot]);
    src += kTileBytes;
    if (++src_kb == a.k_blocks) {  // the next tile's first block: beside this one's, or at the next 128 rows
      src_kb = 0, ++src_tile;
      src += kUnit - (src_tile % kParts ? (int64_t)a.k_blocks * kTileBytes : kTileBytes);
    }
    if (++src_slot == slots) src_slot = 0;
  };
  stage_x<8 * kNt>(a, xs, pitch, most, unscale, [&]() {
    if (u0 + lane < u1 && lane < slots) {
      const int u = u0 + lane, tile = u / a.k_blocks;
      tc::mbar_arrive_expect_tx(&full[warp][lane], kUnit);
      tc::bulk_g2s(ring + lane * kUnit, source(tile0 + tile, u - tile * a.k_blocks), kUnit, &full[warp][lane]);
    }
  });
  bool ok = true;
  // this lane's rows of x (columns from T on are dropped), its chunk of word 0
  const uint8_t* xr[kNt];
#pragma unroll
  for (int m = 0; m < kNt; ++m) xr[m] = xs + min(8 * m + g, a.T - 1) * pitch + t * 64;

  float acc[kGroups][kNt][4] = {};
  int kb = kb0, tile = first, s = 0;
  uint32_t phase = 0;
  int sent = min(u1, u0 + slots);  // (lane 0) where the units end whose copies have begun
  bool whole = kb == 0;
  for (int u = u0; u < u1; ++u) {
    tc::mbar_wait_or(&full[warp][s], phase, ok);  // (sums of what stands there, and a status, where it gives up; no more copies)
    __syncwarp();
    uint4 lo[kGroups], hi[kGroups];
    uint32_t sc[kGroups];
#pragma unroll
    for (int i = 0; i < kGroups; ++i) {
      const uint8_t* b = ring + s * kUnit + i * kBlockBytes;
      lo[i] = *reinterpret_cast<const uint4*>(b + fp4_unit(g, t));
      hi[i] = *reinterpret_cast<const uint4*>(b + fp4_unit(g + 8, t));
      sc[i] = *reinterpret_cast<const uint32_t*>(b + kBlockCodes + 4 * lane);
    }
    __syncwarp();
    if (lane == 0 && ok && u + slots < u1) fetch(), ++sent;
    if (++s == slots) s = 0, phase ^= 1;
    uint32_t f[kGroups][4];  // scales of words 0, 1 and 2, 3 of row g, of row g + 8
#pragma unroll
    for (int i = 0; i < kGroups; ++i) {
      const uint32_t p = scales2(sc[i] & 0xFFFFu), q = scales2(sc[i] >> 16);
      f[i][0] = __byte_perm(p, 0, 0x1010), f[i][1] = __byte_perm(p, 0, 0x3232);
      f[i][2] = __byte_perm(q, 0, 0x1010), f[i][3] = __byte_perm(q, 0, 0x3232);
    }
    // A unit's products are summed by themselves first, then added to the tile's sums: the tensor
    // core's own additions cut off, and over a long run that adds up.  16 rows of 4096 -> 32768
    // in fp32, error relative to the outputs' norm: 9.0e-8 so, 6.1e-7 with one running sum.  It
    // costs 16 rows over 128001 words 71.7 -> 75.1 us, 8 rows 50.5 -> 50.8 us.
    float part[kGroups][kNt][4] = {};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      uint4 x[kNt];
#pragma unroll
      for (int m = 0; m < kNt; ++m) x[m] = *reinterpret_cast<const uint4*>(xr[m] + kb * 256 + (j ^ t) * 16);
#pragma unroll
      for (int i = 0; i < kGroups; ++i) {
        const uint32_t wl = j == 0 ? lo[i].x : j == 1 ? lo[i].y : j == 2 ? lo[i].z : lo[i].w;
        const uint32_t wh = j == 0 ? hi[i].x : j == 1 ? hi[i].y : j == 2 ? hi[i].z : hi[i].w;
        uint32_t l[4], h[4];
        fp4_f16(wl, f[i][j / 2], l);
        fp4_f16(wh, f[i][2 + j / 2], h);
#pragma unroll
        for (int m = 0; m < kNt; ++m) {
          mma(part[i][m], l[0], h[0], l[1], h[1], x[m].x, x[m].y);
          mma(part[i][m], l[2], h[2], l[3], h[3], x[m].z, x[m].w);
        }
      }
    }
#pragma unroll
    for (int i = 0; i < kGroups; ++i)
#pragma unroll
      for (int m = 0; m < kNt; ++m)
#pragma unroll
        for (int c = 0; c < 4; ++c) acc[i][m][c] += part[i][m][c];
    if (++kb == a.k_blocks || u + 1 == u1) {  // the end of the tile, or of the warp's part of it
      const bool all = whole && kb == a.k_blocks, end = u + 1 == u1;
      // the warp's last piece goes to its ring, which is empty by then
      float4* piece = end ? reinterpret_cast<float4*>(ring) : firsts + warp * kPiece;
#pragma unroll
      for (int i = 0; i < kGroups; ++i)
#pragma unroll
        for (int m = 0; m < kNt; ++m) {
          float(&d)[4] = acc[i][m];
          const float4 v = make_float4(d[0], d[1], d[2], d[3]);
          if (all) store_group(a, ((tile0 + tile) * kGroups + i) * kBlockRows + g, 8 * m + 2 * t, unscale, v);
          else piece[(i * kNt + m) * 32 + lane] = v;
          d[0] = d[1] = d[2] = d[3] = 0.0f;
        }
      if (!all && lane == 0) piece_tile[2 * warp + (end ? 1 : 0)] = tile;
      if (kb == a.k_blocks) kb = 0, ++tile;
      whole = true;
    }
  }
  if (!ok) {
    report(a.status, CSA2_ERR_TIMEOUT);
    // nothing may land in shared memory after the CTA has left
    for (int u = max(u0, sent - slots); lane == 0 && u < sent; ++u) tc::mbar_wait(&full[warp][(u - u0) % slots], ((u - u0) / slots) & 1);
  }
  __syncthreads();
  // a shared tile's pieces stand in the order of its channels, two places a warp, a place
  // a lane here: the warp with the first of them joins them
  const int of_lane = piece_tile[lane];
#pragma unroll
  for (int p = 0; p < 2; ++p) {
    const int at = piece_tile[2 * warp + p];
    uint32_t same = __ballot_sync(0xffffffffu, of_lane == at);
    if (at < 0 || __ffs(same) - 1 != 2 * warp + p) continue;
    float4 sum[kGroups * kNt];
#pragma unroll
    for (int i = 0; i < kGroups * kNt; ++i) sum[i] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    for (; same; same &= same - 1) {
      const int q = __ffs(same) - 1;
      const float4* piece = q & 1 ? reinterpret_cast<const float4*>(smem + (q >> 1) * slots * kUnit) : firsts + (q >> 1) * kPiece;
#pragma unroll
      for (int i = 0; i < kGroups * kNt; ++i) {
        const float4 e = piece[i * 32 + lane];
        sum[i].x += e.x, sum[i].y += e.y, sum[i].z += e.z, sum[i].w += e.w;
      }
    }
#pragma unroll
    for (int i = 0; i < kGroups; ++i)
#pragma unroll
      for (int m = 0; m < kNt; ++m)
        store_group(a, ((tile0 + at) * kGroups + i) * kBlockRows + g, 8 * m + 2 * t, unscale, sum[i * kNt + m]);
  }
}

template <int kGroups, int kNt>
cudaError_t launch_of(const Fp4Linear& a, const Shape& s, cudaStream_t stream) {
  auto kern = fp4_rows_kernel<kGroups, kNt>;
  static std::atomic<bool> done[64];
  const cudaError_t e = allow_smem(kern, kSmemMost, done);
  if (e != cudaSuccess) return e;
  const int tiles = (a.n + 16 * kGroups - 1) / (16 * kGroups);
  return launch_k(kern, dim3((unsigned)std::min(tiles, num_sms())), dim3(kThreads), s.smem, stream, 0, a, tiles, s.slots);
}

}  // namespace

bool fp4_rows_ok(const Fp4Linear& a) { return a.T <= kFp4FewRows && shape_of(a, 1).slots != 0; }

cudaError_t launch_fp4_rows(const Fp4Linear& a, cudaStream_t stream) {
  // 32 rows a tile, which halve x's way through shared memory and what a unit costs beside
  // its products, where the rings stay deep and the SM with the most tiles has less of
  // them: a unit of 32 rows takes 1.5 times one of 16
  const Shape two = shape_of(a, 2);
  const int sms = num_sms(), tiles1 = (a.n + 15) / 16, tiles2 = (a.n + 31) / 32;
  const bool wide = two.slots >= 3 && 3 * ((tiles2 + sms - 1) / sms) <= 2 * ((tiles1 + sms - 1) / sms);
  if (a.T <= 8) return wide ? launch_of<2, 1>(a, two, stream) : launch_of<1, 1>(a, shape_of(a, 1), stream);
  return wide ? launch_of<2, 2>(a, two, stream) : launch_of<1, 2>(a, shape_of(a, 1), stream);
}

}  // namespace csa2
