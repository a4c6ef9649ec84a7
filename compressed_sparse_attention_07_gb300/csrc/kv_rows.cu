// Attention of few query rows over the paged key / value cache (single-token
// decode, drafted blocks): every key and value is read once from HBM for up to
// 32 rows (query heads of a kv head x new tokens), so the cache's bytes decide.
//
// One CTA takes one kv head, its rows (8 NT at most) and a part of the keys; its warps
// (four) take tiles of 64 keys (FP4, one page) or 32 (bf16) in turn, each with
// its own two-stage ring of bulk copies, its own running maximum, sum and
// output in registers, joined through shared memory at the end.  With several
// parts a second kernel joins them (in part order, so results do not vary);
// where up to eight parts of every head run at once, one CTA an SM, the parts of
// a head are a cluster of CTAs of eight warps, which join through distributed
// shared memory: one launch, and no workspace.
//
// The products are formed transposed, S^T = K Q^T (m16n8k16: 16 keys, 8 rows)
// and O^T = V^T P^T (16 channels, 8 rows), so 8 rows fill an instruction where
// the usual order would fill half of one, and the softmax's statistics of a row
// stand in the same threads in both.  P^T gets from the first product's
// register layout to the second's by an 8x8 transpose in registers (movmatrix).
//
// FP4: a thread reads 16 bytes of a key (32 channels) and 8 of a value (16
// channels): the order of channels inside a product and of keys inside a tile
// is free, so it is chosen to make these reads whole words without bank
// conflicts.  Key nibbles convert in place; value nibbles of two keys are first
// brought into one byte, which then converts to the pair the second product
// wants.  E2M1 x E4M3 is exact in f16; a query row is scaled by a power of two
// so that its largest channel lies in [1, 2) (below 4 at the end of bf16's range;
// the inverse goes into the softmax scale), so bf16 queries of any size are exact
// too (channels below 2^-14 of the row's largest lose bits).
//
// Measured: one token of each of 32 sequences of 32767, 64 over 8 heads of 128, FP4:
// 214 us, 5.7 TB/s (84 % of a copy's rate; 1180 instructions a page and head keep
// the ALU at 50 %); of 48 sequences of 0 .. 16383, 28 over 4 heads of 64, bf16: 70 us,
// 5.7 TB/s; of one sequence of 4095: 7.7 us in a graph, launches and look-ups mostly.
#include <algorithm>

#include "kv.cuh"
#include "tc.cuh"

namespace csa2 {
namespace {

constexpr int kMostCluster = 8;  // CTAs that join through distributed shared memory

template <int D, bool kFp4, int NT, bool kCluster>
struct Rows {
  static constexpr int kWarps = kCluster && (kFp4 || D == 64) ? 8 : 4;
  static constexpr int kTile = kFp4 ? 64 : 32;                   // keys of a tile
  static constexpr int kPerPage = kPage / kTile;
  static constexpr int kSub = (kFp4 && NT < 4) ? 64 : 32;        // keys of a softmax step
  static constexpr int kData = kFp4 ? kTile * D / 2 : kTile * D * 2;
  static constexpr int kScales = kFp4 ? kTile * D / 16 : 0;
  static constexpr int kStage = 2 * (kData + kScales);           // K, V, K scales, V scales
  static constexpr int kWarpBytes = 2 * kStage;
  static constexpr int kOPitch = D + 8;                          // floats of a row in the joining area
  static constexpr int kQFrag = NT * (D / 16) * 32 * 8;  // query fragments
  static constexpr int kJoined = kCluster ? 8 * NT * D * 4 : 0;  // this CTA's part, for the cluster to read
  static constexpr int kSmem = kWarps * kWarpBytes + kQFrag + kJoined;
  static_assert(8 * NT * kOPitch * 4 <= kWarpBytes, "the joining area fits a warp's ring");
  static constexpr int kCtas = kCluster || kSmem > 112 * 1024 ? 1 : (kSmem > 72 * 1024 || NT > 1) ? 2 : 3;
};

template <bool kF16>
__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1) {
  if constexpr (kF16)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
template <bool kTrans>
__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
  if constexpr (kTrans)
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
  else
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}

template <int D, bool kFp4, int NT, bool kCluster>
__global__ void __launch_bounds__(Rows<D, kFp4, NT, kCluster>::kWarps * 32, Rows<D, kFp4, NT, kCluster>::kCtas)
    kv_rows_kernel(KvAtt a) {
  using R = Rows<D, kFp4, NT, kCluster>;
  constexpr int kWarps = R::kWarps, kRows = 8 * NT, KS = D / 16, MT = D / 16;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ __align__(8) uint64_t bars[kWarps][2];
  __shared__ int row_hi[kRows], row_lo[kRows];
  __shared__ float row_scale[kRows];
  __shared__ float join_m[kWarps][kRows], join_l[kWarps][kRows];
  __shared__ float part_l[kRows];  // (cluster) this CTA's log2-sum-exp2 of each row

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  const int part = blockIdx.x, kh = blockIdx.y, b = blockIdx.z;
  if (lane < 2) tc::mbar_init(&bars[warp][lane], 1);
  tc::fence_mbar_init();
  griddep_wait();
  if (kv_joined(a)) griddep_launch();
  int row0, rows, keys;
  if (!kv_sequence(a, b, row0, rows, keys)) return;
  if (rows == 0) return;
  const int n_rows = rows * a.group;  // of this kv head, kRows at most
  int p0, p1;
  kv_pages(a, 0, rows - 1, rows, keys, p0, p1);
  const int n_act = kv_parts(a, p0, p1);
  if (!kCluster && part > 0 && part >= n_act) return;
  const int pb = min(p0 + part * a.part_pages, p1), pe = min(pb + a.part_pages, p1);
  const int key_end = kv_hi(a, rows - 1, rows, keys);  // no row sees keys from here on
  const int tb = pb * R::kPerPage, te = min(pe * R::kPerPage, (key_end + R::kTile - 1) / R::kTile);

  uint8_t* ring = smem + warp * R::kWarpBytes;
  const int32_t* table = a.c.table + (int64_t)b * a.c.max_pages;
  auto load = [&](int tile, int stage) -> bool {  // the whole warp; whether the tile's page is in the pool
    const int32_t page = __ldg(table + tile / R::kPerPage);
    if (page < 0 || page >= a.c.num_pages) {
      if (lane == 0) report(a.status, CSA2_ERR_BAD_PAGE);
      return false;
    }
    uint8_t* dst = ring + stage * R::kStage;
    uint64_t* bar = &bars[warp][stage];
    const int64_t block = (int64_t)page * a.kv_heads + kh;
    if (lane == 0) tc::mbar_arrive_expect_tx(bar, R::kStage);
    __syncwarp();
    if constexpr (kFp4) {
      if (tc::elect_one()) {
        tc::bulk_g2s(dst, a.c.k + block * R::kData, R::kData, bar);
        tc::bulk_g2s(dst + R::kData, a.c.v + block * R::kData, R::kData, bar);
        tc::bulk_g2s(dst + 2 * R::kData, a.c.ks + block * R::kScales, R::kScales, bar);
        tc::bulk_g2s(dst + 2 * R::kData + R::kScales, a.c.vs + block * R::kScales, R::kScales, bar);
      }
      __syncwarp();
    } else {
      constexpr int kRun = R::kTile * 16;  // bytes of one channel chunk of the tile
      const int half = tile % R::kPerPage;
      if (lane < 2 * (D / 8)) {
        const int v = lane / (D / 8), c = lane % (D / 8);
        tc::bulk_g2s(dst + v * R::kData + c * kRun,
                     (v ? a.c.v : a.c.k) + block * (2 * R::kData) + c * (kPage * 16) + half * kRun, kRun, bar);
      }
    }
    return true;
  };
  int tile = tb + warp;
  uint32_t filled = 0;  // bit s: stage s has a tile on its way
  __syncwarp();
  if (tile < te) filled |= load(tile, 0) ? 1u : 0u;
  if (tile + kWarps < te) filled |= load(tile + kWarps, 1) ? 2u : 0u;

  // this CTA's rows: what they see, their scale, and their fragments of Q
  float qs = a.scale * kLog2e;
  uint2* qfrag = reinterpret_cast<uint2*>(smem + kWarps * R::kWarpBytes);  // [KS][NT][32]
  for (int n = warp; n < NT; n += kWarps) {
    const int r = 8 * n + g;
    const bool live = r < n_rows;
    const int i = live ? group_of(a, r) : 0, h = live ? kh * a.group + r - group_of(a, r) * a.group : 0;
    const uint16_t* q = a.q + (int64_t)(row0 + i) * a.q_stride + h * D;
    if constexpr (kFp4) {
      uint4 w[D / 32];  // channels D/4 * t .. of row g
#pragma unroll
      for (int x = 0; x < D / 32; ++x) {
        w[x] = make_uint4(0, 0, 0, 0);
        if (live) w[x] = __ldg(reinterpret_cast<const uint4*>(q + (D / 4) * t) + x);
      }
      uint32_t most = 0;
#pragma unroll
      for (int x = 0; x < D / 32; ++x) {
        const uint32_t u[4] = {w[x].x, w[x].y, w[x].z, w[x].w};
#pragma unroll
        for (int y = 0; y < 4; ++y) most = max(most, max(u[y] & 0x7F80u, (u[y] >> 16) & 0x7F80u));
      }
      most = max(most, __shfl_xor_sync(0xffffffffu, most, 1));
      most = max(most, __shfl_xor_sync(0xffffffffu, most, 2));
      // the largest channel's exponent, biased, where its power of two and the
      // inverse are both normal numbers
      const uint32_t e = min(max(most >> 7, 1u), 253u);
      const float down = __uint_as_float((254u - e) << 23), up = __uint_as_float(e << 23);
#pragma unroll
      for (int x = 0; x < D / 32; ++x) {
        const uint32_t u[4] = {w[x].x, w[x].y, w[x].z, w[x].w};
#pragma unroll
        for (int y = 0; y < 2; ++y) {  // four channels: one product step's share
          const uint32_t l = u[2 * y], m = u[2 * y + 1];
          const uint32_t f0 = f16x2(__uint_as_float(l << 16) * down, __uint_as_float(l & 0xFFFF0000u) * down);
          const uint32_t f1 = f16x2(__uint_as_float(m << 16) * down, __uint_as_float(m & 0xFFFF0000u) * down);
          qfrag[((2 * x + y) * NT + n) * 32 + lane] = make_uint2(f0, f1);
        }
      }
      if (t == 0) row_scale[8 * n + g] = qs * up;
    } else {
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        uint32_t f0 = 0, f1 = 0;
        if (live) {
          f0 = __ldg(reinterpret_cast<const uint32_t*>(q + 16 * ks + 2 * t));
          f1 = __ldg(reinterpret_cast<const uint32_t*>(q + 16 * ks + 8 + 2 * t));
        }
        qfrag[(ks * NT + n) * 32 + lane] = make_uint2(f0, f1);
      }
      if (t == 0) row_scale[8 * n + g] = qs;
    }
    if (t == 0) {
      row_hi[8 * n + g] = live ? kv_hi(a, i, rows, keys) : 0;
      row_lo[8 * n + g] = live ? kv_lo(a, i, rows, keys) : 0;
    }
  }
  __syncthreads();
  // keys that every row sees: no masks inside
  const int all_lo = kv_lo(a, rows - 1, rows, keys), all_hi = kv_hi(a, 0, rows, keys);

  float sc[NT][2], m[NT][2], l[NT][2], o[MT][NT][4];
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      sc[n][e] = row_scale[8 * n + 2 * t + e];
      m[n][e] = -INFINITY;
      l[n][e] = 0.0f;
    }
#pragma unroll
  for (int x = 0; x < MT; ++x)
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[x][n][e] = 0.0f;
  uint2 qreg[KS];
  if constexpr (NT == 1) {
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) qreg[ks] = qfrag[ks * 32 + lane];
  }
  auto qf = [&](int ks, int n) -> uint2 {
    if constexpr (NT == 1) return qreg[ks];
    else return qfrag[(ks * NT + n) * 32 + lane];
  };

  const int sig = kFp4 ? (g >> 1) + 4 * (g & 1) : g;  // key of fragment row g within 8
  uint32_t phase = 0;
  bool late = false;
  for (int it = 0; tile < te; tile += kWarps, ++it) {
    const int stage = it & 1;
    if ((filled >> stage) & 1u) {
      if (!__all_sync(0xffffffffu, tc::mbar_wait(&bars[warp][stage], (phase >> stage) & 1u))) {
        late = true;
        // nothing may land in shared memory after the CTA has left
        if ((filled >> (stage ^ 1)) & 1u) tc::mbar_wait(&bars[warp][stage ^ 1], (phase >> (stage ^ 1)) & 1u);
        tc::mbar_wait(&bars[warp][stage], (phase >> stage) & 1u);
        break;
      }
      phase ^= 1u << stage;
      filled &= ~(1u << stage);
      uint8_t* kd = ring + stage * R::kStage;
      uint8_t* vd = kd + R::kData;
      const uint8_t* ks_ = vd + R::kData;
      uint8_t* vs_ = vd + R::kData + R::kScales;
      const int k0 = tile * R::kTile;
      if (k0 + R::kTile > keys) {
        // slots from kv_len on hold anything: their weights are 0, and so have
        // to be their values
        const int first = keys - k0;
        if constexpr (kFp4) {
          for (int x = first * (D / 16) + lane; x < R::kScales; x += 32) vs_[x] = 0;
        } else {
          for (int x = lane; x < R::kTile * (D / 8); x += 32)
            if (x % R::kTile >= first) reinterpret_cast<uint4*>(vd)[x] = make_uint4(0, 0, 0, 0);
        }
        __syncwarp();
      }
      const bool masked = k0 < all_lo || k0 + R::kTile > all_hi;
#pragma unroll 1
      for (int s0 = 0; s0 < R::kTile; s0 += R::kSub) {
        constexpr int SM = R::kSub / 16;  // 16-key steps
        float s[SM][NT][4];
#pragma unroll
        for (int x = 0; x < SM; ++x)
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) s[x][n][e] = 0.0f;
        if constexpr (kFp4) {
          constexpr int W = D / 32;  // words of a thread's share of a key
          uint32_t w[SM][2][W], f[SM][2];
#pragma unroll
          for (int x = 0; x < SM; ++x)
#pragma unroll
            for (int y = 0; y < 2; ++y) {
              const int key = s0 + 16 * x + 8 * y + sig;
              if constexpr (D == 128) {
                const uint4 v = *reinterpret_cast<const uint4*>(kd + key * (D / 2) + t * 16);
                w[x][y][0] = v.x, w[x][y][1] = v.y, w[x][y][2] = v.z, w[x][y][3] = v.w;
                f[x][y] = scales2(*reinterpret_cast<const uint16_t*>(ks_ + key * (D / 16) + 2 * t));
              } else {
                const uint2 v = *reinterpret_cast<const uint2*>(kd + key * (D / 2) + t * 8);
                w[x][y][0] = v.x, w[x][y][1] = v.y;
                f[x][y] = scales2(ks_[key * (D / 16) + t]);
              }
            }
#pragma unroll
          for (int j = 0; j < W; ++j) {  // eight channels, two product steps
            uint2 q0[NT], q1[NT];
#pragma unroll
            for (int n = 0; n < NT; ++n) q0[n] = qf(2 * j, n), q1[n] = qf(2 * j + 1, n);
#pragma unroll
            for (int x = 0; x < SM; ++x) {
              uint32_t r0[4], r1[4];
              codes8(w[x][0][j], r0);
              codes8(w[x][1][j], r1);
              const uint32_t sel = j < 2 ? 0x1010u : 0x3232u;
              const uint32_t s0_ = __byte_perm(f[x][0], 0, sel), s1_ = __byte_perm(f[x][1], 0, sel);
#pragma unroll
              for (int y = 0; y < 4; ++y) r0[y] = mul2(r0[y], s0_), r1[y] = mul2(r1[y], s1_);
#pragma unroll
              for (int n = 0; n < NT; ++n) {
                mma<true>(s[x][n], r0[0], r1[0], r0[1], r1[1], q0[n].x, q0[n].y);
                mma<true>(s[x][n], r0[2], r1[2], r0[3], r1[3], q1[n].x, q1[n].y);
              }
            }
          }
        } else {
          // matrices of a load: keys 0-7 and 8-15 of chunk 2 ks, then of 2 ks + 1
          const uint32_t base = tc::smem_u32(kd) + (((lane >> 4) * R::kTile) + (lane & 15)) * 16;
#pragma unroll
          for (int ks = 0; ks < KS; ++ks) {
            uint2 q[NT];
#pragma unroll
            for (int n = 0; n < NT; ++n) q[n] = qf(ks, n);
#pragma unroll
            for (int x = 0; x < SM; ++x) {
              uint32_t r[4];
              ldsm4<false>(base + (2 * ks * R::kTile + s0 + 16 * x) * 16, r);
#pragma unroll
              for (int n = 0; n < NT; ++n) mma<false>(s[x][n], r[0], r[1], r[2], r[3], q[n].x, q[n].y);
            }
          }
        }
        // ---- softmax of the step
        float top[NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            int lo = 0, hi = 0;
            if (masked) lo = row_lo[8 * n + 2 * t + e] - k0 - s0, hi = row_hi[8 * n + 2 * t + e] - k0 - s0;
            float best = -INFINITY;
#pragma unroll
            for (int x = 0; x < SM; ++x)
#pragma unroll
              for (int y = 0; y < 2; ++y) {
                float v = s[x][n][2 * y + e] * sc[n][e];
                if (masked) {
                  const int key = 16 * x + 8 * y + sig;
                  if (key < lo || key >= hi) v = -INFINITY;
                }
                s[x][n][2 * y + e] = v;
                best = fmaxf(best, v);
              }
#pragma unroll
            for (int d = 4; d < 32; d <<= 1) best = fmaxf(best, __shfl_xor_sync(0xffffffffu, best, d));
            top[n][e] = best;
          }
        bool grew = false;
#pragma unroll
        for (int n = 0; n < NT; ++n) grew |= top[n][0] > m[n][0] || top[n][1] > m[n][1];
        if (__any_sync(0xffffffffu, grew)) {
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const float m2 = fmaxf(m[n][e], top[n][e]);
              const float f = m[n][e] == -INFINITY ? 0.0f : ex2(m[n][e] - m2);
              m[n][e] = m2;
              l[n][e] *= f;
#pragma unroll
              for (int x = 0; x < MT; ++x) o[x][n][e] *= f, o[x][n][2 + e] *= f;
            }
        }
        uint32_t pt[SM][NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          const float z0 = m[n][0] == -INFINITY ? 0.0f : m[n][0], z1 = m[n][1] == -INFINITY ? 0.0f : m[n][1];
#pragma unroll
          for (int x = 0; x < SM; ++x)
#pragma unroll
            for (int y = 0; y < 2; ++y) {
              const float u = ex2(s[x][n][2 * y] - z0), v = ex2(s[x][n][2 * y + 1] - z1);
              l[n][0] += u, l[n][1] += v;
              pt[x][n][y] = transpose8(kFp4 ? f16x2(u, v) : bf16x2(u, v));
            }
        }
        // ---- O^T += V^T P^T
#pragma unroll
        for (int x = 0; x < SM; ++x) {
          if constexpr (kFp4) {
            constexpr int W = D / 64;  // words of a thread's share of a value
            const int k = s0 + 16 * x + t;
            uint32_t w[4][W], f[4];
#pragma unroll
            for (int y = 0; y < 4; ++y) {
              const uint8_t* p = vd + (k + 4 * y) * (D / 2) + g * (D / 16);
              if constexpr (D == 128) {
                const uint2 v = *reinterpret_cast<const uint2*>(p);
                w[y][0] = v.x, w[y][1] = v.y;
                f[y] = vs_[(k + 4 * y) * 8 + g];
              } else {
                w[y][0] = *reinterpret_cast<const uint32_t*>(p);
                f[y] = vs_[(k + 4 * y) * 4 + (g >> 1)];
              }
            }
            const uint32_t fa = scales2(f[0] | (f[1] << 8)), fb = scales2(f[2] | (f[3] << 8));
#pragma unroll
            for (int j = 0; j < W; ++j) {
              const uint32_t la = (w[0][j] & 0x0F0F0F0Fu) | ((w[1][j] << 4) & 0xF0F0F0F0u);
              const uint32_t ha = ((w[0][j] >> 4) & 0x0F0F0F0Fu) | (w[1][j] & 0xF0F0F0F0u);
              const uint32_t lb = (w[2][j] & 0x0F0F0F0Fu) | ((w[3][j] << 4) & 0xF0F0F0F0u);
              const uint32_t hb = ((w[2][j] >> 4) & 0x0F0F0F0Fu) | (w[3][j] & 0xF0F0F0F0u);
              uint32_t a0[4], a1[4], a2[4], a3[4];
              codes8(la, a0);
              codes8(ha, a1);
              codes8(lb, a2);
              codes8(hb, a3);
#pragma unroll
              for (int y = 0; y < 4; ++y) {
                const uint32_t r0 = mul2(a0[y], fa), r1 = mul2(a1[y], fa), r2 = mul2(a2[y], fb), r3 = mul2(a3[y], fb);
#pragma unroll
                for (int n = 0; n < NT; ++n) mma<true>(o[4 * j + y][n], r0, r1, r2, r3, pt[x][n][0], pt[x][n][1]);
              }
            }
          } else {
            // matrices: chunk 2 mt (channels of rows 0-7), 2 mt + 1; then keys 8-15
            const uint32_t base = tc::smem_u32(vd) + ((((lane >> 3) & 1) * R::kTile) + s0 + 16 * x + 8 * (lane >> 4) + (lane & 7)) * 16;
#pragma unroll
            for (int y = 0; y < MT; ++y) {
              uint32_t r[4];
              ldsm4<true>(base + 2 * y * R::kTile * 16, r);
#pragma unroll
              for (int n = 0; n < NT; ++n) mma<false>(o[y][n], r[0], r[1], r[2], r[3], pt[x][n][0], pt[x][n][1]);
            }
          }
        }
      }
      __syncwarp();  // the stage is read: it may be filled again
    }
    if (tile + 2 * kWarps < te && load(tile + 2 * kWarps, stage)) filled |= 1u << stage;
  }
  if (late && lane == 0) report(a.status, CSA2_ERR_TIMEOUT);
  late = __syncthreads_or(late);
  if (!kCluster && late) return;

  // ---- join the warps
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float v = l[n][e];
#pragma unroll
      for (int d = 4; d < 32; d <<= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
      if (g == 0) join_m[warp][8 * n + 2 * t + e] = m[n][e], join_l[warp][8 * n + 2 * t + e] = v;
    }
  float* mine = reinterpret_cast<float*>(ring);
#pragma unroll
  for (int x = 0; x < MT; ++x)
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e)
        *reinterpret_cast<float2*>(mine + (8 * n + 2 * t + e) * R::kOPitch + x * 16 + 2 * g) =
            make_float2(o[x][n][e], o[x][n][2 + e]);
  __syncthreads();
  const bool whole = n_act <= 1;
  float* joined = reinterpret_cast<float*>(smem + kWarps * R::kWarpBytes + R::kQFrag);  // [kRows][D] (cluster)
  for (int x = tid; x < kRows * (D / 2); x += kWarps * 32) {
    const int r = x / (D / 2), c = 2 * (x % (D / 2));
    if (r >= n_rows) break;
    float top = -INFINITY;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) top = fmaxf(top, join_m[w][r]);
    float sum = 0.0f, v0 = 0.0f, v1 = 0.0f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float f = join_m[w][r] == -INFINITY ? 0.0f : ex2(join_m[w][r] - top);
      sum += f * join_l[w][r];
      const float* src = reinterpret_cast<const float*>(smem + w * R::kWarpBytes) + r * R::kOPitch;
      if constexpr (kFp4) {  // channel (D / 8) g + 2 mt + e at [mt][g][e]
        const float2 v = *reinterpret_cast<const float2*>(src + ((c % (D / 8)) / 2) * 16 + 2 * (c / (D / 8)));
        v0 += f * v.x, v1 += f * v.y;
      } else {  // channel 16 mt + g + 8 e
        const float* p = src + (c / 16) * 16 + 2 * (c % 8) + (c % 16) / 8;
        v0 += f * p[0], v1 += f * p[2];
      }
    }
    const float inv = sum > 0.0f ? 1.0f / sum : (sum == 0.0f ? 0.0f : NAN);
    const int i = row0 + group_of(a, r), h = kh * a.group + (r - group_of(a, r) * a.group);
    const int64_t at = (int64_t)i * a.n_heads + h;
    const float lse2 = sum == 0.0f ? -INFINITY : top + log2f(sum);
    if (whole) {
      if (kCluster && part > 0) break;
      *reinterpret_cast<uint32_t*>(a.out + (int64_t)i * a.out_stride + h * D + c) = bf16x2(v0 * inv, v1 * inv);
      if (a.lse && c == 0) a.lse[at] = lse2 * kLn2;
    } else if (kCluster) {
      *reinterpret_cast<float2*>(joined + r * D + c) = make_float2(v0 * inv, v1 * inv);
      if (c == 0) part_l[r] = lse2;
    } else {
      const int64_t pa = part * a.part_step + at;
      *reinterpret_cast<float2*>(a.part_o + pa * D + c) = make_float2(v0 * inv, v1 * inv);
      if (c == 0) a.part_l[pa] = lse2;
    }
  }
  if constexpr (kCluster) {
    // ---- join the parts through distributed shared memory, each CTA a share of
    // the channels, in part order
    __syncthreads();
    tc::cluster_sync();
    if (!whole) {
      const uint32_t mine_o = tc::smem_u32(joined), mine_l = tc::smem_u32(part_l);
      for (int x = part * (kWarps * 32) + tid; x < kRows * (D / 4); x += gridDim.x * (kWarps * 32)) {
        const int r = x / (D / 4), c = 4 * (x % (D / 4));
        if (r >= n_rows) break;
        float lp[kMostCluster];
        float4 v[kMostCluster];
        float top = -INFINITY;
#pragma unroll
        for (int p = 0; p < kMostCluster; ++p) {
          lp[p] = -INFINITY;
          if (p < n_act) {
            lp[p] = tc::ld_dsmem(tc::map_rank(mine_l + 4 * r, p));
            v[p] = tc::ld_dsmem_v4(tc::map_rank(mine_o + 4 * (r * D + c), p));
            top = fmaxf(top, lp[p]);
          }
        }
        float sum = 0.0f, o0 = 0.0f, o1 = 0.0f, o2 = 0.0f, o3 = 0.0f;
#pragma unroll
        for (int p = 0; p < kMostCluster; ++p) {
          if (p < n_act) {
            const float f = lp[p] == -INFINITY ? 0.0f : ex2(lp[p] - top);
            sum += f;
            o0 += f * v[p].x, o1 += f * v[p].y, o2 += f * v[p].z, o3 += f * v[p].w;
          }
        }
        const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
        const int i = row0 + group_of(a, r), h = kh * a.group + (r - group_of(a, r) * a.group);
        *reinterpret_cast<uint2*>(a.out + (int64_t)i * a.out_stride + h * D + c) =
            make_uint2(bf16x2(o0 * inv, o1 * inv), bf16x2(o2 * inv, o3 * inv));
        if (a.lse && c == 0) a.lse[(int64_t)i * a.n_heads + h] = sum == 0.0f ? -INFINITY : (top + log2f(sum)) * kLn2;
      }
    }
    __syncthreads();
    tc::cluster_sync();  // nobody leaves while his part may be read
  }
}

// Joins the parts of each row of the divided tiles: out = sum 2^(l_p - l) o_p, one
// warp a row.  Bound by latency (a row's parts are some 4 KB): eight parts are on their
// way at a time, which took 48 ragged sequences in parts from 72.7 to 70.9 us.
template <int D>
__global__ void __launch_bounds__(256) kv_join_kernel(KvAtt a, int tile_rows, int per) {
  griddep_wait();
  const int lane = threadIdx.x & 31, id = a.whole + blockIdx.x / per;  // per: CTAs of a tile
  int b = id / a.kv_heads, kh = id % a.kv_heads, tile = 0;  // kv_rows_kernel: one a kv head
  if (tile_rows > kMostRows && !kv_tile(a, tile_rows, id, b, kh, tile)) return;
  const int tile0 = tile * tile_rows;
  int row0, rows, keys;
  if (!kv_sequence(a, b, row0, rows, keys)) return;
  const int r = tile0 + blockIdx.x % per * 8 + threadIdx.x / 32;
  if (r >= rows * a.group) return;
  const int i = group_of(a, r), h = kh * a.group + r - i * a.group;
  const int last = min(tile0 + tile_rows, rows * a.group) - 1;
  int p0, p1;
  kv_pages(a, group_of(a, tile0), group_of(a, last), rows, keys, p0, p1);
  const int n = kv_parts(a, p0, p1);
  if (n <= 1) return;
  const int64_t at = (int64_t)(row0 + i) * a.n_heads + h, step = a.part_step;
  const int64_t from = kv_part_row(a, id, r, tile0, at);
  // The outputs of eight parts are on their way while the maximum is formed, and of
  // the next eight while these are added.
  constexpr int kAhead = 8, kLane = D / 32;  // channels of a lane
  const float* src = a.part_o + from * D + lane * kLane;
  float x[kAhead][kLane];
  auto load = [&](int p0) {
#pragma unroll
    for (int p = 0; p < kAhead; ++p) {
      if (p0 + p >= n) break;
      if constexpr (D == 128) {
        const float4 v = *reinterpret_cast<const float4*>(src + (p0 + p) * step * D);
        x[p][0] = v.x, x[p][1] = v.y, x[p][2] = v.z, x[p][3] = v.w;
      } else {
        const float2 v = *reinterpret_cast<const float2*>(src + (p0 + p) * step * D);
        x[p][0] = v.x, x[p][1] = v.y;
      }
    }
  };
  load(0);
  float lp[4];  // of parts lane, lane + 32, .. (128 at most)
  float top = -INFINITY;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    lp[k] = lane + 32 * k < n ? a.part_l[(lane + 32 * k) * step + from] : -INFINITY;
    top = fmaxf(top, lp[k]);
  }
#pragma unroll
  for (int d = 16; d; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
#pragma unroll
  for (int k = 0; k < 4; ++k) lp[k] = lp[k] == -INFINITY ? 0.0f : ex2(lp[k] - top);
  float sum = 0.0f, v[kLane] = {};
  for (int p0 = 0; p0 < n; p0 += kAhead) {
    float y[kAhead][kLane];
#pragma unroll
    for (int p = 0; p < kAhead; ++p)
#pragma unroll
      for (int c = 0; c < kLane; ++c) y[p][c] = x[p][c];
    if (p0 + kAhead < n) load(p0 + kAhead);
#pragma unroll
    for (int p = 0; p < kAhead; ++p) {
      const int at_p = p0 + p;
      const float all = at_p < 32 ? lp[0] : at_p < 64 ? lp[1] : at_p < 96 ? lp[2] : lp[3];
      const float f = __shfl_sync(0xffffffffu, all, at_p & 31);
      if (at_p < n) {
        sum += f;
#pragma unroll
        for (int c = 0; c < kLane; ++c) v[c] += f * y[p][c];
      }
    }
  }
  const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
  uint16_t* out = a.out + (int64_t)(row0 + i) * a.out_stride + h * D + lane * (D / 32);
  if constexpr (D == 128)
    *reinterpret_cast<uint2*>(out) = make_uint2(bf16x2(v[0] * inv, v[1] * inv), bf16x2(v[2] * inv, v[3] * inv));
  else
    *reinterpret_cast<uint32_t*>(out) = bf16x2(v[0] * inv, v[1] * inv);
  if (a.lse && lane == 0) a.lse[at] = sum == 0.0f ? -INFINITY : (top + log2f(sum)) * kLn2;
}

template <int D, bool kFp4, int NT, bool kCluster>
cudaError_t launch(int B, const KvAtt& a, cudaStream_t stream) {
  using R = Rows<D, kFp4, NT, kCluster>;
  auto kern = kv_rows_kernel<D, kFp4, NT, kCluster>;
  static std::atomic<bool> done[64];
  const cudaError_t e = allow_smem(kern, R::kSmem, done);
  if (e != cudaSuccess) return e;
  return launch_k(kern, dim3(a.n_parts, a.kv_heads, B), dim3(R::kWarps * 32), R::kSmem, stream,
                  kCluster ? a.n_parts : 0, a);
}

template <int D, bool kFp4>
cudaError_t launch_rows(int nt, int B, const KvAtt& a, cudaStream_t stream) {
  if (a.cluster)
    return nt == 1   ? launch<D, kFp4, 1, true>(B, a, stream)
           : nt == 2 ? launch<D, kFp4, 2, true>(B, a, stream)
                     : launch<D, kFp4, 4, true>(B, a, stream);
  return nt == 1   ? launch<D, kFp4, 1, false>(B, a, stream)
         : nt == 2 ? launch<D, kFp4, 2, false>(B, a, stream)
                   : launch<D, kFp4, 4, false>(B, a, stream);
}

// CTAs of an SM without clusters, and warps of a CTA with.
template <int D, bool kFp4>
void shape(int nt, int* ctas, int* warps) {
  *ctas = nt == 1 ? Rows<D, kFp4, 1, false>::kCtas : nt == 2 ? Rows<D, kFp4, 2, false>::kCtas : Rows<D, kFp4, 4, false>::kCtas;
  *warps = Rows<D, kFp4, 1, true>::kWarps;
}

// Blocks of eight rows for n rows of a kv head: a CTA takes them all.
static_assert(kMostRows == 32, "a CTA of four blocks, and kv_join_kernel, take every row of a kv head");
int row_blocks(int64_t n) { return n <= 8 ? 1 : n <= 16 ? 2 : 4; }

}  // namespace

KvPlan kv_plan(const csa2_kv_cfg& cfg, int B, int T, int max_q, int max_kv, bool cross, size_t room) {
  const int group = cfg.n_heads / cfg.kv_heads;
  if ((int64_t)max_q * group > kMostRows) return kv_tiles_plan(cfg, B, T, max_q, max_kv, cross, room);
  KvPlan plan = {1, 1, false, 0, 0, 0, (int64_t)T * cfg.n_heads, 0, 0};
  const size_t part_bytes = (size_t)plan.part_step * (cfg.head_dim + 1) * 4;
  const int nt = row_blocks((int64_t)max_q * group);
  int64_t pages = ((int64_t)max_kv + kPage - 1) / kPage;
  if (cfg.window && !cross)  // max_q rows see window + max_q - 1 keys
    pages = std::min<int64_t>(pages, ((int64_t)cfg.window + max_q + kPage - 2) / kPage + 1);
  if (pages < 1) pages = 1;
  const bool fp4 = cfg.cache_dtype == CSA2_CACHE_FP4;
  int per_sm, wide;
  if (cfg.head_dim == 128) fp4 ? shape<128, true>(nt, &per_sm, &wide) : shape<128, false>(nt, &per_sm, &wide);
  else fp4 ? shape<64, true>(nt, &per_sm, &wide) : shape<64, false>(nt, &per_sm, &wide);
  const int64_t sms = num_sms(), base = (int64_t)B * cfg.kv_heads;
  // The number of parts that ends soonest, in units of a page's share of an
  // SM's throughput: an SM's CTAs (n at most, each its pages and about three
  // pages' work besides) share it, but one warp alone needs about ten units for
  // a page and a CTA eight to start and end; joining in a second kernel costs
  // ten, in a cluster four.  Clusters, of `wide` warps a CTA, where they all run
  // at once, one CTA an SM.
  int best = 1;
  double cost = 1e30;
  for (int s = 1; s <= 128; ++s) {
    const int64_t pp = (pages + s - 1) / s, n = (base * s + sms - 1) / sms;
    if (s > 1 && pp < 4) break;
    if (s == 1 || s * part_bytes <= room) {
      const double c = std::max((double)n * (pp + 3), (double)((n + per_sm - 1) / per_sm) * ((pp + 3) / 4 * 10 + 8)) +
                       (s > 1 ? 10 : 0);
      if (c < cost * 0.999) cost = c, best = s, plan.cluster = false;
    }
    if (s > 1 && s <= kMostCluster && n == 1) {
      const double c = std::max((double)(pp + 3), (double)((pp + wide - 1) / wide * 10 + 8)) + 4;
      if (c < cost * 0.999) cost = c, best = s, plan.cluster = true;
    }
  }
  plan.part_pages = (int)((pages + best - 1) / best);
  plan.n_parts = (int)((pages + plan.part_pages - 1) / plan.part_pages);
  if (plan.n_parts == 1) plan.cluster = false;
  if (plan.n_parts > 1 && !plan.cluster) plan.bytes = plan.n_parts * part_bytes;
  return plan;
}

cudaError_t launch_kv_attend(const csa2_kv_cfg& cfg, int B, KvAtt& a, cudaStream_t stream) {
  const int nt = row_blocks((int64_t)a.max_q * a.group);
  const bool fp4 = cfg.cache_dtype == CSA2_CACHE_FP4, many = (int64_t)a.max_q * a.group > kMostRows;
  const int tile_rows = many ? kv_tiles_rows() : 8 * nt;
  cudaError_t e;
  if (many) e = launch_kv_tiles(cfg, B, a, stream);
  else if (cfg.head_dim == 128) e = fp4 ? launch_rows<128, true>(nt, B, a, stream) : launch_rows<128, false>(nt, B, a, stream);
  else e = fp4 ? launch_rows<64, true>(nt, B, a, stream) : launch_rows<64, false>(nt, B, a, stream);
  if (e != cudaSuccess || a.n_parts <= 1 || a.cluster) return e;
  const int per = (int)(std::min<int64_t>(tile_rows, (int64_t)a.max_q * a.group) + 7) / 8;
  const unsigned grid = (many ? a.tiles - a.whole : (unsigned)B * a.kv_heads) * per;
  return cfg.head_dim == 128 ? launch_k(kv_join_kernel<128>, dim3(grid), dim3(256), 0, stream, 0, a, tile_rows, per)
                             : launch_k(kv_join_kernel<64>, dim3(grid), dim3(256), 0, stream, 0, a, tile_rows, per);
}

}  // namespace csa2
