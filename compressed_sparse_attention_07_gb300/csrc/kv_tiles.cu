// Attention of many query rows over the paged key / value cache (prompts,
// chunks, a decoder's rows over its encoder) on the tensor cores.
//
// One CTA takes one kv head, 256 rows (two tiles of 128; a row is one query
// head at one token) and a part of the keys, 128 at a time:
//   S_j = Q_j K^T  (M = 128 rows, N = 128 keys)   TMEM columns 128 j
//   P_j = exp2(S_j - m) as f16 (bf16 caches: bf16) over S_j, read by
//   O_j += P_j V   (A from TMEM, N = head_dim)    TMEM columns 256 + D j
// with the softmax of tile 0 beside the products of tile 1 and the other way
// round.  A CTA with no more than 128 rows (drafts, short texts) gives both
// places to the same rows and key tiles in turn, and joins the two at the end; with
// no more than 64 rows these stand in the tile twice, each half of the lanes for
// one page of a key tile, which halves the softmax's way.
//
// Warps 0-3 and 4-7 hold the rows (thread = row = TMEM lane, with registers for
// its 128 scores); warps 8-11 bring keys, 12-15 values into shared memory as
// [channel chunk][128 keys][16 B] (copied values: [page][chunk][64 keys][16 B]),
// which is K-major for the first product and MN-major for the second: FP4 decoded
// to f16 on the way, one row a thread, from a ring of pages that warps 18 and 19
// fill with bulk copies; bf16 pages, stored in that order, by bulk copies (warps
// 8-11 and 12).  Warp 16 issues the products (a warp for each place made their
// batches longer, not the pauses between them shorter).  FP4 pages that many
// rows read are decoded ahead by kv_decode_kernel and then taken as bf16 pages are.
//
// The output in TMEM is rescaled only when a row's maximum grew by more than
// 2^8 since its last rescaling (weights up to 2^8 are as exact as those up to
// 1), which after the first keys is rare.  Query rows over FP4 caches are
// scaled by a power of two as in kv_rows.cu.
//
// Measured, 64 over 8 heads of 128 (calls back to back): 2048 tokens on 16384 811 us in
// FP4, 1.44 PFLOP/s (tensor pipe 74 % of the busiest SM's cycles), 835 us in bf16, two
// such in bf16 1.64 ms, 1.43 PFLOP/s.  128 keys of 256 rows are 2048 cycles of products;
// the rest is the way from one product through the softmax to the other, which the other
// place's products cover only in part.  Drafts of 5 tokens on 8 x 32763, FP4: 150 us, a
// key tile of 128 in 2200 cycles of decoding and of the operands' way through shared
// memory (1600).
#include <algorithm>

#include "kv.cuh"
#include "tc.cuh"

namespace csa2 {
namespace {

constexpr int kTileRows = 128, kCtaRows = 256, kTileKeys = 128, kStages = 2;
constexpr int kSoftWarps = 8, kThreads = 640;
constexpr int kKeyWarp = 8, kValueWarp = 12, kProductWarp = 16, kFetchWarp = 18;  // keys 8-11, values 12-15
// registers of a thread: 96 at the launch, then by role (640 x 96 = 256 x 152 + 256 x 48 + 128 x 80)
constexpr int kSoftRegs = 152, kDecodeRegs = 48, kIssueRegs = 80;
// Undecoded tiles on their way (turns: the long ring).  Both even: keys and values
// alternate, so that a place in the ring belongs to one of the two, whose reading
// threads see every one of its phases.
constexpr int kRing = 2, kLongRing = 6, kTailSlots = 3;

template <int D>
struct Tiles {
  static constexpr int kOperand = 128 * D * 2;  // one operand tile
  static constexpr int kQ = 0, kK = 2 * kOperand, kV = kK + kStages * kOperand;
  // undecoded FP4 tiles: the first kTailSlots behind the operands, the others
  // (turns) in the place of the second tile of queries
  static constexpr int kRaw = kV + kStages * kOperand, kRawData = kTileKeys * D / 2, kRawScales = kTileKeys * D / 16;
  static constexpr int kRawTile = kRawData + kRawScales;
  static_assert(kRing % 2 == 0 && kLongRing % 2 == 0 && (kLongRing - kTailSlots) * kRawTile <= kOperand, "the long ring fits");
  // one CTA per SM: it takes all of TMEM
  static constexpr int kSmem = std::max(kRaw + kTailSlots * kRawTile, 120 * 1024);
  __device__ static __forceinline__ int raw(int slot) {
    return slot < kTailSlots ? kRaw + slot * kRawTile : kQ + kOperand + (slot - kTailSlots) * kRawTile;
  }
};

// Rows that read a key (of a sequence of mean length) from which FP4 pages are decoded once for the call, into the
// workspace (up to kMostPlain bytes of it).  Decoding in every CTA takes issue slots
// from the softmax beside it; ahead, a write and reads from L2.  64 over 8 heads of
// 128 on 16384 keys, in passing / ahead: 256 tokens (2048 rows) 138 / 142 us, 512
// 233 / 225, 2048 (keys not divided) 947 / 872; 2 x 4096 on themselves 527 / 480 (GPU
// time in graphs of calls, as at the plan below).
constexpr int64_t kPlainRows = 4096;
constexpr size_t kMostPlain = (size_t)2 << 30;

template <int N>
__device__ __forceinline__ void regs_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// A number that a generic lambda sees at compile time.
template <int N>
struct Num {
  __device__ constexpr int operator()() const { return N; }
};

// Chunk-major operand tile: element (row, channel) at ((c / 8) * 128 + row) * 16 + (c % 8) * 2.
constexpr uint32_t kChunk = 128 * 16;

// kPlain: FP4 pages that kv_decode_kernel has decoded.
template <int D, bool kFp4, bool kPlain>
__global__ void __launch_bounds__(kThreads, 1) kv_tiles_kernel(KvAtt a) {
  using L = Tiles<D>;
  constexpr bool kCodes = kFp4 && !kPlain;  // decoded here
  extern __shared__ __align__(1024) uint8_t smem[];
  __shared__ __align__(8) uint64_t k_full[kStages], v_full[kStages], k_free[kStages], v_free[kStages], s_ready[2],
      p_ready[2], o_full[2];
  __shared__ uint32_t tmem_base;
  __shared__ int late_flag;
  __shared__ __align__(8) uint64_t raw_full[kLongRing], raw_free[kLongRing], tail_full, q_full, drained;
  __shared__ int raw_pages[kLongRing];  // which of a tile's two pages are there
  __shared__ float half_m[2][kTileRows], half_l[2][kTileRows];

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  int id = blockIdx.x, part = 0, kh, b, tile;
  const bool divided = id >= a.whole;
  if (divided) {
    const int x = id - a.whole, q = quotient(x, a.by_parts);
    part = x - q * a.n_parts, id = a.whole + q;
  }
  griddep_wait();
  if (kv_joined(a)) griddep_launch();
  if (!kv_tile(a, kCtaRows, id, b, kh, tile)) return;
  const int tile0 = tile * kCtaRows;
  int row0, rows, keys;
  if (!kv_sequence(a, b, row0, rows, keys)) return;
  const int n_rows = rows * a.group;
  const int last = min(tile0 + kCtaRows, n_rows) - 1;
  int p0, p1;
  kv_pages(a, group_of(a, tile0), group_of(a, last), rows, keys, p0, p1);
  const int part_pages = divided ? a.part_pages : p1 - p0;
  const int n_act = divided ? kv_parts(a, p0, p1) : 1;
  if (part > 0 && part >= n_act) return;
  const int pb = p0 + part * part_pages, pe = min(pb + part_pages, p1);
  const int key0 = pb * kPage;
  const int n_it = (pe - pb + 1) / 2;  // key tiles
  // turns: no second tile of rows, so that place 0 takes the even key tiles of
  // the one there is and place 1 the odd ones
  const bool turns = tile0 + kTileRows >= n_rows;
  // split: no more than 64 rows, which stand in the tile twice: lanes 0-63 take the
  // first page of each key tile, 64-127 the second, half the softmax for each
  const bool split = tile0 + kTileRows / 2 >= n_rows;
  const int32_t* table = a.c.table + (int64_t)b * a.c.max_pages;

  if (tid == 0) {
    for (int s = 0; s < kLongRing; ++s) {
      tc::mbar_init(&raw_full[s], 1);
      tc::mbar_init(&raw_free[s], 4);
    }
    for (int s = 0; s < kStages; ++s) {
      tc::mbar_init(&k_full[s], 4);               // warps
      tc::mbar_init(&v_full[s], kCodes ? 4 : 32);  // warps; or lanes of the one that copies
      tc::mbar_init(&k_free[s], 1);
      tc::mbar_init(&v_free[s], 1);
    }
    for (int j = 0; j < 2; ++j) {
      const int rows_of = n_rows - tile0 - (turns ? 0 : kTileRows * j);  // rows of place j
      const int live = split && rows_of > 32 ? kTileRows : split ? 64 : rows_of;
      tc::mbar_init(&s_ready[j], 1);
      tc::mbar_init(&p_ready[j], max(1, min(4, (live + 31) / 32)));  // warps with rows
      tc::mbar_init(&o_full[j], 1);
    }
    tc::mbar_init(&tail_full, 1);
    tc::mbar_init(&drained, 1);
    tc::mbar_init(&q_full, kSoftWarps);
    late_flag = 0;
    tc::fence_mbar_init();
  }
  if (warp == kProductWarp) {
    tc::tmem_alloc(&tmem_base, 512);
    tc::tmem_relinquish();
  }

  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tb = tmem_base;
  const uint32_t sbase = tc::smem_u32(smem);
  bool ok = true;
  // one arrival for a warp, once all its lanes are here
  auto warp_arrive = [&](uint64_t* bar) {
    __syncwarp();
    if (lane == 0) tc::mbar_arrive(bar);
  };

  if (warp < kSoftWarps) {
    // ---------------------------------------------------------- softmax --
    regs_inc<kSoftRegs>();
    // the query rows, f16 (bf16 caches: bf16)
    float scale;
    int hi = 0, lo = 0;
    const int r = tile0 + (split ? tid % (kTileRows / 2) : turns ? tid % kTileRows : tid);
    if (r < n_rows) hi = kv_hi(a, group_of(a, r), rows, keys), lo = kv_lo(a, group_of(a, r), rows, keys);
    {
      // A lane loads parts of four rows, 8 x + its number & 7 of the warp's: 64
      // neighbouring bytes of eight rows at a time (a lane with a row to itself, 16
      // bytes of 32 rows at a time, took 8 000 cycles for 64 channels), and eight
      // lanes store the same chunk of neighbouring rows.
      const int sub = lane & 7, c0 = lane >> 3;
      const uint32_t sign = a.scale < 0.0f ? 0x80008000u : 0u;  // into the query: the scale is positive below
      scale = fabsf(a.scale) * kLog2e;
      uint4 w[4][D / 32];
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const int rr = r - lane + 8 * x + sub;
        const bool live = rr < n_rows;
        const uint16_t* q = a.q;
        if (live) q += (int64_t)(row0 + group_of(a, rr)) * a.q_stride + (kh * a.group + rr - group_of(a, rr) * a.group) * D;
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
          w[x][c] = make_uint4(0, 0, 0, 0);
          if (live) w[x][c] = __ldg(reinterpret_cast<const uint4*>(q) + 4 * c + c0);
        }
      }
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        float down = 1.0f;
        if constexpr (kFp4) {
          uint32_t most = 0;
#pragma unroll
          for (int c = 0; c < D / 32; ++c) {
            const uint32_t u[4] = {w[x][c].x, w[x][c].y, w[x][c].z, w[x][c].w};
#pragma unroll
            for (int y = 0; y < 4; ++y) most = max(most, max(u[y] & 0x7F80u, (u[y] >> 16) & 0x7F80u));
          }
          most = max(most, __shfl_xor_sync(0xffffffffu, most, 8));
          most = max(most, __shfl_xor_sync(0xffffffffu, most, 16));
          // the largest channel's exponent, biased, where its power of two and the
          // inverse are both normal numbers
          const uint32_t e = min(max(most >> 7, 1u), 253u);
          down = __uint_as_float((254u - e) << 23);
          if (c0 == x) scale *= __uint_as_float(e << 23);  // this lane's own row
        }
        if (!turns || tid < kTileRows) {
          uint8_t* dst = smem + L::kQ + (tid / kTileRows) * L::kOperand + (32 * (warp & 3) + 8 * x + sub) * 16;
#pragma unroll
          for (int c = 0; c < D / 32; ++c) {
            uint32_t u[4] = {w[x][c].x, w[x][c].y, w[x][c].z, w[x][c].w};
#pragma unroll
            for (int y = 0; y < 4; ++y) {
              if constexpr (kFp4)
                u[y] = f16x2(__uint_as_float(u[y] << 16) * down, __uint_as_float(u[y] & 0xFFFF0000u) * down);
              u[y] ^= sign;
            }
            *reinterpret_cast<uint4*>(dst + (4 * c + c0) * kChunk) = make_uint4(u[0], u[1], u[2], u[3]);
          }
        }
      }
      scale = fmaxf(scale, 1e-37f);  // above 0: a hidden key's -inf stays -inf
    }
    tc::fence_async_smem();
    warp_arrive(&q_full);
    const int j = warp / 4;
    const uint32_t lane_base = 32 * (warp & 3);
    const uint32_t s_addr = tc::taddr(tb, lane_base, 128 * j), o_addr = tc::taddr(tb, lane_base, 256 + D * j);
    const bool warp_live = r - lane < n_rows;
    float m = -INFINITY, l = 0.0f;
    // this place's key tiles: 32 kChunks keys of each from 32 first on
    auto soft = [&](auto chunks, int first) {
      constexpr int kChunks = chunks();
      int u = 0;  // key tiles so far
      for (int it = turns ? j : 0; it < n_it; it += turns ? 2 : 1, ++u) {
        const int k0 = key0 + it * kTileKeys;
        int v_lo = lo - k0, v_hi = hi - k0;  // the row's keys in this tile
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const int pg = pb + 2 * it + x;
          if (pg >= pe) {
            v_hi = min(v_hi, 64 * x);
          } else {
            const int32_t id = __ldg(table + pg);
            if (id < 0 || id >= a.c.num_pages) {
              if (x == 0) v_lo = max(v_lo, 64);
              else v_hi = min(v_hi, 64);
            }
          }
        }
        v_lo -= 32 * first, v_hi -= 32 * first;
        const bool masked = __any_sync(0xffffffffu, v_lo > 0 || v_hi < 32 * kChunks);
        if (!__all_sync(0xffffffffu, tc::mbar_wait(&s_ready[j], u & 1))) {
          ok = false;
          return;
        }
        tc::fence_after_sync();
        uint32_t s[kChunks][32];
#pragma unroll
        for (int c = 0; c < kChunks; ++c) tc::tmem_ld32(s_addr + 32 * (first + c), s[c]);
        tc::tmem_wait_ld();
        if (masked) {
#pragma unroll
          for (int c = 0; c < kChunks; ++c) {
            const int from = min(max(v_lo - 32 * c, 0), 32), to = min(max(v_hi - 32 * c, 0), 32);
            const uint32_t bits = (uint32_t)((1ull << to) - 1) & (uint32_t)(0xFFFFFFFFull << from);
#pragma unroll
            for (int x = 0; x < 32; ++x)
              if (!(bits & (1u << x))) s[c][x] = 0xFF800000u;  // -inf
          }
        }
        constexpr int kRun = 8 * kChunks;  // four maxima at once
        float t4[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          t4[c] = __uint_as_float(s[c * kRun / 32][c * kRun % 32]);
#pragma unroll
          for (int x = 1; x < kRun; ++x) t4[c] = fmaxf(t4[c], __uint_as_float(s[(c * kRun + x) / 32][(c * kRun + x) % 32]));
        }
        float top = fmaxf(fmaxf(t4[0], t4[1]), fmaxf(t4[2], t4[3]));
        if (top > -INFINITY) top *= scale;
        const bool grew = top > m + 8.0f || (m == -INFINITY && top > -INFINITY);
        if (__any_sync(0xffffffffu, grew)) {
          const float f = (grew && m > -INFINITY) ? ex2(m - top) : 1.0f;
          if (grew) m = top;
          l *= f;
          if (u > 0) {
#pragma unroll 1
            for (int c = 0; c < D / 16; ++c) {
              uint32_t o[16];
              tc::tmem_ld16(o_addr + 16 * c, o);
              tc::tmem_wait_ld();
#pragma unroll
              for (int x = 0; x < 16; ++x) o[x] = __float_as_uint(__uint_as_float(o[x]) * f);
              tc::tmem_st16(o_addr + 16 * c, o);
            }
          }
        }
        const uint64_t scale2 = pack2(scale, scale);
        const float z = m == -INFINITY ? 0.0f : -m;
        const uint64_t z2 = pack2(z, z);
        uint64_t sum[2] = {pack2(l, 0.0f), 0ull};
#pragma unroll
        for (int c = 0; c < kChunks; ++c) {
          uint32_t p[16];
#pragma unroll
          for (int x = 0; x < 16; ++x) {
            float y0, y1;
            unpack2(fma2(pack2(__uint_as_float(s[c][2 * x]), __uint_as_float(s[c][2 * x + 1])), scale2, z2), y0, y1);
            y0 = ex2(y0), y1 = ex2(y1);
            sum[x & 1] = add2(sum[x & 1], pack2(y0, y1));
            p[x] = kFp4 ? f16x2(y0, y1) : bf16x2(y0, y1);
          }
          tc::tmem_st16(s_addr + 16 * (first + c), p);
        }
        if constexpr (kChunks == 2) {  // the other lanes' keys
          const uint32_t none[16] = {};
          tc::tmem_st16(s_addr + 16 * (2 - first), none);
          tc::tmem_st16(s_addr + 16 * (3 - first), none);
        }
        {
          float y0, y1;
          unpack2(add2(sum[0], sum[1]), y0, y1);
          l = y0 + y1;
        }
        tc::tmem_wait_st();
        tc::fence_before_sync();
        warp_arrive(&p_ready[j]);
      }
    };
    const int half = (warp >> 1) & 1;
    if (warp_live) {
      if (split) soft(Num<2>{}, 2 * half);
      else soft(Num<4>{}, 0);
    }
    // ---- the rows' outputs: place 0's, place 1's, or (turns) both for one row
    float f[2] = {0.0f, 0.0f};  // factors of the places' outputs
    f[j] = 1.0f;
    if (turns) {
      const int at = tid % kTileRows;
      half_m[j][at] = m, half_l[j][at] = l;
      asm volatile("bar.sync 1, 256;" ::: "memory");
      const float m0 = half_m[0][at], m1 = half_m[1][at], n0 = half_m[0][at ^ 64], n1 = half_m[1][at ^ 64];
      m = fmaxf(m0, m1);
      if (split) m = fmaxf(m, fmaxf(n0, n1));
      f[0] = m0 == -INFINITY ? 0.0f : ex2(m0 - m);
      f[1] = m1 == -INFINITY ? 0.0f : ex2(m1 - m);
      l = f[0] * half_l[0][at] + f[1] * half_l[1][at];
      if (split)
        l += (n0 == -INFINITY ? 0.0f : ex2(n0 - m)) * half_l[0][at ^ 64] + (n1 == -INFINITY ? 0.0f : ex2(n1 - m)) * half_l[1][at ^ 64];
    }
    bool write = false;  // the products are over and this warp has rows
    if (warp_live && ok) {
      // The outputs pass through the queries' place: the products have read them, or
      // (rows that see nothing) every warp has stored its own.
      if (n_it == 0) ok = tc::mbar_wait(&q_full, 0);
      else if (!turns) ok = tc::mbar_wait(&o_full[j], 0);
      else ok = tc::mbar_wait(&o_full[0], 0) && (n_it < 2 || tc::mbar_wait(&o_full[1], 0));
      ok = __all_sync(0xffffffffu, ok);
      write = ok;
      tc::fence_after_sync();
    }
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
    const float g0 = inv * (turns ? f[0] : 1.0f), g1 = inv * f[1];
    const uint32_t o0 = tc::taddr(tb, lane_base, 256), o1 = tc::taddr(tb, lane_base, 256 + D);
    auto take = [&](int c, uint32_t (&o)[32]) {  // this lane's share of 32 channels of the output
      if (n_it > 0) {
        tc::tmem_ld32((j == 1 && !turns ? o1 : o0) + 32 * c, o);
        tc::tmem_wait_ld();
#pragma unroll
        for (int x = 0; x < 32; ++x) o[x] = __float_as_uint(__uint_as_float(o[x]) * g0);
      }
      if (turns && n_it > 1) {
        uint32_t o2[32];
        tc::tmem_ld32(o1 + 32 * c, o2);
        tc::tmem_wait_ld();
#pragma unroll
        for (int x = 0; x < 32; ++x) o[x] = __float_as_uint(fmaf(__uint_as_float(o2[x]), g1, __uint_as_float(o[x])));
      }
      if (l == 0.0f) {
#pragma unroll
        for (int x = 0; x < 32; ++x) o[x] = 0u;
      }
    };
    // (turns) each place writes one half of the channels; (split) lanes 64-127 hand
    // theirs over first, in the place of the keys, which are done with
    float* other = reinterpret_cast<float*>(smem + L::kK) + tid % (kTileRows / 2);
    if (split) {
      if (write && half) {
#pragma unroll 1
        for (int c = j * (D / 64); c < (j + 1) * (D / 64); ++c) {
          uint32_t o[32];
          take(c, o);
#pragma unroll
          for (int x = 0; x < 32; ++x) other[(32 * c + x) * (kTileRows / 2)] = __uint_as_float(o[x]);
        }
      }
      asm volatile("bar.sync 2, 256;" ::: "memory");
      if (half) write = false;
    }
    if (write) {
      const bool live = r < n_rows;
      const int i = row0 + (live ? group_of(a, r) : 0), h = kh * a.group + (live ? r - group_of(a, r) * a.group : 0);
      const int64_t at = (int64_t)i * a.n_heads + h, pa = part * a.part_step + kv_part_row(a, id, r, tile0, at);
      const bool whole = n_act <= 1;
      const float lse2 = l == 0.0f ? -INFINITY : m + log2f(l);
      if (live && (!turns || j == 0)) {
        if (!whole) a.part_l[pa] = lse2;
        else if (a.lse) a.lse[at] = lse2 * kLn2;
      }
      // where this lane's row goes, or 0
      const uint64_t home = !live ? 0 : whole ? reinterpret_cast<uint64_t>(a.out + (int64_t)i * a.out_stride + h * D)
                                              : reinterpret_cast<uint64_t>(a.part_o + pa * D);
      // The rows pass through shared memory (the place's queries are done with),
      // so that neighbouring lanes write neighbouring 16 bytes of a row: its unit x
      // of 64 bytes stands at x ^ (row / 2 & 3).
      uint8_t* pad = smem + L::kQ + j * L::kOperand + (warp & 3) * 2048;
      uint64_t to[4];  // four lanes a row, eight rows at a time
#pragma unroll
      for (int x = 0; x < 4; ++x) to[x] = __shfl_sync(0xffffffffu, home, 8 * x + lane / 4);
      auto pass = [&](const uint32_t* w, int offset) {  // 64 bytes of each row, to `offset` in it
        __syncwarp();
#pragma unroll
        for (int x = 0; x < 4; ++x)
          *reinterpret_cast<uint4*>(pad + lane * 64 + ((x ^ ((lane >> 1) & 3)) * 16)) =
              make_uint4(w[4 * x], w[4 * x + 1], w[4 * x + 2], w[4 * x + 3]);
        __syncwarp();
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const int row = 8 * x + lane / 4, unit = lane & 3;
          const uint4 v = *reinterpret_cast<const uint4*>(pad + row * 64 + ((unit ^ ((row >> 1) & 3)) * 16));
          if (to[x]) *reinterpret_cast<uint4*>(to[x] + offset + 16 * unit) = v;
        }
      };
#pragma unroll 1
      for (int c = turns ? j * (D / 64) : 0; c < (turns ? (j + 1) * (D / 64) : D / 32); ++c) {
        uint32_t o[32];
        take(c, o);
        if (split) {
#pragma unroll
          for (int x = 0; x < 32; ++x)
            o[x] = __float_as_uint(__uint_as_float(o[x]) + other[(32 * c + x) * (kTileRows / 2)]);
        }
        if (whole) {
          uint32_t u[16];
#pragma unroll
          for (int x = 0; x < 16; ++x) u[x] = bf16x2(__uint_as_float(o[2 * x]), __uint_as_float(o[2 * x + 1]));
          pass(u, 64 * c);
        } else {
          pass(o, 128 * c);
          pass(o + 16, 128 * c + 64);
        }
      }
    }
  } else if (warp < kProductWarp) {
    regs_dec<kDecodeRegs>();
    const int ring = turns ? kLongRing : kRing;
    if (kCodes) {
      // -------------------------------------------------------- decoding --
      // a row of each tile for each thread: warps 8-11 keys, 12-15 values
      constexpr int W = D / 32;  // 16-byte pieces of a row
      const bool v = warp >= kValueWarp;
      const int key = tid % kTileKeys;
      // The pieces are taken from another one on by each few keys, so that the
      // eight keys of a quarter warp's read lie in different banks.
      const int turn = key / (256 / D);
      for (int it = 0; it < n_it; ++it) {
        const int op = 2 * it + v, slot = op % ring, s = it % kStages;
        ok = __all_sync(0xffffffffu, tc::mbar_wait(&raw_full[slot], (op / ring) & 1));
        if (!ok) break;
        const uint8_t* raw = smem + L::raw(slot);
        const bool seen = key0 + it * kTileKeys + key < keys && pb + 2 * it + key / 64 < pe && ((raw_pages[slot] >> (key / 64)) & 1);
        uint4 w[W];
        uint32_t f[W];
#pragma unroll
        for (int x = 0; x < W; ++x) {
          const int piece = (x + turn) % W;
          w[x] = *reinterpret_cast<const uint4*>(raw + key * (D / 2) + piece * 16);
          f[x] = *reinterpret_cast<const uint16_t*>(raw + L::kRawData + key * (D / 16) + 2 * piece);
          if (!seen) w[x] = make_uint4(0, 0, 0, 0), f[x] = 0;  // not there: anything
        }
        warp_arrive(&raw_free[slot]);
        if (it >= kStages) {
          ok = __all_sync(0xffffffffu, tc::mbar_wait(v ? &v_free[s] : &k_free[s], ((it / kStages) & 1) ^ 1));
          if (!ok) break;
        }
        uint8_t* dst = smem + (v ? L::kV : L::kK) + s * L::kOperand + key * 16;
#pragma unroll
        for (int x = 0; x < W; ++x) {  // 32 channels: two scales, four chunks
          uint8_t* at = dst + ((x + turn) % W) * (4 * kChunk);
          const uint32_t c[4] = {w[x].x, w[x].y, w[x].z, w[x].w};
          const uint32_t sc = scales2(f[x]);
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            uint32_t h[4];
            codes8(c[y], h);
            const uint32_t one = __byte_perm(sc, 0, y < 2 ? 0x1010u : 0x3232u);
            *reinterpret_cast<uint4*>(at + y * kChunk) =
                make_uint4(mul2(h[0], one), mul2(h[1], one), mul2(h[2], one), mul2(h[3], one));
          }
        }
        tc::fence_async_smem();
        warp_arrive(v ? &v_full[s] : &k_full[s]);
      }
    } else if (warp <= kValueWarp) {
      // ---- pages as they are: keys by four warps, each a quarter of the chunks (a copy
      // of 1 KB takes a warp some 90 cycles), values, a page at once, by one
      const bool v = warp == kValueWarp;
      uint64_t* full = v ? v_full : k_full;
      uint64_t* free_ = v ? v_free : k_free;
      int it = 0;
      for (; it < n_it; ++it) {
        const int s = it % kStages;
        uint8_t* dst = smem + (v ? L::kV : L::kK) + s * L::kOperand;
        if (it >= kStages && !__all_sync(0xffffffffu, tc::mbar_wait(&free_[s], ((it / kStages) & 1) ^ 1))) {
          ok = false;
          break;
        }
        int64_t at[2];  // the tile's pages; -1: not there
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const int pg = pb + 2 * it + x;
          if constexpr (kPlain) {
            at[x] = pg < pe ? (((int64_t)b * a.plain_pages + pg) * a.kv_heads + kh) * kv_block_bytes(D, false) : -1;
            continue;
          }
          const int32_t page = pg < pe ? __ldg(table + pg) : -1;
          const bool there = page >= 0 && page < a.c.num_pages;
          if (pg < pe && !there && lane == 0) report(a.status, CSA2_ERR_BAD_PAGE);
          at[x] = there ? ((int64_t)page * a.kv_heads + kh) * kv_block_bytes(D, false) : -1;
        }
        // Scores of keys that are not seen are never used, but values are
        // multiplied by weight 0: what lies in slots from kv_len on (anything) and
        // in the place of a page outside the pool has to be 0 (and is in plain pages).
        const int live = keys - key0 - it * kTileKeys;
        const bool tail = !kPlain && v && live < kTileKeys && (live < kPage ? at[0] : at[1]) >= 0;
        uint64_t* bar = tail ? &tail_full : &full[s];
        if (lane == 0) tc::mbar_arrive_expect_tx(bar, ((at[0] >= 0) + (at[1] >= 0)) * (L::kOperand / (v ? 2 : 8)));
        __syncwarp();
        if (tc::elect_one()) {
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            if (at[x] < 0) continue;
            if (v) {
              tc::bulk_g2s(dst + x * (L::kOperand / 2), (kPlain ? a.plain_v : a.c.v) + at[x], L::kOperand / 2, bar);
              continue;
            }
#pragma unroll
            for (int y = 0; y < D / 32; ++y) {
              const int c = (warp - kKeyWarp) * (D / 32) + y;
              tc::bulk_g2s(dst + c * kChunk + x * (kPage * 16), (kPlain ? a.plain_k : a.c.k) + at[x] + c * (kPage * 16),
                           kPage * 16, bar);
            }
          }
        }
        __syncwarp();
        if (v) {
          auto clear = [&](int from, int to) {  // values of these keys
            for (int key = from + lane; key < to; key += 32)
#pragma unroll
              for (int c = 0; c < D / 8; ++c)
                *reinterpret_cast<uint4*>(dst + key / kPage * (L::kOperand / 2) + (c * kPage + key % kPage) * 16) =
                    make_uint4(0, 0, 0, 0);
            tc::fence_async_smem();
          };
          if (tail) {  // the last tile
            ok = __all_sync(0xffffffffu, tc::mbar_wait(&tail_full, 0));
            if (!ok) break;
            clear(live, live < kPage ? kPage : kTileKeys);
          }
          if (!kPlain && at[0] < 0) clear(0, kPage);
          if (!kPlain && at[1] < 0 && pb + 2 * it + 1 < pe) clear(kPage, kTileKeys);
          if (lane != 0 || tail) tc::mbar_arrive(&full[s]);
        }
      }
      // nothing may land in shared memory after the CTA has left
      for (int i = max(0, it - kStages); !ok && i < it; ++i) tc::mbar_wait(&full[i % kStages], (i / kStages) & 1);
    }
  } else {
    regs_dec<kIssueRegs>();
    const int ring = turns ? kLongRing : kRing;
    if (warp == kProductWarp && n_it > 0) {
      // ------------------------------------------------------- products --
      constexpr uint32_t kIdS = tc::idesc_f16(128, kTileKeys, !kFp4, !kFp4, false, false);
      constexpr uint32_t kIdO = tc::idesc_f16(128, D, !kFp4, !kFp4, false, true);
      // values decoded: 128 keys of a chunk together; copied: 64, a page after the other
      constexpr uint32_t kHiK = tc::sdesc_hi(128), kHiV = tc::sdesc_hi(kCodes ? kChunk : kChunk / 2);
      constexpr uint32_t kTile16 = L::kOperand / 16;
      static_assert(kStages == 2, "the loops below go over two key tiles");
      // Place and stage are compile-time numbers, the descriptors' low words formed
      // once: see tc.cuh.
      const uint32_t q_lo = tc::sdesc_lo(sbase + L::kQ, kChunk), k_lo = tc::sdesc_lo(sbase + L::kK, kChunk);
      const uint32_t v_lo = tc::sdesc_lo(sbase + L::kV, 128);
      auto wait = [&](uint64_t* bar, int parity) { return __all_sync(0xffffffffu, tc::mbar_wait(bar, parity)); };
      // S_j = Q_q K^T with the keys of stage s, the last to read them if `over`
      auto scores = [&](auto q, auto j, auto s, bool over) {
        tc::fence_after_sync();
        if (tc::elect_one()) {
#pragma unroll
          for (int ks = 0; ks < D / 16; ++ks)
            tc::mma_ss_lo(tb + 128 * j(), q_lo + q() * kTile16 + ks * (2 * kChunk / 16),
                          k_lo + s() * kTile16 + ks * (2 * kChunk / 16), kHiK, kHiK, kIdS, ks > 0);
          tc::mma_commit(&s_ready[j()]);
          if (over) tc::mma_commit(&k_free[s()]);
        }
        __syncwarp();
      };
      // O_j += P_j V with the values of stage s, the u-th tile of place j
      // (half: the tile has one page)
      auto outputs = [&](auto j, auto s, int u, uint64_t* done, bool half) {
        tc::fence_after_sync();
        if (tc::elect_one()) {
          tc::mma_ts_lo(tb + 256 + D * j(), tb + 128 * j(), v_lo + s() * kTile16, kHiV, kIdO, u > 0);
#pragma unroll
          for (int ks = 1; ks < kTileKeys / 16; ++ks) {
            if (ks >= kPage / 16 && half) break;
            tc::mma_ts_lo(tb + 256 + D * j(), tb + 128 * j() + 8 * ks, v_lo + s() * kTile16 + ks * (256 / 16) + (kCodes || ks < kPage / 16 ? 0 : kTile16 / 2 - kPage),
                          kHiV, kIdO,
                          1u);
          }
          if (done) tc::mma_commit(done);
        }
        __syncwarp();
      };
      const bool odd = (pe - pb) & 1;  // the last tile has one page
      ok = wait(&q_full, 0);
      if (turns) {
        // tile `it`, of stage and place s, and the outputs of the place's last one
        auto step = [&](auto s, int it) {
          ok = wait(&k_full[s()], (it / kStages) & 1);
          if (it >= 2) {
            ok = ok && wait(&v_full[s()], (it / kStages - 1) & 1) && wait(&p_ready[s()], (it / 2 - 1) & 1);
            if (ok) outputs(s, s, it / 2 - 1, &v_free[s()], false);
          }
          if (ok) scores(Num<0>{}, s, s, true);
        };
        auto end = [&](auto s, int it) {
          ok = wait(&v_full[s()], (it / kStages) & 1) && wait(&p_ready[s()], (it / 2) & 1);
          if (ok) outputs(s, s, it / 2, &o_full[s()], odd && it == n_it - 1);
        };
        for (int it = 0; it < n_it && ok; it += 2) {
          step(Num<0>{}, it);
          if (ok && it + 1 < n_it) step(Num<1>{}, it + 1);
        }
        for (int it = max(0, n_it - 2); it < n_it && ok; ++it) {
          if (it & 1) end(Num<1>{}, it);
          else end(Num<0>{}, it);
        }
      } else {
        // tile `it` (stage s), and the outputs of the one before it (stage p)
        auto step = [&](auto s, auto p, int it) {
          ok = wait(&k_full[s()], (it / kStages) & 1);
          if (it > 0) {
            ok = ok && wait(&v_full[p()], ((it - 1) / kStages) & 1) && wait(&p_ready[0], (it - 1) & 1);
            if (ok) outputs(Num<0>{}, p, it - 1, nullptr, false);
          }
          if (ok) scores(Num<0>{}, Num<0>{}, s, false);
          if (it > 0) {
            ok = ok && wait(&p_ready[1], (it - 1) & 1);
            if (ok) outputs(Num<1>{}, p, it - 1, &v_free[p()], false);
          }
          if (ok) scores(Num<1>{}, Num<1>{}, s, true);
        };
        auto end = [&](auto s) {
          ok = wait(&v_full[s()], ((n_it - 1) / kStages) & 1) && wait(&p_ready[0], (n_it - 1) & 1);
          if (ok) outputs(Num<0>{}, s, n_it - 1, &o_full[0], odd);
          ok = ok && wait(&p_ready[1], (n_it - 1) & 1);
          if (ok) outputs(Num<1>{}, s, n_it - 1, &o_full[1], odd);
        };
        for (int it = 0; it < n_it && ok; it += 2) {
          step(Num<0>{}, Num<1>{}, it);
          if (ok && it + 1 < n_it) step(Num<1>{}, Num<0>{}, it + 1);
        }
        if (ok) {
          if (n_it & 1) end(Num<0>{});
          else end(Num<1>{});
        }
      }
      if (!ok) {  // nothing may run on after TMEM is given back
        if (tc::elect_one()) tc::mma_commit(&drained);
        __syncwarp();
        tc::mbar_wait(&drained, 0);
      }
    } else if (kCodes && (warp == kFetchWarp || warp == kFetchWarp + 1)) {
      // ---------------- pages into the ring (K, V, K ..), a warp for each --
      const bool v = warp != kFetchWarp;
      int32_t id[2], next[2] = {-1, -1};
      auto find = [&](int it) {
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const int pg = pb + 2 * it + x;
          next[x] = it < n_it && pg < pe ? __ldg(table + pg) : -1;
        }
      };
      find(0);
      for (int it = 0; it < n_it; ++it) {
        const int op = 2 * it + v, slot = op % ring;
        id[0] = next[0], id[1] = next[1];
        find(it + 1);
        const bool bad = id[0] < 0 || id[0] >= a.c.num_pages ||
                         (pb + 2 * it + 1 < pe && (id[1] < 0 || id[1] >= a.c.num_pages));
        if (bad && lane == 0) report(a.status, CSA2_ERR_BAD_PAGE);
        if (op >= ring && !__all_sync(0xffffffffu, tc::mbar_wait(&raw_free[slot], ((op / ring) & 1) ^ 1))) {
          ok = false;
          break;
        }
        const int there = (id[0] >= 0 && id[0] < a.c.num_pages ? 1 : 0) | (id[1] >= 0 && id[1] < a.c.num_pages ? 2 : 0);
        if (lane == 0) {
          raw_pages[slot] = there;
          tc::mbar_arrive_expect_tx(&raw_full[slot], __popc(there) * (L::kRawTile / 2));
        }
        __syncwarp();
        if (tc::elect_one()) {
          uint8_t* dst = smem + L::raw(slot);
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            if (!((there >> x) & 1)) continue;
            const int64_t block = (int64_t)id[x] * a.kv_heads + kh;
            tc::bulk_g2s(dst + x * (L::kRawData / 2), (v ? a.c.v : a.c.k) + block * (L::kRawData / 2), L::kRawData / 2,
                         &raw_full[slot]);
            tc::bulk_g2s(dst + L::kRawData + x * (L::kRawScales / 2), (v ? a.c.vs : a.c.ks) + block * (L::kRawScales / 2),
                         L::kRawScales / 2, &raw_full[slot]);
          }
        }
        __syncwarp();
      }
      // nothing may land in shared memory after the CTA has left
      for (int op = max(0, 2 * n_it - ring); !ok && op < 2 * n_it; ++op)
        tc::mbar_wait(&raw_full[op % ring], (op / ring) & 1);
    }
  }
  __syncwarp();
  if (!ok) late_flag = 1;
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  if (tid == 0 && late_flag) report(a.status, CSA2_ERR_TIMEOUT);
  if (warp == kProductWarp) tc::tmem_dealloc(tb, 512);
}

// The FP4 pages that a sequence's rows see, as f16 in a BF16 page's order; slots from
// kv_len on and pages outside the pool are 0.  A CTA for a page and kv head: four (two)
// threads a key, 32 channels each, read neighbouring 16 bytes and write neighbouring 16
// bytes of eight (16) keys.  Bound by latency and L2's writes: 8704 keys of 8 heads of 128
// (46 MB) in 10.5 us.
template <int D>
__global__ void __launch_bounds__(256) kv_decode_kernel(KvAtt a) {
  griddep_wait();
  griddep_launch();
  const int pg = blockIdx.x, kh = blockIdx.y, b = blockIdx.z;
  int row0, rows, keys, p0, p1;
  if (!kv_sequence(a, b, row0, rows, keys) || rows == 0) return;
  kv_pages(a, 0, rows - 1, rows, keys, p0, p1);
  if (pg < p0 || pg >= p1) return;
  const int32_t page = __ldg(a.c.table + (int64_t)b * a.c.max_pages + pg);
  const bool there = page >= 0 && page < a.c.num_pages;
  if (!there && threadIdx.x == 0) report(a.status, CSA2_ERR_BAD_PAGE);
  constexpr int W = D / 32;  // 16-byte pieces of a key
  const int64_t block = (int64_t)page * a.kv_heads + kh;
  const int64_t to = (((int64_t)b * a.plain_pages + pg) * a.kv_heads + kh) * kv_block_bytes(D, false);
#pragma unroll
  for (int i0 = 0; i0 < 2 * kPage * W; i0 += 256) {
    const int i = i0 + threadIdx.x, piece = i % W, key = i / W % kPage;
    const bool v = i >= kPage * W;
    uint4 w = make_uint4(0, 0, 0, 0);
    uint32_t sc = 0;
    if (there && pg * kPage + key < keys) {
      w = __ldg(reinterpret_cast<const uint4*>((v ? a.c.v : a.c.k) + block * kv_block_bytes(D, true) + key * (D / 2)) + piece);
      sc = scales2(__ldg(reinterpret_cast<const uint16_t*>((v ? a.c.vs : a.c.ks) + block * kv_scale_bytes(D) + key * (D / 16)) + piece));
    }
    uint8_t* dst = (v ? a.plain_v : a.plain_k) + to + (4 * piece * kPage + key) * 16;
    const uint32_t c[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int y = 0; y < 4; ++y) {
      uint32_t h[4];
      codes8(c[y], h);
      const uint32_t one = __byte_perm(sc, 0, y < 2 ? 0x1010u : 0x3232u);
      *reinterpret_cast<uint4*>(dst + y * (kPage * 16)) =
          make_uint4(mul2(h[0], one), mul2(h[1], one), mul2(h[2], one), mul2(h[3], one));
    }
  }
}

template <int D, bool kFp4, bool kPlain>
cudaError_t launch(int B, const KvAtt& a, cudaStream_t stream) {
  auto kern = kv_tiles_kernel<D, kFp4, kPlain>;
  static std::atomic<bool> done[64];
  cudaError_t e = allow_smem(kern, Tiles<D>::kSmem, done);
  if (e != cudaSuccess) return e;
  if constexpr (kPlain) {
    e = launch_k(kv_decode_kernel<D>, dim3(a.plain_pages, a.kv_heads, B), dim3(256), 0, stream, 0, a);
    if (e != cudaSuccess) return e;
  }
  const dim3 grid(a.whole + (unsigned)(a.tiles - a.whole) * a.n_parts);
  return launch_k(kern, grid, dim3(kThreads), Tiles<D>::kSmem, stream, 0, a);
}

}  // namespace

// Partial outputs stand by row and head of the batch up to this many bytes of them, else
// only the divided tiles' rows, tile by tile, where that is less: 2048 tokens on 16384 (64
// over 8 heads of 128, 56 of 512 tiles in five parts) take 37 MB instead of 338.
constexpr size_t kMostByRow = (size_t)64 << 20;

KvPlan kv_tiles_plan(const csa2_kv_cfg& cfg, int B, int T, int max_q, int64_t max_kv, bool cross, size_t room) {
  const int group = cfg.n_heads / cfg.kv_heads;
  const int64_t rows = (int64_t)max_q * group;
  // at most: each sequence's longest, or what all rows fill and a last one each
  const int64_t tiles = std::min(B * ((rows + kCtaRows - 1) / kCtaRows), (int64_t)T * group / kCtaRows + B);
  int64_t pages = (max_kv + kPage - 1) / kPage;
  if (cfg.window && !cross)
    pages = std::min<int64_t>(pages, ((int64_t)cfg.window + std::min<int64_t>(max_q, kCtaRows / group + 2) + kPage - 2) / kPage + 1);
  const int64_t steps = std::max<int64_t>(1, (pages + 1) / 2), base = cfg.kv_heads * tiles, slots = num_sms();
  // The number of parts whose waves of CTAs end soonest, in key tiles: a CTA's start
  // and end cost about three, the joining kernel two and its reading two and a half
  // for each CTA of an SM.  Divided are all row tiles, or those of the last wave, if
  // it wins 3 %: 2048 tokens on 16384 (64 over 8 heads of 128, FP4 decoded ahead; 512
  // tiles, the last 56 in five parts) take 806 us so and 872 us whole, three such
  // sequences of 512 tokens 637 and 665.
  const double read = 2.5 * std::min<int64_t>(rows, kCtaRows) / kCtaRows / slots;
  const int64_t tile_rows = std::min<int64_t>(rows, kCtaRows), all = (int64_t)T * cfg.n_heads;
  const size_t row_bytes = (size_t)(cfg.head_dim + 1) * 4;
  // rows of a part, with `rest` tiles divided in s; by_tile: tile by tile
  auto part_step = [&](int64_t s, int64_t rest, bool* by_tile) {
    *by_tile = rest * tile_rows < all && s * all * row_bytes > std::min(room, kMostByRow);
    return *by_tile ? rest * tile_rows : all;
  };
  int64_t best = 1, whole = 0;
  bool by_tile = false;
  double cost = 1e30;
  for (int64_t s = 1; s <= 64; ++s) {
    const int64_t n = (steps + s - 1) / s;
    if (s > 1 && n < 2) break;
    for (const int64_t w : {(int64_t)0, base / slots * slots}) {
      const int64_t rest = base - w;
      if (w && (s == 1 || rest == 0)) continue;
      if (s > 1 && s * part_step(s, rest, &by_tile) * row_bytes > room) continue;
      const double c = (double)(w / slots) * (steps + 3) + (double)((rest * s + slots - 1) / slots) * (n + 3) +
                       (s > 1 ? 2 + read * rest * s : 0);
      if (c < cost * 0.999) cost = s == 1 ? 0.97 * c : c, best = s, whole = w;
    }
  }
  const int64_t per = (steps + best - 1) / best, parts = (steps + per - 1) / per;
  if (parts == 1) whole = 0;
  const int64_t ctas = whole + (base - whole) * std::max<int64_t>(parts, parts > 1 ? kCtaRows / 8 : 1);
  const int64_t step = part_step(parts, base - whole, &by_tile);
  return KvPlan{(int)parts, (int)(2 * per), false, base, whole, ctas, step, by_tile ? (int)tile_rows : 0,
                parts > 1 ? parts * step * row_bytes : 0};
}

cudaError_t launch_kv_tiles(const csa2_kv_cfg& cfg, int B, const KvAtt& a, cudaStream_t stream) {
  const bool fp4 = cfg.cache_dtype == CSA2_CACHE_FP4, plain = a.plain_k != nullptr;
  if (cfg.head_dim == 128)
    return !fp4 ? launch<128, false, false>(B, a, stream) : plain ? launch<128, true, true>(B, a, stream)
                                                                  : launch<128, true, false>(B, a, stream);
  return !fp4 ? launch<64, false, false>(B, a, stream) : plain ? launch<64, true, true>(B, a, stream)
                                                               : launch<64, true, false>(B, a, stream);
}

size_t kv_plain_bytes(const csa2_kv_cfg& cfg, int B, int T, int max_q, int64_t max_kv, bool cross) {
  if (cfg.cache_dtype != CSA2_CACHE_FP4) return 0;
  const int mean = std::min(max_q, T / B);  // rows of a sequence
  const int64_t seen = cfg.window && !cross ? std::min(mean, cfg.window) : mean;
  if (seen * (cfg.n_heads / cfg.kv_heads) < kPlainRows) return 0;
  const size_t bytes = (size_t)B * ((max_kv + kPage - 1) / kPage) * cfg.kv_heads * 2 * kv_block_bytes(cfg.head_dim, false);
  return bytes <= kMostPlain ? bytes : 0;
}

int kv_tiles_rows() { return kCtaRows; }

}  // namespace csa2
