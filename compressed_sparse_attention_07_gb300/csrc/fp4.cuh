// Shared by the projections with 4-bit weights (fp4_pack.cu, fp4_rows.cu,
// fp4_tiles.cu): how the weights are laid out, and their decoding to bf16.
//
// A block is 16 rows x 128 channels in 1152 bytes: 1024 of codes, 128 of scales; the
// eight blocks of 128 rows and 128 channels follow one another, these along k, then the
// next 128 rows.  In a block the codes are in units of 16 bytes, 32 channels of a row:
// those of row r and channels 32 t .. at fp4_unit(r, t).  A warp reads them conflict-free
// both as the left operand of eight 16x8x16 products (lane 4 g + t: unit t of rows g and
// g + 8) and a row a lane.  The i-th word of unit t has the eight channels of 16-byte
// chunk i ^ t of the unit's 32 in bf16, so that lanes of neighbouring t read different
// banks of rows of x too.  The two scales of a row's unit stand at fp4_unit_scales(r, t),
// that of words 0 and 1 first.
// Nibble p of a word is the code of the chunk's channel 2 p, nibble 4 + p of channel
// 2 p + 1, so that a mask and two shifts bring two neighbouring channels to the halves of a
// register (fp4_bf16), and its bytes hold channels (0, 2), (4, 6), (1, 3), (5, 7) for the
// conversion of pairs to f16 (fp4_f16).
//
// To bf16, for x as it comes: a code's sign at bit 15 and the rest at bits 8..6 of a bf16
// is code x 2^-126 (subnormal where the exponent is 0), exactly; times scale x 2^118 it is
// the weight x 2^-8, exactly, as a code has 2 significant bits and a scale 4.  Eight
// codes take 15 + 4 instructions and 4.4 cycles of a warp and SM.  To f16, which the
// kernel for few rows brings x to: 4 + 4 instructions, 1.4 cycles; at HBM's rate there are
// 6, of which the products of 8 rows of x take 2.
#pragma once

#include "kv.cuh"

namespace csa2 {

constexpr int kBlockRows = 16, kBlockK = 128, kBlockBytes = 1152, kBlockCodes = 1024;
constexpr float kFp4Unit = 256.0f;  // what fp4_bf16's weights are short of

constexpr int kTileRows = 128, kTileBlocks = kTileRows / kBlockRows, kTileBytes = kTileBlocks * kBlockBytes;

__host__ __device__ constexpr int fp4_unit(int r, int t) { return t * 256 + (r >> 3) * 128 + ((r & 7) ^ (2 * t)) * 16; }
__host__ __device__ constexpr int fp4_unit_scales(int r, int t) {
  return kBlockCodes + ((r & 7) * 4 + t) * 4 + (r >> 3) * 2;
}
__host__ __device__ __forceinline__ int fp4_row_tiles(int n) { return (n + kTileRows - 1) / kTileRows; }
__host__ __device__ __forceinline__ int fp4_k_blocks(int k) { return (k + kBlockK - 1) / kBlockK; }

struct Fp4Linear {
  const uint8_t* w;
  int n, k, k_blocks, T;
  const uint16_t* x;
  int64_t x_stride;
  const uint16_t* bias;
  void* out;
  int64_t out_stride;
  int f32;      // out's type
  float alpha;
  int32_t* status;
};

__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
// Byte i of w, an E4M3 scale >= 0, as a pair of bf16 scale x 2^118: its bits are a bf16
// scale x 2^-120.
__device__ __forceinline__ uint32_t fp4_scale(uint32_t w, int i) {
  const uint32_t b = __byte_perm(w, 0, 0x4040 | i | i << 8) * 16u;
  return mul_bf16x2(mul_bf16x2(b, 0x7F007F00u), 0x77007700u);  // 2^127, 2^111
}
// The eight weights of a word, times 2^-8: pair p holds channels 2p and 2p + 1.
__device__ __forceinline__ void fp4_bf16(uint32_t w, uint32_t scale, uint32_t (&r)[4]) {
  constexpr uint32_t kRest = 0x01C001C0u, kSign = 0x80008000u;
  r[0] = mul_bf16x2(((w << 6) & kRest) | ((w << 12) & kSign), scale);
  r[1] = mul_bf16x2(((w << 2) & kRest) | ((w << 8) & kSign), scale);
  r[2] = mul_bf16x2(((w >> 2) & kRest) | ((w << 4) & kSign), scale);
  r[3] = mul_bf16x2(((w >> 6) & kRest) | (w & kSign), scale);
}
// The eight weights of a word in f16, channels (0, 2), (4, 6), (1, 3), (5, 7); scale a pair.
__device__ __forceinline__ void fp4_f16(uint32_t w, uint32_t scale, uint32_t (&r)[4]) {
  codes8(w, r);
#pragma unroll
  for (int i = 0; i < 4; ++i) r[i] = mul2(r[i], scale);
}
// sum x alpha + bias, stored in out's type.
__device__ __forceinline__ void fp4_store(const Fp4Linear& a, int t, int i, float sum, float alpha, float bias) {
  const float y = fmaf(sum, alpha, bias);
  if (a.f32) static_cast<float*>(a.out)[t * a.out_stride + i] = y;
  else static_cast<__nv_bfloat16*>(a.out)[t * a.out_stride + i] = __float2bfloat16_rn(y);
}
__device__ __forceinline__ float fp4_bias(const Fp4Linear& a, int i) {
  return a.bias ? bf16_bits_to_float(__ldg(a.bias + i)) : 0.0f;
}

cudaError_t launch_fp4_encode(int n, int k, const uint16_t* w, int64_t stride, float gain, uint8_t* packed,
                              int32_t* status, cudaStream_t stream);
cudaError_t launch_fp4_pack(int n, int k, const uint8_t* codes, const uint8_t* scales, uint8_t* packed,
                            int32_t* status, cudaStream_t stream);
// Up to kFp4FewRows rows whose x fits shared memory (fp4_rows_ok), and any.
constexpr int kFp4FewRows = 16;
bool fp4_rows_ok(const Fp4Linear& a);
cudaError_t launch_fp4_rows(const Fp4Linear& a, cudaStream_t stream);
cudaError_t launch_fp4_tiles(const Fp4Linear& a, cudaStream_t stream);

}  // namespace csa2
