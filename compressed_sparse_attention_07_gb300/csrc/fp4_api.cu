// C ABI of the projections with 4-bit weights: argument validation on the host, then
// the launches of fp4_pack.cu, fp4_rows.cu and fp4_tiles.cu.
#include <cmath>

#include "fp4.cuh"

using namespace csa2;

namespace {

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
int32_t cuda_status(cudaError_t e) { return e == cudaSuccess ? CSA2_OK : CSA2_ERR_CUDA; }
bool sizes_ok(int32_t n, int32_t k) { return n >= 1 && k >= 16 && k % 16 == 0 && n < (1 << 24) && k < (1 << 24); }

}  // namespace

extern "C" {

size_t csa2_fp4_weight_bytes(int32_t n, int32_t k) {
  return sizes_ok(n, k) ? (size_t)fp4_row_tiles(n) * fp4_k_blocks(k) * kTileBytes : 0;
}

int32_t csa2_fp4_encode(int32_t n, int32_t k, const uint16_t* w, int64_t stride, float gain, void* packed,
                        int32_t* status, void* stream) {
  if (!sizes_ok(n, k) || !w || !packed || !aligned(w, 16) || stride < k || stride % 8 || !std::isfinite(gain) ||
      !aligned(packed, 128) || !aligned(status, 4))
    return CSA2_ERR_INVALID_ARG;
  return cuda_status(launch_fp4_encode(n, k, w, stride, gain, static_cast<uint8_t*>(packed), status,
                                       static_cast<cudaStream_t>(stream)));
}

int32_t csa2_fp4_pack(int32_t n, int32_t k, const uint8_t* codes, const uint8_t* scales, void* packed, int32_t* status,
                      void* stream) {
  if (!sizes_ok(n, k) || !codes || !scales || !packed || !aligned(codes, 4) || !aligned(packed, 128) || !aligned(status, 4))
    return CSA2_ERR_INVALID_ARG;
  return cuda_status(launch_fp4_pack(n, k, codes, scales, static_cast<uint8_t*>(packed), status,
                                     static_cast<cudaStream_t>(stream)));
}

int32_t csa2_fp4_linear(const csa2_fp4_weights* w, int32_t T, const uint16_t* x, int64_t x_stride, const uint16_t* bias,
                        void* out, int32_t out_dtype, int64_t out_stride, int32_t* status, void* stream) {
  if (!w || w->reserved != 0 || !sizes_ok(w->n, w->k) || !w->data || !aligned(w->data, 128) || !std::isfinite(w->alpha) ||
      T < 0 || (out_dtype != CSA2_BF16 && out_dtype != CSA2_F32))
    return CSA2_ERR_INVALID_ARG;
  if (T == 0) return CSA2_OK;
  if (T > (1 << 30)) return CSA2_ERR_UNSUPPORTED;  // (rows rounded up to a tile, in 32 bits)
  if (!x || !out || !aligned(x, 16) || x_stride < w->k || x_stride % 8 || !aligned(bias, 2) ||
      !aligned(out, out_dtype == CSA2_F32 ? 4 : 2) || out_stride < w->n || !aligned(status, 4))
    return CSA2_ERR_INVALID_ARG;
  Fp4Linear a{static_cast<const uint8_t*>(w->data), w->n, w->k, fp4_k_blocks(w->k), T, x, x_stride, bias, out, out_stride,
              out_dtype == CSA2_F32 ? 1 : 0, w->alpha, status};
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return cuda_status(fp4_rows_ok(a) ? launch_fp4_rows(a, s) : launch_fp4_tiles(a, s));
}

}  // extern "C"
