// C ABI of the paged key / value operators: argument validation on the host,
// then the launches of kv_append.cu, kv_rows.cu, kv_tiles.cu and kv_reorder.cu.
#include <cmath>
#include <cstring>

#include "kv.cuh"

using namespace csa2;

namespace {

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

int32_t check_cfg(const csa2_kv_cfg* c) {
  if (!c || c->reserved != 0) return CSA2_ERR_INVALID_ARG;
  if ((c->cache_dtype != CSA2_CACHE_FP4 && c->cache_dtype != CSA2_CACHE_BF16) || c->window < 0 || c->kv_heads < 1 ||
      c->n_heads < 1 || c->n_heads % c->kv_heads || c->rope_dims < 0 || c->rope_dims % 16 ||
      c->rope_dims > c->head_dim || (c->rope_style != CSA2_ROPE_INTERLEAVED && c->rope_style != CSA2_ROPE_HALF))
    return CSA2_ERR_INVALID_ARG;
  if ((c->head_dim != 64 && c->head_dim != 128) || c->n_heads > 1024) return CSA2_ERR_UNSUPPORTED;
  return CSA2_OK;
}

bool cache_ok(const csa2_kv_cfg& cfg, const csa2_kv_cache* c) {
  if (!c || !c->k_data || !c->v_data || !c->block_table || c->max_pages <= 0 || c->num_pages <= 0) return false;
  // positions are 32-bit in the kernels
  if (c->max_pages > (INT32_MAX - 1024) / kPage) return false;
  const bool fp4 = cfg.cache_dtype == CSA2_CACHE_FP4;
  if (fp4 && (!c->k_scales || !c->v_scales)) return false;
  return aligned(c->k_data, 16) && aligned(c->v_data, 16) && aligned(c->k_scales, 16) && aligned(c->v_scales, 16) &&
         aligned(c->block_table, 4);
}

KvView view_of(const csa2_kv_cache& c) {
  return KvView{static_cast<uint8_t*>(c.k_data), static_cast<uint8_t*>(c.k_scales), static_cast<uint8_t*>(c.v_data),
                static_cast<uint8_t*>(c.v_scales), c.block_table, c.max_pages, c.num_pages};
}

// A row array: 16-byte aligned rows at least `width` elements apart.
bool rows_ok(const void* p, int64_t stride, int64_t width) {
  return p && aligned(p, 16) && stride >= width && stride % 8 == 0;
}

int32_t cuda_status(cudaError_t e) { return e == cudaSuccess ? CSA2_OK : CSA2_ERR_CUDA; }

int32_t attend(const csa2_kv_cfg* cfg, bool cross, int32_t B, int32_t T, const uint16_t* q, int64_t q_stride,
               const int32_t* cu, const csa2_kv_cache* cache, const int32_t* kv_len, int32_t max_q, int32_t max_kv,
               float scale, uint16_t* out, int64_t out_stride, float* lse, void* workspace, size_t workspace_bytes,
               int32_t* status, void* stream) {
  const int32_t rc = check_cfg(cfg);
  if (rc) return rc;
  if (cross && cfg->window) return CSA2_ERR_INVALID_ARG;
  if (B < 0 || T < 0 || max_q < 0 || max_kv < 0 || !std::isfinite(scale)) return CSA2_ERR_INVALID_ARG;
  if (B == 0 || T == 0 || max_q == 0) return CSA2_OK;
  const int64_t width = (int64_t)cfg->n_heads * cfg->head_dim;
  if (!rows_ok(q, q_stride, width) || !rows_ok(out, out_stride, width) || !cu || !kv_len || !aligned(cu, 4) ||
      !aligned(kv_len, 4) || !aligned(lse, 4) || !aligned(status, 4) || !cache_ok(*cfg, cache))
    return CSA2_ERR_INVALID_ARG;
  if (workspace ? !aligned(workspace, 256) : workspace_bytes != 0) return CSA2_ERR_INVALID_ARG;
  const int64_t most = max_q < T ? max_q : T;  // rows of a sequence; row numbers are 32-bit in the kernels
  if (B > 65535 || most * cfg->n_heads > (1 << 30)) return CSA2_ERR_UNSUPPORTED;
  if (max_kv > (int64_t)cache->max_pages * kPage) return CSA2_ERR_CAPACITY;
  KvAtt a = {};
  a.B = B, a.T = T, a.n_heads = cfg->n_heads, a.kv_heads = cfg->kv_heads, a.group = cfg->n_heads / cfg->kv_heads;
  a.by_group = divisor(a.group), a.by_heads = divisor(a.kv_heads);
  a.window = cfg->window >= max_kv ? 0 : cfg->window;  // as wide as the keys: none
  a.causal = cross ? 0 : 1, a.max_q = (int)most, a.max_kv = max_kv;
  a.q = q, a.q_stride = q_stride, a.cu = cu, a.c = view_of(*cache), a.kv_len = kv_len, a.scale = scale;
  a.out = out, a.out_stride = out_stride, a.lse = lse, a.status = status;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  if (const size_t plain = kv_plain_bytes(*cfg, B, T, a.max_q, max_kv, cross); plain && plain <= workspace_bytes) {
    a.plain_k = ws, a.plain_v = ws + plain / 2, a.plain_pages = (max_kv + kPage - 1) / kPage;
    ws += plain, workspace_bytes -= plain;
  }
  KvPlan plan = kv_plan(*cfg, B, T, a.max_q, max_kv, cross, SIZE_MAX);
  if (plan.bytes > workspace_bytes) plan = kv_plan(*cfg, B, T, a.max_q, max_kv, cross, workspace_bytes);
  if (plan.ctas > INT32_MAX) return CSA2_ERR_UNSUPPORTED;
  a.n_parts = plan.n_parts, a.by_parts = divisor(plan.n_parts), a.cluster = plan.cluster ? 1 : 0;
  a.part_pages = plan.part_pages, a.by_pages = divisor(plan.part_pages);
  a.tiles = (int)plan.tiles, a.whole = (int)plan.whole;
  if (plan.bytes) {
    a.part_step = plan.part_step, a.part_rows = plan.part_rows;
    a.part_o = reinterpret_cast<float*>(ws);
    a.part_l = a.part_o + a.n_parts * a.part_step * cfg->head_dim;
  }
  return cuda_status(launch_kv_attend(*cfg, B, a, static_cast<cudaStream_t>(stream)));
}

int32_t append(const csa2_kv_cfg* cfg, int32_t B, int32_t T, const uint16_t* q, int64_t q_stride,
                       const uint16_t* k, int64_t k_stride, const uint16_t* v, int64_t v_stride, const int32_t* cu,
                       const int64_t* pos0, const KvAxes& axes, const float* rope, int64_t rope_rows, const csa2_kv_cache* cache,
                       uint16_t* q_out, int64_t q_out_stride, uint16_t* k_out, uint16_t* v_out, int32_t* status,
                       void* stream) {
  const int32_t rc = check_cfg(cfg);
  if (rc) return rc;
  if (B < 0 || T < 0 || rope_rows < 0) return CSA2_ERR_INVALID_ARG;
  if (B == 0 || T == 0) return CSA2_OK;
  const int64_t kw = (int64_t)cfg->kv_heads * cfg->head_dim, qw = (int64_t)cfg->n_heads * cfg->head_dim;
  if (!rows_ok(k, k_stride, kw) || !rows_ok(v, v_stride, kw) || !cu || !pos0 || !aligned(cu, 4) || !aligned(pos0, 8) ||
      !aligned(k_out, 16) || !aligned(v_out, 16) || !aligned(status, 4) || !cache_ok(*cfg, cache))
    return CSA2_ERR_INVALID_ARG;
  if ((q != nullptr) != (q_out != nullptr)) return CSA2_ERR_INVALID_ARG;
  if (q && (!rows_ok(q, q_stride, qw) || !rows_ok(q_out, q_out_stride, qw))) return CSA2_ERR_INVALID_ARG;
  if ((rope != nullptr) != (cfg->rope_dims != 0) || !aligned(rope, 16)) return CSA2_ERR_INVALID_ARG;
  return cuda_status(launch_kv_append(*cfg, B, T, q, q_stride, k, k_stride, v, v_stride, cu, pos0, axes, rope, rope_rows,
                                      view_of(*cache), q_out, q_out_stride, k_out, v_out, status,
                                      static_cast<cudaStream_t>(stream)));
}

}  // namespace

extern "C" {

size_t csa2_kv_page_bytes(const csa2_kv_cfg* cfg, int32_t which) {
  if (check_cfg(cfg) || which < 0 || which > 1) return 0;
  const bool fp4 = cfg->cache_dtype == CSA2_CACHE_FP4;
  if (which == 0) return (size_t)cfg->kv_heads * kv_block_bytes(cfg->head_dim, fp4);
  return fp4 ? (size_t)cfg->kv_heads * kv_scale_bytes(cfg->head_dim) : 0;
}

int32_t csa2_kv_append(const csa2_kv_cfg* cfg, int32_t B, int32_t T, const uint16_t* q, int64_t q_stride,
                       const uint16_t* k, int64_t k_stride, const uint16_t* v, int64_t v_stride, const int32_t* cu,
                       const int64_t* pos0, const float* rope, int64_t rope_rows, const csa2_kv_cache* cache,
                       uint16_t* q_out, int64_t q_out_stride, uint16_t* k_out, uint16_t* v_out, int32_t* status,
                       void* stream) {
  return append(cfg, B, T, q, q_stride, k, k_stride, v, v_stride, cu, pos0, KvAxes{}, rope, rope_rows, cache, q_out,
                q_out_stride, k_out, v_out, status, stream);
}

int32_t csa2_kv_append_axes(const csa2_kv_cfg* cfg, int32_t B, int32_t T, const uint16_t* q, int64_t q_stride,
                            const uint16_t* k, int64_t k_stride, const uint16_t* v, int64_t v_stride, const int32_t* cu,
                            const int64_t* pos0, const int32_t* axes, int32_t n_axes, const uint8_t* axis_of,
                            const float* rope, int64_t rope_rows, const csa2_kv_cache* cache, uint16_t* q_out,
                            int64_t q_out_stride, uint16_t* k_out, uint16_t* v_out, int32_t* status, void* stream) {
  const int32_t rc = check_cfg(cfg);
  if (rc) return rc;
  if (n_axes < 1 || n_axes > 4 || !axis_of || cfg->rope_dims == 0) return CSA2_ERR_INVALID_ARG;
  for (int i = 0; i < cfg->rope_dims / 2; ++i)
    if (axis_of[i] >= n_axes) return CSA2_ERR_INVALID_ARG;
  if (B > 0 && T > 0 && (!axes || !aligned(axes, 4))) return CSA2_ERR_INVALID_ARG;
  return append(cfg, B, T, q, q_stride, k, k_stride, v, v_stride, cu, pos0, KvAxes{axes, n_axes, axis_of}, rope, rope_rows,
                cache, q_out, q_out_stride, k_out, v_out, status, stream);
}

int32_t csa2_kv_reorder(const csa2_kv_cfg* cfg, int32_t layers, const csa2_kv_cache* caches, int32_t groups,
                        int32_t beams, const int32_t* parents, const int32_t* kv_len, int32_t* status, void* stream) {
  const int32_t rc = check_cfg(cfg);
  if (rc) return rc;
  if (layers < 0 || groups < 0 || beams < 1 || beams > 64) return CSA2_ERR_INVALID_ARG;
  if (layers > CSA2_MAX_LAYERS || (int64_t)groups * beams > (1 << 24)) return CSA2_ERR_UNSUPPORTED;
  if (layers == 0 || groups == 0) return CSA2_OK;
  if (!caches || !parents || !kv_len || !aligned(parents, 4) || !aligned(kv_len, 4) || !aligned(status, 4))
    return CSA2_ERR_INVALID_ARG;
  for (int i = 0; i < layers; ++i)
    if (!cache_ok(*cfg, caches + i) || caches[i].block_table != caches[0].block_table ||
        caches[i].max_pages != caches[0].max_pages || caches[i].num_pages != caches[0].num_pages)
      return CSA2_ERR_INVALID_ARG;
  return cuda_status(launch_kv_reorder(*cfg, layers, caches, groups, beams, parents, kv_len, status,
                                       static_cast<cudaStream_t>(stream)));
}

size_t csa2_kv_workspace_bytes(const csa2_kv_cfg* cfg, int32_t B, int32_t T, int32_t max_q, int32_t max_kv) {
  if (check_cfg(cfg) || B < 0 || T < 0 || max_q < 0 || max_kv < 0 || B == 0 || T == 0 || max_q == 0) return 0;
  if (max_q > T) max_q = T;
  size_t most = 0;
  for (const bool cross : {false, true}) {
    if (cross && cfg->window) break;
    const size_t n = kv_plain_bytes(*cfg, B, T, max_q, max_kv, cross) + kv_plan(*cfg, B, T, max_q, max_kv, cross, SIZE_MAX).bytes;
    if (n > most) most = n;
  }
  return most;
}

int32_t csa2_kv_attend(const csa2_kv_cfg* cfg, int32_t B, int32_t T, const uint16_t* q, int64_t q_stride,
                       const int32_t* cu, const csa2_kv_cache* cache, const int32_t* kv_len, int32_t max_q,
                       int32_t max_kv, float scale, uint16_t* out, int64_t out_stride, float* lse, void* workspace,
                       size_t workspace_bytes, int32_t* status, void* stream) {
  return attend(cfg, false, B, T, q, q_stride, cu, cache, kv_len, max_q, max_kv, scale, out, out_stride, lse,
                workspace, workspace_bytes, status, stream);
}

int32_t csa2_kv_cross_attend(const csa2_kv_cfg* cfg, int32_t B, int32_t T, const uint16_t* q, int64_t q_stride,
                             const int32_t* cu, const csa2_kv_cache* cache, const int32_t* kv_len, int32_t max_q,
                             int32_t max_kv, float scale, uint16_t* out, int64_t out_stride, float* lse,
                             void* workspace, size_t workspace_bytes, int32_t* status, void* stream) {
  return attend(cfg, true, B, T, q, q_stride, cu, cache, kv_len, max_q, max_kv, scale, out, out_stride, lse, workspace,
                workspace_bytes, status, stream);
}

}  // extern "C"
