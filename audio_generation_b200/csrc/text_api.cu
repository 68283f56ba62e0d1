// C ABI entry points of the text model's operators: argument checks and the
// library-owned error word. The kernels are in int8_linear.cu,
// prompt_attention.cu and kv_cache.cu.
#include <math.h>

#include <new>

#include "internal.cuh"
#include "sm100.cuh"

namespace h3 {
namespace {

// A wait that runs out in a text operator records H3_DEVERR_TIMEOUT here, a
// device table that makes no sense H3_DEVERR_LAYOUT (one int per GPU that loads
// the library); h3_text_error reads and clears it.
static __device__ int g_text_err;

SymbolAddressCache g_text_err_cache;

cudaError_t lookup_text_err(void** p) { return cudaGetSymbolAddress(p, g_text_err); }

inline cudaStream_t as_stream(h3_stream_t s) { return reinterpret_cast<cudaStream_t>(s); }

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

inline h3_status cuda_status(cudaError_t e) {
  if (e == cudaSuccess) return H3_OK;
  if (e == cudaErrorInvalidValue) return H3_ERR_ARG;
  return H3_ERR_CUDA;
}

// Rows of `width` 2-byte elements, `stride` apart: aligned, apart, and within
// the 2^40 bytes a tensor map's stride may have.
inline bool row_stride_ok(int64_t stride, int64_t width) {
  return stride >= width && stride % 8 == 0 && stride < (1ll << 38);
}

// Positive and finite, in log2 units too.
inline bool scale_ok(float scale) { return scale > 0.f && isfinite(scale * 1.4426950408889634f); }

inline bool known_type(h3_type t) { return t == H3_BF16 || t == H3_F16 || t == H3_F32; }

h3_status check_cache(const h3_kv_cache* c) {
  if (!c || c->n_blocks < 0 || c->kv_heads <= 0) return H3_ERR_ARG;
  if (c->block_tokens != 32 && c->block_tokens != 64 && c->block_tokens != 128)
    return H3_ERR_SHAPE;
  if (c->head_dim != 64 && c->head_dim != 128) return H3_ERR_SHAPE;
  return H3_OK;
}

// The parts that a call with work to do dereferences.
h3_status check_cache_pointers(const h3_kv_cache* c) {
  if (!c->k_codes || !c->v_codes || !c->k_scales || !c->v_scales) return H3_ERR_ARG;
  if (!aligned16(c->k_codes) || !aligned16(c->v_codes) || !aligned16(c->k_scales) ||
      !aligned16(c->v_scales))
    return H3_ERR_ALIGN;
  return H3_OK;
}

// A table of `width` blocks per sequence whose token numbers fit an int.
h3_status check_table(const h3_kv_cache* c, int width) {
  if (width < 0) return H3_ERR_ARG;
  return (long long)width * c->block_tokens > 0x7fffffffLL ? H3_ERR_SHAPE : H3_OK;
}

}  // namespace

h3_status text_error_word(int** out) {
  void* p = nullptr;
  const h3_status rc = symbol_address(g_text_err_cache, lookup_text_err, &p);
  *out = static_cast<int*>(p);
  return rc;
}

}  // namespace h3

using namespace h3;

extern "C" {

h3_status h3_text_error(void) {
  int* p = nullptr;
  if (text_error_word(&p) != H3_OK) return H3_ERR_CUDA;
  int v = 0;
  if (cudaDeviceSynchronize() != cudaSuccess) return H3_ERR_CUDA;
  if (cudaMemcpy(&v, p, 4, cudaMemcpyDeviceToHost) != cudaSuccess) return H3_ERR_CUDA;
  // cleared for good before the caller launches anything more, on any stream
  if (v != 0 && (cudaMemset(p, 0, 4) != cudaSuccess || cudaDeviceSynchronize() != cudaSuccess))
    return H3_ERR_CUDA;
  return v == 0 ? H3_OK : v == H3_DEVERR_LAYOUT ? H3_ERR_LAYOUT : H3_ERR_TIMEOUT;
}

h3_status h3_quantize_int8_rows(h3_type type, int rows, int K, const void* x, int64_t x_stride,
                                void* codes, float* scales, h3_stream_t stream) {
  if (!known_type(type) || rows < 0 || K <= 0) return H3_ERR_ARG;
  if (K % 16 != 0 || x_stride < K || x_stride % 8 != 0) return H3_ERR_SHAPE;
  if (rows == 0) return H3_OK;
  if (!x || !codes || !scales) return H3_ERR_ARG;
  if (!aligned16(x) || !aligned16(codes) || !aligned16(scales)) return H3_ERR_ALIGN;
  return cuda_status(
      launch_quantize_rows_int8(type, rows, K, x, x_stride, codes, scales, as_stream(stream)));
}

h3_status h3_matmul_int8(int M, int N, int K, const void* a_codes, const float* a_scales,
                         const void* w_codes, const float* w_scales, h3_type out_type, void* out,
                         int64_t out_stride, h3_stream_t stream) {
  if (!known_type(out_type) || M < 0 || N < 0 || K <= 0) return H3_ERR_ARG;
  // |sum| <= 128 * 128 * K must stay below 2^31; rows of codes start 16-byte aligned
  if (K % 16 != 0 || K > 131056 || out_stride < N || M > 1 << 30 || N > 1 << 30)
    return H3_ERR_SHAPE;
  if (M == 0 || N == 0) return H3_OK;
  if (!a_codes || !a_scales || !w_codes || !w_scales || !out) return H3_ERR_ARG;
  if (!aligned16(a_codes) || !aligned16(a_scales) || !aligned16(w_codes) ||
      !aligned16(w_scales) || !aligned16(out))
    return H3_ERR_ALIGN;
  int* err = nullptr;
  const h3_status rc = text_error_word(&err);
  if (rc != H3_OK) return rc;
  return cuda_status(launch_matmul_int8(M, N, K, a_codes, a_scales, w_codes, w_scales, out_type,
                                        out, out_stride, err, as_stream(stream)));
}

h3_status h3_prompts_prepare(const int32_t* offsets_host, int n_prompts, int q_heads,
                             int kv_heads, int head_dim, h3_prompts_t* out) {
  if (!out) return H3_ERR_ARG;
  *out = nullptr;
  if (!offsets_host || n_prompts < 0 || q_heads <= 0 || kv_heads <= 0) return H3_ERR_ARG;
  if (q_heads % kv_heads != 0 || q_heads / kv_heads > 128 || (head_dim != 64 && head_dim != 128))
    return H3_ERR_SHAPE;
  if (offsets_host[0] < 0) return H3_ERR_LAYOUT;
  for (int i = 0; i < n_prompts; ++i)
    if (offsets_host[i + 1] < offsets_host[i]) return H3_ERR_LAYOUT;
  h3_prompts* p = new (std::nothrow) h3_prompts();
  if (!p) return H3_ERR_CUDA;
  p->q_heads = q_heads;
  p->kv_heads = kv_heads;
  p->head_dim = head_dim;
  p->rows = offsets_host[n_prompts];
  h3_status rc = cudaGetDevice(&p->device) == cudaSuccess ? H3_OK : H3_ERR_CUDA;
  if (rc == H3_OK) rc = build_prompts(p, offsets_host, n_prompts);
  if (rc != H3_OK) {
    delete p;
    return rc;
  }
  *out = p;
  return H3_OK;
}

void h3_prompts_destroy(h3_prompts_t p) {
  if (!p) return;
  if (p->items) {
    int current = 0;
    const bool known = cudaGetDevice(&current) == cudaSuccess;
    if (known && current != p->device) cudaSetDevice(p->device);
    cudaDeviceSynchronize();
    cudaFree(p->items);
    if (known && current != p->device) cudaSetDevice(current);
  }
  delete p;
}

h3_status h3_prompt_attention(h3_prompts_t p, h3_type type, const void* q, int64_t q_stride,
                              const void* k, int64_t k_stride, const void* v, int64_t v_stride,
                              float scale, void* o, int64_t o_stride, h3_stream_t stream) {
  if (!p || (type != H3_BF16 && type != H3_F16)) return H3_ERR_ARG;
  if (!scale_ok(scale)) return H3_ERR_ARG;
  const int64_t qw = (int64_t)p->q_heads * p->head_dim, kw = (int64_t)p->kv_heads * p->head_dim;
  if (!row_stride_ok(q_stride, qw) || !row_stride_ok(o_stride, qw) ||
      !row_stride_ok(k_stride, kw) || !row_stride_ok(v_stride, kw))
    return H3_ERR_SHAPE;
  if (p->n_items == 0) return H3_OK;
  if (!q || !k || !v || !o) return H3_ERR_ARG;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o)) return H3_ERR_ALIGN;
  int device = 0;
  if (cudaGetDevice(&device) != cudaSuccess) return H3_ERR_CUDA;
  if (device != p->device) return H3_ERR_ARG;
  int* err = nullptr;
  const h3_status rc = text_error_word(&err);
  if (rc != H3_OK) return rc;
  return cuda_status(launch_prompt_attention(p, type == H3_F16, q, q_stride, k, k_stride, v,
                                             v_stride, scale, o, o_stride, err,
                                             as_stream(stream)));
}

h3_status h3_kv_cache_store(const h3_kv_cache* cache, int n_seq, int max_new,
                            const int32_t* block_table, int table_width, const int32_t* lengths,
                            const int32_t* offsets, h3_type type, int rows, const void* k,
                            int64_t k_stride, const void* v, int64_t v_stride,
                            h3_stream_t stream) {
  h3_status rc = check_cache(cache);
  if (rc != H3_OK) return rc;
  if (n_seq < 0 || max_new < 0 || rows < 0 || (type != H3_BF16 && type != H3_F16))
    return H3_ERR_ARG;
  if ((rc = check_table(cache, table_width)) != H3_OK) return rc;
  const int64_t w = (int64_t)cache->kv_heads * cache->head_dim;
  if (!row_stride_ok(k_stride, w) || !row_stride_ok(v_stride, w)) return H3_ERR_SHAPE;
  if (n_seq == 0 || max_new == 0 || rows == 0) return H3_OK;
  if (table_width == 0) return H3_ERR_SHAPE;  // new tokens, and no block to hold them
  if (!block_table || !lengths || !offsets || !k || !v) return H3_ERR_ARG;
  if ((rc = check_cache_pointers(cache)) != H3_OK) return rc;
  if (!aligned16(block_table) || !aligned16(lengths) || !aligned16(offsets) || !aligned16(k) ||
      !aligned16(v))
    return H3_ERR_ALIGN;
  int* err = nullptr;
  if ((rc = text_error_word(&err)) != H3_OK) return rc;
  return cuda_status(launch_kv_cache_store(*cache, n_seq, max_new, block_table, table_width,
                                           lengths, offsets, type == H3_F16, rows, k, k_stride, v,
                                           v_stride, err, as_stream(stream)));
}

size_t h3_cache_attention_workspace_size(const h3_kv_cache* cache, int n_seq, int q_heads,
                                         int table_width) {
  if (check_cache(cache) != H3_OK || n_seq <= 0 || q_heads <= 0 ||
      q_heads % cache->kv_heads != 0 || check_table(cache, table_width) != H3_OK ||
      table_width == 0)
    return 0;
  return cache_attention_workspace(*cache, n_seq, q_heads, table_width);
}

h3_status h3_cache_attention(const h3_kv_cache* cache, int n_seq, int q_heads,
                             const int32_t* block_table, int table_width, const int32_t* lengths,
                             h3_type type, const void* q, int64_t q_stride, float scale, void* o,
                             int64_t o_stride, void* ws, size_t ws_bytes, h3_stream_t stream) {
  h3_status rc = check_cache(cache);
  if (rc != H3_OK) return rc;
  if (n_seq < 0 || q_heads <= 0 || (type != H3_BF16 && type != H3_F16) || !scale_ok(scale))
    return H3_ERR_ARG;
  if ((rc = check_table(cache, table_width)) != H3_OK) return rc;
  const int64_t w = (int64_t)q_heads * cache->head_dim;
  if (q_heads % cache->kv_heads != 0 || !row_stride_ok(q_stride, w) ||
      !row_stride_ok(o_stride, w))
    return H3_ERR_SHAPE;
  if (n_seq == 0) return H3_OK;
  if (table_width == 0) return H3_ERR_SHAPE;
  if (!block_table || !lengths || !q || !o) return H3_ERR_ARG;
  if ((rc = check_cache_pointers(cache)) != H3_OK) return rc;
  const size_t need = cache_attention_workspace(*cache, n_seq, q_heads, table_width);
  if (ws_bytes < need) return H3_ERR_WORKSPACE;
  if (need > 0 && !ws) return H3_ERR_ARG;
  if (!aligned16(block_table) || !aligned16(lengths) || !aligned16(q) || !aligned16(o) ||
      (need > 0 && !aligned16(ws)))
    return H3_ERR_ALIGN;
  int* err = nullptr;
  if ((rc = text_error_word(&err)) != H3_OK) return rc;
  return cuda_status(launch_cache_attention(*cache, n_seq, q_heads, block_table, table_width,
                                            lengths, type == H3_F16, q, q_stride, scale, o,
                                            o_stride, ws, err, as_stream(stream)));
}

}  // extern "C"
