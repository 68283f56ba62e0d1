// C ABI entry points of the text model's operators: argument checks and the
// library-owned error word. The kernels are in int8_linear.cu.
#include "internal.cuh"
#include "sm100.cuh"

namespace h3 {
namespace {

// A wait that runs out in a text operator records H3_DEVERR_TIMEOUT here (one
// int per GPU that loads the library); h3_text_error reads and clears it.
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

inline bool known_type(h3_type t) { return t == H3_BF16 || t == H3_F16 || t == H3_F32; }

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
  if (v != 0 && cudaMemset(p, 0, 4) != cudaSuccess) return H3_ERR_CUDA;
  return v == 0 ? H3_OK : H3_ERR_TIMEOUT;
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
  if (K % 16 != 0 || K > 131056 || out_stride < N) return H3_ERR_SHAPE;
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

}  // extern "C"
