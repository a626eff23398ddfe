// gemm_int8.hip -- grouped products of 8-bit integer rows with 8-bit integer expert
// weights, a scale for each row and each column of the result, and the SwiGLU expert FFN
// made of two of them.
#include "gemm_int8.h"
#include "launch.h"

namespace moe {

hipError_t launch_gemm_int8(const Int8Rows& a, int64_t rows, int E, const int32_t* offs,
                            const int32_t* cnts, const void* w, const float* wsc, int N, int K,
                            int out_dtype, void* out, hipStream_t s) {
  if (rows == 0) return hipSuccess;
  return launch_gemm_int8_stream(false, out_dtype == MOE_F32, a, rows, E, offs, cnts, w, wsc, N, K,
                                 out, s);
}

hipError_t launch_expert_swiglu_int8(const Int8Rows& a, int64_t rows, int H, int I, int E,
                                     const int32_t* offs, const int32_t* cnts,
                                     const void* w_gate_up, const float* gsc, const void* w_down,
                                     const float* dsc, float* h, void* hq, float* hs, void* out,
                                     hipStream_t s) {
  if (rows == 0) return hipSuccess;
  hipError_t err =
      launch_gemm_int8_stream(true, true, a, rows, E, offs, cnts, w_gate_up, gsc, 2 * I, H, h, s);
  if (err != hipSuccess) return err;
  err = launch_quantize_int8(h, MOE_F32, rows, I, hq, hs, s);
  if (err != hipSuccess) return err;
  return launch_gemm_int8({hq, hs, nullptr, rows}, rows, E, offs, cnts, w_down, dsc, H, I, MOE_BF16,
                          out, s);
}

}  // namespace moe
