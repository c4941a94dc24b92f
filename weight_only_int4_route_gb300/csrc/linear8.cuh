// What the kernels of the 8-bit product share (linear8.cu, linear8_tc.cu).
#pragma once

#include "moe_internal.cuh"

namespace moe {

struct LinearArgs {
  const int8_t *a, *w;
  const float *a_scale, *w_scale, *bias;
  void *out;
  int64_t M, a_stride, w_stride, out_stride;   // strides in elements (= bytes for a and w)
  int N, K;       // K as given; w's rows start on 16 bytes and hold K rounded up to 16, zeros past K
  int out_dtype;
};

// The definition's fp32 operations, each rounded.
__device__ __forceinline__ float scaled(int acc, float sa, float sw, bool with_bias, float bias) {
  const float v = __fmul_rn(__fmul_rn(float(acc), sa), sw);
  return with_bias ? __fadd_rn(v, bias) : v;
}
__device__ __forceinline__ void store_out(void *out, int dtype, int64_t at, float v) {
  if (dtype == MOE_F32) static_cast<float *>(out)[at] = v;
  else if (dtype == MOE_F16) static_cast<__half *>(out)[at] = from_f32<__half>(v);
  else static_cast<__nv_bfloat16 *>(out)[at] = from_f32<__nv_bfloat16>(v);
}

// Many rows, on tcgen05: bytes of the rows as f16, and the launch (rows16: that many bytes, 256-byte aligned).
size_t linear8_tc_rows_bytes(int64_t M, int64_t K);
int launch_linear8_tc(const LinearArgs &p, void *rows16, cudaStream_t st);
int linear8_error_take(int *out);   // device error word of the tcgen05 kernel

}  // namespace moe
