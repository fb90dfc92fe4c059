// grad.cuh -- backward pass of the ternary layer (straight-through
// estimator: the rounding of x and W passes gradients unchanged).
//
//   dx[m,k] = gamma * sum_n dy[m,n] W~[n,k]
//   dW[n,k] = sum_m dy[m,n] (x~[m,k] eta_m / 127)
//
// One thread per output element, fp32 sums.
#pragma once

#include "common.cuh"

namespace bl {

template <typename T>
__device__ __forceinline__ float ld_f32(const T* p);
template <>
__device__ __forceinline__ float ld_f32<float>(const float* p) { return *p; }
template <>
__device__ __forceinline__ float ld_f32<__nv_bfloat16>(const __nv_bfloat16* p) { return __bfloat162float(*p); }

template <typename DyT, typename OutT>
__global__ void __launch_bounds__(256)
    k_grad_input(const DyT* __restrict__ dy, int64_t M, int64_t N, const uint8_t* __restrict__ packed,
                 const float* __restrict__ gamma, int64_t K, void* __restrict__ dx) {
  const int64_t P = (K + 3) / 4;
  const int64_t total = M * K;
  for (int64_t i = blockIdx.x * 256ll + threadIdx.x; i < total; i += gridDim.x * 256ll) {
    const int64_t m = i / K, k = i % K;
    float s = 0.0f;
    for (int64_t n = 0; n < N; ++n) {
      const int c = (packed[n * P + (k >> 2)] >> (2 * (k & 3))) & 3;
      s = __fmaf_rn(ld_f32(dy + m * N + n), static_cast<float>(c - 1), s);
    }
    store_out<OutT>(dx, i, __fmul_rn(s, *gamma));
  }
}

template <typename DyT, typename OutT>
__global__ void __launch_bounds__(256)
    k_grad_weight(const DyT* __restrict__ dy, const int8_t* __restrict__ xq, const float* __restrict__ eta,
                  int64_t M, int64_t N, int64_t K, void* __restrict__ dw) {
  const int64_t total = N * K;
  for (int64_t i = blockIdx.x * 256ll + threadIdx.x; i < total; i += gridDim.x * 256ll) {
    const int64_t n = i / K, k = i % K;
    float s = 0.0f;
    for (int64_t m = 0; m < M; ++m)
      s = __fmaf_rn(ld_f32(dy + m * N + n), __fmul_rn(static_cast<float>(xq[m * K + k]), div127_rn(eta[m])), s);
    store_out<OutT>(dw, i, s);
  }
}

}  // namespace bl
