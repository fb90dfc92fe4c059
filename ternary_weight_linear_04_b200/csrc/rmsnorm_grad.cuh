// rmsnorm_grad.cuh -- backward pass of the RMSNorm without affine parameters
// from the 8-bit tokens the forward pass kept.
//
// The forward pass is n = x r, r = 1 / sqrt(mean(x^2) + eps), so
//   dx = r (dn - n mean_k(n dn)),
// and n is read back from its codes, n = x~ eta / 127 (the quantiser's
// rounding passes gradients unchanged); x itself is not needed.
#pragma once

#include "common.cuh"
#include "grad.cuh"

namespace bl {

template <typename DnT, typename OutT>
__global__ void __launch_bounds__(256)
    k_rmsnorm_grad(const DnT* __restrict__ dn, const int8_t* __restrict__ xq, const float* __restrict__ eta,
                   const float* __restrict__ rstd, int64_t M, int64_t K, void* __restrict__ dx) {
  __shared__ float red[8];
  for (int64_t m = blockIdx.x; m < M; m += gridDim.x) {
    float s = 0.0f;
    for (int64_t k = threadIdx.x; k < K; k += 256)
      s = __fmaf_rn(static_cast<float>(xq[m * K + k]), ld_f32(dn + m * K + k), s);
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = s;
    __syncthreads();
    s = 0.0f;
    for (int w = 0; w < 8; ++w) s += red[w];
    const float f = div127_rn(eta[m]);
    const float c = __fdiv_rn(__fmul_rn(__fmul_rn(s, f), f), static_cast<float>(K));  // x~ c = n mean(n dn)
    const float r = rstd[m];
    for (int64_t k = threadIdx.x; k < K; k += 256) {
      const float d = __fmaf_rn(-static_cast<float>(xq[m * K + k]), c, ld_f32(dn + m * K + k));
      store_out<OutT>(dx, m * K + k, __fmul_rn(r, d));
    }
    __syncthreads();
  }
}

}  // namespace bl
