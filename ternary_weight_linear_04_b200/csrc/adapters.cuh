// adapters.cuh -- low-rank adapters of many requests beside one ternary
// projection.  Token m uses adapter a = ids[m] (none when outside [0, L)):
//
//   u[m,:]   = scale_a (eta_m / 127) x~[m,:] A_a^T         (r values)
//   y[m,n]   = (ternary projection) + sum_j u[m,j] B_a[n,j]
//   v[m,:]   = scale_a dy[m,:] B_a
//   dx[m,k]  = (ternary input gradient) + sum_j v[m,j] A_a[j,k]
//   dA_a     = sum_{m of a} v[m,:]^T (eta_m / 127) x~[m,:]
//   dB_a     = sum_{m of a} dy[m,:]^T u[m,:]
//
// A is L x r x K, B is L x N x r (bf16); sums in fp32.
#pragma once

#include "common.cuh"
#include "grad.cuh"

namespace bl {

__device__ __forceinline__ float warp_sum(float s) {
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
  return s;
}

// One warp per (token, rank index).
__global__ void __launch_bounds__(256)
    k_adapter_u(const int8_t* __restrict__ xq, const float* __restrict__ eta, int64_t M, int64_t K,
                const __nv_bfloat16* __restrict__ A, const float* __restrict__ scale,
                const int32_t* __restrict__ ids, int L, int r, float* __restrict__ u) {
  const int lane = threadIdx.x & 31;
  for (int64_t i = blockIdx.x * 8ll + (threadIdx.x >> 5); i < M * r; i += gridDim.x * 8ll) {
    const int64_t m = i / r, j = i % r;
    const int a = adapter_of(ids, m, L);
    float s = 0.0f;
    if (a >= 0) {
      const __nv_bfloat16* row = A + (static_cast<int64_t>(a) * r + j) * K;
      for (int64_t k = lane; k < K; k += 32)
        s = __fmaf_rn(static_cast<float>(xq[m * K + k]), __bfloat162float(row[k]), s);
      s = __fmul_rn(__fmul_rn(warp_sum(s), div127_rn(eta[m])), scale[a]);
    }
    if (lane == 0) u[i] = s;
  }
}

template <typename DyT>
__global__ void __launch_bounds__(256)
    k_adapter_v(const DyT* __restrict__ dy, int64_t M, int64_t N, const __nv_bfloat16* __restrict__ B,
                const float* __restrict__ scale, const int32_t* __restrict__ ids, int L, int r,
                float* __restrict__ v) {
  const int lane = threadIdx.x & 31;
  for (int64_t i = blockIdx.x * 8ll + (threadIdx.x >> 5); i < M * r; i += gridDim.x * 8ll) {
    const int64_t m = i / r, j = i % r;
    const int a = adapter_of(ids, m, L);
    float s = 0.0f;
    if (a >= 0) {
      for (int64_t n = lane; n < N; n += 32)
        s = __fmaf_rn(ld_f32(dy + m * N + n), __bfloat162float(B[(a * N + n) * r + j]), s);
      s = __fmul_rn(warp_sum(s), scale[a]);
    }
    if (lane == 0) v[i] = s;
  }
}

// out[m,n] = base[m,n] + sum_j u[m,j] B_a[n,j]; jstride/nstride address the
// factor so that the same kernel adds v A (factor A_a[j,k]).
template <typename OutT>
__global__ void __launch_bounds__(256)
    k_adapter_add(const float* __restrict__ base, int64_t M, int64_t N, const float* __restrict__ u,
                  const __nv_bfloat16* __restrict__ F, int64_t nstride, int64_t jstride,
                  const int32_t* __restrict__ ids, int L, int r, void* __restrict__ out) {
  for (int64_t i = blockIdx.x * 256ll + threadIdx.x; i < M * N; i += gridDim.x * 256ll) {
    const int64_t m = i / N, n = i % N;
    const int a = adapter_of(ids, m, L);
    float s = base[i];
    if (a >= 0) {
      const __nv_bfloat16* f = F + static_cast<int64_t>(a) * r * N + n * nstride;
      float t = 0.0f;
      for (int j = 0; j < r; ++j) t = __fmaf_rn(u[m * r + j], __bfloat162float(f[j * jstride]), t);
      s = __fadd_rn(s, t);
    }
    store_out<OutT>(out, i, s);
  }
}

template <typename OutT>
__global__ void __launch_bounds__(256)
    k_adapter_da(const float* __restrict__ v, const int8_t* __restrict__ xq, const float* __restrict__ eta,
                 int64_t M, int64_t K, const int32_t* __restrict__ ids, int L, int r, void* __restrict__ dA) {
  for (int64_t i = blockIdx.x * 256ll + threadIdx.x; i < L * r * K; i += gridDim.x * 256ll) {
    const int64_t k = i % K, aj = i / K, j = aj % r, a = aj / r;
    float s = 0.0f;
    for (int64_t m = 0; m < M; ++m)
      if (ids[m] == a)
        s = __fmaf_rn(__fmul_rn(v[m * r + j], div127_rn(eta[m])), static_cast<float>(xq[m * K + k]), s);
    store_out<OutT>(dA, i, s);
  }
}

template <typename DyT, typename OutT>
__global__ void __launch_bounds__(256)
    k_adapter_db(const DyT* __restrict__ dy, const float* __restrict__ u, int64_t M, int64_t N,
                 const int32_t* __restrict__ ids, int L, int r, void* __restrict__ dB) {
  for (int64_t i = blockIdx.x * 256ll + threadIdx.x; i < L * N * r; i += gridDim.x * 256ll) {
    const int64_t j = i % r, an = i / r, n = an % N, a = an / N;
    float s = 0.0f;
    for (int64_t m = 0; m < M; ++m)
      if (ids[m] == a) s = __fmaf_rn(ld_f32(dy + m * N + n), u[m * r + j], s);
    store_out<OutT>(dB, i, s);
  }
}

}  // namespace bl
