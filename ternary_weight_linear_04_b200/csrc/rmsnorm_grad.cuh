// rmsnorm_grad.cuh -- backward pass of the RMSNorm without affine parameters
// from the 8-bit tokens the forward pass kept.
//
// The forward pass is n = x r, r = 1 / sqrt(mean(x^2) + eps), so
//   dx = r (dn - n mean_k(n dn)),
// and n is read back from its codes, n = x~ eta / 127 (the quantiser's
// rounding passes gradients unchanged); x itself is not needed.
//
// Memory bound: dn and x~ are read once and dx is written once (5 bytes a
// value in bf16).  One CTA per row; a thread holds its 8-value chunks (up to
// kRgHeld of them) in registers between the sum and the result, so rows of up
// to 16384 values are read once and longer ones twice (the second time from
// L2).  Rows that do not start on 16 bytes are read value by value in the
// same order, so a row's result does not depend on where it lies.  2048 x 8640
// bf16: 20.4 us on rotating inputs, 4.3 TB/s of the 6.5 a copy reaches (the
// sum and the result of a row do not overlap; the CTAs beside it fill in).
#pragma once

#include "common.cuh"
#include "decode.cuh"
#include "grad.cuh"

namespace bl {

constexpr int kRgHeld = 4;           // chunks of 8 a thread holds
constexpr int kRgMaxThreads = 512;

// Eight values (n of them inside the row) as they lie in memory, and value j.
template <typename T>
struct Raw8 {
  uint32_t w[sizeof(T) * 2];

  __device__ __forceinline__ void load(const T* p, int n, bool vec) {
    if (vec) {
#pragma unroll
      for (int i = 0; i < static_cast<int>(sizeof(T)) / 2; ++i) {
        const uint4 a = reinterpret_cast<const uint4*>(p)[i];
        w[4 * i] = a.x; w[4 * i + 1] = a.y; w[4 * i + 2] = a.z; w[4 * i + 3] = a.w;
      }
    } else if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int i = 0; i < 8; ++i) w[i] = i < n ? reinterpret_cast<const uint32_t*>(p)[i] : 0u;
    } else {
      const uint16_t* h = reinterpret_cast<const uint16_t*>(p);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        w[i] = (2 * i < n ? h[2 * i] : 0u) | (2 * i + 1 < n ? static_cast<uint32_t>(h[2 * i + 1]) << 16 : 0u);
    }
  }

  __device__ __forceinline__ float get(int j) const {
    if constexpr (sizeof(T) == 4) return __uint_as_float(w[j]);
    else return __uint_as_float((j & 1) ? w[j / 2] & 0xFFFF0000u : w[j / 2] << 16);
  }
};

// Eight codes with their sign bits flipped (c + 128 as unsigned bytes).
__device__ __forceinline__ uint2 load8_codes(const int8_t* p, int n, bool vec) {
  uint2 w = make_uint2(0, 0);
  if (vec) {
    w = *reinterpret_cast<const uint2*>(p);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t b = i < n ? static_cast<uint32_t>(static_cast<uint8_t>(p[i])) << (8 * (i & 3)) : 0u;
      if (i < 4) w.x |= b;
      else w.y |= b;
    }
  }
  return make_uint2(w.x ^ 0x80808080u, w.y ^ 0x80808080u);
}

// Code j of load8_codes as fp32: the byte in the mantissa of 2^23, minus
// 2^23 + 128 (exact; int-to-float conversions have a quarter of the rate).
__device__ __forceinline__ float code_f32(const uint2& w, int j) {
  const uint32_t u = __byte_perm(j < 4 ? w.x : w.y, 0x4B000000u, 0x7540 | (j & 3));
  return __fsub_rn(__uint_as_float(u), 8388736.0f);
}

template <typename T>
__device__ __forceinline__ void store8(void* out, int64_t at, int n, bool vec, const float (&f)[8]) {
  if (vec) {
    if constexpr (sizeof(T) == 4) {
      float4* p = reinterpret_cast<float4*>(static_cast<float*>(out) + at);
      p[0] = make_float4(f[0], f[1], f[2], f[3]);
      p[1] = make_float4(f[4], f[5], f[6], f[7]);
    } else {
      *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(out) + at) =
          make_uint4(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]), pack_bf16(f[6], f[7]));
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) store_out<T>(out, at + i, f[i]);
  }
}

// vec: K is a multiple of 8 and every row of dn, xq and dx can be read and
// written in chunks of 8.  HELD: K <= 8 kRgHeld blockDim.x.
template <typename DnT, typename OutT, bool HELD>
__global__ void __launch_bounds__(kRgMaxThreads, sizeof(DnT) == 2 ? 2 : 1)
    k_rmsnorm_grad(const DnT* dn, const int8_t* __restrict__ xq, const float* __restrict__ eta,
                   const float* __restrict__ rstd, int64_t M, int64_t K, void* dx, int vec) {
  __shared__ float red[2][kRgMaxThreads / 32];
  const int warps = blockDim.x >> 5, step = 8 * blockDim.x;
  const int first = 8 * threadIdx.x, cols = static_cast<int>(K);
  pdl_wait();
  if (threadIdx.x == 0) pdl_trigger();
  int flip = 0;
  for (int64_t m = blockIdx.x; m < M; m += gridDim.x, flip ^= 1) {
    const DnT* row = dn + m * K;
    const int8_t* codes = xq + m * K;
    Raw8<DnT> d[kRgHeld];
    uint2 q[kRgHeld];
    const float e = __ldg(eta + m), r = __ldg(rstd + m);
    float s = 0.0f;
    for (int base = first; base < (HELD ? first + 1 : cols); base += kRgHeld * step) {
#pragma unroll
      for (int i = 0; i < kRgHeld; ++i) {
        const int k = base + i * step;
        if (k < cols) {
          d[i].load(row + k, cols - k, vec);
          q[i] = load8_codes(codes + k, cols - k, vec);
        }
      }
#pragma unroll
      for (int i = 0; i < kRgHeld; ++i)
        if (base + i * step < cols) {
#pragma unroll
          for (int j = 0; j < 8; ++j) s = __fmaf_rn(code_f32(q[i], j), d[i].get(j), s);
        }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
    if ((threadIdx.x & 31) == 0) red[flip][threadIdx.x >> 5] = s;
    __syncthreads();
    s = 0.0f;
    for (int w = 0; w < warps; ++w) s += red[flip][w];
    const float f = div127_rn(e);
    const float c = __fdiv_rn(__fmul_rn(__fmul_rn(s, f), f), static_cast<float>(K));  // x~ c = n mean(n dn)
    for (int base = first; base < (HELD ? first + 1 : cols); base += kRgHeld * step) {
#pragma unroll
      for (int i = 0; i < kRgHeld; ++i) {
        const int k = base + i * step;
        if (k < cols) {
          if (!HELD) {
            d[i].load(row + k, cols - k, vec);
            q[i] = load8_codes(codes + k, cols - k, vec);
          } else {
            // keep the codes, not the 32 floats they were in the sum (120 registers)
            asm volatile("" : "+r"(q[i].x), "+r"(q[i].y));
          }
          float o[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) o[j] = __fmul_rn(r, __fmaf_rn(-code_f32(q[i], j), c, d[i].get(j)));
          store8<OutT>(dx, m * K + k, cols - k, vec, o);
        }
      }
    }
  }
}

}  // namespace bl
