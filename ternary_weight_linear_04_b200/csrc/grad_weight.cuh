// grad_weight.cuh -- gradient of the latent weights from the 8-bit tokens,
//
//   dW[n,k] = sum_m (dy[m,n] f_m) x~[m,k],   f_m = eta_m / 127,
//
// as an exact integer contraction on the tensor core (tcgen05 kind::i8).
//
// The tokens are int8 already.  The other factor, g[m,n] = dy[m,n] f_m, is
// held in fixed point: over each chunk of 512 tokens a column n gets the
// power of two that brings its largest |g| just below the top of ND signed
// base-256 digits (k_gw_digits), q = round(g 2^e) = sum_j d_j 256^j with
// d_j in [-128, 127].  The MMA sums d_j x~ over a chunk without any rounding
// (at most 512 * 128 * 127 < 2^23), and the epilogue adds D_j 256^j 2^-e to
// fp32 accumulators in registers.  ND = 3 (23 bits beside the column's
// largest value in the chunk) for fp32 results, ND = 2 (15 bits, against
// the 8 of the result) for bf16 ones.
//
// Why integers: bf16 operands would need the token's value x~ f rounded to
// 8 bits, or two such parts and two products (measured: 2.4e-6 off in the
// 2-norm, and the fp32 accumulator of kind::f16 truncates, which pulls a
// sum of 2048 tokens 4e-6 towards zero).  Two or three int8 products take
// the time of 1 or 1.5 bf16 products and sum exactly.
//
// Both operands are rewritten once with the tokens contiguous (K-major):
// the digits by k_gw_digits, the codes by k_gw_codes.
#pragma once

#include <cuda.h>

#include "common.cuh"
#include "grad.cuh"
#include "tc_bf16.cuh"

namespace bl {

constexpr int kGwChunk = 512;  // tokens that share a column's exponent

// ---------------------------------------------------------------- operands

// Digits of a 32-column, 512-token tile: lane = column, a warp takes 64
// tokens in groups of 4, whose digits fill one word.  digits: ND planes of
// N x Mp bytes (Mp a multiple of 16, zero past M); scale[chunk * N + n] =
// 2^-e, or NaN where the column holds an infinity or a NaN (its whole
// gradient row is then NaN, as it would be in floating point).
template <typename DyT, int ND>
__global__ void __launch_bounds__(256)
    k_gw_digits(const DyT* __restrict__ dy, const float* __restrict__ eta, int64_t M, int64_t N, int64_t Mp,
                uint8_t* __restrict__ digits, float* __restrict__ scale) {
  constexpr int kPitch = kGwChunk + 4;  // bytes: 129 words, so 32 columns lie in 32 banks
  constexpr float kTop = ND == 3 ? 8355711.0f : 32639.0f;  // 127 (1 + 256 (+ 65536)): the largest q
  constexpr int kBits = ND == 3 ? 22 : 14;
  extern __shared__ uint8_t smem[];  // ND x 32 x kPitch
  __shared__ uint32_t s_max[8][32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t ntiles = (N + 31) / 32;
  const int64_t chunk = blockIdx.x / ntiles;
  const int64_t n0 = (blockIdx.x % ntiles) * 32, n = n0 + lane;
  const int64_t mc = chunk * kGwChunk, mw = mc + warp * 64;
  float g[64];
  uint32_t mx = 0;
#pragma unroll
  for (int i = 0; i < 64; ++i) {
    const int64_t m = mw + i;
    g[i] = n < N && m < M ? ld_f32(dy + m * N + n) : 0.0f;
  }
#pragma unroll
  for (int i = 0; i < 64; ++i) {
    const int64_t m = mw + i;
    if (m < M) g[i] = __fmul_rn(g[i], div127_rn(__ldg(eta + m)));
    mx = max(mx, __float_as_uint(g[i]) & 0x7FFFFFFFu);  // orders magnitudes, infinities and NaN last
  }
  s_max[warp][lane] = mx;
  __syncthreads();
  for (int w = 0; w < 8; ++w) mx = max(mx, s_max[w][lane]);
  // 2^e with the largest |g| 2^e in [2^kBits, 2^(kBits+1)), one less if that
  // passes kTop; kept where 2^e and 2^-e are normal numbers
  int e = kBits + 127 - static_cast<int>(mx >> 23);
  e = min(max(e, -113), 120);
  if (__fmul_rn(__uint_as_float(mx), __uint_as_float(static_cast<uint32_t>(e + 127) << 23)) > kTop) --e;
  const bool finite = mx < 0x7F800000u;
  const float up = finite ? __uint_as_float(static_cast<uint32_t>(e + 127) << 23) : 0.0f;
  if (warp == 0 && n < N)
    scale[chunk * N + n] = finite ? __uint_as_float(static_cast<uint32_t>(127 - e) << 23) : __uint_as_float(0x7FC00000u);
#pragma unroll
  for (int i = 0; i < 64; i += 4) {
    uint32_t w[ND];
#pragma unroll
    for (int j = 0; j < ND; ++j) w[j] = 0;
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      int q = finite ? __float2int_rn(__fmul_rn(g[i + b], up)) : 0;
#pragma unroll
      for (int j = 0; j < ND; ++j) {  // low digit first; d in [-128, 127]
        const int d = static_cast<int>(static_cast<int8_t>(q & 0xFF));
        w[j] |= static_cast<uint32_t>(d & 0xFF) << (8 * b);
        q = (q - d) >> 8;
      }
    }
#pragma unroll
    for (int j = 0; j < ND; ++j)
      *reinterpret_cast<uint32_t*>(smem + (j * 32 + lane) * kPitch + warp * 64 + i) = w[j];
  }
  __syncthreads();
  // out: a warp writes one column's 512 bytes at a time
  for (int c = warp; c < 32 * ND; c += 8) {
    const int j = c >> 5, col = c & 31;
    const int64_t m = mc + lane * 16;
    if (n0 + col < N && m < Mp) {
      const uint32_t* src = reinterpret_cast<const uint32_t*>(smem + (j * 32 + col) * kPitch) + lane * 4;
      *reinterpret_cast<uint4*>(digits + (j * N + n0 + col) * Mp + m) = make_uint4(src[0], src[1], src[2], src[3]);
    }
  }
}

// The codes with the tokens contiguous: xt (K x Mp) from xq (M x K), zero
// past M.  Tiles of 64 inputs by 128 tokens, transposed 4 x 4 bytes at a time
// on the way into shared memory.
__global__ void __launch_bounds__(256)
    k_gw_codes(const int8_t* __restrict__ xq, int64_t M, int64_t K, int64_t Mp, uint8_t* __restrict__ xt) {
  __shared__ uint32_t tile[64][33];
  const int64_t ktiles = (K + 63) / 64;
  const int64_t k0 = (blockIdx.x % ktiles) * 64, m0 = (blockIdx.x / ktiles) * 128;
  const int kq = threadIdx.x & 15, mq = threadIdx.x >> 4;
  const bool words = (K & 3) == 0;
#pragma unroll
  for (int it = 0; it < 2; ++it) {
    const int64_t k = k0 + 4 * kq, m = m0 + 4 * (mq + 16 * it);
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      w[i] = 0;
      if (m + i < M && k < K) {
        const int8_t* p = xq + (m + i) * K + k;
        if (words) {
          w[i] = *reinterpret_cast<const uint32_t*>(p);
        } else {
#pragma unroll
          for (int b = 0; b < 4; ++b)
            if (k + b < K) w[i] |= static_cast<uint32_t>(static_cast<uint8_t>(p[b])) << (8 * b);
        }
      }
    }
    uint32_t o[4];
    transpose4x4_bytes(w[0], w[1], w[2], w[3], o[0], o[1], o[2], o[3]);
#pragma unroll
    for (int i = 0; i < 4; ++i) tile[4 * kq + i][mq + 16 * it] = o[i];
  }
  __syncthreads();
#pragma unroll
  for (int it = 0; it < 2; ++it) {
    const int row = (threadIdx.x >> 3) + 32 * it, c = threadIdx.x & 7;
    const int64_t m = m0 + 16 * c;
    if (k0 + row < K && m < Mp)
      *reinterpret_cast<uint4*>(xt + (k0 + row) * Mp + m) =
          make_uint4(tile[row][4 * c], tile[row][4 * c + 1], tile[row][4 * c + 2], tile[row][4 * c + 3]);
  }
}

// ---------------------------------------------------------------- product
//
// Persistent CTAs, tiles of 128 outputs n (TMEM lanes) by 256 inputs k
// (columns).  For each chunk of 512 tokens the codes' four 256 x 128-token
// blocks stay in shared memory while the ND digit planes pass through a ring
// of 128 x 128-token tiles against them: one digit of one chunk is a pass of
// four steps into one of two TMEM accumulators, and eight warps add the
// finished pass to their registers (128 values a thread) while the next one
// runs into the other.  Digits go from high to low.

constexpr int kGwBM = 128;   // tokens per step
constexpr int kGwBN = 256;   // inputs per tile
constexpr int kGwSlots = 4;  // code blocks held
constexpr int kGwStages = 6;
constexpr int kGwThreads = 32 * 10;
constexpr int kGwABytes = 128 * kGwBM, kGwBBytes = kGwBN * kGwBM;
constexpr int kGwBars = 2 * kGwStages + 2 * kGwSlots + 4 + 1;
constexpr size_t kGwSmem = 1024 + kGwStages * kGwABytes + kGwSlots * kGwBBytes + 8 * kGwBars + 16;
static_assert(kGwSmem <= 227 * 1024, "shared memory per CTA");
static_assert(kGwChunk == kGwSlots * kGwBM, "a chunk's codes are held whole");

// Position in a ring of n barriers: slot and phase parity.  A consumer waits
// for `full` with the parity, a producer for `empty` with its opposite (a
// fresh barrier counts as empty).
struct Ring {
  int s = 0;
  uint32_t ph = 0;
  __device__ __forceinline__ void next(int n) {
    if (++s == n) {
      s = 0;
      ph ^= 1u;
    }
  }
};

template <int ND, typename OutT>
__global__ void __launch_bounds__(kGwThreads, 1)
    k_grad_weight(const __grid_constant__ CUtensorMap tm_d, const __grid_constant__ CUtensorMap tm_x,
                  const float* __restrict__ scale, int M, int N, int K, void* __restrict__ dw, int vec) {
  constexpr int S = kGwStages, SB = kGwSlots;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint8_t* sA = base;
  uint8_t* sB = sA + S * kGwABytes;
  uint64_t* full_a = reinterpret_cast<uint64_t*>(sB + SB * kGwBBytes);
  uint64_t* empty_a = full_a + S;
  uint64_t* full_b = empty_a + S;
  uint64_t* empty_b = full_b + SB;
  uint64_t* acc_full = empty_b + SB;   // [2] a pass is in TMEM
  uint64_t* acc_empty = acc_full + 2;  // [2] it has been read (8 warps)
  uint64_t* drain = acc_empty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int ktiles = (K + kGwBN - 1) / kGwBN;
  const int64_t tiles = static_cast<int64_t>(ktiles) * ((N + 127) / 128);
  const int chunks = (M + kGwChunk - 1) / kGwChunk;
  const int steps = (M + kGwBM - 1) / kGwBM;  // of 128 tokens

  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(full_a + s, 1);
      mbar_init(empty_a + s, 1);
    }
    for (int s = 0; s < SB; ++s) {
      mbar_init(full_b + s, 1);
      mbar_init(empty_b + s, 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(acc_full + b, 1);
      mbar_init(acc_empty + b, 8);
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    mbar_init_fence();
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_d = *tmem_slot;
  Ring mine;  // warp 0: the lane's next slot

  if (warp == 0) {
    if (lane == 0) {  // digit tiles
      bool ok = true;
      for (int64_t t = blockIdx.x; ok && t < tiles; t += gridDim.x) {
        const int n0 = static_cast<int>(t / ktiles) * 128;
        for (int c = 0; ok && c < chunks; ++c)
          for (int j = ND - 1; ok && j >= 0; --j)
            for (int st = c * SB; st < steps && st < (c + 1) * SB; ++st, mine.next(S)) {
              ok = mbar_wait(empty_a + mine.s, mine.ph ^ 1u, abort_flag);
              if (!ok) break;
              mbar_arrive_expect_tx(full_a + mine.s, kGwABytes);
              tma_load_3d(sA + mine.s * kGwABytes, &tm_d, full_a + mine.s, st * kGwBM, n0, j);
            }
      }
    } else if (lane == 1) {  // code blocks
      bool ok = true;
      for (int64_t t = blockIdx.x; ok && t < tiles; t += gridDim.x) {
        const int k0 = static_cast<int>(t % ktiles) * kGwBN;
        for (int st = 0; st < steps; ++st, mine.next(SB)) {
          ok = mbar_wait(empty_b + mine.s, mine.ph ^ 1u, abort_flag);
          if (!ok) break;
          mbar_arrive_expect_tx(full_b + mine.s, kGwBBytes);
          tma_load_2d(sB + mine.s * kGwBBytes, &tm_x, full_b + mine.s, st * kGwBM, k0);
        }
      }
    }
  } else if (warp == 1) {
    if (lane == 0) {
      constexpr uint32_t idesc = make_idesc_i8(128, kGwBN);
      const uint64_t a_desc0 = make_sw128_kmajor_desc(smem_u32(sA));
      const uint64_t b_desc0 = make_sw128_kmajor_desc(smem_u32(sB));
      Ring ra, rb, acc;  // rb: the chunk's first block
      bool ok = true;
      for (int64_t t = blockIdx.x; ok && t < tiles; t += gridDim.x)
        for (int c = 0; ok && c < chunks; ++c) {
          const int nst = min(SB, steps - c * SB);
          Ring b = rb;
          for (int j = ND - 1; ok && j >= 0; --j, acc.next(2)) {
            ok = mbar_wait(acc_empty + acc.s, acc.ph ^ 1u, abort_flag);
            tc_fence_after();
            b = rb;
            for (int st = 0; ok && st < nst; ++st, ra.next(S), b.next(SB)) {
              ok = (j != ND - 1 || mbar_wait(full_b + b.s, b.ph, abort_flag)) &&
                   mbar_wait(full_a + ra.s, ra.ph, abort_flag);
              if (!ok) break;
              tc_fence_after();
              const uint64_t ad = a_desc0 + static_cast<uint64_t>(ra.s * (kGwABytes >> 4));
              const uint64_t bd = b_desc0 + static_cast<uint64_t>(b.s * (kGwBBytes >> 4));
#pragma unroll
              for (int kk = 0; kk < kGwBM / 32; ++kk)
                tc_mma_i8_ss(tmem_d + 256 * acc.s, ad + 2 * kk, bd + 2 * kk, idesc, st != 0 || kk != 0 ? 1u : 0u);
              tc_commit(empty_a + ra.s);
              if (j == 0) tc_commit(empty_b + b.s);
            }
            if (ok) tc_commit(acc_full + acc.s);
          }
          rb = b;
        }
      if (!ok) {  // let the MMAs in flight finish before TMEM is freed
        tc_commit(drain);
        mbar_drain(drain, 0);
      }
    }
  } else {
    // ---------------- accumulate and store: lane = output n, 128 columns
    const int qd = warp & 3, part = (warp - 2) >> 2;
    const uint32_t trow = tmem_d + 128 * part + (static_cast<uint32_t>(qd * 32) << 16);
    Ring pass;
    bool ok = true;
    for (int64_t t = blockIdx.x; ok && t < tiles; t += gridDim.x) {
      const int k0 = static_cast<int>(t % ktiles) * kGwBN + 128 * part;
      const int64_t n = t / ktiles * 128 + 32 * qd + lane;
      float acc[128];
#pragma unroll
      for (int i = 0; i < 128; ++i) acc[i] = 0.0f;
      for (int c = 0; ok && c < chunks; ++c) {
        float sc = n < N ? __ldg(scale + static_cast<int64_t>(c) * N + n) : 0.0f;
        sc = __fmul_rn(sc, ND == 3 ? 65536.0f : 256.0f);
#pragma unroll 1
        for (int j = 0; j < ND; ++j, pass.next(2)) {
          ok = __all_sync(0xFFFFFFFFu, mbar_wait(acc_full + pass.s, pass.ph, abort_flag));
          if (!ok) break;
          tc_fence_after();
#pragma unroll
          for (int i = 0; i < 128; i += 16) {
            uint32_t v[16];
            tmem_ld_32x32b_x16(trow + 256 * pass.s + i, v);
            tmem_ld_wait();
#pragma unroll
            for (int x = 0; x < 16; ++x)
              acc[i + x] = __fmaf_rn(__int2float_rn(static_cast<int32_t>(v[x])), sc, acc[i + x]);
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(acc_empty + pass.s);
          sc = __fmul_rn(sc, 0.00390625f);
        }
      }
      if (ok && n < N) {
#pragma unroll
        for (int i = 0; i < 128; i += 16) {
          float f[16];
#pragma unroll
          for (int x = 0; x < 16; ++x) f[x] = acc[i + x];
          store16<OutT>(dw, n * K, k0 + i, K, f, vec);
        }
      }
    }
  }

  __syncwarp();
  __syncthreads();
  if (warp == 0 && lane < 2 && *abort_flag) {
    // loads that can still be in flight: the last one into each slot (a slot
    // that never had one passes at once)
    uint64_t* bars = lane == 0 ? full_a : full_b;
    const int ring = lane == 0 ? S : SB;
    for (int i = 0; i < ring; ++i) mbar_drain(bars + i, i < mine.s ? mine.ph : mine.ph ^ 1u);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_d, 512);
  }
}

}  // namespace bl
