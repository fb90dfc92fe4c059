// grad_weight.cuh -- gradient of the latent weights from the 8-bit tokens,
//
//   dW[n,k] = sum_m (dy[m,n] f_m) x~[m,k],   f_m = eta_m / 127,
//
// as an exact integer contraction on the tensor core (tcgen05 kind::i8).
//
// The tokens are int8 already.  The other factor, g[m,n] = dy[m,n] f_m, is
// held in fixed point: over each chunk of 1024 tokens a column n gets the
// power of two that brings its largest |g| just below the top of three signed
// base-256 digits (k_gw_operands), q = round(g 2^e) = sum_p d_p 256^(2-p) with
// d_p in [-128, 127].  The MMA sums d_p x~ over a chunk without any rounding
// (at most 1024 * 128 * 127 < 2^24, so exact in fp32 too), and the epilogue
// adds D_p 256^(2-p) 2^-e to fp32 accumulators in registers.
//
// Three digits are 23 bits beside the column's largest value in the chunk.
// That is finer than an fp32 sum while the values are of like size, but one
// token with a large eta or a large gradient leaves the others few bits, and
// outputs that it does not reach (its codes there are zero) would show it.  So
// a block of 64 columns has a fourth and a fifth digit of g in a chunk where,
// in some column, the largest |g| lies more than 2^4 and 2^12 above the
// geometric mean of those that are not zero (in binary exponents): an error is
// then at most 2^-17.9 of that mean for each token, while the largest is no more
// than 2^20 above it.  Normal gradients are 2^2.5 to 2^3.5 above: three digits.
// (One token 2^10 times the others: outputs without it were 5.8e-5 off in the
// 2-norm with three digits.)
//
// Why integers: bf16 operands would need the token's value x~ f rounded to
// 8 bits, or two such parts and two products (measured: 2.4e-6 off in the
// 2-norm, and the fp32 accumulator of kind::f16 cuts off, which pulls a
// sum of 2048 tokens 4e-6 towards zero).  Three int8 products take the time of
// 1.5 bf16 products and sum exactly.
//
// k_gw_operands rewrites both operands once with the tokens contiguous
// (K-major).
#pragma once

#include <cuda.h>

#include "common.cuh"
#include "decode.cuh"
#include "grad.cuh"
#include "tc_bf16.cuh"

namespace bl {

constexpr int kGwChunk = 1024;  // tokens that share a column's exponent
constexpr int kGdTokens = 512;  // of a CTA that makes digits; two CTAs share a chunk

// ---------------------------------------------------------------- operands

// Digits of a 64-column, 512-token tile (a cluster of two CTAs makes a chunk's
// and shares its maxima): lane = two neighbouring columns, a warp takes 32
// tokens, held as they were read (two bf16 in a register) between the column's
// maximum and the digits.  digits: five planes of N x Mp bytes (Mp a multiple
// of 16, zero past M), the largest digit first, the fourth and fifth written
// where they are used; extra[chunk * groups + n / 64] = 0, 1 or 2, how many of
// those are (groups: column blocks, rounded up to four); scale[chunk * N + n] =
// 2^-e, or NaN where the column holds an infinity or a NaN (its whole gradient
// row is then NaN).
//
// Rounding and splitting use no conversion instruction (a quarter of the
// rate of an add): adding 1.5 2^23 rounds a value below 2^22 to an integer in
// the low bits, and the bytes of q + 0x808080 with their top bits flipped
// are the signed digits.  2048 x 11008, three digits, cold: 101 us with
// conversions, bound by their pipe, 46 us so (44 instructions a value, three
// of them for the spread).
constexpr int kGdCols = 64;
constexpr int kGdThreads = 512;

constexpr int kGdPlanes = 5;

// q + 0x808080, q = p rounded to an integer.
__device__ __forceinline__ uint32_t biased_round(float p) {
  constexpr float kMagic = 12582912.0f;  // 1.5 2^23
  constexpr uint32_t kBits = 0x4B400000u;
  // |p| passes 2^22: a multiple of 4096 first, the rest is exact
  const float h = __fmaf_rn(p, 0x1p-12f, kMagic);
  const float l = __fadd_rn(__fmaf_rn(__fsub_rn(h, kMagic), -4096.0f, p), kMagic);
  return __float_as_uint(h) * 4096u + (__float_as_uint(l) + (0x808080u - 4097u * kBits));
}

// The same of p 2^16 with five digits: the upper three (PLANE 0) or the lower
// two (PLANE 3) in the low bytes.
template <int PLANE>
__device__ __forceinline__ uint32_t biased_round_wide(float p) {
  const long long q = __float2ll_rn(__fmul_rn(p, 65536.0f)) + 0x8080808080ll;
  return static_cast<uint32_t>(PLANE == 0 ? q >> 16 : q & 0xFFFF);
}

// Digits of a tile's outputs in a chunk, from the four bytes of `extra`.
__device__ __forceinline__ int gw_digits(uint32_t extra4) { return (extra4 & 0x02020202u) ? 5 : (extra4 & 0x01010101u) ? 4 : 3; }

// The codes with the tokens contiguous: a tile of 64 inputs by 128 tokens of
// xt (K x Mp) from xq (M x K), zero past M, transposed 4 x 4 bytes at a time
// on the way into shared memory.
__device__ __forceinline__ void gw_codes_tile(const int8_t* __restrict__ xq, int64_t M, int64_t K, int64_t Mp,
                                              int64_t at, uint32_t (&tile)[64][33], uint8_t* __restrict__ xt) {
  const int64_t ktiles = (K + 63) / 64;
  const int64_t k0 = (at % ktiles) * 64, m0 = (at / ktiles) * 128;
  const int kq = threadIdx.x & 15, mq = threadIdx.x >> 4;
  const int64_t k = k0 + 4 * kq, m = m0 + 4 * mq;
  uint32_t w[4], o[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    w[i] = 0;
    if (m + i < M && k < K) {
      const int8_t* p = xq + (m + i) * K + k;
      if ((K & 3) == 0) {
        w[i] = __ldg(reinterpret_cast<const uint32_t*>(p));
      } else {
#pragma unroll
        for (int b = 0; b < 4; ++b)
          if (k + b < K) w[i] |= static_cast<uint32_t>(static_cast<uint8_t>(__ldg(p + b))) << (8 * b);
      }
    }
  }
  transpose4x4_bytes(w[0], w[1], w[2], w[3], o[0], o[1], o[2], o[3]);
#pragma unroll
  for (int i = 0; i < 4; ++i) tile[4 * kq + i][mq] = o[i];
  __syncthreads();
  const int row = threadIdx.x >> 3, c = threadIdx.x & 7;
  const int64_t mc = m0 + 16 * c;
  if (k0 + row < K && mc < Mp)
    *reinterpret_cast<uint4*>(xt + (k0 + row) * Mp + mc) =
        make_uint4(tile[row][4 * c], tile[row][4 * c + 1], tile[row][4 * c + 2], tile[row][4 * c + 3]);
}

// Both operands in one launch: blocks below digit_blocks make digits, the
// others codes.
template <typename DyT>
__global__ void __launch_bounds__(kGdThreads, sizeof(DyT) == 2 ? 2 : 1)
    k_gw_operands(unsigned digit_blocks, const int8_t* __restrict__ xq, int64_t K, uint8_t* __restrict__ xt,
                  const DyT* __restrict__ dy, const float* __restrict__ eta, int64_t M, int64_t N, int64_t Mp,
                  int pairs, uint8_t* __restrict__ digits, float* __restrict__ scale, uint8_t* __restrict__ extra) {
  constexpr float kTop = 8355711.0f;  // 127 (1 + 256 + 65536): the largest q
  constexpr int kBits = 22;
  constexpr int kRegs = sizeof(DyT) == 2 ? 1 : 2;
  extern __shared__ __align__(16) uint8_t smem[];  // 3 x 64 columns x 512 bytes, words XORed with the lane
  __shared__ __align__(16) uint32_t s_max[16][kGdCols];
  __shared__ uint32_t s_col[2][kGdCols];
  __shared__ float s_f[kGdTokens];
  __shared__ __align__(16) uint32_t s_codes[64][33];
  auto& s_exp = reinterpret_cast<uint32_t(&)[16][kGdCols]>(s_codes);  // (other blocks': two CTAs have to fit an SM)
  uint32_t* words = reinterpret_cast<uint32_t*>(smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t ntiles = (N + kGdCols - 1) / kGdCols;
  const int64_t chunk = (blockIdx.x >> 1) / ntiles;
  const int64_t n0 = ((blockIdx.x >> 1) % ntiles) * kGdCols, n = n0 + 2 * lane;
  const int64_t mc = chunk * kGwChunk + (blockIdx.x & 1) * kGdTokens;
  pdl_wait();
  if (threadIdx.x == 0) pdl_trigger();
  if (blockIdx.x >= digit_blocks) {
    if (blockIdx.x - digit_blocks < (K + 63) / 64 * ((M + 127) / 128)) gw_codes_tile(xq, M, K, Mp, blockIdx.x - digit_blocks, s_codes, xt);
    return;
  }
  uint32_t raw[32][kRegs];
  const int rows = static_cast<int>(min(static_cast<int64_t>(32), M - mc - 32 * warp));  // of this warp, may be < 1
  const DyT* src = dy + (mc + 32 * warp) * N + n;
  const bool in0 = n < N, in1 = n + 1 < N;
  if (pairs) {
#pragma unroll
    for (int i = 0; i < 32; ++i, src += N) {
      if constexpr (kRegs == 1) {
        raw[i][0] = in0 && i < rows ? __ldg(reinterpret_cast<const unsigned*>(src)) : 0u;
      } else {
        const uint2 v = in0 && i < rows ? __ldg(reinterpret_cast<const uint2*>(src)) : make_uint2(0, 0);
        raw[i][0] = v.x;
        raw[i][kRegs - 1] = v.y;
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < 32; ++i, src += N) {
      if constexpr (kRegs == 1) {
        const uint16_t* h = reinterpret_cast<const uint16_t*>(src);
        raw[i][0] = (in0 && i < rows ? static_cast<uint32_t>(__ldg(h)) : 0u) |
                    (in1 && i < rows ? static_cast<uint32_t>(__ldg(h + 1)) << 16 : 0u);
      } else {
        const uint32_t* h = reinterpret_cast<const uint32_t*>(src);
        raw[i][0] = in0 && i < rows ? __ldg(h) : 0u;
        raw[i][kRegs - 1] = in1 && i < rows ? __ldg(h + 1) : 0u;
      }
    }
  }
  {
    const int64_t m = mc + threadIdx.x;
    s_f[threadIdx.x] = m < M ? div127_rn(__ldg(eta + m)) : 0.0f;
  }
  __syncthreads();
  auto g_of = [&](int i, int c) {  // dy f of the warp's token i, column c
    const uint32_t u = kRegs == 2 ? raw[i][kRegs == 2 ? c : 0] : c ? raw[i][0] & 0xFFFF0000u : raw[i][0] << 16;
    return __fmul_rn(__uint_as_float(u), s_f[32 * warp + i]);
  };
  // a column's largest magnitude, and of those that are not zero the number
  // (from bit 20 on) and the sum of the exponents (at most 1024 * 255)
  uint32_t mx[2] = {0, 0}, ex[2] = {0, 0};
#pragma unroll
  for (int i = 0; i < 32; i += 2)
#pragma unroll
    for (int c = 0; c < 2; ++c) {  // orders magnitudes, infinities and NaN last
      const uint32_t a = __float_as_uint(g_of(i, c)) & 0x7FFFFFFFu, b = __float_as_uint(g_of(i + 1, c)) & 0x7FFFFFFFu;
      mx[c] = __vimax3_u32(mx[c], a, b);
      ex[c] += (a >> 23) + (b >> 23) + ((a ? 1u : 0u) << 20) + ((b ? 1u : 0u) << 20);
    }
  *reinterpret_cast<uint2*>(&s_max[warp][2 * lane]) = make_uint2(mx[0], mx[1]);
  *reinterpret_cast<uint2*>(&s_exp[warp][2 * lane]) = make_uint2(ex[0], ex[1]);
  __syncthreads();
  if (threadIdx.x < kGdCols) {
    uint32_t t = 0, x = 0;
#pragma unroll
    for (int w = 0; w < 16; ++w) {
      t = max(t, s_max[w][threadIdx.x]);
      x += s_exp[w][threadIdx.x];
    }
    s_col[0][threadIdx.x] = t;
    s_col[1][threadIdx.x] = x;
  }
  cluster_sync_all();
  const uint32_t other = cluster_ctarank() ^ 1u;
  int more = 0;  // digits beyond three that a column wants
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    mx[c] = max(s_col[0][2 * lane + c], __float_as_uint(ld_cluster_f32(cluster_map(&s_col[0][2 * lane + c], other))));
    ex[c] = s_col[1][2 * lane + c] + __float_as_uint(ld_cluster_f32(cluster_map(&s_col[1][2 * lane + c], other)));
    const uint32_t count = ex[c] >> 20, spread = (mx[c] >> 23) * count - (ex[c] & 0xFFFFFu);  // count times the distance
    if (mx[c] < 0x7F800000u) more = max(more, spread <= 4 * count ? 0 : spread <= 12 * count ? 1 : 2);
  }
  more = __reduce_max_sync(0xFFFFFFFFu, more);  // the block's, the same in every warp
  cluster_sync_all();  // the other CTA has read this one's
  float up[2];
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    // 2^e with the largest |g| 2^e in [2^kBits, 2^(kBits+1)), one less if that
    // passes kTop; kept where 2^e and 2^-e are normal numbers
    int e = kBits + 127 - static_cast<int>(mx[c] >> 23);
    e = min(max(e, -113), 120);
    if (__fmul_rn(__uint_as_float(mx[c]), __uint_as_float(static_cast<uint32_t>(e + 127) << 23)) > kTop) --e;
    const bool finite = mx[c] < 0x7F800000u;
    up[c] = __uint_as_float(static_cast<uint32_t>(e + 127) << 23);  // not finite: the digits do not matter
    if (warp == 0 && n + c < N && (blockIdx.x & 1) == 0)
      scale[chunk * N + n + c] = finite ? __uint_as_float(static_cast<uint32_t>(127 - e) << 23) : __uint_as_float(0x7FC00000u);
  }
  if (threadIdx.x == 0 && (blockIdx.x & 1) == 0) {
    const int64_t groups = (ntiles + 3) / 4 * 4, g = n0 / kGdCols;
    extra[chunk * groups + g] = static_cast<uint8_t>(more);
    for (int64_t r = g + 1; g + 1 == ntiles && r < groups; ++r) extra[chunk * groups + r] = 0;
  }
  // digits of four tokens at a time: byte j of `round`'s words into slot j
  auto fill = [&](auto round) {
#pragma unroll
    for (int i = 0; i < 32; i += 4) {
#pragma unroll
      for (int b = 0; b < 4; ++b) asm volatile("" : "+r"(raw[i + b][0]));  // keep dy, not the products
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        uint32_t u[4], o[4];
#pragma unroll
        for (int b = 0; b < 4; ++b) u[b] = round(__fmul_rn(g_of(i + b, c), up[c]));
        transpose4x4_bytes(u[0], u[1], u[2], u[3], o[0], o[1], o[2], o[3]);
#pragma unroll
        for (int j = 0; j < 3; ++j)
          words[(j * kGdCols + 2 * lane + c) * 128 + ((8 * warp + i / 4) ^ lane)] = o[j] ^ 0x80808080u;
      }
    }
  };
  // slots lo .. hi - 1 out, slot j as plane `top` - j: a warp writes one
  // column's 512 bytes at a time
  auto store = [&](int lo, int hi, int top) {
    for (int r = lo * kGdCols + warp; r < hi * kGdCols; r += 16) {
      const int j = r / kGdCols, col = r % kGdCols, x = col >> 1;  // x: the lane that wrote the column
      const int64_t m = mc + lane * 16;
      if (n0 + col < N && m < Mp) {
        uint4 v = *reinterpret_cast<const uint4*>(words + r * 128 + ((4 * lane) ^ (x & ~3)));
        if (x & 1) v = make_uint4(v.y, v.x, v.w, v.z);
        if (x & 2) v = make_uint4(v.z, v.w, v.x, v.y);
        *reinterpret_cast<uint4*>(digits + ((top - j) * N + n0 + col) * Mp + m) = v;
      }
    }
  };
  if (more == 0) fill([](float p) { return biased_round(p); });
  else fill([](float p) { return biased_round_wide<0>(p); });
  __syncthreads();
  store(0, 3, 2);
  if (more != 0) {
    __syncthreads();
    fill([](float p) { return biased_round_wide<3>(p); });
    __syncthreads();
    store(more == 1 ? 1 : 0, 2, 4);  // the fourth digit is slot 1, the fifth slot 0
  }
}

// ---------------------------------------------------------------- product
//
// Persistent pairs of CTAs, tiles of 256 outputs n (128 TMEM lanes of each
// CTA) by 256 inputs k (columns).  For each chunk of 1024 tokens the codes'
// eight 256 x 128-token blocks (half in each CTA) stay in shared memory while
// the digit planes pass through a ring of 128 x 128-token tiles against
// them: one digit of one chunk is a pass of eight steps into one of two TMEM
// accumulators, and eight warps of each CTA add the finished pass to their
// registers (128 values a thread) while the next one runs into the other.
// Digits go from high to low.  One CTA a tile (128 x 256) reads 12 KB of
// shared memory for each MMA of 128 cycles beside 4 KB that TMA writes, all
// that it can; a pair reads 8 KB in each.  2048 x 4096 x 11008, three digits:
// about 240 us, 2.3e15 integer operations a second; the tensor pipe waits for
// the passes to be added (a TMEM load and its use follow one another in two
// warps a scheduler), which is also why a chunk is 1024 tokens and not 512
// (322 -> 264 us for the whole call).

constexpr int kGwBM = 128;   // tokens per step
constexpr int kGwBN = 256;   // inputs per tile
constexpr int kGwRows = 256;  // outputs per tile
constexpr int kGwPer = kGwChunk / kGwBM;  // blocks of codes in a chunk
constexpr int kGwSlots = kGwPer;  // blocks held: a chunk's, each replaced by the next one's after its last digit
constexpr int kGwStages = 5;
constexpr int kGwAddWarps = 8;  // accumulate: 128 columns each
constexpr int kGwThreads = 32 * (2 + kGwAddWarps);
constexpr int kGwABytes = 128 * kGwBM, kGwBBytes = kGwBN / 2 * kGwBM;  // of one CTA
constexpr int kGwBars = 2 * kGwStages + 2 * kGwSlots + 4 + 1;
constexpr int kGwPatch = 32 * 17;  // floats of a warp's 32 x 16 outputs, turned for the stores
constexpr size_t kGwSmem = 1024 + kGwStages * kGwABytes + kGwSlots * kGwBBytes + kGwAddWarps * 4 * kGwPatch + 8 * kGwBars + 16;
static_assert(kGwSmem <= 227 * 1024, "shared memory per CTA");

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

template <typename OutT>
__global__ void __launch_bounds__(kGwThreads, 1)
    k_grad_weight(const __grid_constant__ CUtensorMap tm_d, const __grid_constant__ CUtensorMap tm_x,
                  const float* __restrict__ scale, const uint8_t* __restrict__ extra, int M, int N, int K,
                  void* __restrict__ dw) {
  constexpr int S = kGwStages, SB = kGwSlots;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint8_t* sA = base;
  uint8_t* sB = sA + S * kGwABytes;
  float* patches = reinterpret_cast<float*>(sB + SB * kGwBBytes);
  uint64_t* full_a = reinterpret_cast<uint64_t*>(patches + kGwAddWarps * kGwPatch);
  uint64_t* empty_a = full_a + S;
  uint64_t* full_b = empty_a + S;
  uint64_t* empty_b = full_b + SB;
  uint64_t* acc_full = empty_b + SB;   // [2] a pass is in TMEM
  uint64_t* acc_empty = acc_full + 2;  // [2] CTA 0: it has been read (8 warps of each CTA)
  uint64_t* drain = acc_empty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int ktiles = (K + kGwBN - 1) / kGwBN;
  const int64_t tiles = static_cast<int64_t>(ktiles) * ((N + kGwRows - 1) / kGwRows);
  const int rank = static_cast<int>(cluster_ctarank());  // in the pair
  const int64_t first = blockIdx.x >> 1, stride = gridDim.x >> 1;
  const int chunks = (M + kGwChunk - 1) / kGwChunk;
  const int steps = (M + kGwBM - 1) / kGwBM;  // of 128 tokens
  const int64_t groups = (static_cast<int64_t>(N) + kGwRows - 1) / kGwRows * 4;
  auto extra_of = [&](int64_t t, int c) {  // of tile t's four blocks of 64 outputs
    return __ldg(reinterpret_cast<const uint32_t*>(extra + c * groups + t / ktiles * 4));
  };

  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(full_a + s, 1);  // CTA 0's: the tiles of both are in
      mbar_init(empty_a + s, 1);
    }
    for (int s = 0; s < SB; ++s) {
      mbar_init(full_b + s, 1);
      mbar_init(empty_b + s, 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(acc_full + b, 1);
      mbar_init(acc_empty + b, 2 * kGwAddWarps);
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    mbar_init_fence();
  }
  if (warp == 1) {
    tmem2_alloc(tmem_slot, 512);
    tmem2_relinquish();
  }
  pdl_wait();
  if (threadIdx.x == 0) pdl_trigger();
  __syncwarp();
  tc_fence_before();
  cluster_sync_all();  // both CTAs' barriers are there
  tc_fence_after();
  const uint32_t tmem_d = *tmem_slot;
  Ring mine;  // warp 0: the lane's next slot

  if (warp == 0) {
    if (lane == 0) {  // digit tiles
      bool ok = true;
      for (int64_t t = first; ok && t < tiles; t += stride) {
        const int n0 = static_cast<int>(t / ktiles) * kGwRows + 128 * rank;
        for (int c = 0; ok && c < chunks; ++c) {
          const int nd = gw_digits(extra_of(t, c));
          for (int j = 0; ok && j < nd; ++j)
            for (int st = c * kGwPer; st < steps && st < (c + 1) * kGwPer; ++st, mine.next(S)) {
              ok = mbar_wait(empty_a + mine.s, mine.ph ^ 1u, abort_flag);
              if (!ok) break;
              if (rank == 0) mbar_arrive_expect_tx(full_a + mine.s, 2 * kGwABytes);
              tma2_load_3d(sA + mine.s * kGwABytes, &tm_d, full_a + mine.s, st * kGwBM, n0, j);
            }
        }
      }
      // the other CTA's commits have arrived here before this one may exit
      for (int i = 0; ok && i < S; ++i, mine.next(S)) ok = mbar_wait(empty_a + mine.s, mine.ph ^ 1u, abort_flag);
    } else if (lane == 1) {  // code blocks
      bool ok = true;
      for (int64_t t = first; ok && t < tiles; t += stride) {
        const int k0 = static_cast<int>(t % ktiles) * kGwBN + kGwBN / 2 * rank;
        for (int st = 0; st < steps; ++st, mine.next(SB)) {
          ok = mbar_wait(empty_b + mine.s, mine.ph ^ 1u, abort_flag);
          if (!ok) break;
          if (rank == 0) mbar_arrive_expect_tx(full_b + mine.s, 2 * kGwBBytes);
          tma2_load_2d(sB + mine.s * kGwBBytes, &tm_x, full_b + mine.s, st * kGwBM, k0);
        }
      }
      for (int i = 0; ok && i < SB; ++i, mine.next(SB)) ok = mbar_wait(empty_b + mine.s, mine.ph ^ 1u, abort_flag);
    }
  } else if (warp == 1) {
    if (lane == 0 && rank == 0) {
      constexpr uint32_t idesc = make_idesc_i8(kGwRows, kGwBN);
      const uint64_t a_desc0 = make_sw128_kmajor_desc(smem_u32(sA));
      const uint64_t b_desc0 = make_sw128_kmajor_desc(smem_u32(sB));
      Ring ra, rb, acc;  // rb: the chunk's first block
      bool ok = true;
      for (int64_t t = first; ok && t < tiles; t += stride)
        for (int c = 0; ok && c < chunks; ++c) {
          const int nst = min(kGwPer, steps - c * kGwPer), nd = gw_digits(extra_of(t, c));
          Ring b = rb;
          for (int j = 0; ok && j < nd; ++j, acc.next(2)) {
            ok = mbar_wait(acc_empty + acc.s, acc.ph ^ 1u, abort_flag);
            tc_fence_after();
            b = rb;
            for (int st = 0; ok && st < nst; ++st, ra.next(S), b.next(SB)) {
              ok = (j != 0 || mbar_wait(full_b + b.s, b.ph, abort_flag)) &&
                   mbar_wait(full_a + ra.s, ra.ph, abort_flag);
              if (!ok) break;
              tc_fence_after();
              const uint64_t ad = a_desc0 + static_cast<uint64_t>(ra.s * (kGwABytes >> 4));
              const uint64_t bd = b_desc0 + static_cast<uint64_t>(b.s * (kGwBBytes >> 4));
#pragma unroll
              for (int kk = 0; kk < kGwBM / 32; ++kk)
                tc2_mma_i8_ss(tmem_d + 256 * acc.s, ad + 2 * kk, bd + 2 * kk, idesc, st != 0 || kk != 0 ? 1u : 0u);
              tc2_commit_both(empty_a + ra.s);
              if (j == nd - 1) tc2_commit_both(empty_b + b.s);
            }
            if (ok) tc2_commit_both(acc_full + acc.s);
          }
          rb = b;
        }
      if (!ok) {  // let the MMAs in flight finish before TMEM is freed
        tc2_commit(drain);
        mbar_drain(drain, 0);
      }
    }
  } else {
    // ---------------- accumulate and store: lane = output n, 128 columns
    const int qd = warp & 3, part = (warp - 2) >> 2;
    const uint32_t trow = tmem_d + 128 * part + (static_cast<uint32_t>(qd * 32) << 16);
    float* patch = patches + (warp - 2) * kGwPatch;
    const int64_t nlast = N - 1;
    Ring pass;
    bool ok = true;
#pragma unroll 1
    for (int t = static_cast<int>(first); ok && t < tiles; t += static_cast<int>(stride)) {
      const int nw = t / ktiles * kGwRows + 128 * rank + 32 * qd;
      const float* sp = scale + min(static_cast<int64_t>(nw + lane), nlast);  // rows past N repeat the last, unused
      float acc[128];
#pragma unroll
      for (int i = 0; i < 128; ++i) acc[i] = 0.0f;
#pragma unroll 1
      for (int c = 0; ok && c < chunks; ++c, sp += N) {
        float sc = __fmul_rn(__ldg(sp), 65536.0f);
        const uint32_t ex = extra_of(t, c);
        const int nd = gw_digits(ex), own = 3 + static_cast<int>((ex >> (8 * ((nw >> 6) & 3))) & 0xFFu);
#pragma unroll 1
        for (int j = 0; j < nd; ++j, pass.next(2)) {
          ok = __all_sync(0xFFFFFFFFu, mbar_wait(acc_full + pass.s, pass.ph, abort_flag));
          if (!ok) break;
          tc_fence_after();
#pragma unroll
          for (int i = 0; i < 128; i += 16) {
            if (j >= own) continue;  // a digit of other outputs in the tile, not written for these
            uint32_t v[16];
            tmem_ld_32x32b_x16(trow + 256 * pass.s + i, v);
            tmem_ld_wait();
#pragma unroll
            for (int x = 0; x < 16; ++x)  // at most 2^24: exact in fp32
              acc[i + x] = __fmaf_rn(__int2float_rn(static_cast<int32_t>(v[x])), sc, acc[i + x]);
          }
          tc_fence_before();
          __syncwarp();
#ifdef BL_TEST_HOOKS
          const bool held = (g_test_fault == 5 && rank == 0 || g_test_fault == 6 && rank == 1) && warp == 2 && t == first && c == 0 && j == 0;
          if (!held)
#endif
            if (lane == 0) mbar_arrive_remote(acc_empty + pass.s, 0);
          sc = __fmul_rn(sc, 0.00390625f);
        }
      }
      if (ok) {
        // turned 16 columns at a time, so that a store takes 16 columns of
        // two rows and not one of 32 (which is 32 sectors)
        const int k0 = t % ktiles * kGwBN + 128 * part, col = lane & 15;
        const int rows = min(32, N - nw);  // may be < 1
#pragma unroll
        for (int i = 0; i < 128; i += 16) {
          __syncwarp();
#pragma unroll
          for (int x = 0; x < 16; ++x) patch[lane * 17 + x] = acc[i + x];
          __syncwarp();
          if (k0 + i + col < K) {
            int64_t at = static_cast<int64_t>(nw + (lane >> 4)) * K + k0 + i + col;
#pragma unroll 4
            for (int r = lane >> 4; r < rows; r += 2, at += 2 * static_cast<int64_t>(K))
              store_out<OutT>(dw, at, patch[r * 17 + col]);
          }
        }
      }
    }
  }

  __syncwarp();
  __syncthreads();
  if (rank == 0 && warp == 0 && lane < 2 && *abort_flag) {
    // loads that can still be in flight: the last one into each slot (a slot
    // that never had one passes at once)
    uint64_t* bars = lane == 0 ? full_a : full_b;
    const int ring = lane == 0 ? S : SB;
    for (int i = 0; i < ring; ++i) mbar_drain(bars + i, i < mine.s ? mine.ph : mine.ph ^ 1u);
  }
  __syncwarp();
  tc_fence_before();
  cluster_sync_all();  // the pair's MMAs, reads of TMEM and arrivals are done
  if (warp == 1) {
    tc_fence_after();
    tmem2_dealloc(tmem_d, 512);
  }
}

}  // namespace bl
