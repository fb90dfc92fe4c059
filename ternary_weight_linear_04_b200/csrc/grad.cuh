// grad.cuh -- backward pass of the ternary layer on the tensor core.
//
// The straight-through estimator passes gradients through the roundings
// unchanged, so with W^ = gamma W~ and x^ = x~ eta / 127
//
//   dx[m,k] = gamma sum_n dy[m,n] W~[n,k]          (k_grad_input)
//   dW[n,k] = sum_m dy[m,n] x~[m,k] eta_m / 127    (grad_weight.cuh)
//
// k_grad_input (here) contracts bf16 with bf16 values into fp32 accumulators
// (tcgen05 kind::f16, accumulators in TMEM): W~ has the values -1, 0, +1,
// exact in bf16, so the products are exact and only the sum rounds; gamma is
// applied to the finished sum.  kind::f16 cuts its fp32 sums off instead of
// rounding them, 16 terms at a time, so the planes of an fp32 dy come smallest
// first: behind the tops, each of their steps would lose up to a last bit of
// the whole sum (dx of 4096 x 4096 x 4096: 1.4e-5 off in the 2-norm that way,
// 3e-7 this way).  k_grad_weight (grad_weight.cuh) contracts integers.
#pragma once

#include <cuda.h>

#include "adapter_add.cuh"
#include "common.cuh"
#include "decode.cuh"
#include "tc_bf16.cuh"

namespace bl {

template <typename T>
__device__ __forceinline__ float ld_f32(const T* p);
template <>
__device__ __forceinline__ float ld_f32<float>(const float* p) { return *p; }
template <>
__device__ __forceinline__ float ld_f32<__nv_bfloat16>(const __nv_bfloat16* p) { return __bfloat162float(*p); }

// ---------------------------------------------------------------- operand copies

// Rows of `bytes` bytes copied into rows of `stride` bytes (a multiple of
// 16), the rest zero: operands whose rows do not start on 16 bytes cannot be
// read by TMA.  One pass over the operand, small beside the product; two
// operands in one launch.
struct PadJob {
  const uint8_t* src;
  int64_t rows, bytes, stride;  // rows 0: nothing to do
  uint8_t* dst;
};

// Item `at` and every `step`-th after it (16 bytes each).
__device__ __forceinline__ void pad_rows(const PadJob& first, const PadJob& second, int64_t at, int64_t step) {
  const int64_t n1 = first.rows * (first.stride / 16), n2 = second.rows * (second.stride / 16);
  for (int64_t it = at; it < n1 + n2; it += step) {
    const PadJob& job = it < n1 ? first : second;
    const int64_t i = it < n1 ? it : it - n1;
    const uint8_t* src = job.src;
    const int64_t chunks = job.stride / 16;
    const int64_t row = i / chunks, c = (i - row * chunks) * 16;
    const int64_t left = job.bytes - c;
    const int64_t off = row * job.bytes + c;
    uint32_t w[4];
    if (off + 20 <= job.rows * job.bytes) {  // rows start anywhere: five aligned words, shifted together
      const uint32_t* s4 = reinterpret_cast<const uint32_t*>(src + (off & ~int64_t{3}));
      const unsigned sh = 8 * static_cast<unsigned>(off & 3);
      uint32_t in[5];
#pragma unroll
      for (int j = 0; j < 5; ++j) in[j] = __ldg(s4 + j);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        w[j] = __funnelshift_r(in[j], in[j + 1], sh);
        const int64_t keep = left - 4 * j;  // bytes of this word inside the row
        if (keep < 4) w[j] = keep <= 0 ? 0u : w[j] & (0xFFFFFFFFu >> (8 * (4 - keep)));
      }
    } else {  // the end of the tensor byte by byte
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        w[j] = 0;
#pragma unroll
        for (int b = 0; b < 4; ++b)
          if (4 * j + b < left) w[j] |= static_cast<uint32_t>(src[off + 4 * j + b]) << (8 * b);
      }
    }
    *reinterpret_cast<uint4*>(job.dst + row * job.stride + c) = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

__global__ void __launch_bounds__(256) k_pad_rows(const PadJob first, const PadJob second) {
  pdl_wait();
  if (threadIdx.x == 0) pdl_trigger();
  pad_rows(first, second, blockIdx.x * 256ll + threadIdx.x, gridDim.x * 256ll);
}

// fp32 rows as three bf16 planes (rows x cols_pad each, zero past cols) whose
// sum is the fp32 value (bf16_part).
__global__ void __launch_bounds__(256)
    k_split_planes(const float* __restrict__ src, int64_t rows, int64_t cols, int64_t cols_pad,
                   __nv_bfloat16* __restrict__ dst) {
  const int64_t plane = rows * cols_pad;
  pdl_wait();
  if (threadIdx.x == 0) pdl_trigger();
  for (int64_t i = blockIdx.x * 256ll + threadIdx.x; i < plane; i += gridDim.x * 256ll) {
    const int64_t row = i / cols_pad, c = i - row * cols_pad;
    const float f = c < cols ? src[row * cols + c] : 0.0f;
#pragma unroll
    for (int p = 0; p < 3; ++p) dst[p * plane + i] = __ushort_as_bfloat16(static_cast<unsigned short>(__float_as_uint(bf16_part(f, p)) >> 16));
  }
}

// ---------------------------------------------------------------- input gradient
//
// Tile: 128 H tokens (TMEM lanes, H accumulators) by 256 inputs k (columns),
// the contraction over n in steps of 64.  Per step:
//   * the dy tile (128 H x 64, K-major, 128-byte swizzle) by TMA;
//   * the packed tile (64 rows n x 64 bytes) by TMA through its own ring of
//     stages, expanded by eight warps to bf16 (64 x 256, MN-major: k
//     contiguous as in the packed rows, so nothing is transposed).  A code c
//     in {0,1,2} becomes bits 0x4300 | c = 128 + c in bf16, minus 129: two
//     codes a lane-instruction.  The pair in one register is (k, k + 8) of
//     its 16, which leaves the columns of a 16-group in the order 0 8 1 9 ..
//     7 15; the epilogue puts them back by naming registers;
//   * eight (H = 2) MMAs 128 x 256 x 16.
// Two groups of eight expanding warps take the steps in turn, which hides
// the chain wait - load - store - fence of one step behind the other's.
// H = 2 shares one expanded tile between two MMAs of 128 tokens and fills
// TMEM, for token counts that fill the GPU; H = 1 is for the rest, where a
// cluster splits the steps and adds the tiles through distributed shared
// memory.  2048 x 11008 x 4096 (H = 2): 124 us on warm inputs, 143 on
// rotating ones, 1.5 and 1.3 PFLOP/s of the 1.64 that a library product
// reaches.  It reads 12 KB of shared memory for an MMA of 128 cycles and
// writes 8 KB beside it, which is all that an SM can.  77 x 3200 x 8640
// (H = 1): 17 us, about 8 of them before and after the steps.
//
// Adapters: behind the steps over n come steps of 64 entries, an entry being
// one (adapter of the tile's tokens, part of v, rank index): v (each token's
// row masked to its own adapter, divided by gamma because the sum is
// multiplied by it at the end; three bf16 parts) against A_a's row, written
// by the expanding warps.

constexpr int kGiBK = 64;    // n per step
constexpr int kGiBN = 256;   // inputs k per tile
constexpr int kGiGroup = 8;  // warps that expand a step
constexpr int kGiGroups = 2;
constexpr int kGiThreads = 32 * (2 + kGiGroup * kGiGroups);
constexpr int kGiTilePitch = kGiBN + 4;  // floats of a token's row in the finished tile (H = 1)

template <int H>
struct GiCfg {
  static constexpr int kStages = H == 2 ? 3 : 4;
  static constexpr int kPStages = 6;
  static constexpr int kABytes = H * 128 * 128;    // dy tile
  static constexpr int kBBytes = kGiBK * kGiBN * 2;  // expanded weights
  static constexpr int kPBytes = kGiBK * kGiBN / 4;  // packed weights
  static constexpr int kBars = 3 * kStages + 2 * kPStages + 2;
  static constexpr int kTail = 8 * kBars + 32 + 4 * (2 * 128 * H + 8);
  static constexpr size_t kSmem = 1024 + static_cast<size_t>(kStages) * (kABytes + kBBytes) + kPStages * kPBytes + kTail;
  static_assert(kSmem <= 227 * 1024, "shared memory per CTA");
  static_assert(H == 2 || 128 * kGiTilePitch * 4 <= kStages * (kABytes + kBBytes), "the finished tile in the stages");
};

struct GiArgs {
  const float* gamma;
  int M, N, K;       // N: contraction, K: output columns
  int planes;        // bf16 planes of dy
  void* dx;
  int vec;           // rows of dx take 16-byte stores
  // adapters (v NULL: none)
  const float* v;    // M x rank_stride(r)
  const __nv_bfloat16* A;  // L x r x K
  const int32_t* ids;
  int L, r;
};

// Sixteen bf16 of a row of the factor in the column order of the expanded
// weights (pairs (i, i + 8)); zero past `left`, and in the place of values
// that are not finite, in which case it returns true.
__device__ __forceinline__ bool load16_paired(const __nv_bfloat16* p, int64_t left, bool vec, uint32_t (&o)[8]) {
  uint32_t w[8];
  if (left >= 16 && vec) {
    const uint4 a = *reinterpret_cast<const uint4*>(p), b = *reinterpret_cast<const uint4*>(p + 8);
    w[0] = a.x; w[1] = a.y; w[2] = a.z; w[3] = a.w;
    w[4] = b.x; w[5] = b.y; w[6] = b.z; w[7] = b.w;
  } else {
    const uint16_t* h = reinterpret_cast<const uint16_t*>(p);
#pragma unroll
    for (int i = 0; i < 8; ++i)
      w[i] = (2 * i < left ? h[2 * i] : 0u) | (2 * i + 1 < left ? static_cast<uint32_t>(h[2 * i + 1]) << 16 : 0u);
  }
  uint32_t bad = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) bad |= nonfinite2(w[i]);
  if (bad)
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t b = nonfinite2(w[i]);
      w[i] &= ((b & 0x8000u) ? 0u : 0xFFFFu) | ((b & 0x80000000u) ? 0u : 0xFFFF0000u);
    }
#pragma unroll
  for (int i = 0; i < 8; ++i) o[i] = __byte_perm(w[i >> 1], w[4 + (i >> 1)], (i & 1) ? 0x7632 : 0x5410);
  return bad != 0;
}

// What load16_paired left out of one output: the terms of its adapter's
// values that are not finite.
__device__ __noinline__ float gi_nonfinite(const float* v, const __nv_bfloat16* A, int a, int r, int m, int k, int K) {
  float s = 0.0f;
  for (int j = 0; j < r; ++j) {
    const float w = __bfloat162float(A[(static_cast<int64_t>(a) * r + j) * K + k]);
    if (__fsub_rn(w, w) != 0.0f) s = __fmaf_rn(v[static_cast<int64_t>(m) * rank_stride(r) + j], w, s);
  }
  return s;
}

// Grid (tiles, 1, CTAs of a cluster along the contraction; H = 2: 1).
template <int H, typename OutT>
__global__ void __launch_bounds__(kGiThreads, 1)
    k_grad_input(const __grid_constant__ CUtensorMap tm_dy, const __grid_constant__ CUtensorMap tm_w, const GiArgs a) {
  using Cfg = GiCfg<H>;
  constexpr int S = Cfg::kStages, SP = Cfg::kPStages, kParts = kFactorParts;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint8_t* sA = base;
  uint8_t* sB = sA + S * Cfg::kABytes;
  uint8_t* sP = sB + S * Cfg::kBBytes;
  uint64_t* full_a = reinterpret_cast<uint64_t*>(sP + SP * Cfg::kPBytes);  // dy tile in
  uint64_t* full_b = full_a + S;      // weights expanded (a group's warps)
  uint64_t* empty = full_b + S;       // the MMAs are done with the stage
  uint64_t* full_p = empty + S;       // packed tile in
  uint64_t* empty_p = full_p + SP;    // packed tile read (a group's warps)
  uint64_t* accum_full = empty_p + SP;
  uint64_t* drain = accum_full + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  volatile float* s_bad = reinterpret_cast<volatile float*>(tmem_slot + 2);  // not zero: a value of A is not finite
  int* s_ids = reinterpret_cast<int*>(tmem_slot + 4);
  int* s_list = s_ids + 128 * H;
  int* s_cnt = s_list + 128 * H;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int ktiles = (a.K + kGiBN - 1) / kGiBN;
  const int k0 = static_cast<int>(blockIdx.x % ktiles) * kGiBN, m0 = static_cast<int>(blockIdx.x / ktiles) * (128 * H);
  const int steps_n = (a.N + kGiBK - 1) / kGiBK;
  const int CS = H == 1 ? static_cast<int>(cluster_nctarank()) : 1;
  const int z = CS > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  // this CTA's steps over n: [lo, lo + nst) of all planes', the last plane's
  // first
  const int64_t all = static_cast<int64_t>(steps_n) * a.planes;
  const int lo = static_cast<int>(all * z / CS), nst = static_cast<int>(all * (z + 1) / CS) - lo;

  auto issue_p = [&](int i) {
    const int s = i % SP;
    mbar_arrive_expect_tx(full_p + s, Cfg::kPBytes);
    tma_load_2d(sP + s * Cfg::kPBytes, &tm_w, full_p + s, k0 / 4, ((lo + i) % steps_n) * kGiBK);
  };
  auto issue_a = [&](int i) {
    const int s = i % S;
    mbar_arrive_expect_tx(full_a + s, Cfg::kABytes);
    tma_load_3d(sA + s * Cfg::kABytes, &tm_dy, full_a + s, ((lo + i) % steps_n) * kGiBK, m0, a.planes - 1 - (lo + i) / steps_n);
  };
  const int a_first = nst < S ? nst : S, p_first = nst < SP ? nst : SP;
  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(full_a + s, 1);
      mbar_init(full_b + s, kGiGroup);
      mbar_init(empty + s, 1);
    }
    for (int s = 0; s < SP; ++s) {
      mbar_init(full_p + s, 1);
      mbar_init(empty_p + s, kGiGroup);
    }
    mbar_init(accum_full, 1);
    mbar_init(drain, 1);
    *abort_flag = 0;
    *s_bad = 0.0f;
    mbar_init_fence();
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, 256 * H);
    tmem_relinquish();
  }
  pdl_wait();
  if (threadIdx.x == 0) {
    pdl_trigger();
    for (int i = 0; i < p_first; ++i) issue_p(i);
    for (int i = 0; i < a_first; ++i) issue_a(i);
  }
  int entries = 0, ast = 0, alo = 0;  // entries of the tile's adapters, this CTA's steps of 64 of them
  if (a.v) {
    entries = tile_adapters(a.ids, nullptr, m0, a.M, 128 * H, a.L, s_ids, s_list, s_cnt) * kParts * padded_rank(a.r);
    const int asteps = (entries + kGiBK - 1) / kGiBK;
    alo = asteps * z / CS;
    ast = asteps * (z + 1) / CS - alo;
  }
  const int nall = nst + ast;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_d = *tmem_slot;
  bool epi_ok = false;
  int issued = 0;

  if (warp == 0) {
    if (lane == 0) {  // dy tiles
      issued = a_first;
      for (int i = S; i < nst; ++i) {
        if (!mbar_wait(empty + i % S, static_cast<uint32_t>(i / S - 1) & 1u, abort_flag)) break;
        issue_a(i);
        issued = i + 1;
      }
    } else if (lane == 1) {  // packed tiles
      issued = p_first;
      for (int i = SP; i < nst; ++i) {
        if (!mbar_wait(empty_p + i % SP, static_cast<uint32_t>(i / SP - 1) & 1u, abort_flag)) break;
        issue_p(i);
        issued = i + 1;
      }
    }
  } else if (warp == 1) {
    if (lane == 0) {
      constexpr uint32_t idesc = make_idesc_bf16(128, kGiBN, false, true);
      const uint64_t a_desc0 = make_sw128_kmajor_desc(smem_u32(sA));
      const uint64_t b_desc0 = make_sw128_mnmajor_desc(smem_u32(sB), kGiBK * 128);
      bool ok = true;
      for (int i = 0; i < nall; ++i) {
        const int s = i % S;
        const uint32_t par = static_cast<uint32_t>(i / S) & 1u;
        ok = (i >= nst || mbar_wait(full_a + s, par, abort_flag)) && mbar_wait(full_b + s, par, abort_flag);
        if (!ok) {
          if (i > 0) {
            tc_commit(drain);
            mbar_drain(drain, 0);
          }
          break;
        }
        tc_fence_after();
        const uint64_t ad = a_desc0 + static_cast<uint64_t>(s * (Cfg::kABytes >> 4));
        const uint64_t bd = b_desc0 + static_cast<uint64_t>(s * (Cfg::kBBytes >> 4));
#pragma unroll
        for (int kk = 0; kk < kGiBK / 16; ++kk)
#pragma unroll
          for (int h = 0; h < H; ++h)
            tc_mma_bf16_ss(tmem_d + 256 * h, ad + h * (16384 >> 4) + 2 * kk, bd + kk * (2048 >> 4), idesc,
                           i != 0 || kk != 0 ? 1u : 0u);
        tc_commit(empty + s);
      }
      if (ok) tc_commit(accum_full);
    }
  } else {
    // ---------------- expand: thread = row n of the tile and 64 of its inputs
    const int grp = (warp - 2) / kGiGroup;
    const int t = (threadIdx.x - 64) & (32 * kGiGroup - 1);
    const int n = t & 63, q = t >> 6;
    const uint32_t src_off = n * 64 + ((q ^ ((n >> 1) & 3)) << 4);  // 64-byte swizzle
    uint8_t* const dst0 = sB + q * (kGiBK * 128) + (n >> 3) * 1024 + (n & 7) * 128;
    bool ok = true;
    int i = grp;
    for (; i < nst; i += kGiGroups) {
      const int s = i % S, sp = i % SP;
      ok = __all_sync(0xFFFFFFFFu, mbar_wait(full_p + sp, static_cast<uint32_t>(i / SP) & 1u, abort_flag));
      if (!ok) break;
      const uint4 p = *reinterpret_cast<const uint4*>(sP + sp * Cfg::kPBytes + src_off);
      __syncwarp();
      if (lane == 0) mbar_arrive(empty_p + sp);
      if (i >= S) {
        ok = __all_sync(0xFFFFFFFFu, mbar_wait(empty + s, static_cast<uint32_t>(i / S - 1) & 1u, abort_flag));
        if (!ok) break;
      }
      const uint32_t pw[4] = {p.x, p.y, p.z, p.w};
      uint8_t* dst = dst0 + s * Cfg::kBBytes;
#pragma unroll
      for (int wi = 0; wi < 4; ++wi) {
        uint32_t o[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const uint32_t c = ((pw[wi] >> (2 * j)) & 0x00030003u) | 0x43004300u;  // 128 + code
          const __nv_bfloat162 d = __hsub2(reinterpret_cast<const __nv_bfloat162&>(c),
                                           __nv_bfloat162(__float2bfloat16(129.0f), __float2bfloat16(129.0f)));
          o[j] = reinterpret_cast<const uint32_t&>(d);
        }
        *reinterpret_cast<uint4*>(dst + (((2 * wi) ^ (n & 7)) << 4)) = make_uint4(o[0], o[1], o[2], o[3]);
        *reinterpret_cast<uint4*>(dst + (((2 * wi + 1) ^ (n & 7)) << 4)) = make_uint4(o[4], o[5], o[6], o[7]);
      }
      fence_proxy_async_smem();
      __syncwarp();
#ifdef BL_TEST_HOOKS
      if (g_test_fault == 4 && warp == 2 && i == 2) continue;  // behind two steps whose MMAs are in flight
#endif
      if (lane == 0) mbar_arrive(full_b + s);
    }
    // ---------------- adapters
    const int r = a.r, rp = padded_rank(r), group = kParts * rp;
    const float inv_gamma = ok && i < nall ? __frcp_rn(*a.gamma) : 0.0f;
    const bool avec = (a.K & 7) == 0;
    for (; ok && i < nall; i += kGiGroups) {
      const int s = i % S, e0 = (alo + i - nst) * kGiBK;
      if (i >= S) {
        ok = __all_sync(0xFFFFFFFFu, mbar_wait(empty + s, static_cast<uint32_t>(i / S - 1) & 1u, abort_flag));
        if (!ok) break;
      }
      {  // A: entry t / 4, 16 inputs of each 64 (four lanes read 128 bytes of a row)
        const int en = t >> 2, wi = t & 3, e = e0 + en, pair = e / rp, j = e - pair * rp;
        uint32_t o[4][8];
        bool bad = false;
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const int k = k0 + 64 * x + 16 * wi;
#pragma unroll
          for (int b = 0; b < 8; ++b) o[x][b] = 0;
          if (e < entries && j < r && k < a.K)
            bad |= load16_paired(a.A + (static_cast<int64_t>(s_list[pair / kParts]) * r + j) * a.K + k, a.K - k, avec, o[x]);
        }
        if (bad) *s_bad = 1.0f;
        uint8_t* dst = sB + s * Cfg::kBBytes + (en >> 3) * 1024 + (en & 7) * 128;
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          *reinterpret_cast<uint4*>(dst + x * (kGiBK * 128) + (((2 * wi) ^ (en & 7)) << 4)) =
              make_uint4(o[x][0], o[x][1], o[x][2], o[x][3]);
          *reinterpret_cast<uint4*>(dst + x * (kGiBK * 128) + (((2 * wi + 1) ^ (en & 7)) << 4)) =
              make_uint4(o[x][4], o[x][5], o[x][6], o[x][7]);
        }
      }
      // v: piece t % 8 (8 entries) of the tokens t / 8 + 32 x
      constexpr int kEach = 128 * H / 32;
      const int piece = t & 7, tok0 = t >> 3, e = e0 + 8 * piece;
      uint8_t* row = sA + s * Cfg::kABytes + (tok0 >> 3) * 1024 + (tok0 & 7) * 128 + ((piece ^ (tok0 & 7)) << 4);
#pragma unroll
      for (int x4 = 0; x4 < kEach; x4 += 4) {
        uint4 o[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const int tok = tok0 + 32 * (x4 + c), own = s_ids[tok] * group;
          o[c] = make_uint4(0, 0, 0, 0);
          if (own < 0 || e + 8 <= own || e >= own + group) continue;
          o[c] = own_entries(e, own, r, rp, a.v + static_cast<int64_t>(m0 + tok) * rank_stride(r), inv_gamma);
        }
#pragma unroll
        for (int c = 0; c < 4; ++c) *reinterpret_cast<uint4*>(row + 4096 * (x4 + c)) = o[c];
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(full_b + s);
    }
    if (ok) ok = __all_sync(0xFFFFFFFFu, mbar_wait(accum_full, 0, abort_flag));
    epi_ok = ok && __all_sync(0xFFFFFFFFu, *abort_flag == 0);
  }

  // After an abort the producers wait (bounded) for the loads that can still
  // be in flight, so none lands in shared memory freed at exit.
  __syncwarp();
  __syncthreads();
  if (warp == 0 && lane < 2 && *abort_flag) {
    uint64_t* bars = lane == 0 ? full_a : full_p;
    const int ring = lane == 0 ? S : SP;
    for (int i = issued > ring ? issued - ring : 0; i < issued; ++i)
      mbar_drain(bars + i % ring, static_cast<uint32_t>(i / ring) & 1u);
  }

  // ---------------- epilogue: one TMEM lane = one token; four warps share a
  // lane quarter: H = 2: two for each half of the tokens, half of the columns
  // each; H = 1: a quarter of the columns each.
  float* tile = reinterpret_cast<float*>(sA);  // H = 1: 128 x kGiTilePitch; H = 2: a 32 x 33 patch for each warp
  const int qd = warp & 3, part = (warp - 2) >> 2;
  if (warp >= 2 && epi_ok) {
    tc_fence_after();
    const float gamma = *a.gamma;
    const int h = H == 2 ? part >> 1 : 0;
    const int c_begin = H == 2 ? (part & 1) * 128 : part * 64, c_end = c_begin + (H == 2 ? 128 : 64);
    const int trow = 128 * h + 32 * qd;
    const int64_t m = static_cast<int64_t>(m0) + trow + lane;
    const uint32_t taddr = tmem_d + 256 * h + (static_cast<uint32_t>(qd * 32) << 16);
    const bool fix = a.v && *s_bad != 0.0f;
#pragma unroll 1
    for (int c = c_begin; c < c_end; c += 32) {
      uint32_t v[32];
      if (nall > 0) {
        tmem_ld_32x32b_x32(taddr + c, v);
        tmem_ld_wait();
      } else {
#pragma unroll
        for (int j = 0; j < 32; ++j) v[j] = 0;
      }
      float f[32];
#pragma unroll
      for (int g = 0; g < 32; g += 16)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          f[g + j] = __fmul_rn(__uint_as_float(v[g + 2 * j]), gamma);
          f[g + 8 + j] = __fmul_rn(__uint_as_float(v[g + 2 * j + 1]), gamma);
        }
      if (fix && m < a.M  // (every CTA that saw one adds the same infinities and NaN)
           && s_ids[trow + lane] >= 0)
#pragma unroll
        for (int j = 0; j < 32; ++j)
          if (k0 + c + j < a.K)
            f[j] = __fadd_rn(f[j], gi_nonfinite(a.v, a.A, s_list[s_ids[trow + lane]], a.r, static_cast<int>(m), k0 + c + j, a.K));
      if constexpr (H == 1) {
#pragma unroll
        for (int j = 0; j < 32; j += 4)
          *reinterpret_cast<float4*>(tile + (trow + lane) * kGiTilePitch + c + j) =
              make_float4(f[j], f[j + 1], f[j + 2], f[j + 3]);
      } else if (a.vec) {
#pragma unroll
        for (int g = 0; g < 32; g += 16) {
          float o[16];
#pragma unroll
          for (int j = 0; j < 16; ++j) o[j] = f[g + j];
          if (m < a.M) store16<OutT>(a.dx, m * a.K, k0 + c + g, a.K, o, true);
        }
      } else {  // turned, so that a warp stores consecutive columns
        float* patch = tile + (warp - 2) * (32 * 33);
        __syncwarp();
#pragma unroll
        for (int j = 0; j < 32; ++j) patch[lane * 33 + j] = f[j];
        __syncwarp();
        const int k = k0 + c + lane, rows = min(32, a.M - m0 - trow);
        if (k < a.K)
          for (int x = 0; x < rows; ++x)
            store_out<OutT>(a.dx, static_cast<int64_t>(m0 + trow + x) * a.K + k, patch[x * 33 + lane]);
      }
    }
  }
  if constexpr (H == 1) {
    __syncwarp();
    if (CS > 1) cluster_sync_all();
    else __syncthreads();
    // this CTA's rows of the finished tile, four columns a thread
    const int row0 = 128 * z / CS, rows = 128 * (z + 1) / CS - row0;
    if (*abort_flag == 0)
      for (int e = threadIdx.x; e < rows * (kGiBN / 4); e += kGiThreads) {
        const int row = row0 + e / (kGiBN / 4), c = e % (kGiBN / 4) * 4, k = k0 + c;
        if (m0 + row >= a.M || k >= a.K) continue;
        const float* p = tile + row * kGiTilePitch + c;
        float4 v = *reinterpret_cast<const float4*>(p);
        if (CS > 1) v = cluster_total4(p, CS);
        const int64_t at = static_cast<int64_t>(m0 + row) * a.K + k;
        if (a.vec) {
          if constexpr (sizeof(OutT) == 4)
            *reinterpret_cast<float4*>(static_cast<float*>(a.dx) + at) = v;
          else
            *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.dx) + at) = make_uint2(pack_bf16(v.x, v.y), pack_bf16(v.z, v.w));
        } else {
          store_out<OutT>(a.dx, at, v.x);
          if (k + 1 < a.K) store_out<OutT>(a.dx, at + 1, v.y);
          if (k + 2 < a.K) store_out<OutT>(a.dx, at + 2, v.z);
          if (k + 3 < a.K) store_out<OutT>(a.dx, at + 3, v.w);
        }
      }
    __syncwarp();
    if (CS > 1) cluster_sync_all();  // the tile stays until it is read
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_d, 256 * H);
  }
}

}  // namespace bl
