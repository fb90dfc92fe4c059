// adapter_add.cuh -- what the accumulate kernels need to add a low-rank
// adapter to their outputs (adapters.cuh holds the rest).
//
// Token m uses adapter a = ids[m] (none when outside [0, L)); with u[m,:]
// given, output n gains sum_j u[m,j] B_a[n,j], added to the rescaled integer
// sum in fp32, so that the output is rounded once.
#pragma once

#include "common.cuh"

namespace bl {

// u and v are kept with rows of rank_stride(r) values, zeros past r.
__host__ __device__ constexpr int rank_stride(int r) { return (r + 3) / 4 * 4; }

struct AdapterAdd {
  const float* u;  // M x rank_stride(r); NULL: no adapters
  const __nv_bfloat16* B;  // L x N x r
  const int32_t* ids;
  int L, r;
};

// The adapter of token m: ids[m], or -1 (none) when outside [0, L).
__device__ __forceinline__ int adapter_of(const int32_t* ids, int64_t m, int L) {
  const int a = ids[m];
  return static_cast<unsigned>(a) < static_cast<unsigned>(L) ? a : -1;
}

// base + sum_j u[m,j] B_a[n,j] for one output of the decode kernels, which
// call it where they store (out of line: it costs them no registers).
__device__ __noinline__ float adapter_add(const float* u, const __nv_bfloat16* B, const int32_t* ids, int L, int r, int m,
                                          int n, int N, float base) {
  const int a = adapter_of(ids, m, L);
  if (a < 0) return base;
  const __nv_bfloat16* b = B + (static_cast<int64_t>(a) * N + n) * r;
  u += static_cast<int64_t>(m) * rank_stride(r);
  float s = 0.0f;
  int j = 0;
  if ((r & 7) == 0) {
    for (; j < r; j += 8) {
      const uint4 v = __ldg(reinterpret_cast<const uint4*>(b + j));
      const float4 p = *reinterpret_cast<const float4*>(u + j), q = *reinterpret_cast<const float4*>(u + j + 4);
      s = __fmaf_rn(p.x, __uint_as_float(v.x << 16), s);
      s = __fmaf_rn(p.y, __uint_as_float(v.x & 0xFFFF0000u), s);
      s = __fmaf_rn(p.z, __uint_as_float(v.y << 16), s);
      s = __fmaf_rn(p.w, __uint_as_float(v.y & 0xFFFF0000u), s);
      s = __fmaf_rn(q.x, __uint_as_float(v.z << 16), s);
      s = __fmaf_rn(q.y, __uint_as_float(v.z & 0xFFFF0000u), s);
      s = __fmaf_rn(q.z, __uint_as_float(v.w << 16), s);
      s = __fmaf_rn(q.w, __uint_as_float(v.w & 0xFFFF0000u), s);
    }
  }
  for (; j < r; ++j) s = __fmaf_rn(u[j], __bfloat162float(b[j]), s);
  return __fadd_rn(base, s);
}

// The distinct adapters of a tile's tokens in order of first use: s_list, and
// s_ids[t], t < BM, the place of token t's in it (-1: none); returns their
// number.  Token t is rows[m0 + t], or m0 + t where rows is NULL.  Called by whole warps, the
// threads t = 0 .. (BM at least) that `sync` brings together; BM <= 256;
// s_cnt has 8 entries.
template <typename Sync>
__device__ __forceinline__ int tile_adapters(const int32_t* ids, const int32_t* rows, int64_t m0, int64_t M, int BM, int L,
                                             int* s_ids, int* s_list, int* s_cnt, int t, Sync sync) {
  const int lane = t & 31, warp = t >> 5, groups = (BM + 31) >> 5;
  const int id = t < BM && m0 + t < M ? adapter_of(ids, rows ? rows[m0 + t] : m0 + t, L) : -1;
  // each warp's distinct ones, then those that no warp before has
  const unsigned same = __match_any_sync(0xFFFFFFFFu, id);
  bool first = id >= 0 && lane == __ffs(same) - 1;
  const unsigned below = (1u << lane) - 1;
  unsigned firsts = __ballot_sync(0xFFFFFFFFu, first);
  if (first) s_list[32 * warp + __popc(firsts & below)] = id;
  if (lane == 0 && warp < groups) s_cnt[warp] = __popc(firsts);
  sync();
  for (int w = 0; first && w < warp; ++w)
    for (int j = 0; j < s_cnt[w]; ++j)
      if (s_list[32 * w + j] == id) {
        first = false;
        break;
      }
  firsts = __ballot_sync(0xFFFFFFFFu, first);
  sync();
  if (lane == 0 && warp < groups) s_cnt[warp] = __popc(firsts);
  sync();
  int before = 0, total = 0;
  for (int w = 0; w < groups; ++w) {
    if (w < warp) before += s_cnt[w];
    total += s_cnt[w];
  }
  if (first) s_list[before + __popc(firsts & below)] = id;
  sync();
  if (t < BM) {
    int at = -1;
    for (int j = 0; id >= 0 && j < total; ++j)
      if (s_list[j] == id) {
        at = j;
        break;
      }
    s_ids[t] = at;
  }
  sync();
  return total;
}

__device__ __forceinline__ int tile_adapters(const int32_t* ids, const int32_t* rows, int64_t m0, int64_t M, int BM, int L,
                                             int* s_ids, int* s_list, int* s_cnt) {
  return tile_adapters(ids, rows, m0, M, BM, L, s_ids, s_list, s_cnt, static_cast<int>(threadIdx.x), [] { __syncthreads(); });
}

// u and v enter the tensor cores' products as this many bf16 values whose sum
// they are (8 of the 24 bits each): two would drop 2^-17 of them, which shows
// in a bf16 result wherever terms cancel.
constexpr int kFactorParts = 3;

// The bf16 values x0 + x1 + x2 that hold an fp32: its top 16 bits, those of
// the rest, and the last 8 bits (differences exact).  Cutting off instead of
// rounding takes no conversion, and the top of a large number stays finite;
// an infinity has no rest.
__device__ __forceinline__ float bf16_top(float x) { return __uint_as_float(__float_as_uint(x) & 0xFFFF0000u); }
__device__ __forceinline__ float bf16_rest(float x) {
  const float h = bf16_top(x);
  return x == h ? 0.0f : __fsub_rn(x, h);
}
// Its part p, in the top half of the word.
__device__ __forceinline__ float bf16_part(float x, int p) {
  if (p >= 1) x = bf16_rest(x);
  return p >= 2 ? bf16_rest(x) : x;
}
// Two parts as a bf16 pair (lo in the low half).
__device__ __forceinline__ uint32_t pack_tops(float lo, float hi) {
  return __byte_perm(__float_as_uint(lo), __float_as_uint(hi), 0x7632);
}

// n words from an address that need not be on four bytes (all of the n + 1
// aligned words that cover them have to be readable).
template <int n>
__device__ __forceinline__ void load_words(const void* p, uint32_t* o) {
  const uint64_t at = reinterpret_cast<uint64_t>(p);
  const uint32_t* w = reinterpret_cast<const uint32_t*>(at & ~uint64_t{3});
  const unsigned sh = 8 * static_cast<unsigned>(at & 3);
  uint32_t in[n + 1];
#pragma unroll
  for (int i = 0; i <= n; ++i) in[i] = __ldg(w + i);
#pragma unroll
  for (int i = 0; i < n; ++i) o[i] = __funnelshift_r(in[i], in[i + 1], sh);
}

// Entries of the adapters' contraction in the tensor-core kernels: for each
// adapter of a tile three parts of its r values, padded to rp (a multiple of 8,
// or 1, 2 or 4), so that eight entries from a multiple of 8 on are whole
// pairs (adapter, part), or lie inside one, and need one division.  The small
// part comes first: the MMA cuts its sums off, and would cut it off of a sum
// that the large ones have made already.
__host__ __device__ constexpr int padded_rank(int r) { return r > 4 ? (r + 7) / 8 * 8 : r == 3 ? 4 : r; }

// Eight entries from e on of a token's row: its own adapter's begin at entry
// `own`, the rest are zeros.  x: the token's row of u (or v), scaled by f.
__device__ __forceinline__ uint4 own_entries(int e, int own, int r, int rp, const float* x, float f) {
  constexpr int P = kFactorParts;
  const int i0 = e - own, rs = rank_stride(r);
  float v[8];
  if (rp >= 8) {  // all of one part
    const int at = i0 >= 2 * rp ? 2 : i0 >= rp ? 1 : 0, p = P - 1 - at, j = i0 - at * rp;
    const float4 lo = *reinterpret_cast<const float4*>(x + j);
    const float4 hi = j + 4 < rs ? *reinterpret_cast<const float4*>(x + j + 4) : make_float4(0, 0, 0, 0);
    const float y[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
#pragma unroll
    for (int b = 0; b < 8; ++b) v[b] = bf16_part(__fmul_rn(y[b], f), p);
  } else {
    const float4 y = *reinterpret_cast<const float4*>(x);
#pragma unroll
    for (int b = 0; b < 8; ++b) {
      const int i = i0 + b, at = i >= 2 * rp ? 2 : i >= rp ? 1 : 0, p = P - 1 - at, j = i - at * rp;
      const float w = j == 0 ? y.x : j == 1 ? y.y : j == 2 ? y.z : y.w;  // zero past r
      v[b] = i >= 0 && i < P * rp ? bf16_part(__fmul_rn(w, f), p) : 0.0f;
    }
  }
  return make_uint4(pack_tops(v[0], v[1]), pack_tops(v[2], v[3]), pack_tops(v[4], v[5]), pack_tops(v[6], v[7]));
}

// Which of a pair of bf16 are infinities or NaN (the top bit of each half).
// The tensor-core kernels multiply a factor of one adapter by the zeros that
// stand for the tokens of the others, and zero times infinity is NaN.  Where
// a sum can be formed again cheaply they do so for what comes out not
// finite; the input gradient, whose sums are long, leaves such values out and
// adds their terms for their own tokens.
__device__ __forceinline__ uint32_t nonfinite2(uint32_t w) {
  return ((w & 0x7F807F80u) + 0x00800080u) & 0x80008000u;
}

}  // namespace bl
