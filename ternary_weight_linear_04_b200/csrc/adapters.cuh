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
// A is L x r x K, B is L x N x r (bf16); sums in fp32.  Here: u and v, and
// the two gradients.  y's sum over j sits in the accumulate kernels
// (adapter_add.cuh, gemm_tc.cuh), dx's in grad.cuh.
#pragma once

#include <type_traits>

#include "adapter_add.cuh"
#include "common.cuh"
#include "grad.cuh"
#include "quant.cuh"
#include "rmsnorm_grad.cuh"

namespace bl {

// ---------------------------------------------------------------- small pieces

__device__ __forceinline__ void mma_bf16_16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                               uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void ldmatrix_x4_trans(uint32_t (&d)[4], const void* row) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(d[0]), "=r"(d[1]), "=r"(d[2]), "=r"(d[3])
               : "r"(smem_u32(row))
               : "memory");
}

// The codes in bytes 0 and 2 of w as a bf16 pair: the low seven bits on 128
// (one step of bf16 there is one), minus 128 or, for a negative code, 256.
__device__ __forceinline__ uint32_t codes_bf16(uint32_t w) {
  const uint32_t low = (w & 0x007F007Fu) | 0x43004300u, off = (w & 0x00800080u) | 0x43004300u;
  const __nv_bfloat162 d = __hsub2(reinterpret_cast<const __nv_bfloat162&>(low), reinterpret_cast<const __nv_bfloat162&>(off));
  return reinterpret_cast<const uint32_t&>(d);
}

// ---------------------------------------------------------------- u of up to 16 tokens
//
// Few tokens: every (token, rank index) is a dot product over K that reads
// its own row of A, so the time is that of reading the adapters in use (and
// a launch).  One CTA per token and group of rank indices; a thread holds its
// chunks of the token's codes.  FUSE: the CTA quantises the token itself
// (the exact rule of the quantiser kernels) and the first group's CTA
// writes x~, eta and xsum, which saves the quantiser's launch.  Measured with
// the accumulate kernel behind it: 7.8 us for one token (3200 -> 8640, rank
// 16; the layer alone 3.5), 16 us for 16 (8640 -> 3200, rank 32; 10.9), both
// below what issuing the call from Python costs.

constexpr int kAuThreads = 256;
constexpr int kAuChunks = 8;  // chunks of 8 codes a thread: K <= 16384

template <bool FUSE>
__global__ void __launch_bounds__(kAuThreads)
    k_adapter_u(const __nv_bfloat16* __restrict__ x, int8_t* xq, float* eta, int32_t* xsum, int K,
                const __nv_bfloat16* __restrict__ A, const float* __restrict__ scale,
                const int32_t* __restrict__ ids, int L, int r, int group, float* __restrict__ u) {
  __shared__ float s_red[2][kAuThreads / 32];
  __shared__ int32_t s_sum[kAuThreads / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t m = blockIdx.y;
  const int nch = K >> 3;
  pdl_wait();
  if (tid == 0) pdl_trigger();
  const int a = adapter_of(ids, m, L);
  const bool writes = FUSE && xq != nullptr && blockIdx.x == 0;
  const int rs = rank_stride(r);
  if (blockIdx.x == 0 && r + tid < rs) u[m * rs + r + tid] = 0.0f;
  if (a < 0) {
    for (int j = blockIdx.x * group + tid; j < min(r, static_cast<int>(blockIdx.x + 1) * group); j += kAuThreads)
      u[m * rs + j] = 0.0f;
    if (!writes) return;
  }
  uint2 q[kAuChunks];
  float e;
  if constexpr (FUSE) {
    const uint4* row = reinterpret_cast<const uint4*>(x + m * K);
    uint4 v[kAuChunks];
    uint32_t amax = 0;
#pragma unroll
    for (int i = 0; i < kAuChunks; ++i) {
      const int c = tid + kAuThreads * i;
      v[i] = c < nch ? __ldg(row + c) : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int i = 0; i < kAuChunks; ++i) {
      const uint32_t w4[4] = {v[i].x & 0x7FFF7FFFu, v[i].y & 0x7FFF7FFFu, v[i].z & 0x7FFF7FFFu, v[i].w & 0x7FFF7FFFu};
#pragma unroll
      for (int k = 0; k < 4; ++k) amax = max(amax, max(w4[k] << 16, w4[k] & 0xFFFF0000u));
    }
    amax = __reduce_max_sync(0xFFFFFFFFu, amax);
    if (lane == 0) s_red[0][warp] = __uint_as_float(amax);
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kAuThreads / 32; ++w) amax = max(amax, __float_as_uint(s_red[0][w]));
    e = fmaxf(__uint_as_float(amax), 1e-5f);
    const float rr = rcp_approx(e), qs = __fmul_rn(127.0f, rr), heta = __fmul_rn(0.5f, e);
    const bool eta_bf16 = is_bf16_value(e);  // else eta is the 1e-5 floor: exact quotients
    int32_t sum = 0;
#pragma unroll
    for (int i = 0; i < kAuChunks; ++i) {
      const int c = tid + kAuThreads * i;
      q[i] = make_uint2(0, 0);
      if (c < nch) {
        q[i] = eta_bf16 ? codes8_bf16<4>(v[i], e, heta, qs, rr) : codes8_exact(v[i], e);
        if (writes) {
          sum = __dp4a(static_cast<int>(q[i].x), 0x01010101, sum);
          sum = __dp4a(static_cast<int>(q[i].y), 0x01010101, sum);
          *reinterpret_cast<uint2*>(xq + m * K + 8 * c) = q[i];
        }
      }
    }
    if (writes) {
      sum = __reduce_add_sync(0xFFFFFFFFu, sum);
      if (lane == 0) s_sum[warp] = sum;
      __syncthreads();
      if (tid == 0) {
        sum = 0;
        for (int w = 0; w < kAuThreads / 32; ++w) sum += s_sum[w];
        eta[m] = e;
        xsum[m] = sum;
      }
      if (a < 0) return;
    }
  } else {
    e = eta[m];
    const uint2* row = reinterpret_cast<const uint2*>(xq + m * K);
#pragma unroll
    for (int i = 0; i < kAuChunks; ++i) {
      const int c = tid + kAuThreads * i;
      q[i] = c < nch ? row[c] : make_uint2(0, 0);
    }
  }
#pragma unroll
  for (int i = 0; i < kAuChunks; ++i) q[i] = make_uint2(q[i].x ^ 0x80808080u, q[i].y ^ 0x80808080u);
  const float f = div127_rn(e), sc = __ldg(scale + a);
  for (int jj = 0; jj < group; ++jj) {
    const int j = blockIdx.x * group + jj;
    if (j >= r) break;
    const uint4* row = reinterpret_cast<const uint4*>(A + (static_cast<int64_t>(a) * r + j) * K);
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < kAuChunks; ++i) {
      const int c = tid + kAuThreads * i;
      if (c < nch) {
        const uint4 v = __ldg(row + c);
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          s = __fmaf_rn(code_f32(q[i], 2 * k), __uint_as_float(w[k] << 16), s);
          s = __fmaf_rn(code_f32(q[i], 2 * k + 1), __uint_as_float(w[k] & 0xFFFF0000u), s);
        }
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
    if (lane == 0) s_red[(jj & 1) ^ 1][warp] = s;
    __syncthreads();
    if (tid == 0) {
      s = 0.0f;
      for (int w = 0; w < kAuThreads / 32; ++w) s += s_red[(jj & 1) ^ 1][w];
      u[m * rs + j] = __fmul_rn(__fmul_rn(s, f), sc);
    }
  }
}

// ---------------------------------------------------------------- tokens by adapter
//
// rows: the tokens in the order of their adapters (those without one last),
// within an adapter in their own; start[a]: where adapter a's begin, start[L]
// where those without one do.  One CTA: a stable counting sort by the adapter's
// low and (L > 255) high eight bits.  Each of 32 warps counts and places its
// own stretch of the tokens, ranks within a step of 32 by matching keys, so
// the order needs no atomics.  7 us for 2048 tokens (cold caches), all latency.
// With it u, v, dA and dB read one or two adapters a tile whatever the order of
// the requests.

constexpr int kSortThreads = 1024;

__global__ void __launch_bounds__(kSortThreads)
    k_adapter_sort(const int32_t* __restrict__ ids, int64_t M, int L, int32_t* first, int32_t* rows,
                   int32_t* __restrict__ start, const PadJob pad0, const PadJob pad1) {
  __shared__ int s_count[32][257];  // a warp's tokens with a digit, then where the next of them goes
  __shared__ int s_sum[8];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int64_t seg = (M + 1023) / 1024 * 32, lo = warp * seg, hi = min(M, lo + seg);
  const int passes = L > 255 ? 2 : 1;
  pdl_wait();
  if (tid == 0) pdl_trigger();
  if (blockIdx.x > 0) {
    pad_rows(pad0, pad1, (blockIdx.x - 1) * int64_t{kSortThreads} + tid, (gridDim.x - 1) * int64_t{kSortThreads});
    return;
  }
  auto key_of = [&](int64_t m) {
    const int a = adapter_of(ids, m, L);
    return a < 0 ? L : a;
  };
  for (int pass = 0; pass < passes; ++pass) {
    const int32_t* src = pass ? first : nullptr;
    int32_t* dst = pass == passes - 1 ? rows : first;
    auto digit = [&](int64_t i, int& item) {
      item = src ? src[i] : static_cast<int>(i);
      return (key_of(item) >> (8 * pass)) & 255;
    };
    for (int i = tid; i < 32 * 257; i += kSortThreads) (&s_count[0][0])[i] = 0;
    __syncthreads();
    for (int64_t i0 = lo; i0 < hi; i0 += 32) {
      int item, d = 256;
      if (i0 + lane < hi) d = digit(i0 + lane, item);
      const unsigned same = __match_any_sync(0xFFFFFFFFu, d);
      if (lane == __ffs(same) - 1) s_count[warp][d] += __popc(same);
      __syncwarp();
    }
    __syncthreads();
    int total = 0, inc = 0;
    if (tid < 256) {
      for (int w = 0; w < 32; ++w) {  // where a warp's go among its digit's
        const int n = s_count[w][tid];
        s_count[w][tid] = total;
        total += n;
      }
      inc = total;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int up = __shfl_up_sync(0xFFFFFFFFu, inc, o);
        if (lane >= o) inc += up;
      }
      if (lane == 31) s_sum[warp] = inc;
    }
    __syncthreads();
    if (tid < 256) {
      int before = inc - total;  // the digits below
      for (int w = 0; w < warp; ++w) before += s_sum[w];
      for (int w = 0; w < 32; ++w) s_count[w][tid] += before;
    }
    __syncthreads();
    for (int64_t i0 = lo; i0 < hi; i0 += 32) {
      int item = 0, d = 256;
      const bool in = i0 + lane < hi;
      if (in) d = digit(i0 + lane, item);
      const unsigned same = __match_any_sync(0xFFFFFFFFu, d);
      const int base = s_count[warp][d];
      __syncwarp();
      if (in) dst[base + __popc(same & ((1u << lane) - 1))] = item;
      if (lane == __ffs(same) - 1) s_count[warp][d] = base + __popc(same);
      __syncwarp();
    }
    __syncthreads();  // this pass's order is there for the whole CTA
  }
  for (int64_t p = tid; p <= M; p += kSortThreads) {
    const int k = p < M ? key_of(rows[p]) : L, before = p > 0 ? key_of(rows[p - 1]) : -1;
    for (int b = before + 1; b <= k; ++b) start[b] = static_cast<int>(p);
  }
}

// ---------------------------------------------------------------- u and v of many tokens
//
// One CTA per 16 tokens; its 16 warps take the contraction's steps of 64 in
// turn and add their sums at the end (with few tokens a cluster splits the
// contraction too).  Products on mma.sync m16n8k16: bf16 by bf16, fp32 sums;
// x~ is exact in bf16, an fp32 dy goes in as three parts.  The MMA cuts its
// sums off: a step's is added to the running one by an addition that rounds.
// (tcgen05 would need its operands in shared memory: the work is small beside
// reading dy, and these fragments come straight from global memory.)  The
// order of the contraction is free, so lane q of a row reads 16 consecutive
// codes, and A's row the same 16; for v, B's rows lie across the contraction
// and pass through shared memory (ldmatrix.trans).  A row's fragment is zeroed
// for the adapters that are not its own.  The tokens' values of the next step
// are loaded while this one's are multiplied: a warp's steps are a chain of
// loads, and the time of the kernel: 36 us for u and v of 2048 tokens (K 4096,
// N 11008, rank 16, cold caches; reading dy takes 7).

struct UvSide {
  int is_v;                // u: x = codes, F = A; v: x = dy, F = B
  const void* x;           // M x C
  int64_t C;               // contraction
  const __nv_bfloat16* F;
  const float* eta;        // u
  float* out;              // M x rank_stride(r)
  int vec;                 // rows of x (and of A) can be read in vectors
};

struct UvArgs {
  UvSide side[2];
  const float* scale;
  const int32_t* ids;
  const int32_t* rows;     // the order of the tokens (k_adapter_sort), or NULL: as they are
  int64_t M;
  int L, r;
};

constexpr int kUvWarps = 16;
constexpr int kUvThreads = 32 * kUvWarps;
constexpr int kUvRedPitch = 40;  // floats of a row of sums: 32 and 8 that spread the banks
constexpr int kUvPitch = 40;     // bf16 of a staged row of B, the same
constexpr size_t kUvSmem = kUvWarps * 64 * kUvPitch * 2;  // staged rows; the sums (16 rows a warp) take half
static_assert(kUvWarps * 16 * kUvRedPitch * 4 <= kUvSmem, "the sums in the staged rows' place");

// The plain sum for one output.
template <typename DyT>
__device__ __noinline__ float uv_plain(const UvArgs& g, const UvSide& s, int64_t m, int a, int j) {
  float t = 0.0f;
  for (int64_t c = 0; c < s.C; ++c) {
    const float x = s.is_v ? ld_f32(static_cast<const DyT*>(s.x) + m * s.C + c)
                           : static_cast<float>(static_cast<const int8_t*>(s.x)[m * s.C + c]);
    const int64_t at = s.is_v ? (a * s.C + c) * g.r + j : (static_cast<int64_t>(a) * g.r + j) * s.C + c;
    t = __fmaf_rn(x, __bfloat162float(s.F[at]), t);
  }
  return t;
}

// A lane's share of two token rows (g and g + 8) at a step: 16 codes from
// 16 q on, or values 16 i + 4 q .. + 3 for each of the step's four MMAs.
template <typename XT>
struct UvRaw {
  static constexpr int kWords = 4 * static_cast<int>(sizeof(XT));
  uint32_t w[2][kWords];

  __device__ __forceinline__ void load(const XT* const (&row)[2], int64_t k0, int64_t C, int q, bool vec) {
    constexpr int kEach = sizeof(XT) == 1 ? 16 : 4;  // values in a row
    constexpr int kW = kEach * static_cast<int>(sizeof(XT)) / 4;
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int i = 0; i < 16 / kEach; ++i) {
        const int64_t k = k0 + (sizeof(XT) == 1 ? 16 * q : 16 * i + 4 * q);
        const XT* p = row[h] + k;
        uint32_t* o = w[h] + kW * i;
#pragma unroll
        for (int j = 0; j < kW; ++j) o[j] = 0;
        if (vec) {
          if (k < C) {
            if constexpr (kW == 2) {
              const uint2 v = __ldg(reinterpret_cast<const uint2*>(p));
              o[0] = v.x; o[1] = v.y;
            } else {
              const uint4 v = __ldg(reinterpret_cast<const uint4*>(p));
              o[0] = v.x; o[1] = v.y; o[2] = v.z; o[3] = v.w;
            }
          }
        } else if (sizeof(XT) == 1 && k + 20 <= C) {
          load_words<kW>(p, o);
        } else {
#pragma unroll
          for (int j = 0; j < kEach; ++j) {
            if (k + j >= C) continue;
            if constexpr (sizeof(XT) == 1) o[j >> 2] |= static_cast<uint32_t>(static_cast<uint8_t>(__ldg(p + j))) << (8 * (j & 3));
            else if constexpr (sizeof(XT) == 2) o[j >> 1] |= static_cast<uint32_t>(__ldg(reinterpret_cast<const uint16_t*>(p) + j)) << (16 * (j & 1));
            else o[j] = __ldg(reinterpret_cast<const uint32_t*>(p) + j);
          }
        }
      }
  }

  // A fragment of MMA i: registers 0, 1 the rows' first pairs, 2, 3 the
  // second (of codes 0, 2 and 1, 3 of the four).
  __device__ __forceinline__ void fragment(uint32_t (&xf)[4], int i, int part) const {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if constexpr (sizeof(XT) == 1) {
        xf[h] = codes_bf16(w[h][i]);
        xf[2 + h] = codes_bf16(w[h][i] >> 8);
      } else if constexpr (sizeof(XT) == 2) {
        xf[h] = w[h][2 * i];
        xf[2 + h] = w[h][2 * i + 1];
      } else {
        float f[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) f[j] = bf16_part(__uint_as_float(w[h][4 * i + j]), part);
        xf[h] = pack_tops(f[0], f[1]);
        xf[2 + h] = pack_tops(f[2], f[3]);
      }
    }
  }
};

// NT: tiles of 8 rank indices at a time (r <= 8 NT, or 32 of them after one
// another); four such tiles are in flight, so 4 / NT adapters.
template <typename XT, int NT>
__device__ __forceinline__ void uv_tile(const UvArgs& g, const UvSide& s, uint8_t* smem, const int* s_ids,
                                        const int* s_list, int nad) {
  constexpr bool V = sizeof(XT) > 1;
  constexpr int PX = sizeof(XT) == 4 ? 3 : 1;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, gr = lane >> 2, q = lane & 3;
  const int64_t m0 = static_cast<int64_t>(blockIdx.x) * 16;
  const int CS = static_cast<int>(cluster_nctarank()), z = CS > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  const int64_t C = s.C;
  const int64_t nst = (C + 63) >> 6;
  const int step = kUvWarps * CS;
  const int r = g.r;
  const bool vec = s.vec != 0, bvec = (r & 7) == 0;
  float* red = reinterpret_cast<float*>(smem);
  __nv_bfloat16* stage = reinterpret_cast<__nv_bfloat16*>(smem) + warp * 64 * kUvPitch;
  const int own0 = s_ids[gr], own1 = s_ids[8 + gr];
  auto token = [&](int i) {  // of the tile's row i; rows past M repeat the last
    const int64_t at = min(m0 + i, g.M - 1);
    return g.rows ? static_cast<int64_t>(g.rows[at]) : at;
  };
  const XT* const row[2] = {static_cast<const XT*>(s.x) + token(gr) * C, static_cast<const XT*>(s.x) + token(8 + gr) * C};
  for (int jb = 0; jb < r; jb += 8 * NT) {
    float acc[NT][4];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[n][i] = 0.0f;
    constexpr bool kAhead = sizeof(XT) < 4;  // fp32 rows: not enough registers for two steps
    UvRaw<XT> next;
    const int64_t first = warp * CS + z;
    if (kAhead && nad && first < nst) next.load(row, first << 6, C, q, vec);
    for (int64_t st = first; nad && st < nst; st += step) {
      const int64_t k0 = st << 6;
      UvRaw<XT> raw;
      if constexpr (kAhead) {
        raw = next;
        if (st + step < nst) next.load(row, (st + step) << 6, C, q, vec);
      } else {
        raw.load(row, k0, C, q, vec);
      }
      float sum[NT][4] = {};  // this step's terms
      for (int lb = 0; lb < nad; lb += 4 / NT) {
        // slot x of the four: rank indices jb + 8 (x % NT) .. of adapter lb + x / NT
        uint4 w[4][2];
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          w[x][0] = w[x][1] = make_uint4(0, 0, 0, 0);
          const int li = lb + x / NT, j0 = jb + 8 * (x % NT);
          if (li >= nad || j0 >= r) continue;
          const int64_t a = s_list[li];
          if constexpr (!V) {  // A's row j0 + g: 16 values
            const int64_t k = k0 + 16 * q;
            const int j = j0 + gr;
            const __nv_bfloat16* f = s.F + (a * r + j) * C + k;
            if (j < r && k < C) {
              if (vec) {
                w[x][0] = __ldg(reinterpret_cast<const uint4*>(f));
                w[x][1] = __ldg(reinterpret_cast<const uint4*>(f) + 1);
              } else {
                uint32_t e[8] = {0, 0, 0, 0, 0, 0, 0, 0};
                if (k + 18 <= C)
                  load_words<8>(f, e);
                else
#pragma unroll
                for (int i = 0; i < 16; ++i)
                  if (k + i < C)
                    e[i >> 1] |= static_cast<uint32_t>(__ldg(reinterpret_cast<const uint16_t*>(f) + i)) << (16 * (i & 1));
                w[x][0] = make_uint4(e[0], e[1], e[2], e[3]);
                w[x][1] = make_uint4(e[4], e[5], e[6], e[7]);
              }
            }
          } else {  // B's rows k0 + lane and k0 + lane + 32: 8 values
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const int64_t k = k0 + lane + 32 * h;
              if (k >= C) continue;
              const __nv_bfloat16* f = s.F + (a * C + k) * r + j0;
              if (bvec) {
                w[x][h] = __ldg(reinterpret_cast<const uint4*>(f));
              } else {
                uint32_t e[4] = {0, 0, 0, 0};
#pragma unroll
                for (int i = 0; i < 8; ++i)
                  if (j0 + i < r)
                    e[i >> 1] |= static_cast<uint32_t>(__ldg(reinterpret_cast<const uint16_t*>(f) + i)) << (16 * (i & 1));
                w[x][h] = make_uint4(e[0], e[1], e[2], e[3]);
              }
            }
          }
        }
        uint32_t own[4 / NT][2];
#pragma unroll
        for (int x = 0; x < 4 / NT; ++x) {
          own[x][0] = own0 == lb + x ? 0xFFFFFFFFu : 0u;
          own[x][1] = own1 == lb + x ? 0xFFFFFFFFu : 0u;
        }
        if constexpr (!V) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint32_t xf[4];
            raw.fragment(xf, i, 0);
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              if (lb + x / NT >= nad) continue;
              const uint32_t k0m = own[x / NT][0], k1m = own[x / NT][1];
              const uint4 f = w[x][i >> 1];
              const uint32_t lo = (i & 1) ? f.z : f.x, hi = (i & 1) ? f.w : f.y;
              mma_bf16_16816(sum[x % NT], xf[0] & k0m, xf[1] & k1m, xf[2] & k0m, xf[3] & k1m,
                             __byte_perm(lo, hi, 0x5410), __byte_perm(lo, hi, 0x7632));
            }
          }
        } else {
          __syncwarp();
#pragma unroll
          for (int x = 0; x < 4; ++x)
#pragma unroll
            for (int h = 0; h < 2; ++h)
              *reinterpret_cast<uint4*>(stage + (lane + 32 * h) * kUvPitch + 8 * x) = w[x][h];
          __syncwarp();
          // matrix lane / 8: rows of the contraction 0 1 4 5 .. (registers
          // 0) or 2 3 6 7 .. (1), slots 0 or 1 of the pair
          const int mat = lane >> 3, kk = lane & 7;
          const __nv_bfloat16* at = stage + (4 * (kk >> 1) + (kk & 1) + 2 * (mat & 1)) * kUvPitch + 8 * (mat >> 1);
#pragma unroll 1
          for (int part = PX - 1; part >= 0; --part)  // the small parts first
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              uint32_t xf[4];
              raw.fragment(xf, i, part);
#pragma unroll
              for (int x = 0; x < 4; x += 2) {
                if (lb + x / NT >= nad) continue;
                uint32_t d[4];
                ldmatrix_x4_trans(d, at + 16 * i * kUvPitch + 8 * x);
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                  const uint32_t k0m = own[(x + y) / NT][0], k1m = own[(x + y) / NT][1];
                  mma_bf16_16816(sum[(x + y) % NT], xf[0] & k0m, xf[1] & k1m, xf[2] & k0m, xf[3] & k1m, d[2 * y], d[2 * y + 1]);
                }
              }
            }
        }
      }
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[n][i] = __fadd_rn(acc[n][i], sum[n][i]);
    }
    __syncthreads();  // the staged rows are read
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int h = 0; h < 2; ++h)
        *reinterpret_cast<float2*>(red + (warp * 16 + 8 * h + gr) * kUvRedPitch + 8 * n + 2 * q) =
            make_float2(acc[n][2 * h], acc[n][2 * h + 1]);
    __syncthreads();
    static_assert(kUvThreads == 16 * 32, "one sum a thread");
    float* mine = red + (tid >> 5) * kUvRedPitch + (tid & 31);
    float t = 0.0f;
#pragma unroll
    for (int w = 0; w < kUvWarps; ++w) t = __fadd_rn(t, mine[w * 16 * kUvRedPitch]);
    if (CS > 1) {  // CTA 0 adds the cluster's
      *mine = t;
      cluster_sync_all();
      if (z == 0) t = cluster_total(mine, CS);
    }
    const int i = tid >> 5, j = tid & 31;
    if (z == 0 && j < 8 * NT && jb + j < rank_stride(r) && m0 + i < g.M) {
      const int64_t m = token(i);
      if (s_ids[i] >= 0) {
        const int a = s_list[s_ids[i]];
        // zero times another adapter's infinity or NaN: the plain sum, in
        // which it has no part
        if (__fsub_rn(t, t) != 0.0f && jb + j < r) t = uv_plain<typename std::conditional<V, XT, float>::type>(g, s, m, a, jb + j);
        if constexpr (!V) t = __fmul_rn(t, div127_rn(s.eta[m]));
        t = __fmul_rn(t, g.scale[a]);
      } else {
        t = 0.0f;
      }
      s.out[m * rank_stride(r) + jb + j] = jb + j < r ? t : 0.0f;
    }
    if (CS > 1) cluster_sync_all();
    else __syncthreads();
  }
}

// Grid (tiles of 16 tokens, sides, CTAs of a cluster).
template <typename DyT, int NT>
__global__ void __launch_bounds__(kUvThreads, 1) k_adapter_uv(const __grid_constant__ UvArgs g) {
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ int s_ids[32], s_list[32], s_cnt[8];
  pdl_wait();
  if (threadIdx.x == 0) pdl_trigger();
  const UvSide& s = g.side[blockIdx.y];
  const int nad = tile_adapters(g.ids, g.rows, static_cast<int64_t>(blockIdx.x) * 16, g.M, 16, g.L, s_ids, s_list, s_cnt);
  if (s.is_v) uv_tile<DyT, NT>(g, s, smem, s_ids, s_list, nad);
  else uv_tile<int8_t, NT>(g, s, smem, s_ids, s_list, nad);
}

// ---------------------------------------------------------------- dA and dB
//
// One CTA per adapter and 64 columns of A or B (a cluster splits the tokens
// where there are few of these): it takes the adapter's tokens
// (k_adapter_sort) 64 at a time
//   out[j][c] += coef[m][j] x[m][c],   dA: coef = v eta / 127, x = x~;
//                                      dB: coef = u,           x = dy
// on mma.sync, both operands transposed out of shared memory by ldmatrix.
// The coefficients go in as three bf16 parts.  The MMA cuts its sums off, which
// would pull a long one towards zero: 16 tokens' terms are added to the running
// sum by an addition that rounds.  The next chunk's rows are loaded while one is
// multiplied.
// Bound by the longest adapter's chain of chunks.  2048 tokens of 4 adapters,
// K 4096, N 11008: 47 us with cold caches (x~ and dy are 53 MB: 8 us).

struct DabSide {
  const void* x;     // M x C: codes (dA) or dy (dB)
  int64_t C;
  const float* coef;  // M x rank_stride(r)
  void* out;
  int vec;           // rows of x can be read in 16-byte pieces
};

struct DabArgs {
  DabSide a, b;
  const float* eta;
  const int32_t *rows, *start;  // k_adapter_sort
  int r;
  unsigned slabs_a;  // blocks x below this: dA
};

constexpr int kDabThreads = 128;
constexpr int kDabTokens = 64;   // a chunk
constexpr int kDabCols = 64;
constexpr int kDabXPitch = kDabCols + 8;

__host__ __device__ constexpr int dab_rows(int r) { return (r + 15) / 16 * 16; }
__host__ __device__ constexpr size_t dab_smem(int r, int xparts) {
  const size_t tiles = static_cast<size_t>(kDabTokens) * 2 * (kFactorParts * (dab_rows(r) + 8) + xparts * kDabXPitch);
  const size_t out = static_cast<size_t>(dab_rows(r)) * (kDabCols + 4) * 4;
  return tiles > out ? tiles : out;
}

// JT: tiles of 16 rank indices (r <= 16 JT).
template <typename XT, typename OutT, int JT>
__device__ __forceinline__ void dab_tile(const DabArgs& g, const DabSide& s, int64_t c0, bool is_a, uint8_t* smem) {
  constexpr int P = kFactorParts, PX = sizeof(XT) == 4 ? 3 : 1;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int CS = static_cast<int>(cluster_nctarank()), z = CS > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  const int r = g.r, rows = dab_rows(r), cpitch = rows + 8;
  const int a = blockIdx.y;
  const int from = g.start[a], to = g.start[a + 1];
  __nv_bfloat16* s_coef = reinterpret_cast<__nv_bfloat16*>(smem);          // [P][token][cpitch]
  __nv_bfloat16* s_x = s_coef + P * kDabTokens * cpitch;                   // [PX][token][kDabXPitch]
  float acc[JT][2][4];
#pragma unroll
  for (int t = 0; t < JT; ++t)
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[t][n][i] = 0.0f;

  // A thread takes one token of a chunk and half of its columns and rank
  // indices: into registers, then (next chunk) into shared memory.
  const int xt = tid >> 1, xh = tid & 1;
  constexpr int kXRegs = 8 * static_cast<int>(sizeof(XT));  // 32 columns
  constexpr int kCoefs = 8 * JT;
  uint32_t xr[kXRegs];
  float cf[kCoefs];
  auto load = [&](int at) {  // the 64 tokens from place `at` on
    const bool in = at + xt < to;
    const int64_t m = in ? g.rows[at + xt] : 0;
    const XT* src = static_cast<const XT*>(s.x) + m * s.C + c0 + 32 * xh;
    const int64_t cols = in ? s.C - c0 - 32 * xh : 0;
    constexpr int kPer = 16 / static_cast<int>(sizeof(XT));  // values of a 16-byte piece
    if (s.vec) {
#pragma unroll
      for (int i = 0; i < kXRegs / 4; ++i) {
        const uint4 v = kPer * i < cols ? __ldg(reinterpret_cast<const uint4*>(src) + i) : make_uint4(0, 0, 0, 0);
        xr[4 * i] = v.x; xr[4 * i + 1] = v.y; xr[4 * i + 2] = v.z; xr[4 * i + 3] = v.w;
      }
    } else {
#pragma unroll
      for (int i = 0; i < kXRegs; ++i) {
        if constexpr (sizeof(XT) == 4) {
          xr[i] = i < cols ? __ldg(reinterpret_cast<const uint32_t*>(src) + i) : 0u;
        } else if constexpr (sizeof(XT) == 2) {
          const uint16_t* h = reinterpret_cast<const uint16_t*>(src) + 2 * i;
          xr[i] = (2 * i < cols ? __ldg(h) : 0u) | (2 * i + 1 < cols ? static_cast<uint32_t>(__ldg(h + 1)) << 16 : 0u);
        } else {
          const uint8_t* h = reinterpret_cast<const uint8_t*>(src) + 4 * i;
          xr[i] = 0;
#pragma unroll
          for (int b = 0; b < 4; ++b)
            if (4 * i + b < cols) xr[i] |= static_cast<uint32_t>(__ldg(h + b)) << (8 * b);
        }
      }
    }
    const float f = in && is_a ? div127_rn(__ldg(g.eta + m)) : 1.0f;
    const float* cp = s.coef + m * rank_stride(r);
#pragma unroll
    for (int i = 0; i < kCoefs; i += 4) {
      const int j = xh * (rows / 2) + i;  // rows / 2 <= kCoefs; what passes it is not stored
      const float4 v = in && i < rows / 2 && j < r ? *reinterpret_cast<const float4*>(cp + j) : make_float4(0, 0, 0, 0);
      cf[i] = __fmul_rn(v.x, f);
      cf[i + 1] = __fmul_rn(v.y, f);
      cf[i + 2] = __fmul_rn(v.z, f);
      cf[i + 3] = __fmul_rn(v.w, f);
    }
  };
  auto put = [&]() {
    uint4* dst = reinterpret_cast<uint4*>(s_x + xt * kDabXPitch + 32 * xh);
    if constexpr (sizeof(XT) == 1) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint32_t o[4];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const uint32_t e = codes_bf16(xr[2 * i + k]), d = codes_bf16(xr[2 * i + k] >> 8);  // codes 0, 2 and 1, 3
          o[2 * k] = __byte_perm(e, d, 0x5410);
          o[2 * k + 1] = __byte_perm(e, d, 0x7632);
        }
        dst[i] = make_uint4(o[0], o[1], o[2], o[3]);
      }
    } else if constexpr (sizeof(XT) == 2) {
#pragma unroll
      for (int i = 0; i < 4; ++i) dst[i] = make_uint4(xr[4 * i], xr[4 * i + 1], xr[4 * i + 2], xr[4 * i + 3]);
    } else {
#pragma unroll
      for (int p = 0; p < PX; ++p)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint32_t o[4];
#pragma unroll
          for (int k = 0; k < 4; ++k)
            o[k] = pack_tops(bf16_part(__uint_as_float(xr[8 * i + 2 * k]), p),
                             bf16_part(__uint_as_float(xr[8 * i + 2 * k + 1]), p));
          dst[p * (kDabTokens * kDabXPitch / 8) + i] = make_uint4(o[0], o[1], o[2], o[3]);
        }
    }
#pragma unroll
    for (int i = 0; i < kCoefs; i += 4) {
      if (i >= rows / 2) continue;
#pragma unroll
      for (int p = 0; p < P; ++p)
        *reinterpret_cast<uint2*>(s_coef + (p * kDabTokens + xt) * cpitch + xh * (rows / 2) + i) =
            make_uint2(pack_tops(bf16_part(cf[i], p), bf16_part(cf[i + 1], p)),
                       pack_tops(bf16_part(cf[i + 2], p), bf16_part(cf[i + 3], p)));
    }
  };
  int c = from + z * kDabTokens;  // this CTA's chunks: every CS-th
  if (c < to) load(c);
  for (; c < to; c += CS * kDabTokens) {
    put();
    __syncthreads();
    // the next chunk's rows are on their way while this one is multiplied
    if (c + CS * kDabTokens < to) load(c + CS * kDabTokens);
    const int kk = lane & 7, mat = lane >> 3;
#pragma unroll
    for (int ks = 0; ks < kDabTokens / 16; ++ks) {
      uint32_t bx[PX][4];  // columns 16 warp + 0-7 (registers 0, 1) and 8-15 (2, 3)
#pragma unroll
      for (int p = 0; p < PX; ++p)
        ldmatrix_x4_trans(bx[p], s_x + (p * kDabTokens + 16 * ks + kk + 8 * (mat & 1)) * kDabXPitch + 16 * warp + 8 * (mat >> 1));
#pragma unroll
      for (int t = 0; t < JT; ++t) {
        if (16 * t >= rows) continue;
        float sum[2][4] = {};  // these 16 tokens' terms, the small parts first
#pragma unroll
        for (int p = P - 1; p >= 0; --p) {
          uint32_t f[4];  // rows j 0-7, 8-15 at tokens 0-7, then at 8-15
          ldmatrix_x4_trans(f, s_coef + (p * kDabTokens + 16 * ks + kk + 8 * (mat >> 1)) * cpitch + 16 * t + 8 * (mat & 1));
#pragma unroll
          for (int px = PX - 1; px >= 0; --px) {
            mma_bf16_16816(sum[0], f[0], f[1], f[2], f[3], bx[px][0], bx[px][1]);
            mma_bf16_16816(sum[1], f[0], f[1], f[2], f[3], bx[px][2], bx[px][3]);
          }
        }
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[t][n][i] = __fadd_rn(acc[t][n][i], sum[n][i]);
      }
    }
    __syncthreads();
  }

  // out: the CTA's sums into shared memory, a cluster's added up by rows
  float* s_out = reinterpret_cast<float*>(smem);
  constexpr int kOPitch = kDabCols + 4;
  __syncthreads();
#pragma unroll
  for (int t = 0; t < JT; ++t) {
    if (16 * t >= rows) continue;
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
      for (int h = 0; h < 2; ++h)
        *reinterpret_cast<float2*>(s_out + (16 * t + 8 * h + (lane >> 2)) * kOPitch + 16 * warp + 8 * n + 2 * (lane & 3)) =
            make_float2(acc[t][n][2 * h], acc[t][n][2 * h + 1]);
  }
  if (CS > 1) cluster_sync_all();
  else __syncthreads();
  const int cols = static_cast<int>(min(static_cast<int64_t>(kDabCols), s.C - c0));
  const int64_t base = is_a ? static_cast<int64_t>(a) * r * s.C + c0 : (static_cast<int64_t>(a) * s.C + c0) * r;
  for (int e = z * kDabThreads + tid; e < r * kDabCols; e += CS * kDabThreads) {
    // neighbouring threads take neighbouring outputs: A is r x K, B is N x r
    const int j = is_a ? e / kDabCols : e % r, c = is_a ? e % kDabCols : e / r;
    if (c >= cols) continue;
    float v = s_out[j * kOPitch + c];
    if (CS > 1) v = cluster_total(s_out + j * kOPitch + c, CS);
    store_out<OutT>(s.out, base + (is_a ? j * s.C + c : static_cast<int64_t>(c) * r + j), v);
  }
  if (CS > 1) cluster_sync_all();  // the sums stay until they are read
}

// Grid (slabs of A, then of B; adapters; CTAs of a cluster).
template <typename DyT, typename OutT, int JT>
__global__ void __launch_bounds__(kDabThreads) k_adapter_dab(const __grid_constant__ DabArgs g) {
  extern __shared__ __align__(16) uint8_t smem[];
  pdl_wait();
  if (threadIdx.x == 0) pdl_trigger();
  if (blockIdx.x < g.slabs_a)
    dab_tile<int8_t, OutT, JT>(g, g.a, static_cast<int64_t>(blockIdx.x) * kDabCols, true, smem);
  else
    dab_tile<DyT, OutT, JT>(g, g.b, static_cast<int64_t>(blockIdx.x - g.slabs_a) * kDabCols, false, smem);
}

}  // namespace bl
