// train_host.cuh -- argument checks and launches of the backward pass and of
// the adapters (grad.cuh, rmsnorm_grad.cuh, adapters.cuh).  Included by
// bitlinear.cu after its own helpers.
#pragma once

namespace {

constexpr int64_t kTrainMaxDim = INT32_MAX / 2;
constexpr int kAdapterMaxRank = 128;
constexpr int kAdapterMaxCount = 65535;

inline bool dtype_ok(bl_dtype t) { return t == BL_F32 || t == BL_BF16; }
inline int64_t dtype_bytes(bl_dtype t) { return t == BL_F32 ? 4 : 2; }
inline int64_t round_up(int64_t v, int64_t to) { return (v + to - 1) / to * to; }

// Sizes every call of the backward pass shares: M >= 0, N, K >= 1, each
// below 2^30, N * K and M * max(N, K) at most 2^40, 127 K < 2^31.
inline bl_status train_sizes(int64_t M, int64_t N, int64_t K) {
  if (M < 0 || N < 1 || K < 1) return BL_ERR_INVALID_ARG;
  if (M > kTrainMaxDim || N > kTrainMaxDim || 127 * K >= (int64_t{1} << 31)) return BL_ERR_UNSUPPORTED;
  if (N * K > (int64_t{1} << 40) || M * (N > K ? N : K) > (int64_t{1} << 40)) return BL_ERR_UNSUPPORTED;
  return BL_OK;
}

inline bl_status adapter_sizes(int64_t L, int64_t r, int64_t N, int64_t K) {
  if (L < 1 || r < 1) return BL_ERR_INVALID_ARG;
  if (r > kAdapterMaxRank || L > kAdapterMaxCount) return BL_ERR_UNSUPPORTED;
  if (L * r * (N > K ? N : K) > (int64_t{1} << 40)) return BL_ERR_UNSUPPORTED;
  return BL_OK;
}

// Device scratch handed out of the caller's workspace in 256-byte pieces.
struct Scratch {
  char* base;
  size_t used;
  explicit Scratch(void* p) : base(static_cast<char*>(p)), used(0) {}
  void* take(size_t bytes) {
    void* p = base ? base + used : nullptr;
    used += static_cast<size_t>(round_up(static_cast<int64_t>(bytes), 256));
    return p;
  }
};

inline unsigned grid_for(int64_t items, int64_t per, int sms) {
  int64_t g = (items + per - 1) / per;
  if (g > static_cast<int64_t>(sms) * 32) g = static_cast<int64_t>(sms) * 32;
  return static_cast<unsigned>(g < 1 ? 1 : g);
}

// Row-major matrix (planes of it) of elem-byte values for TMA: cols of rows
// of `stride` bytes, box of box_cols x box_rows; out-of-bounds values read as
// zero.
bool make_tmap(CUtensorMap* map, CUtensorMapDataType type, const void* ptr, uint64_t cols, uint64_t rows,
               uint64_t planes, uint64_t stride, uint32_t box_cols, uint32_t box_rows, CUtensorMapSwizzle swizzle) {
  auto enc = get_encode_fn();
  if (!enc) return false;
  const cuuint64_t dims[3] = {cols, rows, planes ? planes : 1};
  const cuuint64_t strides[2] = {stride, stride * rows};
  const cuuint32_t box[3] = {box_cols, box_rows, 1};
  const cuuint32_t estr[3] = {1, 1, 1};
  return enc(map, type, planes ? 3 : 2, const_cast<void*>(ptr), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// An operand as TMA can read it: the caller's own rows when they start on 16
// bytes, else a copy in the workspace (taken from it in either case of a
// null base, so that queries and calls agree).
struct Rows {
  const void* p;
  int64_t stride;  // bytes
  int planes;
};

inline bl_status pad_rows(const void* src, int64_t rows, int64_t bytes, Scratch* ws, Rows* out, int sms,
                          cudaStream_t s) {
  *out = {src, bytes, 1};
  if (bytes % 16 == 0) return BL_OK;
  out->stride = round_up(bytes, 16);
  void* dst = ws->take(static_cast<size_t>(rows * out->stride));
  out->p = dst;
  if (!ws->base || rows == 0) return BL_OK;
  bl::k_pad_rows<<<grid_for(rows * (out->stride / 16), 256, sms), 256, 0, s>>>(
      static_cast<const uint8_t*>(src), rows, bytes, out->stride, static_cast<uint8_t*>(dst));
  return launch_status();
}

// dy as bf16 planes: one, or three of an fp32 dy.
inline bl_status dy_rows(const void* dy, bl_dtype dydt, int64_t M, int64_t N, Scratch* ws, Rows* out, int sms,
                         cudaStream_t s) {
  if (dydt == BL_BF16) return pad_rows(dy, M, 2 * N, ws, out, sms, s);
  const int64_t cols = round_up(N, 8);
  void* dst = ws->take(static_cast<size_t>(3 * M * cols * 2));
  *out = {dst, 2 * cols, 3};
  if (!ws->base || M == 0) return BL_OK;
  bl::k_split_planes<<<grid_for(M * cols, 256, sms), 256, 0, s>>>(static_cast<const float*>(dy), M, N, cols,
                                                                   static_cast<__nv_bfloat16*>(dst));
  return launch_status();
}

// Whether rows of `cols` values of type dt take 16-byte stores.
inline int vec_rows(int64_t cols, bl_dtype dt) { return cols % (16 / dtype_bytes(dt)) == 0 ? 1 : 0; }

template <int H, typename OutT>
bl_status launch_gi(const CUtensorMap& tdy, const CUtensorMap& tw, const bl::GiArgs& a, cudaStream_t s) {
  static int done[kMaxDevices] = {0};
  auto kern = bl::k_grad_input<H, OutT>;
  constexpr size_t smem = bl::GiCfg<H>::kSmem;
  if (!ensure_smem(kern, smem, done)) return BL_ERR_CUDA;
  const int64_t tiles = ((a.K + bl::kGiBN - 1) / bl::kGiBN) * ((int64_t{a.M} + 128 * H - 1) / (128 * H));
  if (tiles > INT32_MAX) return BL_ERR_UNSUPPORTED;
  kern<<<static_cast<unsigned>(tiles), bl::kGiThreads, smem, s>>>(tdy, tw, a);
  return launch_status();
}

// dx = gamma dy W~ (+ v A where a.v is given); the operands' copies come out of ws.
bl_status run_grad_input(const Rows& dy, const uint8_t* packed, bl_dtype dxdt, bl::GiArgs a, Scratch* ws, int sms,
                         cudaStream_t s) {
  Rows w;
  bl_status st = pad_rows(packed, a.N, (a.K + 3) / 4, ws, &w, sms, s);
  if (st != BL_OK) return st;
  const int H = a.M > 128 ? 2 : 1;
  CUtensorMap tdy, tw;
  if (!make_tmap(&tdy, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, dy.p, a.N, a.M, dy.planes, dy.stride, bl::kGiBK, 128 * H,
                 CU_TENSOR_MAP_SWIZZLE_128B) ||
      !make_tmap(&tw, CU_TENSOR_MAP_DATA_TYPE_UINT8, w.p, (a.K + 3) / 4, a.N, 0, w.stride, bl::kGiBN / 4,
                 bl::kGiBK, CU_TENSOR_MAP_SWIZZLE_64B))
    return BL_ERR_CUDA;
  a.planes = dy.planes;
  a.vec = vec_rows(a.K, dxdt);
  if (H == 2) return dxdt == BL_F32 ? launch_gi<2, float>(tdy, tw, a, s) : launch_gi<2, __nv_bfloat16>(tdy, tw, a, s);
  return dxdt == BL_F32 ? launch_gi<1, float>(tdy, tw, a, s) : launch_gi<1, __nv_bfloat16>(tdy, tw, a, s);
}

template <typename DyT, int ND>
bl_status launch_gw_digits(const void* dy, const float* eta, int64_t M, int64_t N, int64_t Mp, uint8_t* digits,
                           float* scale, cudaStream_t s) {
  static int done[kMaxDevices] = {0};
  auto kern = bl::k_gw_digits<DyT, ND>;
  constexpr size_t smem = ND * bl::kGdCols * bl::kGwChunk;
  if (!ensure_smem(kern, smem, done)) return BL_ERR_CUDA;
  const int64_t blocks = ((N + bl::kGdCols - 1) / bl::kGdCols) * ((M + bl::kGwChunk - 1) / bl::kGwChunk);
  if (blocks > INT32_MAX) return BL_ERR_UNSUPPORTED;
  return launch_pdl(kern, dim3(static_cast<unsigned>(blocks)), dim3(bl::kGdThreads), smem, s,
                    static_cast<const DyT*>(dy), eta, M, N, Mp, N % 2 == 0 ? 1 : 0, digits, scale);
}

template <int ND, typename OutT>
bl_status launch_gw(const CUtensorMap& td, const CUtensorMap& tx, const float* scale, int M, int N, int K, void* dw,
                    int vec, int sms, cudaStream_t s) {
  static int done[kMaxDevices] = {0};
  auto kern = bl::k_grad_weight<ND, OutT>;
  if (!ensure_smem(kern, bl::kGwSmem, done)) return BL_ERR_CUDA;
  const int64_t tiles = ((int64_t{K} + bl::kGwBN - 1) / bl::kGwBN) * ((int64_t{N} + 127) / 128);
  const int64_t grid = tiles < sms ? tiles : sms;
  return launch_pdl(kern, dim3(static_cast<unsigned>(grid)), dim3(bl::kGwThreads), bl::kGwSmem, s, td, tx, scale, M, N,
                    K, dw, vec);
}

// Workspace of grad_weight: the digit planes, their exponents, the codes.
struct GwScratch {
  int64_t Mp;
  uint8_t *digits, *codes;
  float* scale;
};

inline GwScratch gw_scratch(int64_t M, int64_t N, int64_t K, int nd, Scratch* ws) {
  GwScratch g;
  g.Mp = round_up(M, 16);
  g.digits = static_cast<uint8_t*>(ws->take(static_cast<size_t>(nd * N * g.Mp)));
  g.codes = static_cast<uint8_t*>(ws->take(static_cast<size_t>(K * g.Mp)));
  g.scale = static_cast<float*>(ws->take(static_cast<size_t>((M + bl::kGwChunk - 1) / bl::kGwChunk * N * 4)));
  return g;
}

// One CTA per row, of as many warps as hold the row at kRgHeld chunks a thread.
template <typename DnT, typename OutT>
bl_status launch_rg(const void* dn, const int8_t* xq, const float* eta, const float* rstd, int64_t M, int64_t K,
                    void* dx, bool vec, int sms, cudaStream_t s) {
  const int64_t per_warp = 32 * 8 * bl::kRgHeld, warps = (K + per_warp - 1) / per_warp;
  const bool held = warps <= bl::kRgMaxThreads / 32;
  const auto* d = static_cast<const DnT*>(dn);
  const dim3 grid(grid_for(M, 1, sms)), block(static_cast<unsigned>(held ? 32 * warps : bl::kRgMaxThreads));
  if (held) return launch_pdl(bl::k_rmsnorm_grad<DnT, OutT, true>, grid, block, 0, s, d, xq, eta, rstd, M, K, dx, vec ? 1 : 0);
  return launch_pdl(bl::k_rmsnorm_grad<DnT, OutT, false>, grid, block, 0, s, d, xq, eta, rstd, M, K, dx, vec ? 1 : 0);
}

struct AdapterSet {
  const __nv_bfloat16 *A, *B;
  const float* scale;
  const int32_t* ids;
  int L, r;
};

template <typename DyT>
bl_status launch_adapters_grad(const void* dy, const int8_t* xq, const float* eta, int64_t M, int64_t K,
                               int64_t N, const AdapterSet& ad, void* dA, void* dB, bl_dtype dabdt, float* u,
                               float* v, int sms, cudaStream_t s) {
  const auto* d = static_cast<const DyT*>(dy);
  bl::k_adapter_v<DyT><<<grid_for(M * ad.r, 8, sms), 256, 0, s>>>(d, M, N, ad.B, ad.scale, ad.ids, ad.L, ad.r, v);
  if (!dA) return launch_status();
  bl::k_adapter_u<<<grid_for(M * ad.r, 8, sms), 256, 0, s>>>(xq, eta, M, K, ad.A, ad.scale, ad.ids, ad.L, ad.r, u);
  const unsigned ga = grid_for(int64_t{1} * ad.L * ad.r * K, 256, sms), gb = grid_for(int64_t{1} * ad.L * ad.r * N, 256, sms);
  if (dabdt == BL_F32) {
    bl::k_adapter_da<float><<<ga, 256, 0, s>>>(v, xq, eta, M, K, ad.ids, ad.L, ad.r, dA);
    bl::k_adapter_db<DyT, float><<<gb, 256, 0, s>>>(d, u, M, N, ad.ids, ad.L, ad.r, dB);
  } else {
    bl::k_adapter_da<__nv_bfloat16><<<ga, 256, 0, s>>>(v, xq, eta, M, K, ad.ids, ad.L, ad.r, dA);
    bl::k_adapter_db<DyT, __nv_bfloat16><<<gb, 256, 0, s>>>(d, u, M, N, ad.ids, ad.L, ad.r, dB);
  }
  return launch_status();
}

}  // namespace

extern "C" {

size_t bitlinear_grad_input_workspace_bytes(int64_t M, int64_t N, int64_t K, bl_dtype dydt) {
  if (train_sizes(M, N, K) != BL_OK || !dtype_ok(dydt)) return 0;
  Scratch ws(nullptr);
  Rows r;
  dy_rows(nullptr, dydt, M, N, &ws, &r, 1, nullptr);
  pad_rows(nullptr, N, (K + 3) / 4, &ws, &r, 1, nullptr);
  return ws.used;
}

bl_status bitlinear_grad_input(const void* dy, bl_dtype dydt, int64_t M, int64_t N, const uint8_t* packed,
                               const float* gamma, int64_t K, void* dx, bl_dtype dxdt, void* workspace,
                               size_t workspace_bytes, void* stream) {
  bl_status st = train_sizes(M, N, K);
  if (st == BL_ERR_INVALID_ARG) return st;
  if (!dtype_ok(dydt) || !dtype_ok(dxdt) || !packed || !gamma) return BL_ERR_INVALID_ARG;
  if (st != BL_OK) return st;
  if (M == 0) return BL_OK;
  const size_t need = bitlinear_grad_input_workspace_bytes(M, N, K, dydt);
  if (!dy || !dx || (need && !workspace) || workspace_bytes < need) return BL_ERR_INVALID_ARG;
  if (!aligned(dy, 16) || !aligned(packed, 16) || !aligned(dx, 16) || !aligned(gamma, 4) || !aligned(workspace, 256))
    return BL_ERR_ALIGNMENT;
  int sms = 148;
  if ((st = device_info(&sms)) != BL_OK) return st;
  const cudaStream_t s = as_stream(stream);
  Scratch ws(workspace);
  Rows rdy;
  if ((st = dy_rows(dy, dydt, M, N, &ws, &rdy, sms, s)) != BL_OK) return st;
  bl::GiArgs a = {};
  a.gamma = gamma; a.M = static_cast<int>(M); a.N = static_cast<int>(N); a.K = static_cast<int>(K); a.dx = dx;
  return run_grad_input(rdy, packed, dxdt, a, &ws, sms, s);
}

size_t bitlinear_grad_weight_workspace_bytes(int64_t M, int64_t N, int64_t K, bl_dtype dydt, bl_dtype dwdt) {
  if (train_sizes(M, N, K) != BL_OK || !dtype_ok(dydt) || !dtype_ok(dwdt)) return 0;
  Scratch ws(nullptr);
  gw_scratch(M, N, K, dwdt == BL_F32 ? 3 : 2, &ws);
  return ws.used;
}

bl_status bitlinear_grad_weight(const void* dy, bl_dtype dydt, const int8_t* xq, const float* eta, int64_t M,
                                int64_t N, int64_t K, void* dw, bl_dtype dwdt, void* workspace,
                                size_t workspace_bytes, void* stream) {
  bl_status st = train_sizes(M, N, K);
  if (st == BL_ERR_INVALID_ARG) return st;
  if (!dtype_ok(dydt) || !dtype_ok(dwdt) || !dw) return BL_ERR_INVALID_ARG;
  if (st != BL_OK) return st;
  const size_t need = bitlinear_grad_weight_workspace_bytes(M, N, K, dydt, dwdt);
  if (M > 0 && (!dy || !xq || !eta)) return BL_ERR_INVALID_ARG;
  if ((need && !workspace) || workspace_bytes < need) return BL_ERR_INVALID_ARG;
  if (!aligned(dy, 16) || !aligned(xq, 16) || !aligned(eta, 4) || !aligned(dw, 16) || !aligned(workspace, 256))
    return BL_ERR_ALIGNMENT;
  int sms = 148;
  if ((st = device_info(&sms)) != BL_OK) return st;
  const cudaStream_t s = as_stream(stream);
  if (M == 0) {
    if (cudaMemsetAsync(dw, 0, static_cast<size_t>(N * K * dtype_bytes(dwdt)), s) == cudaSuccess) return BL_OK;
    (void)cudaGetLastError();
    return BL_ERR_CUDA;
  }
  Scratch ws(workspace);
  const int nd = dwdt == BL_F32 ? 3 : 2;
  const GwScratch g = gw_scratch(M, N, K, nd, &ws);
  if (dydt == BL_F32)
    st = nd == 3 ? launch_gw_digits<float, 3>(dy, eta, M, N, g.Mp, g.digits, g.scale, s)
                 : launch_gw_digits<float, 2>(dy, eta, M, N, g.Mp, g.digits, g.scale, s);
  else
    st = nd == 3 ? launch_gw_digits<__nv_bfloat16, 3>(dy, eta, M, N, g.Mp, g.digits, g.scale, s)
                 : launch_gw_digits<__nv_bfloat16, 2>(dy, eta, M, N, g.Mp, g.digits, g.scale, s);
  if (st != BL_OK) return st;
  const int64_t blocks = ((K + 63) / 64) * ((M + 127) / 128);
  if (blocks > INT32_MAX) return BL_ERR_UNSUPPORTED;
  if ((st = launch_pdl(bl::k_gw_codes, dim3(static_cast<unsigned>(blocks)), dim3(256), 0, s, xq, M, K, g.Mp, g.codes)) !=
      BL_OK)
    return st;
  CUtensorMap td, tx;
  if (!make_tmap(&td, CU_TENSOR_MAP_DATA_TYPE_UINT8, g.digits, g.Mp, N, nd, g.Mp, bl::kGwBM, 128,
                 CU_TENSOR_MAP_SWIZZLE_128B) ||
      !make_tmap(&tx, CU_TENSOR_MAP_DATA_TYPE_UINT8, g.codes, g.Mp, K, 0, g.Mp, bl::kGwBM, bl::kGwBN,
                 CU_TENSOR_MAP_SWIZZLE_128B))
    return BL_ERR_CUDA;
  const int m = static_cast<int>(M), n = static_cast<int>(N), k = static_cast<int>(K);
  const int vec = vec_rows(K, dwdt);
  return nd == 3 ? launch_gw<3, float>(td, tx, g.scale, m, n, k, dw, vec, sms, s)
                 : launch_gw<2, __nv_bfloat16>(td, tx, g.scale, m, n, k, dw, vec, sms, s);
}

bl_status bitlinear_rmsnorm_grad(const void* dn, bl_dtype dndt, const int8_t* xq, const float* eta,
                                 const float* rstd, int64_t M, int64_t K, void* dx, bl_dtype dxdt, void* stream) {
  if (M < 0 || K < 1 || !dtype_ok(dndt) || !dtype_ok(dxdt)) return BL_ERR_INVALID_ARG;
  if (K > (int64_t{1} << 24) || M > (int64_t{1} << 40) / K) return BL_ERR_UNSUPPORTED;
  if (M == 0) return BL_OK;
  if (!dn || !xq || !eta || !rstd || !dx) return BL_ERR_INVALID_ARG;
  if (!aligned(dn, dtype_bytes(dndt)) || !aligned(dx, dtype_bytes(dxdt)) || !aligned(eta, 4) || !aligned(rstd, 4))
    return BL_ERR_ALIGNMENT;
  int sms = 148;
  const bl_status st = device_info(&sms);
  if (st != BL_OK) return st;
  const cudaStream_t s = as_stream(stream);
  const bool vec = K % 8 == 0 && aligned(dn, 16) && aligned(xq, 8) && aligned(dx, 16);
  if (dndt == BL_F32)
    return dxdt == BL_F32 ? launch_rg<float, float>(dn, xq, eta, rstd, M, K, dx, vec, sms, s)
                          : launch_rg<float, __nv_bfloat16>(dn, xq, eta, rstd, M, K, dx, vec, sms, s);
  return dxdt == BL_F32 ? launch_rg<__nv_bfloat16, float>(dn, xq, eta, rstd, M, K, dx, vec, sms, s)
                        : launch_rg<__nv_bfloat16, __nv_bfloat16>(dn, xq, eta, rstd, M, K, dx, vec, sms, s);
}

size_t bitlinear_forward_adapters_workspace_bytes(int64_t M, int64_t K, int64_t N, int64_t L, int64_t r) {
  if (train_sizes(M, N, K) != BL_OK || adapter_sizes(L, r, N, K) != BL_OK) return 0;
  Scratch ws(nullptr);
  ws.take(static_cast<size_t>(M) * r * 4);  // u
  ws.take(static_cast<size_t>(M) * N * 4);  // the projection in fp32
  return ws.used;
}

bl_status bitlinear_forward_adapters(const int8_t* xq, const float* eta, const int32_t* xsum, int64_t M,
                                     int64_t K, const uint8_t* packed, const float* gamma, int64_t N,
                                     const void* A, const void* B, const float* scale, const int32_t* ids,
                                     int64_t L, int64_t r, void* y, bl_dtype ydt, void* workspace,
                                     size_t workspace_bytes, unsigned flags, void* stream) {
  bl_status st = train_sizes(M, N, K), sa = adapter_sizes(L, r, N, K);
  if (st == BL_ERR_INVALID_ARG || sa == BL_ERR_INVALID_ARG) return BL_ERR_INVALID_ARG;
  if (!dtype_ok(ydt) || !packed || !gamma || !A || !B || !scale) return BL_ERR_INVALID_ARG;
  if (st != BL_OK || sa != BL_OK) return BL_ERR_UNSUPPORTED;
  if (M == 0) return BL_OK;
  const size_t need = bitlinear_forward_adapters_workspace_bytes(M, K, N, L, r);
  if (!xq || !eta || !xsum || !ids || !y || !workspace || workspace_bytes < need) return BL_ERR_INVALID_ARG;
  if (!aligned(xq, 16) || !aligned(packed, 16) || !aligned(A, 16) || !aligned(B, 16) || !aligned(y, 16) ||
      !aligned(eta, 4) || !aligned(xsum, 4) || !aligned(gamma, 4) || !aligned(scale, 4) || !aligned(ids, 4) ||
      !aligned(workspace, 256))
    return BL_ERR_ALIGNMENT;
  int sms = 148;
  if ((st = device_info(&sms)) != BL_OK) return st;
  const cudaStream_t s = as_stream(stream);
  Scratch ws(workspace);
  float* u = static_cast<float*>(ws.take(static_cast<size_t>(M) * r * 4));
  float* base = static_cast<float*>(ws.take(static_cast<size_t>(M) * N * 4));
  const auto* a = static_cast<const __nv_bfloat16*>(A);
  const auto* b = static_cast<const __nv_bfloat16*>(B);
  if ((st = forward_impl(xq, eta, xsum, M, K, packed, gamma, N, base, BL_F32, nullptr, BL_PATH_AUTO, flags,
                         stream)) != BL_OK)
    return st;
  bl::k_adapter_u<<<grid_for(M * r, 8, sms), 256, 0, s>>>(xq, eta, M, K, a, scale, ids, static_cast<int>(L),
                                                          static_cast<int>(r), u);
  const unsigned g = grid_for(M * N, 256, sms);
  if (ydt == BL_F32)
    bl::k_adapter_add<float><<<g, 256, 0, s>>>(base, M, N, u, b, r, 1, ids, static_cast<int>(L), static_cast<int>(r), y);
  else
    bl::k_adapter_add<__nv_bfloat16><<<g, 256, 0, s>>>(base, M, N, u, b, r, 1, ids, static_cast<int>(L),
                                                       static_cast<int>(r), y);
  return launch_status();
}

size_t bitlinear_adapters_grad_workspace_bytes(int64_t M, int64_t N, int64_t K, int64_t L, int64_t r,
                                               bl_dtype dydt) {
  if (train_sizes(M, N, K) != BL_OK || adapter_sizes(L, r, N, K) != BL_OK || !dtype_ok(dydt)) return 0;
  Scratch ws(nullptr);
  ws.take(static_cast<size_t>(M) * r * 4);  // u
  ws.take(static_cast<size_t>(M) * r * 4);  // v
  Rows rows;
  dy_rows(nullptr, dydt, M, N, &ws, &rows, 1, nullptr);
  pad_rows(nullptr, N, (K + 3) / 4, &ws, &rows, 1, nullptr);
  return ws.used;
}

bl_status bitlinear_adapters_grad(const void* dy, bl_dtype dydt, const int8_t* xq, const float* eta, int64_t M,
                                  int64_t N, int64_t K, const uint8_t* packed, const float* gamma, const void* A,
                                  const void* B, const float* scale, const int32_t* ids, int64_t L, int64_t r,
                                  void* dx, bl_dtype dxdt, void* dA, void* dB, bl_dtype dabdt, void* workspace,
                                  size_t workspace_bytes, void* stream) {
  bl_status st = train_sizes(M, N, K), sa = adapter_sizes(L, r, N, K);
  if (st == BL_ERR_INVALID_ARG || sa == BL_ERR_INVALID_ARG) return BL_ERR_INVALID_ARG;
  if (!dtype_ok(dydt) || !dtype_ok(dxdt) || !dtype_ok(dabdt) || !A || !B || !scale) return BL_ERR_INVALID_ARG;
  if (!dx && !dA && !dB) return BL_ERR_INVALID_ARG;
  if ((dA == nullptr) != (dB == nullptr) || (dx && (!packed || !gamma))) return BL_ERR_INVALID_ARG;
  if (st != BL_OK || sa != BL_OK) return BL_ERR_UNSUPPORTED;
  const size_t need = bitlinear_adapters_grad_workspace_bytes(M, N, K, L, r, dydt);
  if (M > 0 && (!dy || !xq || !eta || !ids || !workspace)) return BL_ERR_INVALID_ARG;
  if (workspace_bytes < need) return BL_ERR_INVALID_ARG;
  if (!aligned(dy, 16) || !aligned(xq, 16) || !aligned(packed, 16) || !aligned(A, 16) || !aligned(B, 16) ||
      !aligned(dx, 16) || !aligned(dA, 16) || !aligned(dB, 16) || !aligned(eta, 4) || !aligned(gamma, 4) ||
      !aligned(scale, 4) || !aligned(ids, 4) || !aligned(workspace, 256))
    return BL_ERR_ALIGNMENT;
  int sms = 148;
  if ((st = device_info(&sms)) != BL_OK) return st;
  const cudaStream_t s = as_stream(stream);
  Scratch ws(workspace);
  float* u = static_cast<float*>(ws.take(static_cast<size_t>(M) * r * 4));
  float* v = static_cast<float*>(ws.take(static_cast<size_t>(M) * r * 4));
  const AdapterSet ad = {static_cast<const __nv_bfloat16*>(A), static_cast<const __nv_bfloat16*>(B), scale, ids,
                         static_cast<int>(L), static_cast<int>(r)};
  st = dydt == BL_F32
           ? launch_adapters_grad<float>(dy, xq, eta, M, K, N, ad, dA, dB, dabdt, u, v, sms, s)
           : launch_adapters_grad<__nv_bfloat16>(dy, xq, eta, M, K, N, ad, dA, dB, dabdt, u, v, sms, s);
  if (st != BL_OK || !dx || M == 0) return st;
  Rows rdy;
  if ((st = dy_rows(dy, dydt, M, N, &ws, &rdy, sms, s)) != BL_OK) return st;
  bl::GiArgs g = {};
  g.gamma = gamma; g.M = static_cast<int>(M); g.N = static_cast<int>(N); g.K = static_cast<int>(K); g.dx = dx;
  g.v = v; g.A = ad.A; g.ids = ids; g.L = ad.L; g.r = ad.r;
  return run_grad_input(rdy, packed, dxdt, g, &ws, sms, s);
}

}  // extern "C"
