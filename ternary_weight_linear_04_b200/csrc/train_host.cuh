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

template <typename DyT>
bl_status launch_grad_input(const void* dy, int64_t M, int64_t N, const uint8_t* packed, const float* gamma,
                            int64_t K, void* dx, bl_dtype dxdt, int sms, cudaStream_t s) {
  const auto* d = static_cast<const DyT*>(dy);
  const unsigned g = grid_for(M * K, 256, sms);
  if (dxdt == BL_F32) bl::k_grad_input<DyT, float><<<g, 256, 0, s>>>(d, M, N, packed, gamma, K, dx);
  else bl::k_grad_input<DyT, __nv_bfloat16><<<g, 256, 0, s>>>(d, M, N, packed, gamma, K, dx);
  return launch_status();
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
  return 0;
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
  return dydt == BL_F32 ? launch_grad_input<float>(dy, M, N, packed, gamma, K, dx, dxdt, sms, s)
                        : launch_grad_input<__nv_bfloat16>(dy, M, N, packed, gamma, K, dx, dxdt, sms, s);
}

size_t bitlinear_grad_weight_workspace_bytes(int64_t M, int64_t N, int64_t K, bl_dtype dydt, bl_dtype dwdt) {
  if (train_sizes(M, N, K) != BL_OK || !dtype_ok(dydt) || !dtype_ok(dwdt)) return 0;
  return 0;
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
  const unsigned g = grid_for(N * K, 256, sms);
  if (dydt == BL_F32) {
    const auto* d = static_cast<const float*>(dy);
    if (dwdt == BL_F32) bl::k_grad_weight<float, float><<<g, 256, 0, s>>>(d, xq, eta, M, N, K, dw);
    else bl::k_grad_weight<float, __nv_bfloat16><<<g, 256, 0, s>>>(d, xq, eta, M, N, K, dw);
  } else {
    const auto* d = static_cast<const __nv_bfloat16*>(dy);
    if (dwdt == BL_F32) bl::k_grad_weight<__nv_bfloat16, float><<<g, 256, 0, s>>>(d, xq, eta, M, N, K, dw);
    else bl::k_grad_weight<__nv_bfloat16, __nv_bfloat16><<<g, 256, 0, s>>>(d, xq, eta, M, N, K, dw);
  }
  return launch_status();
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
  const unsigned g = grid_for(M, 1, sms);
  if (dndt == BL_F32) {
    const auto* d = static_cast<const float*>(dn);
    if (dxdt == BL_F32) bl::k_rmsnorm_grad<float, float><<<g, 256, 0, s>>>(d, xq, eta, rstd, M, K, dx);
    else bl::k_rmsnorm_grad<float, __nv_bfloat16><<<g, 256, 0, s>>>(d, xq, eta, rstd, M, K, dx);
  } else {
    const auto* d = static_cast<const __nv_bfloat16*>(dn);
    if (dxdt == BL_F32) bl::k_rmsnorm_grad<__nv_bfloat16, float><<<g, 256, 0, s>>>(d, xq, eta, rstd, M, K, dx);
    else bl::k_rmsnorm_grad<__nv_bfloat16, __nv_bfloat16><<<g, 256, 0, s>>>(d, xq, eta, rstd, M, K, dx);
  }
  return launch_status();
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
  ws.take(static_cast<size_t>(M) * K * 4);  // the projection's input gradient in fp32
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
  float* base = static_cast<float*>(ws.take(static_cast<size_t>(M) * K * 4));
  const AdapterSet ad = {static_cast<const __nv_bfloat16*>(A), static_cast<const __nv_bfloat16*>(B), scale, ids,
                         static_cast<int>(L), static_cast<int>(r)};
  st = dydt == BL_F32
           ? launch_adapters_grad<float>(dy, xq, eta, M, K, N, ad, dA, dB, dabdt, u, v, sms, s)
           : launch_adapters_grad<__nv_bfloat16>(dy, xq, eta, M, K, N, ad, dA, dB, dabdt, u, v, sms, s);
  if (st != BL_OK || !dx || M == 0) return st;
  st = dydt == BL_F32 ? launch_grad_input<float>(dy, M, N, packed, gamma, K, base, BL_F32, sms, s)
                      : launch_grad_input<__nv_bfloat16>(dy, M, N, packed, gamma, K, base, BL_F32, sms, s);
  if (st != BL_OK) return st;
  const unsigned g = grid_for(M * K, 256, sms);
  if (dxdt == BL_F32) bl::k_adapter_add<float><<<g, 256, 0, s>>>(base, M, K, v, ad.A, 1, K, ids, ad.L, ad.r, dx);
  else bl::k_adapter_add<__nv_bfloat16><<<g, 256, 0, s>>>(base, M, K, v, ad.A, 1, K, ids, ad.L, ad.r, dx);
  return launch_status();
}

}  // extern "C"
