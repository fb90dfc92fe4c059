// train_host.cuh -- argument checks and launches of the backward pass and of
// the adapters (grad.cuh, rmsnorm_grad.cuh, adapters.cuh).  Included by
// bitlinear.cu after its own helpers.
#pragma once

#include <initializer_list>

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

// Whether an output shares memory with one of the inputs: kernels write while
// other CTAs still read.
struct Span {
  const void* p;
  int64_t bytes;
};

inline bool overlaps(const Span& out, std::initializer_list<Span> in) {
  const auto at = [](const Span& s) { return reinterpret_cast<uintptr_t>(s.p); };
  for (const Span& s : in)
    if (out.p && s.p && at(out) < at(s) + static_cast<uint64_t>(s.bytes) && at(s) < at(out) + static_cast<uint64_t>(out.bytes))
      return true;
  return false;
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

// Up to two copies, made by one launch.
struct Pads {
  bl::PadJob job[2] = {};
  int n = 0;
};

inline void pad_rows(const void* src, int64_t rows, int64_t bytes, int64_t multiple, Scratch* ws, Rows* out, Pads* pads) {
  *out = {src, bytes, 1};
  if (bytes % multiple == 0) return;
  out->stride = round_up(bytes, multiple);
  void* dst = ws->take(static_cast<size_t>(rows * out->stride));
  out->p = dst;
  pads->job[pads->n++] = {static_cast<const uint8_t*>(src), rows, bytes, out->stride, static_cast<uint8_t*>(dst)};
}

inline int64_t pad_items(const Pads& pads) {
  return pads.job[0].rows * (pads.job[0].stride / 16) + pads.job[1].rows * (pads.job[1].stride / 16);
}

inline bl_status run_pads(const Pads& pads, int sms, cudaStream_t s) {
  if (!pads.n) return BL_OK;
  return launch_pdl(bl::k_pad_rows, dim3(grid_for(pad_items(pads), 256, sms)), dim3(256), 0, s, pads.job[0], pads.job[1]);
}

// dy as bf16 planes: one, or three of an fp32 dy.
inline bl_status dy_rows(const void* dy, bl_dtype dydt, int64_t M, int64_t N, Scratch* ws, Rows* out, Pads* pads,
                         int sms, cudaStream_t s) {
  if (dydt == BL_BF16) {
    pad_rows(dy, M, 2 * N, 16, ws, out, pads);
    return BL_OK;
  }
  const int64_t cols = round_up(N, 8);
  void* dst = ws->take(static_cast<size_t>(3 * M * cols * 2));
  *out = {dst, 2 * cols, 3};
  if (!ws->base || M == 0) return BL_OK;
  return launch_pdl(bl::k_split_planes, dim3(grid_for(M * cols, 256, sms)), dim3(256), 0, s,
                    static_cast<const float*>(dy), M, N, cols, static_cast<__nv_bfloat16*>(dst));
}

// Whether rows of `cols` values of type dt take 16-byte stores.
inline int vec_rows(int64_t cols, bl_dtype dt) { return cols % (16 / dtype_bytes(dt)) == 0 ? 1 : 0; }

template <int H, typename OutT>
bl_status launch_gi(const CUtensorMap& tdy, const CUtensorMap& tw, const bl::GiArgs& a, cudaStream_t s) {
  static int done[kMaxDevices] = {0}, room[kMaxDevices][9] = {{0}};
  auto kern = bl::k_grad_input<H, OutT>;
  constexpr size_t smem = bl::GiCfg<H>::kSmem;
  if (!ensure_smem(kern, smem, done)) return BL_ERR_CUDA;
  const int64_t tiles = ((a.K + bl::kGiBN - 1) / bl::kGiBN) * ((int64_t{a.M} + 128 * H - 1) / (128 * H));
  if (tiles > INT32_MAX) return BL_ERR_UNSUPPORTED;
  int split = 1;
  if (H == 1) {
    // as many CTAs along the contraction, up to 8, as the GPU has room for
    // beside the tiles, four steps each at least.  77 x 3200 x 8640, 34 tiles:
    // 32 us with one CTA a tile, 21 with two, 17 with three, 27 with four, which
    // do not all fit
    const int64_t steps = (int64_t{a.N} + bl::kGiBK - 1) / bl::kGiBK * a.planes;
    split = steps >= 32 ? 8 : steps >= 8 ? static_cast<int>(steps / 4) : 1;
    while (split > 1 && tiles > cluster_room(kern, bl::kGiThreads, smem, split, room)) --split;
  }
  const dim3 grid(static_cast<unsigned>(tiles), 1, static_cast<unsigned>(split));
  return launch_pdl_cluster(kern, grid, dim3(bl::kGiThreads), smem, s, grid.z, tdy, tw, a);
}

// The operands of dx as TMA reads them; `pads`: the copies to be made first.
struct GiOperands {
  Rows dy, w;
  Pads pads;
};

bl_status gi_operands(const void* dy, bl_dtype dydt, const uint8_t* packed, int64_t M, int64_t N, int64_t K, Scratch* ws,
                      GiOperands* o, int sms, cudaStream_t s) {
  const bl_status st = dy_rows(dy, dydt, M, N, ws, &o->dy, &o->pads, sms, s);
  pad_rows(packed, N, (K + 3) / 4, 16, ws, &o->w, &o->pads);
  return st;
}

// Tokens of an input gradient's tile: 256 where such tiles fill most of the
// GPU, else 128.
inline int gi_tokens(int64_t M, int64_t K, int sms) {
  const int64_t ktiles = (K + bl::kGiBN - 1) / bl::kGiBN;
  return M > 128 && ktiles * ((M + 255) / 256) * 4 > int64_t{3} * sms ? 256 : 128;
}

// dx = gamma dy W~ (+ v A where a.v is given), the copies made.
bl_status run_grad_input(const GiOperands& o, bl_dtype dxdt, bl::GiArgs a, int sms, cudaStream_t s) {
  const Rows &dy = o.dy, &w = o.w;
  const int H = gi_tokens(a.M, a.K, sms) / 128;
  CUtensorMap tdy, tw;
  if (!make_tmap(&tdy, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, dy.p, a.N, a.M, dy.planes, dy.stride, bl::kGiBK, 128 * H,
                 CU_TENSOR_MAP_SWIZZLE_128B) ||
      !make_tmap(&tw, CU_TENSOR_MAP_DATA_TYPE_UINT8, w.p, (a.K + 3) / 4, a.N, 0, w.stride, bl::kGiBN / 4,
                 bl::kGiBK, CU_TENSOR_MAP_SWIZZLE_64B))
    return BL_ERR_CUDA;
  a.planes = dy.planes;
  a.vec = vec_rows(a.K, dxdt);
  if (H == 2)
    return dxdt == BL_F32 ? launch_gi<2, float>(tdy, tw, a, s) : launch_gi<2, __nv_bfloat16>(tdy, tw, a, s);
  return dxdt == BL_F32 ? launch_gi<1, float>(tdy, tw, a, s) : launch_gi<1, __nv_bfloat16>(tdy, tw, a, s);
}

// Launch of `blocks` (an even number) CTAs in clusters of two along x, with
// programmatic dependent launch allowed.
template <typename... KArgs, typename... Args>
bl_status launch_pdl_pairs(void (*kern)(KArgs...), unsigned blocks, int threads, size_t smem, cudaStream_t st,
                           Args&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(blocks);
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = 2;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  if (cudaLaunchKernelEx(&cfg, kern, std::forward<Args>(args)...) != cudaSuccess) {
    (void)cudaGetLastError();
    return BL_ERR_CUDA;
  }
  return launch_status();
}

template <typename OutT>
bl_status launch_gw(const CUtensorMap& td, const CUtensorMap& tx, const float* scale, const uint8_t* extra, int M, int N,
                    int K, void* dw, int sms, cudaStream_t s) {
  static int done[kMaxDevices] = {0};
  auto kern = bl::k_grad_weight<OutT>;
  if (!ensure_smem(kern, bl::kGwSmem, done)) return BL_ERR_CUDA;
  const int64_t tiles = ((int64_t{K} + bl::kGwBN - 1) / bl::kGwBN) * ((int64_t{N} + bl::kGwRows - 1) / bl::kGwRows);
  if (tiles > INT32_MAX / 2) return BL_ERR_UNSUPPORTED;
  const int64_t pairs = tiles < sms / 2 ? tiles : sms / 2;
  return launch_pdl_pairs(kern, static_cast<unsigned>(2 * pairs), bl::kGwThreads, bl::kGwSmem, s, td, tx, scale, extra, M, N, K,
                          dw);
}

// Workspace of grad_weight: the digit planes, the codes, the planes' exponents
// and which of them are used.
struct GwScratch {
  int64_t Mp;
  uint8_t *digits, *codes;
  float* scale;
  uint8_t* extra;
};

inline GwScratch gw_scratch(int64_t M, int64_t N, int64_t K, Scratch* ws) {
  GwScratch g;
  g.Mp = round_up(M, 16);
  g.digits = static_cast<uint8_t*>(ws->take(static_cast<size_t>(bl::kGdPlanes * N * g.Mp)));
  g.codes = static_cast<uint8_t*>(ws->take(static_cast<size_t>(K * g.Mp)));
  const int64_t chunks = (M + bl::kGwChunk - 1) / bl::kGwChunk;
  g.scale = static_cast<float*>(ws->take(static_cast<size_t>(chunks * N * 4)));
  g.extra = static_cast<uint8_t*>(ws->take(static_cast<size_t>(chunks * (round_up(N, bl::kGwRows) / bl::kGdCols))));
  return g;
}

template <typename DyT>
bl_status launch_gw_operands(const void* dy, const int8_t* xq, const float* eta, int64_t M, int64_t N, int64_t K,
                             const GwScratch& g, cudaStream_t s) {
  static int done[kMaxDevices] = {0};
  auto kern = bl::k_gw_operands<DyT>;
  constexpr size_t smem = 3 * bl::kGdCols * bl::kGdTokens;
  if (!ensure_smem(kern, smem, done)) return BL_ERR_CUDA;
  const int64_t digits = 2 * ((N + bl::kGdCols - 1) / bl::kGdCols) * ((M + bl::kGwChunk - 1) / bl::kGwChunk);
  const int64_t blocks = round_up(digits + ((K + 63) / 64) * ((M + 127) / 128), 2);
  if (blocks > INT32_MAX) return BL_ERR_UNSUPPORTED;
  return launch_pdl_pairs(kern, static_cast<unsigned>(blocks), bl::kGdThreads, smem, s, static_cast<unsigned>(digits), xq, K, g.codes, static_cast<const DyT*>(dy), eta, M, N, g.Mp,
                    N % 2 == 0 ? 1 : 0, g.digits, g.scale, g.extra);
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

// u of up to 16 tokens (k_adapter_u): rows of x~ (or of x, quantised there)
// and of A in 16-byte pieces, K within a CTA's registers.
inline bool few_tokens_u(int64_t M, int64_t K) {
  return M <= 16 && K % 8 == 0 && K <= 8 * bl::kAuChunks * bl::kAuThreads;
}

bl_status launch_u_few(const void* x, int8_t* xq, float* eta, int32_t* xsum, int64_t M, int64_t K, const AdapterSet& ad,
                       float* u, int sms, cudaStream_t s) {
  // rank indices per CTA: one while the CTAs fit on the GPU about at once
  // (eight of 256 threads an SM), more where every CTA would read its token
  // again for little work
  const int64_t group = (M * ad.r + sms * 8 - 1) / (sms * 8);
  const dim3 grid(static_cast<unsigned>((ad.r + group - 1) / group), static_cast<unsigned>(M));
  auto kern = x ? bl::k_adapter_u<true> : bl::k_adapter_u<false>;
  return launch_pdl(kern, grid, dim3(bl::kAuThreads), 0, s, static_cast<const __nv_bfloat16*>(x), xq, eta, xsum,
                    static_cast<int>(K), ad.A, ad.scale, ad.ids, ad.L, ad.r, static_cast<int>(group), u);
}

// Scratch of k_adapter_sort.
struct Order {
  int32_t *rows, *start, *first;
};

inline Order order_scratch(int64_t M, int64_t L, Scratch* ws) {
  Order o;
  o.rows = static_cast<int32_t*>(ws->take(static_cast<size_t>(M * 4)));
  o.start = static_cast<int32_t*>(ws->take(static_cast<size_t>((L + 1) * 4)));
  o.first = L > 255 ? static_cast<int32_t*>(ws->take(static_cast<size_t>(M * 4))) : nullptr;
  return o;
}

// With the copies of `pads` in the same launch.
bl_status launch_sort(const AdapterSet& ad, int64_t M, const Order& o, const Pads& pads, int sms, cudaStream_t s) {
  const int64_t n = pad_items(pads);
  const unsigned grid = 1 + (n ? grid_for(n, bl::kSortThreads, sms) : 0);
  return launch_pdl(bl::k_adapter_sort, dim3(grid), dim3(bl::kSortThreads), 0, s, ad.ids, M, ad.L, o.first, o.rows,
                    o.start, pads.job[0], pads.job[1]);
}

template <typename DyT, int NT>
bl_status launch_uv_nt(const bl::UvArgs& g, int sides, int64_t steps, cudaStream_t s) {
  static int done[kMaxDevices] = {0}, room[kMaxDevices][9] = {{0}};
  auto kern = bl::k_adapter_uv<DyT, NT>;
  if (!ensure_smem(kern, bl::kUvSmem, done)) return BL_ERR_CUDA;
  const int64_t tiles = (g.M + 15) / 16;
  if (tiles > INT32_MAX) return BL_ERR_UNSUPPORTED;
  // CTAs of a cluster along the contraction: while the GPU has room for all
  // of them at once and there are steps for all their warps
  int cs = 1;
  while (cs < 8 && steps > bl::kUvWarps * cs &&
         tiles * sides <= cluster_room(kern, bl::kUvThreads, bl::kUvSmem, 2 * cs, room))
    cs *= 2;
  const dim3 grid(static_cast<unsigned>(tiles), static_cast<unsigned>(sides), static_cast<unsigned>(cs));
  return launch_pdl_cluster(kern, grid, dim3(bl::kUvThreads), bl::kUvSmem, s, grid.z, g);
}

template <typename DyT>
bl_status launch_uv_t(const bl::UvArgs& g, int sides, int64_t steps, cudaStream_t s) {
  if (g.r <= 8) return launch_uv_nt<DyT, 1>(g, sides, steps, s);
  return g.r <= 16 ? launch_uv_nt<DyT, 2>(g, sides, steps, s) : launch_uv_nt<DyT, 4>(g, sides, steps, s);
}

// u (where out_u is given) and v (out_v) of any number of tokens, in the
// order of `rows` where it is given.
bl_status launch_uv(const void* dy, bl_dtype dydt, const int8_t* xq, const float* eta, int64_t M, int64_t K, int64_t N,
                    const AdapterSet& ad, const int32_t* rows, float* out_u, float* out_v, cudaStream_t s) {
  bl::UvArgs g = {};
  g.scale = ad.scale; g.ids = ad.ids; g.rows = rows; g.M = M; g.L = ad.L; g.r = ad.r;
  int n = 0;
  if (out_v) g.side[n++] = {1, dy, N, ad.B, nullptr, out_v, N % 4 == 0 ? 1 : 0};
  if (out_u) g.side[n++] = {0, xq, K, ad.A, eta, out_u, K % 16 == 0 ? 1 : 0};
  int64_t steps = out_v ? (N + 63) / 64 : 0;
  if (out_u && (K + 63) / 64 > steps) steps = (K + 63) / 64;
  return out_v && dydt == BL_F32 ? launch_uv_t<float>(g, n, steps, s) : launch_uv_t<__nv_bfloat16>(g, n, steps, s);
}

template <typename DyT, typename OutT, int JT>
bl_status launch_dab_jt(const bl::DabArgs& g, dim3 grid, cudaStream_t s) {
  static int done[kMaxDevices] = {0};
  auto kern = bl::k_adapter_dab<DyT, OutT, JT>;
  constexpr int xparts = sizeof(DyT) == 4 ? 3 : 1;
  if (!ensure_smem(kern, bl::dab_smem(16 * JT, xparts), done)) return BL_ERR_CUDA;
  return launch_pdl_cluster(kern, grid, dim3(bl::kDabThreads), bl::dab_smem(g.r, xparts), s, grid.z, g);
}

template <typename DyT, typename OutT>
bl_status launch_dab(const void* dy, const int8_t* xq, const float* eta, int64_t M, int64_t K, int64_t N,
                     const AdapterSet& ad, const Order& o, const float* u, const float* v, void* dA, void* dB, int sms,
                     cudaStream_t s) {
  const int64_t sa = (K + bl::kDabCols - 1) / bl::kDabCols, sb = (N + bl::kDabCols - 1) / bl::kDabCols;
  bl::DabArgs g = {};
  g.a = {xq, K, v, dA, K % 16 == 0 ? 1 : 0};
  g.b = {dy, N, u, dB, N % (sizeof(DyT) == 4 ? 4 : 8) == 0 ? 1 : 0};
  g.eta = eta; g.rows = o.rows; g.start = o.start; g.r = ad.r; g.slabs_a = static_cast<unsigned>(sa);
  // CTAs of a cluster along the tokens: while there are fewer than four CTAs
  // an SM, and two chunks of tokens for each; two where one adapter may have
  // more than 16 chunks (2048 tokens: dA and dB 3 us less)
  int cs = M > 16 * bl::kDabTokens ? 2 : 1;
  while (cs < 8 && (sa + sb) * ad.L * cs < 4 * sms && M >= 4 * bl::kDabTokens * cs) cs *= 2;
  const dim3 grid(static_cast<unsigned>(sa + sb), static_cast<unsigned>(ad.L), static_cast<unsigned>(cs));
  if (ad.r <= 16) return launch_dab_jt<DyT, OutT, 1>(g, grid, s);
  if (ad.r <= 32) return launch_dab_jt<DyT, OutT, 2>(g, grid, s);
  if (ad.r <= 64) return launch_dab_jt<DyT, OutT, 4>(g, grid, s);
  return launch_dab_jt<DyT, OutT, 8>(g, grid, s);
}

// Scratch of the forward pass: u, then the operands' copies where K is not a
// multiple of 64 (rows of x~ padded with zeros, which meet any code).
struct FaScratch {
  float* u;
  Order order;  // rows NULL: not sorted
  Rows x, w;
  Pads pads;
};

// Tokens are sorted where a tile of 16 could meet several adapters.
inline void fa_scratch(const int8_t* xq, const uint8_t* packed, int64_t M, int64_t K, int64_t N, int64_t L, int64_t r,
                       Scratch* ws, FaScratch* f) {
  f->u = static_cast<float*>(ws->take(static_cast<size_t>(M * bl::rank_stride(static_cast<int>(r)) * 4)));
  f->order = M > 16 && L > 1 ? order_scratch(M, L, ws) : Order{nullptr, nullptr, nullptr};
  if (K % 64 == 0) {
    f->x = {xq, K, 1};
    f->w = {packed, K / 4, 1};
    return;
  }
  const int64_t kp = round_up(K, 64);
  auto* x = static_cast<uint8_t*>(ws->take(static_cast<size_t>(M * kp)));
  auto* w = static_cast<uint8_t*>(ws->take(static_cast<size_t>(N * (kp / 4))));
  f->x = {x, kp, 1};
  f->w = {w, kp / 4, 1};
  f->pads.job[0] = {reinterpret_cast<const uint8_t*>(xq), M, K, kp, x};
  f->pads.job[1] = {packed, N, (K + 3) / 4, kp / 4, w};
  f->pads.n = 2;
}

// u of the forward pass, and the operands' copies.
bl_status run_u(const FaScratch& f, int8_t* xq, float* eta, int64_t M, int64_t K, int64_t N, const AdapterSet& ad, int sms,
                cudaStream_t s) {
  if (few_tokens_u(M, K)) {
    const bl_status st = launch_u_few(nullptr, xq, eta, nullptr, M, K, ad, f.u, sms, s);
    return st == BL_OK ? run_pads(f.pads, sms, s) : st;
  }
  const bl_status st = f.order.rows ? launch_sort(ad, M, f.order, f.pads, sms, s) : run_pads(f.pads, sms, s);
  if (st != BL_OK) return st;
  return launch_uv(nullptr, BL_BF16, xq, eta, M, K, N, ad, f.order.rows, f.u, nullptr, s);
}

// The projection with adapters, u given in f.
bl_status run_forward_adapters(const FaScratch& f, const float* eta, const int32_t* xsum, int64_t M, const float* gamma,
                               int64_t N, const AdapterSet& ad, void* y, bl_dtype ydt, unsigned flags, int sms,
                               cudaStream_t s) {
  if (f.pads.n) flags &= ~static_cast<unsigned>(BL_FLAG_WEIGHTS_STATIC);  // the copy is new
  const bl::AdapterAdd add = {f.u, ad.B, ad.ids, ad.L, ad.r};
  return forward_impl(static_cast<const int8_t*>(f.x.p), eta, xsum, M, f.x.stride, static_cast<const uint8_t*>(f.w.p),
                      gamma, N, y, ydt, nullptr, BL_PATH_AUTO, flags, s, add);
}

// Scratch of linear_adapters: the quantised tokens, then the forward pass's.
struct LaScratch {
  int8_t* xq;
  float* eta;
  int32_t* xsum;
};

inline void la_scratch(int64_t M, int64_t K, Scratch* ws, LaScratch* q) {
  q->xq = static_cast<int8_t*>(ws->take(static_cast<size_t>(M * K)));
  q->eta = static_cast<float*>(ws->take(static_cast<size_t>(M * 4)));
  q->xsum = static_cast<int32_t*>(ws->take(static_cast<size_t>(M * 4)));
}

// Sizes of the forward pass with adapters: those above, K padded to 64 and
// the projection's grid (65535 tiles of 256 tokens).
inline bl_status fa_sizes(int64_t M, int64_t N, int64_t K, int64_t L, int64_t r) {
  const bl_status st = train_sizes(M, N, K), sa = adapter_sizes(L, r, N, K);
  if (st == BL_ERR_INVALID_ARG || sa == BL_ERR_INVALID_ARG) return BL_ERR_INVALID_ARG;
  if (st != BL_OK || sa != BL_OK || 127 * round_up(K, 64) >= (int64_t{1} << 31) || M > 65535 * 256) return BL_ERR_UNSUPPORTED;
  return BL_OK;
}

// Checks that forward_adapters and linear_adapters share, in the order of
// the other calls: arguments, sizes, then (after M = 0) the rest.
bl_status fa_check(int64_t M, int64_t N, int64_t K, int64_t L, int64_t r, const uint8_t* packed, const float* gamma,
                   const void* A, const void* B, const float* scale, bl_dtype ydt) {
  const bl_status st = fa_sizes(M, N, K, L, r);
  if (st == BL_ERR_INVALID_ARG || !dtype_ok(ydt) || !packed || !gamma || !A || !B || !scale) return BL_ERR_INVALID_ARG;
  return st;
}

inline bool adapters_aligned(const uint8_t* packed, const float* gamma, const void* A, const void* B, const float* scale,
                             const int32_t* ids) {
  return aligned(packed, 16) && aligned(A, 16) && aligned(B, 16) && aligned(gamma, 4) && aligned(scale, 4) &&
         aligned(ids, 4);
}

inline AdapterSet adapter_set(const void* A, const void* B, const float* scale, const int32_t* ids, int64_t L, int64_t r) {
  return {static_cast<const __nv_bfloat16*>(A), static_cast<const __nv_bfloat16*>(B), scale, ids, static_cast<int>(L),
          static_cast<int>(r)};
}

}  // namespace

extern "C" {

size_t bitlinear_grad_input_workspace_bytes(int64_t M, int64_t N, int64_t K, bl_dtype dydt) {
  if (train_sizes(M, N, K) != BL_OK || !dtype_ok(dydt)) return 0;
  Scratch ws(nullptr);
  GiOperands o;
  gi_operands(nullptr, dydt, nullptr, M, N, K, &ws, &o, 1, nullptr);
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
  if (overlaps({dx, M * K * dtype_bytes(dxdt)}, {{dy, M * N * dtype_bytes(dydt)}, {packed, N * ((K + 3) / 4)}, {gamma, 4}}))
    return BL_ERR_INVALID_ARG;
  int sms = 148;
  if ((st = device_info(&sms)) != BL_OK) return st;
  const cudaStream_t s = as_stream(stream);
  Scratch ws(workspace);
  bl::GiArgs a = {};
  a.gamma = gamma; a.M = static_cast<int>(M); a.N = static_cast<int>(N); a.K = static_cast<int>(K); a.dx = dx;
  GiOperands o;
  if ((st = gi_operands(dy, dydt, packed, M, N, K, &ws, &o, sms, s)) != BL_OK) return st;
  if ((st = run_pads(o.pads, sms, s)) != BL_OK) return st;
  return run_grad_input(o, dxdt, a, sms, s);
}

int32_t bitlinear_tile_tokens(int grad, int64_t M, int64_t K, int64_t N, int sms) {
  if (M < 1 || sms < 1 || (grad ? train_sizes(M, N, K) : fa_sizes(M, N, K, 1, 1)) != BL_OK) return 0;
  return grad ? gi_tokens(M, K, sms)
              : tc_tokens<true>(static_cast<int>(M), static_cast<int>(round_up(K, 64)), static_cast<int>(N), sms);
}

size_t bitlinear_grad_weight_workspace_bytes(int64_t M, int64_t N, int64_t K, bl_dtype dydt, bl_dtype dwdt) {
  if (train_sizes(M, N, K) != BL_OK || !dtype_ok(dydt) || !dtype_ok(dwdt)) return 0;
  Scratch ws(nullptr);
  gw_scratch(M, N, K, &ws);
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
  if (overlaps({dw, N * K * dtype_bytes(dwdt)}, {{dy, M * N * dtype_bytes(dydt)}, {xq, M * K}, {eta, 4 * M}}))
    return BL_ERR_INVALID_ARG;
  int sms = 148;
  if ((st = device_info(&sms)) != BL_OK) return st;
  const cudaStream_t s = as_stream(stream);
  if (M == 0) {
    if (cudaMemsetAsync(dw, 0, static_cast<size_t>(N * K * dtype_bytes(dwdt)), s) == cudaSuccess) return BL_OK;
    (void)cudaGetLastError();
    return BL_ERR_CUDA;
  }
  Scratch ws(workspace);
  const GwScratch g = gw_scratch(M, N, K, &ws);
  st = dydt == BL_F32 ? launch_gw_operands<float>(dy, xq, eta, M, N, K, g, s)
                      : launch_gw_operands<__nv_bfloat16>(dy, xq, eta, M, N, K, g, s);
  if (st != BL_OK) return st;
  CUtensorMap td, tx;
  if (!make_tmap(&td, CU_TENSOR_MAP_DATA_TYPE_UINT8, g.digits, g.Mp, N, bl::kGdPlanes, g.Mp, bl::kGwBM, 128,
                 CU_TENSOR_MAP_SWIZZLE_128B) ||
      !make_tmap(&tx, CU_TENSOR_MAP_DATA_TYPE_UINT8, g.codes, g.Mp, K, 0, g.Mp, bl::kGwBM, bl::kGwBN / 2,
                 CU_TENSOR_MAP_SWIZZLE_128B))
    return BL_ERR_CUDA;
  const int m = static_cast<int>(M), n = static_cast<int>(N), k = static_cast<int>(K);
  return dwdt == BL_F32 ? launch_gw<float>(td, tx, g.scale, g.extra, m, n, k, dw, sms, s)
                        : launch_gw<__nv_bfloat16>(td, tx, g.scale, g.extra, m, n, k, dw, sms, s);
}

bl_status bitlinear_rmsnorm_grad(const void* dn, bl_dtype dndt, const int8_t* xq, const float* eta,
                                 const float* rstd, int64_t M, int64_t K, void* dx, bl_dtype dxdt, void* stream) {
  if (M < 0 || K < 1 || !dtype_ok(dndt) || !dtype_ok(dxdt)) return BL_ERR_INVALID_ARG;
  if (K > (int64_t{1} << 24) || M > (int64_t{1} << 40) / K) return BL_ERR_UNSUPPORTED;
  if (M == 0) return BL_OK;
  if (!dn || !xq || !eta || !rstd || !dx) return BL_ERR_INVALID_ARG;
  if (!aligned(dn, dtype_bytes(dndt)) || !aligned(dx, dtype_bytes(dxdt)) || !aligned(eta, 4) || !aligned(rstd, 4))
    return BL_ERR_ALIGNMENT;
  const Span out = {dx, M * K * dtype_bytes(dxdt)};
  const bool in_place = dx == dn && dxdt == dndt;  // a thread reads what it writes before
  if (overlaps(out, {{xq, M * K}, {eta, 4 * M}, {rstd, 4 * M}}) || (!in_place && overlaps(out, {{dn, M * K * dtype_bytes(dndt)}})))
    return BL_ERR_INVALID_ARG;
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
  if (fa_sizes(M, N, K, L, r) != BL_OK) return 0;
  Scratch ws(nullptr);
  FaScratch f;
  fa_scratch(nullptr, nullptr, M, K, N, L, r, &ws, &f);
  return ws.used;
}

bl_status bitlinear_forward_adapters(const int8_t* xq, const float* eta, const int32_t* xsum, int64_t M,
                                     int64_t K, const uint8_t* packed, const float* gamma, int64_t N,
                                     const void* A, const void* B, const float* scale, const int32_t* ids,
                                     int64_t L, int64_t r, void* y, bl_dtype ydt, void* workspace,
                                     size_t workspace_bytes, unsigned flags, void* stream) {
  bl_status st = fa_check(M, N, K, L, r, packed, gamma, A, B, scale, ydt);
  if (st != BL_OK || M == 0) return st;
  const size_t need = bitlinear_forward_adapters_workspace_bytes(M, K, N, L, r);
  if (!xq || !eta || !xsum || !ids || !y || !workspace || workspace_bytes < need) return BL_ERR_INVALID_ARG;
  if (!adapters_aligned(packed, gamma, A, B, scale, ids) || !aligned(xq, 16) || !aligned(y, 16) || !aligned(eta, 4) ||
      !aligned(xsum, 4) || !aligned(workspace, 256))
    return BL_ERR_ALIGNMENT;
  if (overlaps({y, M * N * dtype_bytes(ydt)}, {{xq, M * K}, {eta, 4 * M}, {xsum, 4 * M}, {packed, N * ((K + 3) / 4)},
                                              {gamma, 4}, {A, 2 * L * r * K}, {B, 2 * L * r * N}, {scale, 4 * L}, {ids, 4 * M}}))
    return BL_ERR_INVALID_ARG;
  int sms = 148;
  if ((st = device_info(&sms)) != BL_OK) return st;
  const cudaStream_t s = as_stream(stream);
  Scratch ws(workspace);
  FaScratch f;
  fa_scratch(xq, packed, M, K, N, L, r, &ws, &f);
  const AdapterSet ad = adapter_set(A, B, scale, ids, L, r);
  st = run_u(f, const_cast<int8_t*>(xq), const_cast<float*>(eta), M, K, N, ad, sms, s);  // neither is written
  return st == BL_OK ? run_forward_adapters(f, eta, xsum, M, gamma, N, ad, y, ydt, flags, sms, s) : st;
}

size_t bitlinear_linear_adapters_workspace_bytes(int64_t M, int64_t K, int64_t N, int64_t L, int64_t r) {
  const size_t fwd = bitlinear_forward_adapters_workspace_bytes(M, K, N, L, r);
  if (!fwd) return 0;
  Scratch ws(nullptr);
  LaScratch q;
  la_scratch(M, K, &ws, &q);
  return ws.used + fwd;
}

bl_status bitlinear_linear_adapters(const void* x, bl_dtype xdt, int64_t M, int64_t K, const uint8_t* packed,
                                    const float* gamma, int64_t N, const void* A, const void* B,
                                    const float* scale, const int32_t* ids, int64_t L, int64_t r, void* y,
                                    bl_dtype ydt, void* workspace, size_t workspace_bytes, unsigned flags,
                                    void* stream) {
  bl_status st = fa_check(M, N, K, L, r, packed, gamma, A, B, scale, ydt);
  if (st == BL_ERR_INVALID_ARG || !dtype_ok(xdt)) return BL_ERR_INVALID_ARG;
  const bool norm = (flags & BL_FLAG_RMSNORM) != 0;
  if (st != BL_OK || (norm && xdt != BL_BF16)) return BL_ERR_UNSUPPORTED;
  if (M == 0) return BL_OK;
  const size_t need = bitlinear_linear_adapters_workspace_bytes(M, K, N, L, r);
  if (!x || !ids || !y || !workspace || workspace_bytes < need) return BL_ERR_INVALID_ARG;
  if (!adapters_aligned(packed, gamma, A, B, scale, ids) || !aligned(x, dtype_bytes(xdt)) || !aligned(y, 16) ||
      !aligned(workspace, 256))
    return BL_ERR_ALIGNMENT;
  if (overlaps({y, M * N * dtype_bytes(ydt)}, {{x, M * K * dtype_bytes(xdt)}, {packed, N * ((K + 3) / 4)}, {gamma, 4},
                                              {A, 2 * L * r * K}, {B, 2 * L * r * N}, {scale, 4 * L}, {ids, 4 * M}}))
    return BL_ERR_INVALID_ARG;
  int sms = 148;
  if ((st = device_info(&sms)) != BL_OK) return st;
  const cudaStream_t s = as_stream(stream);
  Scratch ws(workspace);
  LaScratch q;
  la_scratch(M, K, &ws, &q);
  FaScratch f;
  fa_scratch(q.xq, packed, M, K, N, L, r, &ws, &f);
  const AdapterSet ad = adapter_set(A, B, scale, ids, L, r);
  if (!norm && xdt == BL_BF16 && aligned(x, 16) && few_tokens_u(M, K)) {
    RegGeom rg;
    const bool one = M == 1 && g_decode_reg.load(std::memory_order_relaxed) != 0 && reg_decode_geometry(K, N, sms, &rg);
    // one token: the accumulate kernel quantises again, x~ need not be written
    if ((st = launch_u_few(x, one ? nullptr : q.xq, q.eta, q.xsum, M, K, ad, f.u, sms, s)) != BL_OK) return st;
    if (one) {
      bl::RegDecodeArgs a = {};
      a.x = static_cast<const __nv_bfloat16*>(x);
      a.K = static_cast<int>(K); a.N = static_cast<int>(N);
      a.packed = packed; a.gamma = gamma; a.y = y; a.y_bf16 = ydt == BL_BF16 ? 1 : 0;
      a.rows_per_cta = rg.rows_per_cta;
      a.weights_static = (flags & BL_FLAG_WEIGHTS_STATIC) ? 1 : 0;
      a.ad = {f.u, ad.B, ids, ad.L, ad.r};
      return launch_decode_reg(a, rg, s);
    }
    if ((st = run_pads(f.pads, sms, s)) != BL_OK) return st;
  } else {
    st = norm ? rmsnorm_quant_impl(x, xdt, M, K, q.xq, q.eta, q.xsum, nullptr, stream)
              : bitlinear_quant_act(x, xdt, M, K, q.xq, q.eta, q.xsum, stream);
    if (st != BL_OK) return st;
    if ((st = run_u(f, q.xq, q.eta, M, K, N, ad, sms, s)) != BL_OK) return st;
  }
  return run_forward_adapters(f, q.eta, q.xsum, M, gamma, N, ad, y, ydt, flags, sms, s);
}

size_t bitlinear_adapters_grad_workspace_bytes(int64_t M, int64_t N, int64_t K, int64_t L, int64_t r,
                                               bl_dtype dydt) {
  if (train_sizes(M, N, K) != BL_OK || adapter_sizes(L, r, N, K) != BL_OK || !dtype_ok(dydt)) return 0;
  Scratch ws(nullptr);
  for (int i = 0; i < 2; ++i) ws.take(static_cast<size_t>(M) * bl::rank_stride(static_cast<int>(r)) * 4);  // u, v
  order_scratch(M, L, &ws);
  return ws.used + bitlinear_grad_input_workspace_bytes(M, N, K, dydt);
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
  if (M > 0 && (!dy || !xq || !eta || !ids)) return BL_ERR_INVALID_ARG;
  if ((need && !workspace) || workspace_bytes < need) return BL_ERR_INVALID_ARG;
  if (!adapters_aligned(packed, gamma, A, B, scale, ids) || !aligned(dy, 16) || !aligned(xq, 16) ||
      !aligned(dx, 16) || !aligned(dA, 16) || !aligned(dB, 16) || !aligned(eta, 4) || !aligned(workspace, 256))
    return BL_ERR_ALIGNMENT;
  for (const Span& out : {Span{dx, M * K * dtype_bytes(dxdt)}, Span{dA, L * r * K * dtype_bytes(dabdt)},
                          Span{dB, L * r * N * dtype_bytes(dabdt)}})
    if (overlaps(out, {{dy, M * N * dtype_bytes(dydt)}, {xq, M * K}, {eta, 4 * M}, {packed, N * ((K + 3) / 4)}, {gamma, 4},
                       {A, 2 * L * r * K}, {B, 2 * L * r * N}, {scale, 4 * L}, {ids, 4 * M}}))
      return BL_ERR_INVALID_ARG;
  int sms = 148;
  if ((st = device_info(&sms)) != BL_OK) return st;
  const cudaStream_t s = as_stream(stream);
  Scratch ws(workspace);
  const size_t rank_bytes = static_cast<size_t>(M) * bl::rank_stride(static_cast<int>(r)) * 4;
  float* u = static_cast<float*>(ws.take(rank_bytes));
  float* v = static_cast<float*>(ws.take(rank_bytes));
  const Order order = order_scratch(M, L, &ws);
  const AdapterSet ad = adapter_set(A, B, scale, ids, L, r);
  const bool sorted = dA != nullptr || (M > 16 && L > 1), has_dx = dx && M > 0;
  GiOperands o;
  if (has_dx && (st = gi_operands(dy, dydt, packed, M, N, K, &ws, &o, sms, s)) != BL_OK) return st;
  if ((st = sorted ? launch_sort(ad, M, order, o.pads, sms, s) : run_pads(o.pads, sms, s)) != BL_OK) return st;
  if (M > 0 && (st = launch_uv(dy, dydt, xq, eta, M, K, N, ad, sorted ? order.rows : nullptr, dA ? u : nullptr, v, s)) !=
                   BL_OK)
    return st;
  if (dA) {  // no tokens: zeros
    if (dydt == BL_F32)
      st = dabdt == BL_F32 ? launch_dab<float, float>(dy, xq, eta, M, K, N, ad, order, u, v, dA, dB, sms, s)
                           : launch_dab<float, __nv_bfloat16>(dy, xq, eta, M, K, N, ad, order, u, v, dA, dB, sms, s);
    else
      st = dabdt == BL_F32 ? launch_dab<__nv_bfloat16, float>(dy, xq, eta, M, K, N, ad, order, u, v, dA, dB, sms, s)
                           : launch_dab<__nv_bfloat16, __nv_bfloat16>(dy, xq, eta, M, K, N, ad, order, u, v, dA, dB, sms, s);
    if (st != BL_OK) return st;
  }
  if (!has_dx) return BL_OK;
  bl::GiArgs g = {};
  g.gamma = gamma; g.M = static_cast<int>(M); g.N = static_cast<int>(N); g.K = static_cast<int>(K); g.dx = dx;
  g.v = v; g.A = ad.A; g.ids = ids; g.L = ad.L; g.r = ad.r;
  return run_grad_input(o, dxdt, g, sms, s);
}

}  // extern "C"
