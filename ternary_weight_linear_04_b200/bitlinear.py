"""Python binding of the BitLinear C ABI (``include/bitlinear.h``).

Argument marshalling only: torch supplies device memory and the current
CUDA stream; every step of the layer runs in the library's CUDA kernels.
Names follow the C entry points: ``pack_weights``, ``quant_act``,
``forward`` (plus ``BitLinear``, a small holder of one packed matrix).
"""
import contextlib
import ctypes
import functools

import torch

from . import _lib
from ._lib import check

PATHS = {"auto": _lib.BL_PATH_AUTO, "gemv": _lib.BL_PATH_GEMV,
         "tcgen05": _lib.BL_PATH_TCGEN05, "generic": _lib.BL_PATH_GENERIC}
PATH_NAMES = {v: k for k, v in PATHS.items()}
_DTYPES = {torch.float32: _lib.BL_F32, torch.bfloat16: _lib.BL_BF16}


def _stream(stream):
    # the raw handle: building a Stream object costs as much as a launch
    return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device()) if stream is None else stream.cuda_stream


def _ptr(t):
    return t.data_ptr() if t is not None else None


def _require_cuda(*ts):
    for t in ts:
        if t is not None and (not t.is_cuda or not t.is_contiguous()):
            raise ValueError("tensors must be contiguous CUDA tensors")


def packed_bytes(N, K):
    return int(_lib.lib().bitlinear_packed_bytes(N, K))


def _pack_workspace(workspace, dev):
    """The caller's pack scratch, checked for size, or a new one."""
    need = int(_lib.lib().bitlinear_pack_workspace_bytes())
    if workspace is None:
        return torch.empty(need, dtype=torch.uint8, device=dev)
    _require_cuda(workspace)
    if workspace.numel() * workspace.element_size() < need or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous buffer of at least %d bytes" % need)
    return workspace


def pack_weights(W, stream=None, workspace=None, packed=None, gamma=None):
    """fp32 latent weights (N x K, CUDA) -> (packed uint8 N x ceil(K/4), gamma fp32[1])."""
    _require_cuda(W)
    if W.dtype != torch.float32 or W.dim() != 2:
        raise ValueError("W must be a 2-D float32 tensor")
    N, K = W.shape
    L = _lib.lib()
    dev = W.device
    if packed is None:
        packed = torch.empty((N, (K + 3) // 4), dtype=torch.uint8, device=dev)
    if gamma is None:
        gamma = torch.empty(1, dtype=torch.float32, device=dev)
    workspace = _pack_workspace(workspace, dev)
    check(L.bitlinear_pack_weights(_ptr(W), N, K, _ptr(packed), _ptr(gamma), _ptr(workspace),
                                   _stream(stream)), "bitlinear_pack_weights")
    return packed, gamma


def absmean_buckets(W, stream=None, out=None):
    """Exact |W| exponent buckets of a row shard (fp32 N x K, CUDA) -> int64[256]
    (uint64 totals in two's complement; sum them over shards with an int64
    all-reduce)."""
    _require_cuda(W)
    if W.dtype != torch.float32 or W.dim() != 2:
        raise ValueError("W must be a 2-D float32 tensor")
    N, K = W.shape
    b = out if out is not None else torch.empty(256, dtype=torch.int64, device=W.device)
    check(_lib.lib().bitlinear_absmean_buckets(_ptr(W), N, K, _ptr(b), _stream(stream)),
          "bitlinear_absmean_buckets")
    return b


def gamma_from_buckets(buckets, count, stream=None, out=None):
    """gamma (fp32[1]) from bucket totals of a whole matrix of `count` elements."""
    _require_cuda(buckets)
    if buckets.dtype != torch.int64 or buckets.numel() != 256:
        raise ValueError("buckets must be 256 int64 values")
    g = out if out is not None else torch.empty(1, dtype=torch.float32, device=buckets.device)
    check(_lib.lib().bitlinear_gamma_from_buckets(_ptr(buckets), int(count), _ptr(g),
                                                  _stream(stream)), "bitlinear_gamma_from_buckets")
    return g


def ternarise_pack(W, gamma, stream=None, out=None):
    """Rows of W (fp32 N x K, CUDA) ternarised with a given gamma and packed
    (uint8 N x ceil(K/4))."""
    _require_cuda(W, gamma)
    if W.dtype != torch.float32 or W.dim() != 2:
        raise ValueError("W must be a 2-D float32 tensor")
    N, K = W.shape
    p = out if out is not None else torch.empty((N, (K + 3) // 4), dtype=torch.uint8,
                                                 device=W.device)
    check(_lib.lib().bitlinear_ternarise_pack(_ptr(W), N, K, _ptr(gamma), _ptr(p), _stream(stream)),
          "bitlinear_ternarise_pack")
    return p


def quant_act(x, stream=None, out=None):
    """Activations (M x K, fp32 or bf16, CUDA) -> (xq int8 M x K, eta fp32 M, xsum int32 M)."""
    _require_cuda(x)
    if x.dim() != 2 or x.dtype not in _DTYPES:
        raise ValueError("x must be a 2-D float32 or bfloat16 tensor")
    M, K = x.shape
    dev = x.device
    if out is None:
        out = (torch.empty((M, K), dtype=torch.int8, device=dev),
               torch.empty(M, dtype=torch.float32, device=dev),
               torch.empty(M, dtype=torch.int32, device=dev))
    xq, eta, xsum = out
    check(_lib.lib().bitlinear_quant_act(_ptr(x), _DTYPES[x.dtype], M, K, _ptr(xq), _ptr(eta),
                                         _ptr(xsum), _stream(stream)), "bitlinear_quant_act")
    return xq, eta, xsum


def rmsnorm_quant_act(x, stream=None, out=None, want_rstd=False):
    """RMSNorm (no affine, eps 1e-6) fused with the per-token quantiser.
    Activations (M x K, bf16, CUDA) -> (xq int8 M x K, eta fp32 M, xsum int32 M)
    of the normalised rows; with want_rstd also rstd (fp32 M), the factor each
    row was multiplied by (what rmsnorm_grad needs)."""
    if x.dim() != 2 or x.dtype != torch.bfloat16:
        raise ValueError("x must be a 2-D bfloat16 tensor")
    M, K = x.shape
    dev = x.device
    with _place(stream, x):
        if out is None:
            out = (torch.empty((M, K), dtype=torch.int8, device=dev),
                   torch.empty(M, dtype=torch.float32, device=dev),
                   torch.empty(M, dtype=torch.int32, device=dev))
        xq, eta, xsum = out
        if want_rstd:
            rstd = torch.empty(M, dtype=torch.float32, device=dev)
            check(_lib.lib().bitlinear_rmsnorm_quant_act_rstd(
                _ptr(x), _DTYPES[x.dtype], M, K, _ptr(xq), _ptr(eta), _ptr(xsum), _ptr(rstd),
                _stream_of(x)), "bitlinear_rmsnorm_quant_act_rstd")
            return xq, eta, xsum, rstd
        check(_lib.lib().bitlinear_rmsnorm_quant_act(_ptr(x), _DTYPES[x.dtype], M, K, _ptr(xq),
                                                     _ptr(eta), _ptr(xsum), _stream_of(x)),
              "bitlinear_rmsnorm_quant_act")
    return xq, eta, xsum


def forward(xq, eta, xsum, packed, gamma, N, out_dtype=torch.bfloat16, want_int=False,
            path="auto", stream=None, out=None, out_int=None, weights_static=False):
    """Integer accumulation + rescale.  Returns y (M x N), or (y, y_int) if want_int.
    weights_static: packed/gamma are not written by pending work on the stream
    (lets the decode kernel start streaming them early)."""
    _require_cuda(xq, eta, xsum, packed, gamma)
    M, K = xq.shape
    if packed.shape != (N, (K + 3) // 4):
        raise ValueError("packed shape %s does not match N=%d, K=%d" % (tuple(packed.shape), N, K))
    dev = xq.device
    y = out if out is not None else torch.empty((M, N), dtype=out_dtype, device=dev)
    y_int = out_int
    if want_int and y_int is None:
        y_int = torch.empty((M, N), dtype=torch.int32, device=dev)
    check(_lib.lib().bitlinear_forward_path(
        _ptr(xq), _ptr(eta), _ptr(xsum), M, K, _ptr(packed), _ptr(gamma), N, _ptr(y),
        _DTYPES[y.dtype], _ptr(y_int), PATHS[path],
        _lib.BL_FLAG_WEIGHTS_STATIC if weights_static else 0, _stream(stream)), "bitlinear_forward")
    return (y, y_int) if want_int else y


def fused_decode_ok(M, K):
    """Whether bitlinear_linear runs its single fused decode kernel for (M, K)
    with bf16 activations: one or two tokens (the same rule as the library;
    otherwise it needs x~ scratch)."""
    mt = 1 if M <= 1 else 2
    return 1 <= M <= 2 and K >= 64 and K % 64 == 0 and K * mt <= 131072


DECODE_SHAPE_FIELDS = ("team_warps", "rows_per_block", "teams", "words_per_lane", "rows_per_cta",
                       "ctas", "blocks_per_stage", "stages", "x_staged", "smem_bytes")


def decode_shape(M, K, N, fused=True):
    """The decode kernel's launch shape for (M, K, N) on the current device,
    as a dict (see bitlinear_decode_shape)."""
    buf = (ctypes.c_int32 * len(DECODE_SHAPE_FIELDS))()
    check(_lib.lib().bitlinear_decode_shape(M, K, N, 1 if fused else 0, buf), "bitlinear_decode_shape")
    return dict(zip(DECODE_SHAPE_FIELDS, list(buf)))


def decode_reg_shape(K, N, sms=None):
    """Shape of the one-token register-resident kernel of bitlinear_linear for
    (K, N) as a dict, or None when that kernel does not take the layer.  sms
    defaults to the current device's SM count."""
    if sms is None:
        sms = torch.cuda.get_device_properties(torch.cuda.current_device()).multi_processor_count
    buf = (ctypes.c_int32 * 4)()
    st = _lib.lib().bitlinear_decode_reg_shape(K, N, sms, buf)
    if st == _lib.BL_ERR_UNSUPPORTED:
        return None
    check(st, "bitlinear_decode_reg_shape")
    return dict(zip(("rows_per_warp", "words_per_lane", "rows_per_cta", "ctas"), list(buf)))


def decode_regm_shape(M, K, N, sms=None):
    """Shape of the register-resident kernel for 2..8 tokens with x~ given,
    as a dict, or None when that kernel does not take (M, K, N).  sms
    defaults to the current device's SM count."""
    if sms is None:
        sms = torch.cuda.get_device_properties(torch.cuda.current_device()).multi_processor_count
    buf = (ctypes.c_int32 * 5)()
    st = _lib.lib().bitlinear_decode_regm_shape(M, K, N, sms, buf)
    if st == _lib.BL_ERR_UNSUPPORTED:
        return None
    check(st, "bitlinear_decode_regm_shape")
    return dict(zip(("token_slots", "rows_per_warp", "words_per_lane", "rows_per_cta", "ctas"), list(buf)))


def decode_mma_shape(M, K, N, sms=None):
    """Shape of the warp-MMA decode kernel for 9..16 tokens with x~ given, as
    a dict, or None when that kernel does not take (M, K, N).  sms defaults
    to the current device's SM count."""
    if sms is None:
        sms = torch.cuda.get_device_properties(torch.cuda.current_device()).multi_processor_count
    buf = (ctypes.c_int32 * 7)()
    st = _lib.lib().bitlinear_decode_mma_shape(M, K, N, sms, buf)
    if st == _lib.BL_ERR_UNSUPPORTED:
        return None
    check(st, "bitlinear_decode_mma_shape")
    return dict(zip(("token_slots", "row_blocks", "k_parts", "k_steps", "rows_per_cta", "ctas",
                     "smem_bytes"), list(buf)))


def set_decode_mma(enable=True):
    """Turn the warp-MMA decode kernel on (default) or off for later launches
    in this process."""
    check(_lib.lib().bitlinear_set_decode_mma(1 if enable else 0), "bitlinear_set_decode_mma")


def set_decode_reg(enable=True):
    """Turn the register-resident kernels (one token fused; 2..8 tokens with
    x~ given) on (default) or off for later launches in this process (off:
    the shared-memory decode kernel)."""
    check(_lib.lib().bitlinear_set_decode_reg(1 if enable else 0), "bitlinear_set_decode_reg")


def set_tc_split(k_split=0):
    """Force the K split (CTAs per cluster) of the tensor-core kernel for later
    launches in this process (0 = the library's choice)."""
    check(_lib.lib().bitlinear_set_tc_split(k_split), "bitlinear_set_tc_split")


def set_decode_shape(team_warps=0, rows_per_block=0):
    """Force the decode kernel's team width and row-block height for later
    launches in this process (0 = the library's choice)."""
    check(_lib.lib().bitlinear_set_decode_shape(team_warps, rows_per_block), "bitlinear_set_decode_shape")


def linear(x, packed, gamma, N, out_dtype=torch.bfloat16, want_quant=False, want_int=False,
           weights_static=False, stream=None, out=None, scratch=None):
    """The whole per-token layer (quantise + accumulate + rescale) in one call.
    Returns y, plus (xq, eta, xsum) if want_quant and y_int if want_int."""
    _require_cuda(x, packed, gamma)
    if x.dim() != 2 or x.dtype not in _DTYPES:
        raise ValueError("x must be a 2-D float32 or bfloat16 tensor")
    M, K = x.shape
    if packed.shape != (N, (K + 3) // 4):
        raise ValueError("packed shape %s does not match N=%d, K=%d" % (tuple(packed.shape), N, K))
    dev = x.device
    y = out if out is not None else torch.empty((M, N), dtype=out_dtype, device=dev)
    decode = fused_decode_ok(M, K) and x.dtype == torch.bfloat16
    if scratch is not None:
        xq, eta, xsum = scratch
    elif want_quant or not decode:
        xq = torch.empty((M, K), dtype=torch.int8, device=dev)
        eta = torch.empty(M, dtype=torch.float32, device=dev)
        xsum = torch.empty(M, dtype=torch.int32, device=dev)
    else:
        xq = eta = xsum = None
    y_int = torch.empty((M, N), dtype=torch.int32, device=dev) if want_int else None
    check(_lib.lib().bitlinear_linear(
        _ptr(x), _DTYPES[x.dtype], M, K, _ptr(packed), _ptr(gamma), N, _ptr(y), _DTYPES[y.dtype],
        _ptr(xq), _ptr(eta), _ptr(xsum), _ptr(y_int),
        _lib.BL_FLAG_WEIGHTS_STATIC if weights_static else 0, _stream(stream)), "bitlinear_linear")
    out_ = (y,)
    if want_quant:
        out_ += ((xq, eta, xsum),)
    if want_int:
        out_ += (y_int,)
    return out_[0] if len(out_) == 1 else out_


def linear_group(x, packed, gamma, out_dtype=torch.bfloat16, weights_static=False, stream=None,
                 out=None):
    """bitlinear_linear_group: the per-token layer for up to 4 matrices that
    share the activations x (bf16 M x K, M <= 4), in one launch.  packed and
    gamma are lists (one per matrix); returns the list of outputs."""
    _require_cuda(x, *packed, *gamma)
    if x.dim() != 2 or x.dtype != torch.bfloat16:
        raise ValueError("x must be a 2-D bfloat16 tensor")
    M, K = x.shape
    n = len(packed)
    if n != len(gamma) or not 1 <= n <= 4:
        raise ValueError("one gamma per packed matrix, 1 to 4 matrices")
    Ns = [p.shape[0] for p in packed]
    for p in packed:
        if p.shape[1] != (K + 3) // 4:
            raise ValueError("packed shape %s does not match K=%d" % (tuple(p.shape), K))
    ys = out if out is not None else [torch.empty((M, N), dtype=out_dtype, device=x.device) for N in Ns]
    arr = ctypes.c_void_p * n
    check(_lib.lib().bitlinear_linear_group(
        _ptr(x), _lib.BL_BF16, M, K, n, arr(*[_ptr(p) for p in packed]), arr(*[_ptr(g) for g in gamma]),
        (ctypes.c_int64 * n)(*Ns), arr(*[_ptr(y) for y in ys]), _DTYPES[ys[0].dtype],
        _lib.BL_FLAG_WEIGHTS_STATIC if weights_static else 0, _stream(stream)), "bitlinear_linear_group")
    return ys


def packed3_stride(K):
    """Row stride (bytes) of the base-3 layout."""
    return int(_lib.lib().bitlinear_packed3_stride(K))


def pack_weights3(W, stream=None, workspace=None):
    """bitlinear_pack_weights3: (packed3 N x stride uint8, gamma) on W's device."""
    _require_cuda(W)
    N, K = W.shape
    dev = W.device
    packed3 = torch.empty((N, packed3_stride(K)), dtype=torch.uint8, device=dev)
    gamma = torch.empty(1, dtype=torch.float32, device=dev)
    ws = _pack_workspace(workspace, dev)
    check(_lib.lib().bitlinear_pack_weights3(_ptr(W), N, K, _ptr(packed3), _ptr(gamma), _ptr(ws),
                                             _stream(stream)), "bitlinear_pack_weights3")
    return packed3, gamma


def forward3(xq, eta, xsum, packed3, gamma, N, out_dtype=torch.float32, want_int=False,
             stream=None, out=None):
    """bitlinear_forward3: the accumulate + rescale on base-3 packed weights."""
    _require_cuda(xq, eta, xsum, packed3, gamma)
    M, K = xq.shape
    if packed3.shape != (N, packed3_stride(K)):
        raise ValueError("packed3 shape %s does not match N=%d, K=%d" % (tuple(packed3.shape), N, K))
    y = out if out is not None else torch.empty((M, N), dtype=out_dtype, device=xq.device)
    y_int = torch.empty((M, N), dtype=torch.int32, device=xq.device) if want_int else None
    check(_lib.lib().bitlinear_forward3(_ptr(xq), _ptr(eta), _ptr(xsum), M, K, _ptr(packed3), _ptr(gamma),
                                        N, _ptr(y), _DTYPES[y.dtype], _ptr(y_int), _stream(stream)),
          "bitlinear_forward3")
    return (y, y_int) if want_int else y


# ------------------------------------------------------------ backward pass, adapters

_HERE = contextlib.nullcontext()


def _place(stream, *ts):
    """A context that makes the tensors' device, and `stream` where one is
    given, the current ones, so that scratch and outputs belong to the stream
    that the kernels run on.  All tensors have to be on one CUDA device (and
    the stream on it) and contiguous."""
    index = -1
    for t in ts:
        if t is None:
            continue
        at = t.get_device()  # -1: not a CUDA tensor
        if at < 0 or not t.is_contiguous():
            raise ValueError("tensors must be contiguous CUDA tensors")
        if at != index:
            if index >= 0:
                raise ValueError("tensors must be on one device")
            index = at
    if stream is not None:
        if stream.device.index != index:
            raise ValueError("stream must be on the tensors' device")
        return torch.cuda.stream(stream)
    return _HERE if index == torch.cuda.current_device() else torch.cuda.device(index)


def _stream_of(t):
    """The current stream of the tensor's device (which _place made current)."""
    return torch._C._cuda_getCurrentRawStream(t.get_device())


def _al16(t):
    """The tensor itself, or a copy where its data does not start on 16 bytes
    (a slice of a ragged tensor)."""
    return t if t is None or t.data_ptr() % 16 == 0 else t.clone()


def _check(name, t, shape, *dtypes):
    if t.shape != shape or t.dtype not in dtypes:
        raise ValueError("%s must be %s of shape %s, not %s of %s" % (
            name, " or ".join(str(d).replace("torch.", "") for d in dtypes), tuple(shape),
            str(t.dtype).replace("torch.", ""), tuple(t.shape)))


def _out(out, shape, dtype, like, name="out"):
    """The caller's output, checked, or a new one on the device of `like`."""
    if dtype not in _DTYPES:
        raise ValueError("%s must be float32 or bfloat16" % name)
    if out is None:
        return like.new_empty(shape) if dtype is like.dtype else like.new_empty(shape, dtype=dtype)
    _check(name, out, shape, *_DTYPES)
    if not out.is_cuda or out.device != like.device or not out.is_contiguous() or out.data_ptr() % 16:
        raise ValueError("%s must be contiguous, on the inputs' device and 16-byte aligned" % name)
    return out


def _scratch(nbytes, like):
    return like.new_empty((nbytes,), dtype=torch.uint8) if nbytes else None


@functools.lru_cache(maxsize=4096)
def _ws_bytes(call, *sizes):
    """bitlinear_<call>_workspace_bytes(*sizes), a function of the sizes alone."""
    return getattr(_lib.lib(), "bitlinear_%s_workspace_bytes" % call)(*sizes)


def _codes(xq, eta, M):
    if xq.dtype is torch.int8 and eta.dtype is torch.float32 and eta.shape == (M,) and xq.dim() == 2 and xq.shape[0] == M:
        return
    if xq.dim() != 2 or xq.shape[0] != M:
        raise ValueError("xq must be int8 with %d rows" % M)
    _check("xq", xq, xq.shape, torch.int8)
    _check("eta", eta, (M,), torch.float32)


def _packed(packed, gamma, N, K):
    if (packed.dtype is torch.uint8 and gamma.dtype is torch.float32 and packed.shape == (N, (K + 3) // 4)
            and gamma.shape == (1,)):
        return
    _check("packed", packed, (N, (K + 3) // 4), torch.uint8)
    _check("gamma", gamma, (1,), torch.float32)


def _adapters(A, B, scale, ids, M, N, K):
    """(L, r) of an adapter set whose shapes fit."""
    if A.dim() != 3 or B.dim() != 3:
        raise ValueError("A must be L x r x K and B L x N x r")
    L, r, k = A.shape
    if (A.dtype is torch.bfloat16 and B.dtype is torch.bfloat16 and scale.dtype is torch.float32
            and ids.dtype is torch.int32 and k == K and B.shape == (L, N, r) and scale.shape == (L,) and ids.shape == (M,)):
        return L, r
    _check("A", A, (L, r, K), torch.bfloat16)
    _check("B", B, (L, N, r), torch.bfloat16)
    _check("scale", scale, (L,), torch.float32)
    _check("ids", ids, (M,), torch.int32)
    return L, r


def grad_input(dy, packed, gamma, K, out_dtype=torch.bfloat16, stream=None, out=None):
    """Input gradient dx = gamma (dy W~) (M x K) of the layer's output gradient
    dy (M x N, fp32 or bf16), through the packed weights."""
    if dy.dim() != 2 or dy.dtype not in _DTYPES:
        raise ValueError("dy must be a 2-D float32 or bfloat16 tensor")
    M, N = dy.shape
    _packed(packed, gamma, N, K)
    with _place(stream, dy, packed, gamma):
        dx = _out(out, (M, K), out_dtype, dy)
        L = _lib.lib()
        dt = _DTYPES[dy.dtype]
        nws = _ws_bytes("grad_input", M, N, K, dt)
        ws = _scratch(nws, dy)
        dy, packed = _al16(dy), _al16(packed)
        check(L.bitlinear_grad_input(_ptr(dy), dt, M, N, _ptr(packed), _ptr(gamma), K, _ptr(dx),
                                     _DTYPES[dx.dtype], _ptr(ws), nws, _stream_of(dy)), "bitlinear_grad_input")
    return dx


def grad_weight(dy, xq, eta, out_dtype=torch.float32, stream=None, out=None):
    """Gradient of the latent weights dW = dy^T (x~ eta / 127) (N x K) from the
    8-bit tokens that the forward pass kept."""
    if dy.dim() != 2 or dy.dtype not in _DTYPES:
        raise ValueError("dy must be a 2-D float32 or bfloat16 tensor")
    M, N = dy.shape
    _codes(xq, eta, M)
    K = xq.shape[1]
    with _place(stream, dy, xq, eta):
        dw = _out(out, (N, K), out_dtype, dy)
        L = _lib.lib()
        dt, wt = _DTYPES[dy.dtype], _DTYPES[dw.dtype]
        nws = _ws_bytes("grad_weight", M, N, K, dt, wt)
        ws = _scratch(nws, dy)
        dy, xq = _al16(dy), _al16(xq)
        check(L.bitlinear_grad_weight(_ptr(dy), dt, _ptr(xq), _ptr(eta), M, N, K, _ptr(dw), wt, _ptr(ws), nws,
                                      _stream_of(dy)), "bitlinear_grad_weight")
    return dw


def rmsnorm_grad(dn, xq, eta, rstd, out_dtype=torch.bfloat16, stream=None, out=None):
    """Input gradient of the RMSNorm from the 8-bit tokens: dn (M x K, fp32 or
    bf16) is the gradient of the normalised rows, xq, eta and rstd as
    rmsnorm_quant_act(want_rstd=True) returned them."""
    if dn.dim() != 2 or dn.dtype not in _DTYPES:
        raise ValueError("dn must be a 2-D float32 or bfloat16 tensor")
    M, K = dn.shape
    _codes(xq, eta, M)
    _check("xq", xq, (M, K), torch.int8)
    _check("rstd", rstd, (M,), torch.float32)
    with _place(stream, dn, xq, eta, rstd):
        dx = _out(out, (M, K), out_dtype, dn)
        check(_lib.lib().bitlinear_rmsnorm_grad(_ptr(dn), _DTYPES[dn.dtype], _ptr(xq), _ptr(eta), _ptr(rstd),
                                                M, K, _ptr(dx), _DTYPES[dx.dtype], _stream_of(dn)),
              "bitlinear_rmsnorm_grad")
    return dx


def forward_adapters(xq, eta, xsum, packed, gamma, N, A, B, scale, ids, out_dtype=torch.bfloat16,
                     weights_static=False, stream=None, out=None):
    """The projection plus each token's own low-rank adapter, from the 8-bit
    tokens: y = x^ W^T + scale_a (x^ A_a^T) B_a^T with a = ids[m] (none where
    ids[m] is outside [0, L)).  A bf16 L x r x K, B bf16 L x N x r, scale fp32
    L, ids int32 M."""
    if xq.dim() != 2:
        raise ValueError("xq must be 2-D")
    M, K = xq.shape
    _codes(xq, eta, M)
    _check("xsum", xsum, (M,), torch.int32)
    _packed(packed, gamma, N, K)
    n_ad, r = _adapters(A, B, scale, ids, M, N, K)
    with _place(stream, xq, eta, xsum, packed, gamma, A, B, scale, ids):
        y = _out(out, (M, N), out_dtype, xq)
        L = _lib.lib()
        nws = _ws_bytes("forward_adapters", M, K, N, n_ad, r)
        ws = _scratch(nws, xq)
        xq, packed, A, B = _al16(xq), _al16(packed), _al16(A), _al16(B)
        check(L.bitlinear_forward_adapters(
            _ptr(xq), _ptr(eta), _ptr(xsum), M, K, _ptr(packed), _ptr(gamma), N, _ptr(A), _ptr(B),
            _ptr(scale), _ptr(ids), n_ad, r, _ptr(y), _DTYPES[y.dtype], _ptr(ws), nws,
            _lib.BL_FLAG_WEIGHTS_STATIC if weights_static else 0, _stream_of(xq)), "bitlinear_forward_adapters")
    return y


def linear_adapters(x, packed, gamma, N, A, B, scale, ids, out_dtype=torch.bfloat16, rmsnorm=False,
                    weights_static=False, stream=None, out=None):
    """forward_adapters on tokens it quantises itself: x (M x K, fp32 or bf16),
    RMS-normalised first with rmsnorm (bf16)."""
    if x.dim() != 2 or x.dtype not in _DTYPES:
        raise ValueError("x must be a 2-D float32 or bfloat16 tensor")
    M, K = x.shape
    _packed(packed, gamma, N, K)
    n_ad, r = _adapters(A, B, scale, ids, M, N, K)
    with _place(stream, x, packed, gamma, A, B, scale, ids):
        y = _out(out, (M, N), out_dtype, x)
        L = _lib.lib()
        nws = _ws_bytes("linear_adapters", M, K, N, n_ad, r)
        ws = _scratch(nws, x)
        packed, A, B = _al16(packed), _al16(A), _al16(B)
        flags = (_lib.BL_FLAG_WEIGHTS_STATIC if weights_static else 0) | (_lib.BL_FLAG_RMSNORM if rmsnorm else 0)
        check(L.bitlinear_linear_adapters(
            _ptr(x), _DTYPES[x.dtype], M, K, _ptr(packed), _ptr(gamma), N, _ptr(A), _ptr(B), _ptr(scale), _ptr(ids),
            n_ad, r, _ptr(y), _DTYPES[y.dtype], _ptr(ws), nws, flags, _stream_of(x)), "bitlinear_linear_adapters")
    return y


def adapters_grad(dy, xq, eta, packed, gamma, A, B, scale, ids, out_dtype=torch.bfloat16,
                  grad_dtype=torch.bfloat16, want_dx=True, want_dab=True, stream=None):
    """Backward pass of forward_adapters from the 8-bit tokens, the projection
    frozen: (dx, dA, dB).  dx has out_dtype, dA and dB grad_dtype; what is not
    wanted is None (packed and gamma may be None without dx)."""
    if dy.dim() != 2 or dy.dtype not in _DTYPES:
        raise ValueError("dy must be a 2-D float32 or bfloat16 tensor")
    if not (want_dx or want_dab):
        raise ValueError("nothing is wanted")
    M, N = dy.shape
    _codes(xq, eta, M)
    K = xq.shape[1]
    if want_dx:
        _packed(packed, gamma, N, K)
    n_ad, r = _adapters(A, B, scale, ids, M, N, K)
    with _place(stream, dy, xq, eta, packed, gamma, A, B, scale, ids):
        dx = _out(None, (M, K), out_dtype, dy) if want_dx else None
        dA = _out(None, A.shape, grad_dtype, dy) if want_dab else None
        dB = _out(None, B.shape, grad_dtype, dy) if want_dab else None
        L = _lib.lib()
        dt = _DTYPES[dy.dtype]
        nws = _ws_bytes("adapters_grad", M, N, K, n_ad, r, dt)
        ws = _scratch(nws, dy)
        dy, xq, packed, A, B = _al16(dy), _al16(xq), _al16(packed), _al16(A), _al16(B)
        check(L.bitlinear_adapters_grad(
            _ptr(dy), dt, _ptr(xq), _ptr(eta), M, N, K, _ptr(packed), _ptr(gamma), _ptr(A), _ptr(B),
            _ptr(scale), _ptr(ids), n_ad, r, _ptr(dx), _DTYPES[out_dtype], _ptr(dA), _ptr(dB),
            _DTYPES[grad_dtype], _ptr(ws), nws, _stream_of(dy)), "bitlinear_adapters_grad")
    return dx, dA, dB


def tile_tokens(M, K, N, grad=False, sms=None):
    """Tokens of a tile of the projection with adapters (more than 16 tokens),
    or with grad of the input gradient (see bitlinear_tile_tokens).  sms
    defaults to the current device's SM count."""
    if sms is None:
        sms = torch.cuda.get_device_properties(torch.cuda.current_device()).multi_processor_count
    return int(_lib.lib().bitlinear_tile_tokens(1 if grad else 0, M, K, N, sms))


def select_path(M, K, N, xq, packed, y, y_int=None):
    return PATH_NAMES[int(_lib.lib().bitlinear_select_path(M, K, N, _ptr(xq), _ptr(packed),
                                                           _ptr(y), _ptr(y_int)))]


def device_error(stream=None):
    code = ctypes.c_int32(0)
    check(_lib.lib().bitlinear_device_error(ctypes.byref(code), _stream(stream)),
          "bitlinear_device_error")
    return int(code.value)


class BitLinear:
    """One packed ternary matrix and its gamma, applied to activations.

    ``BitLinear.from_latent(W)`` packs fp32 latent weights (N x K) once;
    calling the object quantises x (M x K) per token and runs the integer
    accumulate + rescale.  With ``rmsnorm=True`` the tokens are first
    RMS-normalised (no affine weight, eps 1e-6; bf16 x), as BitLinear158.forward
    does in [Production] "2. Absmax Dynamic Activation Quantization"."""

    def __init__(self, packed, gamma, in_features, out_features, rmsnorm=False):
        self.packed, self.gamma = packed, gamma
        self.in_features, self.out_features = in_features, out_features
        self.rmsnorm = rmsnorm

    @classmethod
    def from_latent(cls, W, stream=None, rmsnorm=False):
        packed, gamma = pack_weights(W, stream=stream)
        return cls(packed, gamma, W.shape[1], W.shape[0], rmsnorm=rmsnorm)

    def __call__(self, x, out_dtype=torch.bfloat16, stream=None):
        if self.rmsnorm:
            xq, eta, xsum = rmsnorm_quant_act(x, stream=stream)
            return forward(xq, eta, xsum, self.packed, self.gamma, self.out_features,
                           out_dtype=out_dtype, stream=stream, weights_static=True)
        return linear(x, self.packed, self.gamma, self.out_features, out_dtype=out_dtype,
                      weights_static=True, stream=stream)
