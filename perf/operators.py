"""The adapter and training operators of the ternary layer as measured cases.

Five operators, each with its plain form (elementary torch operations in
fp32) and the framework's call:

* ``adapters``       y = BitLinear(x) + scale_a (x^ A_a^T) B_a^T, the adapter a
                     chosen per token (serving many requests at once)
* ``adapters_grad``  its backward pass from the 8-bit tokens: dx, dA, dB
* ``grad_input``     dx = gamma dy W~, through the packed ternary weights
* ``grad_weight``    dW = dy^T x^, x^ read back from the 8-bit tokens
* ``rmsnorm_grad``   the normalisation's backward pass from the 8-bit tokens

x^ = x~ eta / 127 are the activations as their int8 codes x~ and absmax eta
hold them; the same codes feed the forward product and are what the forward
pass keeps for the backward pass.
"""
import math

import torch

own = False

OUT = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # one token of one request, the layer's up projection at 3B size
        dict(name="adapters_decode_1", op="adapters", M=1, K=3200, N=8640, r=16, L=8,
             order="mixed", out="bf16"),
        # sixteen requests decoding together, the down projection
        dict(name="adapters_decode_16", op="adapters", M=16, K=8640, N=3200, r=32, L=16,
             order="mixed", out="bf16"),
        # ragged sizes: a few short prompts, rank 5, fp32 results
        dict(name="adapters_ragged_333", op="adapters", M=333, K=1003, N=777, r=5, L=3,
             order="packed", out="f32"),
        # prompts of several requests packed behind one another, 7B size
        dict(name="adapters_prompts_2048", op="adapters", M=2048, K=4096, N=11008, r=16, L=8,
             order="packed", out="bf16"),
        # a small fine-tuning step, examples of four adapters interleaved
        dict(name="adapters_grad_96", op="adapters_grad", M=96, K=3200, N=8640, r=8, L=4,
             order="mixed", out="bf16"),
        # a fine-tuning step of packed examples, 7B size
        dict(name="adapters_grad_2048", op="adapters_grad", M=2048, K=4096, N=11008, r=16, L=4,
             order="packed", out="bf16"),
        # the input gradient of a short example through the down projection
        dict(name="grad_input_77", op="grad_input", M=77, K=8640, N=3200, out="bf16"),
        # the input gradient of a full micro-batch
        dict(name="grad_input_2048", op="grad_input", M=2048, K=4096, N=11008, out="bf16"),
        # the latent weights' gradient, ragged sizes, in the type of its all-reduce
        dict(name="grad_weight_ragged_129", op="grad_weight", M=129, K=1501, N=901, out="bf16"),
        # the latent weights' gradient of a full micro-batch, in the weights' own fp32
        dict(name="grad_weight_2048", op="grad_weight", M=2048, K=4096, N=11008, out="f32"),
        # the normalisation's backward pass of a handful of tokens
        dict(name="rmsnorm_grad_16", op="rmsnorm_grad", M=16, K=3200, out="bf16"),
        # and of a full micro-batch
        dict(name="rmsnorm_grad_2048", op="rmsnorm_grad", M=2048, K=8640, out="bf16"),
    ]


def _between(rng, lo, hi):
    """A size between lo and hi, spread over its logarithm."""
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng):
    """A layer width: every other one a multiple of 64, as model widths are."""
    n = _between(rng, 64, 11008)
    return max(64, n // 64 * 64) if rng.random() < 0.5 else n


def draw(rng):
    op = rng.choice(["adapters", "adapters", "adapters_grad", "grad_input", "grad_weight", "rmsnorm_grad"])
    most = 2048 * 4096 * 11008
    while True:
        case = dict(op=op, M=_between(rng, 1, 4096), K=_width(rng), out=rng.choice(["bf16", "f32"]))
        if op == "rmsnorm_grad":
            return case
        case["N"] = _width(rng)
        if op.startswith("adapters"):
            case |= dict(r=_between(rng, 1, 64), L=_between(rng, 1, 32),
                         order=rng.choice(["packed", "mixed"]))
        if op == "adapters_grad":
            case["out"] = "bf16"
        if case["M"] * case["K"] * case["N"] <= most:
            return case


def _inputs(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def randn(*shape):
        return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)

    M, K, op = case["M"], case["K"], case["op"]
    s = {"op": op, "out": OUT[case["out"]], "K": K}
    x = randn(M, K).to(torch.bfloat16)
    if op == "rmsnorm_grad":
        s["rstd"] = torch.rsqrt(x.float().square().mean(1) + 1e-6)
        n = x.float() * s["rstd"][:, None]
        s["xq"], s["eta"] = _codes(n)
        s["dn"] = (randn(M, K) * 0.01).to(torch.bfloat16)
        return s
    N = s["N"] = case["N"]
    if op == "adapters":
        s["x"] = x
    else:
        s["xq"], s["eta"] = _codes(x.float())
        s["dy"] = (randn(M, N) * 0.01).to(torch.bfloat16)
    if op != "grad_weight":
        # a third of the ternary weights of each value; the codes of the packed bytes
        trits = torch.randint(0, 3, (N, (K + 3) // 4 * 4), generator=g, device="cuda", dtype=torch.int32)
        trits[:, K:] = 1
        t = trits.view(N, -1, 4)
        s["packed"] = (t[..., 0] | t[..., 1] << 2 | t[..., 2] << 4 | t[..., 3] << 6).to(torch.uint8)
        s["gamma"] = 0.01 + 0.01 * torch.rand(1, generator=g, device="cuda")
    if op.startswith("adapters"):
        r, L = case["r"], case["L"]
        s["A"] = (randn(L, r, K) / math.sqrt(K)).to(torch.bfloat16)
        s["B"] = (randn(L, N, r) * 0.1).to(torch.bfloat16)
        s["scale"] = 0.5 + 1.5 * torch.rand(L, generator=g, device="cuda")
        # one token in eight (or request in eight) has no adapter
        ids = torch.randint(0, L, (M,), generator=g, device="cuda", dtype=torch.int32)
        ids[torch.rand(M, generator=g, device="cuda") < 0.125] = -1
        if case["order"] == "packed":  # L + 1 prompts of drawn lengths, one behind the other
            cuts = torch.rand(L, generator=g, device="cuda").sort()[0] * M
            at = torch.arange(M, device="cuda")
            ids = ((at[:, None] >= cuts).sum(1) - 1).to(torch.int32)  # the first has none
        s["ids"] = ids
    return s


def _codes(x):
    """int8 codes and absmax of fp32 rows."""
    eta = x.abs().amax(1).clamp(min=1e-5)
    return (x * 127 / eta[:, None]).round().clamp(-127, 127).to(torch.int8), eta


def prepare(case, seed):
    return _inputs(case, seed)


def run(s):
    return _own(s) if own else PLAIN[s["op"]](s)


def _own(s):
    from ternary_weight_linear_04_b200 import bitlinear as bl

    op = s["op"]
    if op == "adapters":
        return bl.linear_adapters(s["x"], s["packed"], s["gamma"], s["N"], s["A"], s["B"], s["scale"],
                                  s["ids"], out_dtype=s["out"], weights_static=True)
    if op == "adapters_grad":
        return bl.adapters_grad(s["dy"], s["xq"], s["eta"], s["packed"], s["gamma"], s["A"], s["B"],
                                s["scale"], s["ids"])
    if op == "grad_input":
        return bl.grad_input(s["dy"], s["packed"], s["gamma"], s["K"], out_dtype=s["out"])
    if op == "grad_weight":
        return bl.grad_weight(s["dy"], s["xq"], s["eta"], out_dtype=s["out"])
    return bl.rmsnorm_grad(s["dn"], s["xq"], s["eta"], s["rstd"], out_dtype=s["out"])


# ---------------------------------------------------------------- plain forms

def _trits(s):
    """The ternary weights (fp32 N x K) of the packed bytes."""
    p = s["packed"].to(torch.int32)
    codes = torch.stack([p & 3, p >> 2 & 3, p >> 4 & 3, p >> 6], 2).view(p.shape[0], -1)
    return (codes[:, :s["K"]] - 1).to(torch.float32)


def _chosen(s):
    """(M x L r) scale of each token's own adapter, zero elsewhere."""
    L, r, _ = s["A"].shape
    hot = s["ids"][:, None] == torch.arange(L, device=s["ids"].device)
    return (hot * s["scale"]).repeat_interleave(r, 1)


def _flat(s):
    """All adapters side by side: A (L r x K), B (N x L r)."""
    L, r, K = s["A"].shape
    return s["A"].float().view(L * r, K), s["B"].float().transpose(0, 1).reshape(-1, L * r)


def _plain_adapters(s):
    xq, eta = _codes(s["x"].float())
    A, B = _flat(s)
    y = (xq.float() @ _trits(s).t()) * (eta * s["gamma"] / 127)[:, None]
    u = (xq.float() * (eta / 127)[:, None]) @ A.t() * _chosen(s)
    return (y + u @ B.t()).to(s["out"])


def _plain_adapters_grad(s):
    L, r, K = s["A"].shape
    A, B = _flat(s)
    dy, c = s["dy"].float(), _chosen(s)
    xh = s["xq"].float() * (s["eta"] / 127)[:, None]
    u, v = xh @ A.t() * c, dy @ B * c
    dx = dy @ _trits(s) * s["gamma"] + v @ A
    dB = (dy.t() @ u).view(-1, L, r).transpose(0, 1).contiguous()
    return dx.to(torch.bfloat16), (v.t() @ xh).view(L, r, K).to(torch.bfloat16), dB.to(torch.bfloat16)


def _plain_grad_input(s):
    return (s["dy"].float() @ _trits(s) * s["gamma"]).to(s["out"])


def _plain_grad_weight(s):
    return (s["dy"].float().t() @ (s["xq"].float() * (s["eta"] / 127)[:, None])).to(s["out"])


def _plain_rmsnorm_grad(s):
    n = s["xq"].float() * (s["eta"] / 127)[:, None]
    dn = s["dn"].float()
    return ((dn - n * (n * dn).mean(1, keepdim=True)) * s["rstd"][:, None]).to(s["out"])


PLAIN = {"adapters": _plain_adapters, "adapters_grad": _plain_adapters_grad,
         "grad_input": _plain_grad_input, "grad_weight": _plain_grad_weight,
         "rmsnorm_grad": _plain_rmsnorm_grad}


# ---------------------------------------------------------------- 64 bits

def exact(case, seed):
    s = _inputs(case, seed)
    f8 = torch.float64
    K, op = case["K"], case["op"]
    if op == "adapters":
        # the codes' definition is in fp32: round half even of fl(fl(127 x) / eta)
        x = s["x"].float()
        eta32 = x.abs().max(dim=1).values.clamp_min(1e-5)
        xq = torch.round(x.mul(127.0).div(eta32.unsqueeze(1))).clamp(-127, 127).to(f8)
        eta = eta32.to(f8)
    else:
        xq, eta = s["xq"].to(f8), s["eta"].to(f8)
    xh = xq * eta.div(127).unsqueeze(1)
    if op == "rmsnorm_grad":
        dn = s["dn"].to(f8)
        proj = torch.einsum("mk,mk->m", xh, dn) / K
        return s["rstd"].to(f8).unsqueeze(1) * (dn - proj.unsqueeze(1) * xh)
    if op == "grad_weight":
        return torch.einsum("mn,mk->nk", s["dy"].to(f8), xh)
    W = torch.empty(case["N"], s["packed"].shape[1] * 4, dtype=f8, device="cuda")
    for j in range(4):
        W[:, j::4] = ((s["packed"] >> (2 * j)) & 3).to(f8) - 1
    W = W[:, :K] * s["gamma"].to(f8)
    if op == "grad_input":
        return torch.einsum("mn,nk->mk", s["dy"].to(f8), W)
    A, B, scale = s["A"].to(f8), s["B"].to(f8), s["scale"].to(f8)
    if op == "adapters":
        y = torch.einsum("mk,nk->mn", xh, W)
        for a in range(case["L"]):  # each adapter on its own tokens
            of = (s["ids"] == a).nonzero().squeeze(1)
            y[of] += scale[a] * (xh[of] @ A[a].t()) @ B[a].t()
        return y
    dy = s["dy"].to(f8)
    dx = torch.einsum("mn,nk->mk", dy, W)
    dA, dB = torch.zeros_like(A), torch.zeros_like(B)
    for a in range(case["L"]):
        of = (s["ids"] == a).nonzero().squeeze(1)
        v = scale[a] * dy[of] @ B[a]
        dx[of] += v @ A[a]
        dA[a] = v.t() @ xh[of]
        dB[a] = scale[a] * dy[of].t() @ (xh[of] @ A[a].t())
    return dx, dA, dB


def work(case):
    M, K, op = case["M"], case["K"], case["op"]
    wide = 2 if case["out"] == "bf16" else 4
    if op == "rmsnorm_grad":
        return {"bytes": M * (K * (2 + 1 + wide) + 8), "flops": 7 * M * K}
    N = case["N"]
    packed = N * ((K + 3) // 4) + 4
    if op == "grad_input":
        return {"bytes": 2 * M * N + packed + wide * M * K, "flops": 2 * M * N * K}
    if op == "grad_weight":
        return {"bytes": 2 * M * N + M * (K + 4) + wide * N * K, "flops": 2 * M * N * K}
    r, L = case["r"], case["L"]
    pairs = 2 * min(L, M) * r * (K + N)  # the adapters in use, bf16
    if op == "adapters":
        return {"bytes": 2 * M * K + packed + pairs + 4 * (M + L) + wide * M * N,
                "flops": 2 * M * N * K + 2 * M * r * (K + N)}
    return {"bytes": 2 * M * N + M * (K + 4) + packed + pairs + 4 * (M + L) + 2 * M * K + 2 * L * r * (K + N),
            "flops": 2 * M * N * K + 2 * M * r * (3 * K + 2 * N)}
