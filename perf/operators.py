"""The 8-bit dense operators beside the experts: cases, their plain forms and their definitions in 64 bits.

Three operators, each reached through ``sparse_moe_rmsnorm_b200.Fp8Ops``:

* ``norm``: RMS norm with the residual's addition; the normalised rows in E4M3 with a scale for each 128 elements.
* ``matmul``: the product of two E4M3 matrices, a scale for each 128 elements of a row of ``a`` and for each 128 x 128
  block of ``b``, with an optional bias and residual.
* ``gated``: both projections of a gated feed-forward block, the activation and the product, the result in E4M3 with
  a scale for each 128 elements (what the block's second product reads).

``own`` is False for the plain form (elementary torch operations in 32 bits) and True for the framework's kernels.
"""
import math

import torch

own = False

BLOCK = 128            # elements that share a scale
E4M3_MAX = 448.0
SCALE_MIN = 2.0 ** -126   # the scale of a block of zeros
EPS = 1e-5
# (alpha, limit, shift) of h = min(g, limit) * sigmoid(alpha * min(g, limit)) * (clamp(u, -limit, limit) + shift)
ACTIVATIONS = {"clamped": (1.702, 7.0, 1.0), "silu": (1.0, math.inf, 0.0)}
TYPES = {"bfloat16": torch.bfloat16, "float16": torch.float16, "float32": torch.float32}


def listed():
    return [
        # One decoded token of the 2880-wide model: latency alone counts.
        {"name": "norm, one token", "op": "norm", "T": 1, "d": 2880, "type": "bfloat16", "residual": True},
        # The larger of the two decode batches.
        {"name": "norm, decode batch", "op": "norm", "T": 64, "d": 2880, "type": "bfloat16", "residual": True},
        # The prefill batch.
        {"name": "norm, prefill", "op": "norm", "T": 8192, "d": 2880, "type": "bfloat16", "residual": True},
        # A ragged batch with a residual stream in 32 bits, the last block of a row an eighth full.
        {"name": "norm, ragged, 32 bits", "op": "norm", "T": 1237, "d": 4112, "type": "float32", "residual": True},
        # The query/key/value projection (64 query heads and 2 x 8 key/value heads of 64) of one token.
        {"name": "projection, one token", "op": "matmul", "M": 1, "N": 5120, "K": 2880, "type": "bfloat16", "bias": True, "residual": False},
        # The same for a decode batch.
        {"name": "projection, decode batch", "op": "matmul", "M": 32, "N": 5120, "K": 2880, "type": "bfloat16", "bias": True, "residual": False},
        # The logits of a decode batch over the 201088 tokens of the vocabulary, in 32 bits for the sampler.
        {"name": "logits, decode batch", "op": "matmul", "M": 64, "N": 201088, "K": 2880, "type": "float32", "bias": False, "residual": False},
        # The projection of the prefill batch: the largest product.
        {"name": "projection, prefill", "op": "matmul", "M": 8192, "N": 5120, "K": 2880, "type": "bfloat16", "bias": True, "residual": False},
        # A ragged batch whose rows end inside every tile and block, with the residual's addition, in half precision.
        {"name": "product, ragged", "op": "matmul", "M": 1237, "N": 2885, "K": 4112, "type": "float16", "bias": True, "residual": True},
        # The dense (or shared) expert of one token.
        {"name": "gated, one token", "op": "gated", "M": 1, "F": 2880, "K": 2880, "act": "clamped", "bias": True},
        # ... of the prefill batch.
        {"name": "gated, prefill", "op": "gated", "M": 8192, "F": 2880, "K": 2880, "act": "clamped", "bias": True},
        # A middling ragged batch of a block without biases or clamps.
        {"name": "gated, ragged, silu", "op": "gated", "M": 333, "F": 1360, "K": 1552, "act": "silu", "bias": False},
    ]


def _log(rng, lo, hi):
    return min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))


def draw(rng):
    op = rng.choice(["norm", "matmul", "gated"])
    type_ = rng.choice(["bfloat16", "bfloat16", "float16", "float32"])
    if op == "norm":
        return {"op": op, "T": _log(rng, 1, 8192), "d": 16 * _log(rng, 4, 384), "type": type_, "residual": rng.random() < 0.75}
    M, K = _log(rng, 1, 8192), 16 * _log(rng, 4, 384)
    most = 8192 * 5120 * 2880 // (M * K)      # columns that cost what the largest listed product does
    if op == "matmul":
        N = _log(rng, 16, max(16, min(20000, most)))
        return {"op": op, "M": M, "N": N, "K": K, "type": type_, "bias": rng.random() < 0.5, "residual": rng.random() < 0.5}
    F = 16 * _log(rng, 4, max(4, min(384, most // 32)))
    return {"op": op, "M": M, "F": F, "K": K, "act": rng.choice(["clamped", "silu"]), "bias": rng.random() < 0.5}


def work(case):
    kb = lambda n: -(-n // BLOCK)  # noqa: E731
    if case["op"] == "norm":
        T, d, e = case["T"], case["d"], 4 if case["type"] == "float32" else 2
        streams = 3 if case["residual"] else 1          # x, and with a residual it and the sum
        return {"bytes": T * d * (e * streams + 1) + T * kb(d) * 4 + 2 * d, "flops": 8 * T * d}
    M, K = case["M"], case["K"]
    if case["op"] == "matmul":
        N, e = case["N"], 4 if case["type"] == "float32" else 2
        out = M * N * e * (2 if case["residual"] else 1) + (2 * N if case["bias"] else 0)
        return {"bytes": M * K + N * K + 4 * (M * kb(K) + kb(N) * kb(K)) + out, "flops": 2 * M * N * K}
    F = case["F"]
    out = M * F + 4 * M * kb(F) + (4 * F if case["bias"] else 0)
    return {"bytes": M * K + 2 * F * K + 4 * (M * kb(K) + 2 * kb(F) * kb(K)) + out, "flops": 4 * M * F * K}


# ------------------------------------------------------------------ inputs

def _pad(x, rows, cols):
    return torch.nn.functional.pad(x, (0, -x.shape[1] % cols, 0, -x.shape[0] % rows))


def _quantised(x, rows):
    """x in E4M3 with a scale for each block of `rows` rows x 128 columns: an activation's (1) or a weight's (128)."""
    M, K = x.shape
    b = _pad(x, rows, BLOCK)
    b = b.view(b.shape[0] // rows, rows, b.shape[1] // BLOCK, BLOCK)
    s = (b.abs().amax(dim=(1, 3)) / E4M3_MAX).clamp_min(SCALE_MIN)
    q = (b / s[:, None, :, None]).reshape(b.shape[0] * rows, -1)[:M, :K]
    return q.to(torch.float8_e4m3fn).contiguous(), s.contiguous()


def _activations(M, K, g):
    """Rows as a norm leaves them: unit variance, a few channels that stand out."""
    loud = 1 + 7 * (torch.rand(K, generator=g, device="cuda") < 0.01)
    return _quantised(torch.randn(M, K, generator=g, device="cuda") * loud, 1)


def _weights(N, K, g):
    """Projection weights of variance 1/K, rows of differing size."""
    size = 0.5 + torch.rand(N, 1, generator=g, device="cuda")
    return _quantised(torch.randn(N, K, generator=g, device="cuda").mul_(size / math.sqrt(K)), BLOCK)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    randn = lambda *n: torch.randn(*n, generator=g, device="cuda")  # noqa: E731
    s = {"case": case}
    if case["op"] == "norm":
        T, d, t = case["T"], case["d"], TYPES[case["type"]]
        loud = 1 + 30 * (torch.rand(d, generator=g, device="cuda") < 0.005)
        s["x"] = randn(T, d).to(t)
        s["residual"] = (randn(T, d) * loud).to(t) if case["residual"] else None
        s["weight"] = (1 + 0.3 * randn(d)).to(torch.bfloat16)
        return s
    M, K = case["M"], case["K"]
    s["a"], s["a_scale"] = _activations(M, K, g)
    if case["op"] == "matmul":
        N, t = case["N"], TYPES[case["type"]]
        s["b"], s["b_scale"] = _weights(N, K, g)
        s["bias"] = (0.1 * randn(N)).to(torch.bfloat16) if case["bias"] else None
        s["residual"] = randn(M, N).to(t) if case["residual"] else None
        return s
    F = case["F"]
    gate, linear = _weights(F, K, g), _weights(F, K, g)
    s["w13"] = torch.cat([gate[0].view(torch.uint8), linear[0].view(torch.uint8)]).view(torch.float8_e4m3fn)
    s["w13_scale"] = torch.stack([gate[1], linear[1]])
    s["b13"] = (0.1 * randn(2 * F)).to(torch.bfloat16) if case["bias"] else None
    return s


# ------------------------------------------------- the framework's operators

_ops = None


def _framework():
    """The operators' handle, which a program makes once."""
    global _ops
    if _ops is None:
        import sparse_moe_rmsnorm_b200 as moe
        _ops = moe.Fp8Ops()
    return _ops


def _run_own(s):
    case, ops = s["case"], _framework()
    if case["op"] == "norm":
        return ops.add_rmsnorm(s["x"], s["weight"], residual=s["residual"], eps=EPS)
    if case["op"] == "matmul":
        return ops.matmul(s["a"], s["a_scale"], s["b"], s["b_scale"], bias=s["bias"], residual=s["residual"], out_dtype=TYPES[case["type"]])
    alpha, limit, shift = ACTIVATIONS[case["act"]]
    return ops.gated_matmul(s["a"], s["a_scale"], s["w13"], s["w13_scale"], bias=s["b13"], alpha=alpha, limit=limit, shift=shift)


# ------------------------------------------------------------ the plain form

def _value(q, scale, rows):
    """The numbers that E4M3 codes and their blocks' scales stand for, in 32 bits."""
    s = scale.repeat_interleave(BLOCK, 1)[:, :q.shape[1]]
    return q.float() * (s if rows == 1 else s.repeat_interleave(rows, 0)[:q.shape[0]])


def _run_plain(s):
    case = s["case"]
    if case["op"] == "norm":
        n = s["x"].float()
        if s["residual"] is not None:
            n = n + s["residual"].float()
        y = n * torch.rsqrt((n * n).mean(dim=1, keepdim=True) + EPS) * s["weight"].float()
        q, scale = _quantised(y, 1)
        return (q, scale, n.to(s["x"].dtype)) if s["residual"] is not None else (q, scale)
    a = _value(s["a"], s["a_scale"], 1)
    if case["op"] == "matmul":
        c = a @ _value(s["b"], s["b_scale"], BLOCK).t()
        if s["bias"] is not None:
            c = c + s["bias"].float()
        if s["residual"] is not None:
            c = c + s["residual"].float()
        return c.to(TYPES[case["type"]])
    F = case["F"]
    z = [a @ _value(s["w13"][i * F:(i + 1) * F], s["w13_scale"][i], BLOCK).t() for i in (0, 1)]
    if s["b13"] is not None:
        z = [z[i] + s["b13"][i * F:(i + 1) * F].float() for i in (0, 1)]
    alpha, limit, shift = ACTIVATIONS[case["act"]]
    gate, linear = z[0].clamp(max=limit), z[1].clamp(-limit, limit)
    return _quantised(gate / (1 + torch.exp(-alpha * gate)) * (linear + shift), 1)


def run(state):
    return _run_own(state) if own else _run_plain(state)


# --------------------------------------------------- the definition, 64 bits

def _spread(scale, n, dim):
    """scale[..., i // 128, ...] for i in 0 .. n - 1 along `dim`, in 64 bits."""
    return scale.double().index_select(dim, torch.arange(n, device=scale.device) // BLOCK)


def _codes(y):
    """y over its block's scale, before the rounding to E4M3, and the scales."""
    T, d = y.shape
    nb = -(-d // BLOCK)
    at = (torch.arange(d, device=y.device) // BLOCK).expand(T, d)
    most = torch.zeros(T, nb, dtype=torch.float64, device=y.device).scatter_reduce_(1, at, y.abs(), "amax")
    scale = torch.maximum(most / E4M3_MAX, torch.full_like(most, SCALE_MIN))
    return y / scale.gather(1, at), scale


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        n = s["x"].double()
        if case["residual"]:
            n = n + s["residual"].double()
        rms = torch.sqrt(n.square().sum(dim=1) / case["d"] + EPS)
        q, scale = _codes(n / rms[:, None] * s["weight"].double())
        return (q, scale, n) if case["residual"] else (q, scale)
    K = case["K"]
    a = s["a"].double() * _spread(s["a_scale"], K, 1)

    def product(w, scale):
        return torch.einsum("mk,nk->mn", a, w.double() * _spread(_spread(scale, K, 1), w.shape[0], 0))

    if case["op"] == "matmul":
        c = product(s["b"], s["b_scale"])
        for more in (s["bias"], s["residual"]):
            if more is not None:
                c += more.double()
        return c
    F = case["F"]
    gate, linear = product(s["w13"][:F], s["w13_scale"][0]), product(s["w13"][F:], s["w13_scale"][1])
    if case["bias"]:
        gate, linear = gate + s["b13"][:F].double(), linear + s["b13"][F:].double()
    alpha, limit, shift = ACTIVATIONS[case["act"]]
    gate = torch.minimum(gate, torch.full_like(gate, limit))
    linear = torch.maximum(torch.minimum(linear, torch.full_like(linear, limit)), torch.full_like(linear, -limit))
    return _codes(gate * torch.sigmoid(alpha * gate) * (linear + shift))
