"""Dense 8-bit operators beside the routed experts, and the dense feed-forward block built of them.

A matrix in 8 bits is a pair of tensors: E4M3 codes (``torch.float8_e4m3fn``, or the same bytes as
``torch.uint8``) and fp32 scales.  Activations ``[M, K]`` have a scale for each 128 consecutive elements
of a row (``[M, ceil(K/128)]``), weights ``[N, K]`` one for each 128 x 128 block
(``[ceil(N/128), ceil(K/128)]``).

Like the rest of the package this only checks and marshals arguments (``Fp8Ops`` does so in C++,
``csrc/binding.cpp``): the work is in the CUDA library, every call raises where the library or a B200
is missing, and a call returns when its kernel is queued.

There is no backward pass: results carry no gradient, also where an operand asks for one, and a tracer that
runs these calls would record their results as constants.
"""
from __future__ import annotations

import ctypes
import dataclasses
import math
from typing import Dict, Optional

import sparse_moe_rmsnorm_b200 as _moe

__all__ = [
    "MOE_BF16", "MOE_FP16", "MOE_FP32", "Fp8Ops", "DenseFFN", "DenseWeights", "quantize_fp8_rows", "quantize_fp8_weight",
    "moe_fp8_init", "moe_fp8_destroy", "moe_fp8_sync_status", "moe_fp8_set_wait_limit_ns",
    "moe_fp8_selftest_wait_timeout", "moe_add_rmsnorm_fp8", "moe_fp8_matmul", "moe_fp8_gated_matmul", "moe_fp8_debug_plan",
]

MOE_BF16, MOE_FP16, MOE_FP32 = 0, 1, 2

FP8_BLOCK = 128
FP8_MAX = 448.0
FP8_SCALE_MIN = 2.0 ** -126


# ------------------------------------------------------- C-ABI-named wrappers

def moe_fp8_init() -> int:
    h = ctypes.c_void_p()
    _moe._check(_moe.lib().moe_fp8_init(ctypes.byref(h)), "moe_fp8_init")
    return h.value


def moe_fp8_destroy(ctx: int) -> None:
    _moe.lib().moe_fp8_destroy(ctx)


def moe_fp8_sync_status(ctx, stream=None) -> int:
    return int(_moe.lib().moe_fp8_sync_status(ctx, _moe._stream(stream)))


def moe_fp8_set_wait_limit_ns(ctx, ns: int) -> None:
    _moe._check(_moe.lib().moe_fp8_set_wait_limit_ns(ctx, int(ns)), "moe_fp8_set_wait_limit_ns")


def moe_fp8_selftest_wait_timeout(ctx, stream=None) -> None:
    _moe._check(_moe.lib().moe_fp8_selftest_wait_timeout(ctx, _moe._stream(stream)), "moe_fp8_selftest_wait_timeout")


def moe_add_rmsnorm_fp8(ctx, T, d, type, x, ldx, residual, ldr, norm_scale, eps, sum_out, lds, q, q_scale,
                        stream=None) -> None:
    p = _moe._ptr
    _moe._check(_moe.lib().moe_add_rmsnorm_fp8(ctx, T, d, type, p(x), ldx, p(residual), ldr, p(norm_scale), eps,
                                               p(sum_out), lds, p(q), p(q_scale), _moe._stream(stream)),
                "moe_add_rmsnorm_fp8")


def moe_fp8_matmul(ctx, M, N, K, a, lda, a_scale, b, b_scale, bias, residual, ldr, c, ldc, type, stream=None) -> None:
    p = _moe._ptr
    _moe._check(_moe.lib().moe_fp8_matmul(ctx, M, N, K, p(a), lda, p(a_scale), p(b), p(b_scale), p(bias), p(residual),
                                          ldr, p(c), ldc, type, _moe._stream(stream)), "moe_fp8_matmul")


def moe_fp8_gated_matmul(ctx, M, F, K, a, lda, a_scale, w13, w13_scale, b13, alpha, limit, shift, h, h_scale,
                         stream=None) -> None:
    p = _moe._ptr
    _moe._check(_moe.lib().moe_fp8_gated_matmul(ctx, M, F, K, p(a), lda, p(a_scale), p(w13), p(w13_scale), p(b13), alpha,
                                                limit, shift, p(h), p(h_scale), _moe._stream(stream)),
                "moe_fp8_gated_matmul")


FP8_PLAN_FIELDS = ("few", "bn", "ctas", "split", "a_rows", "n_stages", "m_tiles", "tiles", "grid", "smem_needed")


def moe_fp8_debug_plan(gated: bool, M: int, N: int, K: int, num_sms: int) -> Dict[str, int]:
    """The launch plan of one product, computed on the host (N = F for the gated one)."""
    out = (ctypes.c_int * len(FP8_PLAN_FIELDS))()
    _moe._check(_moe.lib().moe_fp8_debug_plan(int(gated), int(M), int(N), int(K), int(num_sms), out),
                "moe_fp8_debug_plan")
    return dict(zip(FP8_PLAN_FIELDS, list(out)))


# ------------------------------------------------------------- torch layer

_binding_module = None


def _binding():
    """The operators on torch tensors (``csrc/binding.cpp``): checks, output allocation and the C call."""
    global _binding_module
    if _binding_module is None:
        import importlib

        import torch  # noqa: F401  (its libraries have to be loaded first)
        _moe.lib()
        try:
            mod = importlib.import_module("sparse_moe_rmsnorm_b200._binding")
        except ImportError as e:
            raise RuntimeError("the torch binding is not built for this torch; run `python -m sparse_moe_rmsnorm_b200.build` "
                               "(%s)" % e) from e
        mod.set_error(_moe.MoEError)
        _binding_module = mod
    return _binding_module


class Fp8Ops:
    """The operators on one device.  One object serves any number of streams and captured graphs at once;
    make it outside a capture.

    ``stream``: where a call runs (a ``torch.cuda.Stream`` or a raw handle), by default the device's current
    one; outputs that the call allocates belong to it.
    """

    def __init__(self, device=None):
        import torch
        dev = torch.device("cuda" if device is None else device)
        if dev.type != "cuda":
            raise _moe.MoEError(_moe.MOE_ERR_ARG, "Fp8Ops: not a CUDA device")
        self._index = torch.cuda.current_device() if dev.index is None else dev.index
        self.device = torch.device("cuda", self._index)
        self._c = _binding()
        with torch.cuda.device(self._index):
            self.ctx = moe_fp8_init()

    def close(self) -> None:
        if getattr(self, "ctx", None):
            moe_fp8_destroy(self.ctx)
            self.ctx = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def _on(self, stream):
        import torch
        if isinstance(stream, int):
            stream = torch.cuda.ExternalStream(stream, device=self.device)
        if stream.device != self.device:        # the device's own current stream would be taken in its place
            raise _moe.MoEError(_moe.MOE_ERR_ARG, f"stream of {stream.device}, operators of {self.device}")
        return torch.cuda.stream(stream)

    def add_rmsnorm(self, x, norm_scale, residual=None, eps: float = 1e-5, sum_out=None, stream=None):
        """RMS norm of ``x + residual`` (of ``x`` without one) in 8 bits: ``(q, q_scale, sum)``, without a
        residual ``(q, q_scale)``.

        ``x``, ``residual``: bf16, fp16 or fp32 ``[T, d]``, rows at any distance of whole 16 bytes;
        ``norm_scale``: bf16 ``[d]``.  ``sum`` is ``x + residual`` in their type, written to ``sum_out`` if
        given, which may be ``x`` or ``residual``.
        """
        if stream is not None:
            with self._on(stream):
                return self._c.add_rmsnorm(self.ctx, self._index, x, norm_scale, residual, eps, sum_out)
        return self._c.add_rmsnorm(self.ctx, self._index, x, norm_scale, residual, eps, sum_out)

    def matmul(self, a, a_scale, b, b_scale, bias=None, residual=None, out=None, out_dtype=None, stream=None):
        """``a @ b.T (+ bias) (+ residual)`` of 8-bit ``a [M, K]`` and ``b [N, K]``, rounded once to
        ``out_dtype`` (bf16 by default, fp16 or fp32; ``out``'s or ``residual``'s where one is given).

        ``bias``: bf16 ``[N]``; ``residual``: ``[M, N]`` of the output's type, which may be ``out`` itself.
        K is a multiple of 16; rows of ``a`` at any distance of whole 16 bytes, of ``residual`` and ``out`` at any.
        """
        if stream is not None:
            with self._on(stream):
                return self._c.matmul(self.ctx, self._index, a, a_scale, b, b_scale, bias, residual, out, out_dtype)
        return self._c.matmul(self.ctx, self._index, a, a_scale, b, b_scale, bias, residual, out, out_dtype)

    def gated_matmul(self, a, a_scale, w13, w13_scale, bias=None, alpha: float = 1.702, limit: float = 7.0,
                     shift: float = 1.0, stream=None):
        """Both projections of a gated feed-forward block, its activation and the product: ``(h, h_scale)``,
        ``h [M, F]`` in 8 bits for the block's second product.

        ``w13``: ``[2 F, K]`` (or ``[2, F, K]``), gate rows, then linear rows; ``w13_scale``:
        ``[2, ceil(F/128), ceil(K/128)]``; ``bias``: bf16 ``[2 F]``.  With ``g = min(gate, limit)`` and
        ``u = clamp(linear, -limit, limit)``, ``h = g * sigmoid(alpha * g) * (u + shift)``: the experts'
        activation by default, silu(gate) * linear for ``alpha=1, limit=math.inf, shift=0``.
        """
        if stream is not None:
            with self._on(stream):
                return self._c.gated_matmul(self.ctx, self._index, a, a_scale, w13, w13_scale, bias, alpha, limit, shift)
        return self._c.gated_matmul(self.ctx, self._index, a, a_scale, w13, w13_scale, bias, alpha, limit, shift)

    def sync_status(self, stream=None) -> int:
        """Waits for ``stream`` and returns MOE_OK, or MOE_ERR_TIMEOUT where a device-side wait of any call of this
        object ran out since this stream last asked: each stream hears of it once.  Streams that have to know whose
        it was take an ``Fp8Ops`` each."""
        import torch
        return moe_fp8_sync_status(self.ctx, torch.cuda.current_stream(self._index) if stream is None else stream)


def _quantize(x, rows: int):
    import torch
    M, K = x.shape
    b = torch.nn.functional.pad(x.float(), (0, -K % FP8_BLOCK, 0, -M % rows))
    b = b.view(b.shape[0] // rows, rows, b.shape[1] // FP8_BLOCK, FP8_BLOCK)
    s = (b.abs().amax(dim=(1, 3)) / FP8_MAX).clamp_min(FP8_SCALE_MIN)
    q = (b / s[:, None, :, None]).reshape(b.shape[0] * rows, b.shape[2] * FP8_BLOCK)[:M, :K]
    return q.to(torch.float8_e4m3fn).contiguous(), s.contiguous()


def quantize_fp8_weight(w):
    """A weight ``[N, K]`` in 8 bits: codes and a scale for each 128 x 128 block.  Done once, when weights are
    loaded, so in elementary torch operations, on any device."""
    return _quantize(w, FP8_BLOCK)


def quantize_fp8_rows(x):
    """Rows ``[M, K]`` in 8 bits: codes and a scale for each 128 elements, in elementary torch operations."""
    return _quantize(x, 1)


@dataclasses.dataclass
class DenseWeights:
    """The parameters of one dense feed-forward block, its matrices in 8 bits."""
    norm_scale: "torch.Tensor"    # bf16 [d]
    w13: "torch.Tensor"           # e4m3 [2F, d]: gate rows, then linear rows
    w13_scale: "torch.Tensor"     # fp32 [2, ceil(F/128), ceil(d/128)]
    b13: Optional["torch.Tensor"]  # bf16 [2F]
    w2: "torch.Tensor"            # e4m3 [d, F]
    w2_scale: "torch.Tensor"      # fp32 [ceil(d/128), ceil(F/128)]
    b2: Optional["torch.Tensor"]  # bf16 [d]

    @classmethod
    def from_float(cls, norm_scale, w13, w2, b13=None, b2=None, device="cuda") -> "DenseWeights":
        """From matrices in any floating type: ``w13 [2F, d]`` (gate rows, then linear rows), ``w2 [d, F]``."""
        import torch
        F = w13.shape[0] // 2
        gate, linear = quantize_fp8_weight(w13[:F].to(device)), quantize_fp8_weight(w13[F:].to(device))
        w2q, w2s = quantize_fp8_weight(w2.to(device))
        bf16 = lambda t: None if t is None else t.to(device=device, dtype=torch.bfloat16).contiguous()  # noqa: E731
        codes = torch.cat([gate[0].view(torch.uint8), linear[0].view(torch.uint8)]).view(torch.float8_e4m3fn)
        return cls(bf16(norm_scale), codes, torch.stack([gate[1], linear[1]]), bf16(b13), w2q, w2s, bf16(b2))


class DenseFFN:
    """The dense (or shared-expert) counterpart of ``MoE``: RMSNorm, gated feed-forward, residual, three launches.

    ``forward(x)`` is ``x + W2 h + b2`` with ``h`` the gated activation of ``W13 norm(x) + b13``;
    ``forward(x, residual)`` takes ``x + residual`` in the place of ``x`` (a layer's pending addition).
    """

    def __init__(self, ops: Optional[Fp8Ops] = None, eps: float = 1e-5, alpha: float = 1.702, limit: float = 7.0,
                 shift: float = 1.0):
        self.ops = Fp8Ops() if ops is None else ops
        self.eps, self.alpha, self.limit, self.shift = float(eps), float(alpha), float(limit), float(shift)

    def forward(self, x, w: DenseWeights, residual=None, y=None, stream=None):
        ops = self.ops
        if residual is None:
            q, s = ops.add_rmsnorm(x, w.norm_scale, eps=self.eps, stream=stream)
            n = x
        else:
            q, s, n = ops.add_rmsnorm(x, w.norm_scale, residual=residual, eps=self.eps, stream=stream)
        h, hs = ops.gated_matmul(q, s, w.w13, w.w13_scale, bias=w.b13, alpha=self.alpha, limit=self.limit,
                                 shift=self.shift, stream=stream)
        return ops.matmul(h, hs, w.w2, w.w2_scale, bias=w.b2, residual=n, out=y, out_dtype=x.dtype, stream=stream)

    def sync_status(self, stream=None) -> int:
        return self.ops.sync_status(stream)
