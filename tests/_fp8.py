"""Definitions in 64 bits and error bounds of the dense 8-bit operators, for their tests.

Every bound counts roundings; none is fitted to an output.  ``h(t) = finfo(t).eps / 2`` is half a step of
type t relative to the value (E4M3: 2^-4, and half its smallest step, 2^-10, near zero).
"""
import math

import torch

BLOCK, E4M3_MAX, SCALE_MIN = 128, 448.0, 2.0 ** -126
U32 = 2.0 ** -24


def half_step(t):
    return torch.finfo(t).eps / 2


def spread(s, n, dim):
    """s[..., i // 128, ...] for i < n along dim, in 64 bits."""
    return s.double().index_select(dim, torch.arange(n, device=s.device) // BLOCK)


def value(q, s, rows):
    """What codes q [M, K] and their scales stand for, in 64 bits; rows: 1 (activations) or 128 (weights)."""
    s = spread(s, q.shape[1], 1)
    return q.view(torch.float8_e4m3fn).double() * (s if rows == 1 else spread(s, q.shape[0], 0))


def block_max(y):
    """max |y| over each row's blocks of 128 (a NaN stays)."""
    y = torch.nn.functional.pad(y.abs(), (0, -y.shape[1] % BLOCK))
    return y.view(y.shape[0], -1, BLOCK).amax(2)


def check_codes(q, s, y, tol):
    """Codes and scales against rows y in 64 bits that the kernel knows to within `tol` (same shape)."""
    T, d = y.shape
    assert q.dtype == torch.float8_e4m3fn and q.shape == (T, d) and s.shape == (T, -(-d // BLOCK))
    want = (block_max(y) / E4M3_MAX).clamp_min(SCALE_MIN)
    off = block_max(tol) / E4M3_MAX + 4 * U32 * want       # the maximum's error, the division's and the clamp's
    assert ((s.double() - want).abs() <= off).all(), ((s.double() - want).abs() / off).max()
    sd = spread(s, d, 1)
    got = q.double() * sd
    # half a step of E4M3 (relative, or 2^-10 of the scale among the smallest), of y / s in fp32 (three
    # roundings before it: 1 / s, the product, and y's own error)
    step = (y.abs() + tol) * (half_step(torch.float8_e4m3fn) + 4 * U32) + 2.0 ** -10 * sd
    assert ((got - y).abs() <= step + tol).all(), ((got - y).abs() / (step + tol)).max()


def norm_ref(x, residual, w, eps):
    """(sum, y) of the norm in 64 bits and y's error bound."""
    n = x.double() if residual is None else x.double() + residual.double()
    y = n / torch.sqrt(n.square().mean(1, keepdim=True) + eps) * w.double()
    # n rounds once.  The mean of squares: a square, at most 16 serial and 10 tree additions, the division and eps, so
    # 29 roundings and twice n's; its root halves them and adds 2 (the root, the reciprocal); y takes 2 products.
    return n, y, y.abs() * (29 / 2 + 1 + 1 + 2 + 2) * U32 * 1.01


def product_ref(a, a_scale, b, b_scale):
    """The product in 64 bits and its error bound before bias, residual and the output's rounding.

    An E4M3 product is exact; K products and ceil(K/128) scaled sums are added in fp32, each addition off by
    at most 2^-23 (a truncation) of the magnitudes added so far; the scales' product and its own with the
    block's sum round twice."""
    A, B = value(a, a_scale, 1), value(b, b_scale, BLOCK)
    K = A.shape[1]
    return A @ B.t(), (A.abs() @ B.abs().t()) * (K + -(-K // BLOCK) + 2) * 2 * U32


def gated_ref(a, a_scale, w13, w13_scale, bias, alpha, limit, shift):
    F = w13.shape[0] // 2
    z = []
    for i in (0, 1):
        c, t = product_ref(a, a_scale, w13[i * F:(i + 1) * F], w13_scale[i])
        if bias is not None:
            c = c + bias[i * F:(i + 1) * F].double()
            t = t + (c.abs() + t) * U32
        z.append((c, t))
    (g, tg), (u, tu) = z
    g, u = g.clamp(max=limit), u.clamp(-limit, limit)
    f = g * torch.sigmoid(alpha * g)
    h = f * (u + shift)
    # |d/dg (g sigmoid(alpha g))| < 1.1 for every alpha > 0; the exponential's argument is rounded
    # (|alpha g| half steps), it and the quotient are off by at most 4 steps, and the two products and
    # the sum round once each
    slack = h.abs() * (2 * (alpha * g).abs().clamp(max=128) + 16) * U32
    return h, 1.1 * tg * ((u + shift).abs() + tu) + f.abs() * tu + f.abs() * abs(shift) * U32 + slack


def rows(M, K, seed, device="cuda"):
    import sparse_moe_rmsnorm_b200 as moe
    g = torch.Generator(device=device).manual_seed(seed)
    x = torch.randn(M, K, generator=g, device=device)
    x[:, ::37] *= 20
    return moe.quantize_fp8_rows(x)


def weight(N, K, seed, device="cuda"):
    import sparse_moe_rmsnorm_b200 as moe
    g = torch.Generator(device=device).manual_seed(seed + 1000)
    size = torch.exp2(torch.randint(-6, 3, (-(-N // 64), -(-K // 64)), generator=g, device=device).float())
    size = size.repeat_interleave(64, 0)[:N].repeat_interleave(64, 1)[:, :K]
    return moe.quantize_fp8_weight(torch.randn(N, K, generator=g, device=device) * size / math.sqrt(K))
