"""The dense 8-bit operators on a B200 against their definitions in 64 bits.

Bounds count roundings (see ``_fp8``); inputs are seeded.  Sizes sit at the edges of the kernels' tiles: rows
around 8, 32, 64, 128 and 256, columns around 16, 32, 64, 128 and 256, K from one 16-byte unit to many blocks.
"""
import math

import pytest

torch = pytest.importorskip("torch")

import sparse_moe_rmsnorm_b200 as moe
from _fp8 import (BLOCK, E4M3_MAX, SCALE_MIN, U32, check_codes, gated_ref, half_step, norm_ref, product_ref, rows, value,
                  weight)

pytestmark = pytest.mark.gpu

BF16, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32
ACTS = {"clamped": (1.702, 7.0, 1.0), "silu": (1.0, math.inf, 0.0)}


@pytest.fixture(scope="module")
def ops():
    o = moe.Fp8Ops()
    yield o
    assert o.sync_status() == moe.MOE_OK
    o.close()


def randn(*shape, seed=0, dtype=FP32):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(*shape, generator=g, device="cuda").to(dtype)


# ------------------------------------------------------------------ the norm

@pytest.mark.parametrize("dtype", [BF16, FP16, FP32])
@pytest.mark.parametrize("T,d", [(1, 16), (1, 2880), (3, 64), (5, 144), (33, 128), (64, 2880), (7, 1040), (130, 4112),
                                 (2, 8192), (3, 8208), (2, 16384), (1000, 272)])
@pytest.mark.parametrize("with_residual", [False, True])
def test_norm(ops, T, d, dtype, with_residual):
    x, w = randn(T, d, seed=T + d, dtype=dtype), (1 + 0.3 * randn(d, seed=5)).to(BF16)
    x[:, ::29] *= 16
    res = randn(T, d, seed=9, dtype=dtype) if with_residual else None
    out = ops.add_rmsnorm(x, w, residual=res, eps=1e-5)
    n, y, tol = norm_ref(x, res, w, 1e-5)
    check_codes(out[0], out[1], y, tol)
    assert len(out) == (3 if with_residual else 2)
    if with_residual:
        assert out[2].dtype == dtype
        assert ((out[2].double() - n).abs() <= n.abs() * (half_step(dtype) * 1.001 + U32) + 2.0 ** -25).all()


def test_norm_in_place_and_strided(ops):
    """The sum may replace the residual or x; rows may lie apart, and what lies between them stays."""
    T, d, ld = 37, 272, 320
    w = (1 + 0.3 * randn(d, seed=5)).to(BF16)
    base_x, base_r = randn(T + 2, ld, seed=1, dtype=BF16), randn(T + 2, ld, seed=2, dtype=BF16)
    want = ops.add_rmsnorm(base_x[1:T + 1, 8:8 + d].contiguous(), w, residual=base_r[1:T + 1, 16:16 + d].contiguous())
    for target in ("residual", "x"):
        bx, br = base_x.clone(), base_r.clone()
        x, r = bx[1:T + 1, 8:8 + d], br[1:T + 1, 16:16 + d]
        out = ops.add_rmsnorm(x, w, residual=r, sum_out=r if target == "residual" else x)
        for a, b in zip(out, want):
            assert torch.equal(a.float(), b.float())
        b, base, c0 = (br, base_r, 16) if target == "residual" else (bx, base_x, 8)
        keep = torch.ones_like(base, dtype=torch.bool)
        keep[1:T + 1, c0:c0 + d] = False
        assert torch.equal(b[keep], base[keep])


def test_norm_of_a_row_added_to_itself(ops):
    """x as its own residual, and its sum in its place."""
    x, w = randn(9, 400, seed=1, dtype=BF16), torch.ones(400, dtype=BF16, device="cuda")
    want = ops.add_rmsnorm(x, w, residual=x.clone())
    got = ops.add_rmsnorm(x, w, residual=x, sum_out=x)
    assert got[2].data_ptr() == x.data_ptr()
    for a, b in zip(got, want):
        assert torch.equal(a.float(), b.float())


def test_one_row_in_place_under_another_stride(ops):
    """One row's distance to the next means nothing: the same row is the same place whatever view it is."""
    d, K = 272, 144
    w = (1 + 0.3 * randn(d, seed=5)).to(BF16)
    a, sa = rows(1, K, 1)
    b, sb = weight(d, K, 2)
    base, x = randn(4, 400, seed=1, dtype=BF16), randn(1, d, seed=2, dtype=BF16)
    want = ops.add_rmsnorm(x, w, residual=base[1:2, :d].clone())
    want_c = ops.matmul(a, sa, b, sb, residual=base[1:2, :d].clone())
    for out_of in (lambda t: t[1, :d][None], lambda t: t[1:2, :d]):
        for r_of in (lambda t: t[1, :d][None], lambda t: t[1:2, :d]):
            buf = base.clone()
            got = ops.add_rmsnorm(x, w, residual=r_of(buf), sum_out=out_of(buf))
            for p, q in zip(got, want):
                assert torch.equal(p.float(), q.float())
            assert torch.equal(buf[1, :d], want[2][0])
            buf[1, :d] = base[1, :d]
            assert torch.equal(buf, base)
            ops.matmul(a, sa, b, sb, residual=r_of(buf), out=out_of(buf))
            assert torch.equal(buf[1, :d], want_c[0])
            buf[1, :d] = base[1, :d]
            assert torch.equal(buf, base)
    # a column of results: its elements lie apart by the rows' distance alone
    col = torch.zeros(6, 4, dtype=BF16, device="cuda")
    a, sa = rows(6, K, 1)
    b, sb = weight(1, K, 2)
    want_c = ops.matmul(a, sa, b, sb, residual=col[:, 1:2].clone())
    ops.matmul(a, sa, b, sb, residual=col[:, 1:2], out=col.t()[1:2].t())
    assert torch.equal(col[:, 1:2], want_c) and (col[:, [0, 2, 3]] == 0).all()
    with pytest.raises(moe.MoEError):                              # over its neighbour's first half
        ops.matmul(a, sa, b, sb, residual=col[:, 1:2], out=col.view(-1)[:6].view(6, 1))


def test_norm_zeros_infinities_and_nan(ops):
    """A row of zeros, and blocks of zeros, have the smallest scale and zero codes; a NaN spoils its own row
    only, an infinity makes its own block NaN and the rest of its row zero."""
    d = 300 // 16 * 16
    x = randn(6, d, seed=3)
    x[0] = 0
    x[1, :128] = 0
    x[2, 5] = math.nan
    x[3, 130] = math.inf
    w = torch.ones(d, dtype=BF16, device="cuda")
    q, s = ops.add_rmsnorm(x, w)
    assert (s[0] == SCALE_MIN).all() and (q[0].float() == 0).all()
    assert s[1, 0] == SCALE_MIN and (q[1, :128].float() == 0).all() and s[1, 1] > SCALE_MIN
    assert s[2].isnan().all() and q[2].float().isnan().all()
    assert s[3, 1].isnan() and q[3, 128:256].float().isnan().all()
    assert s[3, 0] == SCALE_MIN and (q[3, :128].float() == 0).all() and (q[3, 256:].float() == 0).all()
    _, y, tol = norm_ref(x[4:], None, w, 1e-5)
    check_codes(q[4:], s[4:], y, tol)


# --------------------------------------------------------------- the product

SIZES = [(1, 1, 16), (1, 5, 32), (3, 16, 48), (8, 33, 128), (9, 31, 144), (32, 64, 256), (33, 65, 272), (64, 127, 400),
         (65, 129, 640), (127, 128, 1040), (128, 257, 128), (129, 255, 2064), (255, 130, 512), (257, 300, 784),
         (1, 5120, 2880), (17, 2885, 2880), (300, 1000, 4112), (1000, 2880, 576), (2049, 1303, 304), (256, 5120, 2880), (200, 4901, 784),
         (40, 19100, 144), (70, 20001, 272), (777, 5001, 400), (1100, 2885, 528)]
RES_SIZES = [(1, 40, 64), (30, 2885, 272), (130, 257, 400), (513, 1024, 1552), (45, 19101, 144), (1100, 2885, 528), (300, 19000, 144)]
GATED_SIZES = [(1, 16, 16), (2, 48, 64), (9, 128, 144), (32, 144, 256), (64, 272, 400), (65, 112, 128),
               (128, 384, 1040), (129, 1360, 272), (257, 640, 528), (1, 2880, 2880), (31, 2880, 2880),
               (1025, 2000, 304), (1030, 4112, 144), (100, 9600, 128), (150, 19104, 128)]


@pytest.mark.parametrize("M,N,K", SIZES)
@pytest.mark.parametrize("dtype", [BF16, FP16, FP32])
def test_matmul(ops, M, N, K, dtype):
    a, sa = rows(M, K, M)
    b, sb = weight(N, K, N)
    c = ops.matmul(a, sa, b, sb, out_dtype=dtype)
    want, tol = product_ref(a, sa, b, sb)
    assert c.dtype == dtype and c.shape == (M, N)
    assert ((c.double() - want).abs() <= tol + (want.abs() + tol) * half_step(dtype) + 2.0 ** -25).all()


@pytest.mark.parametrize("M,N,K", RES_SIZES)
@pytest.mark.parametrize("dtype", [BF16, FP16, FP32])
def test_matmul_bias_and_residual(ops, M, N, K, dtype):
    a, sa = rows(M, K, M)
    b, sb = weight(N, K, N)
    bias, res = randn(N, seed=3, dtype=BF16), randn(M, N, seed=4, dtype=dtype)
    want, tol = product_ref(a, sa, b, sb)
    for bb, rr in ((bias, None), (None, res), (bias, res)):
        w, t = want, tol
        for more in (bb, rr):
            if more is not None:
                w = w + more.double()
                t = t + (w.abs() + t) * U32
        c = ops.matmul(a, sa, b, sb, bias=bb, residual=rr, out_dtype=dtype)
        assert ((c.double() - w).abs() <= t + (w.abs() + t) * half_step(dtype) + 2.0 ** -25).all()
    # in place of the residual, the same bits
    r2 = res.clone()
    c2 = ops.matmul(a, sa, b, sb, bias=bias, residual=r2, out=r2)
    assert c2.data_ptr() == r2.data_ptr() and torch.equal(c2, c)


@pytest.mark.parametrize("M,N", [(20, 100), (200, 257), (300, 512)])
@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_matmul_strides_leave_the_rest(ops, M, N, dtype):
    """Rows of a, residual and c at odd places and distances; what lies around c stays as it was."""
    K = 272
    a, sa = rows(M, K, 1)
    b, sb = weight(N, K, 2)
    abuf = torch.zeros(M + 1, K + 64, dtype=torch.uint8, device="cuda")
    abuf[1:, 32:32 + K] = a.view(torch.uint8)
    res = randn(M, N, seed=7, dtype=dtype)
    want = ops.matmul(a, sa, b, sb, residual=res)
    for pad, off in ((5, 3), (24, 16)):           # odd places, and whole 16-byte units at the same time
        cbuf = torch.full((M + 2, N + pad + off), 7.0, dtype=dtype, device="cuda")
        rbuf = torch.zeros(M, N + pad, dtype=dtype, device="cuda")
        rbuf[:, :N] = res
        c = cbuf[1:M + 1, off:off + N]
        ops.matmul(abuf[1:, 32:32 + K], sa, b.view(torch.uint8), sb, residual=rbuf[:, :N], out=c)
        assert torch.equal(c, want)
        keep = torch.ones_like(cbuf, dtype=torch.bool)
        keep[1:M + 1, off:off + N] = False
        assert (cbuf[keep] == 7).all()


@pytest.mark.parametrize("M,N,K", [(300, 19000, 144), (70, 19101, 144), (37, 2886, 272)])
@pytest.mark.parametrize("dtype", [BF16, FP16, FP32])
@pytest.mark.parametrize("c_at,c_pad,r_at,r_pad", [(0, 1, 0, 1), (1, 0, 1, 0), (1, 3, 1, 2), (2, 2, 1, 4), (3, 1, 0, 4), (4, 4, 4, 8)])
def test_matmul_rows_that_start_anywhere(ops, M, N, K, dtype, c_at, c_pad, r_at, r_pad):
    """Every element comes out the same wherever the rows of the result and of the residual start, and what lies
    around them stays; in place of the residual too."""
    a, sa = rows(M, K, M)
    b, sb = weight(N, K, N)
    bias, res = randn(N, seed=3, dtype=BF16), randn(M, N, seed=4, dtype=dtype)
    plain, want = (ops.matmul(a, sa, b, sb, bias=bias, residual=r, out_dtype=dtype) for r in (None, res))
    exact, tol = product_ref(a, sa, b, sb)
    for more in (bias, res):
        exact = exact + more.double()
        tol = tol + (exact.abs() + tol) * U32
    assert ((want.double() - exact).abs() <= tol + (exact.abs() + tol) * half_step(dtype) + 2.0 ** -25).all()

    def lain(at, pad, fill):
        base = torch.full((at + M * (N + pad) + 7,), -77.0, dtype=dtype, device="cuda")
        view = base[at:at + M * (N + pad)].view(M, N + pad)[:, :N]
        if fill is not None:
            view.copy_(fill)
        return base, view

    for same in (False, True):
        r_base, r = lain(c_at if same else r_at, c_pad if same else r_pad, res)
        c_base, c = (r_base, r) if same else lain(c_at, c_pad, None)
        ops.matmul(a, sa, b, sb, bias=bias, residual=r, out=c)
        assert torch.equal(c, want)
        c.fill_(-77.0)
        assert (c_base == -77.0).all()
        if not same:
            assert torch.equal(r, res)
            ops.matmul(a, sa, b, sb, bias=bias, out=c)
            assert torch.equal(c, plain)
            c.fill_(-77.0)
            assert (c_base == -77.0).all()


def test_matmul_padded_batch_leaves_rows_behind(ops):
    """A batch of 70 rows in a buffer of 200: the rows behind stay, whatever the operand holds there."""
    M, N, K = 70, 300, 528
    a, sa = rows(200, K, 1)
    b, sb = weight(N, K, 2)
    want = ops.matmul(a[:M].contiguous(), sa[:M].contiguous(), b, sb)
    a.view(torch.uint8)[M:] = 0x7F               # NaN codes
    buf = torch.full((200, N), 3.0, dtype=BF16, device="cuda")
    ops.matmul(a[:M], sa[:M], b, sb, out=buf[:M])
    assert torch.equal(buf[:M], want) and (buf[M:] == 3).all()


def test_matmul_nan_stays_in_its_row(ops):
    M, N, K = 140, 300, 400
    a, sa = rows(M, K, 1)
    b, sb = weight(N, K, 2)
    want = ops.matmul(a, sa, b, sb)
    a2 = a.clone()
    a2.view(torch.uint8)[17, 33] = 0x7F
    sa2 = sa.clone()
    sa2[131, 2] = math.inf
    c = ops.matmul(a2, sa2, b, sb)
    assert c[17].isnan().all() and not torch.isfinite(c[131]).any()
    rest = [i for i in range(M) if i not in (17, 131)]
    assert torch.equal(c[rest], want[rest])


def test_matmul_far_scales(ops):
    """Scales that are no powers of two, across the fp32 range: exact products of the block sums."""
    M, N, K = 40, 200, 384
    a, sa = rows(M, K, 3)
    b, sb = weight(N, K, 4)
    sa = sa * torch.tensor([1e-18, 1.0, 3e-7], device="cuda")
    sb = sb * torch.tensor([1e9, 0.0, 1.7], device="cuda")
    c = ops.matmul(a, sa, b, sb, out_dtype=FP32)
    want, tol = product_ref(a, sa, b, sb)
    assert ((c.double() - want).abs() <= tol + (want.abs() + tol) * half_step(FP32) + 1e-37).all()


@pytest.mark.parametrize("M,N,K", [(1, 2880, 2880), (256, 5120, 2880), (2048, 5120, 2880)])
def test_matmul_repeats_bit_for_bit(ops, M, N, K):
    a, sa = rows(M, K, 3)
    b, sb = weight(N, K, 4)
    c = ops.matmul(a, sa, b, sb)
    for _ in range(3):
        assert torch.equal(ops.matmul(a, sa, b, sb), c)


def test_matmul_output_past_32_bits(ops):
    """An output of more than 2^32 bytes, rows far apart: the last rows land where they belong."""
    M, N, K, ld = 257, 48, 64, 1 << 23
    a, sa = rows(M, K, 3)
    b, sb = weight(N, K, 4)
    want = ops.matmul(a, sa, b, sb)
    buf = torch.empty(M * ld, dtype=BF16, device="cuda")
    c = buf.view(M, ld)[:, :N]
    ops.matmul(a, sa, b, sb, out=c)
    assert torch.equal(c, want)


# ----------------------------------------------------------- the gated product

@pytest.mark.parametrize("M,F,K", GATED_SIZES)
@pytest.mark.parametrize("act", sorted(ACTS))
@pytest.mark.parametrize("with_bias", [False, True])
def test_gated(ops, M, F, K, act, with_bias):
    a, sa = rows(M, K, M)
    gate, linear = weight(F, K, F), weight(F, K, F + 1)
    w13 = torch.cat([gate[0].view(torch.uint8), linear[0].view(torch.uint8)])
    w13s = torch.stack([gate[1], linear[1]])
    bias = randn(2 * F, seed=8, dtype=BF16) if with_bias else None
    alpha, limit, shift = ACTS[act]
    h, hs = ops.gated_matmul(a, sa, w13, w13s, bias=bias, alpha=alpha, limit=limit, shift=shift)
    want, tol = gated_ref(a, sa, w13, w13s, bias, alpha, limit, shift)
    check_codes(h, hs, want, tol)
    # 3-D weights, and the same bits again
    h2, hs2 = ops.gated_matmul(a, sa, w13.view(torch.float8_e4m3fn).view(2, F, K), w13s, bias=bias, alpha=alpha,
                               limit=limit, shift=shift)
    assert torch.equal(h.view(torch.uint8), h2.view(torch.uint8)) and torch.equal(hs, hs2)


@pytest.mark.parametrize("M,F,K", [(129, 640, 6144), (200, 272, 2064), (333, 144, 2880), (1200, 256, 2880), (400, 1360, 4112)])
@pytest.mark.parametrize("act", sorted(ACTS))
def test_gated_split_over_many_row_tiles(ops, M, F, K, act):
    """K split over a cluster where there are several tiles of rows, too: a long K and few columns."""
    pl = moe.moe_fp8_debug_plan(True, M, F, K, torch.cuda.get_device_properties(0).multi_processor_count)
    assert pl["split"] > 1 and pl["m_tiles"] > 1 and not pl["few"]
    test_gated(ops, M, F, K, act, True)


def test_gated_zero_and_nan_rows(ops):
    M, F, K = 40, 272, 256
    a, sa = rows(M, K, 1)
    gate, linear = weight(F, K, 2), weight(F, K, 3)
    w13 = torch.cat([gate[0].view(torch.uint8), linear[0].view(torch.uint8)])
    w13s = torch.stack([gate[1], linear[1]])
    a.view(torch.uint8)[5] = 0
    want = ops.gated_matmul(a, sa, w13, w13s)
    a.view(torch.uint8)[7, 0] = 0x7F
    h, s = ops.gated_matmul(a, sa, w13, w13s)
    assert (s[5] == SCALE_MIN).all() and (h[5].float() == 0).all()
    assert s[7].isnan().all() and h[7].float().isnan().all()
    rest = [i for i in range(M) if i != 7]
    assert torch.equal(h.view(torch.uint8)[rest], want[0].view(torch.uint8)[rest]) and torch.equal(s[rest], want[1][rest])


# -------------------------------------------------------------------- together

def ffn(T, d, F, seed=0, b=True):
    w13, w2 = randn(2 * F, d, seed=seed) / math.sqrt(d), randn(d, F, seed=seed + 1) / math.sqrt(F)
    return moe.DenseWeights.from_float(1 + 0.2 * randn(d, seed=seed + 2), w13, w2, randn(2 * F, seed=seed + 3) if b else None,
                                       randn(d, seed=seed + 4) if b else None)


def ffn_ref(x, w, residual, eps, act):
    """The block in 64 bits, its 8-bit roundings left out: (y, the size of the feed-forward part)."""
    alpha, limit, shift = act
    n = x.double() if residual is None else x.double() + residual.double()
    z = n / torch.sqrt(n.square().mean(1, keepdim=True) + eps) * w.norm_scale.double()
    F = w.w13.shape[0] // 2
    g, u = (z @ value(w.w13[i * F:(i + 1) * F], w.w13_scale[i], BLOCK).t() + (0 if w.b13 is None else w.b13[i * F:(i + 1) * F].double())
            for i in (0, 1))
    g, u = g.clamp(max=limit), u.clamp(-limit, limit)
    f = g * torch.sigmoid(alpha * g) * (u + shift) @ value(w.w2, w.w2_scale, BLOCK).t() + (0 if w.b2 is None else w.b2.double())
    return n + f, f


@pytest.mark.parametrize("T,d,F", [(1, 2880, 2880), (32, 2880, 2880), (70, 272, 144), (300, 1040, 640), (2048, 2880, 2880)])
@pytest.mark.parametrize("with_residual", [False, True])
def test_dense_ffn(ops, T, d, F, with_residual):
    """The three operators as a block.  Each of the two 8-bit roundings is off by at most 2^-4 of an element,
    with either sign: over sums of hundreds of terms that is below 2^-4 of the result's size in the 2-norm."""
    w, act = ffn(T, d, F), ACTS["clamped"]
    x = randn(T, d, seed=11, dtype=BF16)
    res = randn(T, d, seed=12, dtype=BF16) if with_residual else None
    layer = moe.DenseFFN(ops)
    y = layer.forward(x, w, residual=res)
    want, f = ffn_ref(x, w, res, 1e-5, act)
    assert (y.double() - want).norm() <= (2 * 2.0 ** -4) * f.norm() + 2 * half_step(BF16) * want.norm()
    assert layer.sync_status() == moe.MOE_OK
    # step by step, the same bits
    q = ops.add_rmsnorm(x, w.norm_scale, residual=res)
    h = ops.gated_matmul(q[0], q[1], w.w13, w.w13_scale, bias=w.b13)
    assert torch.equal(y, ops.matmul(*h, w.w2, w.w2_scale, bias=w.b2, residual=q[2] if with_residual else x))


def test_dense_ffn_beside_the_routed_block(ops):
    """A layer with a shared expert: the routed block and the dense one on the same stream, as a user runs them."""
    from moe_inputs import CONFIGS, make_config_inputs
    cfg = CONFIGS["tiny"]
    inp = make_config_inputs(cfg)
    import numpy as np
    x = torch.from_numpy(inp["x"].view(np.int16)).view(BF16).cuda()
    m, mw, dw, dense = moe.MoE(cfg.T, cfg.d, cfg.F, cfg.E, cfg.k, cfg.eps), moe.MoEWeights.from_numpy(inp), ffn(cfg.T, cfg.d, 256), moe.DenseFFN(ops)
    alone = dense.forward(m.forward(x, mw), dw)
    torch.cuda.synchronize()
    for _ in range(20):
        y = dense.forward(m.forward(x, mw), dw)
    torch.cuda.synchronize()
    assert torch.equal(y, alone) and m.sync_status() == moe.MOE_OK
    m.close()


def test_captured_and_replayed_with_new_inputs(ops):
    """One graph of the block, replayed on other inputs, and two graphs at once on two streams."""
    T, d, F = 48, 528, 400
    w, layer = ffn(T, d, F), moe.DenseFFN(ops)
    xs = [randn(T, d, seed=20 + i, dtype=BF16) for i in range(4)]
    want = [layer.forward(x, w) for x in xs]
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        x, y = torch.empty_like(xs[0]), torch.empty_like(xs[0])
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            layer.forward(x, w, y=y)
        graphs.append((g, x, y, torch.cuda.Stream()))
    for i in (0, 2):
        for k, (g, x, y, s) in enumerate(graphs):
            x.copy_(xs[i + k])
        torch.cuda.synchronize()
        for g, x, y, s in graphs:
            with torch.cuda.stream(s):
                for _ in range(10):
                    g.replay()
        torch.cuda.synchronize()
        for k, (g, x, y, s) in enumerate(graphs):
            assert torch.equal(y, want[i + k])


def test_other_streams(ops):
    """Calls of every size at once on three streams give what they give alone."""
    sizes = [(1, 512, 2880), (64, 2880, 528), (700, 640, 1040)]
    data = [(rows(M, K, 5), weight(N, K, 6)) for M, N, K in sizes]
    want = [ops.matmul(*a, *b) for a, b in data]
    gate = [(rows(M, 256, 5), weight(2 * 144, 256, 7)) for M, _, _ in sizes]
    gs = [torch.stack([weight(144, 256, 8)[1], weight(144, 256, 9)[1]]) for _ in sizes]
    want_g = [ops.gated_matmul(*a, w[0], s) for (a, w), s in zip(gate, gs)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sizes]
    for _ in range(10):
        got, got_g = [], []
        for i, s in enumerate(streams):
            (a, b), (ga, gw) = data[i], gate[i]
            got.append(ops.matmul(*a, *b, stream=s))
            got_g.append(ops.gated_matmul(*ga, gw[0], gs[i], stream=s.cuda_stream if i else s))
        torch.cuda.synchronize()
        for x, y in zip(got, want):
            assert torch.equal(x, y)
        for x, y in zip(got_g, want_g):
            assert torch.equal(x[0].view(torch.uint8), y[0].view(torch.uint8)) and torch.equal(x[1], y[1])


def test_wait_that_runs_out(ops):
    """The status reports it once; the object stays usable."""
    ops2 = moe.Fp8Ops()
    moe.moe_fp8_set_wait_limit_ns(ops2.ctx, 2_000_000)
    moe.moe_fp8_selftest_wait_timeout(ops2.ctx)
    assert ops2.sync_status() == moe.MOE_ERR_TIMEOUT
    assert ops2.sync_status() == moe.MOE_OK
    moe.moe_fp8_set_wait_limit_ns(ops2.ctx, 2_000_000_000)
    for M in (1, 40, 600):
        a, b = rows(M, 272, 1), weight(300, 272, 2)
        assert torch.equal(ops2.matmul(*a, *b), ops.matmul(*a, *b))
    assert ops2.sync_status() == moe.MOE_OK
    ops2.close()


def test_new_objects_start_clean_on_any_stream():
    """The count is zero for a stream that is not ordered behind the default one, which is kept busy here."""
    s = torch.cuda.Stream()
    for _ in range(20):
        torch.cuda._sleep(2_000_000)
        ops2 = moe.Fp8Ops()
        moe.moe_fp8_set_wait_limit_ns(ops2.ctx, 1_000_000)
        with torch.cuda.stream(s):
            assert ops2.sync_status() == moe.MOE_OK
        moe.moe_fp8_selftest_wait_timeout(ops2.ctx, stream=s)      # (its memory is not zero for the next one)
        assert ops2.sync_status(s) == moe.MOE_ERR_TIMEOUT
        ops2.close()


def test_every_stream_hears_of_a_wait_that_ran_out():
    """Whichever asks first: the answer to one stream leaves another's alone; so does one between two timeouts."""
    ops2 = moe.Fp8Ops()
    moe.moe_fp8_set_wait_limit_ns(ops2.ctx, 2_000_000)
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    assert ops2.sync_status(a) == ops2.sync_status(b) == moe.MOE_OK
    moe.moe_fp8_selftest_wait_timeout(ops2.ctx, stream=b)
    b.synchronize()
    assert ops2.sync_status(a) == moe.MOE_ERR_TIMEOUT
    assert ops2.sync_status(b) == moe.MOE_ERR_TIMEOUT
    assert ops2.sync_status(a) == ops2.sync_status(b) == moe.MOE_OK
    for s in (a, b):
        moe.moe_fp8_selftest_wait_timeout(ops2.ctx, stream=s)
    assert [ops2.sync_status(s) for s in (b, a, b, a)][:2] == [moe.MOE_ERR_TIMEOUT] * 2
    torch.cuda.synchronize()
    for s in (a, b):
        ops2.sync_status(s)
    assert ops2.sync_status(a) == ops2.sync_status(b) == moe.MOE_OK
    assert ops2.sync_status() == moe.MOE_ERR_TIMEOUT            # the default stream's first question
    assert ops2.sync_status() == moe.MOE_OK
    ops2.close()


def test_waits_do_not_count_the_kernel_before():
    """A product of few tiles and a very long K lasts longer than the limit of a single wait; the next product, which
    has SMs to start on meanwhile, waits for it without running out."""
    ops2, limit_ns = moe.Fp8Ops(), 1_000_000
    M, N, K = 17, 16, 1 << 24
    a, sa = torch.zeros(M, K, dtype=torch.uint8, device="cuda"), torch.ones(M, K // 128, device="cuda")
    b, sb = torch.zeros(N, K, dtype=torch.uint8, device="cuda"), torch.ones(1, K // 128, device="cuda")
    data = [((M, K), (N, K)) for M, N, K in ((40, 300, 272), (600, 5000, 272), (70, 19101, 144))]
    data = [(rows(*ra, 1), weight(*rb, 2)) for ra, rb in data]
    want = [ops2.matmul(*x, *w) for x, w in data]
    long_out = torch.empty(M, N, dtype=BF16, device="cuda")
    ops2.matmul(a, sa, b, sb, out=long_out)
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    start.record()
    ops2.matmul(a, sa, b, sb, out=long_out)
    end.record()
    torch.cuda.synchronize()
    assert start.elapsed_time(end) * 1e6 > 2 * limit_ns         # (or the test shows nothing)
    assert ops2.sync_status() == moe.MOE_OK
    moe.moe_fp8_set_wait_limit_ns(ops2.ctx, limit_ns)
    for (x, w), y in zip(data, want):
        out = torch.empty_like(y)
        torch.cuda.synchronize()
        ops2.matmul(a, sa, b, sb, out=long_out)
        ops2.matmul(*x, *w, out=out)
        assert ops2.sync_status() == moe.MOE_OK
        assert torch.equal(out, y) and (long_out == 0).all()
    ops2.close()


CAPTURE_FIRST = """
import sys, torch
sys.path[:0] = [%r, %r]
import sparse_moe_rmsnorm_b200 as moe
from _fp8 import rows, weight
ops = moe.Fp8Ops()
w = torch.ones(272, dtype=torch.bfloat16, device="cuda")
data = [(rows(M, 272, M), weight(N, 272, N), torch.randn(M, 272, device="cuda").bfloat16()) for M, N in ((1, 300), (40, 300), (600, 5000))]
gs = [torch.stack([weight(N // 32 * 16, 272, 3)[1]] * 2) for N in (300, 300, 5000)]
g = torch.cuda.CUDAGraph()
def call():
    return [(ops.matmul(*a, *b), *ops.gated_matmul(*a, b[0][:b[0].shape[0] // 32 * 32], s), *ops.add_rmsnorm(x, w, residual=x))
            for (a, b, x), s in zip(data, gs)]
with torch.cuda.graph(g):
    out = call()
g.replay()
torch.cuda.synchronize()
for one, other in zip(out, call()):
    for p, q in zip(one, other):
        assert torch.equal(p.float(), q.float())
assert ops.sync_status() == moe.MOE_OK
print("captured first")
"""


def test_first_calls_captured():
    """A process whose first calls, of every form, are inside a capture."""
    import os
    import subprocess
    import sys
    here = os.path.dirname(os.path.abspath(__file__))
    r = subprocess.run([sys.executable, "-c", CAPTURE_FIRST % (os.path.dirname(here), here)], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "captured first" in r.stdout, r.stderr[-2000:]


def test_empty_batches(ops):
    K, N = 272, 96
    w = torch.ones(K, dtype=BF16, device="cuda")
    q, s, n = ops.add_rmsnorm(torch.empty(0, K, dtype=BF16, device="cuda"), w, residual=torch.empty(0, K, dtype=BF16, device="cuda"))
    assert q.shape == (0, K) and s.shape == (0, 3) and n.shape == (0, K)
    b, sb = weight(N, K, 1)
    assert ops.matmul(q, s, b, sb).shape == (0, N)
    h, hs = ops.gated_matmul(q, s, b, torch.stack([weight(48, K, 1)[1]] * 2))
    assert h.shape == (0, 48) and hs.shape == (0, 1)


def test_refusals(ops):
    """What the documentation does not allow raises before anything is launched."""
    M, N, K = 8, 64, 256
    a, sa = rows(M, K, 1)
    b, sb = weight(N, K, 2)
    w13s = torch.stack([weight(32, K, 3)[1]] * 2)
    x, w = randn(M, K, dtype=BF16), torch.ones(K, dtype=BF16, device="cuda")
    odd = torch.zeros(M * K + 16, dtype=torch.uint8, device="cuda")
    cases = [
        lambda: ops.matmul(a, sa, b[:, :128], sb),                                   # K differs
        lambda: ops.matmul(a, sa, b, sb.t()),                                        # scales of another shape
        lambda: ops.matmul(a, sa.half(), b, sb),
        lambda: ops.matmul(a.float(), sa, b, sb),
        lambda: ops.matmul(a.cpu(), sa, b, sb),
        lambda: ops.matmul(a, sa, b.cpu(), sb),
        lambda: ops.matmul(a, sa, b.t().contiguous().t(), sb),                       # rows not contiguous
        lambda: ops.matmul(a[:1].expand(M, K), sa, b, sb),                           # the same row again
        lambda: ops.matmul(odd[1:1 + M * K].view(M, K), sa, b, sb),                  # not on 16 bytes
        lambda: ops.matmul(a, sa, b, sb, out_dtype=torch.float64),
        lambda: ops.matmul(a, sa, b, sb, bias=randn(N)),                             # bias not bf16
        lambda: ops.matmul(a, sa, b, sb, residual=randn(M, N), out_dtype=BF16),      # another type
        lambda: ops.matmul(a, sa, b, sb, residual=randn(M, N + 1, dtype=BF16)),
        lambda: ops.matmul(a, sa, b, sb, out=a.view(BF16)[:, :N]),                   # over an operand
        lambda: ops.matmul(*rows(M, 24, 1), *weight(N, 24, 2)),                      # K not of 16
        lambda: ops.gated_matmul(a, sa, b, w13s, limit=0.0),
        lambda: ops.gated_matmul(a, sa, b, w13s, limit=math.nan),
        lambda: ops.gated_matmul(a, sa, b, sb),
        lambda: ops.gated_matmul(a, sa, b[:63], w13s),
        lambda: ops.gated_matmul(a, sa, b[:40], w13s[:, :1]),                        # F = 20
        lambda: ops.add_rmsnorm(x.double(), w),
        lambda: ops.add_rmsnorm(x, w.float()),
        lambda: ops.add_rmsnorm(x, w, residual=x.float()),
        lambda: ops.add_rmsnorm(x, w, residual=x[:4]),
        lambda: ops.add_rmsnorm(x, w, sum_out=x),
        lambda: ops.add_rmsnorm(x[:, :40].contiguous(), w[:40]),                     # d not of 16
        lambda: ops.add_rmsnorm(x[:, 1:17], w[:16]),                                 # not on 16 bytes
        lambda: ops.add_rmsnorm(x, w, eps=-1.0),
        lambda: ops.add_rmsnorm(x[:4], w, residual=x[4:], sum_out=x[2:6]),           # over half of both
        lambda: ops.add_rmsnorm(randn(1, 16400, dtype=BF16), torch.ones(16400, dtype=BF16, device="cuda")),
    ]
    for i, call in enumerate(cases):
        with pytest.raises(moe.MoEError) as e:
            call()
            pytest.fail("case %d was accepted" % i)
        assert e.value.code == moe.MOE_ERR_ARG
    torch.cuda.synchronize()


# ------------------------------------------------- the hard cases, in every form

# few rows, single tiles, K split over a cluster, CTA pairs; gated: few rows, a split tile, one CTA's, CTA pairs
FORMS = {"few": (9, 300, 400), "single": (70, 19101, 144), "split": (140, 300, 400), "pair": (600, 5000, 272)}
GATED_FORMS = {"few": (9, 272, 256), "split": (40, 272, 256), "single": (100, 19104, 128), "pair": (600, 2496, 272)}


def as_planned(form, gated):
    M, N, K = (GATED_FORMS if gated else FORMS)[form]
    pl = moe.moe_fp8_debug_plan(gated, M, N, K, torch.cuda.get_device_properties(0).multi_processor_count)
    assert form == ("few" if pl["few"] else "pair" if pl["ctas"] == 2 else "split" if pl["split"] > 1 else "single")
    return M, N, K


def gated_weight(F, K, seed):
    gate, linear = weight(F, K, seed), weight(F, K, seed + 1)
    return torch.cat([gate[0].view(torch.uint8), linear[0].view(torch.uint8)]), torch.stack([gate[1], linear[1]])


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("with_residual", [False, True])
def test_nan_and_infinity_in_every_form(ops, form, with_residual):
    """A NaN code or an infinite scale of a row spoils its row, of a weight its column (its 128 columns); a row of zeros
    gives zeros (or the residual); everything else comes out with the same bits."""
    M, N, K = as_planned(form, False)
    a, sa = rows(M, K, 1)
    b, sb = weight(N, K, 2)
    res = randn(M, N, seed=3, dtype=BF16) if with_residual else None
    zero, nan, inf, col, block = M // 2, 1, M - 2, 17, (N - 1) // 128
    a.view(torch.uint8)[zero] = 0
    want = ops.matmul(a, sa, b, sb, residual=res)
    assert torch.equal(want[zero], res[zero] if with_residual else torch.zeros_like(want[zero]))
    a2, sa2, b2, sb2 = a.clone(), sa.clone(), b.clone(), sb.clone()
    a2.view(torch.uint8)[nan, K - 1] = 0x7F
    sa2[inf, -1] = math.inf
    b2.view(torch.uint8)[col, 5] = 0xFF
    sb2[block, 0] = math.nan
    c = ops.matmul(a2, sa2, b2, sb2, residual=res)
    keep = torch.ones(M, N, dtype=torch.bool, device="cuda")
    keep[nan] = keep[inf] = False
    keep[:, col] = False
    keep[:, 128 * block:] = False
    assert c[nan].isnan().all() and not torch.isfinite(c[inf]).any()
    assert c[:, col].isnan().all() and c[:, 128 * block:].isnan().all()
    assert torch.equal(c[keep], want[keep])


@pytest.mark.parametrize("form", FORMS)
def test_far_scales_in_every_form(ops, form):
    """Scales that are no powers of two, across the fp32 range, and zero ones."""
    M, N, K = as_planned(form, False)
    a, sa = rows(M, K, 3)
    b, sb = weight(N, K, 4)
    kb = torch.arange(sa.shape[1], device="cuda")
    sa = sa * torch.tensor([1e-18, 3e-7, 1.0, 1e12], device="cuda")[kb] * torch.tensor([1.0, 1e-3, 0.0, 7.7], device="cuda")[torch.arange(M, device="cuda") % 4, None]
    sb = sb * torch.tensor([1e15, 1e6, 1.7, 1e-12], device="cuda")[kb]
    c = ops.matmul(a, sa, b, sb, out_dtype=FP32)
    want, tol = product_ref(a, sa, b, sb)
    # (and a step of the smallest numbers for each product of codes)
    assert ((c.double() - want).abs() <= tol + (want.abs() + tol) * half_step(FP32) + K * 448 ** 2 * 2.0 ** -149).all()
    assert (c[2::4] == 0).all()


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("dtype", [BF16, FP16, FP32])
@pytest.mark.parametrize("place", ["odd", "even", "16 bytes"])
def test_strides_in_every_form(ops, form, dtype, place):
    """Rows of a, of the residual and of the result apart and anywhere: the same bits, and nothing around the result
    or between its rows is touched; in place of the residual too."""
    M, N, K = as_planned(form, False)
    a, sa = rows(M, K, 1)
    b, sb = weight(N, K, 2)
    bias, res = randn(N, seed=3, dtype=BF16), randn(M, N, seed=7, dtype=dtype)
    want = ops.matmul(a, sa, b, sb, bias=bias, residual=res)
    abuf = torch.full((M + 1, K + 48), 0x7F, dtype=torch.uint8, device="cuda")      # NaN between the rows
    abuf[1:, 16:16 + K] = a.view(torch.uint8)
    at, pad, rpad = {"odd": (3, 5, 2), "even": (2, 2 + N % 2, 4 + N % 2), "16 bytes": (16, 16 - N % 8, 24 - N % 8)}[place]
    base = torch.full((at + M * (N + pad) + 9,), 7.0, dtype=dtype, device="cuda")
    c = base[at:at + M * (N + pad)].view(M, N + pad)[:, :N]
    rbuf = torch.zeros(M, N + rpad, dtype=dtype, device="cuda")
    rbuf[:, :N] = res
    for r in (rbuf[:, :N], c):
        if r is c:
            c.copy_(res)
        got = ops.matmul(abuf[1:, 16:16 + K], sa, b, sb, bias=bias, residual=r, out=c)
        assert got.data_ptr() == c.data_ptr() and torch.equal(c, want)
        c.fill_(7.0)
        assert (base == 7).all()


@pytest.mark.parametrize("form", GATED_FORMS)
def test_gated_nan_and_zero_rows_in_every_form(ops, form):
    """A NaN in a row makes that row's scales and codes NaN, a row of zeros (without a bias) the smallest scale and
    zero codes; the other rows keep their bits.  Rows of a apart, NaN codes between them."""
    M, F, K = as_planned(form, True)
    a, sa = rows(M, K, 1)
    w13, w13s = gated_weight(F, K, 2)
    zero, nan = M // 2, M - 2
    a.view(torch.uint8)[zero] = 0
    want = ops.gated_matmul(a, sa, w13, w13s)
    assert (want[1][zero] == SCALE_MIN).all() and (want[0][zero].float() == 0).all()
    abuf = torch.full((M + 1, K + 48), 0x7F, dtype=torch.uint8, device="cuda")
    abuf[1:, 16:16 + K] = a.view(torch.uint8)
    got = ops.gated_matmul(abuf[1:, 16:16 + K], sa, w13, w13s)
    assert torch.equal(got[0].view(torch.uint8), want[0].view(torch.uint8)) and torch.equal(got[1], want[1])
    a.view(torch.uint8)[nan, K - 1] = 0x7F
    h, s = ops.gated_matmul(a, sa, w13, w13s)
    assert s[nan].isnan().all() and h[nan].float().isnan().all()
    rest = [i for i in range(M) if i != nan]
    assert torch.equal(h.view(torch.uint8)[rest], want[0].view(torch.uint8)[rest]) and torch.equal(s[rest], want[1][rest])


@pytest.mark.parametrize("form", GATED_FORMS)
def test_gated_infinities_in_every_form(ops, form):
    """The clamps take an infinite gate (+) and linear value (+ or -) as they take any large one; a gate of -inf is
    -inf * 0: its block's scale and codes are NaN.  Without clamps an infinite value makes its block's scale infinite,
    its own code NaN and the others zero.  Other blocks keep their bits."""
    M, F, K = as_planned(form, True)
    a, sa = rows(M, K, 5)
    w13, w13s = gated_weight(F, K, 6)
    bias = randn(2 * F, seed=8, dtype=BF16)
    last = F - 1
    big, inf = bias.clone(), bias.clone()
    for col, v in ((3, 1e4), (F + 5, 1e4), (F + last, -1e4), (F + 64, 1e4)):
        big[col], inf[col] = v, math.copysign(math.inf, v)
    want, got = ops.gated_matmul(a, sa, w13, w13s, bias=big), ops.gated_matmul(a, sa, w13, w13s, bias=inf)
    assert torch.equal(got[0].view(torch.uint8), want[0].view(torch.uint8)) and torch.equal(got[1], want[1])
    y, tol = gated_ref(a, sa, w13, w13s, big, *ACTS["clamped"])
    check_codes(want[0], want[1], y, tol)

    inf[130] = -math.inf
    h, s = ops.gated_matmul(a, sa, w13, w13s, bias=inf)
    other = torch.ones(F, dtype=torch.bool, device="cuda")
    other[128:256] = False
    assert s[:, 1].isnan().all() and h.float()[:, ~other].isnan().all()
    assert torch.equal(h.view(torch.uint8)[:, other], want[0].view(torch.uint8)[:, other])
    assert torch.equal(torch.cat([s[:, :1], s[:, 2:]], 1), torch.cat([want[1][:, :1], want[1][:, 2:]], 1))

    silu = dict(alpha=1.0, limit=math.inf, shift=0.0)
    want = ops.gated_matmul(a, sa, w13, w13s, bias=bias, **silu)
    bias2 = bias.clone()
    bias2[130] = math.inf
    h, s = ops.gated_matmul(a, sa, w13, w13s, bias=bias2, **silu)
    assert (s[:, 1] == math.inf).all() and h[:, 130].float().isnan().all()
    rest = ~other
    rest[130] = False
    assert (h.float()[:, rest] == 0).all()
    assert torch.equal(h.view(torch.uint8)[:, other], want[0].view(torch.uint8)[:, other])
