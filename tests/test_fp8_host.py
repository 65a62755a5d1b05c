"""The dense 8-bit operators without a GPU: argument checks before any device work, the launch plan, the
quantisers against their definition."""
import ctypes
import math
import os
import subprocess
import sys

import pytest
import torch

import sparse_moe_rmsnorm_b200 as moe
from sparse_moe_rmsnorm_b200 import build as moe_build

@pytest.fixture(scope="module")
def lib():
    moe_build.build()
    return moe.lib()


def test_null_context_and_null_results(lib):
    assert lib.moe_fp8_init(None) == moe.MOE_ERR_ARG
    assert lib.moe_fp8_destroy(None) == moe.MOE_OK
    assert lib.moe_fp8_sync_status(None, None) == moe.MOE_ERR_ARG
    assert lib.moe_fp8_set_wait_limit_ns(None, 5) == moe.MOE_ERR_ARG
    assert lib.moe_fp8_selftest_wait_timeout(None, None) == moe.MOE_ERR_ARG
    assert lib.moe_add_rmsnorm_fp8(None, 1, 64, 0, None, 64, None, 0, None, 1e-5, None, 0, None, None, None) == moe.MOE_ERR_ARG
    assert lib.moe_fp8_matmul(None, 1, 1, 16, None, 16, None, None, None, None, None, 0, None, 1, 0, None) == moe.MOE_ERR_ARG
    assert lib.moe_fp8_gated_matmul(None, 1, 16, 16, None, 16, None, None, None, None, 1.0, 7.0, 1.0, None, None, None) == moe.MOE_ERR_ARG


class Ctx(ctypes.Structure):
    """The context's layout: enough to reach the argument checks, which use nothing of the device."""
    _fields_ = [("device", ctypes.c_int), ("num_sms", ctypes.c_int), ("err", ctypes.c_void_p), ("limit", ctypes.c_ulonglong)]


def test_sizes_types_strides_and_alignment(lib):
    c = ctypes.byref(Ctx(0, 148, None, 1))
    P = 1 << 20                                  # a pointer on every boundary; nothing reads it
    norm = dict(T=4, d=64, type=0, x=P, ldx=64, r=None, ldr=0, w=P, eps=1e-5, sum=None, lds=0, q=P, s=P)
    bad = [dict(T=-1), dict(d=0), dict(d=24), dict(d=16400), dict(type=3), dict(type=-1), dict(eps=-1.0), dict(eps=math.nan),
           dict(x=None), dict(x=P + 8), dict(w=None), dict(w=P + 2), dict(q=P + 8), dict(q=None), dict(s=None), dict(s=P + 2),
           dict(ldx=63), dict(ldx=68), dict(ldx=0), dict(r=P, ldr=32), dict(r=P + 4, ldr=64), dict(sum=P + 16, lds=12),
           dict(sum=P, lds=128), dict(r=P + 4096, ldr=64, sum=P + 4096, lds=72)]
    for b in bad:
        v = {**norm, **b}
        assert lib.moe_add_rmsnorm_fp8(c, v["T"], v["d"], v["type"], v["x"], v["ldx"], v["r"], v["ldr"], v["w"], v["eps"],
                                       v["sum"], v["lds"], v["q"], v["s"], None) == moe.MOE_ERR_ARG, b
    mm = dict(M=4, N=8, K=64, a=P, lda=64, sa=P, b=P, sb=P, bias=None, r=None, ldr=0, c=P, ldc=8, type=0)
    bad = [dict(M=-1), dict(N=0), dict(K=0), dict(K=8), dict(K=72), dict(a=None), dict(a=P + 8), dict(lda=48), dict(lda=72),
           dict(lda=1 << 40), dict(sa=None), dict(b=None), dict(b=P + 1), dict(sb=P + 1), dict(bias=P + 1), dict(c=None),
           dict(c=P + 1), dict(ldc=7), dict(type=7), dict(r=P + 64, ldr=7), dict(r=P + 1, ldr=8), dict(r=P, ldr=16)]
    for b in bad:
        v = {**mm, **b}
        assert lib.moe_fp8_matmul(c, v["M"], v["N"], v["K"], v["a"], v["lda"], v["sa"], v["b"], v["sb"], v["bias"], v["r"],
                                  v["ldr"], v["c"], v["ldc"], v["type"], None) == moe.MOE_ERR_ARG, b
    g = dict(M=4, F=32, K=64, a=P, lda=64, sa=P, b=P, sb=P, bias=None, alpha=1.0, limit=7.0, shift=1.0, h=P, hs=P)
    bad = [dict(F=0), dict(F=40), dict(K=24), dict(M=-2), dict(limit=0.0), dict(limit=-1.0), dict(limit=math.nan),
           dict(alpha=math.nan), dict(shift=math.nan), dict(alpha=math.inf), dict(shift=-math.inf), dict(h=None), dict(h=P + 4), dict(hs=P + 2), dict(b=P + 4), dict(lda=56)]
    for b in bad:
        v = {**g, **b}
        assert lib.moe_fp8_gated_matmul(c, v["M"], v["F"], v["K"], v["a"], v["lda"], v["sa"], v["b"], v["sb"], v["bias"],
                                        v["alpha"], v["limit"], v["shift"], v["h"], v["hs"], None) == moe.MOE_ERR_ARG, b
    # no rows: nothing to do, whatever the pointers are
    assert lib.moe_add_rmsnorm_fp8(c, 0, 64, 0, None, 0, None, 0, None, 1e-5, None, 0, None, None, None) == moe.MOE_OK
    assert lib.moe_fp8_matmul(c, 0, 8, 64, None, 0, None, None, None, None, None, 0, None, 0, 0, None) == moe.MOE_OK
    assert lib.moe_fp8_gated_matmul(c, 0, 32, 64, None, 0, None, None, None, None, 1.0, 7.0, 1.0, None, None, None) == moe.MOE_OK


def test_alpha_past_the_range_of_its_exponent_is_refused(lib):
    """The exponent is alpha log2(e) g in fp32: where alpha log2(e) is no number, 0 times it would not be 0."""
    c, P = ctypes.byref(Ctx(0, 148, None, 1)), 1 << 20
    for alpha in (2.0 ** 127 * 1.5, -2.0 ** 127 * 1.5, 3.4e38):
        assert lib.moe_fp8_gated_matmul(c, 4, 32, 64, P, 64, P, P, P, None, alpha, 7.0, 1.0, P, P, None) == moe.MOE_ERR_ARG
    # (no rows: nothing else to check)
    assert lib.moe_fp8_gated_matmul(c, 0, 32, 64, None, 64, None, None, None, None, 2.0 ** 127, 7.0, 1.0, None, None, None) == moe.MOE_OK


def test_wait_limits_shorter_than_a_drain_are_refused(lib):
    """A CTA whose wait ran out waits as long again for its copies in flight: a limit of microseconds would let it
    leave before they land."""
    c = Ctx(0, 148, None, 2_000_000_000)
    for ns in (0, 1, 1000, 999_999):
        assert lib.moe_fp8_set_wait_limit_ns(ctypes.byref(c), ns) == moe.MOE_ERR_ARG
        assert c.limit == 2_000_000_000
    for ns in (1_000_000, 2_000_000, 1 << 62):
        assert lib.moe_fp8_set_wait_limit_ns(ctypes.byref(c), ns) == moe.MOE_OK
        assert c.limit == ns


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("M", [1, 7, 8, 9, 32, 64, 65, 128, 129, 255, 333, 1000, 2048, 8192, 100000])
def test_plans_fit_and_cover(lib, gated, M):
    """Whatever the sizes: the rings (and a split tile's sums) fit the shared memory, two MMA warps taking every
    other K block keep to their own stages, the tiles cover every row and column, every CTA of a cluster that splits
    K has a block, and the clusters of a split are all resident."""
    for N in (16, 48, 128, 144, 1360, 2880, 5120, 20000):
        for K in (16, 128, 144, 2880, 6144):
            pl = moe.moe_fp8_debug_plan(gated, M, N, K, 148)
            assert pl["smem_needed"] <= 227 * 1024 and 2 <= pl["n_stages"] <= 16
            assert pl["bn"] == 256 or pl["n_stages"] % 2 == 0
            assert pl["a_rows"] % 8 == 0 and (pl["a_rows"] == 128 or M <= pl["a_rows"] < 128 and pl["m_tiles"] == 1)
            assert pl["m_tiles"] * 128 * pl["ctas"] >= M > (pl["m_tiles"] - 1) * 128 * pl["ctas"]
            n_tiles = pl["tiles"] // pl["m_tiles"]
            assert n_tiles * pl["m_tiles"] == pl["tiles"]
            width = 128 if gated else pl["bn"]
            assert n_tiles * width >= N > (n_tiles - 1) * width
            assert pl["ctas"] in (1, 2) and 1 <= pl["split"] <= min(8, -(-K // 128)) and (pl["ctas"] == 1 or pl["split"] == 1)
            if pl["split"] > 1:
                assert pl["grid"] == pl["tiles"] * pl["split"] <= 148
            else:
                assert pl["grid"] % pl["ctas"] == 0 and pl["grid"] // pl["ctas"] <= pl["tiles"]
            assert not pl["few"] or M <= 16


def test_gated_form_that_measured_faster(lib):
    """Pairs or K split, at the sizes whose times stand beside the rule."""
    for form, sizes in (("pair", [(256, 2880, 512), (333, 1360, 1552), (512, 2880, 2880), (2000, 272, 1040)]),
                        ("split", [(260, 1360, 2880), (256, 2880, 6144), (1200, 256, 2880), (64, 2880, 2880)])):
        for s in sizes:
            assert (moe.moe_fp8_debug_plan(True, *s, 148)["ctas"] == 2) == (form == "pair"), s


def test_gpu_sizes_cover_every_form(lib):
    """The sizes of the GPU tests run every kernel: the one for a few rows, pairs, single tiles, split K (and, gated,
    a split tile with one CTA), each with ragged rows and columns."""
    import importlib.util
    import os
    spec = importlib.util.spec_from_file_location("gpu_fp8", os.path.join(os.path.dirname(__file__), "test_gpu_fp8.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)

    def form(gated, size):
        pl = moe.moe_fp8_debug_plan(gated, *size, 148)
        return "few" if pl["few"] else "pair" if pl["ctas"] == 2 else "split" if pl["split"] > 1 else "single"

    for gated, sizes in ((False, mod.SIZES), (False, mod.RES_SIZES), (True, mod.GATED_SIZES)):
        forms = {form(gated, s) for s in sizes if s[0] % 128 and s[1] % 128}
        assert forms == {"few", "pair", "single", "split"}, (gated, forms)


def test_plan_rejects_bad_arguments(lib):
    out = (ctypes.c_int * 10)()
    for args in [(0, 0, 8, 64, 148), (0, 1, 0, 64, 148), (0, 1, 8, 60, 148), (0, 1, 8, 64, 0), (1, 1, 24, 64, 148),
                 (0, 2 ** 31 - 1, 2 ** 31 - 1, 64, 148)]:
        assert lib.moe_fp8_debug_plan(*args, out) == moe.MOE_ERR_ARG, args
    assert lib.moe_fp8_debug_plan(0, 1, 8, 64, 148, None) == moe.MOE_ERR_ARG


@pytest.mark.parametrize("M,K", [(1, 16), (5, 130), (200, 300)])
def test_quantisers(M, K):
    """A code times its scale is within half a step of the element; the scale is the block's maximum over 448."""
    x = torch.randn(M, K, generator=torch.Generator().manual_seed(K)) * 3
    x[0, :16] = 0
    for (q, s), rows in ((moe.quantize_fp8_rows(x), 1), (moe.quantize_fp8_weight(x), 128)):
        assert q.dtype == torch.float8_e4m3fn and q.shape == (M, K) and q.is_contiguous()
        assert s.shape == (-(-M // rows), -(-K // 128)) and s.dtype == torch.float32
        for i in range(s.shape[0]):
            for j in range(s.shape[1]):
                b = x[i * rows:(i + 1) * rows, 128 * j:128 * (j + 1)].double()
                v = q[i * rows:(i + 1) * rows, 128 * j:128 * (j + 1)].double() * s[i, j].double()
                assert abs(s[i, j].double() - max(b.abs().max() / 448, 2.0 ** -126)) <= 2.0 ** -23 * s[i, j].double()
                assert ((v - b).abs() <= b.abs() * (2.0 ** -4 + 2.0 ** -22) + s[i, j].double() * 2.0 ** -10).all()


def test_build_goes_on_without_the_binding(lib, monkeypatch, tmp_path):
    """Where the binding cannot be built the library is there all the same, and the operators that need the binding
    say why they are not."""
    for e in (FileNotFoundError("g++"), ModuleNotFoundError("No module named 'torch'"), subprocess.CalledProcessError(1, "g++")):
        def fails(*_, e=e, **__):
            raise e
        monkeypatch.setattr(moe_build, "build_binding", fails)
        with pytest.warns(UserWarning, match="torch binding"):
            assert moe_build.build() == moe_build.LIB
    monkeypatch.undo()
    from sparse_moe_rmsnorm_b200 import fp8
    monkeypatch.setattr(fp8, "_binding_module", None)
    monkeypatch.setitem(sys.modules, "sparse_moe_rmsnorm_b200._binding", None)
    with pytest.raises(RuntimeError, match="build.*None in sys.modules"):
        fp8._binding()


def test_binding_of_another_torch_is_built_again(lib, monkeypatch, tmp_path):
    """A binding is kept only for the torch that it was built for, whatever the files' times are."""
    import importlib.metadata
    before = os.stat(moe_build.BINDING).st_mtime_ns
    assert moe_build.build_binding() == moe_build.BINDING and os.stat(moe_build.BINDING).st_mtime_ns == before
    copy = tmp_path / "_binding.so"
    built = open(moe_build.BINDING, "rb").read()
    copy.write_bytes(built)
    monkeypatch.setattr(moe_build, "BINDING", str(copy))
    ran = []
    monkeypatch.setattr(moe_build.subprocess, "run", lambda cmd, **_: (ran.append(cmd), open(cmd[cmd.index("-o") + 1], "wb").close()))
    moe_build.build_binding()
    assert not ran
    have = importlib.metadata.version("torch")
    for other in ("0.0.1", have + "0", have[:-1]):
        monkeypatch.setattr(moe_build.importlib.metadata, "version", lambda name, other=other: other)
        moe_build.build_binding()
        assert len(ran) == 1 and any(other in word for word in ran.pop())
        copy.write_bytes(built)


@pytest.mark.parametrize("M,K", [(0, 272), (0, 128), (3, 0), (0, 0)])
def test_quantisers_of_nothing(M, K):
    """An empty batch's rows and scales, as the operators take and give them."""
    for quantise, rows in ((moe.quantize_fp8_rows, 1), (moe.quantize_fp8_weight, 128)):
        q, s = quantise(torch.empty(M, K, dtype=torch.bfloat16))
        assert q.shape == (M, K) and q.dtype == torch.float8_e4m3fn
        assert s.shape == (-(-M // rows), -(-K // 128)) and s.dtype == torch.float32


def test_stream_of_another_device_is_refused():
    """Its calls would run on the operators' device's current stream instead."""
    import types
    ops = object.__new__(moe.Fp8Ops)
    ops.device, ops.ctx = torch.device("cuda", 0), None
    with pytest.raises(moe.MoEError):
        ops._on(types.SimpleNamespace(device=torch.device("cuda", 1)))
