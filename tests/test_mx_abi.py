"""MXFP4 on the CPU: the oracle against hand values and a second reading of
the format, and what the entry points refuse before any HIP call."""
import numpy as np
import pytest

from oracle import mxref

qgm = pytest.importorskip("bit_weight_only_dequant_amd")
torch = pytest.importorskip("torch")
lib = qgm._lib

OK, E_ARG, E_UNSUP, E_ALIGN, E_DEVICE = 0, 1, 2, 3, 4
A = 0x10000   # an aligned fake address: validation never dereferences it
F16, BF16, F32, FP4 = 0, 1, 2, 3


def gpu_present():
    return torch.cuda.is_available()


# ---------------------------------------------------------------- the oracle

def block(*head):
    v = np.zeros((1, 32))
    v[0, :len(head)] = head
    return v


def test_oracle_hand_values():
    # largest magnitude 6: scale 2^0; every value of the format is itself
    codes, scales = mxref.mx_quantize(block(6, 4, 3, 2, 1.5, 1, 0.5, 0, -0.5, -6))
    assert scales[0, 0] == 127
    assert list(codes[0, :5]) == [7 | 6 << 4, 5 | 4 << 4, 3 | 2 << 4, 1 | 0 << 4, 9 | 15 << 4]
    # ties go to the even code: 0.25 -> 0, 0.75 -> 1, 1.25 -> 1, 1.75 -> 2, 2.5 -> 2, 3.5 -> 4, 5 -> 4
    codes, scales = mxref.mx_quantize(block(4, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5))
    assert list(mxref.mx_values(codes, scales)[0, :8]) == [4, 0, 1, 1, 2, 2, 4, 4]
    # 7.9: the scale follows the exponent of the largest, the value saturates at 6
    codes, scales = mxref.mx_quantize(block(7.9, 1))
    assert scales[0, 0] == 127 and mxref.mx_values(codes, scales)[0, 0] == 6
    codes, scales = mxref.mx_quantize(block(8.0))
    assert scales[0, 0] == 128 and mxref.mx_values(codes, scales)[0, 0] == 8


def test_oracle_edges():
    assert mxref.mx_quantize(block())[1][0, 0] == 0
    tiny = 2.0 ** -149
    codes, scales = mxref.mx_quantize(block(tiny))
    assert scales[0, 0] == 0 and codes[0, 0] == 0             # 2^-22 of the smallest scale
    codes, scales = mxref.mx_quantize(block(2.0 ** -127))
    assert scales[0, 0] == 0 and codes[0, 0] == 2
    for bad in (np.inf, -np.inf, np.nan):
        codes, scales = mxref.mx_quantize(block(1, bad, 2))
        assert scales[0, 0] == 255 and not codes.any()
        assert np.isnan(mxref.mx_values(codes, scales)).all()
    codes, _ = mxref.mx_quantize(block(1.0, -0.0, -1e-9))
    assert codes[0, 0] >> 4 == 8 and codes[0, 1] & 15 == 8    # the sign stays on a zero


def test_oracle_rounding_by_exhaustion():
    # a step's half at most away, and no other value nearer
    rng = np.random.default_rng(0)
    x = rng.standard_normal((64, 96)) * np.exp2(rng.integers(-30, 30, (64, 1)))
    codes, scales = mxref.mx_quantize(x)
    v = mxref.mx_values(codes, scales).reshape(64, 3, 32)
    unit = np.exp2(scales.astype(float) - 127)[:, :, None]
    grid = np.concatenate([mxref.VALUES, -mxref.VALUES]) * unit[..., None]
    best = np.abs(x.reshape(64, 3, 32, 1) - grid).min(axis=-1)
    assert np.array_equal(np.abs(x.reshape(64, 3, 32) - v), best)


def test_oracle_products_by_loops():
    rng = np.random.default_rng(1)
    wc, wsc = mxref.mx_quantize(rng.standard_normal((2 * 3, 64)))
    w = mxref.mx_values(wc, wsc).reshape(2, 3, 64)
    x = rng.standard_normal((4, 64))
    y, a = mxref.mx_gemm_ref(x, w[0], residual=np.ones((4, 3)))
    for m in range(4):
        for n in range(3):
            assert abs(y[m, n] - 1 - sum(x[m, k] * w[0, n, k] for k in range(64))) < 1e-12
            assert a[m, n] >= abs(y[m, n])
    y, _ = mxref.mx_grouped_ref(x, w, [0, 1, 3], rows=[2, -1, 2, 0], row_scale=[2.0, 1, 3.0, 1], fill=7)
    assert np.allclose(y[0], 2 * w[0] @ x[2]) and not y[1].any()
    assert np.allclose(y[2], 3 * w[1] @ x[2]) and (y[3] == 7).all()


# ------------------------------------------------------------- the refusals

def quantize(x=A, ldx=None, xt=F16, M=2, K=64, codes=A, scales=A):
    return lib.qmx_quantize(x, K if ldx is None else ldx, xt, M, K, codes, scales, None)


def dequantize(y=A, ldy=None, yt=F16, M=2, K=64, codes=A, scales=A):
    return lib.qmx_dequantize(codes, scales, M, K, y, K if ldy is None else ldy, yt, None)


def gemm(x=A, ldx=None, xt=F16, xs=None, w=A, ws=A, res=None, ldr=None, M=2, N=16, K=64, y=A, ldy=None, yt=F16):
    return lib.qmx_gemm(x, K if ldx is None else ldx, xt, xs, w, ws, res, N if ldr is None else ldr, M, N, K, y,
                        N if ldy is None else ldy, yt, None)


def grouped(x=A, ldx=None, xt=F16, xs=None, xr=8, rows=A, w=A, ws=A, off=A, E=3, T=8, rsc=None, N=16, K=64, y=A,
            ldy=None, yt=F16):
    return lib.qmx_gemm_grouped(x, K if ldx is None else ldx, xt, xs, xr, rows, w, ws, off, E, T, rsc, N, K, y,
                                N if ldy is None else ldy, yt, None)


@pytest.mark.parametrize("kw,expect", [
    (dict(xt=FP4), E_ARG), (dict(xt=-1), E_ARG), (dict(xt=4), E_ARG), (dict(M=-1), E_ARG), (dict(K=-32), E_ARG),
    (dict(K=48), E_ARG), (dict(x=None), E_ARG), (dict(codes=None), E_ARG), (dict(scales=None), E_ARG),
    (dict(ldx=32), E_ARG), (dict(x=A + 2), E_ALIGN), (dict(codes=A + 8), E_ALIGN), (dict(ldx=68), E_ALIGN),
    (dict(M=0, x=None), OK), (dict(K=0, codes=None), OK)])
def test_quantize_refuses(kw, expect):
    assert quantize(**kw) == expect
    kw = {{"x": "y", "xt": "yt", "ldx": "ldy"}.get(k, k): v for k, v in kw.items()}
    assert dequantize(**kw) == expect


PRODUCT_REFUSALS = [
    (dict(xt=F32), E_ARG), (dict(xt=9), E_ARG), (dict(yt=FP4), E_ARG), (dict(yt=-1), E_ARG), (dict(N=-1), E_ARG),
    (dict(K=-32), E_ARG), (dict(K=40), E_ARG), (dict(x=None), E_ARG), (dict(w=None), E_ARG), (dict(ws=None), E_ARG),
    (dict(y=None), E_ARG), (dict(ldx=32), E_ARG), (dict(ldy=15), E_ARG), (dict(xs=A), E_ARG),
    (dict(xt=FP4), E_ARG), (dict(xt=FP4, xs=A, ldx=96), E_ARG), (dict(x=A + 8), E_ALIGN), (dict(w=A + 4), E_ALIGN),
    (dict(y=A + 2), E_ALIGN), (dict(ldx=68), E_ALIGN), (dict(N=0, y=None), OK)]


@pytest.mark.parametrize("kw,expect", PRODUCT_REFUSALS + [
    (dict(M=-1), E_ARG), (dict(res=A, ldr=8), E_ARG), (dict(res=A, ldr=32), E_ARG), (dict(res=A + 2), E_ALIGN),
    (dict(M=0, x=None), OK)])
def test_gemm_refuses(kw, expect):
    assert gemm(**kw) == expect


@pytest.mark.parametrize("kw,expect", PRODUCT_REFUSALS + [
    (dict(T=-1), E_ARG), (dict(E=-1), E_ARG), (dict(xr=-1), E_ARG), (dict(off=None), E_ARG),
    (dict(rows=None, xr=7), E_ARG), (dict(off=A + 2), E_ALIGN), (dict(rows=A + 1), E_ALIGN),
    (dict(rsc=A + 2), E_ALIGN), (dict(E=65536), E_UNSUP), (dict(T=0, x=None), OK), (dict(E=0), OK)])
def test_grouped_refuses(kw, expect):
    assert grouped(**kw) == expect


@pytest.mark.parametrize("tile,call", [
    (None, lambda: gemm(xt=BF16, M=1 << 30, N=16, K=32)), (None, lambda: gemm(xt=F16, M=(1 << 31) - 600, N=4, K=64)),
    (0, lambda: gemm(M=65535 * 16 + 1)), (1, lambda: gemm(xt=FP4, xs=A, M=1 << 30)),
    (1, lambda: gemm(M=1 << 18, N=1 << 18)), (4, lambda: gemm(xt=BF16, M=1 << 19, N=1 << 19)),
    (4, lambda: gemm(xt=FP4, xs=A, M=1 << 20, N=1 << 19)), (2, lambda: grouped(T=1 << 30, E=5)),
    (None, lambda: grouped(xt=BF16, T=(1 << 30) + 7, xr=1 << 30, E=1)), (None, lambda: grouped(K=0, N=1 << 30)),
    (None, lambda: grouped(xr=0, x=None, N=(1 << 30) - 15)), (None, lambda: gemm(M=(1 << 31) - 1)),
    (None, lambda: gemm(N=(1 << 31) - 512)), (None, lambda: grouped(T=(1 << 31) - 100))])
def test_more_than_a_grid_holds(monkeypatch, tile, call):
    if tile is not None:
        monkeypatch.setenv("QMX_TILE", str(tile))
    assert call() == E_UNSUP


@pytest.mark.skipif(gpu_present(), reason="checks the no-device status; a GPU is present")
@pytest.mark.parametrize("tile,call", [
    (None, lambda: gemm(xt=FP4, xs=A, M=(1 << 30) + 70, N=16, K=32)), (None, lambda: gemm(M=1 << 22, K=0)),
    (0, lambda: gemm(M=65535 * 16)), (1, lambda: gemm(M=(1 << 18) - 64, N=1 << 18)),
    (4, lambda: gemm(xt=FP4, xs=A, M=(1 << 20) - 256, N=1 << 19)), (None, lambda: grouped(K=0, N=(1 << 30) - 16)),
    (None, lambda: gemm(M=(1 << 31) - 600, K=0))])
def test_what_a_grid_holds_comes_to_the_device(monkeypatch, tile, call):
    if tile is not None:
        monkeypatch.setenv("QMX_TILE", str(tile))
    assert call() == E_DEVICE


@pytest.mark.skipif(gpu_present(), reason="checks the no-device status; a GPU is present")
def test_no_device_status():
    assert quantize() == E_DEVICE and dequantize() == E_DEVICE
    assert gemm() == E_DEVICE and gemm(xt=FP4, xs=A + 1) == E_DEVICE
    assert grouped() == E_DEVICE and grouped(xr=0, x=None) == E_DEVICE


def test_plans(monkeypatch):
    plan = qgm.mx_plan
    # few rows: a wave for each chunk of 512 k, at most 16 and what LDS holds
    assert plan(1, 6144, 2048, F16) == dict(tile=0, blocks=1, waves=4, pieces=384)
    assert plan(8, 2048, 8192, BF16) == dict(tile=0, blocks=1, waves=16, pieces=128)
    assert plan(16, 8192, 8192, BF16)["waves"] == 8 and plan(16, 8192, 8192, BF16)["blocks"] == 2
    assert plan(16, 8192, 8192, FP4)["waves"] == 16
    assert plan(1, 64, 96, BF16)["waves"] == 1 and plan(1, 64, 0, BF16)["tile"] == 0
    # larger tiles as the rows grow
    tiles = [plan(m, 8192, 8192, BF16)["tile"] for m in (1, 64, 512, 4096)]
    assert tiles[0] == 0 and tiles == sorted(tiles) and tiles[-1] == 4
    assert plan(4096, 8192, 8192, FP4) == dict(tile=4, blocks=0, waves=0, pieces=512)
    assert plan(32, 2048, 2048, BF16, groups=32)["tile"] == 0
    assert plan(16384, 4096, 2048, BF16, groups=32)["tile"] > 1
    # the rows kernel's grid has 65535 blocks of 16 rows
    assert plan(1 << 21, 16, 32, BF16)["tile"] > 0
    for v in range(5):
        monkeypatch.setenv("QMX_TILE", str(v))
        assert plan(100, 300, 512, F16)["tile"] == v
    out = (qgm.ctypes.c_int * 4)()
    for bad in ((-1, 1, 32, 0, 0), (1, -1, 32, 0, 0), (1, 1, 40, 0, 0), (1, 1, 32, -1, 0), (1, 1, 32, 0, F32)):
        assert lib.qmx_plan(*bad, out) == E_ARG
    assert lib.qmx_plan(1, 1, 32, 0, 0, None) == E_ARG


@pytest.mark.parametrize("x_type", [F16, BF16, FP4])
@pytest.mark.parametrize("groups", [0, 1, 4, 65535])
@pytest.mark.parametrize("M,N", [(0, 16), (16, 0), (0, 0)])
def test_plan_of_nothing(M, N, groups, x_type):
    for K in (0, 64, 8192):
        assert qgm.mx_plan(M, N, K, x_type, groups=groups) == dict(tile=0, blocks=1, waves=1, pieces=0)


def test_plan_limits():
    # what the products refuse by their sizes alone; the largest they take has a plan, grouped or not
    out = (qgm.ctypes.c_int * 4)()
    top = (1 << 31) - 1
    for bad in ((1 << 29, 16, 64, 1 << 29, BF16), (1, 16, 64, 65536, F16), (top, 16, 64, 0, FP4), (16, top, 64, 0, F16)):
        assert lib.qmx_plan(*bad, out) == E_UNSUP
    for M, E in ((1, 65535), (1 << 29, 65535), (top - 512, 65535), (top - 512, 1), (top - 512, 0)):
        for x_type in (F16, BF16, FP4):
            assert lib.qmx_plan(M, 16, 64, E, x_type, out) == OK and out[3] > 0


def test_binding_refuses_sizes_and_strides_past_32_bits(monkeypatch):
    """Before the library is called: a stride, a number of rows or a length that 32 bits cut off would read as a
    small one there.  Tensors without memory stand for the large ones."""
    class Never:
        def __getattr__(self, name):
            raise AssertionError(f"{name} was called")
    monkeypatch.setattr(qgm, "_lib", Never())
    monkeypatch.setattr(qgm, "_mx_elsewhere", lambda x, stream: None)
    monkeypatch.setattr(qgm, "_dev", lambda t, what: t)

    def t(shape, dtype=torch.float16, stride=None):
        return torch.empty_strided(shape, stride or [int(np.prod(shape[i + 1:])) for i in range(len(shape))],
                                   dtype=dtype, device="meta")
    u8, i32, f32 = torch.uint8, torch.int32, torch.float32

    def mx(*shape):
        return t((*shape[:-1], shape[-1] // 2), u8), t((*shape[:-1], shape[-1] // 32), u8)
    big = 1 << 32
    few, far, many, wide = t((2, 64)), t((2, 64), stride=(big + 64, 1)), t((big + 2, 64)), t((1, big + 64))
    w, ws = mx(64, 64)
    gw, gs = mx(3, 64, 64)
    off = t((4,), i32)
    calls = [
        lambda: qgm.mx_quantize(far), lambda: qgm.mx_quantize(many), lambda: qgm.mx_quantize(wide),
        lambda: qgm.mx_quantize(t((2, 64), stride=(1 << 31, 1))), lambda: qgm.mx_quantize(t((1 << 31, 64))),
        lambda: qgm.mx_dequantize(*mx(2, 64), out=far), lambda: qgm.mx_dequantize(*mx(big + 2, 64)),
        lambda: qgm.mx_dequantize(*mx(1, big + 64)),
        lambda: qgm.mx_gemm(far, w, ws), lambda: qgm.mx_gemm(many, w, ws), lambda: qgm.mx_gemm(few, w, ws, out=far),
        lambda: qgm.mx_gemm(few, w, ws, residual=far), lambda: qgm.mx_gemm(few, *mx(big + 3, 64)),
        lambda: qgm.mx_gemm(wide, *mx(3, big + 64)), lambda: qgm.mx_gemm(mx(big + 2, 64)[0], w, ws, x_scales=mx(big + 2, 64)[1]),
        lambda: qgm.mx_gemm_grouped(far, gw, gs, off), lambda: qgm.mx_gemm_grouped(many, gw, gs, off),
        lambda: qgm.mx_gemm_grouped(few, gw, gs, off, out=far), lambda: qgm.mx_gemm_grouped(few, gw, gs, off, rows=t((big + 2,), i32)),
        lambda: qgm.mx_gemm_grouped(few, *mx(big + 3, 0, 64), t((big + 4,), i32)),
        lambda: qgm.MXLinear(*mx(big + 3, 64)),
        lambda: qgm.mx_plan(big + 1, 16, 64, BF16), lambda: qgm.mx_plan(1, big + 16, 64, BF16),
        lambda: qgm.mx_plan(1, 16, big + 64, BF16), lambda: qgm.mx_plan(1, 16, 64, BF16, groups=big + 1),
    ]
    for call in calls:
        with pytest.raises(ValueError, match="2147483647"):
            call()
    monkeypatch.undo()
    with pytest.raises(qgm.QGemmError):
        qgm.mx_plan(-1, 16, 64, BF16)


def test_binding_refuses_cpu_tensors():
    x = torch.zeros(2, 64, dtype=torch.float16)
    c, s = torch.zeros(2, 32, dtype=torch.uint8), torch.zeros(2, 2, dtype=torch.uint8)
    off = torch.zeros(2, dtype=torch.int32)
    for call in (lambda: qgm.mx_quantize(x), lambda: qgm.mx_dequantize(c, s), lambda: qgm.mx_gemm(x, c, s),
                 lambda: qgm.mx_gemm_grouped(x, c[None], s[None], off), lambda: qgm.MXLinear(c, s),
                 lambda: qgm.MXLinear.from_weight(x)):
        with pytest.raises(ValueError, match="GPU"):
            call()
