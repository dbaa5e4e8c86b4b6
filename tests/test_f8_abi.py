"""8-bit floating point with blocks of 128 on the CPU: the oracle against hand
values and a second reading of the format, and what the entry points refuse
before any HIP call."""
from fractions import Fraction

import numpy as np
import pytest

from oracle import f8ref

qgm = pytest.importorskip("bit_weight_only_dequant_amd")
torch = pytest.importorskip("torch")
lib = qgm._lib

OK, E_ARG, E_UNSUP, E_ALIGN, E_DEVICE = 0, 1, 2, 3, 4
A = 0x10000   # an aligned fake address: validation never dereferences it
F16, BF16, F32, FP4, F8 = 0, 1, 2, 3, 4


def gpu_present():
    return torch.cuda.is_available()


# ---------------------------------------------------------------- the oracle

def test_oracle_values_are_the_formats():
    t = torch.arange(256, dtype=torch.int16).to(torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(f8ref.VALUES, t, equal_nan=True)
    assert f8ref.VALUES[126] == 448 and f8ref.VALUES[1] == 2.0 ** -9 and f8ref.VALUES[8] == 2.0 ** -6


def test_oracle_hand_values():
    # largest magnitude 448: scale 1, every value of the format is itself
    x = np.zeros((1, 128))
    x[0, :8] = [448, 1, -1.125, 2.0 ** -9, 0.0, -0.0, 17, 19]
    codes, scales = f8ref.f8_quantize(x)
    assert scales[0, 0] == 1
    # 17 lies midway between 16 (code 88) and 18 (89): the even code; 19 between 18 and 20 (90)
    assert list(codes[0, :8]) == [126, 56, 185, 1, 0, 128, 88, 90]
    # half the smallest subnormal goes to 0, more than that up
    x[0, 1:4] = [2.0 ** -10, 2.0 ** -10 * 1.001, 3 * 2.0 ** -10]
    assert list(f8ref.f8_quantize(x)[0][0, 1:4]) == [0, 1, 2]


def test_oracle_rounding_in_rationals():
    # by exact arithmetic: no code is nearer to 448 v / A, and of two as near the even one is taken
    rng = np.random.default_rng(0)
    x = rng.standard_normal((3, 128)).astype(np.float32)
    x[1] = rng.integers(-224, 225, 128)        # A = 224: 448 v / A = 2 v, many middles
    x[1, 0] = 224
    codes, _ = f8ref.f8_quantize(x)
    grid = [f8ref.code_value(b) for b in range(127)]
    ties = 0
    for r in range(3):
        a = max(Fraction(float(abs(v))) for v in x[r])
        for k in range(128):
            q = abs(Fraction(float(x[r, k]))) * 448 / a
            best = min(abs(q - v) for v in grid)
            near = [b for b in range(127) if abs(q - grid[b]) == best]
            ties += len(near) == 2
            want = near[0] if len(near) == 1 else [b for b in near if b % 2 == 0][0]
            assert codes[r, k] == want + (128 if np.signbit(x[r, k]) else 0)
    assert ties > 5


def test_oracle_blocks_edges_and_transpose():
    rng = np.random.default_rng(1)
    x = rng.standard_normal((130, 144))
    x[5, 3], x[129, 143] = np.inf, np.nan
    c, s = f8ref.f8_quantize(x, 128)
    assert c.shape == (130, 144) and s.shape == (2, 2)
    assert np.isnan(s[0, 0]) and not c[:128, :128].any() and np.isnan(s[1, 1]) and np.isfinite(s[0, 1])
    ct, st = f8ref.f8_quantize(x, 128, transpose=True)
    assert ct.shape == (144, 144) and np.array_equal(ct[:, :130], c.T) and not ct[:, 130:].any()
    assert np.array_equal(st, s.T, equal_nan=True)
    c1, s1 = f8ref.f8_quantize(x, 1, transpose=True)
    assert c1.shape == (144, 144) and s1.shape == (144, 2)
    assert np.isclose(s1[7, 0], np.abs(x[:128, 7]).max() / 448) and np.isclose(s1[7, 1], np.abs(x[128:, 7]).max() / 448)
    z, zs = f8ref.f8_quantize(np.zeros((1, 16)))
    assert not z.any() and zs[0, 0] == np.float32(2.0 ** -100 / 448)
    assert np.isnan(f8ref.f8_values(c, s)[:128, :128]).all()
    assert np.abs(f8ref.f8_values(*f8ref.f8_quantize(rng.standard_normal((4, 256)))).max()) < 6


def test_oracle_products_by_loops():
    rng = np.random.default_rng(2)
    wc, ws = f8ref.f8_quantize(rng.standard_normal((2 * 16, 144)), 128)
    w = f8ref.f8_values(wc, ws)
    for n in range(32):
        for k in (0, 127, 128, 143):
            assert w[n, k] == f8ref.VALUES[wc[n, k]] * np.float64(ws[0, k // 128])
    x = rng.standard_normal((3, 144))
    y, a = f8ref.f8_gemm_ref(x, w, residual=np.ones((3, 32)))
    assert abs(y[2, 5] - 1 - sum(x[2, k] * w[5, k] for k in range(144))) < 1e-12 and a[2, 5] >= abs(y[2, 5])


@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
def test_oracle_gate_and_its_gradient(act):
    g = torch.linspace(-12, 12, 97, dtype=torch.float64, requires_grad=True)
    ref = torch.nn.functional.silu(g) if act == "silu" else torch.nn.functional.gelu(g, approximate="tanh")
    slope, = torch.autograd.grad(ref.sum(), g)
    a, da = f8ref.act_ref(g.detach().numpy(), act)
    assert np.allclose(a, ref.detach().numpy(), atol=1e-13) and np.allclose(da, slope.numpy(), atol=1e-13)
    # the block's gradients against differences
    rng = np.random.default_rng(3)
    x, w, dh = rng.standard_normal((4, 16)), rng.standard_normal((2 * 5, 16)), rng.standard_normal((4, 5))
    d = f8ref.gated_grad_ref(dh, x, w, act)
    dx, dw = d @ w, d.T @ x
    f = lambda x, w: (f8ref.gated_ref(x, w, act)[0] * dh).sum()  # noqa: E731
    e = 1e-6
    for m, k in ((0, 0), (3, 15), (2, 7)):
        up, down = x.copy(), x.copy()
        up[m, k] += e
        down[m, k] -= e
        assert abs((f(up, w) - f(down, w)) / (2 * e) - dx[m, k]) < 1e-6 * (1 + abs(dx[m, k]))
    for n, k in ((0, 0), (4, 3), (5, 1), (9, 15)):
        up, down = w.copy(), w.copy()
        up[n, k] += e
        down[n, k] -= e
        assert abs((f(x, up) - f(x, down)) / (2 * e) - dw[n, k]) < 1e-6 * (1 + abs(dw[n, k]))


# ------------------------------------------------------------- the refusals

def quantize(x=A, ldx=None, xt=F16, M=2, K=64, block=1, turn=0, codes=A, scales=A):
    return lib.qf8_quantize(x, K if ldx is None else ldx, xt, M, K, block, turn, codes, scales, None)


def dequantize(codes=A, scales=A, block=1, M=2, K=64, y=A, ldy=None, yt=F16):
    return lib.qf8_dequantize(codes, scales, block, M, K, y, K if ldy is None else ldy, yt, None)


def gemm(x=A, ldx=None, xt=F16, xs=None, w=A, ws=A, block=128, res=None, ldr=None, M=2, N=16, K=64, y=A, ldy=None, yt=F16):
    return lib.qf8_gemm(x, K if ldx is None else ldx, xt, xs, w, ws, block, res, N if ldr is None else ldr, M, N, K, y,
                        N if ldy is None else ldy, yt, None)


def gated(x=A, ldx=None, xt=F16, xs=None, w=A, ws=A, act=0, M=2, N=16, K=64, y=A, ldy=None, yt=F16):
    return lib.qf8_gated(x, K if ldx is None else ldx, xt, xs, w, ws, act, M, N, K, y, N if ldy is None else ldy, yt, None)


def grad(dh=2 * A, ldd=None, x=A, ldx=None, xt=F16, xs=None, w=A, ws=A, act=0, M=2, N=16, K=64, y=A, ldy=None, yt=F16):
    return lib.qf8_gated_grad(dh, N if ldd is None else ldd, x, K if ldx is None else ldx, xt, xs, w, ws, act, M, N, K, y,
                              2 * N if ldy is None else ldy, yt, None)


@pytest.mark.parametrize("kw,expect", [
    (dict(xt=FP4), E_ARG), (dict(xt=-1), E_ARG), (dict(xt=F8), E_ARG), (dict(M=-1), E_ARG), (dict(K=-16), E_ARG),
    (dict(K=24), E_ARG), (dict(block=64), E_ARG), (dict(block=0), E_ARG), (dict(turn=2), E_ARG), (dict(turn=-1), E_ARG),
    (dict(x=None), E_ARG), (dict(codes=None), E_ARG), (dict(scales=None), E_ARG), (dict(ldx=48), E_ARG),
    (dict(x=A + 2), E_ALIGN), (dict(codes=A + 8), E_ALIGN), (dict(scales=A + 2), E_ALIGN), (dict(ldx=68), E_ALIGN),
    (dict(M=(1 << 31) - 100), E_UNSUP), (dict(K=(1 << 31) - 16), E_UNSUP), (dict(M=65535 * 128 + 1, block=128), E_UNSUP),
    (dict(M=65535 * 128 + 1, turn=1), E_UNSUP), (dict(K=(1 << 30) - 112, turn=1), E_UNSUP),
    (dict(M=0, x=None), OK), (dict(K=0, codes=None), OK)])
def test_quantize_refuses(kw, expect):
    assert quantize(**kw) == expect


@pytest.mark.parametrize("kw,expect", [
    (dict(yt=FP4), E_ARG), (dict(yt=F8), E_ARG), (dict(M=-1), E_ARG), (dict(K=-16), E_ARG), (dict(K=24), E_ARG),
    (dict(block=2), E_ARG), (dict(y=None), E_ARG), (dict(codes=None), E_ARG), (dict(scales=None), E_ARG),
    (dict(ldy=48), E_ARG), (dict(y=A + 2), E_ALIGN), (dict(codes=A + 8), E_ALIGN), (dict(scales=A + 2), E_ALIGN),
    (dict(ldy=68), E_ALIGN), (dict(M=0, y=None), OK), (dict(K=0, codes=None), OK)])
def test_dequantize_refuses(kw, expect):
    assert dequantize(**kw) == expect


PRODUCT_REFUSALS = [
    (dict(xt=F32), E_ARG), (dict(xt=FP4), E_ARG), (dict(xt=9), E_ARG), (dict(yt=F8), E_ARG), (dict(yt=-1), E_ARG),
    (dict(M=-1), E_ARG), (dict(N=-16), E_ARG), (dict(K=-16), E_ARG), (dict(K=40), E_ARG), (dict(x=None), E_ARG),
    (dict(w=None), E_ARG), (dict(ws=None), E_ARG), (dict(y=None), E_ARG), (dict(ldx=32), E_ARG), (dict(ldy=15), E_ARG),
    (dict(xs=A), E_ARG), (dict(xt=F8), E_ARG), (dict(xt=F8, xs=A, ldx=96), E_ARG), (dict(x=A + 8), E_ALIGN),
    (dict(w=A + 4), E_ALIGN), (dict(ws=A + 2), E_ALIGN), (dict(xt=F8, xs=A + 1), E_ALIGN), (dict(y=A + 2), E_ALIGN),
    (dict(ldx=68), E_ALIGN), (dict(M=(1 << 31) - 512), E_UNSUP), (dict(K=(1 << 31) - 16), E_UNSUP),
    (dict(N=0, y=None), OK), (dict(M=0, x=None), OK)]


@pytest.mark.parametrize("kw,expect", PRODUCT_REFUSALS + [
    (dict(block=1), E_ARG), (dict(block=64, xt=F8, xs=A), E_ARG), (dict(res=A, ldr=8), E_ARG),
    (dict(res=A, ldr=32), E_ARG), (dict(res=A + 2), E_ALIGN), (dict(N=(1 << 31) - 512), E_UNSUP)])
def test_gemm_refuses(kw, expect):
    assert gemm(**kw) == expect


GATED_REFUSALS = [(dict(act=2), E_ARG), (dict(act=-1), E_ARG), (dict(N=24), E_ARG), (dict(N=1 << 30), E_ARG)]


@pytest.mark.parametrize("kw,expect", PRODUCT_REFUSALS + GATED_REFUSALS)
def test_gated_refuses(kw, expect):
    assert gated(**kw) == expect


@pytest.mark.parametrize("kw,expect", PRODUCT_REFUSALS + GATED_REFUSALS + [
    (dict(dh=None), E_ARG), (dict(dh=A), E_ARG), (dict(ldd=8), E_ARG), (dict(ldy=31), E_ARG), (dict(dh=A + 2), E_ALIGN)])
def test_grad_refuses(kw, expect):
    assert grad(**kw) == expect


def test_features_up_to_their_limit():
    # 2^30 - 513 features at most: the largest multiple of 16 below it goes on, the next is refused by name
    last, out = (1 << 30) - 528, (qgm.ctypes.c_int * 3)()
    for call in (gated, grad):
        assert call(N=last + 16) == E_ARG and call(N=last + 16, xt=F8, xs=A) == E_ARG
        assert call(N=last, M=0) == OK and call(N=last, ldy=16) == E_ARG and call(N=last, w=A + 4) == E_ALIGN
    assert lib.qf8_plan(1, 2, last, 64, F16, F16, 128, out) == OK and out[2] > 0
    assert lib.qf8_plan(1, 2, last + 16, 64, F16, F16, 128, out) == E_UNSUP


@pytest.mark.skipif(gpu_present(), reason="checks the no-device status; a GPU is present")
def test_no_device_status():
    assert quantize() == E_DEVICE and quantize(block=128, turn=1) == E_DEVICE and dequantize() == E_DEVICE
    assert gemm() == E_DEVICE and gemm(xt=F8, xs=A + 4, block=1) == E_DEVICE and gemm(K=0, x=None, w=None) == E_DEVICE
    assert gated() == E_DEVICE and gated(act=1, xt=F8, xs=A) == E_DEVICE and grad() == E_DEVICE


# ------------------------------------------------------------- the binding

def meta(shape, dtype=torch.float16, stride=None):
    return torch.empty_strided(shape, stride or [int(np.prod(shape[i + 1:])) for i in range(len(shape))],
                               dtype=dtype, device="meta")


def f8(R, K, block=128):
    return (meta((R, K), torch.float8_e4m3fn),
            meta((R if block == 1 else -(-R // 128), -(-K // 128)), torch.float32))


class Never:
    def __getattr__(self, name):
        raise AssertionError(f"{name} was called")


@pytest.fixture
def no_library(monkeypatch):
    """Tensors without memory stand for those on a GPU; the library must not be called."""
    monkeypatch.setattr(qgm, "_lib", Never())
    monkeypatch.setattr(qgm, "_mx_elsewhere", lambda x, stream: None)
    monkeypatch.setattr(qgm, "_dev", lambda t, what: t)


def test_binding_refuses_sizes_and_strides_past_32_bits(no_library):
    big = 1 << 32
    few, far, many = meta((2, 64)), meta((2, 64), stride=(big + 64, 1)), meta((big + 2, 64))
    w, ws = f8(64, 64)
    for call in (lambda: qgm.f8_quantize(far), lambda: qgm.f8_quantize(many), lambda: qgm.f8_quantize(meta((1, big + 64))),
                 lambda: qgm.f8_dequantize(*f8(2, 64), out=far), lambda: qgm.f8_dequantize(*f8(big + 2, 64)),
                 lambda: qgm.f8_gemm(far, w, ws), lambda: qgm.f8_gemm(many, w, ws), lambda: qgm.f8_gemm(few, w, ws, out=far),
                 lambda: qgm.f8_gemm(few, w, ws, residual=far), lambda: qgm.f8_gemm(few, *f8(big + 3, 64)),
                 lambda: qgm.f8_gemm(meta((1, big + 64)), *f8(3, big + 64)),
                 lambda: qgm.f8_gemm(f8(big + 2, 64)[0], w, ws, x_scales=f8(big + 2, 64, 1)[1]),
                 lambda: qgm.f8_gated(far, w, ws), lambda: qgm.f8_gated(few, *f8(big + 64, 64)),
                 lambda: qgm.f8_gated(few, w, ws, out=meta((2, 32), stride=(big + 32, 1))),
                 lambda: qgm.f8_gated_grad(meta((2, 32), stride=(big + 32, 1)), few, w, ws),
                 lambda: qgm.f8_gated_grad(meta((2, 32)), few, w, ws, out=far), lambda: qgm.F8Linear(*f8(big + 3, 64))):
        with pytest.raises(ValueError, match="2147483647"):
            call()


def test_binding_refuses_what_does_not_fit(no_library):
    x, (w, ws), (c, cs) = meta((2, 256)), f8(64, 256), f8(2, 256, 1)
    w1 = f8(64, 256, 1)[1]
    h = meta((2, 32))
    for call in (lambda: qgm.f8_quantize(meta((2, 40))), lambda: qgm.f8_quantize(x, block=64), lambda: qgm.f8_quantize(c),
                 lambda: qgm.f8_quantize(meta((2, 64), stride=(1, 2))), lambda: qgm.f8_quantize(x, codes=w),
                 lambda: qgm.f8_quantize(x, scales=ws), lambda: qgm.f8_quantize(x, transpose=True, codes=c),
                 lambda: qgm.f8_dequantize(c, cs, dtype=torch.float64), lambda: qgm.f8_dequantize(c, cs, out=h),
                 lambda: qgm.f8_dequantize(c, w1), lambda: qgm.f8_dequantize(x, cs),
                 lambda: qgm.f8_gemm(meta((2, 128)), w, ws), lambda: qgm.f8_gemm(meta((2, 256), torch.float32), w, ws),
                 lambda: qgm.f8_gemm(c, w, ws), lambda: qgm.f8_gemm(c, w, ws, x_scales=cs.t()),
                 lambda: qgm.f8_gemm(x, w, w1), lambda: qgm.f8_gemm(x, w, ws, x_scales=cs),
                 lambda: qgm.f8_gemm(x, w.view(torch.uint8), ws), lambda: qgm.f8_gemm(x, w, ws.double()),
                 lambda: qgm.f8_gemm(x, w.t(), ws), lambda: qgm.f8_gemm(x, w, ws, out=h),
                 lambda: qgm.f8_gemm(x, w, ws, out_dtype=torch.float64), lambda: qgm.f8_gemm(x, w, ws, residual=h),
                 lambda: qgm.f8_gemm(x, w, ws, residual=meta((2, 64), torch.float32)),
                 lambda: qgm.f8_gemm(x, w, ws, out=meta((2, 64)), out_dtype=torch.float32),
                 lambda: qgm.f8_gated(x, w, ws, act="relu"), lambda: qgm.f8_gated(x, *f8(48, 256)),
                 lambda: qgm.f8_gated(x, w, w1), lambda: qgm.f8_gated(x, w, ws, out=meta((2, 64))),
                 lambda: qgm.f8_gated_grad(meta((2, 64)), x, w, ws), lambda: qgm.f8_gated_grad(h, x, w, ws, out=h),
                 lambda: qgm.f8_gated_grad(h, x, w, ws, out=meta((2, 64), torch.float32)),
                 lambda: qgm.f8_gated_grad(c, x, w, ws), lambda: qgm.F8Linear(w, w1), lambda: qgm.F8Gated(w, ws, act="tanh"),
                 lambda: qgm.F8Gated(*f8(40, 256))):
        with pytest.raises(ValueError):
            call()


def test_binding_refuses_cpu_tensors():
    x = torch.zeros(2, 64, dtype=torch.float16)
    c, s = torch.zeros(32, 64, dtype=torch.float8_e4m3fn), torch.zeros(1, 1)
    for call in (lambda: qgm.f8_quantize(x), lambda: qgm.f8_dequantize(c, s), lambda: qgm.f8_gemm(x, c, s), lambda: qgm.f8_gated(x, c, s),
                 lambda: qgm.f8_gated_grad(x[:, :16], x, c, s), lambda: qgm.F8Linear(c, s), lambda: qgm.F8Gated(c, s),
                 lambda: qgm.F8Linear.from_weight(x), lambda: qgm.F8Gated.from_weight(x)):
        with pytest.raises(ValueError, match="GPU"):
            call()


# --------------------------------------------------------------- the plans

def test_plans(monkeypatch):
    plan = qgm.f8_plan
    # few rows: a wave for each chunk of 512 k, as far as LDS holds 16 rows of x for them
    assert plan(1, 6144, 2048, F16, F16) == dict(tile=0, waves=4, pieces=384)
    assert plan(8, 2048, 8192, BF16) == dict(tile=0, waves=16, pieces=128)
    assert plan(1, 8192, 2048, F16, F16, gated=True) == dict(tile=0, waves=4, pieces=512)
    assert plan(16, 2048, 8192, BF16)["waves"] == 8 and plan(1, 64, 96, BF16)["waves"] == 1
    assert plan(1, 64, 0, BF16)["tile"] == 0
    # larger tiles as the rows grow
    tiles = [plan(m, 8192, 8192, F8)["tile"] for m in (1, 100, 1000, 4096)]
    assert tiles[0] == 0 and tiles[1] in (1, 2, 5) and tiles[-1] == 4
    assert plan(4096, 8192, 8192, F8) == dict(tile=4, waves=0, pieces=512)
    assert plan(4096, 8192, 8192, F8, F32)["pieces"] == 1024 == plan(4096, 8192, 8192, F8, w_block=1)["pieces"]
    assert plan(128, 2048, 8192, BF16)["tile"] == 5      # few tiles of a long K: two groups of waves
    # the rows kernel's grid has 65535 blocks of 16 rows; rows of more than 4 MiB are its alone
    assert plan(1 << 21, 16, 16, BF16)["tile"] > 0
    assert plan(4096, 4096, 1 << 23, F8)["tile"] == 0 and plan(4096, 4096, 1 << 22, F8)["tile"] > 0
    for v in range(6):
        monkeypatch.setenv("QF8_TILE", str(v))
        assert plan(100, 300, 512, F16)["tile"] == v and plan(100, 304, 512, F8, gated=True)["tile"] == v
    out = (qgm.ctypes.c_int * 3)()
    for bad in ((2, 1, 1, 16, 0, 0, 128), (0, -1, 1, 16, 0, 0, 128), (0, 1, -1, 16, 0, 0, 128), (0, 1, 1, 24, 0, 0, 128),
                (0, 1, 1, 16, 2, 0, 128), (0, 1, 1, 16, 0, 4, 128), (0, 1, 1, 16, 0, 0, 1), (0, 1, 1, 16, 4, 0, 64),
                (1, 1, 8, 16, 0, 0, 128)):
        assert lib.qf8_plan(*bad, out) == E_ARG
    assert lib.qf8_plan(0, 1, 1, 16, 0, 0, 128, None) == E_ARG
    top = (1 << 31) - 1
    for bad in ((0, top, 16, 16, 0, 0, 128), (0, 16, top, 16, 0, 0, 128), (1, 16, 1 << 30, 16, 0, 0, 128)):
        assert lib.qf8_plan(*bad, out) == E_UNSUP


@pytest.mark.parametrize("forced", [None, 0, 1, 4, 5])
def test_plans_without_a_choice(monkeypatch, forced):
    # nothing to multiply, or rows of x of more than 4 MiB: the setting is not asked
    if forced is not None:
        monkeypatch.setenv("QF8_TILE", str(forced))
    for gated_ in (False, True):
        for M in (1, 40, 5000):
            for x_type in (F16, BF16, F8):
                assert qgm.f8_plan(M, 304, 0, x_type, gated=gated_)["tile"] == 0
                assert qgm.f8_plan(M, 304, 0, x_type, gated=gated_)["waves"] == 1
                assert qgm.f8_plan(M, 304, (1 << 22) + 16, x_type, gated=gated_)["tile"] == 0
            assert qgm.f8_plan(M, 304, (1 << 21) + 16, BF16, gated=gated_)["tile"] == 0
    if forced is not None:
        assert qgm.f8_plan(40, 304, 1 << 21, BF16)["tile"] == forced == qgm.f8_plan(40, 304, 1 << 22, F8)["tile"]


@pytest.mark.parametrize("M,N", [(0, 16), (16, 0), (0, 0)])
def test_plan_of_nothing(M, N):
    for K in (0, 64, 8192):
        for x_type in (F16, BF16, F8):
            assert qgm.f8_plan(M, N, K, x_type) == dict(tile=0, waves=1, pieces=0)


@pytest.mark.parametrize("tile,call", [
    (0, lambda: gemm(M=65535 * 16 + 1)), (1, lambda: gemm(M=1 << 18, N=1 << 18)), (5, lambda: gemm(M=1 << 18, N=1 << 17)),
    (4, lambda: gemm(xt=F8, xs=A, yt=BF16, M=1 << 20, N=1 << 19)), (0, lambda: gated(M=65535 * 16 + 1)),
    (None, lambda: gemm(M=1 << 20, K=1 << 23, xt=F8, xs=A))])
def test_more_than_a_grid_holds(monkeypatch, tile, call):
    if tile is not None:
        monkeypatch.setenv("QF8_TILE", str(tile))
    assert call() == E_UNSUP


@pytest.mark.skipif(gpu_present(), reason="checks the no-device status; a GPU is present")
@pytest.mark.parametrize("tile,call", [
    (0, lambda: gemm(M=65535 * 16)), (1, lambda: gemm(M=(1 << 18) - 64, N=1 << 18)),
    (4, lambda: gemm(xt=F8, xs=A, yt=BF16, M=(1 << 20) - 256, N=1 << 19)), (None, lambda: gemm(M=1 << 22)), (None, lambda: gemm(M=1 << 22, K=0)),
    (None, lambda: gated(M=1 << 22, K=0)), (None, lambda: grad(M=1 << 22, K=0))])
def test_what_a_grid_holds_comes_to_the_device(monkeypatch, tile, call):
    if tile is not None:
        monkeypatch.setenv("QF8_TILE", str(tile))
    assert call() == E_DEVICE
