"""The MXFP4 operators on the GPU against the oracle in 64 bits.

Tolerances.  Quantising and reading back are exact, as are products whose
terms and partial sums are integers times one power of two below 2^24 (fp32
holds every partial sum, in any order).  Elsewhere |y - ref| is at most half a
step of the output type (relative eps / 2, or half its smallest subnormal) plus
the fp32 sums' own error: at most K + 2 additions (and the factor of row_scale),
each off by at most a whole unit (2^-23, matrix cores need not round to
nearest) of a partial sum that the sum of the terms' magnitudes bounds."""
import numpy as np
import pytest

from oracle import mxref

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU visible", allow_module_level=True)
import bit_weight_only_dequant_amd as qgm  # noqa: E402

DEV = "cuda:0"
F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32
TINY = {F16: 2.0 ** -24, BF16: 2.0 ** -133, F32: 2.0 ** -149}


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def f64(t):
    return t.detach().cpu().double().numpy()


def check(y, ref, mag, K):
    """ref rounded to y's type, within the bound of the head of this file."""
    eps = torch.finfo(y.dtype).eps / 2
    tol = eps * np.abs(ref) + TINY[y.dtype] / 2 + (1 + eps) * (K + 3) * 2.0 ** -23 * mag
    err = np.abs(f64(y) - ref)
    assert (err <= tol).all(), (np.unravel_index(np.argmax(err - tol), err.shape), (err / np.maximum(tol, 1e-300)).max())


def rounded(ref, dtype):
    """float64 (exact in fp32) rounded once to dtype, as float64."""
    return f64(torch.from_numpy(np.asarray(ref, dtype=np.float32)).to(dtype))


def random_mx(rng, R, K, spread=4, centre=122):
    codes = rng.integers(0, 256, (R, K // 2), dtype=np.uint8)
    return codes, rng.integers(centre - spread, centre + spread + 1, (R, K // 32)).astype(np.uint8)


def make_x(rng, kind, M, K, exact=False):
    """(device x, device x_scales, float64 values)."""
    if kind == "mx":
        c, s = random_mx(rng, M, K, spread=0 if exact else 6, centre=127)
        return dev(c), dev(s), mxref.mx_values(c, s)
    v = rng.integers(-4, 5, (M, K)) if exact else rng.standard_normal((M, K))
    t = torch.from_numpy(v.astype(np.float32)).to(F16 if kind == "f16" else BF16)
    return t.to(DEV), None, f64(t)


XTYPE = {"f16": F16, "bf16": BF16}


# ----------------------------------------------------- quantise and read back

@pytest.mark.parametrize("dtype", [F16, BF16, F32])
def test_quantize_every_pattern(dtype):
    # every 16-bit pattern (for fp32: random patterns, subnormals and all
    # exponents) beside a block's other values, finite blocks and others
    rng = np.random.default_rng(3)
    if dtype == F32:
        x = torch.from_numpy(rng.integers(0, 1 << 32, (2048, 32), dtype=np.uint32).view(np.float32))
        x[:512] = torch.from_numpy(rng.integers(0, 1 << 25, (512, 32), dtype=np.uint32).view(np.float32))
    else:
        bits = np.arange(65536, dtype=np.uint16)
        x = torch.from_numpy(bits.view(np.int16).copy()).view(dtype).reshape(2048, 32)
        x = torch.cat([x, x.reshape(32, 2048).t().contiguous()])
    codes, scales = qgm.mx_quantize(x.to(DEV))
    want_c, want_s = mxref.mx_quantize(x.double().numpy())
    assert np.array_equal(scales.cpu().numpy(), want_s)
    assert np.array_equal(codes.cpu().numpy(), want_c)


@pytest.mark.parametrize("dtype", [F16, BF16, F32])
@pytest.mark.parametrize("M,K", [(1, 32), (3, 96), (257, 2080), (1, 8192), (70000, 32), (5, 64)])
def test_quantize_sizes_and_strides(dtype, M, K):
    rng = np.random.default_rng(M + K)
    v = rng.standard_normal((M, K)) * np.exp2(rng.integers(-12, 12, (M, 1)))
    v[rng.random((M, K)) < 0.2] *= 0.25   # ties' neighbourhood
    v = np.round(v * 64) / 64
    x = torch.from_numpy(v.astype(np.float32)).to(dtype)
    want_c, want_s = mxref.mx_quantize(x.double().numpy())
    wide = torch.full((M, K + 24), float("nan"), dtype=dtype, device=DEV)
    wide[:, 8:8 + K] = x.to(DEV)
    for t in (x.to(DEV), wide[:, 8:8 + K]):
        codes = torch.full((M + 2, K // 2), 77, dtype=torch.uint8, device=DEV)
        scales = torch.full((M + 2, K // 32), 77, dtype=torch.uint8, device=DEV)
        qgm.mx_quantize(t, codes=codes[:M], scales=scales[:M])
        assert np.array_equal(codes[:M].cpu().numpy(), want_c) and np.array_equal(scales[:M].cpu().numpy(), want_s)
        assert bool((codes[M:] == 77).all()) and bool((scales[M:] == 77).all())


@pytest.mark.parametrize("dtype", [F16, BF16, F32])
def test_dequantize_every_scale_and_code(dtype):
    scales = np.arange(256, dtype=np.uint8).reshape(256, 1)
    nib = np.concatenate([np.arange(16), np.arange(15, -1, -1)]).astype(np.uint8)
    codes = np.tile(nib[0::2] | nib[1::2] << 4, (256, 1)).astype(np.uint8)
    y = qgm.mx_dequantize(dev(codes), dev(scales), dtype=dtype)
    with np.errstate(over="ignore"):
        ref = rounded(mxref.mx_values(codes, scales), dtype)
    assert np.array_equal(f64(y), ref, equal_nan=True)


def test_dequantize_strided_leaves_the_gap():
    rng = np.random.default_rng(8)
    codes, scales = random_mx(rng, 37, 160)
    out = torch.full((37, 176), 5.0, dtype=F32, device=DEV)
    qgm.mx_dequantize(dev(codes), dev(scales), out=out[:, 8:168])
    assert np.array_equal(f64(out[:, 8:168]), mxref.mx_values(codes, scales))
    assert bool((out[:, :8] == 5).all()) and bool((out[:, 168:] == 5).all())


@pytest.mark.parametrize("M,K", [(0, 64), (4, 0)])
def test_quantize_empty(M, K):
    codes, scales = qgm.mx_quantize(torch.zeros(M, K, dtype=F16, device=DEV))
    assert codes.shape == (M, K // 2) and scales.shape == (M, K // 32)
    assert qgm.mx_dequantize(codes, scales).shape == (M, K)


# ------------------------------------------------------------------ products

SIZES = [(1, 1, 32), (1, 16, 64), (1, 250, 2048), (2, 17, 96), (7, 33, 160), (15, 64, 128), (16, 100, 288),
         (17, 48, 512), (31, 16, 1056), (33, 130, 96), (63, 257, 256), (64, 128, 128), (65, 96, 544), (100, 65, 2080),
         (127, 300, 32), (129, 129, 224), (200, 512, 384), (257, 200, 1024), (300, 777, 800), (513, 1030, 288),
         (1100, 530, 416)]


@pytest.mark.parametrize("kind", ["f16", "bf16", "mx"])
@pytest.mark.parametrize("M,N,K", SIZES)
def test_gemm_exact_integers(kind, M, N, K):
    # x integers to 4 (codes to 6, halves), weights with one scale: every partial
    # sum is a multiple of 2^-7 below 2^17 (K 6 6 at most), exact in fp32
    rng = np.random.default_rng(M * 7 + N + K)
    x, xs, xv = make_x(rng, kind, M, K, exact=True)
    wc, wsc = random_mx(rng, N, K, spread=0)
    ref, _ = mxref.mx_gemm_ref(xv, mxref.mx_values(wc, wsc))
    for yt in (F32, XTYPE.get(kind, F16)):
        out = torch.full((M + 1, N), 9.0, dtype=yt, device=DEV)
        y = qgm.mx_gemm(x, dev(wc), dev(wsc), x_scales=xs, out=out[:M])
        assert np.array_equal(f64(y), rounded(ref, yt))
        assert bool((out[M] == 9).all())


@pytest.mark.parametrize("kind", ["f16", "bf16", "mx"])
@pytest.mark.parametrize("yt", [F16, BF16, F32])
@pytest.mark.parametrize("M,N,K", [(1, 300, 2048), (5, 77, 96), (40, 129, 608), (130, 260, 1056), (600, 333, 512)])
def test_gemm_random_with_residual_and_strides(kind, yt, M, N, K):
    rng = np.random.default_rng(M + N * 3 + K)
    x, xs, xv = make_x(rng, kind, M, K)
    if xs is None:
        wide = torch.full((M, K + 16), float("nan"), dtype=x.dtype, device=DEV)
        wide[:, :K] = x
        x = wide[:, :K]
    wc, wsc = random_mx(rng, N, K)
    r = torch.randn(M, N + 3, dtype=F32).to(yt)
    out = torch.full((M, N + 5), 9.0, dtype=yt, device=DEV)
    ref, mag = mxref.mx_gemm_ref(xv, mxref.mx_values(wc, wsc), residual=f64(r[:, :N]))
    qgm.mx_gemm(x, dev(wc), dev(wsc), x_scales=xs, out=out[:, :N], residual=r.to(DEV)[:, :N])
    check(out[:, :N], ref, mag, K)
    assert bool((out[:, N:] == 9).all())
    # in place: the residual is the output itself
    y = r.to(DEV).contiguous()[:, :N].clone()
    qgm.mx_gemm(x, dev(wc), dev(wsc), x_scales=xs, out=y, residual=y)
    assert torch.equal(y, out[:, :N])


@pytest.mark.parametrize("M", [1, 20, 150, 600])
def test_gemm_f16_weights_beyond_f16(M):
    # weights far below and above what fp16 can hold, in the same row as ordinary ones
    rng = np.random.default_rng(M)
    N, K = 70, 640
    wc, wsc = random_mx(rng, N, K)
    wsc[3, :] = 20       # 2^-107
    wsc[4, 2] = 180      # 2^53
    wsc[5, 7:9] = 95     # fp16 would keep some of the codes
    wsc[6, ::2] = 141    # 6 * 2^14: past fp16's largest
    x, _, xv = make_x(rng, "f16", M, K)
    x[0, :4] = torch.tensor([65504.0, -65504.0, 2.0 ** -24, -(2.0 ** -24)], dtype=F16)
    xv = f64(x)
    ref, mag = mxref.mx_gemm_ref(xv, mxref.mx_values(wc, wsc))
    check(qgm.mx_gemm(x, dev(wc), dev(wsc), out_dtype=F32), ref, mag, K)


@pytest.mark.parametrize("kind", ["f16", "bf16", "mx"])
@pytest.mark.parametrize("M,N,K", [(3, 40, 96), (70, 90, 416), (300, 270, 672)])
def test_gemm_nan_and_inf_stay_in_their_row_and_column(kind, M, N, K):
    rng = np.random.default_rng(M * N)
    x, xs, xv = make_x(rng, kind, M, K)
    wc, wsc = random_mx(rng, N, K)
    wsc[5, -1] = 255
    wsc[N - 1, 0] = 255
    if kind == "mx":
        xs[1, 0] = 255
    else:
        x[1, 3] = float("nan")
        x[2, K - 1] = float("inf")
    xv = mxref.mx_values(x.cpu().numpy(), xs.cpu().numpy()) if kind == "mx" else f64(x)
    y = f64(qgm.mx_gemm(x, dev(wc), dev(wsc), x_scales=xs, out_dtype=F32))
    with np.errstate(invalid="ignore"):
        ref, _ = mxref.mx_gemm_ref(xv, mxref.mx_values(wc, wsc))
        gap = np.abs(y - ref)
    assert np.array_equal(np.isnan(y), np.isnan(ref)) and np.array_equal(np.isinf(y), np.isinf(ref))
    ok = np.isfinite(ref)
    ok_rows = [m for m in range(M) if np.isfinite(xv[m]).all()]
    w0 = np.nan_to_num(mxref.mx_values(wc, wsc))
    mag = np.abs(np.nan_to_num(xv, posinf=0)) @ np.abs(w0).T
    assert (gap[ok_rows][ok[ok_rows]] <= ((K + 3) * 2.0 ** -23 * mag[ok_rows] + 2.0 ** -149)[ok[ok_rows]]).all()


# the ends of the scales' range: the smallest make weights down to 2^-128 (16-bit x meets them as subnormal
# bf16 numbers), 252 is the largest that the quantiser writes.  x keeps the products and sums within fp32's
# normal numbers, so the tolerance is the usual one.
@pytest.mark.parametrize("tile", range(5))
@pytest.mark.parametrize("low", [0, 6, 250])
@pytest.mark.parametrize("kind", ["f16", "bf16", "mx"])
@pytest.mark.parametrize("M,N,K", [(3, 40, 96), (20, 70, 1056)])
def test_gemm_ends_of_the_scales(monkeypatch, tile, low, kind, M, N, K):
    monkeypatch.setenv("QMX_TILE", str(tile))
    rng = np.random.default_rng(M + N + low)
    wc, _ = random_mx(rng, N, K)
    wsc = rng.integers(low, low + 3, (N, K // 32)).astype(np.uint8)
    if kind == "mx":
        x, xs, _ = make_x(rng, kind, M, K)
        xs = dev(rng.integers(*((150, 160) if low < 250 else (90, 100)), (M, K // 32)).astype(np.uint8))
        xv = mxref.mx_values(x.cpu().numpy(), xs.cpu().numpy())
    else:
        size = (2.0 ** 12 if low < 250 else 2.0 ** -12) if kind == "f16" else (2.0 ** 60 if low < 250 else 2.0 ** -30)
        x, xs = torch.from_numpy(rng.uniform(1, 2, (M, K)) * size).to(F16 if kind == "f16" else BF16).to(DEV), None
        xv = f64(x)
    ref, mag = mxref.mx_gemm_ref(xv, mxref.mx_values(wc, wsc))
    check(qgm.mx_gemm(x, dev(wc), dev(wsc), x_scales=xs, out_dtype=F32), ref, mag, K)


@pytest.mark.parametrize("kind", ["f16", "bf16", "mx"])
@pytest.mark.parametrize("M,N,K", [(1, 64, 8192), (64, 256, 1024), (512, 512, 1024)])
def test_gemm_equal_inputs_give_equal_bits(kind, M, N, K):
    rng = np.random.default_rng(5)
    x, xs, _ = make_x(rng, kind, M, K)
    w, ws = (dev(a) for a in random_mx(rng, N, K))
    first = qgm.mx_gemm(x, w, ws, x_scales=xs, out_dtype=F32)
    for _ in range(3):
        assert torch.equal(first, qgm.mx_gemm(x, w, ws, x_scales=xs, out_dtype=F32))


# every kernel whatever the rule would take: sizes around their tiles, K around
# the stages (128) and groups of them (512), K that ends inside each
@pytest.mark.parametrize("tile", range(5))
@pytest.mark.parametrize("kind", ["f16", "bf16", "mx"])
@pytest.mark.parametrize("M,N,K", [(1, 129, 512), (70, 257, 544), (17, 64, 992), (130, 300, 1024), (260, 70, 1600),
                                   (3, 40, 128), (66, 130, 352), (5, 17, 32), (129, 513, 480), (33, 100, 2528)])
def test_gemm_every_kernel(monkeypatch, tile, kind, M, N, K):
    monkeypatch.setenv("QMX_TILE", str(tile))
    rng = np.random.default_rng(M + N + K)
    wc, wsc = random_mx(rng, N, K, spread=0)
    x, xs, xv = make_x(rng, kind, M, K, exact=True)
    out = torch.full((M + 1, N), 9.0, dtype=F32, device=DEV)
    qgm.mx_gemm(x, dev(wc), dev(wsc), x_scales=xs, out=out[:M])
    assert np.array_equal(f64(out[:M]), mxref.mx_gemm_ref(xv, mxref.mx_values(wc, wsc))[0])
    assert bool((out[M] == 9).all())
    # scales of every size, some of them too small or too large for fp16, and a NaN block that only
    # reaches its own column
    wsc = rng.integers(95, 150, wsc.shape).astype(np.uint8)
    wsc[N // 2, -1] = 255
    x, xs, xv = make_x(rng, kind, M, K)
    with np.errstate(invalid="ignore"):
        ref, mag = mxref.mx_gemm_ref(xv, mxref.mx_values(wc, wsc))
    y = qgm.mx_gemm(x, dev(wc), dev(wsc), x_scales=xs, out_dtype=F32)
    keep = np.arange(N) != N // 2
    assert bool(torch.isnan(y[:, N // 2]).all())
    check(y[:, torch.from_numpy(keep).to(DEV)], ref[:, keep], mag[:, keep], K)


@pytest.mark.parametrize("kind", ["f16", "bf16", "mx"])
@pytest.mark.parametrize("M", [1, 7, 9, 16])
@pytest.mark.parametrize("N,K", [(200, 8192), (4200, 4128), (40, 20000)])
def test_gemm_few_rows_long_k(monkeypatch, kind, M, N, K):
    # several chunks a wave, x in as much LDS as there is, workgroups with several column blocks
    monkeypatch.setenv("QMX_TILE", "0")
    rng = np.random.default_rng(M + K)
    wc, wsc = random_mx(rng, N, K)
    x, xs, xv = make_x(rng, kind, M, K)
    ref, mag = mxref.mx_gemm_ref(xv, mxref.mx_values(wc, wsc))
    check(qgm.mx_gemm(x, dev(wc), dev(wsc), x_scales=xs, out_dtype=F32), ref, mag, K)


@pytest.mark.parametrize("tile", [0, 1, 4])
@pytest.mark.parametrize("kind", ["bf16", "mx"])
def test_grouped_far_rows_and_weights(monkeypatch, tile, kind):
    # rows of x and a matrix that lie more than 4 GiB into their arrays
    monkeypatch.setenv("QMX_TILE", str(tile))
    rng = np.random.default_rng(1)
    E, N, K = 150, 8192, 8192
    w = torch.zeros(E, N, K // 2, dtype=torch.uint8, device=DEV)
    ws = torch.full((E, N, K // 32), 120, dtype=torch.uint8, device=DEV)
    wc, wsc = random_mx(rng, 64, K)
    w[E - 1, N - 64:], ws[E - 1, N - 64:] = dev(wc), dev(wsc)
    far = 300000 if kind == "bf16" else 1200000
    x = torch.zeros(far, K if kind == "bf16" else K // 2, dtype=BF16 if kind == "bf16" else torch.uint8, device=DEV)
    xs = None if kind == "bf16" else torch.full((far, K // 32), 127, dtype=torch.uint8, device=DEV)
    few, fews, xv = make_x(rng, kind, 3, K)
    x[far - 3:] = few
    if xs is not None:
        xs[far - 3:] = fews
    rows = torch.tensor([far - 1, far - 3, 0, far - 2], dtype=torch.int32, device=DEV)
    off = torch.zeros(E + 1, dtype=torch.int32, device=DEV)
    off[E] = 4
    y = qgm.mx_gemm_grouped(x, w, ws, off, x_scales=xs, rows=rows, out_dtype=F32)
    assert not bool(y[:, :N - 64].any()) and not bool(y[2].any())
    ref, mag = mxref.mx_gemm_ref(xv[[2, 0, 1]], mxref.mx_values(wc, wsc))
    check(y[[0, 1, 3], N - 64:], ref, mag, K)


@pytest.mark.parametrize("M,N,K", [(0, 16, 64), (4, 0, 64), (3, 18, 0), (2, 140000, 0)])
def test_gemm_empty(M, N, K):
    w = torch.zeros(N, K // 2, dtype=torch.uint8, device=DEV)
    ws = torch.zeros(N, K // 32, dtype=torch.uint8, device=DEV)
    r = torch.randn(M, N, device=DEV).to(BF16)
    for kind in ("bf16", "mx"):
        x = torch.zeros(M, K, dtype=BF16, device=DEV) if kind == "bf16" else w.new_zeros(M, K // 2)
        xs = None if kind == "bf16" else w.new_zeros(M, K // 32)
        y = qgm.mx_gemm(x, w, ws, x_scales=xs, out_dtype=BF16, residual=r)
        assert y.shape == (M, N) and (K > 0 or torch.equal(y, r))


# ------------------------------------------------------------------- grouped

def make_groups(sizes, head=0):
    return np.concatenate([[head], head + np.cumsum(sizes)]).astype(np.int32)


GROUPS = [[1], [3, 0, 5], [0, 0, 40], [16, 1, 0, 31], [1] * 20, [0, 200, 3], [130, 0, 70, 1, 64], [300, 260, 0, 513],
          [5] * 70, [0, 0, 0]]


@pytest.mark.parametrize("tile", ["", "0", "1", "2", "3", "4"], ids=lambda t: "tile" + t)
@pytest.mark.parametrize("kind", ["f16", "bf16", "mx"])
@pytest.mark.parametrize("sizes", GROUPS, ids=lambda s: "-".join(map(str, s[:5])))
@pytest.mark.parametrize("N,K", [(40, 96), (260, 544)])
def test_grouped(monkeypatch, kind, sizes, N, K, tile):
    if tile:
        monkeypatch.setenv("QMX_TILE", tile)
    rng = np.random.default_rng(sum(sizes) + N)
    E, head, behind = len(sizes), 3, 2
    off = make_groups(sizes, head)
    T, xr = int(off[-1]) + behind, 50
    rows = rng.integers(0, xr, T).astype(np.int32)     # rows chosen twice and never
    rows[rng.random(T) < 0.1] = -1
    rows[rng.random(T) < 0.05] = xr
    scale = rng.standard_normal(T).astype(np.float32)
    x, xs, xv = make_x(rng, kind, xr, K)
    wc, wsc = random_mx(rng, E * N, K)
    w, ws = dev(wc.reshape(E, N, -1)), dev(wsc.reshape(E, N, -1))
    wv = mxref.mx_values(wc, wsc).reshape(E, N, K)
    yt = XTYPE.get(kind, BF16)
    out = torch.full((T, N), 9.0, dtype=yt, device=DEV)
    qgm.mx_gemm_grouped(x, w, ws, dev(off), x_scales=xs, rows=dev(rows), row_scale=dev(scale), out=out)
    ref, mag = mxref.mx_grouped_ref(xv, wv, off, rows, scale, fill=9.0)
    check(out, ref, mag, K)
    assert bool((out[:head] == 9).all()) and bool((out[T - behind:] == 9).all())
    # rows in slot order, no factor
    xt, xst, xtv = make_x(rng, kind, T, K)
    out = torch.full((T, N), 9.0, dtype=F32, device=DEV)
    qgm.mx_gemm_grouped(xt, w, ws, dev(off), x_scales=xst, out=out)
    ref, mag = mxref.mx_grouped_ref(xtv, wv, off, fill=9.0)
    check(out, ref, mag, K)


@pytest.mark.parametrize("T", [9, 700])
def test_grouped_one_group_is_the_plain_product(T):
    rng = np.random.default_rng(T)
    x, _, _ = make_x(rng, "bf16", T, 256)
    w, ws = (dev(a) for a in random_mx(rng, 200, 256))
    off = torch.tensor([0, T], dtype=torch.int32, device=DEV)
    y, z = qgm.mx_gemm_grouped(x, w[None], ws[None], off, out_dtype=F32), qgm.mx_gemm(x, w, ws, out_dtype=F32)
    mag = np.abs(f64(x)) @ np.abs(f64(qgm.mx_dequantize(w, ws, dtype=F32))).T
    assert (np.abs(f64(y) - f64(z)) <= 2 * 259 * 2.0 ** -23 * mag).all()


@pytest.mark.parametrize("kind", ["f16", "mx"])
@pytest.mark.parametrize("T", [40, 400])
@pytest.mark.parametrize("off", [[0, -5, 1000, 7], [9, 3, 3, 2], [-2147483648, 2147483647, 5, 2147483647]])
def test_grouped_bad_offsets_stay_inside(kind, T, off):
    # what the rows hold is unspecified; what lies around y is not touched
    rng = np.random.default_rng(T)
    N, K = 48, 160
    x, xs, _ = make_x(rng, kind, T, K)
    w, ws = (dev(a).reshape(3, N, -1) for a in random_mx(rng, 3 * N, K))
    out = torch.full((T + 16, N), 9.0, dtype=F16, device=DEV)
    qgm.mx_gemm_grouped(x, w, ws, torch.tensor(off, dtype=torch.int32, device=DEV), x_scales=xs, out=out[8:8 + T])
    assert bool((out[:8] == 9).all()) and bool((out[8 + T:] == 9).all())


def test_grouped_empty():
    w, ws = torch.zeros(3, 16, 32, dtype=torch.uint8, device=DEV), torch.zeros(3, 16, 2, dtype=torch.uint8, device=DEV)
    off = torch.zeros(4, dtype=torch.int32, device=DEV)
    x = torch.zeros(0, 64, dtype=BF16, device=DEV)
    assert qgm.mx_gemm_grouped(x, w, ws, off).shape == (0, 16)
    # no rows of x at all, every slot without one: zeros
    off[1:] = 5
    rows = torch.full((5,), -1, dtype=torch.int32, device=DEV)
    y = qgm.mx_gemm_grouped(x, w, ws, off, rows=rows, out=torch.full((5, 16), 9.0, dtype=BF16, device=DEV))
    assert not bool(y.any())
    # the same where a wave would have work, and many blocks
    big, bigs = torch.zeros(40, 4000, 512, dtype=torch.uint8, device=DEV), torch.zeros(40, 4000, 32, dtype=torch.uint8, device=DEV)
    off = torch.arange(41, dtype=torch.int32, device=DEV)
    y = qgm.mx_gemm_grouped(torch.zeros(0, 1024, dtype=BF16, device=DEV), big, bigs, off,
                            rows=torch.zeros(40, dtype=torch.int32, device=DEV), out=torch.full((40, 4000), 9.0, dtype=BF16, device=DEV))
    assert not bool(y.any())
    off = torch.zeros(4, dtype=torch.int32, device=DEV)
    x = torch.zeros(0, 64, dtype=BF16, device=DEV)
    # no experts: nothing is written
    y = torch.full((4, 16), 9.0, dtype=BF16, device=DEV)
    qgm.mx_gemm_grouped(x.new_zeros(4, 64), w[:0], ws[:0], off[:1], out=y)
    assert bool((y == 9).all())


@pytest.mark.parametrize("tile", range(5))
@pytest.mark.parametrize("kind", ["f16", "bf16", "mx"])
@pytest.mark.parametrize("N,K", [(40, 96), (260, 544), (40, 0)])
def test_grouped_slots_without_a_row_are_zero_whatever_their_factor(monkeypatch, kind, N, K, tile):
    # a padded batch: the padding slots' factors were never written
    monkeypatch.setenv("QMX_TILE", str(tile))
    rng = np.random.default_rng(N + K)
    sizes = [7, 0, 40, 1, 130]
    off, E, T, xr = make_groups(sizes), len(sizes), sum(sizes), 50
    rows = rng.integers(0, xr, T).astype(np.int32)
    pad = rng.random(T) < 0.4
    pad[:2] = True
    rows[pad] = rng.choice(np.array([-1, xr, -2147483648, 2147483647], dtype=np.int32), int(pad.sum()))
    scale = rng.standard_normal(T).astype(np.float32)
    scale[pad] = rng.choice(np.array([np.nan, np.inf, -np.inf, -1.0, 2.0], dtype=np.float32), int(pad.sum()))
    x, xs, xv = make_x(rng, kind, xr, K)
    wc, wsc = random_mx(rng, E * N, K)
    w, ws = dev(wc.reshape(E, N, K // 2)), dev(wsc.reshape(E, N, K // 32))
    out = torch.full((T, N), 9.0, dtype=F32, device=DEV)
    qgm.mx_gemm_grouped(x, w, ws, dev(off), x_scales=xs, rows=dev(rows), row_scale=dev(scale), out=out)
    assert not out[dev(pad)].view(torch.int32).any()          # +0 in every bit
    ref, mag = mxref.mx_grouped_ref(xv, mxref.mx_values(wc, wsc).reshape(E, N, K), off, rows, scale)
    check(out, ref, mag, K)
    # no rows of x at all
    out.fill_(9.0)
    none = x[:0], None if xs is None else xs[:0]
    qgm.mx_gemm_grouped(none[0], w, ws, dev(off), x_scales=none[1], rows=dev(rows), row_scale=dev(scale), out=out)
    assert not out.view(torch.int32).any()


def test_strides_and_sizes_past_32_bits_are_refused():
    # one allocation of 8.6 GB: a far second row, and a row longer than 2^31
    far = (1 << 32) + 64
    flat = torch.empty(far + 64, dtype=F16, device=DEV)
    x, long_row = flat.as_strided((2, 64), (far, 1)), flat[:far].view(1, far)
    w, ws = torch.zeros(64, 32, dtype=torch.uint8, device=DEV), torch.zeros(64, 2, dtype=torch.uint8, device=DEV)
    few, off = torch.zeros(2, 64, dtype=F16, device=DEV), torch.tensor([0, 2], dtype=torch.int32, device=DEV)
    for call in (lambda: qgm.mx_quantize(x), lambda: qgm.mx_quantize(long_row),
                 lambda: qgm.mx_dequantize(w[:2], ws[:2], out=x), lambda: qgm.mx_gemm(x, w, ws),
                 lambda: qgm.mx_gemm(few, w, ws, out=x), lambda: qgm.mx_gemm(few, w, ws, residual=x),
                 lambda: qgm.mx_gemm_grouped(x, w[None], ws[None], off),
                 lambda: qgm.mx_gemm_grouped(few, w[None], ws[None], off, out=x)):
        with pytest.raises(ValueError, match="2147483647"):
            call()
    # one row has no stride that counts
    x = flat.as_strided((1, 64), (far, 1))
    x.normal_()
    assert torch.equal(qgm.mx_gemm(x, w, ws), x.new_zeros(1, 64))


@pytest.mark.parametrize("kind", ["bf16", "mx"])
@pytest.mark.parametrize("yt", [F16, BF16, F32])
@pytest.mark.parametrize("M,N", [(65535 * 16 + 5, 3), (1, 140001), (37, 70), (2100000, 1)])
def test_gemm_without_k_of_any_size(kind, yt, M, N):
    w, ws = torch.zeros(N, 0, dtype=torch.uint8, device=DEV), torch.zeros(N, 0, dtype=torch.uint8, device=DEV)
    x, xs = (torch.zeros(M, 0, dtype=BF16, device=DEV), None) if kind == "bf16" else (w.new_zeros(M, 0), w.new_zeros(M, 0))
    r = torch.randn(M, N + 5, device=DEV).to(yt)[:, :N]
    out = torch.full((M + 1, N + 2), 9.0, dtype=yt, device=DEV)
    for res in (None, r):
        qgm.mx_gemm(x, w, ws, x_scales=xs, out=out[:M, :N], residual=res)
        assert torch.equal(out[:M, :N], torch.zeros_like(r) if res is None else r)
    assert bool((out[:M, N:] == 9).all()) and bool((out[M] == 9).all())
    qgm.mx_gemm(x, w, ws, x_scales=xs, out=out[:M, :N], residual=out[:M, :N])   # in place
    assert torch.equal(out[:M, :N], r)


def test_gemm_a_billion_rows():
    # offsets far past 32 bits, and more 64 x 64 tiles than the 2^32 - 1 lanes of a grid: larger ones are taken
    M, N, K = (1 << 30) + 70, 16, 32
    if torch.cuda.mem_get_info()[0] < 80 << 30:
        pytest.skip("needs 80 GB")
    rng = np.random.default_rng(0)
    x, xs = torch.zeros(M, K // 2, dtype=torch.uint8, device=DEV), torch.full((M, 1), 127, dtype=torch.uint8, device=DEV)
    few, fews, xv = make_x(rng, "mx", 6, K)
    at = torch.tensor([0, 1, 1 << 29, (1 << 30) - 1, M - 70, M - 1], device=DEV)
    x[at], xs[at] = few, fews
    wc, wsc = random_mx(rng, N, K)
    out = torch.full((M + 1, N), 9.0, dtype=F16, device=DEV)
    qgm.mx_gemm(x, dev(wc), dev(wsc), x_scales=xs, out=out[:M])
    ref, mag = mxref.mx_gemm_ref(xv, mxref.mx_values(wc, wsc))
    check(out[at], ref, mag, K)
    assert bool((out[M] == 9).all())
    out[at] = 0
    assert not any(bool(out[i:i + (1 << 27)].any()) for i in range(0, M - 70, 1 << 27)) and not bool(out[M - 70:M].any())


@pytest.mark.parametrize("kind", ["f16", "bf16"])
@pytest.mark.parametrize("M,N,K", [(9, 8192, 4128), (12, 8195, 4608), (16, 8200, 8192), (16, 8193, 9248)])
def test_gemm_two_column_blocks(monkeypatch, kind, M, N, K):
    # 9 to 16 rows against many columns of a long K: two column blocks share a reading of x.  Columns that
    # end inside the first block of a pair, inside the second and with it; K that ends inside a chunk
    monkeypatch.setenv("QMX_TILE", "0")
    assert qgm.mx_plan(M, N, K, qgm.MX_F16)["blocks"] == 2
    rng = np.random.default_rng(M + N + K)
    wc, wsc = random_mx(rng, N, K, spread=0)
    w, wv = dev(wc), mxref.mx_values(wc, wsc)
    x, _, xv = make_x(rng, kind, M, K, exact=True)
    out = torch.full((M + 1, N), 9.0, dtype=F32, device=DEV)
    qgm.mx_gemm(x, w, dev(wsc), out=out[:M])
    assert np.array_equal(f64(out[:M]), mxref.mx_gemm_ref(xv, wv)[0])
    assert bool((out[M] == 9).all())
    # every size of scale, also past fp16's; a residual
    wsc = rng.integers(95, 150, wsc.shape).astype(np.uint8)
    x, _, xv = make_x(rng, kind, M, K)
    r = torch.randn(M, N, dtype=F32)
    ref, mag = mxref.mx_gemm_ref(xv, mxref.mx_values(wc, wsc), residual=f64(r))
    check(qgm.mx_gemm(x, w, dev(wsc), out_dtype=F32, residual=r.to(DEV)), ref, mag, K)


@pytest.mark.parametrize("kind", ["f16", "bf16"])
@pytest.mark.parametrize("sizes", [[10, 0, 9, 21], [33, 1, 0, 6]])
def test_grouped_two_column_blocks(monkeypatch, kind, sizes):
    monkeypatch.setenv("QMX_TILE", "0")
    rng = np.random.default_rng(sizes[0])
    E, N, K = len(sizes), 4100, 8192
    off, T = make_groups(sizes), sum(sizes)
    assert qgm.mx_plan(T, N, K, qgm.MX_F16, groups=E)["blocks"] == 2
    rows, scale = rng.integers(-1, 13, T).astype(np.int32), rng.standard_normal(T).astype(np.float32)
    x, _, xv = make_x(rng, kind, 12, K)
    wc, wsc = random_mx(rng, E * N, K)
    out = torch.full((T + 1, N), 9.0, dtype=F32, device=DEV)
    qgm.mx_gemm_grouped(x, dev(wc).view(E, N, -1), dev(wsc).view(E, N, -1), dev(off), rows=dev(rows),
                        row_scale=dev(scale), out=out[:T])
    ref, mag = mxref.mx_grouped_ref(xv, mxref.mx_values(wc, wsc).reshape(E, N, K), off, rows, scale)
    check(out[:T], ref, mag, K)
    assert bool((out[T] == 9).all())


@pytest.mark.parametrize("kind", ["f16", "bf16", "mx"])
@pytest.mark.parametrize("sizes", [[0] * 15 + [23] + [0] * 4, [9, 0, 17] + [0] * 20, [0, 64] + [0] * 30, [8, 16, 1] + [0] * 12],
                         ids=lambda s: "-".join(map(str, s[:4])))
@pytest.mark.parametrize("N,K", [(50, 416), (50, 1024), (1030, 4128), (70, 9248)])
def test_grouped_skewed_router(monkeypatch, kind, sizes, N, K):
    # few slots a matrix on average, most of them one expert's: its rows go eight (16-bit x) at a time through
    # the same workgroup, with K below a chunk, one chunk a wave and several
    monkeypatch.setenv("QMX_TILE", "0")
    rng = np.random.default_rng(sum(sizes) + K)
    E, off, T, xr = len(sizes), make_groups(sizes), sum(sizes), 11
    assert T <= 2 * E
    rows, scale = rng.integers(-1, xr, T).astype(np.int32), rng.standard_normal(T).astype(np.float32)
    x, xs, xv = make_x(rng, kind, xr, K)
    used = [e for e in range(E) if sizes[e]]
    wc, wsc = np.zeros((E, N, K // 2), dtype=np.uint8), np.full((E, N, K // 32), 255, dtype=np.uint8)   # others: NaN
    for e in used:
        wc[e], wsc[e] = random_mx(rng, N, K)
    wv = np.zeros((E, N, K))
    for e in used:
        wv[e] = mxref.mx_values(wc[e], wsc[e])
    out = torch.full((T + 1, N), 9.0, dtype=F32, device=DEV)
    qgm.mx_gemm_grouped(x, dev(wc), dev(wsc), dev(off), x_scales=xs, rows=dev(rows), row_scale=dev(scale), out=out[:T])
    ref, mag = mxref.mx_grouped_ref(xv, wv, off, rows, scale)
    check(out[:T], ref, mag, K)
    assert bool((out[T] == 9).all())


# -------------------------------------------- as used together, graphs, streams

def moe(x, up, down, offsets, rows, scale):
    """An experts' block: 4-bit activations into the first product, a squared
    ReLU, 16-bit ones into the second, the router's factor in its rounding."""
    codes, scales = qgm.mx_quantize(x)
    h = qgm.mx_gemm_grouped(codes, *up, offsets, x_scales=scales, rows=rows, out_dtype=BF16)
    h = torch.relu(h) ** 2
    return h, qgm.mx_gemm_grouped(h, *down, offsets, row_scale=scale)


@pytest.mark.parametrize("tokens", [5, 300])
def test_chain_and_its_graph(tokens):
    rng = np.random.default_rng(tokens)
    E, D, F, top = 6, 160, 288, 2
    up, down = random_mx(rng, E * F, D), random_mx(rng, E * D, F)
    dup = [dev(a).reshape(E, F, -1) for a in up]
    ddn = [dev(a).reshape(E, D, -1) for a in down]
    ids = rng.integers(0, E, tokens * top)
    order = np.argsort(ids, kind="stable")
    off = make_groups(np.bincount(ids, minlength=E))
    rows = (order // top).astype(np.int32)
    scale = rng.random(tokens * top).astype(np.float32)
    x = torch.from_numpy(rng.standard_normal((tokens, D)).astype(np.float32)).to(DEV, BF16)
    args = (dup, ddn, dev(off), dev(rows), dev(scale))
    h, y = moe(x, *args)
    xv = mxref.mx_values(*mxref.mx_quantize(f64(x)))
    ref, mag = mxref.mx_grouped_ref(xv, mxref.mx_values(*up).reshape(E, F, D), off, rows)
    pre = torch.from_numpy(np.maximum(ref, 0) ** 2)
    # the first product's rounding passes through the square: compare h loosely, y from h itself
    assert np.allclose(f64(h), pre.numpy(), rtol=2 ** -6, atol=1e-2 * float(mag.max()))
    ref, mag = mxref.mx_grouped_ref(f64(h), mxref.mx_values(*down).reshape(E, D, F), off, row_scale=scale)
    check(y, ref, mag, F)
    static = x.clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        moe(static, *args)
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        _, captured = moe(static, *args)
    for i in range(4):
        fresh = torch.from_numpy(rng.standard_normal((tokens, D)).astype(np.float32)).to(DEV, BF16)
        _, eager = moe(fresh, *args)
        static.copy_(fresh)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(captured, eager), i


def test_products_on_a_named_stream():
    rng = np.random.default_rng(0)
    x, _, xv = make_x(rng, "f16", 40, 256)
    wc, wsc = random_mx(rng, 96, 256)
    w, ws = dev(wc), dev(wsc)
    ref, mag = mxref.mx_gemm_ref(xv, mxref.mx_values(wc, wsc))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    lin = qgm.MXLinear(w, ws)
    y = lin(x, stream=s)
    z = qgm.mx_gemm_grouped(x, w[None], ws[None], torch.tensor([0, 40], dtype=torch.int32, device=DEV), stream=s)
    c, sc = qgm.mx_quantize(x, stream=s)
    v = qgm.mx_dequantize(c, sc, stream=s)
    s.synchronize()
    check(y, ref, mag, 256)
    check(z, ref, mag, 256)
    assert np.array_equal(f64(v), rounded(mxref.mx_values(*mxref.mx_quantize(xv)), F16))


def test_binding_refuses():
    x = torch.zeros(4, 64, dtype=F16, device=DEV)
    w, ws = torch.zeros(8, 32, dtype=torch.uint8, device=DEV), torch.zeros(8, 2, dtype=torch.uint8, device=DEV)
    off = torch.tensor([0, 4], dtype=torch.int32, device=DEV)
    xc, xs = w[:4], ws[:4]
    bad = [
        lambda: qgm.mx_quantize(x[:, :48]), lambda: qgm.mx_quantize(x.t()), lambda: qgm.mx_quantize(x.double()),
        lambda: qgm.mx_quantize(x[0]), lambda: qgm.mx_quantize(x, codes=w), lambda: qgm.mx_quantize(x, scales=ws),
        lambda: qgm.mx_dequantize(w, ws[:4]), lambda: qgm.mx_dequantize(w[:, ::2], ws),
        lambda: qgm.mx_dequantize(w, ws, dtype=torch.int8), lambda: qgm.mx_dequantize(w, ws, out=x),
        lambda: qgm.mx_gemm(x.float(), w, ws), lambda: qgm.mx_gemm(x[:, :32], w, ws),
        lambda: qgm.mx_gemm(x, w.int(), ws), lambda: qgm.mx_gemm(x, w, ws[:, :1]), lambda: qgm.mx_gemm(x, w, ws.cpu()),
        lambda: qgm.mx_gemm(xc, w, ws), lambda: qgm.mx_gemm(xc, w, ws, x_scales=xs[:3]),
        lambda: qgm.mx_gemm(x, w, ws, x_scales=xs), lambda: qgm.mx_gemm(x, w, ws, out_dtype=torch.float64),
        lambda: qgm.mx_gemm(x, w, ws, out=x), lambda: qgm.mx_gemm(x, w, ws, residual=x),
        lambda: qgm.mx_gemm(x, w, ws, residual=torch.zeros(4, 8, device=DEV)),
        lambda: qgm.mx_gemm(x, w, ws, out=torch.zeros(4, 8, device=DEV), out_dtype=F16),
        lambda: qgm.mx_gemm_grouped(x, w, ws, off), lambda: qgm.mx_gemm_grouped(x, w[None], ws[None], off.long()),
        lambda: qgm.mx_gemm_grouped(x, w[None], ws[None], off[:1]),
        lambda: qgm.mx_gemm_grouped(x, w[None], ws[None], off, rows=off.float()),
        lambda: qgm.mx_gemm_grouped(x, w[None], ws[None], off, rows=off, row_scale=torch.ones(3, device=DEV)),
        lambda: qgm.mx_gemm_grouped(x, w[None], ws[None], off, row_scale=torch.ones(4, device=DEV, dtype=F16)),
    ]
    for call in bad:
        with pytest.raises(ValueError):
            call()
    with pytest.raises(qgm.QGemmError):
        qgm.mx_quantize(torch.zeros(4, 72, dtype=F16, device=DEV)[:, 4:68])   # rows not 16-byte aligned
