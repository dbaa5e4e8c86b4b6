"""The 8-bit floating-point operators (E4M3, blocks of 128) on the GPU against
the oracle in 64 bits.

Tolerances.  Quantising is exact (codes and scales bit for bit), as are products
whose terms and partial sums are integers times one power of two below 2^24.
Elsewhere an fp32 sum of a product over K is off by at most SUM(K) times the sum
of the terms' magnitudes: K additions within the blocks and one more for each
block, each off by at most a whole unit (2^-23, matrix cores need not round to
nearest), the factor of a block (two scales) and its product 2^-24 each, a
residual's addition 2^-24.  A stored value is off by half a step more (eps / 2 of
its type, or half its smallest subnormal).

With 8-bit x, W in blocks of 128 and bf16 results the larger kernels use 8-bit
matrix instructions, which add the products of 8 consecutive k on a grid of
2^(e - 13), e the largest sum of two codes' exponents among them (a subnormal
code's is -6), and cut what is finer.  The product that has e is a multiple of
2^(e - 6), so at most seven are cut: CUT() bounds that by 7 2^-13 times the
largest |x| times the largest |w| of every 8.

The gate g s(t), s the logistic function: e = exp(-|t|) is off by (|t| + 1) 2^-23
of itself (the product with log2 e rounds twice, exp2 is good to a unit), 1 + e,
its reciprocal and their product by 2.5 2^-23 more, and t, for gelu a polynomial
of six roundings, by 3 |t| 2^-23, which moves s by no more than that part of
itself.  So s and 1 - s are good to (4 |t| + 4) 2^-23 (e below 2^-126 is 0), the
value to (4 |t| + 6) 2^-23, and the slope's two terms to (8 |t| + 16) 2^-23.  Errors
of g and u go through with |act'| <= 1.2 and |act''| <= 1."""
import numpy as np
import pytest

from oracle import f8ref

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU visible", allow_module_level=True)
import bit_weight_only_dequant_amd as qgm  # noqa: E402

DEV = "cuda:0"
F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32
TINY = {F16: 2.0 ** -24, BF16: 2.0 ** -133, F32: 2.0 ** -149}
CODE = torch.float8_e4m3fn
XTYPE = {"f16": F16, "bf16": BF16}
U = 2.0 ** -23


def dev(a):
    """A NumPy array on the GPU, bytes as codes."""
    t = torch.from_numpy(np.ascontiguousarray(a)).to(DEV)
    return t.view(CODE) if t.dtype == torch.uint8 else t


def f64(t):
    return t.detach().cpu().double().numpy()


def codes_of(t):
    return t.view(torch.uint8).cpu().numpy()


def stored(ref, dtype):
    """What storing adds to the tolerance of ref."""
    return torch.finfo(dtype).eps / 2 * np.abs(ref) + TINY[dtype] / 2


def sums(K, mag):
    return (K + -(-K // 128) + 4) * U * mag


def eights(codes, scales):
    """The largest magnitude of every 8 consecutive k, at least 2^-6 times the scale."""
    R, K = codes.shape
    top = np.maximum(np.abs(f8ref.VALUES[codes]), 2.0 ** -6).reshape(R, K // 8, 8).max(axis=2)
    s = np.repeat(np.abs(scales.astype(np.float64)), 16, axis=1)[:, :K // 8]
    return top * (s if scales.shape[0] == R else np.repeat(s, 128, axis=0)[:R])


def cut(x, xs, wc, ws, yt):
    """What 8-bit matrix instructions may leave out (see above); 0 where they are not used."""
    if xs is None or yt != BF16 or (ws.shape[0] == wc.shape[0] and len(wc) > 1):
        return 0.0
    return 7 * 2.0 ** -13 * (eights(codes_of(x), xs.cpu().numpy()) @ eights(wc, ws).T)


def inside(y, ref, tol):
    tol = tol * (1 + torch.finfo(y.dtype).eps) + stored(ref, y.dtype)
    err = np.abs(f64(y) - ref)
    assert (err <= tol).all(), (np.unravel_index(np.argmax(err - tol), err.shape), (err / np.maximum(tol, 1e-300)).max())


def rounded(ref, dtype):
    """float64 (exact in fp32) rounded once to dtype, as float64."""
    return f64(torch.from_numpy(np.asarray(ref, dtype=np.float32)).to(dtype))


def random_f8(rng, R, K, block, size=1.0):
    """Random codes (no NaN) of every size, and scales that differ from block to block."""
    codes = rng.integers(0, 255, (R, K), dtype=np.uint8)
    codes[codes == 127] = 3
    scales = rng.uniform(0.5, 2, (-(-R // block), -(-K // 128))) * size / 64
    return codes, scales.astype(np.float32)


def exact_f8(rng, R, K, block, top=4):
    """Integers to `top` with one scale, a power of two."""
    v = torch.from_numpy(rng.integers(-top, top + 1, (R, K)).astype(np.float32)).to(CODE).view(torch.uint8).numpy()
    return v, np.full((-(-R // block), -(-K // 128)), 0.5, dtype=np.float32)


def make_x(rng, kind, M, K, exact=False):
    """(device x, device x_scales, float64 values)."""
    if kind == "f8":
        c, s = exact_f8(rng, M, K, 1) if exact else random_f8(rng, M, K, 1)
        return dev(c), dev(s), f8ref.f8_values(c, s)
    v = rng.integers(-4, 5, (M, K)) if exact else rng.standard_normal((M, K))
    t = torch.from_numpy(v.astype(np.float32)).to(XTYPE[kind])
    return t.to(DEV), None, f64(t)


# ------------------------------------------------------------------- quantise

def check_quantize(x, block, transpose, given=None):
    """x (on the CPU) through the kernel, with guards behind the outputs."""
    want_c, want_s = f8ref.f8_quantize(x.double().numpy(), block, transpose)
    codes = torch.full((want_c.shape[0] + 2, want_c.shape[1]), 77, dtype=torch.uint8, device=DEV).view(CODE)
    scales = torch.full((want_s.shape[0] + 2, want_s.shape[1]), 77.0, device=DEV)
    c, s = codes[:want_c.shape[0]], scales[:want_s.shape[0]]
    qgm.f8_quantize(x.to(DEV) if given is None else given, block=block, transpose=transpose, codes=c, scales=s)
    assert np.array_equal(s.cpu().numpy(), want_s, equal_nan=True)
    bad = np.argwhere(codes_of(c) != want_c)
    assert len(bad) == 0, (len(bad), bad[0], codes_of(c)[tuple(bad[0])], want_c[tuple(bad[0])])
    assert (codes_of(codes)[want_c.shape[0]:] == 77).all() and bool((scales[want_s.shape[0]:] == 77).all())


@pytest.mark.parametrize("block,transpose", [(1, False), (1, True), (128, False), (128, True)])
@pytest.mark.parametrize("dtype", [F16, BF16, F32])
def test_quantize_every_pattern(dtype, block, transpose):
    # every 16-bit pattern (for fp32: random patterns, subnormals and all exponents), each in a block of its
    # neighbours and in one of numbers of other sizes; infinities and NaN in some blocks only
    rng = np.random.default_rng(3)
    if dtype == F32:
        x = torch.from_numpy(rng.integers(0, 1 << 32, (512, 128), dtype=np.uint32).view(np.float32))
        x[:128] = torch.from_numpy(rng.integers(0, 1 << 25, (128, 128), dtype=np.uint32).view(np.float32))
        x[128:256] = torch.where(torch.isfinite(x[128:256]), x[128:256], torch.zeros(()))
    else:
        bits = np.arange(65536, dtype=np.uint16)
        x = torch.from_numpy(bits.view(np.int16).copy()).view(dtype).reshape(512, 128)
        x = torch.cat([x, x.reshape(128, 512).t().contiguous()])
    check_quantize(x, block, transpose)


@pytest.mark.parametrize("block,transpose", [(1, False), (1, True), (128, False), (128, True)])
@pytest.mark.parametrize("dtype", [F16, BF16, F32])
def test_quantize_middles(dtype, block, transpose):
    # quotients that are middles between two codes, and their neighbours in x's type, for many A
    rng = np.random.default_rng(4)
    tops = np.concatenate([np.arange(128, 256), rng.integers(1 << 10, 1 << 11, 64)])
    out = []
    for a in tops:
        mids = []
        for b in rng.permutation(126)[:43]:
            mid = (f8ref.VALUES[b] + f8ref.VALUES[b + 1]) / 2 * float(a) / 448
            t = torch.tensor(mid, dtype=torch.float64).to(dtype)
            mids += [float(t), float(torch.nextafter(t, t * 0)), float(torch.nextafter(t, t * 0 + 60000))]
        out.append(np.concatenate([[float(a)], rng.permutation(mids)[:127]]))
    x = torch.from_numpy(np.array(out)).to(dtype) * torch.from_numpy(rng.choice([-1.0, 1.0], (len(tops), 128))).to(dtype)
    if block == 128 or transpose:   # a tile of one A
        x = torch.cat([x[i:i + 1].repeat(16, 1) for i in range(0, len(tops), 24)])
        if transpose:
            x = torch.cat([x[16 * i:16 * i + 1].reshape(128, 1).repeat(1, 16) for i in range(len(x) // 16)], dim=1)
    check_quantize(x, block, transpose)


@pytest.mark.parametrize("block,transpose", [(1, False), (1, True), (128, False), (128, True)])
@pytest.mark.parametrize("dtype", [F16, BF16, F32])
@pytest.mark.parametrize("M,K", [(1, 16), (3, 144), (257, 2064), (1, 8192), (1000, 48), (128, 128), (15, 4112), (16, 240)])
def test_quantize_sizes_and_strides(dtype, block, transpose, M, K):
    rng = np.random.default_rng(M + K)
    v = rng.standard_normal((M, K)) * np.exp2(rng.integers(-9, 9, (M, 1)))
    x = torch.from_numpy(v.astype(np.float32)).to(dtype)
    wide = torch.full((M, K + 24), float("nan"), dtype=dtype, device=DEV)
    wide[:, 8:8 + K] = x.to(DEV)
    for given in (None, wide[:, 8:8 + K]):
        check_quantize(x, block, transpose, given)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_quantize_ends_of_the_range(dtype):
    # the largest and the smallest numbers of the type, zeros of both signs, a block below the least A
    x = torch.zeros(6, 256, dtype=dtype)
    x[0, :4] = torch.tensor([torch.finfo(dtype).max, -torch.finfo(dtype).max / 3, 1.0, -0.0], dtype=dtype)
    x[1, :4] = torch.tensor([2.0 ** -126, 2.0 ** -133, -(2.0 ** -127), 2.0 ** -110], dtype=dtype)
    x[2, 128:131] = torch.tensor([2.0 ** -100, 2.0 ** -101, 2.0 ** -99], dtype=dtype)
    x[3, 5] = float("inf")
    x[4, 130] = float("nan")
    for block, transpose in ((1, False), (1, True), (128, False), (128, True)):
        check_quantize(x, block, transpose)


@pytest.mark.parametrize("block", [1, 128])
@pytest.mark.parametrize("dtype", [F16, BF16, F32])
@pytest.mark.parametrize("M,K", [(1, 16), (3, 256), (257, 2064), (1000, 48), (130, 144)])
def test_dequantize(dtype, block, M, K):
    # every code, scales of every size; one fp32 rounding, and one to 16 bits
    rng = np.random.default_rng(M + K)
    codes = rng.permutation(np.arange(M * K) % 256).astype(np.uint8).reshape(M, K)
    scales = (rng.uniform(0.5, 2, (-(-M // block), -(-K // 128))) * np.exp2(rng.integers(-12, 6, (-(-M // block), 1)))).astype(np.float32)
    with np.errstate(over="ignore"):
        want = rounded(f8ref.f8_values(codes, scales), dtype)
    out = torch.full((M + 1, K + 16), 5.0, dtype=dtype, device=DEV)
    for y in (qgm.f8_dequantize(dev(codes), dev(scales), dtype=dtype), qgm.f8_dequantize(dev(codes), dev(scales), out=out[:M, 8:K + 8])):
        assert np.array_equal(f64(y), want, equal_nan=True)
    assert bool((out[M] == 5).all()) and bool((out[:, :8] == 5).all()) and bool((out[:, K + 8:] == 5).all())


@pytest.mark.parametrize("M,K", [(0, 64), (4, 0)])
def test_quantize_empty(M, K):
    for block in (1, 128):
        codes, scales = qgm.f8_quantize(torch.zeros(M, K, dtype=F16, device=DEV), block=block)
        assert qgm.f8_dequantize(codes, scales).shape == (M, K)
        assert codes.shape == (M, K) and scales.shape == (M if block == 1 else -(-M // 128), -(-K // 128))
        codes, scales = qgm.f8_quantize(torch.zeros(M, K, dtype=F16, device=DEV), block=block, transpose=True)
        assert codes.shape == (K, -(-M // 16) * 16)


def test_quantize_far_offsets():
    # rows and columns that lie more than 4 GiB into the arrays
    M, K = 70000, 65536
    x = torch.zeros(M, K, dtype=BF16, device=DEV)
    x[M - 3:] = torch.randn(3, K, device=DEV).to(BF16)
    want_c, want_s = f8ref.f8_quantize(f64(x[M - 3:]))
    codes, scales = qgm.f8_quantize(x)
    assert np.array_equal(codes_of(codes[M - 3:]), want_c) and np.array_equal(scales[M - 3:].cpu().numpy(), want_s)
    assert not bool(codes[:M - 3].view(torch.uint8).any())
    back = qgm.f8_dequantize(codes, scales, dtype=F32)      # 17 GiB
    assert np.array_equal(f64(back[M - 3:]), rounded(f8ref.f8_values(want_c, want_s), F32)) and not bool(back[:M - 3].any())
    del back
    tail = x[M - M % 128:, K - 16:]
    want_c, want_s = f8ref.f8_quantize(f64(tail), transpose=True)
    codes, scales = qgm.f8_quantize(x, transpose=True)
    assert codes.shape == (K, M)
    assert np.array_equal(codes_of(codes[K - 16:, M - M % 128:]), want_c)
    assert np.array_equal(scales[K - 16:, -1:].cpu().numpy(), want_s)


# ------------------------------------------------------------------- products

KINDS = ["f16", "bf16", "f8"]
SIZES = [(1, 1, 16), (1, 16, 64), (1, 250, 2048), (2, 17, 96), (7, 33, 160), (15, 64, 128), (16, 100, 272),
         (17, 48, 512), (31, 16, 1040), (33, 130, 112), (63, 257, 256), (64, 128, 128), (65, 96, 528), (100, 65, 2064),
         (127, 300, 32), (129, 129, 240), (200, 512, 384), (257, 200, 1024), (300, 777, 784), (513, 1030, 272),
         (1100, 530, 400)]


@pytest.mark.parametrize("kind", KINDS + ["rows"])
@pytest.mark.parametrize("M,N,K", SIZES)
def test_gemm_exact_integers(kind, M, N, K):
    # every partial sum is a multiple of 2^-2 below K * 16, exact in fp32; "rows": W in blocks of 1
    rng = np.random.default_rng(M * 7 + N + K)
    block = 1 if kind == "rows" else 128
    x, xs, xv = make_x(rng, "f8" if kind == "rows" else kind, M, K, exact=True)
    wc, ws = exact_f8(rng, N, K, block)
    if block == 1:
        ws *= 2.0 ** rng.integers(-2, 3, ws.shape)
    else:
        ws *= 2.0 ** rng.integers(-1, 2, ws.shape)
    ref, _ = f8ref.f8_gemm_ref(xv, f8ref.f8_values(wc, ws))
    for yt in (F32, XTYPE.get(kind, BF16)):
        out = torch.full((M + 1, N), 9.0, dtype=yt, device=DEV)
        y = qgm.f8_gemm(x, dev(wc), dev(ws), x_scales=xs, out=out[:M])
        assert np.array_equal(f64(y), rounded(ref, yt))
        assert bool((out[M] == 9).all())


@pytest.mark.parametrize("kind", KINDS + ["rows"])
@pytest.mark.parametrize("yt", [F16, BF16, F32])
@pytest.mark.parametrize("M,N,K", [(1, 300, 2048), (5, 77, 96), (40, 129, 592), (130, 260, 1040), (600, 333, 512)])
def test_gemm_random_with_residual_and_strides(kind, yt, M, N, K):
    rng = np.random.default_rng(M + N * 3 + K)
    x, xs, xv = make_x(rng, "f8" if kind == "rows" else kind, M, K)
    if xs is None:
        wide = torch.full((M, K + 16), float("nan"), dtype=x.dtype, device=DEV)
        wide[:, :K] = x
        x = wide[:, :K]
    wc, ws = random_f8(rng, N, K, 1 if kind == "rows" else 128, size=0.05)
    r = torch.randn(M, N + 3, dtype=F32).to(yt)
    out = torch.full((M, N + 5), 9.0, dtype=yt, device=DEV)
    ref, mag = f8ref.f8_gemm_ref(xv, f8ref.f8_values(wc, ws), residual=f64(r[:, :N]))
    qgm.f8_gemm(x, dev(wc), dev(ws), x_scales=xs, out=out[:, :N], residual=r.to(DEV)[:, :N])
    inside(out[:, :N], ref, sums(K, mag) + cut(x, xs, wc, ws, yt))
    assert bool((out[:, N:] == 9).all())
    # in place: the residual is the output itself
    y = r.to(DEV).contiguous()[:, :N].clone()
    qgm.f8_gemm(x, dev(wc), dev(ws), x_scales=xs, out=y, residual=y)
    assert torch.equal(y, out[:, :N])


@pytest.mark.parametrize("kind", KINDS + ["rows"])
@pytest.mark.parametrize("M,N,K", [(3, 40, 96), (20, 270, 416), (70, 90, 416), (300, 270, 672)])
def test_gemm_nan_and_inf_stay_in_their_row_and_column(kind, M, N, K):
    rng = np.random.default_rng(M * N)
    x, xs, xv = make_x(rng, "f8" if kind == "rows" else kind, M, K)
    wc, ws = random_f8(rng, N, K, 1 if kind == "rows" else 128)
    wc[5, K - 1] = 127
    wc[N - 1, 0] = 255
    if kind == "rows":
        ws[7, -1] = np.nan
    if xs is not None:
        xs[1, 0] = float("nan")
        x.view(torch.uint8)[2, K - 1] = 127
        xv = f8ref.f8_values(codes_of(x), xs.cpu().numpy())
    else:
        x[1, 3] = float("nan")
        x[2, K - 1] = float("inf")
        xv = f64(x)
    y = f64(qgm.f8_gemm(x, dev(wc), dev(ws), x_scales=xs, out_dtype=F32))
    wv = f8ref.f8_values(wc, ws)
    with np.errstate(invalid="ignore"):
        ref, _ = f8ref.f8_gemm_ref(xv, wv)
        gap = np.abs(y - ref)
    assert np.array_equal(np.isnan(y), np.isnan(ref)) and np.array_equal(np.isinf(y), np.isinf(ref))
    ok = np.isfinite(ref)
    mag = np.abs(np.nan_to_num(xv, posinf=0)) @ np.abs(np.nan_to_num(wv)).T
    assert (gap[ok] <= (sums(K, mag) + U * mag + 2.0 ** -149)[ok]).all()


@pytest.mark.parametrize("kind", KINDS + ["rows"])
@pytest.mark.parametrize("M,N,K", [(3, 40, 272), (40, 130, 528), (300, 300, 1024)])
def test_gemm_scales_of_every_size(kind, M, N, K):
    # blocks whose scales differ by many powers of two: a block's sum must meet its own scales
    rng = np.random.default_rng(M + K)
    x, xs, xv = make_x(rng, "f8" if kind == "rows" else kind, M, K)
    wc, ws = random_f8(rng, N, K, 1 if kind == "rows" else 128)
    ws = (ws * np.exp2(rng.integers(-20, 20, ws.shape))).astype(np.float32)
    if xs is not None:
        xs = (xs * torch.exp2(torch.randint(-20, 20, xs.shape, device=DEV).float())).contiguous()
        xv = f8ref.f8_values(codes_of(x), xs.cpu().numpy())
    ref, mag = f8ref.f8_gemm_ref(xv, f8ref.f8_values(wc, ws))
    inside(qgm.f8_gemm(x, dev(wc), dev(ws), x_scales=xs, out_dtype=F32), ref, sums(K, mag))


@pytest.mark.parametrize("kind", KINDS + ["rows"])
@pytest.mark.parametrize("M", [1, 7, 9, 16])
@pytest.mark.parametrize("N,K", [(200, 8192), (4200, 4112), (40, 20000), (140000, 48)])
def test_gemm_few_rows(kind, M, N, K):
    # several chunks a wave, x in as much LDS as there is, workgroups with several column blocks
    rng = np.random.default_rng(M + K)
    x, xs, xv = make_x(rng, "f8" if kind == "rows" else kind, M, K)
    wc, ws = random_f8(rng, N, K, 1 if kind == "rows" else 128)
    ref, mag = f8ref.f8_gemm_ref(xv, f8ref.f8_values(wc, ws))
    inside(qgm.f8_gemm(x, dev(wc), dev(ws), x_scales=xs, out_dtype=F32), ref, sums(K, mag))


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("M,N,K", [(0, 16, 64), (4, 0, 64), (3, 18, 0), (2, 140000, 0), (70000, 30, 0), (1100000, 3, 0)])
def test_gemm_empty(kind, M, N, K):
    x = torch.zeros(M, K, dtype=XTYPE.get(kind, F16), device=DEV)
    xs = None
    if kind == "f8":
        x, xs = torch.zeros(M, K, dtype=torch.uint8, device=DEV).view(CODE), torch.zeros(M, -(-K // 128), device=DEV)
    w = torch.zeros(N, K, dtype=torch.uint8, device=DEV).view(CODE)
    ws = torch.zeros(-(-N // 128), -(-K // 128), device=DEV)
    r = torch.randn(M, N, device=DEV).to(BF16)
    assert torch.equal(qgm.f8_gemm(x, w, ws, x_scales=xs, residual=r, out_dtype=BF16), r)
    assert not bool(qgm.f8_gemm(x, w, ws, x_scales=xs, out_dtype=F32).any())


# every kernel whatever the rule would take: sizes around their tiles, K that ends inside a stage of 128 and on it
EVERY = [(1, 129, 512), (70, 257, 528), (17, 64, 992), (130, 300, 1024), (260, 70, 1600), (3, 40, 128), (66, 130, 336),
         (5, 17, 16), (129, 513, 480), (33, 100, 2512), (300, 530, 144), (600, 1100, 272)]


@pytest.mark.parametrize("tile", range(6))
@pytest.mark.parametrize("kind", KINDS + ["rows"])
@pytest.mark.parametrize("M,N,K", EVERY)
def test_gemm_every_kernel(monkeypatch, tile, kind, M, N, K):
    monkeypatch.setenv("QF8_TILE", str(tile))
    rng = np.random.default_rng(M + N + K)
    block, xk = (1, "f8") if kind == "rows" else (128, kind)
    wc, ws = exact_f8(rng, N, K, block)
    ws *= 2.0 ** rng.integers(-1, 2, ws.shape)
    x, xs, xv = make_x(rng, xk, M, K, exact=True)
    ref = f8ref.f8_gemm_ref(xv, f8ref.f8_values(wc, ws))[0]
    for yt in (F32, F16, BF16):
        out = torch.full((M + 1, N + 3), 9.0, dtype=yt, device=DEV)
        qgm.f8_gemm(x, dev(wc), dev(ws), x_scales=xs, out=out[:M, :N])
        assert np.array_equal(f64(out[:M, :N]), rounded(ref, yt))
        assert bool((out[M] == 9).all()) and bool((out[:, N:] == 9).all())
    # codes and scales of every size, a NaN code and a NaN scale that reach their own columns only
    wc, ws = random_f8(rng, N, K, block)
    wc[N // 2, K - 1] = 255
    x, xs, xv = make_x(rng, xk, M, K)
    with np.errstate(invalid="ignore"):
        ref, mag = f8ref.f8_gemm_ref(xv, f8ref.f8_values(wc, ws))
    keep = np.arange(N) != N // 2
    left = cut(x, xs, np.where(wc == 255, 0, wc).astype(np.uint8), ws, BF16)
    for yt in (F32, BF16):
        y = qgm.f8_gemm(x, dev(wc), dev(ws), x_scales=xs, out_dtype=yt)
        assert bool(torch.isnan(y[:, N // 2]).all())
        tol = sums(K, mag) + (left if yt == BF16 else 0.0)
        inside(y[:, torch.from_numpy(keep).to(DEV)], ref[:, keep], tol[:, keep])


@pytest.mark.parametrize("tile", range(6))
@pytest.mark.parametrize("kind", KINDS)
def test_gemm_infinite_last_scale(monkeypatch, tile, kind):
    # three blocks along K: two groups of waves share them unevenly, and the last scale is infinite
    monkeypatch.setenv("QF8_TILE", str(tile))
    rng = np.random.default_rng(tile)
    M, N, K = 70, 40, 384
    x, xs, xv = make_x(rng, kind, M, K)
    wc, ws = random_f8(rng, N, K, 128)
    ws[0, 2] = np.inf
    wc[:, 256:] = 56                                        # 1.0: the last block's sum is x's
    wc[:, 257:] = 0
    x.view(torch.uint8 if kind == "f8" else torch.int16)[:, 256] &= 0x77 if kind == "f8" else 0x7777   # finite, its sign gone
    keep = f64(x[:, 256].float()) > 0
    for yt in (F32, BF16):
        y = f64(qgm.f8_gemm(x, dev(wc), dev(ws), x_scales=xs, out_dtype=yt))
        assert np.isposinf(y[keep]).all() and keep.sum() > 20


@pytest.mark.parametrize("tile", range(6))
@pytest.mark.parametrize("kind", KINDS)
def test_gemm_past_k_is_not_read_into_sums(monkeypatch, tile, kind):
    # rows whose neighbours in memory are NaN: x with a wide pitch, the last row of W before other codes
    monkeypatch.setenv("QF8_TILE", str(tile))
    rng = np.random.default_rng(tile)
    M, N, K = 37, 50, 176
    x, xs, xv = make_x(rng, kind, M, K)
    if xs is None:
        wide = torch.full((M + 1, K + 96), float("nan"), dtype=x.dtype, device=DEV)
        wide[:M, :K] = x
        x = wide[:M, :K]
    else:
        wide = torch.full((M + 300, K), 127, dtype=torch.uint8, device=DEV)
        wide[:M] = x.view(torch.uint8)
        x = wide.view(CODE)[:M]
    wc, ws = random_f8(rng, N, K, 128)
    w = torch.full((N + 300, K), 127, dtype=torch.uint8, device=DEV)
    w[:N] = dev(wc).view(torch.uint8)
    ref, mag = f8ref.f8_gemm_ref(xv, f8ref.f8_values(wc, ws))
    for yt in (F32, BF16):
        inside(qgm.f8_gemm(x, w.view(CODE)[:N], dev(ws), x_scales=xs, out_dtype=yt), ref,
               sums(K, mag) + cut(x, xs, wc, ws, yt))


@pytest.mark.parametrize("tile", range(6))
@pytest.mark.parametrize("kind", ["bf16", "f8"])
def test_gemm_far_rows(monkeypatch, tile, kind):
    # rows of x, of W and of y that lie more than 4 GiB into their arrays
    monkeypatch.setenv("QF8_TILE", str(tile))
    rng = np.random.default_rng(tile)
    K, far = 8192, 600000
    xc, s, xv = make_x(rng, kind, 3, K)
    x = torch.zeros(far, K, dtype=torch.uint8 if kind == "f8" else BF16, device=DEV)
    x[far - 3:] = xc.view(torch.uint8) if kind == "f8" else xc
    xs = None
    if kind == "f8":
        x, xs = x.view(CODE), torch.ones(far, K // 128, device=DEV)
        xs[far - 3:] = s
    wc, ws = random_f8(rng, 48, K, 128)
    y = qgm.f8_gemm(x, dev(wc), dev(ws), x_scales=xs, out_dtype=F32)
    ref, mag = f8ref.f8_gemm_ref(xv, f8ref.f8_values(wc, ws))
    inside(y[far - 3:], ref, sums(K, mag))
    assert not bool(y[:far - 3].any())
    del x, xs, y
    w = torch.zeros(far, K, dtype=torch.uint8, device=DEV)
    w[far - 48:] = dev(wc).view(torch.uint8)
    wsc = torch.ones(-(-far // 128), K // 128, device=DEV)
    wsc[-1:] = dev(ws)
    out = torch.full((3, far), 9.0, device=DEV)
    assert far % 128 == 64
    qgm.f8_gemm(xc, w.view(CODE), wsc, x_scales=s, out=out)
    inside(out[:, far - 48:], ref, sums(K, mag))
    assert not bool(out[:, :far - 48].any())
    del w, out
    big = torch.zeros(40, 1 << 27, dtype=F32, device=DEV)      # 20 GiB: y's own rows
    row = xc[:1].expand(40, K).contiguous()
    rs = None if s is None else s[:1].expand(40, K // 128).contiguous()
    qgm.f8_gemm(row, dev(wc), dev(ws), x_scales=rs, out=big[:, :48])
    inside(big[39:, :48], ref[:1], sums(K, mag[:1]))
    assert not bool(big[:, 48:64].any())


# ------------------------------------------------------- the gated block

ACTS = ["silu", "gelu_tanh"]
GATED = [(1, 16, 16), (1, 208, 2048), (3, 48, 96), (16, 64, 272), (17, 144, 512), (33, 32, 1040), (64, 128, 128),
         (65, 272, 240), (130, 176, 528), (257, 400, 384), (520, 1040, 272)]


def gate_tolerances(x, w, act, K, left=0.0):
    """(h, its tolerance before storing, and what the gradient's needs); left: what cut() gives."""
    F = w.shape[0] // 2
    h, g, u = f8ref.gated_ref(x, w, act)
    mag = np.abs(x) @ np.abs(w).T
    e = sums(K, mag) + left
    eg, eu = e[:, :F], e[:, F:]
    a, da = f8ref.act_ref(g, act)
    t = np.abs(g) if act == "silu" else 1.5957691216057308 * np.abs(g + 0.044715 * g ** 3)
    ea = (4 * t + 6) * U * np.abs(a) + 2.0 ** -126 * np.abs(g) + 1.2 * eg
    th = ea * np.abs(u) + (np.abs(a) + ea) * eu + U * np.abs(h)
    return h, th, (g, u, a, da, eg, eu, ea, t)


@pytest.mark.parametrize("tile", [None, 0, 1, 2, 3, 4, 5])
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("M,F,K", GATED)
def test_gated(monkeypatch, tile, kind, act, M, F, K):
    if tile is not None:
        monkeypatch.setenv("QF8_TILE", str(tile))
    rng = np.random.default_rng(M + F + K)
    x, xs, xv = make_x(rng, kind, M, K)
    wc, ws = random_f8(rng, 2 * F, K, 128, size=0.02 if kind != "f8" else 0.005)
    wv = f8ref.f8_values(wc, ws)
    for yt in (F32, XTYPE.get(kind, BF16)):
        h, tol, _ = gate_tolerances(xv, wv, act, K, cut(x, xs, wc, ws, yt))
        out = torch.full((M + 1, F + 3), 9.0, dtype=yt, device=DEV)
        y = qgm.f8_gated(x, dev(wc), dev(ws), x_scales=xs, act=act, out=out[:M, :F])
        inside(y, h, tol)
        assert bool((out[M] == 9).all()) and bool((out[:, F:] == 9).all())


@pytest.mark.parametrize("tile", [None, 0, 1, 2, 3, 4, 5])
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("M,F,K", GATED)
def test_gated_grad(monkeypatch, tile, kind, act, M, F, K):
    if tile is not None:
        monkeypatch.setenv("QF8_TILE", str(tile))
    rng = np.random.default_rng(M + F + K)
    x, xs, xv = make_x(rng, kind, M, K)
    wc, ws = random_f8(rng, 2 * F, K, 128, size=0.02 if kind != "f8" else 0.005)
    wv = f8ref.f8_values(wc, ws)
    for yt in (F32, XTYPE.get(kind, BF16)):
        _, _, (g, u, a, da, eg, eu, ea, t) = gate_tolerances(xv, wv, act, K, cut(x, xs, wc, ws, yt))
        dh = torch.randn(M, F + 2, device=DEV).to(yt)[:, :F]
        ref = f8ref.gated_grad_ref(f64(dh), xv, wv, act)
        # the slope's two terms: s, and g s (1 - s) t', which is what da leaves over
        s = np.where(g != 0, a / np.where(g != 0, g, 1), 0.5)
        es = (8 * t + 16) * U * (np.abs(s) + np.abs(da - s)) + 2.0 ** -126 * (1 + np.abs(g)) + eg
        d = np.abs(f64(dh))
        tol = np.concatenate([d * (es * np.abs(u) + (np.abs(da) + es) * eu), d * ea], axis=1) + 2 * U * np.abs(ref)
        out = torch.full((M + 1, 2 * F + 3), 9.0, dtype=yt, device=DEV)
        y = qgm.f8_gated_grad(dh, x, dev(wc), dev(ws), x_scales=xs, act=act, out=out[:M, :2 * F])
        inside(y, ref, tol)
        assert bool((out[M] == 9).all()) and bool((out[:, 2 * F:] == 9).all())


@pytest.mark.parametrize("act", ACTS)
def test_gate_far_from_zero(act):
    # one k, so that g is x itself: every exponent of g, both signs, u = 1 and dh = 1
    g = torch.cat([torch.exp2(torch.arange(-14, 16).float()) * f for f in (1.0, -1.0, 1.5, -1.75)] + [torch.zeros(1)]).to(F16)
    M = len(g)
    x = torch.zeros(M, 16, dtype=F16, device=DEV)
    x[:, 0], x[:, 1] = g.to(DEV), 1.0
    w = torch.zeros(32, 16)
    w[:16, 0], w[16:, 1] = 1.0, 1.0
    wc, ws = w.to(CODE).to(DEV), torch.ones(1, 1, device=DEV)
    v = g.double().numpy()
    a, da = f8ref.act_ref(v, act)
    t = np.abs(v) if act == "silu" else 1.5957691216057308 * np.abs(v + 0.044715 * v ** 3)
    h = qgm.f8_gated(x, wc, ws, act=act, out_dtype=F32)
    d = qgm.f8_gated_grad(torch.ones(M, 16, device=DEV), x, wc, ws, act=act)
    ea = (4 * t + 7) * U * np.abs(a) + 2.0 ** -126 * np.abs(v)
    s = np.where(v != 0, a / np.where(v != 0, v, 1), 0.5)
    es = (8 * t + 18) * U * (np.abs(s) + np.abs(da - s)) + 2.0 ** -126 * (1 + np.abs(v))
    for y, ref, tol in ((h, a, ea), (d[:, 16:], a, ea), (d[:, :16], da, es)):
        y = f64(y)
        assert (y == y[:, :1]).all() and (np.abs(y[:, 0] - ref) <= tol + stored(ref, F32)).all()


@pytest.mark.parametrize("M,F,K", [(0, 16, 64), (4, 0, 64), (3, 32, 0), (70, 48, 0), (1100000, 16, 0)])
def test_gated_empty(M, F, K):
    x = torch.zeros(M, K, dtype=BF16, device=DEV)
    w = torch.zeros(2 * F, K, dtype=torch.uint8, device=DEV).view(CODE)
    ws = torch.zeros(-(-2 * F // 128), -(-K // 128), device=DEV)
    h = qgm.f8_gated(x, w, ws)
    d = qgm.f8_gated_grad(torch.ones(M, F, dtype=BF16, device=DEV), x, w, ws)
    assert h.shape == (M, F) and d.shape == (M, 2 * F) and not bool(h.any()) and not bool(d.any())


# ------------------------------------------- together, streams, graphs, ends

def test_training_step():
    # as a training program calls them: weights quantised, forward, the projections' gradients, the input's and the
    # weight's gradient; each stage against the definition on what the one before gave
    torch.manual_seed(1)
    M, K, F = 150, 272, 144
    x = torch.randn(M, K, device=DEV).to(BF16)
    master = torch.randn(2 * F, K, device=DEV) * 0.05
    dh = torch.randn(M, F, device=DEV).to(BF16)
    block = qgm.F8Gated.from_weight(master, act="gelu_tanh")
    back = qgm.F8Linear.from_weight(master, transpose=True)
    assert torch.equal(back.codes.view(torch.uint8), block.codes.view(torch.uint8).t())
    xq, xs = qgm.f8_quantize(x)
    h = block(xq, x_scales=xs, out_dtype=BF16)
    xv = f8ref.f8_values(codes_of(xq), xs.cpu().numpy())
    wc, ws = codes_of(block.codes), block.scales.cpu().numpy()
    wv = f8ref.f8_values(wc, ws)
    ref, tol, _ = gate_tolerances(xv, wv, "gelu_tanh", K, cut(xq, xs, wc, ws, BF16))
    inside(h, ref, tol)
    d = block.grad(dh, xq, x_scales=xs)
    dx = back(d)                                            # 16-bit gradients ..
    ref, mag = f8ref.f8_gemm_ref(f64(d), wv.T)
    inside(dx, ref, sums(2 * F, mag))
    dq, ds = qgm.f8_quantize(d)                             # .. or in 8 bits
    dv = f8ref.f8_values(codes_of(dq), ds.cpu().numpy())
    ref, mag = f8ref.f8_gemm_ref(dv, wv.T)
    left = cut(dq, ds, codes_of(back.codes), back.scales.cpu().numpy(), BF16)
    inside(back(dq, x_scales=ds, out_dtype=BF16), ref, sums(2 * F, mag) + left)
    dt, dts = qgm.f8_quantize(d, transpose=True)
    xt, xts = qgm.f8_quantize(x, transpose=True)
    total = torch.randn(2 * F, K, device=DEV)
    dw = qgm.f8_gemm(dt, xt, xts, x_scales=dts, residual=total, out_dtype=F32)
    dtv, xtv = f8ref.f8_values(codes_of(dt), dts.cpu().numpy()), f8ref.f8_values(codes_of(xt), xts.cpu().numpy())
    ref, mag = f8ref.f8_gemm_ref(dtv, xtv, residual=f64(total))
    inside(dw, ref, sums(M + 10, mag))
    # and the whole against the gradients of the formula on the unrounded operands, by what 4 and 8 bits leave
    xd, wd = x.double().requires_grad_(), block_values(master).double().requires_grad_()
    p = xd @ wd.t()
    out = torch.nn.functional.gelu(p[:, :F], approximate="tanh") * p[:, F:]
    gx, gw = torch.autograd.grad(out, (xd, wd), dh.double())
    for got, want in ((dx, gx), (dw - total, gw)):
        gap = (got.double() - want).norm() / want.norm()
        assert gap < 0.08, gap   # elements off by up to 2^-4 each, 2^-5 in the mean square, of up to three factors


def block_values(master):
    c, s = f8ref.f8_quantize(f64(master), 128)
    return torch.from_numpy(f8ref.f8_values(c, s)).to(DEV)


def small_set(kind="bf16", M=5, F=48, K=272, seed=0):
    rng = np.random.default_rng(seed)
    x, xs, _ = make_x(rng, kind, M, K)
    wc, ws = random_f8(rng, 2 * F, K, 128, size=0.02)
    return x, xs, dev(wc), dev(ws), torch.randn(M, F, device=DEV).to(BF16)


def all_of(x, xs, w, ws, dh):
    d = qgm.f8_gated_grad(dh, x, w, ws, x_scales=xs)
    dq, ds = qgm.f8_quantize(d, transpose=True)
    bq, bs = qgm.f8_quantize(d, block=128)
    return [qgm.f8_gated(x, w, ws, x_scales=xs, out_dtype=BF16), d, dq.view(torch.uint8), ds, bq.view(torch.uint8), bs,
            qgm.f8_gemm(x, w, ws, x_scales=xs, out_dtype=F32), qgm.f8_gemm(dq, dq, ds, x_scales=ds, out_dtype=F32)]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("M", [1, 5, 70, 300])
def test_equal_inputs_give_equal_bits(kind, M):
    s = small_set(kind, M, F=272, K=1040)
    first = all_of(*s)
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(first, all_of(*s)))


@pytest.mark.parametrize("kind", ["bf16", "f8"])
@pytest.mark.parametrize("M", [5, 300])
def test_another_stream_and_graph_replays(kind, M):
    s = small_set(kind, M)
    want = all_of(*s)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    x, xs, w, ws, dh = s
    h = qgm.f8_gated(x, w, ws, x_scales=xs, out_dtype=BF16, stream=side)
    side.synchronize()
    assert torch.equal(h, want[0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        all_of(*s)
        with torch.cuda.graph(graph, stream=side):
            got = all_of(*s)
    torch.cuda.current_stream().wait_stream(side)
    for seed in (1, 2, 3):
        other = small_set(kind, M, seed=seed)
        for a, b in zip(s, other):
            if a is not None:
                a.copy_(b)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, all_of(*other)))


def test_two_streams_at_once():
    # nothing is shared between calls: two sets on two streams, many times over
    sets = [small_set("f8", 300, F=272, K=1040, seed=1), small_set("bf16", 5, F=48, K=272, seed=2)]
    want = [all_of(*s) for s in sets]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(20):
        for i in (0, 1):
            with torch.cuda.stream(streams[i]):
                got[i].append(all_of(*sets[i]))
    torch.cuda.synchronize()
    for i in (0, 1):
        assert all(torch.equal(a, b) for r in got[i] for a, b in zip(r, want[i]))


@pytest.mark.parametrize("M", [1, 40, 300])
def test_rows_of_a_padded_batch_stand_alone(M):
    # rows behind the last sequence hold anything: the others are as without them
    x, xs, w, ws, dh = small_set("bf16", M + 9, F=64, K=400)
    clean = x.clone()
    x[M:] = float("nan")
    dh2 = dh.clone()
    dh2[M:] = float("inf")
    for got, want in ((qgm.f8_gemm(x, w, ws), qgm.f8_gemm(clean, w, ws)), (qgm.f8_gated(x, w, ws), qgm.f8_gated(clean, w, ws)),
                      (qgm.f8_gated_grad(dh2, x, w, ws), qgm.f8_gated_grad(dh, clean, w, ws)),
                      (qgm.f8_quantize(x)[0][:M].view(torch.uint8), qgm.f8_quantize(clean)[0][:M].view(torch.uint8))):
        assert torch.equal(got[:M], want[:M])


# ---------------------------------------- the ends of precision, range and pitch

@pytest.mark.parametrize("tile", range(6))
def test_large_products_cancel_within_eight(monkeypatch, tile):
    # 256 * 256 - 256 * 256 + 6 * 7 in every eight of w, one eight of each row of x: 42 times the scales.  Converted codes
    # give it exactly (every partial sum is an integer below 2^24); the 8-bit matrix instructions may cut up to 7 * 2^3
    # of it, as documented, so nothing of it need be left.
    monkeypatch.setenv("QF8_TILE", str(tile))
    M, N, K = 70, 64, 144
    xv, wv = np.zeros((M, K), np.float32), np.tile(np.array([256, 256] + [4] * 6, np.float32), (N, K // 8))
    for m in range(M):
        at = 8 * (m % (K // 8))
        xv[m, at:at + 8] = [256, -256] + [1.75] * 6
    xc, wc = (torch.from_numpy(v).to(CODE).view(torch.uint8).numpy() for v in (xv, wv))
    rng = np.random.default_rng(tile)
    xsn = np.exp2(rng.integers(-3, 4, (M, 2))).astype(np.float32)
    ws = np.exp2(rng.integers(-8, -4, (1, 2))).astype(np.float32)
    x, xs = dev(xc), dev(xsn)
    xd, wd = f8ref.f8_values(xc, xsn), f8ref.f8_values(wc, ws)
    ref, mag = f8ref.f8_gemm_ref(xd, wd)
    left = cut(x, xs, wc, ws, BF16)
    assert (ref == 42 * np.take_along_axis(xsn * ws, (np.arange(M) % (K // 8) // 16)[:, None], 1)).all()
    assert (left >= ref).all() and (left <= 57 * xsn.max(1, keepdims=True) * ws.max()).all()
    for yt in (F32, F16):
        assert np.array_equal(f64(qgm.f8_gemm(x, dev(wc), dev(ws), x_scales=xs, out_dtype=yt)), rounded(ref, yt))
    y = qgm.f8_gemm(x, dev(wc), dev(ws), x_scales=xs, out_dtype=BF16)
    inside(y, ref, sums(K, mag) + left)
    few = qgm.f8_gemm(x[:3], dev(wc), dev(ws), x_scales=xs[:3], out_dtype=BF16)
    inside(few, ref[:3], sums(K, mag[:3]) + left[:3])
    if tile == 0:   # the kernel for few rows converts the codes
        assert np.array_equal(f64(y), rounded(ref, BF16))
    # the gated forms: their projections are off by as much
    for act in ACTS:
        for yt in (BF16, F32):
            h, tol, (g, u, a, da, eg, eu, ea, t) = gate_tolerances(xd, wd, act, K, cut(x, xs, wc, ws, yt))
            inside(qgm.f8_gated(x, dev(wc), dev(ws), x_scales=xs, act=act, out_dtype=yt), h, tol)
            dh = torch.ones(M, N // 2, dtype=yt, device=DEV)
            s = np.where(g != 0, a / np.where(g != 0, g, 1), 0.5)
            es = (8 * t + 16) * U * (np.abs(s) + np.abs(da - s)) + 2.0 ** -126 * (1 + np.abs(g)) + eg
            want = f8ref.gated_grad_ref(f64(dh), xd, wd, act)
            tol = np.concatenate([es * np.abs(u) + (np.abs(da) + es) * eu, ea], axis=1) + 2 * U * np.abs(want)
            inside(qgm.f8_gated_grad(dh, x, dev(wc), dev(ws), x_scales=xs, act=act), want, tol)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("M", [3, 150])
def test_input_gradient_without_rounding_between(kind, M):
    # d in fp32 and its product with the weights turned over as two: of d rounded to bf16, and of what that leaves,
    # rounded too.  What both leave is at most 2^-8 2^-8 of d, so dx is that of the unrounded d within 2^-16.
    rng = np.random.default_rng(M)
    F, K = 80, 272
    x, xs, xv = make_x(rng, kind, M, K)
    wc, ws = random_f8(rng, 2 * F, K, 128, size=0.02 if kind != "f8" else 0.005)
    wv = f8ref.f8_values(wc, ws)
    back = qgm.F8Linear(dev(wc.T), dev(ws.T))
    dh = torch.randn(M, F, device=DEV)
    d = qgm.f8_gated_grad(dh, x, dev(wc), dev(ws), x_scales=xs)
    assert d.dtype == F32
    high = d.to(BF16)
    dx = back(high, out_dtype=F32)
    back((d - high.float()).to(BF16), out=dx, residual=dx)
    ref, mag = f8ref.f8_gemm_ref(f64(d), wv.T)
    inside(dx, ref, (2.0 ** -16 + 2 * sums(2 * F, 1)) * mag)
    # and of the formula's: half a step of bf16 in d alone would be 2^-8 of each term
    want = f8ref.gated_grad_ref(f64(dh), xv, wv, "silu") @ wv
    gap = np.linalg.norm(f64(dx) - want) / np.linalg.norm(want)
    assert gap < 2.0 ** -15, gap


@pytest.mark.parametrize("tile", range(6))
@pytest.mark.parametrize("kind", KINDS + ["rows"])
@pytest.mark.parametrize("end", ["low", "high", "mixed"])
def test_gemm_ends_of_the_scales_range(monkeypatch, tile, kind, end):
    # factors of a block (the product of its two scales; with 16-bit x the one) from 2^-126 on, and sums up to 2^127:
    # what is documented to be as good as elsewhere, but for results below 2^-126, which are multiples of 2^-149
    monkeypatch.setenv("QF8_TILE", str(tile))
    rng = np.random.default_rng(tile)
    M, N, K = 70, 66, 304
    x, xs, xv = make_x(rng, "f8" if kind == "rows" else kind, M, K)
    wc, ws = random_f8(rng, N, K, 1 if kind == "rows" else 128)
    xe, we = {"low": (-80, -46), "high": (70, 30), "mixed": (119, -108)}[end]
    if xs is None:
        ex = 8 if kind == "f16" else {"low": 0, "high": 90, "mixed": 110}[end]
        x = x * 2.0 ** ex
        xv, we = f64(x), {"low": -126, "high": 108 - ex, "mixed": 0 - ex}[end]
    else:
        xs = dev((rng.uniform(1, 2, tuple(xs.shape)) * 2.0 ** xe).astype(np.float32))
        xv = f8ref.f8_values(codes_of(x), xs.cpu().numpy())
    ws = (rng.uniform(1, 2, ws.shape) * 2.0 ** we).astype(np.float32)
    ref, mag = f8ref.f8_gemm_ref(xv, f8ref.f8_values(wc, ws))
    assert mag.max() < 2.0 ** 127
    for yt in (F32, BF16):
        y = qgm.f8_gemm(x, dev(wc), dev(ws), x_scales=xs, out_dtype=yt)
        inside(y, ref, sums(K, mag) + cut(x, xs, wc, ws, yt) + 4 * 2.0 ** -149)


@pytest.mark.parametrize("tile", range(6))
@pytest.mark.parametrize("kind,least", [("f16", 2.0 ** -24), ("bf16", 2.0 ** -133)])
def test_gemm_subnormal_x(monkeypatch, tile, kind, least):
    # multiples of the type's smallest number count in full
    monkeypatch.setenv("QF8_TILE", str(tile))
    rng = np.random.default_rng(tile)
    M, N, K = 70, 66, 176
    n = rng.integers(-64, 65, (M, K))
    x = torch.from_numpy(n * least).to(XTYPE[kind]).to(DEV)
    wc, ws = exact_f8(rng, N, K, 128)
    ws *= 2.0 ** 20
    ref, _ = f8ref.f8_gemm_ref(n * least, f8ref.f8_values(wc, ws))
    assert np.array_equal(f64(qgm.f8_gemm(x, dev(wc), dev(ws), out_dtype=F32)), ref) and ref.any()


@pytest.mark.parametrize("more", [0, 8])
@pytest.mark.parametrize("tile", [None, 0, 1, 2, 3, 4, 5])
def test_widest_pitch_of_x(monkeypatch, tile, more):
    # rows of x 4 MiB apart, the most that the tiles' 32-bit buffers take, and 16 bytes further, which the kernel for
    # few rows takes whatever is forced: more rows than its 16, several tiles, NaN between them
    if tile is not None:
        monkeypatch.setenv("QF8_TILE", str(tile))
    rng = np.random.default_rng(7)
    M, F, K = 270, 48, 80
    xt, _, xv = make_x(rng, "bf16", M, K)
    wide = torch.full((M, (1 << 21) + more), float("nan"), dtype=BF16, device=DEV)
    wide[:, :K] = xt
    x = wide[:, :K]
    wc, ws = random_f8(rng, 2 * F, K, 128, size=0.02)
    w, s = dev(wc), dev(ws)
    ref, mag = f8ref.f8_gemm_ref(xv, f8ref.f8_values(wc, ws))
    y = qgm.f8_gemm(x, w, s, out_dtype=F32)
    inside(y, ref, sums(K, mag))
    h, tol, _ = gate_tolerances(xv, f8ref.f8_values(wc, ws), "silu", K)
    inside(qgm.f8_gated(x, w, s, out_dtype=F32), h, tol)
    dh = torch.ones(M, F, device=DEV)
    d = qgm.f8_gated_grad(dh, x, w, s)
    if more:   # the same kernel as for rows without gaps: the same bits
        monkeypatch.setenv("QF8_TILE", "0")
    assert torch.equal(y, qgm.f8_gemm(xt, w, s, out_dtype=F32)) and torch.equal(d, qgm.f8_gated_grad(dh, xt, w, s))


def test_results_carry_no_graph():
    # the operators are not joined to autograd; a program that trains wraps them in a function of its own
    x, xs, w, ws, dh = small_set("bf16", 5, F=48, K=272)
    block, back = qgm.F8Gated(w, ws), qgm.F8Linear(w.view(torch.uint8).t().contiguous().view(CODE), ws.t().contiguous())

    class Gated(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x):
            ctx.save_for_backward(x)
            return block(x)

        @staticmethod
        def backward(ctx, dh):
            return back(block.grad(dh, *ctx.saved_tensors))

    x.requires_grad_()
    assert not block(x).requires_grad and not back(block.grad(dh, x)).requires_grad
    h = Gated.apply(x)
    got, = torch.autograd.grad(h, x, dh)
    assert torch.equal(h, block(x)) and torch.equal(got, back(block.grad(dh, x)))
    wv = torch.from_numpy(f8ref.f8_values(codes_of(w), ws.cpu().numpy())).to(DEV)
    xd = x.detach().double().requires_grad_()
    p = xd @ wv.t()
    want, = torch.autograd.grad(torch.nn.functional.silu(p[:, :48]) * p[:, 48:], xd, dh.double())
    gap = (got.double() - want).norm() / want.norm()
    assert gap < 2.0 ** -7, gap   # d and dx rounded once each, by half a step (2^-8) at most


@pytest.mark.parametrize("tile", range(6))
def test_large_products_cancel_across_eights(monkeypatch, tile):
    # 256 * 256 in one eight, -256 * 256 in another and 6 * 7 in a third, of any lane and block: no eight has to cut (the
    # 42 lies on its own grid, 2^(2 - 13)), and between them the sum is fp32's
    monkeypatch.setenv("QF8_TILE", str(tile))
    M, N, K = 330, 64, 272
    rng = np.random.default_rng(tile)
    xv, wv = np.zeros((M, K), np.float32), np.tile(np.array([256, 0] + [4] * 6, np.float32), (N, K // 8))
    for m in range(M):
        a, b, c = rng.permutation(K // 8)[:3] * 8
        xv[m, a], xv[m, b], xv[m, c + 2:c + 8] = 256, -256, 1.75
    x, w = (torch.from_numpy(v).to(CODE).to(DEV) for v in (xv, wv))
    one = torch.ones(M, 3, device=DEV)
    ref, mag = f8ref.f8_gemm_ref(xv.astype(np.float64), wv.astype(np.float64))
    assert (ref == 42).all()
    for yt in (F32, BF16):
        inside(qgm.f8_gemm(x, w, one[:1], x_scales=one, out_dtype=yt), ref, sums(K, mag))
