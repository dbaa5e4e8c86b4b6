"""Measured cases of the 8-bit floating-point operators (E4M3 elements with an
fp32 scale for blocks of 128): quantising, the product, the gated feed-forward
block's two projections with activation and product, and that block's backward
pass.

`run` computes an operator in plain torch operations, or through the package's
entry points where `own` is true.  A matrix [R, K] in this form is a pair:
codes [R, K] (torch.float8_e4m3fn) and scales [R / block, ceil(K / 128)]
(fp32), block = 1 (a scale for 128 elements of a row) or 128 (a scale for
128 x 128).  A value is its code times its block's scale."""
import math

import torch

own = False

DEV = "cuda"
TYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"f16": 2, "bf16": 2, "f32": 4, "f8": 1}
CODE = torch.float8_e4m3fn
TOP = 448.0            # the largest code
LOWEST = 2.0 ** -100   # a block's largest magnitude counts as at least this


def _quantise_case(name, M, K, xt, block, transpose):
    return {"name": name, "op": "quantise", "M": M, "K": K, "xt": xt, "block": block, "transpose": transpose}


def _product_case(name, M, N, K, xt, yt, w_block=128, residual=False):
    return {"name": name, "op": "product", "M": M, "N": N, "K": K, "xt": xt, "yt": yt, "w_block": w_block,
            "residual": residual}


def _gated_case(name, M, F, K, xt, yt, act):
    return {"name": name, "op": "gated", "M": M, "F": F, "K": K, "xt": xt, "yt": yt, "act": act}


def _backward_case(name, M, F, K, xt, yt, act):
    return {"name": name, "op": "backward", "M": M, "F": F, "K": K, "xt": xt, "yt": yt, "act": act}


def listed():
    return [
        # one decoded token's hidden state before an 8-bit product: latency
        _quantise_case("quantise token", 1, 2048, "f16", 1, False),
        # gradients of an odd number of tokens, turned over so that the weight's gradient can sum over tokens
        _quantise_case("quantise turned", 1003, 8192, "bf16", 1, True),
        # a master weight quantised before a training step (or once at load time)
        _quantise_case("quantise weights", 8192, 8192, "f32", 128, False),
        # a decoded token through the fused QKV projection, weights only in 8 bits
        _product_case("product decode", 1, 6144, 2048, "f16", "f16"),
        # eight sequences decoded together through the down projection, residual fused
        _product_case("product batch", 8, 2048, 8192, "bf16", "bf16", residual=True),
        # an odd prefill, width and inner size, both sides in 8 bits
        _product_case("product odd", 1003, 2050, 8208, "f8", "bf16"),
        # a long prefill or a training batch, both sides in 8 bits: the largest product
        _product_case("product long", 4096, 8192, 8192, "f8", "bf16"),
        # a weight's gradient summed over 4096 tokens and added to what earlier batches left
        _product_case("product gradient", 2048, 8192, 4096, "f8", "f32", w_block=1, residual=True),
        # a decoded token through gate and up projection
        _gated_case("gated decode", 1, 8192, 2048, "f16", "f16", "silu"),
        # a prefill of 128 tokens, both sides in 8 bits
        _gated_case("gated prefill", 128, 8192, 2048, "f8", "bf16", "silu"),
        # the gradients of an odd batch, adapters trained on 16-bit activations
        _backward_case("backward ragged", 383, 2064, 2048, "bf16", "bf16", "gelu_tanh"),
        # a training batch's gradients, activations kept in 8 bits
        _backward_case("backward long", 4096, 8192, 2048, "f8", "bf16", "silu"),
    ]


def _log_int(rng, low, high):
    return min(high, max(low, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    op = rng.choice(["quantise", "product", "product", "gated", "gated", "backward"])
    if op == "quantise":
        c = _quantise_case("", _log_int(rng, 1, 4096), 16 * _log_int(rng, 1, 512), rng.choice(["f16", "bf16", "f32"]),
                           rng.choice([1, 128]), rng.random() < 0.5)
    elif op == "product":
        xt = rng.choice(["f16", "bf16", "f8", "f8"])
        yt = rng.choice(["f16", "bf16"]) if xt == "f8" else xt
        gradient = xt == "f8" and rng.random() < 0.3
        c = _product_case("", _log_int(rng, 1, 4096), _log_int(rng, 16, 8192), 16 * _log_int(rng, 2, 512), xt,
                          "f32" if gradient else yt, 1 if gradient else 128, rng.random() < 0.3)
    else:
        xt = rng.choice(["f16", "bf16", "f8"])
        yt = rng.choice(["f16", "bf16"]) if xt == "f8" else xt
        make = _gated_case if op == "gated" else _backward_case
        c = make("", _log_int(rng, 1, 4096), 16 * _log_int(rng, 2, 512), 16 * _log_int(rng, 2, 128), xt, yt,
                 rng.choice(["silu", "gelu_tanh"]))
    del c["name"]
    return c


# ----------------------------------------------------------------------------
# inputs
# ----------------------------------------------------------------------------

def _activations(M, K, g):
    """Normal values with a few channels much larger than the others."""
    x = torch.randn(M, K, generator=g, device=DEV)
    wide = torch.rand(K, generator=g, device=DEV) < 0.01
    return x * torch.where(wide, 20.0, 1.0)


def _gradients(M, K, g):
    """Small values, some tokens' much larger than others'."""
    return torch.randn(M, K, generator=g, device=DEV) * torch.exp(torch.randn(M, 1, generator=g, device=DEV) - 5.0)


def _spread(scales, block, R, K):
    """Each element's scale as a matrix [R, K]."""
    s = scales.repeat_interleave(128, dim=1)[:, :K]
    return s if block == 1 else s.repeat_interleave(block, dim=0)[:R]


def _to_f8(v, block):
    """[R, K] -> (codes, scales) in plain operations: a block's scale is its
    largest magnitude A over 448, a code the nearest to 448 v / A, ties to the
    even one.  In 64 bits: quotients midway between two codes are common (16-bit
    A is a multiple of 7 units in every seventh block), and 32 bits would take
    their neighbours for such."""
    R, K = v.shape
    v = v.double()
    rows, cols = -(-R // block), -(-K // 128)
    a = v.new_zeros(rows * block, cols * 128)
    a[:R, :K] = v.abs()
    a = a.reshape(rows, block, cols, 128).amax(dim=(1, 3)).clamp(min=LOWEST)
    q = TOP * v / _spread(a, block, R, K)
    # of the 52 bits of a quotient's mantissa 3 stay; below 2^-6 the codes are the multiples of 2^-9
    bits = q.view(torch.int64)
    bits = (bits + (2 ** 48 - 1) + (bits >> 49 & 1)) & -2 ** 49
    q = torch.where(q.abs() < 2.0 ** -6, torch.round(q * 512) / 512, bits.view(torch.float64))
    return q.float().to(CODE), (a / torch.full_like(a, TOP)).float()


def _weights(R, K, g):
    """A random weight matrix of the usual size (0.02), blocks of 128 x 128."""
    return _to_f8(torch.randn(R, K, generator=g, device=DEV) * 0.02, 128)


def _turned(v):
    """v [T, R] as [R, T] with rows padded by zeros to a multiple of 16."""
    out = v.new_zeros(v.shape[1], -(-v.shape[0] // 16) * 16)
    out[:, :v.shape[0]] = v.t()
    return out


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed * 7919 + 29)
    s = {"case": case, "xs": None, "residual": None}
    K = case["K"]
    if case["op"] == "quantise":
        make = _gradients if case["transpose"] else _activations
        v = make(case["M"], K, g) if case["block"] == 1 else torch.randn(case["M"], K, generator=g, device=DEV) * 0.02
        s["x"] = v.to(TYPES[case["xt"]])
        return s
    M = case["M"]
    if case["op"] == "product" and case["w_block"] == 1:   # the gradient [M, N] of a weight: K tokens
        s["x"], s["xs"] = _to_f8(_gradients(K, M, g).t().contiguous(), 1)
        s["w"], s["ws"] = _to_f8(_activations(K, case["N"], g).t().contiguous(), 1)
    else:
        x = _activations(M, K, g)
        if case["xt"] == "f8":
            s["x"], s["xs"] = _to_f8(x, 1)
        else:
            s["x"] = x.to(TYPES[case["xt"]])
        s["w"], s["ws"] = _weights(case["N"] if case["op"] == "product" else 2 * case["F"], K, g)
    if case["op"] == "product" and case["residual"]:
        s["residual"] = torch.randn(M, case["N"], generator=g, device=DEV).to(TYPES[case["yt"]])
    if case["op"] == "backward":
        s["dh"] = _gradients(M, case["F"], g).to(TYPES[case["yt"]])
        # the same weights turned over, as the product for the input's gradient reads them
        s["wt"] = s["w"].view(torch.uint8).t().contiguous().view(CODE)
        s["wts"] = s["ws"].t().contiguous()
    return s


# ----------------------------------------------------------------------------
# one pass
# ----------------------------------------------------------------------------

def _values(codes, scales, block):
    return codes.float() * _spread(scales, block, *codes.shape)


def _gate(g, act):
    """(act(g), its derivative): g s(t) with the logistic function s, t = g
    (silu) or 2 sqrt(2 / pi) (g + 0.044715 g^3) (gelu, tanh form)."""
    if act == "silu":
        s = torch.sigmoid(g)
        return g * s, s * (1 + g * (1 - s))
    c = 2 * math.sqrt(2 / math.pi)
    s = torch.sigmoid(c * (g + 0.044715 * g ** 3))
    return g * s, s + g * s * (1 - s) * c * (1 + 3 * 0.044715 * g ** 2)


def _plain(s):
    case = s["case"]
    if case["op"] == "quantise":
        codes, scales = _to_f8(_turned(s["x"]) if case["transpose"] else s["x"], case["block"])
        return _values(codes, scales, case["block"]), scales
    yt = TYPES[case["yt"]]
    x = s["x"].float() if s["xs"] is None else _values(s["x"], s["xs"], 1)
    if case["op"] == "product":
        y = x @ _values(s["w"], s["ws"], case["w_block"]).t()
        if s["residual"] is not None:
            y = y + s["residual"].float()
        return y.to(yt)
    w, F = _values(s["w"], s["ws"], 128), case["F"]
    g, u = x @ w[:F].t(), x @ w[F:].t()
    a, da = _gate(g, case["act"])
    if case["op"] == "gated":
        return (a * u).to(yt)
    dh = s["dh"].float()
    d = torch.cat([dh * u * da, dh * a], dim=1)
    return d.to(yt), (d @ w).to(yt)


def _own(s):
    import bit_weight_only_dequant_amd as qg
    case = s["case"]
    if case["op"] == "quantise":
        codes, scales = qg.f8_quantize(s["x"], block=case["block"], transpose=case["transpose"])
        return qg.f8_dequantize(codes, scales, dtype=torch.float32), scales
    yt = TYPES[case["yt"]]
    if case["op"] == "product":
        return qg.f8_gemm(s["x"], s["w"], s["ws"], x_scales=s["xs"], residual=s["residual"], out_dtype=yt)
    if case["op"] == "gated":
        return qg.f8_gated(s["x"], s["w"], s["ws"], x_scales=s["xs"], act=case["act"], out_dtype=yt)
    d = qg.f8_gated_grad(s["dh"], s["x"], s["w"], s["ws"], x_scales=s["xs"], act=case["act"])
    return d, qg.f8_gemm(d, s["wt"], s["wts"])


def run(state):
    return _own(state) if own else _plain(state)


# ----------------------------------------------------------------------------
# what a pass cannot do without, and the definition in 64 bits
# ----------------------------------------------------------------------------

def _stored(R, K, block):
    """Bytes of a matrix's codes and scales."""
    return R * K + 4 * -(-R // block) * -(-K // 128)


def work(case):
    M, K = case["M"], case["K"]
    if case["op"] == "quantise":   # the input, the codes and scales (reading the values back is not the operator's)
        out = _stored(K, -(-M // 16) * 16, case["block"]) if case["transpose"] else _stored(M, K, case["block"])
        return {"bytes": M * K * SIZE[case["xt"]] + out, "flops": 0}
    x = _stored(M, K, 1) if case["xt"] == "f8" else M * K * SIZE[case["xt"]]
    y = SIZE[case["yt"]]
    if case["op"] == "product":
        N = case["N"]
        return {"bytes": x + _stored(N, K, case["w_block"]) + M * N * y * (2 if case["residual"] else 1),
                "flops": 2.0 * M * N * K}
    F = case["F"]
    if case["op"] == "gated":
        return {"bytes": x + _stored(2 * F, K, 128) + M * F * y, "flops": 4.0 * M * F * K}
    # gate and up again, then the two products for the input's gradient; the weights both ways
    return {"bytes": x + 2 * _stored(2 * F, K, 128) + M * F * y + 2 * M * F * y + M * K * y, "flops": 8.0 * M * F * K}


def _wide(codes, scales, block):
    """64-bit values, from the bits of a code: sign, four exponent bits, three
    mantissa bits; the exponent 0 holds the multiples of 2^-9."""
    b = codes.view(torch.uint8).long()
    ex, man = b // 8 % 16, (b % 8).double()
    v = torch.where(ex == 0, man * 2.0 ** -9, (8 + man) * 2.0 ** (ex - 10).double())
    v = torch.where(b >= 128, -v, v)
    R, K = codes.shape
    row = torch.arange(R, device=DEV) // block
    col = torch.arange(K, device=DEV) // 128
    return v * scales.double()[row][:, col]


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "quantise":
        x = s["x"].double()
        if case["transpose"]:
            x = torch.nn.functional.pad(x, (0, 0, 0, -x.shape[0] % 16)).t()
        R, K = x.shape
        b = case["block"]
        p = torch.nn.functional.pad(x.abs(), (0, -K % 128, 0, -R % b))
        top = torch.stack([t.amax(dim=(1, 2)) for t in p.reshape(p.shape[0] // b, b, -1, 128).unbind(2)], dim=1)
        top = top.clamp(min=LOWEST)
        # the 127 codes' magnitudes and the middles between them; at a middle the even code counts
        size = torch.tensor([n * 2.0 ** -9 if n < 8 else (8 + n % 8) * 2.0 ** (n // 8 - 10) for n in range(127)],
                            dtype=torch.float64, device=DEV)
        middle = (size[1:] + size[:-1]) / 2
        spread = top[torch.arange(R, device=DEV) // b][:, torch.arange(K, device=DEV) // 128]
        q = (x.abs() * TOP / spread).contiguous()
        low, high = torch.bucketize(q, middle), torch.bucketize(q, middle, right=True)
        return size[torch.where(low % 2 == 0, low, high)] * torch.sign(x) * spread / TOP, top / TOP
    x = s["x"].double() if s["xs"] is None else _wide(s["x"], s["xs"], 1)
    if case["op"] == "product":
        y = x @ _wide(s["w"], s["ws"], case["w_block"]).t()
        return y if s["residual"] is None else y + s["residual"].double()
    w = _wide(s["w"], s["ws"], 128)
    p = x @ w.t()
    g, u = p[:, :case["F"]], p[:, case["F"]:]
    if case["act"] == "silu":
        gate = 1 / (1 + torch.exp(-g))
        slope = gate + g * torch.exp(-g.abs()) / (1 + torch.exp(-g.abs())) ** 2
    else:
        t = torch.tanh(math.sqrt(2 / math.pi) * (g + 0.044715 * g * g * g))
        gate = (1 + t) / 2
        slope = gate + g * (1 - t * t) / 2 * math.sqrt(2 / math.pi) * (1 + 3 * 0.044715 * g * g)
    if case["op"] == "gated":
        return g * gate * u
    dh = s["dh"].double()
    d = torch.cat([dh * u * slope, dh * g * gate], dim=1)
    return d, d @ w
