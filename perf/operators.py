"""The microscaled operators as they are measured: `quantize`, `add_rms_norm` and `linear_mx`.

Each case is one call on one set of inputs: in its plain form (elementary torch operations in 32 bits)
or, where `own` is true, as a user calls the library. A microscaled tensor is a byte matrix of element
codes (e4m3, one per byte; e2m1, two per byte, the even column in the low half) and one power-of-two
scale byte (e8m0) per 32 values of a row; the scales lie in tiles of 128 rows x 4 blocks (512 bytes):
row r, block k at ((r / 128) * ceil(K / 128) + k / 4) * 512 + (r % 32) * 16 + ((r % 128) / 32) * 4 + k % 4.
8-bit codes and scales are returned as float8 tensors; what `quantize` makes in 4 bits is read back as
the bf16 values it stands for.
"""
import math

import torch

own = False

EPS = 1e-6
WIDTHS = {"mxfp4": 6.0, "mxfp8": 448.0}


def listed():
    return [
        # the activations of one 1280-token slice before a projection, kept in 4 bits
        {"name": "quantize 1280x1536 mxfp4", "op": "quantize", "m": 1280, "k": 1536, "x": "bf16", "fmt": "mxfp4"},
        # the FFN's hidden activations of three 2880-token streams
        {"name": "quantize 8640x8960 mxfp8", "op": "quantize", "m": 8640, "k": 8960, "x": "bf16", "fmt": "mxfp8"},
        # a single token: latency
        {"name": "norm 1x1536", "op": "norm", "m": 1, "d": 1536, "x": "f32", "res": "bf16", "mod": False, "b": 1,
         "out": "mxfp8"},
        # the norm before a projection: fp32 residual stream, bf16 branch, adaLN modulation
        {"name": "norm 1280x1536", "op": "norm", "m": 1280, "d": 1536, "x": "f32", "res": "bf16", "mod": True, "b": 1,
         "out": "mxfp8"},
        # a row width of 49 blocks, which ends inside a scale tile, and an odd number of rows
        {"name": "norm 777x1568 bf16", "op": "norm", "m": 777, "d": 1568, "x": "bf16", "res": "bf16",
         "mod": False, "b": 1, "out": "mxfp8"},
        # eight streams of 2880 tokens
        {"name": "norm 23040x1536", "op": "norm", "m": 23040, "d": 1536, "x": "f32", "res": "bf16", "mod": True,
         "b": 8, "out": "mxfp8"},
        # one row against a wide weight: the conditioning vector's projection to 6 x 1536
        {"name": "linear 1x9216x1536 mxfp4", "op": "linear", "m": 1, "n": 9216, "k": 1536, "fmt": "mxfp4",
         "act": False, "out": "bf16"},
        # odd and ragged: no size a multiple of a tile
        {"name": "linear 437x1001x1568 mxfp8", "op": "linear", "m": 437, "n": 1001, "k": 1568, "fmt": "mxfp8",
         "act": False, "out": "bf16"},
        # FFN1 of a 1280-token slice in 8 bits: GELU, and the 8-bit operand of FFN2 as its output
        {"name": "linear 1280x8960x1536 mxfp8", "op": "linear", "m": 1280, "n": 8960, "k": 1536, "fmt": "mxfp8",
         "act": True, "out": "mxfp8"},
        # FFN2 of a 1280-token slice: few tiles, a long inner dimension
        {"name": "linear 1280x1536x8960 mxfp4", "op": "linear", "m": 1280, "n": 1536, "k": 8960, "fmt": "mxfp4",
         "act": False, "out": "bf16"},
        # the QKV projection of three 2880-token streams in 8 bits
        {"name": "linear 8640x4608x1536 mxfp8", "op": "linear", "m": 8640, "n": 4608, "k": 1536, "fmt": "mxfp8",
         "act": False, "out": "bf16"},
        # FFN1 of eight 2880-token streams
        {"name": "linear 23040x8960x1536 mxfp4", "op": "linear", "m": 23040, "n": 8960, "k": 1536, "fmt": "mxfp4",
         "act": True, "out": "bf16"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["quantize", "norm", "linear", "linear"])
    if op == "quantize":
        k = 32 * _log(rng, 1, 280)
        m = _log(rng, 1, max(1, min(23040, 8640 * 8960 // k)))
        return {"op": op, "m": m, "k": k, "x": rng.choice(["f32", "bf16"]), "fmt": rng.choice(["mxfp4", "mxfp8"])}
    if op == "norm":
        d = 32 * rng.randint(1, 192)
        b = rng.choice([1, 1, 2, 3, 8])
        rows = _log(rng, 1, max(1, min(2880, 23040 * 1536 // (d * b))))
        return {"op": op, "m": b * rows, "d": d, "x": rng.choice(["f32", "f32", "bf16"]), "res": rng.choice(["f32", "bf16"]),
                "mod": rng.random() < 0.5, "b": b, "out": rng.choice(["mxfp8", "mxfp8", "bf16"])}
    out = rng.choice(["bf16", "bf16", "mxfp8"])
    k = 32 * _log(rng, 1, 280)
    n = _log(rng, 1, 9216) if out == "bf16" else 32 * _log(rng, 1, 288)
    m = _log(rng, 1, max(1, min(23040, 23040 * 8960 * 1536 // (n * k), 23040 * 8960 // n)))
    return {"op": op, "m": m, "n": n, "k": k, "fmt": rng.choice(["mxfp4", "mxfp8"]), "act": rng.random() < 0.5, "out": out}


# ----------------------------------------------------------------------------- plain forms
def _e2m1_codes(y):
    """Codes 0..15 of |y| <= 6, to nearest, ties to the even code."""
    a = y.abs()
    c = (a > 0.25).to(torch.uint8)
    c += a >= 0.75
    c += a > 1.25
    c += a >= 1.75
    c += a > 2.5
    c += a >= 3.5
    c += a > 5.0
    return c + 8 * torch.signbit(y).to(torch.uint8)


def _e2m1_values(codes):
    table = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0],
                         device=codes.device)
    return table[codes.long()]


def _tile_scales(byte):
    """[M, K / 32] scale bytes -> the flat tiled layout, zero where the last tiles go past the tensor."""
    m, kb = byte.shape
    rt, kt = -(-m // 128), -(-kb // 4)
    full = torch.zeros((rt * 128, kt * 4), dtype=torch.uint8, device=byte.device)
    full[:m, :kb] = byte
    return full.view(rt, 4, 32, kt, 4).permute(0, 3, 2, 1, 4).reshape(-1)


def _untile_scales(flat, m, kb):
    rt, kt = -(-m // 128), -(-kb // 4)
    return flat.view(rt, kt, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(rt * 128, kt * 4)[:m, :kb]


def _quantize(x, fmt):
    """x float32 [M, K] -> (codes uint8 [M, K], scale bytes uint8 [M, K / 32])."""
    m, k = x.shape
    blocks = x.view(m, k // 32, 32)
    top = WIDTHS[fmt]
    frac, exp = torch.frexp(blocks.abs().amax(-1))
    half, texp = math.frexp(top)
    e = (exp - texp + (frac > half)).clamp(-127, 127)
    e = torch.where(frac == 0, torch.full_like(e, -127), e)
    y = torch.ldexp(blocks, -e[..., None]).view(m, k)
    codes = _e2m1_codes(y) if fmt == "mxfp4" else y.to(torch.float8_e4m3fn).view(torch.uint8)
    return codes, (e + 127).to(torch.uint8)


def _values(codes, byte, fmt):
    m, k = codes.shape
    v = _e2m1_values(codes) if fmt == "mxfp4" else codes.view(torch.float8_e4m3fn).to(torch.float32)
    return torch.ldexp(v.view(m, k // 32, 32), byte.to(torch.int32)[..., None] - 127).view(m, k)


def _pack(codes, fmt):
    return codes if fmt == "mxfp8" else codes[:, 0::2] | (codes[:, 1::2] << 4)


def _unpack(data, fmt):
    return data if fmt == "mxfp8" else torch.stack((data & 15, data >> 4), -1).flatten(1)


def _returned(y, out):
    """What a call whose output type is `out` returns for the float32 result y."""
    if out in ("bf16", "f32"):
        return y.to(torch.bfloat16 if out == "bf16" else torch.float32)
    codes, byte = _quantize(y, out)
    if out == "mxfp4":
        return _values(codes, byte, out).to(torch.bfloat16)
    return [codes.view(torch.float8_e4m3fn), _tile_scales(byte).view(torch.float8_e8m0fnu)]


def _gelu(y):
    return 0.5 * y * (1.0 + torch.tanh(0.7978845608028654 * (y + 0.044715 * y * y * y)))


def _plain(s):
    c = s["case"]
    if c["op"] == "quantize":
        return _returned(s["x"].float(), c["fmt"])
    if c["op"] == "norm":
        total = (s["x"].float() + s["res"].float()).to(s["x"].dtype)
        t = total.float()
        n = t / torch.sqrt((t * t).mean(-1, keepdim=True) + EPS)
        if c["mod"]:
            m, d = t.shape
            y = (n.view(c["b"], m // c["b"], d) * (1.0 + s["a"][:, None]) + s["c"][:, None]).view(m, d)
        else:
            y = n * s["a"][0]
        return [total, _returned(y, c["out"])]
    m, n, k = c["m"], c["n"], c["k"]
    a = _values(_unpack(s["a"], c["fmt"]), _untile_scales(s["sa"], m, k // 32), c["fmt"])
    w = _values(_unpack(s["w"], c["fmt"]), _untile_scales(s["sw"], n, k // 32), c["fmt"])
    y = a @ w.t() + s["bias"]
    return _returned(_gelu(y) if c["act"] else y, c["out"])


# ----------------------------------------------------------------------------- the library's calls
def _mx(q):
    """A microscaled result as it is compared."""
    import audio_driven_talking_b200 as fh
    if not isinstance(q, fh.MXTensor):
        return q
    if q.fmt == "mxfp4":
        return fh.dequantize(q, torch.bfloat16)
    return [q.data.view(torch.float8_e4m3fn), q.scales.view(torch.float8_e8m0fnu)]


def _own(s):
    import audio_driven_talking_b200 as fh
    c = s["case"]
    out = {"bf16": torch.bfloat16, "f32": torch.float32}
    if c["op"] == "quantize":
        return _mx(fh.quantize(s["x"], c["fmt"]))
    if c["op"] == "norm":
        if c["mod"]:
            total, y = fh.add_rms_norm(s["x"], s["res"], s["a"], s["c"], out=out.get(c["out"], c["out"]), eps=EPS)
        else:
            total, y = fh.add_rms_norm(s["x"], s["res"], s["a"][0], out=out.get(c["out"], c["out"]), eps=EPS)
        return [total, _mx(y)]
    a = fh.MXTensor(s["a"], s["sa"], (c["m"], c["k"]), c["fmt"])
    w = fh.MXTensor(s["w"], s["sw"], (c["n"], c["k"]), c["fmt"])
    return _mx(fh.linear_mx(a, w, s["bias"], act="gelu" if c["act"] else None, out=out.get(c["out"], c["out"])))


def run(state):
    return _own(state) if own else _plain(state)


# ----------------------------------------------------------------------------- inputs
def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, device="cuda", generator=g)

    kinds = {"f32": torch.float32, "bf16": torch.bfloat16}
    s = {"case": case}
    if case["op"] == "quantize":
        # activations with a few columns that are an order of magnitude larger
        s["x"] = (normal(case["m"], case["k"]) * torch.exp(0.7 * normal(case["k"]))).to(kinds[case["x"]])
    elif case["op"] == "norm":
        m, d = case["m"], case["d"]
        s["x"] = (4.0 * normal(m, d)).to(kinds[case["x"]])
        s["res"] = normal(m, d).to(kinds[case["res"]])
        s["a"] = 0.3 * normal(case["b"], d) if case["mod"] else 1.0 + 0.1 * normal(1, d)
        s["c"] = 0.3 * normal(case["b"], d)
    else:
        m, n, k, fmt = case["m"], case["n"], case["k"], case["fmt"]
        for name, scales, x in (("a", "sa", normal(m, k) * torch.exp(0.5 * normal(k))), ("w", "sw", normal(n, k) / math.sqrt(k))):
            codes, byte = _quantize(x, fmt)
            s[name], s[scales] = _pack(codes, fmt).contiguous(), _tile_scales(byte).contiguous()
        s["bias"] = 0.5 * normal(n)
    return s


def _bytes(m, k, kind):
    """Bytes of an [m, k] tensor of that kind, as it is returned or read."""
    if kind in ("f32", "bf16"):
        return m * k * (4 if kind == "f32" else 2)
    return m * k * (32 if kind == "mxfp8" else 16) // 32 + m * k // 32


def work(case):
    if case["op"] == "quantize":
        m, k = case["m"], case["k"]
        kept = "bf16" if case["fmt"] == "mxfp4" else "mxfp8"  # 4-bit results come back as bf16 values
        return {"bytes": _bytes(m, k, case["x"]) + _bytes(m, k, kept), "flops": 2 * m * k}
    kept = case["out"]
    if case["op"] == "norm":
        m, d = case["m"], case["d"]
        return {"bytes": 2 * _bytes(m, d, case["x"]) + _bytes(m, d, case["res"]) + _bytes(m, d, kept) +
                4 * d * (2 * case["b"] if case["mod"] else 1), "flops": 6 * m * d}
    m, n, k, fmt = case["m"], case["n"], case["k"], case["fmt"]
    return {"bytes": _bytes(m, k, fmt) + _bytes(n, k, fmt) + 4 * n + _bytes(m, n, kept), "flops": 2 * m * n * k}


# ----------------------------------------------------------------------------- 64 bits
def _round64(a, low, bits):
    """|a| to the nearest multiple of its binade's step (`bits` fraction bits, exponents from `low` on), ties to even."""
    step = torch.exp2(torch.floor(torch.log2(a.clamp(min=2.0 ** low))) - bits)
    return torch.round(a / step) * step


def _micro64(y, fmt):
    """Elements and scales, as values in 64 bits, of the microscaled form of y."""
    m, k = y.shape
    blocks = y.view(m, k // 32, 32)
    top = WIDTHS[fmt]
    big = blocks.abs().max(-1, keepdim=True).values
    e = torch.ceil(torch.log2(big.clamp(min=1e-300) / top)).clamp(-127, 127)
    e = torch.where(big > top * torch.exp2(e), e + 1, e)                   # the logarithm's rounding
    e = torch.where((big <= top * torch.exp2(e - 1)) & (e > -127), e - 1, e)
    r = blocks / torch.exp2(e)
    v = torch.sign(r) * (_round64(r.abs(), 0, 1) if fmt == "mxfp4" else _round64(r.abs(), -6, 3))
    return v, torch.exp2(e)


def _returned64(y, out):
    if out in ("bf16", "f32"):
        return y
    v, scale = _micro64(y, out)
    m, k = y.shape
    if out == "mxfp4":
        return (v * scale).view(m, k)
    rows, tiles = -(-m // 128), -(-k // 128)
    grid = torch.full((rows, 128, tiles, 4), 2.0 ** -127, dtype=torch.float64, device=y.device)
    grid.view(rows * 128, tiles * 4)[:m, :k // 32] = scale[..., 0]
    flat = torch.stack([grid[:, 32 * q:32 * q + 32] for q in range(4)], 3)   # [rows, 32, tiles, q, 4]
    return [v.view(m, k), flat.transpose(1, 2).reshape(-1)]


def _dense64(data, scales, rows, k, fmt):
    """The values of a microscaled operand from its bytes."""
    if fmt == "mxfp8":
        b = data.to(torch.int64)
        e, f, sign = (b >> 3) & 15, (b & 7).double(), 1.0 - 2.0 * (b >> 7).double()
        v = sign * torch.where(e > 0, (1.0 + f / 8) * torch.exp2(e.double() - 7), f * 2.0 ** -9)
    else:
        b = torch.empty((rows, k), dtype=torch.int64, device=data.device)
        b[:, 0::2], b[:, 1::2] = data % 16, data // 16
        e, f, sign = (b >> 1) & 3, (b & 1).double(), 1.0 - 2.0 * (b >> 3).double()
        v = sign * torch.where(e > 0, (1.0 + f / 2) * torch.exp2(e.double() - 1), f / 2)
    r = torch.arange(rows, device=data.device)[:, None]
    q = torch.arange(k, device=data.device)[None, :] // 32
    at = (r // 128 * -(-k // 128) + q // 4) * 512 + r % 32 * 16 + r % 128 // 32 * 4 + q % 4
    return v * torch.exp2(scales[at].double() - 127.0)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "quantize":
        return _returned64(s["x"].double(), case["fmt"])
    if case["op"] == "norm":
        total = s["x"].double() + s["res"].double()
        t = total if case["x"] == "f32" else total.to(torch.bfloat16).double()  # the norm is of the sum as it is kept
        rows = torch.arange(case["m"], device="cuda") // (case["m"] // case["b"])
        n = t * torch.rsqrt(t.square().sum(1, keepdim=True) / case["d"] + EPS)
        y = n * (1.0 + s["a"].double()[rows]) + s["c"].double()[rows] if case["mod"] else n * s["a"].double()
        return [total, _returned64(y, case["out"])]
    a = _dense64(s["a"], s["sa"], case["m"], case["k"], case["fmt"])
    w = _dense64(s["w"], s["sw"], case["n"], case["k"], case["fmt"])
    y = torch.nn.functional.linear(a, w, s["bias"].double())
    if case["act"]:
        y = torch.nn.functional.gelu(y, approximate="tanh")
    return _returned64(y, case["out"])
