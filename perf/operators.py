"""The 4-bit operators: what is measured, in plain form and through the package.

Microscaled 4-bit values: E2M1 codes (0, 0.5, 1, 1.5, 2, 3, 4, 6 and a sign), two to a byte (even column in
the low nibble), with one 8-bit scale per block along a row:
  mxfp4  blocks of 32, scale a power of two (E8M0: 2^(byte - 127), 255 = NaN);
  nvfp4  blocks of 16, scale an E4M3 value times one fp32 factor of the whole tensor.
Scales lie in tiles of 128 rows x 4 blocks (512 bytes): the scale of row r, block b is byte
(r % 32) * 16 + (r % 128) // 32 * 4 + b % 4 of tile [r // 128, b // 4]; a row has as many tiles as cover a
multiple of 256 columns.

Operators (case key "op"):
  quant        rows -> 4 bits, and their values read back
  linear       y = x W^T + b (tanh-GELU) (+ residual), x quantised in the call, W kept in 4 bits
  ffn          y = x + W2 GELU(W1 x + b1) + b2, the inner activation leaving its product in 4 bits
  norm_linear  LayerNorm of x (returned) that leaves in 4 bits too, and the product that reads them
"""
import math

import torch

own = False

BLOCK = {"mxfp4": 32, "nvfp4": 16}
DTYPE = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
BYTES = {"bf16": 2, "fp16": 2, "fp32": 4}
X_SCALE = 0.0093      # nvfp4: the activations' calibrated tensor factor (covers 25)
NORM_EPS = 1e-12


def listed():
    return [
        # one token's activations on their way into a product (latency)
        {"name": "quant_token", "op": "quant", "rows": 1, "K": 768, "fmt": "mxfp4", "dtype": "bf16", "pad": 0},
        # the FFN activations of a packed batch of 256 sequences
        {"name": "quant_batch", "op": "quant", "rows": 18797, "K": 2048, "fmt": "mxfp4", "dtype": "bf16", "pad": 0},
        # a weight matrix on loading, fp32 with an odd width and a row stride
        {"name": "quant_weights", "op": "quant", "rows": 8191, "K": 8000, "fmt": "nvfp4", "dtype": "fp32", "pad": 24},
        # one token through the Q|K|V projection (latency)
        {"name": "linear_token", "op": "linear", "rows": 1, "N": 2304, "K": 768, "fmt": "mxfp4", "dtype": "bf16",
         "out": "bf16", "bias": True, "gelu": False, "residual": False},
        # eight tokens through a wide layer: the weights' bytes
        {"name": "linear_tokens_wide", "op": "linear", "rows": 8, "N": 16384, "K": 8192, "fmt": "nvfp4",
         "dtype": "bf16", "out": "bf16", "bias": False, "gelu": False, "residual": False},
        # Q|K|V of a packed batch of 256 sequences
        {"name": "linear_qkv_batch", "op": "linear", "rows": 18797, "N": 2304, "K": 768, "fmt": "mxfp4",
         "dtype": "bf16", "out": "bf16", "bias": True, "gelu": False, "residual": False},
        # odd rows, odd columns, a short last block, a residual, fp32 in and out
        {"name": "linear_odd", "op": "linear", "rows": 333, "N": 1001, "K": 1000, "fmt": "nvfp4", "dtype": "fp32",
         "out": "fp32", "bias": True, "gelu": False, "residual": True},
        # a large square product
        {"name": "linear_large", "op": "linear", "rows": 8192, "N": 8192, "K": 8192, "fmt": "nvfp4", "dtype": "bf16",
         "out": "bf16", "bias": True, "gelu": False, "residual": False},
        # the feed-forward block on one short sequence, and on a packed batch
        {"name": "ffn_sequence", "op": "ffn", "rows": 64, "N": 2048, "K": 768, "fmt": "nvfp4", "dtype": "bf16"},
        {"name": "ffn_batch", "op": "ffn", "rows": 18797, "N": 2048, "K": 768, "fmt": "mxfp4", "dtype": "bf16"},
        # LayerNorm and the projection behind it: long sequences, and a few rows in fp16
        {"name": "norm_linear_long", "op": "norm_linear", "rows": 12301, "N": 2304, "K": 768, "fmt": "mxfp4",
         "dtype": "bf16"},
        {"name": "norm_linear_rows", "op": "norm_linear", "rows": 5, "N": 512, "K": 1000, "fmt": "nvfp4",
         "dtype": "fp16"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["quant", "linear", "linear", "ffn", "norm_linear"])
    fmt = rng.choice(["mxfp4", "nvfp4"])
    if op == "quant":
        return {"op": op, "rows": _log(rng, 1, 20000), "K": _log(rng, 16, 8192) if rng.random() < 0.5 else
                32 * _log(rng, 1, 128), "fmt": fmt, "dtype": rng.choice(["bf16", "fp16", "fp32"]),
                "pad": rng.choice([0, 0, 8, 3])}
    if op == "linear":
        few = rng.random() < 0.4
        out = rng.choice(["bf16", "bf16", "fp16", "fp32"])
        m, n = _log(rng, 1, 40) if few else _log(rng, 41, 16384), _log(rng, 16, 8192)
        k = 32 * _log(rng, 1, 256) if rng.random() < 0.6 else _log(rng, 32, 4096)
        return {"op": op, "rows": min(m, 8192 ** 3 // (n * k)), "N": n, "K": k, "fmt": fmt,
                "dtype": "fp32" if out == "fp32" else rng.choice(["bf16", "fp16"]), "out": out,
                "bias": rng.random() < 0.7, "gelu": rng.random() < 0.3, "residual": rng.random() < 0.4}
    if op == "ffn":
        return {"op": op, "rows": _log(rng, 1, 16384), "N": 32 * _log(rng, 4, 128), "K": 32 * _log(rng, 2, 64),
                "fmt": fmt, "dtype": rng.choice(["bf16", "fp16"])}
    return {"op": op, "rows": _log(rng, 1, 16384), "N": _log(rng, 16, 4096), "K": _log(rng, 32, 4096), "fmt": fmt,
            "dtype": rng.choice(["bf16", "fp16"])}


# ------------------------------------------------------------------ inputs --

def _e2m1(a):
    """|a| -> nearest E2M1 magnitude, ties to the even code, saturating."""
    return (0.5 * (a > 0.25) + 0.5 * (a >= 0.75) + 0.5 * (a > 1.25) + 0.5 * (a >= 1.75) + 1.0 * (a > 2.5)
            + 1.0 * (a >= 3.5) + 2.0 * (a > 5.0))


def _blocks(x, fmt):
    b = BLOCK[fmt]
    k = x.shape[1]
    kp = -(-k // 32) * 32
    if kp != k:
        x = torch.cat([x, torch.zeros(x.shape[0], kp - k, dtype=x.dtype, device=x.device)], 1)
    return x.view(x.shape[0], kp // b, b)


def _quantize(x, fmt, ts):
    """fp32 rows -> (E2M1 values [rows, blocks, block], scales as the values they stand for [rows, blocks])."""
    xb = _blocks(x, fmt)
    amax = xb.abs().amax(2)
    bad = ~torch.isfinite(amax)
    if fmt == "mxfp4":
        e = torch.clamp(torch.frexp(amax)[1] - 3, min=-127).to(torch.int32)      # floor(log2 amax) - 2
        e = torch.where(amax == 0, torch.full_like(e, -127), e)
        s = torch.ldexp(torch.ones_like(amax, dtype=torch.float64), e)           # 2^-127 is below fp32's normals
        y = (xb.double() / s[..., None]).float()
        s = s.float()
        zero = bad
    else:
        f = torch.tensor(ts, dtype=torch.float32, device=x.device)
        t = torch.clamp(amax / (6.0 * f), max=448.0)
        s = torch.where(bad, torch.zeros_like(t), t).to(torch.float8_e4m3fn).float()
        zero = bad | (s == 0)
        y = xb * (1.0 / torch.where(zero, torch.ones_like(s), s * f))[..., None]
    y = torch.where(zero[..., None], torch.zeros_like(y), y)
    q = torch.where(torch.signbit(y), -_e2m1(y.abs()), _e2m1(y.abs()))
    return q, torch.where(bad, torch.full_like(s, float("nan")), s)


def _values(q, s, k):
    """What the codes and scales stand for, without the tensor factor: [rows, k]."""
    return (q * s[..., None]).reshape(q.shape[0], -1)[:, :k]


def _pack(q, s, fmt):
    """The stored form: codes [rows, columns / 2] and tiled scales."""
    rows = q.shape[0]
    mag = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], device=q.device)
    code = torch.bucketize(q.abs(), mag).to(torch.uint8) + torch.signbit(q).to(torch.uint8) * 8
    code = code.view(rows, -1)
    codes = code[:, 0::2] | (code[:, 1::2] << 4)
    byte = (torch.frexp(s)[1] + 126).to(torch.uint8) if fmt == "mxfp4" else s.to(torch.float8_e4m3fn).view(torch.uint8)
    kp = q.shape[1] * BLOCK[fmt]
    rt, kt = -(-rows // 128), -(-kp // 256) * 256 // BLOCK[fmt] // 4
    full = torch.zeros(rt * 128, kt * 4, dtype=torch.uint8, device=q.device)
    full[:rows, : byte.shape[1]] = byte
    tiles = full.view(rt, 4, 32, kt, 4).permute(0, 3, 2, 1, 4).contiguous()
    return codes.contiguous(), tiles.view(rt, kt, 512)


def _unpack(codes, tiles, rows, k, fmt):
    """The stored form's values in fp32, without the tensor factor: [rows, k]."""
    mag = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6], device=codes.device)
    q = mag[torch.stack([codes & 15, codes >> 4], 2).reshape(rows, -1).long()]
    rt, kt = tiles.shape[:2]
    byte = tiles.view(rt, kt, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(rt * 128, kt * 4)[:rows, : q.shape[1] // BLOCK[fmt]]
    if fmt == "mxfp4":
        s = torch.ldexp(torch.ones(byte.shape, device=codes.device), byte.int() - 127)
        s = torch.where(byte == 255, torch.full_like(s, float("nan")), s)
    else:
        s = byte.contiguous().view(torch.float8_e4m3fn).float()
    return _values(q.view(rows, -1, BLOCK[fmt]), s, k)


def _weight(g, n, k, fmt):
    """A weight matrix N(0, 1/sqrt(k)) as a program keeps it: codes, tiled scales, tensor factor."""
    w = torch.randn(n, k, generator=g, device="cuda") * (1.0 / math.sqrt(k))
    ts = 1.0
    if fmt == "nvfp4":
        ts = 5.0 / math.sqrt(k) / (6.0 * 448.0)    # covers five standard deviations
    q, s = _quantize(w, fmt, ts)
    codes, tiles = _pack(q, s, fmt)
    return {"codes": codes, "scales": tiles, "rows": n, "cols": k, "fmt": fmt, "ts": ts}


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    m, k, op, fmt = case["rows"], case["K"], case["op"], case["fmt"]
    dt = DTYPE[case["dtype"]]
    ld = k + case.get("pad", 0)
    # activations: unit normals, some columns several times as large
    gain = 1.0 + 4.0 * (torch.rand(ld, generator=g, device="cuda") < 0.02)
    x = (torch.randn(m, ld, generator=g, device="cuda") * gain).to(dt)[:, :k]
    st = {"op": op, "fmt": fmt, "x": x, "dtype": dt, "xs": X_SCALE if fmt == "nvfp4" else 1.0}
    if op == "linear":
        n, out = case["N"], DTYPE[case["out"]]
        st.update(w=_weight(g, n, k, fmt), out=out, gelu=case["gelu"],
                  bias=torch.randn(n, generator=g, device="cuda") * 0.1 if case["bias"] else None,
                  residual=torch.randn(m, n, generator=g, device="cuda").to(out) if case["residual"] else None)
    elif op == "ffn":
        n = case["N"]
        st.update(w1=_weight(g, n, k, fmt), b1=torch.randn(n, generator=g, device="cuda") * 0.1,
                  w2=_weight(g, k, n, fmt), b2=torch.randn(k, generator=g, device="cuda") * 0.1)
    elif op == "norm_linear":
        n = case["N"]
        st.update(gamma=1 + 0.1 * torch.randn(k, generator=g, device="cuda"),
                  beta=0.1 * torch.randn(k, generator=g, device="cuda"), w=_weight(g, n, k, fmt),
                  bias=torch.randn(n, generator=g, device="cuda") * 0.1)
    return st


# --------------------------------------------------------------- plain form --

def _gelu(x):
    return 0.5 * x * (1.0 + torch.tanh(0.7978845608028654 * (x + 0.044715 * x * x * x)))


def _product(x, fmt, xs, w):
    """x (fp32 rows) quantised, times the kept weight: fp32."""
    q, s = _quantize(x, fmt, xs)
    return _values(q, s, x.shape[1]) @ _unpack(w["codes"], w["scales"], w["rows"], w["cols"], fmt).t() * (xs * w["ts"])


def _plain(st):
    x, fmt, xs = st["x"].float(), st["fmt"], st["xs"]
    if st["op"] == "quant":
        q, s = _quantize(x, fmt, xs)
        return (_values(q, s, x.shape[1]) * torch.tensor(xs, dtype=torch.float32, device=x.device)).to(st["dtype"])
    if st["op"] == "linear":
        y = _product(x, fmt, xs, st["w"])
        if st["bias"] is not None:
            y = y + st["bias"]
        if st["gelu"]:
            y = _gelu(y)
        if st["residual"] is not None:
            y = y + st["residual"].float()
        return y.to(st["out"])
    if st["op"] == "ffn":
        h = _gelu(_product(x, fmt, xs, st["w1"]) + st["b1"])
        return (_product(h, fmt, xs, st["w2"]) + st["b2"] + x).to(st["dtype"])
    mean = x.mean(1, keepdim=True)
    d = x - mean
    y = d * torch.rsqrt((d * d).mean(1, keepdim=True) + NORM_EPS) * st["gamma"] + st["beta"]
    return y.to(st["dtype"]), (_product(y, fmt, xs, st["w"]) + st["bias"]).to(st["dtype"])


# -------------------------------------------------- the framework's operators --

def _kept(tea, w):
    return tea.Mx4Tensor(w["codes"], w["scales"], w["rows"], w["cols"], w["fmt"], w["ts"])


def _framework(st):
    import transformer_encoder_albert_b200 as tea
    x, fmt, xs = st["x"], st["fmt"], st["xs"]
    if st["op"] == "quant":
        return tea.mx4_dequantize(tea.mx4_quantize(x, fmt, xs), dtype=st["dtype"])
    if st["op"] == "linear":
        return tea.mx4_linear(x, _kept(tea, st["w"]), bias=st["bias"], residual=st["residual"], gelu=st["gelu"],
                              dtype=st["out"], x_scale=xs)
    if st["op"] == "ffn":
        h = tea.mx4_linear_quant(x, _kept(tea, st["w1"]), bias=st["b1"], gelu=True, x_scale=xs, out_scale=xs)
        return tea.mx4_linear(h, _kept(tea, st["w2"]), bias=st["b2"], residual=x, dtype=st["dtype"])
    y, y4 = tea.mx4_layer_norm(x, st["gamma"], st["beta"], NORM_EPS, fmt, xs)
    return y, tea.mx4_linear(y4, _kept(tea, st["w"]), bias=st["bias"], dtype=st["dtype"])


def run(state):
    if own:
        return _framework(state)
    return _plain(state)


def _packed_bytes(rows, k, fmt):
    return rows * k * (0.5 + 1.0 / BLOCK[fmt])


def work(case):
    m, k, fmt, eb = case["rows"], case["K"], case["fmt"], BYTES[case["dtype"]]
    if case["op"] == "quant":
        return {"bytes": 2 * m * k * eb + _packed_bytes(m, k, fmt), "flops": 4.0 * m * k}
    n = case["N"]
    w = _packed_bytes(n, k, fmt)
    if case["op"] == "linear":
        ob = BYTES[case["out"]]
        return {"bytes": m * k * eb + w + m * n * ob * (2 if case["residual"] else 1) + (4 * n if case["bias"] else 0),
                "flops": 2.0 * m * n * k}
    if case["op"] == "ffn":
        return {"bytes": 2 * m * k * eb + 2 * w + 4 * (n + k), "flops": 4.0 * m * n * k}
    return {"bytes": 2 * m * k * eb + m * n * eb + w + 4 * (n + 2 * k), "flops": 2.0 * m * n * k}


# ------------------------------------------------------- the definition, 64 bits --

def _grid_nearest(v, step):
    return torch.round(v / step) * step        # halves to the even multiple


def _floor_log2(a):
    """floor(log2 a) of a > 0: the logarithm may fall short of a whole number by its last bit."""
    e = torch.floor(torch.log2(a))
    e = torch.where(torch.ldexp(torch.ones_like(a), e + 1) <= a, e + 1, e)
    return torch.where(torch.ldexp(torch.ones_like(a), e) > a, e - 1, e)


def _e2m1_64(v):
    a = v.abs().clamp(max=6.0)
    step = torch.where(a < 2.0, 0.5, torch.where(a < 4.0, 1.0, 2.0))
    return torch.copysign(_grid_nearest(a, step), v)


def _rounded_64(x, fmt, ts):
    """x (64 bits) -> the 64-bit values of its 4-bit form, tensor factor included."""
    m, k = x.shape
    b = BLOCK[fmt]
    pad = -k % b
    xb = torch.nn.functional.pad(x, (0, pad)).reshape(m, -1, b)
    amax = xb.abs().max(2).values
    if fmt == "mxfp4":
        scale = torch.ldexp(torch.ones_like(amax), torch.clamp(_floor_log2(amax.clamp(min=2.0 ** -140)) - 2, min=-127.0))
        v = _e2m1_64(xb / scale[..., None]) * scale[..., None]
    else:
        f = float(torch.tensor(ts, dtype=torch.float32))
        f6 = float(torch.tensor(6.0, dtype=torch.float32) * torch.tensor(ts, dtype=torch.float32))
        t = (amax / f6).float().double().clamp(max=448.0)
        step = torch.ldexp(torch.ones_like(t), _floor_log2(t.clamp(min=2.0 ** -6)) - 3)
        sb = _grid_nearest(t, step)
        d = (sb * f).float().double()
        r = (1.0 / torch.where(d == 0, 1.0, d)).float().double()
        v = _e2m1_64((xb * r[..., None]).float().double()) * sb[..., None] * f
        v = torch.where(sb[..., None] == 0, 0.0, v)
    return v.reshape(m, -1)[:, :k]


def _read_64(w):
    """The kept weight's values in 64 bits, tensor factor included, by gathering each column's scale byte."""
    c, n, k, fmt = w["codes"], w["rows"], w["cols"], w["fmt"]
    dev = c.device
    col, row = torch.arange(k, device=dev), torch.arange(n, device=dev)[:, None]
    nib = (c[:, col // 2].int() >> (4 * (col % 2)).int()) & 15
    e, mnt = (nib >> 1) & 3, (nib & 1).double()
    mag = torch.where(e == 0, 0.5 * mnt, (1 + 0.5 * mnt) * 2.0 ** (e.double() - 1))
    blk = col // BLOCK[fmt]
    at = (row % 32) * 16 + (row % 128) // 32 * 4 + blk % 4
    byte = w["scales"].reshape(-1)[(row // 128 * w["scales"].shape[1] + blk // 4) * 512 + at].int()
    if fmt == "mxfp4":
        s = 2.0 ** (byte.double() - 127)
    else:
        ee, mm = (byte >> 3) & 15, (byte & 7).double()
        s = torch.where(ee == 0, mm / 8 * 2.0 ** -6, (1 + mm / 8) * 2.0 ** (ee.double() - 7))
    return torch.where(nib >= 8, -mag, mag) * s * float(torch.tensor(w["ts"], dtype=torch.float32))


def _gelu_64(x):
    return x / (1.0 + torch.exp(-2.0 * math.sqrt(2.0 / math.pi) * (x + 0.044715 * x ** 3)))


def exact(case, seed):
    st = prepare(case, seed)
    x, fmt, xs = st["x"].double(), st["fmt"], st["xs"]
    if st["op"] == "quant":
        return _rounded_64(x, fmt, xs)
    if st["op"] == "linear":
        y = _rounded_64(x, fmt, xs) @ _read_64(st["w"]).T
        y = y if st["bias"] is None else y + st["bias"].double()
        y = _gelu_64(y) if st["gelu"] else y
        return y if st["residual"] is None else y + st["residual"].double()
    if st["op"] == "ffn":
        h = _gelu_64(_rounded_64(x, fmt, xs) @ _read_64(st["w1"]).T + st["b1"].double())
        return _rounded_64(h, fmt, xs) @ _read_64(st["w2"]).T + st["b2"].double() + x
    mu = x.mean(1, keepdim=True)
    var = ((x - mu) ** 2).mean(1, keepdim=True)
    y = (x - mu) / torch.sqrt(var + NORM_EPS) * st["gamma"].double() + st["beta"].double()
    return y, _rounded_64(y, fmt, xs) @ _read_64(st["w"]).T + st["bias"].double()
