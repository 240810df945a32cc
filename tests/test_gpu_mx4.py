"""Microscaled 4-bit operators on the GPU against the 64-bit oracle (oracle/mx4_quant.py).

Tolerances, derived:
  * quantising fp32-representable rows: codes and scale bytes equal;
  * a read-back value: one rounding to the result's type (nvfp4 has one more, the
    product with the tensor factor in fp32: 2^-24 relative);
  * a product of K terms with fp32 accumulation: every one of at most K + 3 additions
    is off by at most 2^-23 of a partial sum (truncation counted), and no partial sum
    exceeds S = sum |a||w| + |bias|, so |err| <= (K + 3) 2^-23 S before the epilogue;
  * GELU: slope at most 1.13, and an own error of 2^-17 |z| (the exponential's argument,
    at most 30 where the result is not yet z or 0, carries 2^-23 of itself);
  * the result's rounding: half a step, eps / 2 relative (and half the smallest
    subnormal of fp16);
  * a 4-bit result z' of a value known to within t: its scale byte lies between the
    bytes of the block's largest magnitude less and plus t, and |z' - z| is at most the
    largest half step (1 scale; 2 above 6 for mxfp4's clipping to 8) + t.
"""
import math

import numpy as np
import pytest
import torch

import transformer_encoder_albert_b200 as tea
from oracle import mx4_quant as mq

pytestmark = pytest.mark.gpu
FMTS = ["mxfp4", "nvfp4"]
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
TS = {"mxfp4": 1.0, "nvfp4": 0.0093}
WTS = {"mxfp4": 1.0, "nvfp4": 7e-5}


def _rows(rng, m, k, dtype, gain=1.0):
    """fp32 values representable in dtype, and the tensor."""
    t = torch.tensor(rng.normal(0, gain, (m, k)).astype(np.float32)).to(DTYPES[dtype])
    return t.float().numpy(), t.cuda()


def _eps(dtype):
    return torch.finfo(DTYPES[dtype]).eps / 2


def _np(t):
    return t.double().cpu().numpy()


def _stored(t):
    return mq.unpack(t.codes.cpu().numpy(), t.scales.cpu().numpy(), t.rows, t.cols, t.fmt)


def _weight(rng, n, k, fmt, std=0.05):
    w = rng.normal(0, std, (n, k)).astype(np.float32)
    t = tea.mx4_quantize(torch.tensor(w).cuda(), fmt, WTS[fmt])
    return mq.rounded(w, fmt, WTS[fmt]), t


# ------------------------------------------------------- quantise, read back --

@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("rows,cols,pad", [(1, 1, 0), (1, 768, 0), (3, 16, 0), (5, 33, 0), (129, 256, 0), (130, 1000, 8),
                                            (257, 257, 3), (64, 2048, 0), (1300, 1001, 0), (70, 511, 2), (33, 770, 1),
                                            (3, 2, 1)])
def test_codes_and_scales_are_bit_exact(rows, cols, pad, dtype, fmt):
    rng = np.random.default_rng(rows * 7 + cols)
    x, t = _rows(rng, rows, cols + pad, dtype, 2.0)
    x, t = x[:, :cols].copy(), t[:, :cols]
    q = tea.mx4_quantize(t, fmt, TS[fmt])
    codes, byte = _stored(q)
    want_c, want_b = mq.quantize(x, fmt, TS[fmt])
    np.testing.assert_array_equal(byte, want_b)
    np.testing.assert_array_equal(codes, want_c)
    packed, tiles = mq.pack(want_c, want_b, fmt)   # the padding bytes as well
    np.testing.assert_array_equal(q.scales.cpu().numpy(), tiles)
    for out in DTYPES:
        ref = mq.values(want_c, want_b, fmt, TS[fmt], cols)
        got = _np(tea.mx4_dequantize(q, dtype=DTYPES[out]))
        tol = (_eps(out) + (2.0 ** -24 if fmt == "nvfp4" else 0)) * np.abs(ref)
        if out == "fp16":
            tol = np.maximum(tol, 2.0 ** -25)
        assert np.all(np.abs(got - ref) <= tol), out


@pytest.mark.parametrize("fmt", FMTS)
def test_every_midpoint_and_border_of_the_formats(fmt):
    """Blocks with amax 6: every E2M1 value, every midpoint and the fp32 neighbours of each,
    under block scales over the whole range."""
    mids = (mq.GRID[:-1] + mq.GRID[1:]) / 2
    v = np.concatenate([mq.GRID, mids, np.nextafter(mids.astype(np.float32), np.float32(9)),
                        np.nextafter(mids.astype(np.float32), np.float32(0))]).astype(np.float32)
    v = np.concatenate([v, -v])
    b = mq.BLOCK[fmt]
    v = np.concatenate([np.append(v[i:i + b - 1], np.float32(6)) for i in range(0, v.size - b + 1, b - 1)])
    exps = np.arange(-120, 120, 7) if fmt == "mxfp4" else np.arange(-6, 9)
    x = np.stack([(v * np.float32(2.0) ** np.float32(e)).astype(np.float32) for e in exps])
    q = tea.mx4_quantize(torch.tensor(x).cuda(), fmt, 1.0)
    codes, byte = _stored(q)
    want_c, want_b = mq.quantize(x, fmt, 1.0)
    np.testing.assert_array_equal(byte, want_b)
    np.testing.assert_array_equal(codes, want_c)


@pytest.mark.parametrize("fmt", FMTS)
def test_zero_tiny_huge_and_non_finite_blocks(fmt):
    b = mq.BLOCK[fmt]
    x = np.random.default_rng(0).normal(0, 1, (6, 4 * b)).astype(np.float32)
    x[0] = 0
    x[1, :b] = 1e-42          # fp32 subnormals
    x[1, b:2 * b] = 3e38
    x[2, 3] = np.nan
    x[2, b + 5] = np.inf
    x[2, 2 * b + 1] = -np.inf
    x[3] *= np.float32(1e-30)
    x[4] = -0.0
    x[5, 0] = 1e30
    q = tea.mx4_quantize(torch.tensor(x).cuda(), fmt, TS[fmt])
    codes, byte = _stored(q)
    want_c, want_b = mq.quantize(x, fmt, TS[fmt])
    np.testing.assert_array_equal(byte, want_b)
    np.testing.assert_array_equal(codes, want_c)
    got = _np(tea.mx4_dequantize(q, dtype=torch.float32))
    assert np.isnan(got[2, :3 * b]).all() and np.isfinite(got[2, 3 * b:]).all()
    assert np.all(got[0] == 0) and np.all(got[4] == 0)


def test_quantise_into_given_buffers_and_no_rows():
    x = torch.randn(40, 96, device="cuda")
    out = tea.mx4_empty(40, 96, "mxfp4")
    q = tea.mx4_quantize(x, "mxfp4", out=out)
    assert q.codes.data_ptr() == out.codes.data_ptr()
    with pytest.raises(ValueError):
        tea.mx4_quantize(x, "nvfp4", 1.0, out=out)
    e = tea.mx4_quantize(x[:0], "mxfp4")
    assert e.shape == (0, 96) and tea.mx4_dequantize(e).shape == (0, 96)
    y, ye = tea.mx4_layer_norm(x[:0], torch.ones(96, device="cuda"), torch.zeros(96, device="cuda"))
    assert y.shape == (0, 96) and ye.rows == 0
    w = tea.mx4_quantize(x, "mxfp4")
    assert tea.mx4_linear(x[:0], w).shape == (0, 40) and tea.mx4_linear_quant(x[:0], w).shape == (0, 40)


def test_read_back_leaves_the_bytes_between_rows_alone():
    x = torch.randn(9, 70, device="cuda")
    q = tea.mx4_quantize(x, "nvfp4", 0.01)
    buf = torch.full((9, 90), 7.0, device="cuda", dtype=torch.float16)
    tea.mx4_dequantize(q, out=buf[:, :70])
    assert torch.all(buf[:, 70:] == 7)
    assert torch.equal(buf[:, :70], tea.mx4_dequantize(q, dtype=torch.float16))


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("cols,width,offset", [(1, 3, 1), (255, 257, 1), (256, 259, 2), (257, 261, 3), (513, 514, 0),
                                               (512, 515, 1), (770, 784, 8)])
def test_rows_at_any_offset_of_a_wider_buffer(cols, width, offset, dtype):
    """Odd offsets and strides: the values of the same rows laid out whole, nothing beside them."""
    rng = np.random.default_rng(cols + offset)
    _, t = _rows(rng, 67, width, dtype)
    part = t[:, offset:offset + cols]
    q, whole = tea.mx4_quantize(part, "nvfp4", 0.01), tea.mx4_quantize(part.contiguous(), "nvfp4", 0.01)
    assert torch.equal(q.codes, whole.codes) and torch.equal(q.scales, whole.scales)
    buf = torch.full((67, width), 7.0, device="cuda", dtype=DTYPES[dtype])
    tea.mx4_dequantize(q, out=buf[:, offset:offset + cols])
    wide = torch.zeros((67, -(-cols // 16) * 16), device="cuda", dtype=DTYPES[dtype])
    tea.mx4_dequantize(q, out=wide[:, :cols])   # (aligned rows)
    assert torch.equal(buf[:, offset:offset + cols], wide[:, :cols])
    buf[:, offset:offset + cols] = 7
    assert torch.all(buf == 7) and torch.all(wide[:, cols:] == 0)
    g, b = torch.randn(cols, device="cuda"), torch.randn(cols, device="cuda")
    y, z = tea.mx4_layer_norm(part, g, b, 1e-5, "mxfp4")
    wide[:, :cols] = part
    y2, z2 = tea.mx4_layer_norm(wide[:, :cols], g, b, 1e-5, "mxfp4")
    # each within the bound of the next test of the formula's value, then rounded to x's type
    xd = part.double()
    rstd = (xd.var(1, unbiased=False, keepdim=True) + 1e-5).rsqrt()
    tol = (cols / 256 + 16) * 2.0 ** -23 * (xd.abs().amax(1, keepdim=True) * rstd * g.abs() + 4 * y2.double().abs() + b.abs())
    step = _eps(dtype) * (y.double().abs() + y2.double().abs()) + (2.0 ** -24 if dtype == "fp16" else 0)
    assert torch.all((y.double() - y2.double()).abs() <= 2 * tol + step)


# ----------------------------------------------------------------- LayerNorm --

@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("rows,cols,pad", [(1, 768, 0), (1, 1, 0), (7, 40, 5), (133, 768, 0), (20, 1001, 0), (6, 2304, 8),
                                            (3, 9000, 0), (700, 768, 0), (700, 520, 8), (2500, 2048, 0), (40, 1000, 0),
                                            (40, 1000, 8), (700, 2600, 0), (320, 8000, 0), (9, 4001, 0), (600, 1477, 0),
                                            (5, 5001, 1)])
def test_layer_norm_rows_and_their_4_bit_form(rows, cols, pad, dtype, fmt):
    rng = np.random.default_rng(rows + cols)
    x, t = _rows(rng, rows, cols + pad, dtype, 3.0)
    x, t = (x[:, :cols] + 0.0).astype(np.float64), t[:, :cols]
    g = (1 + rng.normal(0, 0.1, cols)).astype(np.float32)
    b = rng.normal(0, 0.1, cols).astype(np.float32)
    eps = 1e-5
    y, q = tea.mx4_layer_norm(t, torch.tensor(g).cuda(), torch.tensor(b).cuda(), eps, fmt, TS[fmt])
    mu = x.mean(1, keepdims=True)
    d = x - mu
    ref = d / np.sqrt((d * d).mean(1, keepdims=True) + eps) * g + b
    # mean off by cols 2^-24 max|x| at the worst, but pairwise in the lanes: 64 additions deep;
    # the variance likewise (2 * 64 additions); the rest a few roundings
    rstd = 1.0 / np.sqrt((d * d).mean(1, keepdims=True) + eps)
    deep = cols / 256 + 16
    tol32 = deep * 2.0 ** -23 * (np.abs(x).max(1, keepdims=True) * rstd * np.abs(g) + 4 * np.abs(ref) + np.abs(b))
    tol = tol32 + _eps(dtype) * np.abs(ref) + (2.0 ** -25 if dtype == "fp16" else 0)
    assert np.all(np.abs(_np(y) - ref) <= tol)
    _check_4bit(q, ref, tol32, fmt, TS[fmt])
    y2, q2 = tea.mx4_layer_norm(t, torch.tensor(g).cuda(), torch.tensor(b).cuda(), eps, fmt, TS[fmt], return_rows=False)
    assert y2 is None and torch.equal(q.codes, q2.codes)


def _check_4bit(q, ref, tol, fmt, ts):
    """q is the 4-bit form of a matrix within tol of ref."""
    codes, byte = _stored(q)
    rb, tb = mq.blocks(np.abs(ref), fmt), mq.blocks(np.broadcast_to(tol, ref.shape), fmt)
    f32 = np.float32
    lo = mq.scale_bytes(np.maximum((rb - tb).max(2), 0).astype(f32) * f32(1 - 2.0 ** -22), fmt, ts)
    hi = mq.scale_bytes((rb + tb).max(2).astype(f32) * f32(1 + 2.0 ** -22), fmt, ts)
    assert np.all((byte >= lo) & (byte <= hi))
    got = mq.values(codes, byte, fmt, ts, ref.shape[1])
    s = mq.scale_values(byte, fmt) * (ts if fmt == "nvfp4" else 1.0)
    s = np.repeat(s, mq.BLOCK[fmt], 1)[:, :ref.shape[1]]
    # the half step at a value: 1/4 below 2, 1/2 below 4, 1 up to 6, beyond it what is clipped
    step = np.where(np.abs(ref) < 1.75 * s, 0.25, np.where(np.abs(ref) < 3.5 * s, 0.5, 1.0)) * s
    clip = np.maximum(np.abs(ref) - 6 * s, 0)
    assert np.all(np.abs(got - ref) <= np.maximum(step, clip) + 2 * tol + s * 2.0 ** -20)
    assert np.all(codes[:, ref.shape[1]:] == 0)


# ------------------------------------------------------------------- product --

LINEAR = [  # rows, n, k
    (1, 1, 1), (1, 16, 32), (1, 2304, 768), (2, 48, 100), (3, 130, 4200), (1, 300, 9000), (32, 200, 2500), (31, 1030, 1300), (8, 130, 256), (16, 512, 2048), (17, 257, 320), (33, 96, 768),
    (64, 129, 1000), (127, 768, 768), (128, 128, 256), (129, 300, 288), (200, 1001, 1000), (257, 2304, 64),
    (300, 256, 2080), (513, 520, 520), (1025, 192, 256),
    # enough 256x256 tiles for CTA pairs, with ragged last tiles, one and several tiles per pair
    (2501, 2001, 544), (5000, 2304, 96), (9000, 1040, 1100),
]


def _linear_ref(a, w, bias, gelu, res, k):
    z = a @ w.T + (0 if bias is None else bias)
    big = np.abs(a) @ np.abs(w).T + (0 if bias is None else np.abs(bias))
    tol = (k + 3) * 2.0 ** -23 * big
    if gelu:
        tol = 1.13 * tol + 2.0 ** -17 * np.abs(z)
        z = mq.gelu(z)
    if res is not None:
        z = z + res
        tol = tol + 2.0 ** -23 * np.abs(z)
    return z, tol


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("rows,n,k", LINEAR)
def test_linear_against_the_oracle(rows, n, k, fmt):
    rng = np.random.default_rng(rows + 3 * n + 5 * k)
    for i, (dtype, out, with_bias, gelu, with_res) in enumerate(
            [("bf16", "bf16", True, False, False), ("fp16", "fp32", False, True, True), ("fp32", "fp16", True, True, False),
             ("bf16", "fp32", False, False, False), ("fp32", "bf16", True, False, True)]):
        x, t = _rows(rng, rows, k, dtype)
        w, wt = _weight(rng, n, k, fmt)
        bias = rng.normal(0, 0.5, n).astype(np.float32) if with_bias else None
        res, rt = _rows(rng, rows, n, out) if with_res else (None, None)
        a = mq.rounded(x, fmt, TS[fmt])
        ref, tol = _linear_ref(a, w, bias, gelu, res, k)
        kw = dict(bias=None if bias is None else torch.tensor(bias).cuda(), residual=rt, gelu=gelu, dtype=DTYPES[out])
        got = tea.mx4_linear(t, wt, x_scale=TS[fmt], **kw)
        tol = tol + _eps(out) * np.abs(ref) + (2.0 ** -25 if out == "fp16" else 0)
        err = np.abs(_np(got) - ref)
        assert np.all(err <= tol), f"{dtype}->{out}: {int((err > tol).sum())} off, worst {err.max():.3e}"
        # from a 4-bit matrix: the same products
        got4 = tea.mx4_linear(tea.mx4_quantize(t, fmt, TS[fmt]), wt, **kw)
        assert np.all(np.abs(_np(got4) - ref) <= tol)
    assert tea.mx4_status() == 0


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("rows,n,k", [(1, 32, 32), (1, 2048, 768), (5, 100, 96), (16, 33, 256), (40, 256, 300), (130, 320, 768),
                                      (300, 2048, 256), (129, 1000, 64), (2600, 2020, 288), (10000, 1030, 96)])
def test_linear_with_a_4_bit_result(rows, n, k, fmt):
    rng = np.random.default_rng(rows + n + k)
    x, t = _rows(rng, rows, k, "bf16")
    w, wt = _weight(rng, n, k, fmt)
    bias = rng.normal(0, 0.5, n).astype(np.float32)
    for gelu in (True, False):
        ref, tol = _linear_ref(mq.rounded(x, fmt, TS[fmt]), w, bias, gelu, None, k)
        q = tea.mx4_linear_quant(t, wt, torch.tensor(bias).cuda(), gelu=gelu, x_scale=TS[fmt], out_scale=TS[fmt])
        _check_4bit(q, ref, tol, fmt, TS[fmt])
        # the whole scale tiles of the rows that exist are written: a product may read them
        nb = q.codes.shape[1] * 2 // mq.BLOCK[fmt]
        tiles = q.scales.cpu().numpy()
        r, b = np.arange(rows)[:, None], np.arange(nb, tiles.shape[1] * 4)[None, :]
        assert np.all(tiles[r // 128, b // 4, (r % 32) * 16 + (r % 128) // 32 * 4 + b % 4] == 0)
    assert tea.mx4_status() == 0


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("rows", [4, 300])
def test_linear_reads_and_writes_strided_rows(rows, fmt):
    rng = np.random.default_rng(3)
    n, k = 200, 100
    x, _ = _rows(rng, rows, k, "bf16")
    w, wt = _weight(rng, n, k, fmt)
    for off, ldx, ldo in ((0, 104, 208), (1, 101, 203), (3, 333, 201)):
        xb = torch.full((rows * ldx + 8,), float("nan"), device="cuda", dtype=torch.bfloat16)
        xv = xb[off:off + rows * ldx].view(rows, ldx)[:, :k]
        xv.copy_(torch.tensor(x))
        ob = torch.full((rows * ldo + 8,), 7.0, device="cuda", dtype=torch.bfloat16)
        ov = ob[off:off + rows * ldo].view(rows, ldo)[:, :n]
        rb = torch.zeros(rows * ldo + 8, device="cuda", dtype=torch.bfloat16)
        rv = rb[off:off + rows * ldo].view(rows, ldo)[:, :n]
        rv.copy_(torch.randn(rows, n, device="cuda"))
        tea.mx4_linear(xv, wt, residual=rv, out=ov, x_scale=TS[fmt])
        ref, tol = _linear_ref(mq.rounded(x, fmt, TS[fmt]), w, None, False, _np(rv), k)
        assert np.all(np.abs(_np(ov) - ref) <= tol + 2.0 ** -8 * np.abs(ref))
        rest = ob.clone()
        rest[off:off + rows * ldo].view(rows, ldo)[:, :n] = 7.0
        assert torch.all(rest == 7.0)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("rows", [3, 150])
def test_non_finite_blocks_stay_in_their_row(rows, fmt):
    rng = np.random.default_rng(9)
    x, t = _rows(rng, rows, 512, "fp32")
    w, wt = _weight(rng, 256, 512, fmt)
    t[1, 40] = float("inf")
    t[2, 500] = float("nan")
    y = _np(tea.mx4_linear(t, wt, dtype=torch.float32, x_scale=TS[fmt]))
    assert np.isnan(y[1:3]).all() and np.isfinite(y[0]).all() and np.isfinite(y[3:]).all()
    q = tea.mx4_linear_quant(t, wt, gelu=True, x_scale=TS[fmt], out_scale=TS[fmt])
    v = _np(tea.mx4_dequantize(q, dtype=torch.float32))
    assert np.isnan(v[1:3]).all() and np.isfinite(v[0]).all() and np.isfinite(v[3:]).all()


@pytest.mark.parametrize("fmt", FMTS)
def test_scales_over_their_range(fmt):
    """Row and column magnitudes 2^-30 .. 2^30 (mxfp4) or E4M3's range (nvfp4): the block
    scales multiply exactly."""
    rng = np.random.default_rng(4)
    m, n, k = 140, 130, 512
    e = 30 if fmt == "mxfp4" else 5
    x = (rng.normal(0, 1, (m, k)) * 2.0 ** rng.integers(-e, e + 1, (m, 1))).astype(np.float32)
    wv = (rng.normal(0, 1, (n, k)) * 2.0 ** rng.integers(-e, e + 1, (n, 1))).astype(np.float32)
    ts = 0.25
    wt = tea.mx4_quantize(torch.tensor(wv).cuda(), fmt, ts)
    a, w = mq.rounded(x, fmt, ts), mq.rounded(wv, fmt, ts)
    ref, tol = _linear_ref(a, w, None, False, None, k)
    for rows in (m, 5):
        got = _np(tea.mx4_linear(torch.tensor(x[:rows]).cuda(), wt, dtype=torch.float32, x_scale=ts))
        assert np.all(np.abs(got - ref[:rows]) <= (tol + 2.0 ** -24 * np.abs(ref))[:rows])


@pytest.mark.parametrize("rows", [9, 140])
def test_far_apart_power_of_two_scales_cancel(rows):
    """mxfp4 rows scaled by 2^e against weights scaled by 2^-e, e up to 100: the products are
    those of e = 0."""
    rng = np.random.default_rng(8)
    x, w = rng.normal(0, 1, (rows, 320)).astype(np.float32), rng.normal(0, 1, (200, 320)).astype(np.float32)
    ref = None
    for e in (0, 100, -100):
        xt = torch.tensor(x * np.float32(2.0 ** e)).cuda()
        wt = tea.mx4_quantize(torch.tensor(w * np.float32(2.0 ** -e)).cuda(), "mxfp4")
        y = tea.mx4_linear(xt, wt, dtype=torch.float32)
        ref = y if ref is None else ref
        assert torch.equal(y, ref)


@pytest.mark.parametrize("rows", [6, 200])
def test_gelu_far_from_zero(rows):
    """GELU of +-1, +-30, +-1e5, +-1e20 next to one another in every order: x or 0, and no
    value disturbs its neighbour."""
    v = torch.tensor([1.0, -1.0, 30.0, -30.0, 1e5, -1e5, 1e20, -1e20, 0.0])
    bias = torch.stack([torch.stack([a, b]) for a in v for b in v]).reshape(-1).cuda()
    w = tea.mx4_quantize(torch.zeros(bias.numel(), 64, device="cuda"), "mxfp4")
    y = _np(tea.mx4_linear(torch.randn(rows, 64, device="cuda"), w, bias=bias, gelu=True, dtype=torch.float32))
    b = _np(bias)
    ref = np.where(np.abs(b) > 10, np.maximum(b, 0), mq.gelu(np.where(np.abs(b) > 10, 0, b)))
    assert np.all(np.abs(y - ref) <= 2.0 ** -17 * np.maximum(np.abs(b) * (np.abs(b) < 10), np.abs(ref)) + np.abs(b) * 2.0 ** -60)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("rows", [7, 300, 5000])
def test_residual_in_place_equals_a_separate_result(rows, fmt):
    x = torch.randn(rows, 256, device="cuda", dtype=torch.bfloat16)
    w = tea.mx4_quantize(torch.randn(1040, 256, device="cuda"), fmt, 0.002)
    r = torch.randn(rows, 1040, device="cuda", dtype=torch.bfloat16)
    ref = tea.mx4_linear(x, w, residual=r, x_scale=TS[fmt])
    same = r.clone()
    out = tea.mx4_linear(x, w, residual=same, out=same, x_scale=TS[fmt])
    assert out.data_ptr() == same.data_ptr() and torch.equal(out, ref)
    assert torch.equal(ref, tea.mx4_linear(x, w, residual=r, x_scale=TS[fmt]))


@pytest.mark.parametrize("fmt", FMTS)
def test_rows_of_a_batch_do_not_depend_on_its_size(fmt):
    """The same rows in batches that take each kernel (few tokens, single tiles, pairs)."""
    x = torch.randn(6000, 768, device="cuda", dtype=torch.bfloat16)
    w = tea.mx4_quantize(torch.randn(2304, 768, device="cuda") * 0.05, fmt, 1e-4)
    whole = tea.mx4_linear(x, w, x_scale=TS[fmt], dtype=torch.float32)
    for n in (1, 20, 64, 300, 3000):
        part = tea.mx4_linear(x[:n], w, x_scale=TS[fmt], dtype=torch.float32)
        # sums of 768 products in another order: (K + 3) 2^-23 of their magnitudes, here as norms
        assert torch.linalg.norm(part - whole[:n]) <= 771 * 2.0 ** -23 * torch.linalg.norm(whole[:n])


def test_a_run_of_the_operators_as_a_feed_forward_block():
    """LayerNorm -> 4 bits -> up + GELU -> 4 bits -> down + residual, as used together, for one
    token, a few, and many; every row alone gives the row of the batch."""
    rng = np.random.default_rng(11)
    h, f = 768, 2048
    for fmt in FMTS:
        w1, w1t = _weight(rng, f, h, fmt, 0.03)
        w2, w2t = _weight(rng, h, f, fmt, 0.03)
        b1, b2 = rng.normal(0, 0.1, f).astype(np.float32), rng.normal(0, 0.1, h).astype(np.float32)
        g, b = torch.ones(h, device="cuda"), torch.zeros(h, device="cuda")

        def block(t):
            y, y4 = tea.mx4_layer_norm(t, g, b, 1e-12, fmt, TS[fmt])
            u = tea.mx4_linear_quant(y4, w1t, torch.tensor(b1).cuda(), gelu=True, out_scale=TS[fmt])
            return tea.mx4_linear(u, w2t, torch.tensor(b2).cuda(), residual=y)

        x, t = _rows(rng, 300, h, "bf16")
        out = _np(block(t))
        mu = x.mean(1, keepdims=True, dtype=np.float64)
        y = (x - mu) / np.sqrt(((x - mu) ** 2).mean(1, keepdims=True) + 1e-12)
        hid = mq.gelu(mq.rounded(y.astype(np.float32), fmt, TS[fmt]) @ w1.T + b1)
        ref = mq.rounded(hid.astype(np.float32), fmt, TS[fmt]) @ w2.T + b2 + y
        # bf16 rounding of y and of the result, and the rare code that falls on the other
        # side of a border (a step of it times one weight)
        assert np.linalg.norm(out - ref) <= 2.0 ** -7 * np.linalg.norm(ref)
        assert np.abs(out - ref).max() <= 2.0 ** -7 * np.abs(ref).max() + 2 * 0.03 * 5 * np.abs(hid).max() / 3
        for lo, hi in ((0, 1), (7, 9), (20, 60)):
            part = _np(block(t[lo:hi]))
            assert np.linalg.norm(part - out[lo:hi]) <= 2.0 ** -7 * np.linalg.norm(out[lo:hi])


# -------------------------------------------------- streams, graphs, repeats --

@pytest.mark.parametrize("rows", [1, 24, 700])
def test_two_streams_and_a_captured_graph_give_the_same_bits(rows):
    x = torch.randn(rows, 768, device="cuda", dtype=torch.bfloat16)
    w = tea.mx4_quantize(torch.randn(2304, 768, device="cuda"), "mxfp4")
    w2 = tea.mx4_quantize(torch.randn(768, 2304, device="cuda"), "mxfp4")

    def go(s=None):
        return tea.mx4_linear(tea.mx4_linear_quant(x, w, gelu=True, stream=s), w2, stream=s)

    ref = go()
    assert torch.equal(ref, go())
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    outs = [go(s) for _ in range(3) for s in (s1, s2)]
    torch.cuda.synchronize()
    assert all(torch.equal(ref, o) for o in outs)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = go()
    graph2 = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph2):
        out2 = go()
    for _ in range(2):
        out.zero_()
        out2.zero_()
        graph.replay()
        graph2.replay()
        torch.cuda.synchronize()
        assert torch.equal(ref, out) and torch.equal(ref, out2)
    assert tea.mx4_status() == 0


def test_wrappers_refuse_mismatched_tensors():
    x = torch.randn(8, 64, device="cuda")
    w = tea.mx4_quantize(torch.randn(48, 64, device="cuda"))
    bad = [dict(x=x[:, :32]), dict(x=x.t()), dict(x=x.int()), dict(x=x.cpu()), dict(bias=torch.zeros(47, device="cuda")),
           dict(bias=torch.zeros(48)), dict(residual=torch.zeros(8, 48, device="cuda")),
           dict(residual=torch.zeros(7, 48, device="cuda", dtype=torch.bfloat16)),
           dict(out=torch.zeros(8, 47, device="cuda")), dict(dtype=torch.float64),
           dict(out=torch.zeros(8, 48, device="cuda"), dtype=torch.float16),
           dict(x=x.clone().requires_grad_()), dict(x=tea.mx4_quantize(x, "nvfp4", 0.1)),
           dict(x=torch.empty_strided((8, 64), (32, 1), device="cuda"))]
    for kw in bad:
        with pytest.raises(ValueError):
            tea.mx4_linear(**{"x": x, "w": w, **kw})
    with pytest.raises((ValueError, tea.AlbertError)):
        tea.mx4_linear(tea.mx4_quantize(x), w, out=torch.zeros(8, 96, device="cuda")[:, ::2])
    with pytest.raises(ValueError):
        tea.mx4_layer_norm(x, torch.ones(63, device="cuda"), torch.zeros(64, device="cuda"))
    with pytest.raises(ValueError):
        tea.mx4_quantize(x, "nvfp4", 0.0)
    with torch.no_grad():
        tea.mx4_linear(x.clone().requires_grad_(), w)


def test_block_scales_of_many_magnitudes_and_tensor_scales():
    """nvfp4: amax / (6 ts) correctly rounded before E4M3, over random magnitudes, E4M3's
    midpoints (and their fp32 neighbours) times 6 ts, and tensor scales of any mantissa."""
    rng = np.random.default_rng(77)
    g = mq.e4m3_grid()
    mids = ((g[:-1] + g[1:]) / 2).astype(np.float32)
    for ts in (1.0, 0.0093, 7e-5, 0.33333334, 1.9999999, 2.0 ** -90, 3e20):
        with np.errstate(over="ignore"):
            near = (mids * (np.float32(6) * np.float32(ts))).astype(np.float32)
        a = np.concatenate([near, np.nextafter(near, np.float32(0)), np.nextafter(near, np.float32(np.inf)),
                            (np.exp(rng.uniform(-12, 8, 4000)) * 6 * ts).astype(np.float32)])
        a = a[np.isfinite(a)]
        x = np.zeros((a.size, 16), np.float32)
        x[:, 3] = a
        q = tea.mx4_quantize(torch.tensor(x).cuda(), "nvfp4", ts)
        codes, byte = _stored(q)
        want_c, want_b = mq.quantize(x, "nvfp4", ts)
        np.testing.assert_array_equal(byte, want_b)
        np.testing.assert_array_equal(codes, want_c)


def test_mixed_calls_on_several_streams_at_once():
    """Products of every kind (few tokens with and without a cluster, single tiles, pairs, 4-bit
    results) interleaved on four streams give the bits they give alone."""
    g = torch.Generator(device="cuda").manual_seed(3)
    calls = []
    for fmt, rows, n, k in [("mxfp4", 1, 2304, 768), ("nvfp4", 12, 512, 2048), ("nvfp4", 30, 256, 256),
                            ("mxfp4", 200, 768, 768), ("nvfp4", 3000, 1024, 512), ("mxfp4", 7, 8192, 1024)]:
        x = torch.randn(rows, k, device="cuda", generator=g).to(torch.bfloat16)
        w = tea.mx4_quantize(torch.randn(n, k, device="cuda", generator=g) * 0.05, fmt, 1e-4)
        calls.append((x, w, TS[fmt]))

    def run(c, s=None):
        x, w, ts = c
        return tea.mx4_linear(x, w, x_scale=ts, stream=s), tea.mx4_linear_quant(x, w, gelu=True, x_scale=ts, out_scale=ts,
                                                                               stream=s)

    alone = [run(c) for c in calls]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(4)]
    for rep in range(6):
        outs = [(i, run(calls[i], streams[(i + rep + j) % 4])) for j in range(4) for i in range(len(calls))]
        torch.cuda.synchronize()
        for i, (y, q) in outs:
            assert torch.equal(y, alone[i][0]) and torch.equal(q.codes, alone[i][1].codes)
    assert tea.mx4_status() == 0
