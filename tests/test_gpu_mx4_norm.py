"""LayerNorm with a 4-bit result where its statistics are hard: rows of one value, rows whose
spread is small beside their mean; and ordinary rows to a few units in the last place.

The tolerance, with u = 2^-24 and m0 the mean that the kernel's first pass finds:
  * a sum of the lanes' values, the shuffles and the warps has at most D additions in a row,
    each off by u of a partial sum: 8 per 2048 columns in the kernels that hold a row, 8 per
    eight chunks of 256 in the one for wider rows, 5 shuffles, 16 warps joined in at most 9,
    6 for the final products and pairs: D = 20 + 8 ceil(cols / 2048) covers them;
  * so |m0 - mean| <= D u max|x|, and d = x - m0 is off by u |d|.  Its mean e and mean square
    q are off by D u mean|d| <= D u sqrt(q) and (D + 2) u q.  The variance v = q - e^2 has
    q = v + e^2 = v r, r = 1 + (D u max|x|)^2 / v at the most, and is off by (D + 2) u q
    + 2 |e| D u sqrt(q) + u q <= (3 D + 3) u r v;
  * rstd: half of that (relative), 2 units of the reciprocal square root (4 u), and one u each
    for the additions of eps; -e rstd, the two fma of the result: one u each of what they give.
With h = (x - mean) rstd:
  |y - ref| <= u (|g| (D sqrt(r) + |h| ((3 D + 3) r / 2 + 8) + 2 sqrt(r)) + 2 |ref| + |b|),
then the rounding to the rows' type."""
import numpy as np
import pytest
import torch

import transformer_encoder_albert_b200 as tea
from oracle import mx4_quant as mq

pytestmark = pytest.mark.gpu
FMTS = ["mxfp4", "nvfp4"]
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
TS = {"mxfp4": 1.0, "nvfp4": 0.0093}
U = 2.0 ** -24
# every kernel: a warp per row, a CTA of 2, 4, 8, 16 warps (by values and by words), wider rows
SHAPES = [(3, 1), (5, 200), (600, 256), (600, 768), (600, 520), (3, 768), (40, 1000), (700, 1000), (40, 1001),
          (600, 2047), (9, 2000), (300, 4096), (9, 4001), (5, 8000), (6, 8191), (3, 9000), (2, 20001)]


def _inputs(rng, cols):
    g = (1 + rng.normal(0, 0.2, cols)).astype(np.float32)
    b = rng.normal(0, 0.2, cols).astype(np.float32)
    return g, b, torch.tensor(g).cuda(), torch.tensor(b).cuda()


def _check(x, t, g, b, tg, tb, eps, dtype, fmt):
    cols = x.shape[1]
    y, q = tea.mx4_layer_norm(t, tg, tb, eps, fmt, TS[fmt])
    d = x - x.mean(1, keepdims=True)
    v = (d * d).mean(1, keepdims=True) + eps
    h = d / np.sqrt(v)
    ref = h * g + b
    D = 20 + 8 * -(-cols // 2048)
    r = 1 + (D * U * np.abs(x).max(1, keepdims=True)) ** 2 / v
    tol = U * (np.abs(g) * (D * np.sqrt(r) + np.abs(h) * ((3 * D + 3) * r / 2 + 8) + 2 * np.sqrt(r)) + 2 * np.abs(ref) + np.abs(b))
    got = y.double().cpu().numpy()
    err = np.abs(got - ref)
    half = torch.finfo(DTYPES[dtype]).eps / 2 if dtype != "fp32" else 0
    assert np.all(err <= tol + half * np.abs(ref) * (1 + half) + (2.0 ** -25 if dtype == "fp16" else 0)), float((err - tol).max())
    # the 4-bit form is that of values within tol: its scale bytes lie between those of the
    # largest magnitude less and plus tol, its values a step of the code away at the most
    codes, byte = mq.unpack(q.codes.cpu().numpy(), q.scales.cpu().numpy(), q.rows, q.cols, fmt)
    rb, tb_ = mq.blocks(np.abs(ref), fmt), mq.blocks(tol, fmt)
    lo = mq.scale_bytes(np.maximum((rb - tb_).max(2), 0).astype(np.float32) * np.float32(1 - 2.0 ** -22), fmt, TS[fmt])
    hi = mq.scale_bytes((rb + tb_).max(2).astype(np.float32) * np.float32(1 + 2.0 ** -22), fmt, TS[fmt])
    assert np.all((byte >= lo) & (byte <= hi))
    val = mq.values(codes, byte, fmt, TS[fmt], cols)
    s = np.repeat(mq.scale_values(byte, fmt) * (TS[fmt] if fmt == "nvfp4" else 1.0), mq.BLOCK[fmt], 1)[:, :cols]
    step = np.where(np.abs(ref) < 1.75 * s, 0.25, np.where(np.abs(ref) < 3.5 * s, 0.5, 1.0)) * s
    assert np.all(np.abs(val - ref) <= np.maximum(step, np.maximum(np.abs(ref) - 6 * s, 0)) + 2 * tol + s * 2.0 ** -20)


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_rows_to_a_few_units_in_the_last_place(rows, cols, dtype):
    rng = np.random.default_rng(rows + cols)
    t = torch.tensor(rng.normal(0, 3, (rows, cols)).astype(np.float32)).to(DTYPES[dtype])
    for fmt in FMTS:
        _check(t.double().numpy(), t.cuda(), *_inputs(rng, cols), 1e-5, dtype, fmt)


@pytest.mark.parametrize("rows,cols", SHAPES)
def test_rows_whose_spread_is_small_beside_their_mean(rows, cols):
    """fp32 rows of mean 1000 and spread 0.01: the mean's rounding alone is up to a tenth of it."""
    rng = np.random.default_rng(rows * cols)
    t = torch.tensor((1000 + 0.01 * rng.normal(0, 1, (rows, cols))).astype(np.float32))
    _check(t.double().numpy(), t.cuda(), *_inputs(rng, cols), 1e-12, "fp32", "mxfp4")


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_rows_of_one_value_give_beta(rows, cols, dtype):
    """d = x - m0 is the same for all, at most (D + 1) u |c|; e is that within D u of itself, and
    rstd at most 1 / sqrt(eps): |y - b| <= |g| (D + 2)^2 u^2 |c| / sqrt(eps) + u |b|."""
    rng = np.random.default_rng(cols)
    g, b, tg, tb = _inputs(rng, cols)
    c = torch.tensor([3.0, 100.0, 0.1, -7.3, 0.0]).to(DTYPES[dtype])[torch.arange(rows) % 5]
    y, _ = tea.mx4_layer_norm(c[:, None].repeat(1, cols).cuda(), tg, tb, 1e-12)
    D = 20 + 8 * -(-cols // 2048)
    tol = np.abs(g) * (D + 2) ** 2 * U * U * c.double().abs().numpy()[:, None] / 1e-6 + 2 * U * np.abs(b)
    half = torch.finfo(DTYPES[dtype]).eps / 2
    assert np.all(np.abs(y.double().cpu().numpy() - b) <= tol + half * (np.abs(b) + tol) + (2.0 ** -25 if dtype == "fp16" else 0))


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_normalized_rows_at_any_offset_of_a_wider_buffer(rows, cols, dtype):
    """y by its C entry in rows of every alignment (gamma, beta too): the same values whatever the
    kernel's way of moving them allows, nothing beside them, and x's own rows as y."""
    rng = np.random.default_rng(cols + 1)
    t = torch.tensor(rng.normal(0, 3, (rows, cols)).astype(np.float32)).to(DTYPES[dtype]).cuda()
    g, b, tg, tb = _inputs(rng, cols)
    typ = {"bf16": tea.ALBERT_BF16, "fp16": tea.ALBERT_FP16, "fp32": tea.ALBERT_FP32}[dtype]
    ref, q = tea.mx4_layer_norm(t, tg, tb, 1e-5, "mxfp4")
    params = torch.zeros(2, cols + 8, device="cuda")
    half = torch.finfo(DTYPES[dtype]).eps / 2
    for off, ld, shift in ((0, -(-cols // 16) * 16 + 16, 0), (8, -(-cols // 8) * 8 + 8, 4), (1, cols + 2, 1), (3, cols + 5, 3)):
        buf = torch.full((rows * ld + 16,), 7.0, device="cuda", dtype=DTYPES[dtype])
        y = buf[off:off + rows * ld].view(rows, ld)[:, :cols]
        pg, pb = params[0, shift:shift + cols], params[1, shift:shift + cols]
        pg.copy_(tg)
        pb.copy_(tb)
        for x in (t, y):
            if x is y:
                y.copy_(t)
            rc = tea.lib().albert_mx4_layer_norm(x.data_ptr(), typ, cols if x is t else ld, pg.data_ptr(), pb.data_ptr(), 1e-5,
                                                 rows, cols, tea.ALBERT_MXFP4, 1.0, y.data_ptr(), ld, q.codes.data_ptr(),
                                                 q.scales.data_ptr(), torch.cuda.current_stream().cuda_stream)
            assert rc == 0
            # (two kernels may sum in another order: twice the bound of the statistics, and a step)
            D = 20 + 8 * -(-cols // 2048)
            yd, rd = y.double(), ref.double()
            h = ((rd - tb.double()) / tg.double()).abs()
            tol = 2 * U * (tg.double().abs() * (D + h * (1.5 * D + 12) + 2) + 2 * rd.abs() + tb.double().abs())
            assert torch.all((yd - rd).abs() <= 2 * tol + 2 * half * rd.abs() + (2.0 ** -24 if dtype == "fp16" else 0))
        y.fill_(7.0)
        assert torch.all(buf == 7.0)


@pytest.mark.parametrize("rows,cols", SHAPES)
def test_rows_with_a_nan_or_an_infinity_are_nan_and_no_others(rows, cols):
    rows = max(rows, 5)
    x = torch.randn(rows, cols, device="cuda")
    x[0, cols // 2] = float("nan")
    x[1, 0] = float("inf")
    x[2, cols - 1] = -float("inf")
    y, q = tea.mx4_layer_norm(x, torch.ones(cols, device="cuda"), torch.zeros(cols, device="cuda"), 1e-5)
    back = tea.mx4_dequantize(q, dtype=torch.float32)
    assert torch.isnan(y[:3]).all() and torch.isnan(back[:3]).all()
    assert torch.isfinite(y[3:]).all() and torch.isfinite(back[3:]).all()
    # and far beyond fp32's square: beta, not NaN
    y, _ = tea.mx4_layer_norm(torch.full((2, cols), 1e33, device="cuda") * torch.linspace(-1, 1, cols, device="cuda"),
                              torch.ones(cols, device="cuda"), torch.full((cols,), 0.5, device="cuda"), 1e-5)
    assert torch.isfinite(y).all()
