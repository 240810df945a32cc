"""Linear layers on 4-bit operands at the edges of their formula: GELU far from zero, residuals of
every type, in place and at any alignment, what a call leaves in the scale tiles, calls on another
stream than their inputs'."""
import numpy as np
import pytest
import torch

import transformer_encoder_albert_b200 as tea
from oracle import mx4_quant as mq

pytestmark = pytest.mark.gpu
FMTS = ["mxfp4", "nvfp4"]
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
TS = {"mxfp4": 1.0, "nvfp4": 0.0093}


def _np(t):
    return t.double().cpu().numpy()


# ---------------------------------------------------------------------- GELU --

FAR = [-7.6, -7.62, -7.7, -8.0, -9.5, -16.0, -30.0, -1e3, -1e5, -1e10, -1e19, -1e20, -1e30, -3e38]


@pytest.mark.parametrize("rows", [6, 200, 5000])
def test_gelu_far_below_zero_is_zero(rows):
    """z = the bias alone.  Below -7.6 the formula's value is under 10^-18 in magnitude, and so is
    the result, whatever stands beside it; -infinity gives NaN as 0.5 z (1 + tanh) does."""
    v = FAR + [1.0, -1.0, 5.0, 3e38]
    bias = torch.tensor([[a, b] for a in v for b in v] + [[-float("inf"), -9.0], [2.0, -float("inf")]]).reshape(-1)
    w = tea.mx4_quantize(torch.zeros(bias.numel(), 64, device="cuda"), "mxfp4")
    y = _np(tea.mx4_linear(torch.randn(rows, 64, device="cuda"), w, bias=bias.cuda(), gelu=True, dtype=torch.float32))
    b = bias.double().numpy()
    with np.errstate(over="ignore", invalid="ignore"):
        ref = b / (1.0 + np.exp(-2 * np.sqrt(2 / np.pi) * (b + 0.044715 * b ** 3)))
    none = np.isinf(b)
    assert np.isnan(y[:, none]).all()
    # (2^-17: the bound of the exponential's argument where the result is neither z nor 0)
    assert np.all(np.abs(y - ref)[:, ~none] <= 1e-18 + 2.0 ** -17 * np.abs(ref)[~none])


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("rows", [6, 200, 5000])
def test_far_values_do_not_set_a_blocks_scale(rows, fmt):
    """Blocks of -1e20 beside one ordinary value, and of -1e20 alone: the scale is the ordinary
    value's (0 without one), the others read back as 0."""
    n = 96
    bias = torch.full((n,), -1e20)
    bias[5], bias[40] = 1.0, 2.5
    w = tea.mx4_quantize(torch.zeros(n, 64, device="cuda"), fmt, 1.0)
    q = tea.mx4_linear_quant(torch.randn(rows, 64, device="cuda"), w, bias.cuda(), gelu=True, x_scale=TS[fmt], out_scale=TS[fmt])
    ref = np.where(bias.numpy() < 0, 0, mq.gelu(bias.double().numpy()))[None].repeat(rows, 0)
    got = _np(tea.mx4_dequantize(q, dtype=torch.float32))
    assert np.all(got[:, ref[0] == 0] == 0)
    # the nearest code of a value known to within 2^-17: half a step (mxfp4 up to 1/4 of a binade
    # of 4 codes, nvfp4 the scale's rounding by 1/16 more)
    assert np.all(np.abs(got - ref) <= np.abs(ref) * (0.25 + 2.0 ** -16))
    _, byte = mq.unpack(q.codes.cpu().numpy(), q.scales.cpu().numpy(), rows, n, fmt)
    assert np.all(byte[:, -1] == 0)
