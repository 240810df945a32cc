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


# ----------------------------------------------------------------- residuals --

RES = [(5, 200, 100), (24, 1000, 768), (40, 1001, 300), (300, 512, 256), (2600, 2020, 288)]


def _residual_case(rng, rows, n, k, dtype, fmt):
    """x, w and the residual with the 64-bit result, and how far fp32 sums and the rounding to
    dtype may be from it: every one of K + 3 additions off by 2^-23 of a partial sum, the residual's
    by 2^-23 of the result, half a step of dtype (and of fp16's smallest subnormal)."""
    x = torch.tensor(rng.normal(0, 1, (rows, k)).astype(np.float32)).to(torch.bfloat16)
    wv = rng.normal(0, 0.05, (n, k)).astype(np.float32)
    res = torch.tensor(rng.normal(0, 1, (rows, n)).astype(np.float32)).to(DTYPES[dtype])
    wts = 1e-4 if fmt == "nvfp4" else 1.0
    a, w = mq.rounded(x.float().numpy(), fmt, TS[fmt]), mq.rounded(wv, fmt, wts)
    ref = a @ w.T + res.double().numpy()
    tol = (k + 3) * 2.0 ** -23 * (np.abs(a) @ np.abs(w).T) + 2.0 ** -23 * np.abs(ref)
    half = torch.finfo(DTYPES[dtype]).eps / 2
    tol = tol + half * (np.abs(ref) + tol) + (2.0 ** -25 if dtype == "fp16" else 0)
    return x.cuda(), tea.mx4_quantize(torch.tensor(wv).cuda(), fmt, wts), res.cuda(), ref, tol


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("rows,n,k", RES)
def test_residuals_of_every_type_in_place_and_at_any_offset(rows, n, k, dtype, fmt):
    rng = np.random.default_rng(rows + n + k)
    x, w, res, ref, tol = _residual_case(rng, rows, n, k, dtype, fmt)
    want = tea.mx4_linear(x, w, residual=res, dtype=DTYPES[dtype], x_scale=TS[fmt])
    err = np.abs(_np(want) - ref)
    assert np.all(err <= tol), float((err - tol).max())
    same = res.clone()
    tea.mx4_linear(x, w, residual=same, out=same, x_scale=TS[fmt])
    assert torch.equal(same, want)
    # rows 16-byte aligned or not, the residual's and the result's apart; nothing beside them
    for off_r, pad_r, off_o, pad_o in ((8, 16 - n % 8, 0, 24 - n % 8), (1, 3, 8, 16 - n % 8), (8, 8 - n % 8, 3, 5), (1, 1, 1, 2)):
        rb = torch.full((rows * (n + pad_r) + 16,), float("nan"), device="cuda", dtype=DTYPES[dtype])
        rv = rb[off_r:off_r + rows * (n + pad_r)].view(rows, n + pad_r)[:, :n]
        rv.copy_(res)
        ob = torch.full((rows * (n + pad_o) + 16,), 7.0, device="cuda", dtype=DTYPES[dtype])
        ov = ob[off_o:off_o + rows * (n + pad_o)].view(rows, n + pad_o)[:, :n]
        tea.mx4_linear(x, w, residual=rv, out=ov, x_scale=TS[fmt])
        assert torch.equal(ov, want)
        ov.fill_(7.0)
        assert torch.all(ob == 7.0)
        tea.mx4_linear(x, w, residual=rv, out=rv, x_scale=TS[fmt])
        assert torch.equal(rv, want)
    assert tea.mx4_status() == 0


# -------------------------------------------------------- what a call writes --

def _tensor(rows, cols, fmt):
    """A 4-bit matrix over buffers filled with 0xAA, and the bytes behind each."""
    c, s = tea.mx4_shapes(rows, cols, fmt)
    n, m = c[0] * c[1], s[0] * s[1] * s[2]
    cb, sb = (torch.full((k + 512,), 0xAA, dtype=torch.uint8, device="cuda") for k in (n, m))
    return tea.Mx4Tensor(cb[:n].view(c), sb[:m].view(s), rows, cols, fmt, TS[fmt]), cb[n:], sb[m:]


def _check_past_rows(q, behind_codes, behind_scales):
    t = q.scales.cpu().numpy()
    r, b = np.arange(q.rows, t.shape[0] * 128)[:, None], np.arange(t.shape[1] * 4)[None]
    assert np.all(t[r // 128, b // 4, (r % 32) * 16 + (r % 128) // 32 * 4 + b % 4] == 0)
    r, b = np.arange(q.rows)[:, None], np.arange(q.codes.shape[1] * 2 // mq.BLOCK[q.fmt], t.shape[1] * 4)[None]
    assert np.all(t[r // 128, b // 4, (r % 32) * 16 + (r % 128) // 32 * 4 + b % 4] == 0)
    assert torch.all(behind_codes == 0xAA) and torch.all(behind_scales == 0xAA)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 200), (7, 768), (600, 700), (128, 256), (700, 768), (1, 1000), (129, 1001),
                                       (9, 2000), (5, 4096), (3, 8001), (1, 8200), (140, 9000)])
def test_layer_norm_writes_whole_scale_tiles(rows, cols, fmt):
    q, cb, sb = _tensor(rows, cols, fmt)
    x, g, b = torch.randn(rows, cols, device="cuda"), torch.ones(cols, device="cuda"), torch.zeros(cols, device="cuda")
    rc = tea.lib().albert_mx4_layer_norm(x.data_ptr(), tea.ALBERT_FP32, cols, g.data_ptr(), b.data_ptr(), 1e-5, rows, cols,
                                         tea.MX4_FORMATS[fmt], TS[fmt], None, 0, q.codes.data_ptr(), q.scales.data_ptr(),
                                         torch.cuda.current_stream().cuda_stream)
    assert rc == 0
    _check_past_rows(q, cb, sb)
    ref = tea.mx4_layer_norm(x, g, b, 1e-5, fmt, TS[fmt], return_rows=False)[1]
    assert torch.equal(q.codes, ref.codes) and torch.equal(q.scales, ref.scales)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("rows,n,k", [(1, 32, 32), (1, 2048, 768), (5, 100, 96), (16, 300, 4200), (31, 33, 256), (32, 640, 768),
                                      (33, 256, 300), (130, 320, 768), (129, 1000, 64), (300, 2048, 256), (2600, 2020, 288),
                                      (10000, 1030, 96)])
def test_a_4_bit_result_writes_whole_scale_tiles(rows, n, k, fmt):
    import ctypes as C
    q, cb, sb = _tensor(rows, n, fmt)
    w = tea.mx4_quantize(torch.randn(n, k, device="cuda") * 0.05, fmt, 1e-4)
    x = tea.mx4_quantize(torch.randn(rows, k, device="cuda"), fmt, TS[fmt])
    a = tea.albert_mx4_linear_args()
    for f, v in dict(a_codes=x.codes.data_ptr(), a_scales=x.scales.data_ptr(), w_codes=w.codes.data_ptr(),
                     w_scales=w.scales.data_ptr(), q_codes=q.codes.data_ptr(), q_scales=q.scales.data_ptr(), x_scale=TS[fmt],
                     w_scale=1e-4, q_scale=TS[fmt], rows=rows, n=n, k=k, fmt=tea.MX4_FORMATS[fmt]).items():
        setattr(a, f, v)
    assert tea.lib().albert_mx4_linear(C.byref(a), torch.cuda.current_stream().cuda_stream) == 0
    _check_past_rows(q, cb, sb)
    ref = tea.mx4_linear_quant(x, w, out_scale=TS[fmt])
    assert torch.equal(q.codes, ref.codes) and torch.equal(q.scales, ref.scales)


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("rows", [1, 30, 40, 300, 5000])
def test_a_result_leaves_the_columns_beside_it_alone(rows, dtype):
    """Results of every width modulo 8 in 16-byte aligned rows of a wider buffer."""
    x = torch.randn(rows, 300, device="cuda", dtype=torch.bfloat16)
    for n in (1, 33, 200, 1001, 1002, 1003, 1004, 1005, 1006, 1007, 1008):
        w = tea.mx4_quantize(torch.randn(n, 300, device="cuda"), "mxfp4")
        ld = -(-n // 8) * 8 + 16
        ref = tea.mx4_linear(x, w, dtype=DTYPES[dtype])
        buf = torch.full((rows, ld), 7.0, device="cuda", dtype=DTYPES[dtype])
        tea.mx4_linear(x, w, out=buf[:, :n])
        assert torch.equal(buf[:, :n], ref) and torch.all(buf[:, n:] == 7.0), n
        res = torch.full((rows, ld), float("nan"), device="cuda", dtype=DTYPES[dtype])
        res[:, :n] = 0
        buf[:, :n] = 0
        tea.mx4_linear(x, w, residual=res[:, :n], out=buf[:, :n])
        assert torch.equal(buf[:, :n], ref) and torch.all(buf[:, n:] == 7.0), n


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("rows", [1, 5, 32, 33, 300, 5000])
def test_a_result_over_its_own_input(rows, fmt):
    """x and out are the same rows, share columns of one buffer, or lie beside one another in it."""
    buf = torch.randn(rows, 1600, device="cuda", dtype=torch.bfloat16)
    w = tea.mx4_quantize(torch.randn(768, 768, device="cuda") * 0.05, fmt, 1e-4)
    ref = tea.mx4_linear(buf[:, :768].clone(), w, x_scale=TS[fmt])
    for at in (0, 64, 767, 800):
        b = buf.clone()
        out = tea.mx4_linear(b[:, :768], w, out=b[:, at:at + 768], x_scale=TS[fmt])
        assert torch.equal(out, ref)
        b[:, at:at + 768] = buf[:, at:at + 768]
        assert torch.equal(b, buf)


# ------------------------------------------------------------------- streams --

def test_inputs_of_a_call_on_another_stream_keep_their_memory(monkeypatch):
    """Every tensor of a call on another stream is recorded on it, so that the allocator does not
    hand its memory out before the call has run where the caller drops it at once; the results
    are those of the call alone."""
    g = torch.Generator(device="cuda").manual_seed(5)
    rows, n, k = 300, 512, 256
    x = torch.randn(rows, k, device="cuda", generator=g).to(torch.bfloat16)
    gamma, beta = (torch.randn(k, device="cuda", generator=g) for _ in range(2))
    bias = torch.randn(n, device="cuda", generator=g)
    res = torch.randn(rows, n, device="cuda", generator=g).to(torch.bfloat16)
    w = tea.mx4_quantize(torch.randn(n, k, device="cuda", generator=g) * 0.05, "mxfp4")
    u = tea.mx4_quantize(x, "mxfp4")
    v = tea.Mx4Tensor(u.codes.clone(), u.scales.clone(), rows, k, "mxfp4")
    out = torch.empty(rows, n, device="cuda", dtype=torch.bfloat16)
    given = tea.mx4_empty(rows, k)
    calls = [((x, given), lambda s: tea.mx4_quantize(x, "mxfp4", out=given, stream=s).codes),
             ((u,), lambda s: tea.mx4_dequantize(u, stream=s)),
             ((v, out), lambda s: tea.mx4_dequantize(v, out=out[:, :k], stream=s)),
             ((x, gamma, beta), lambda s: tea.mx4_layer_norm(x, gamma, beta, 1e-5, stream=s)[0]),
             ((x, w, bias, res, out), lambda s: tea.mx4_linear(x, w, bias, res, out=out, stream=s)),
             ((x, w), lambda s: tea.mx4_linear(x[:4], w, stream=s)),
             ((v, w, bias), lambda s: tea.mx4_linear_quant(v, w, bias, stream=s).codes)]
    side, seen = torch.cuda.Stream(), set()
    keep = torch.Tensor.record_stream
    monkeypatch.setattr(torch.Tensor, "record_stream",
                        lambda t, s: (seen.add((t.untyped_storage().data_ptr(), s.cuda_stream)), keep(t, s))[1])
    for used, call in calls:
        ref = call(None).clone()
        assert not seen
        torch.cuda.synchronize()
        got = call(side)
        torch.cuda.synchronize()
        assert torch.equal(got, ref)
        parts = [p for t in used for p in ((t.codes, t.scales) if type(t) is tea.Mx4Tensor else (t,))]
        assert {(p.untyped_storage().data_ptr(), side.cuda_stream) for p in parts} == seen
        seen.clear()


# ------------------------------------------------------------- expired waits --

@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("rows,n,k", [(5, 300, 768), (5, 256, 200), (20, 2304, 4200), (32, 40000, 512), (64, 300, 768),
                                      (300, 640, 4200), (5000, 2304, 256)])
@pytest.mark.parametrize("four_bit", [False, True])
def test_expired_waits_are_reported_and_later_calls_are_right(rows, n, k, fmt, four_bit):
    """Withheld loads with a limit of 2 ms: in a cluster and alone, one tile and several per CTA,
    CTA pairs.  The call returns, the status says so once, the next call is as before."""
    import ctypes as C
    x = tea.mx4_quantize(torch.randn(rows, k, device="cuda"), fmt, TS[fmt])
    w = tea.mx4_quantize(torch.randn(n, k, device="cuda") * 0.05, fmt, 1e-4)
    good = tea.mx4_linear_quant(x, w, out_scale=TS[fmt]).codes if four_bit else tea.mx4_linear(x, w)
    assert tea.mx4_status() == 0
    a = tea.albert_mx4_linear_args()
    for f, v in dict(a_codes=x.codes.data_ptr(), a_scales=x.scales.data_ptr(), w_codes=w.codes.data_ptr(),
                     w_scales=w.scales.data_ptr(), x_scale=TS[fmt], w_scale=1e-4, q_scale=TS[fmt], rows=rows, n=n, k=k,
                     fmt=tea.MX4_FORMATS[fmt]).items():
        setattr(a, f, v)
    out, q = torch.empty(rows, n, device="cuda", dtype=torch.bfloat16), tea.mx4_empty(rows, n, fmt, TS[fmt])
    if four_bit:
        a.q_codes, a.q_scales = q.codes.data_ptr(), q.scales.data_ptr()
    else:
        a.out, a.ld_out = out.data_ptr(), n
    stream = torch.cuda.current_stream().cuda_stream
    assert tea.lib().albert_test_mx4_linear_stall(C.byref(a), 0, stream) == 2
    assert tea.lib().albert_test_mx4_linear_stall(C.byref(a), 2_000_000, stream) == 0
    assert tea.mx4_status() == 8  # ALBERT_ERR_TIMEOUT
    assert tea.mx4_status() == 0
    again = tea.mx4_linear_quant(x, w, out_scale=TS[fmt]).codes if four_bit else tea.mx4_linear(x, w)
    assert torch.equal(again, good) and tea.mx4_status() == 0


def test_one_of_several_callers_takes_a_recorded_status():
    import ctypes as C
    import threading
    x, w = (tea.mx4_quantize(torch.randn(n, 256, device="cuda"), "mxfp4") for n in (3, 128))
    out = torch.empty(3, 128, device="cuda", dtype=torch.bfloat16)
    a = tea.albert_mx4_linear_args()
    for f, v in dict(a_codes=x.codes.data_ptr(), a_scales=x.scales.data_ptr(), w_codes=w.codes.data_ptr(),
                     w_scales=w.scales.data_ptr(), out=out.data_ptr(), ld_out=128, rows=3, n=128, k=256,
                     fmt=tea.ALBERT_MXFP4).items():
        setattr(a, f, v)
    assert tea.mx4_status() == 0
    streams = [torch.cuda.Stream() for _ in range(8)]
    for rep in range(5):
        assert tea.lib().albert_test_mx4_linear_stall(C.byref(a), 1_000_000, torch.cuda.current_stream().cuda_stream) == 0
        torch.cuda.synchronize()
        got, start = [], threading.Barrier(8)

        def ask(s):
            start.wait()
            got.append(tea.mx4_status(s))

        threads = [threading.Thread(target=ask, args=(s,)) for s in streams]
        for t in threads:
            t.start()
        for t in threads:
            t.join()
        assert sorted(got) == [0] * 7 + [8]


def test_calls_with_a_stream_may_be_captured_on_it():
    x, g, b = torch.randn(300, 768, device="cuda", dtype=torch.bfloat16), torch.ones(768, device="cuda"), torch.zeros(768, device="cuda")
    w = tea.mx4_quantize(torch.randn(512, 768, device="cuda") * 0.05, "mxfp4")

    def go(s):
        y, y4 = tea.mx4_layer_norm(x, g, b, 1e-5, stream=s)
        h = tea.mx4_linear_quant(y4, w, gelu=True, stream=s)
        return y, tea.mx4_dequantize(h, stream=s), tea.mx4_linear(x, w, stream=s), tea.mx4_linear(x[:3], w, stream=s)

    ref = go(None)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = go(torch.cuda.current_stream())
    for _ in range(2):
        for o in out:
            o.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(o, r) for o, r in zip(out, ref))


def test_the_first_calls_of_a_process_may_be_captured():
    """Nothing that the entries look up or set up on their first call keeps it out of a graph."""
    import subprocess
    import sys
    code = """
import torch, transformer_encoder_albert_b200 as tea
x, wv = (torch.randn(*s, device="cuda", dtype=torch.bfloat16) for s in ((300, 768), (512, 768)))
g, b = torch.ones(768, device="cuda"), torch.zeros(768, device="cuda")
torch.cuda.synchronize()
def go():
    w = tea.mx4_quantize(wv, "nvfp4", 0.001)
    y, y4 = tea.mx4_layer_norm(x, g, b, 1e-5, "nvfp4", 0.01)
    h = tea.mx4_linear_quant(y4, w, gelu=True, out_scale=0.01)
    return y, tea.mx4_dequantize(h), tea.mx4_linear(x, w, x_scale=0.01), tea.mx4_linear(x[:3], w, x_scale=0.01)
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    out = go()
graph.replay()
torch.cuda.synchronize()
assert all(torch.equal(o, r) for o, r in zip(out, go())) and tea.mx4_status() == 0
print("captured")
"""
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "captured" in r.stdout, r.stderr[-2000:]


def test_offsets_past_32_bits():
    """1,100,000 rows of 2048: more than 2^31 values in, out and between; the last rows are those of
    the same rows alone."""
    rows, k = 1_100_000, 2048
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.empty(rows, k, device="cuda", dtype=torch.bfloat16).normal_(generator=g)
    w = tea.mx4_quantize(torch.randn(k, k, device="cuda", generator=g) * 0.02, "mxfp4")
    part = slice(rows - 300, rows)
    q, alone = tea.mx4_quantize(x, "mxfp4"), tea.mx4_quantize(x[part], "mxfp4")
    assert torch.equal(q.codes[part], alone.codes)
    back = tea.mx4_dequantize(q)
    assert torch.equal(back[part], tea.mx4_dequantize(alone))
    del back
    y = tea.mx4_linear(q, w)
    assert torch.equal(y[part], tea.mx4_linear(alone, w))
    r = tea.mx4_linear(x, w, residual=y, out=y)
    assert torch.equal(r[part], tea.mx4_linear(alone, w, residual=tea.mx4_linear(alone, w)))
    del y, r
    gamma, beta = torch.ones(k, device="cuda"), torch.zeros(k, device="cuda")
    n, n4 = tea.mx4_layer_norm(x, gamma, beta, 1e-5)
    m, m4 = tea.mx4_layer_norm(x[part], gamma, beta, 1e-5)
    assert torch.equal(n[part], m) and torch.equal(n4.codes[part], m4.codes)
    del n
    u = tea.mx4_linear_quant(n4, w, gelu=True)
    assert torch.equal(u.codes[part], tea.mx4_linear_quant(m4, w, gelu=True).codes)
    assert tea.mx4_status() == 0
