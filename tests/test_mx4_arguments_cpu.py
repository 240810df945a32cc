"""Arguments of the 4-bit operators without a GPU: calls that the host must refuse, and what the
Python wrappers do with the tensors they are given."""
import ctypes as C

import pytest

import transformer_encoder_albert_b200 as tea
from transformer_encoder_albert_b200 import build as tea_build

P = 1 << 20  # a non-NULL, aligned pointer value that the host checks never dereference
CONFIG = 2


@pytest.fixture(scope="module")
def lib():
    tea_build.build()
    return tea.lib()


def _linear(lib, **kw):
    a = tea.albert_mx4_linear_args()
    base = dict(a_codes=P, a_scales=P, w_codes=P, w_scales=P, out=P, ld_out=48, x_scale=1.0, w_scale=1.0, q_scale=1.0,
                rows=4, n=48, k=64, fmt=3)
    for k, v in {**base, **kw}.items():
        setattr(a, k, v)
    return lib.albert_mx4_linear(C.byref(a), None)


@pytest.mark.parametrize("rows", [4, 300])
def test_a_residual_with_a_4_bit_result_is_refused(lib, rows):
    for fmt in (tea.ALBERT_MXFP4, tea.ALBERT_NVFP4):
        assert _linear(lib, rows=rows, fmt=fmt, out=None, q_codes=P, q_scales=P, residual=P, ld_residual=48) == CONFIG


def test_few_rows_of_x_and_out_that_overlap_are_refused(lib):
    """The few-row kernel reads x while other parts of it write: any shared byte is refused; rows
    that lie between one another, or more than 32 rows, are not."""
    def f(x, out, **kw):
        return _linear(lib, **{**dict(x=x, ld_x=64, out=out, ld_out=48, workspace=8 * P, k=64, n=48), **kw})

    for kw in (dict(), dict(x_type=tea.ALBERT_FP32, out_type=tea.ALBERT_FP32), dict(rows=32)):
        assert f(P, P, **kw) == CONFIG
    assert f(P, P + 126) == CONFIG and f(P, P + 3 * 128 + 126) == CONFIG and f(P + 3 * 96 + 94, P) == CONFIG
    ok = [f(P, P + 4 * 128), f(P + 3 * 96 + 96, P),                         # one behind the other
          f(P, P + 128, ld_x=200, ld_out=200), f(P + 96, P, ld_x=200, ld_out=200),  # columns of one buffer
          f(P, P, rows=33), f(None, P)]                                     # quantized first; 4-bit rows
    assert CONFIG not in ok, ok
    assert f(P, P + 126, ld_x=200, ld_out=200) == CONFIG                   # its columns, one too many
    assert f(P, P + 128, ld_x=200, ld_out=112) == CONFIG                   # (strides apart: some pair of rows meets)


def test_status_is_asked_on_the_streams_device(monkeypatch):
    import contextlib
    import types

    import torch
    log = []

    @contextlib.contextmanager
    def device(d):
        log.append(("on", str(d)))
        yield
        log.append(("off", str(d)))

    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(tea, "lib", lambda: types.SimpleNamespace(albert_mx4_get_status=lambda s: log.append(("ask", s)) or 8))
    stream = types.SimpleNamespace(device=torch.device("cuda", 3), cuda_stream=77)
    assert tea.mx4_status(stream) == 8
    assert log == [("on", "cuda:3"), ("ask", 77), ("off", "cuda:3")]


def test_bench_knows_the_4_bit_kernels_classes():
    import bench
    for cls in ("quant_mx4", "layer_norm_mx4"):
        assert bench.source_set(cls) == "mx4_rows" and bench.sources_digest(cls) != bench.sources_digest("attention")
    assert bench.PRODUCT_RATE["mxfp4"] == bench.PRODUCT_RATE["nvfp4"] == (4.0, "E2M1")
