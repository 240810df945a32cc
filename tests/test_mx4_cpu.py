"""Microscaled 4-bit rows without a GPU: the oracle against the formats' definitions,
the storage sizes, and the refusals of every entry (host checks return before any
CUDA call; the Python wrappers refuse tensors they must not pass on)."""
import ctypes as C
import os
import re

import numpy as np
import pytest
import torch

import transformer_encoder_albert_b200 as tea
from oracle import mx4_quant as mq
from transformer_encoder_albert_b200 import build as tea_build

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "albert.h")
FMTS = ["mxfp4", "nvfp4"]
P = 4096  # a non-NULL, aligned pointer value that the host checks never dereference


@pytest.fixture(scope="module")
def lib():
    tea_build.build()
    return tea.lib()


# ---------------------------------------------------------------- the oracle --

def test_e2m1_rounding_is_nearest_even_on_every_midpoint():
    for lo, hi in zip(mq.GRID[:-1], mq.GRID[1:]):
        mid = (lo + hi) / 2
        below, above = mq.GRID[mq.e2m1_codes([np.nextafter(mid, 0)])], mq.GRID[mq.e2m1_codes([np.nextafter(mid, 9)])]
        assert below[0] == lo and above[0] == hi
        tie = int(mq.e2m1_codes([mid])[0])
        assert mq.GRID[tie] in (lo, hi) and tie % 2 == 0
    np.testing.assert_array_equal(mq.e2m1_codes([7.0, 1e30, -7.0, -0.0]), [7, 7, 15, 8])


def test_scales_follow_the_definitions():
    assert list(mq.scale_bytes([0, 1, 6, 8, 2.0 ** -125, 1e-45, np.inf, np.nan], "mxfp4")) == \
        [0, 125, 127, 128, 0, 0, 255, 255]
    g = mq.e4m3_grid()
    assert g[126] == 448 and g[1] == 2.0 ** -9 and np.all(np.diff(g) > 0)
    assert list(mq.scale_bytes([6.0, 6 * 448, 1e9, 0, np.inf], "nvfp4")) == [56, 126, 126, 0, 127]


@pytest.mark.parametrize("fmt", FMTS)
def test_rounding_error_is_bounded_by_the_block_scale(fmt):
    x = np.random.default_rng(1).normal(0, 3, (7, 100)).astype(np.float32)
    ts = 0.01
    c, b = mq.quantize(x, fmt, ts)
    v = mq.values(c, b, fmt, ts, 100)
    s = mq.scale_values(b, fmt) * (ts if fmt == "nvfp4" else 1)
    s = np.repeat(s, mq.BLOCK[fmt], axis=1)[:, :100]
    # the widest step is 2 (between 4 and 6); mxfp4 clips 8 to 6, nvfp4 rounds its scale by 1/16
    assert np.all(np.abs(v - x) <= s * (2.0 if fmt == "mxfp4" else 1.5))
    p, t = mq.pack(c, b, fmt)
    c2, b2 = mq.unpack(p, t, 7, 100, fmt)
    np.testing.assert_array_equal(c, c2)
    np.testing.assert_array_equal(b, b2)


# ------------------------------------------------------------------ storage --

@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 768), (128, 256), (129, 257), (5, 1000), (300, 32)])
@pytest.mark.parametrize("fmt", FMTS)
def test_storage_sizes_agree(lib, fmt, rows, cols):
    c, b = mq.quantize(np.zeros((rows, cols), np.float32), fmt)
    p, t = mq.pack(c, b, fmt)
    assert tea.mx4_shapes(rows, cols, fmt) == (p.shape, t.shape)
    assert lib.albert_mx4_codes_bytes(rows, cols) == p.size
    assert lib.albert_mx4_scales_bytes(rows, cols, tea.MX4_FORMATS[fmt]) == t.size
    ws = lib.albert_mx4_linear_workspace_bytes(rows, cols, tea.MX4_FORMATS[fmt])
    assert (ws == 0) == (rows <= tea._MX4_MAX_TOKENS) and (ws == 0 or ws >= p.size + t.size)


def test_storage_sizes_of_invalid_shapes_are_zero(lib):
    for rows, cols in ((0, 4), (-1, 4), (4, 0), (4, (1 << 24) + 1)):
        assert lib.albert_mx4_codes_bytes(rows, cols) == 0
        assert lib.albert_mx4_scales_bytes(rows, cols, tea.ALBERT_MXFP4) == 0
    assert lib.albert_mx4_scales_bytes(4, 4, 0) == 0


def test_linear_args_struct_matches_header_field_order():
    with open(HEADER) as f:
        body = re.search(r"typedef struct \{([^}]*)\} albert_mx4_linear_args;", f.read(), re.S).group(1)
    body = re.sub(r"/\*.*?\*/", "", body, flags=re.S)
    names = [n for decl in body.split(";") for n in re.findall(r"\b(\w+)\s*(?:,|$)", decl.strip())]
    assert names == [f for f, _ in tea.albert_mx4_linear_args._fields_]


# ----------------------------------------------------------------- refusals --

NULL, CONFIG, SHAPE = 1, 2, 3


def test_quantize_and_dequantize_refuse_on_the_host(lib):
    def q(x=P, typ=0, ld=64, rows=4, cols=64, fmt=3, ts=1.0, codes=P, scales=P):
        return lib.albert_mx4_quantize(x, typ, ld, rows, cols, fmt, ts, codes, scales, None)

    def d(codes=P, scales=P, rows=4, cols=64, fmt=3, ts=1.0, out=P, typ=0, ld=64):
        return lib.albert_mx4_dequantize(codes, scales, rows, cols, fmt, ts, out, typ, ld, None)

    for f in (q, d):
        assert f(codes=None) == NULL and f(scales=None) == NULL
        assert f(rows=-1) == SHAPE and f(cols=0) == SHAPE and f(ld=63) == SHAPE and f(cols=(1 << 24) + 1) == SHAPE
        assert f(fmt=0) == CONFIG and f(fmt=5) == CONFIG and f(typ=2) == CONFIG
        for ts in (0.0, -1.0, float("nan"), float("inf"), 2.0 ** -101):
            assert f(fmt=4, ts=ts) == CONFIG, ts
        assert f(codes=P + 8) == CONFIG and f(scales=P + 4) == CONFIG
        assert f(rows=0) == 0
    assert q(x=None) == NULL and q(x=P + 1) == CONFIG and q(x=P + 2, typ=1) == CONFIG
    assert d(out=None) == NULL and d(out=P + 1) == CONFIG


def test_layer_norm_refuses_on_the_host(lib):
    def n(x=P, typ=0, ld=64, g=P, b=P, eps=1e-12, rows=4, cols=64, fmt=3, ts=1.0, y=P, ldy=64, codes=P, scales=P):
        return lib.albert_mx4_layer_norm(x, typ, ld, g, b, eps, rows, cols, fmt, ts, y, ldy, codes, scales, None)

    for kw in ({"x": None}, {"g": None}, {"b": None}, {"codes": None}, {"scales": None}):
        assert n(**kw) == NULL, kw
    for kw in ({"rows": -1}, {"cols": 0}, {"ld": 63}, {"ldy": 63}):
        assert n(**kw) == SHAPE, kw
    for kw in ({"eps": -1.0}, {"eps": float("nan")}, {"eps": float("inf")}, {"fmt": 1}, {"typ": 9}, {"y": P + 1},
               {"g": P + 2}, {"fmt": 4, "ts": 0.0}, {"codes": P + 2}):
        assert n(**kw) == CONFIG, kw
    assert n(rows=0) == 0


def _args(**kw):
    a = tea.albert_mx4_linear_args()
    base = dict(a_codes=P, a_scales=P, w_codes=P, w_scales=P, out=P, ld_out=48, x_scale=1.0, w_scale=1.0, q_scale=1.0,
                rows=4, n=48, k=64, fmt=3)
    for k, v in {**base, **kw}.items():
        setattr(a, k, v)
    return a


def test_linear_refuses_on_the_host(lib):
    def f(**kw):
        return lib.albert_mx4_linear(C.byref(_args(**kw)), None)

    assert lib.albert_mx4_linear(None, None) == NULL
    for kw in ({"w_codes": None}, {"w_scales": None}, {"a_codes": None}, {"a_scales": None}, {"out": None},
               {"out": None, "q_codes": P}, {"rows": 4000, "x": P, "ld_x": 64}):
        assert f(**kw) == NULL, kw
    for kw in ({"rows": -1}, {"rows": (1 << 30) + 1}, {"n": 0}, {"k": 0}, {"ld_out": 47}, {"residual": P, "ld_residual": 47},
               {"x": P, "ld_x": 63, "workspace": P}):
        assert f(**kw) == SHAPE, kw
    for kw in ({"fmt": 0}, {"out_type": 7}, {"x": P, "ld_x": 64, "x_type": 7, "workspace": P}, {"gelu": 2},
               {"w_codes": P + 8}, {"w_scales": P + 8}, {"a_codes": P + 8}, {"bias": P + 2}, {"out": P + 1},
               {"residual": P + 1, "ld_residual": 48}, {"fmt": 4, "w_scale": 0.0}, {"fmt": 4, "x_scale": float("nan")},
               {"fmt": 4, "x_scale": 2.0 ** 60, "w_scale": 2.0 ** 60}, {"fmt": 4, "x_scale": 2.0 ** -60, "w_scale": 2.0 ** -60},
               {"out": None, "q_codes": P + 4, "q_scales": P}, {"fmt": 4, "out": None, "q_codes": P, "q_scales": P, "q_scale": -1.0}):
        assert f(**kw) == CONFIG, kw
    assert f(rows=0) == 0


def test_python_wrappers_refuse_what_the_library_cannot_see():
    x = torch.zeros(4, 64)
    with pytest.raises(ValueError):
        tea.mx4_quantize(x)                                   # not on a GPU
    c, s = (torch.zeros(sh, dtype=torch.uint8) for sh in tea.mx4_shapes(4, 64, "mxfp4"))
    tea.Mx4Tensor(c, s, 4, 64)
    with pytest.raises(ValueError):
        tea.Mx4Tensor(c, s, 5, 64)
    with pytest.raises(ValueError):
        tea.Mx4Tensor(c.float(), s, 4, 64)
    with pytest.raises(ValueError):
        tea.Mx4Tensor(c, s, 4, 64, "fp4")
    with pytest.raises(ValueError):
        tea.Mx4Tensor(c, s[:, :1], 4, 64)
    n = tea.mx4_shapes(4, 64, "nvfp4")
    with pytest.raises(ValueError):
        tea.Mx4Tensor(torch.zeros(n[0], dtype=torch.uint8), torch.zeros(n[1], dtype=torch.uint8), 4, 64, "nvfp4", 0.0)
    with pytest.raises(ValueError):
        tea.mx4_linear(tea.Mx4Tensor(c, s, 4, 64), tea.Mx4Tensor(c, s, 4, 64))   # not on a GPU
    for bad in ((-1, 4), (4, 0), (4, (1 << 24) + 1)):
        with pytest.raises(ValueError):
            tea.mx4_shapes(*bad, "mxfp4")
