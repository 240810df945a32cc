"""The encoder with its layer products on microscaled 4-bit operands (dtypes "mxfp4"
and "nvfp4"): against a plain 64-bit form of the same quantized layer, against the
full-precision encoder, and through every entry of the handle."""
import numpy as np
import pytest
import torch

import oracle
import synth
import transformer_encoder_albert_b200 as tea
from oracle import mx4_quant as mq
from parity_util import record_parity

pytestmark = pytest.mark.gpu
A = synth.ARCH
FMTS = ["mxfp4", "nvfp4"]
ACT = 0.03125  # nvfp4: tensor scale of the activations (albert.h)


@pytest.fixture(scope="module")
def w_bf16():
    return synth.make_weights(seed=1234, bf16=True)


def _bf(x):
    return synth.bf16_round(np.asarray(x, np.float32)).astype(np.float64)


def _mx4_weights(w, fmt):
    """64-bit values of the 4-bit layer matrices (an nvfp4 matrix's tensor scale is its
    largest magnitude over 6 * 448)."""
    mats = {"qkv": np.concatenate([w["wq"], w["wk"], w["wv"]]), "wo": w["wo"], "w1": w["w1"], "w2": w["w2"]}
    out = {}
    for k, m in mats.items():
        m = np.asarray(m, np.float32)
        ts = np.float32(np.abs(m).max()) / np.float32(6 * 448) if fmt == "nvfp4" else 1.0
        out[k] = mq.rounded(m, fmt, ts)
    return out


def _plain(w, q, fmt, E, n_exec, out_dim=True, norms=None):
    """One sequence from its post-embedding-LayerNorm rows E, in 64 bits with the layer's
    rounding points: 4-bit operands, bf16 rows between the kernels."""
    f32 = lambda x: np.asarray(x, np.float32)  # noqa: E731
    q4 = lambda x: mq.rounded(f32(x), fmt, ACT)  # noqa: E731
    mask = np.ones(E.shape[0], np.uint8)
    bqkv = np.concatenate([w["bq"], w["bk"], w["bv"]])
    x = _bf(oracle.linear(_bf(E), w["w_in"], w["b_in"]))
    x4 = q4(x)
    for _ in range(n_exec):
        qkv = _bf(x4 @ q["qkv"].T + bqkv)
        ctx = _bf(oracle.attention(qkv[:, :768], qkv[:, 768:1536], qkv[:, 1536:], mask, 12))
        z = _bf(q4(ctx) @ q["wo"].T + w["bo"] + x)
        y = y1 = oracle.layer_norm(z, w["ln1_g"], w["ln1_b"], A["ln_eps"])
        x1 = _bf(y)
        h = oracle.gelu(q4(y) @ q["w1"].T + w["b1"])
        z = _bf(q4(h) @ q["w2"].T + w["b2"] + x1)
        y = oracle.layer_norm(z, w["ln2_g"], w["ln2_b"], A["ln_eps"])
        if norms is not None:
            n = np.linalg.norm
            z1 = q4(ctx) @ q["wo"].T
            norms.update(wo=n(z1), z1=n(z1 + w["bo"] + x), w1=n(q4(y1) @ q["w1"].T), h=n(h), w2=n(q4(h) @ q["w2"].T),
                         z1n=n(x1), z2=n(z))
        x, x4 = _bf(y), q4(y)
    return oracle.linear(x, w["w_out"], w["b_out"]) if out_dim else x


def _full(w, E):
    x = oracle.linear(E, w["w_in"], w["b_in"])
    layer = oracle.Model(w, A, n_exec=1, out_dim=0)
    for _ in range(A["n_exec"]):
        x = layer.layer(x, np.ones(E.shape[0], np.uint8))
    return oracle.linear(x, w["w_out"], w["b_out"])


def _cos(a, b):
    return float(np.dot(a.ravel(), b.ravel()) / (np.linalg.norm(a) * np.linalg.norm(b)))


def _run(enc, E):
    """E: list of [T, 128] arrays."""
    cu = np.concatenate([[0], np.cumsum([e.shape[0] for e in E])]).astype(np.int32)
    out = enc.forward_embedded(torch.tensor(np.concatenate(E)).cuda(), torch.tensor(cu).cuda(),
                               max(e.shape[0] for e in E)).float().cpu().numpy()
    assert enc.status() == 0
    return [out[cu[i]:cu[i + 1]] for i in range(len(E))]


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("out_dim", [512, 0])
def test_one_layer_matches_its_plain_form(w_bf16, fmt, out_dim):
    """Both sides round at the same points but one: the attention kernel rounds its
    probabilities to bf16, so its output is off by d0 = 2^-8 (that and its own rounding).
    What a relative difference d of a row becomes on the way:
      * rounding to 4 bits: a value off by e comes out a step off with probability e / step,
        so the mean square is e * step; a step is at most the value itself (codes of one
        binade are 1/2 apart at 1, 1 at 2, 2 at 4), so the difference becomes sqrt(d);
      * a sum of terms of norms n_i and differences d_i, of norm n: sum n_i d_i / n;
      * GELU: its slope is at most 1.13; LayerNorm keeps a relative difference.
    The norms are the plain form's own.  (Probabilities, so rows of a few hundred values;
    the largest share of a one-row sequence has no attention error at all.)"""
    rng = np.random.default_rng(5)
    E = [rng.normal(0, 1, (n, 128)).astype(np.float32) for n in (128, 1, 77, 130, 200)]
    q = _mx4_weights(w_bf16, fmt)
    enc = tea.Encoder(w_bf16, A, dtype=fmt, max_tokens=1024, n_exec=1, out_dim=out_dim)
    got = _run(enc, E)
    enc.close()
    for g, e in zip(got, E):
        norms = {}
        ref = _plain(w_bf16, q, fmt, e, 1, out_dim > 0, norms)
        d = np.sqrt(2.0 ** -8) * norms["wo"] / norms["z1"] + 2.0 ** -9       # pre-norm rows, bf16
        h = 1.13 * np.sqrt(d) * norms["w1"] / norms["h"]                     # before the inner rounding
        d = (np.sqrt(h) * norms["w2"] + d * norms["z1n"]) / norms["z2"] + 2.0 ** -8
        assert d < 0.25 and np.linalg.norm(g - ref) <= d * np.linalg.norm(ref)


@pytest.mark.parametrize("fmt", FMTS)
def test_fidelity_to_the_full_precision_encoder(w_bf16, fmt):
    """Cosine and MSE on the pages' protocol for a quantized encoder (N(0,1) inputs of
    [1, 128, 128]): as good as the plain 64-bit form of the same quantization (0.01 of
    cosine for the codes that fall on another side on the way through twelve layers), and
    above the pages' quantized encoder (mean cosine 0.724)."""
    rng = np.random.default_rng(4242)
    E = [rng.normal(0, 1, (128, 128)).astype(np.float32) for _ in range(4)]
    q = _mx4_weights(w_bf16, fmt)
    enc = tea.Encoder(w_bf16, A, dtype=fmt, max_tokens=4 * 128)
    got = _run(enc, E)
    enc.close()
    cos, err = [], 0.0
    for g, e in zip(got, E):
        ref = _full(w_bf16, e)
        err = max(err, float(np.abs(g - ref).max()))
        cos.append(_cos(g, ref))
        assert cos[-1] >= _cos(_plain(w_bf16, q, fmt, e, A["n_exec"]), ref) - 0.01
    record_parity(f"pages' protocol, {fmt}: cosine mean {np.mean(cos):.5f} min {np.min(cos):.5f}", 4, 512, err,
                  float(np.min(cos)), "abs")
    assert np.mean(cos) > 0.724


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("name", ["b8_T128", "b32_T512_long"])
def test_entries_agree(w_bf16, fmt, name):
    """Padded, packed and host-buffer entries give the same rows; padding rows are 0; a
    captured and replayed forward gives the same again."""
    wl = synth.WORKLOADS[name]
    ids, mask, L = synth.make_batch(wl)
    n = min(wl.B, 6)
    ids, mask, L = ids[:n], mask[:n], L[:n]
    enc = tea.Encoder(w_bf16, A, dtype=fmt, max_tokens=n * wl.T)
    di, dm = torch.as_tensor(ids).cuda(), torch.as_tensor(mask).cuda()
    padded = enc.forward(di, dm)
    assert enc.status() == 0
    launches = enc.last_forward_launches()
    assert launches == enc.launches_per_forward(padded_api=True)
    packed = np.concatenate([ids[b, :L[b]] for b in range(n)])
    cu = np.concatenate([[0], np.cumsum(L)]).astype(np.int32)
    out = enc.forward_varlen(torch.as_tensor(packed).cuda(), torch.as_tensor(cu).cuda(), int(L.max()))
    assert enc.status() == 0
    host = torch.empty(n, wl.T, A["out_dim"], dtype=torch.bfloat16)
    assert enc.forward_host(torch.as_tensor(ids), torch.as_tensor(mask), host) == 0
    p, o = padded.float().cpu().numpy(), out.float().cpu().numpy()
    np.testing.assert_array_equal(host.float().numpy(), p)
    for b in range(n):
        np.testing.assert_array_equal(o[cu[b]:cu[b + 1]], p[b, :L[b]])
        assert np.all(p[b, L[b]:] == 0)
    g, buf = torch.cuda.CUDAGraph(), torch.empty_like(padded)
    with torch.cuda.graph(g):
        enc.forward(di, dm, out=buf)
    buf.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(buf, padded) and enc.status() == 0
    del g
    enc.close()


@pytest.mark.parametrize("fmt", FMTS)
def test_grouped_weights_and_transposed_output(fmt):
    """Two weight sets, one execution each, [B, D, T] output, against the full-precision
    encoder (two layers of 4-bit products: cosine 0.95 at the least)."""
    ws = [synth.make_weights(seed=7 + i, bf16=True) for i in range(2)]
    stacked = {k: (np.stack([w[k] for w in ws]) if k in oracle.LAYER_PARAMS else ws[0][k]) for k in ws[0]}
    wl = synth.Workload("g", 3, 40, "uniform", lo=7, hi=40, seed=5)
    ids, mask, L = synth.make_batch(wl)
    enc = tea.Encoder(stacked, A, dtype=fmt, max_tokens=wl.B * wl.T, n_exec=2, n_groups=2, out_layout=1)
    out = enc.forward(torch.as_tensor(ids).cuda(), torch.as_tensor(mask).cuda()).float().cpu().numpy()
    assert enc.status() == 0
    enc.close()
    for b in range(wl.B):
        n = int(L[b])
        ref = oracle.encode_grouped(stacked, A, ids[b], mask[b], 2, n_exec=2)[:n]
        assert _cos(out[b, :, :n].T, ref) >= 0.95
        assert np.all(out[b, :, n:] == 0)


@pytest.mark.parametrize("cls", ["gemm_qkv", "gemm_out_proj_ln", "gemm_ffn_up_gelu", "gemm_ffn_down_ln"])
def test_expired_wait_reports_timeout_and_leaves_output_untouched(w_bf16, cls):
    wl = synth.WORKLOADS["b8_T128"]
    ids, mask, _ = synth.make_batch(wl)
    di, dm = torch.as_tensor(ids).cuda(), torch.as_tensor(mask).cuda()
    enc = tea.Encoder(w_bf16, A, dtype="mxfp4", max_tokens=wl.B * wl.T)
    good = enc.forward(di, dm)
    assert enc.status() == 0
    enc.set_wait_limit(2_000_000)
    enc.test_stall([cls])
    out = torch.full_like(good, 7.0)
    enc.forward(di, dm, out=out)
    assert enc.status() == 8  # ALBERT_ERR_TIMEOUT
    assert torch.all(out == 7.0)
    enc.test_stall([])
    enc.set_wait_limit(0)
    again = enc.forward(di, dm)
    assert enc.status() == 0 and torch.equal(again, good)
    enc.close()


def test_bad_ids_leave_the_output_untouched(w_bf16):
    wl = synth.WORKLOADS["b8_T128"]
    ids, mask, _ = synth.make_batch(wl)
    ids = ids.copy()
    ids[2, 1] = 999
    enc = tea.Encoder(w_bf16, A, dtype="nvfp4", max_tokens=wl.B * wl.T)
    out = torch.full((wl.B, wl.T, A["out_dim"]), 7.0, device="cuda", dtype=torch.bfloat16)
    enc.forward(torch.as_tensor(ids).cuda(), torch.as_tensor(mask).cuda(), out=out)
    assert enc.status() == 4
    assert torch.all(out == 7.0)
    enc.close()


@pytest.mark.parametrize("fmt", FMTS)
def test_a_4_bit_handle_takes_less_memory_than_a_bf16_one(w_bf16, fmt):
    """32768 rows: the FFN activation takes a quarter (4096 -> about 1100 bytes a row), the layer
    matrices likewise, and nothing stays in bf16 that no forward reads."""
    taken = {}
    for dtype in ("bf16", fmt):
        torch.cuda.synchronize()
        before = torch.cuda.mem_get_info()[0]
        enc = tea.Encoder(w_bf16, A, dtype=dtype, max_tokens=32768)
        torch.cuda.synchronize()
        taken[dtype] = before - torch.cuda.mem_get_info()[0]
        enc.close()
    assert taken[fmt] <= taken["bf16"] - 32768 * 2400


def _rows_of_one_layer(w, fmt, x, act):
    """A layer without attention (w["wo"] = 0) out of the operators by themselves, from its
    bf16 input rows: what the handle's kernels must give bit for bit; and its inner activation."""
    cu = lambda k: torch.tensor(np.asarray(w[k], np.float32)).cuda()  # noqa: E731

    def mat(k):
        m = np.asarray(w[k], np.float32)
        ts = float(np.float32(np.abs(m).max()) / np.float32(6 * 448)) if fmt == "nvfp4" else 1.0
        return tea.mx4_quantize(torch.tensor(m).cuda(), fmt, ts if ts >= 1e-30 else 1.0)

    a = act if fmt == "nvfp4" else 1.0
    z = tea.mx4_linear(x, mat("wo"), cu("bo"), residual=x, x_scale=a)
    x1, x4 = tea.mx4_layer_norm(z, cu("ln1_g"), cu("ln1_b"), A["ln_eps"], fmt, a)
    h = tea.mx4_linear_quant(x4, mat("w1"), cu("b1"), gelu=True, out_scale=a)
    z = tea.mx4_linear(h, mat("w2"), cu("b2"), residual=x1)
    return tea.mx4_layer_norm(z, cu("ln2_g"), cu("ln2_b"), A["ln_eps"], fmt, a)[0], h


def _without_attention(w, seed):
    rng = np.random.default_rng(seed)
    w = dict(w)
    w["wo"] = np.zeros_like(w["wo"])
    for k in ("bo", "b1", "b2", "ln1_b", "ln2_b"):
        w[k] = rng.normal(0, 0.3, w[k].shape).astype(np.float32)
    for k in ("ln1_g", "ln2_g"):
        w[k] = (1 + rng.normal(0, 0.2, w[k].shape)).astype(np.float32)
    return w


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("lengths", [(128, 128, 128, 128, 128), (64,), (1, 100, 37, 512, 260)])
def test_a_layer_is_its_operators_bit_for_bit(w_bf16, fmt, lengths):
    """The handle's LayerNorms, products, GELU and residuals against the operators' own entries on
    the same rows: equal, so that no scale, code or bias is anywhere else than there."""
    rng = np.random.default_rng(len(lengths))
    w = _without_attention(w_bf16, 3)
    rows = sum(lengths)
    E = torch.tensor(rng.normal(0, 1, (rows, 128)).astype(np.float32)).cuda()
    cu = torch.tensor(np.concatenate([[0], np.cumsum(lengths)]).astype(np.int32)).cuda()
    got = {}
    for n_exec in (0, 1):
        enc = tea.Encoder(w, A, dtype=fmt, max_tokens=rows, n_exec=n_exec, out_dim=0)
        got[n_exec] = enc.forward_embedded(E, cu, max(lengths))
        assert enc.status() == 0
        enc.close()
    assert torch.equal(got[1], _rows_of_one_layer(w, fmt, got[0], ACT)[0])


def test_the_activation_scale_of_an_nvfp4_encoder(w_bf16):
    """An FFN activation of about 300 (within the eighth and the sixteenth of E2M1's and the scale's
    half steps): cut off at 84 with the scale 1/32, kept with 1/4.  With each scale the layer is its
    operators with that scale."""
    w = _without_attention(w_bf16, 4)
    w["b1"] = w["b1"] + np.where(np.arange(w["b1"].size) % 7 == 0, 300, 0).astype(np.float32)
    E = torch.tensor(np.random.default_rng(6).normal(0, 1, (200, 128)).astype(np.float32)).cuda()
    cu = torch.tensor([0, 200], dtype=torch.int32, device="cuda")
    enc = tea.Encoder(w, A, dtype="nvfp4", max_tokens=200, n_exec=0, out_dim=0)
    x = enc.forward_embedded(E, cu, 200)
    enc.close()
    enc = tea.Encoder(w, A, dtype="nvfp4", max_tokens=200, n_exec=1, out_dim=0)
    for scale in (ACT, 0.25, ACT):
        enc.set_activation_scale(scale)
        y = enc.forward_embedded(E, cu, 200)
        out, h = _rows_of_one_layer(w, "nvfp4", x, scale)
        assert enc.status() == 0 and torch.equal(y, out)
        top = float(tea.mx4_dequantize(h, dtype=torch.float32).abs().max())
        assert top == 84 if scale == ACT else 250 < top < 350
    for bad in (0.0, -1.0, float("nan"), float("inf"), 2.0 ** -21, 2.0 ** 21):
        with pytest.raises(tea.AlbertError):
            enc.set_activation_scale(bad)
    enc.close()
    enc = tea.Encoder(w, A, dtype="mxfp4", max_tokens=64)
    with pytest.raises(tea.AlbertError):
        enc.set_activation_scale(0.25)
    enc.close()
