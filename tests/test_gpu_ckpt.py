"""GPU parity of the 8-bit activation checkpoints and the backward kernels that read them."""
import numpy as np
import pytest
import torch

from oracle import moe_oracle as O
from sparse_moe_layer_sigmoid_amd import inputs as I
from tests.gpu_common import np64, rel_err, say
from tests.test_gpu_norm import _ckpt_reference

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
U = 2.0 ** -24


def M():
    import sparse_moe_layer_sigmoid_amd as m
    return m


SHAPES = [(1, 1), (3, 7), (5, 8), (2, 127), (4, 128), (3, 129), (17, 1000), (200, 15), (9, 2049), (31, 4096), (700, 24),
          (2, 300000)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_pack_bitexact(rows, cols, dtype):
    """Codes and scale codes equal the oracle's rule; the values come back exactly, in both types; with strides."""
    say(f"pack {rows}x{cols} {dtype}")
    pad = 5
    x = I.gen_normal(200 + cols, (rows, cols + pad), 1.0, torch.float32)
    x *= torch.exp2(torch.randint(-30, 30, (rows, 1), generator=torch.Generator().manual_seed(cols)).float())
    x[0, : cols // 2] = 0.0
    xd = x.to(dtype).to(DEV)[:, :cols]
    q, s = M().fp8_ckpt_pack(xd)
    wq, ws, wv = _ckpt_reference(np64(xd))
    assert np.array_equal(s.cpu().numpy(), ws)
    assert np.array_equal(q.cpu().numpy(), wq)
    for out in (torch.float32, torch.bfloat16):
        assert np.array_equal(np64(M().fp8_ckpt_unpack(q, s, out_dtype=out)), wv)


def test_pack_matches_the_e8m0_quantiser():
    x = I.gen_normal(240, (65, 512), 3.0).to(DEV)
    q, s = M().fp8_ckpt_pack(x)
    q2, s2 = M().fp8_quant_1x128_e8m0(x)
    assert torch.equal(q, q2) and torch.equal(s, s2)


def test_pack_special_values():
    """Midpoints, subnormal tiles, the scale rule at its edge, infinities and NaN inside one tile."""
    t = np.zeros((8, 128), dtype=np.float32)
    t[0] = np.linspace(-448, 448, 128)
    t[1, :4] = [448.0, 1.0625, 1.1875, -1.0625]            # ties between codes go to the even one
    t[2, :3] = [np.nextafter(np.float32(448), np.float32(500)), 1.0, -2.0 ** -9]
    t[3, :3] = [1e-38, -3e-39, 1e-45]                      # subnormal f32
    t[4, :3] = [3.4028234663852886e38, 1.0, -1e30]
    t[5] = -0.0
    t[6, :2] = [2.0 ** -9, 448.0]
    t[7, 100] = 7.0
    q, s = M().fp8_ckpt_pack(torch.from_numpy(t).to(DEV))
    wq, ws, wv = _ckpt_reference(t.astype(np.float64))
    assert np.array_equal(s.cpu().numpy(), ws) and np.array_equal(q.cpu().numpy(), wq)
    # the largest f32 is 255.99998 * 2^120: its code is that of 256, whose value 2^128 an f32 output holds as infinity
    with np.errstate(over="ignore"):
        wv = wv.astype(np.float32)
    assert np.isinf(wv).sum() == 1 and np.isinf(wv[4, 0])
    assert np.array_equal(np64(M().fp8_ckpt_unpack(q, s, out_dtype=torch.float32)), wv)
    bad = t[:3].copy()
    bad[0, 5], bad[1, 7], bad[2, 9] = np.inf, np.nan, -np.inf
    bad[2, 10] = np.nan
    for dt in (torch.float32, torch.bfloat16):
        q, s = M().fp8_ckpt_pack(torch.from_numpy(bad).to(dt).to(DEV))
        v = M().fp8_ckpt_unpack(q, s, out_dtype=torch.float32).cpu().numpy()
        assert v[0, 5] == np.inf and np.isfinite(np.delete(v[0], 5)).all()
        assert v[2, 9] == -np.inf and np.isnan(v[2, 10]) and np.isnan(v[1, 7])
        # NaN alone does not change the others' scale
        ref = torch.from_numpy(t[1:2]).to(dt).to(DEV)
        assert np.array_equal(np.delete(v[1], 7), np.delete(np64(M().fp8_ckpt_unpack(*M().fp8_ckpt_pack(ref)))[0], 7))


def test_every_code_and_scale():
    """All 256 codes under all 255 scale codes decode to code * 2^(scale - 127), rounded once to the output."""
    q = torch.arange(256, dtype=torch.uint8).repeat(255, 1)
    s = torch.arange(255, dtype=torch.uint8)[:, None].repeat(1, 2)
    got = M().fp8_ckpt_unpack(q.to(DEV), s.to(DEV), out_dtype=torch.float32).cpu().numpy()
    v = O.e4m3_decode(q.numpy().astype(np.uint8)) * np.exp2(np.arange(255.0) - 127)[:, None]
    with np.errstate(over="ignore"):
        want = v.astype(np.float32)
    nan = np.isnan(v)
    assert np.array_equal(np.isnan(got), nan) and np.array_equal(got[~nan], want[~nan])


def test_every_code_and_scale_in_bf16():
    """The same in bf16: one rounding to nearest even of the f32 value, and none for scales of 2^-124 or more whose value
    stays below 2^128."""
    q = torch.arange(256, dtype=torch.uint8).repeat(255, 1)
    s = torch.arange(255, dtype=torch.uint8)[:, None].repeat(1, 2)
    got = M().fp8_ckpt_unpack(q.to(DEV), s.to(DEV)).cpu()
    v = O.e4m3_decode(q.numpy().astype(np.uint8)) * np.exp2(np.arange(255.0) - 127)[:, None]
    with np.errstate(over="ignore"):
        want = torch.from_numpy(v.astype(np.float32)).to(torch.bfloat16)
    nan = torch.from_numpy(np.isnan(v))
    assert torch.equal(torch.isnan(got), nan)
    assert torch.equal(got.view(torch.int16)[~nan], want.view(torch.int16)[~nan])
    exact = (~np.isnan(v)) & (np.abs(v) < 2.0 ** 128) & (np.arange(255) >= 3)[:, None]
    assert np.array_equal(got.double().numpy()[exact], v[exact])
    assert not np.array_equal(got.double().numpy()[:3][~np.isnan(v[:3])], v[:3][~np.isnan(v[:3])])


@pytest.mark.parametrize("cols", [1, 9, 128, 1001, 2048])
def test_unpack_affine(cols):
    """v * w + b rounded once each in fp32: two half steps, then bf16's."""
    x = I.gen_normal(250, (13, cols), 1.0).to(DEV)
    ck = M().fp8_ckpt_pack(x)
    v = np64(M().fp8_ckpt_unpack(*ck, out_dtype=torch.float32))
    for wt in (torch.bfloat16, torch.float32):
        w, b = I.gen_normal(251, (cols,), 1.0, wt).to(DEV), I.gen_normal(252, (cols,), 1.0, wt).to(DEV)
        for out, half in ((torch.float32, 0.0), (torch.bfloat16, 2.0 ** -8)):
            for ww, bb in ((w, b), (w, None), (None, b)):
                p = v * (np64(ww) if ww is not None else 1.0)
                want = p + (np64(bb) if bb is not None else 0.0)
                got = np64(M().fp8_ckpt_unpack(*ck, weight=ww, bias=bb, out_dtype=out))
                assert np.all(np.abs(got - want) <= U * (np.abs(p) + np.abs(want)) * 1.001 + half * np.abs(want) + 1e-30)


@pytest.mark.parametrize("rows,inter", [(1, 4), (1, 8), (3, 12), (5, 64), (7, 68), (33, 128), (2, 132), (9, 200), (65, 2048),
                                        (1, 16384)])
def test_swiglu_backward_ckpt(rows, inter):
    """Against float64 on the checkpoint's own values.  The device's sigmoid is off by a relative (|a| + 4) u (the
    product with log2 e, exp2 and the reciprocal, one step each); a product of four factors adds 4 u; bf16 half a step."""
    say(f"swiglu_backward_ckpt {rows}x{inter}")
    ac = (I.gen_normal(260 + inter, (rows, 2 * inter), 1.5, torch.float32)).to(DEV)
    dh = I.gen_normal(261, (rows, inter), 0.3, torch.float32).to(DEV)
    q, s = M().fp8_ckpt_pack(ac)
    v = np64(M().fp8_ckpt_unpack(q, s, out_dtype=torch.float32))
    dac, h = M().moe_swiglu_backward_ckpt(q, s, dh)
    a, c, g = v[:, :inter], v[:, inter:], np64(dh)
    sg = 1.0 / (1.0 + np.exp(-a))
    rel = (2 * np.abs(a) + 16) * U
    da, dc, hh = g * c * sg * (1 + a * (1 - sg)), g * a * sg, a * sg * c
    tda = np.abs(g * c * sg) * (1 + np.abs(a)) * rel * 4 + 2.0 ** -8 * np.abs(da)
    got = np64(dac)
    assert np.all(np.abs(got[:, :inter] - da) <= tda + 1e-38)
    assert np.all(np.abs(got[:, inter:] - dc) <= np.abs(dc) * (2.0 ** -8 + rel * 1.01) + 1e-38)
    assert np.all(np.abs(np64(h) - hh) <= np.abs(hh) * (2.0 ** -8 + rel * 1.01) + 1e-38)
    dac2, none = M().moe_swiglu_backward_ckpt(q, s, dh, want_h=False)
    assert none is None and torch.equal(dac, dac2)
    # the same gradient as from f32 a | c that hold the checkpoint's values
    if inter % 4 == 0:
        ref = M()._lib.moe_swiglu_backward(M().fp8_ckpt_unpack(q, s, out_dtype=torch.float32), dh)
        assert rel_err(np64(dac), np64(ref)) <= 2.0 ** -7
    if inter % 128 == 0:
        d3, dq, ds, h3 = M().moe_swiglu_backward_ckpt(q, s, dh, fp8=True)
        assert torch.equal(d3, dac) and torch.equal(h3, h)
        wq, ws = O.quant_1x128(dac.float().cpu().numpy())
        assert np.array_equal(dq.cpu().numpy(), wq) and np.array_equal(ds.cpu().numpy(), ws)


def test_swiglu_backward_ckpt_extremes():
    """Saturated gates: silu'(a) tends to 1 and to 0 without NaN; zero rows stay zero."""
    a = torch.tensor([[-100.0, 100.0, 0.0, -30.0, 30.0, 1.0, -1.0, 0.5]])
    ac = torch.cat([a, torch.ones_like(a)], 1).to(DEV)
    dac, h = M().moe_swiglu_backward_ckpt(*M().fp8_ckpt_pack(ac), torch.ones((1, 8), device=DEV))
    assert torch.isfinite(dac).all() and torch.isfinite(h).all()
    v = np64(M().fp8_ckpt_unpack(*M().fp8_ckpt_pack(ac), out_dtype=torch.float32))[:, :8]
    assert np.allclose(np64(h), v / (1 + np.exp(-v)), rtol=2.0 ** -8, atol=1e-30)
    z = torch.zeros((3, 16), device=DEV)
    dac, h = M().moe_swiglu_backward_ckpt(*M().fp8_ckpt_pack(z), torch.ones((3, 8), device=DEV))
    assert not dac.any() and not h.any()
    e = torch.empty((0, 16), device=DEV)
    dac, h = M().moe_swiglu_backward_ckpt(*M().fp8_ckpt_pack(e), torch.empty((0, 8), device=DEV))
    assert dac.shape == (0, 16) and h.shape == (0, 8)


def _route(seed, T, K, N):
    idx, gate = I.gen_routing(seed, T, K, N)
    scores = torch.from_numpy(np.random.default_rng(seed).uniform(0.05, 0.95, (T, N)).astype(np.float32))
    return idx.to(DEV), gate.to(DEV), scores.to(DEV)


@pytest.mark.parametrize("T,K,N,d", [(1, 1, 4, 8), (5, 2, 8, 40), (33, 8, 16, 128), (7, 9, 16, 520), (3, 32, 40, 136),
                                     (64, 8, 256, 7168), (2, 4, 8, 2056)])
def test_combine_backward_ckpt(T, K, N, d):
    """dy as moe_combine_backward gives it, bit for bit; du within the fp32 sums' bound of float64: dg is a sum of at
    most 8 d / 448 + 6 + 8 roundings, du combines K + 1 of them."""
    say(f"combine_backward_ckpt T={T} K={K} N={N} d={d}")
    idx, gate, scores = _route(300 + d, T, K, N)
    _, _, pp = M().moe_permute(idx, N, 1)
    y = I.gen_normal(301, (T * K, d), 0.2).to(DEV)
    d_out = I.gen_normal(302, (T, d), 1.0).to(DEV)
    q, s = M().fp8_ckpt_pack(y)
    yv = M().fp8_ckpt_unpack(q, s)
    dy, du, du_row = M().moe_combine_backward_ckpt(d_out, q, s, idx, gate, scores, pp)
    dy0, du0, _ = M()._lib.moe_combine_backward(d_out, yv, idx, gate, scores, pp)
    assert torch.equal(dy, dy0)
    p = pp.cpu().numpy()
    y64, o64, g64 = np64(yv), np64(d_out), np64(gate)
    prod = y64[p] * o64[:, None, :]
    dg, adg = prod.sum(2), np.abs(prod).sum(2)
    sv = np.take_along_axis(np64(scores), idx.cpu().numpy().astype(np.int64), 1)
    S = sv.sum(1, keepdims=True)
    f = sv * (1 - sv) / S
    want = f * (dg - (g64 * dg).sum(1, keepdims=True))
    n = 8 * -(-d // 448) + 8 * -(-d // 8 // 64) / 8 + 14
    tol = f * (n * U * (adg + (g64 * adg).sum(1, keepdims=True))) + f * (K + 12) * U * (np.abs(dg) + (g64 * np.abs(dg)).sum(1, keepdims=True))
    assert np.all(np.abs(np64(du) - want) <= tol + 1e-30)
    assert np.array_equal(np64(du_row)[p], np64(du))
    if d % 128 == 0:
        out = M().moe_combine_backward_ckpt(d_out, q, s, idx, gate, scores, pp, fp8=True)
        ref = M()._lib.moe_combine_backward(d_out, yv, idx, gate, scores, pp, fp8=True)
        assert torch.equal(out[0], dy) and torch.equal(out[3], ref[3]) and torch.equal(out[4], ref[4])
        assert torch.equal(out[1], du)


def test_combine_backward_ckpt_skipped_pair():
    """A pair the permutation skips carries nothing: its du is 0 and no row of dy is written for it."""
    T, K, N, d = 4, 3, 8, 64
    idx = torch.tensor([[1, 4, 6], [0, -1, 3], [2, 5, 7], [7, 9, 0]], dtype=torch.int32, device=DEV)
    gate = torch.full((T, K), 1 / 3, device=DEV)
    scores = torch.full((T, N), 0.4, device=DEV)
    _, _, pp = M().moe_permute(idx, N, 1)
    y = I.gen_normal(310, (T * K, d), 1.0).to(DEV)
    q, s = M().fp8_ckpt_pack(y)
    d_out = I.gen_normal(311, (T, d), 1.0).to(DEV)
    dy, du, du_row = M().moe_combine_backward_ckpt(d_out, q, s, idx, gate, scores, pp)
    dy0, du0, _ = M()._lib.moe_combine_backward(d_out, M().fp8_ckpt_unpack(q, s), idx, gate, scores, pp)
    assert float(du[1, 1]) == 0.0 and float(du[3, 1]) == 0.0
    assert torch.allclose(du, du0, rtol=1e-5, atol=1e-6)
    used = pp.flatten()[pp.flatten() >= 0].long()
    assert torch.equal(dy[used], dy0[used]) and torch.equal(dy[T * K:], d_out)


def _layer(fp8, norm, T=160, d=256, N=16, K=4, Inter=128, seed=7):
    cfg = I.small(I.V3_BF16, name="ckpt_layer", T=T, d=d, n_experts=N, top_k=K, inter=Inter, w_std=0.05, router_std=0.05,
                  seed=seed)
    ex = [I.gen_expert(cfg, e) for e in range(cfg.groups)]
    W13 = torch.stack([a for a, _ in ex]).to(torch.bfloat16).to(DEV)
    W2 = torch.stack([b for _, b in ex]).to(torch.bfloat16).to(DEV)
    nw = (1.0 + I.gen_normal(seed + 1, (d,), 0.1, torch.float32)).to(DEV) if norm else None
    nb = I.gen_normal(seed + 2, (d,), 0.1, torch.float32).to(DEV) if norm == "layer" else None
    layer = M().MoELayer(I.gen_router(cfg).to(DEV), W13, W2, I.gen_bias(cfg).to(DEV), K, fp8=fp8, norm=norm, norm_weight=nw,
                         norm_bias=nb)
    return cfg, layer, I.gen_x(cfg).to(DEV), I.gen_normal(seed + 3, (T, d), 1.0).to(DEV)


@pytest.mark.parametrize("norm", [None, "rms", "layer"])
@pytest.mark.parametrize("fp8", [False, True])
def test_layer_checkpointed_training_step(fp8, norm):
    """forward(checkpoint=True) and its backward, end to end: the output is that of the plain forward bit for bit; the
    backward equals the plain backward run on what the checkpoints stand for (the same kernels on the same values, so
    up to the order of one fp32 sum, 2^-7 after the bf16 roundings that follow); against the exact gradients, in
    the 2-norm: an E4M3 rounding is uniform within 2^-4 of a value, 3.6% in the root mean square, and at most four
    independent ones meet in a product (x, a, c and the FP8 path's operand): 7.2%, so 8% with the bf16 roundings."""
    # the FP8 backward's GEMMs take widths in multiples of 256
    cfg, layer, x, d_out = _layer(fp8, norm, Inter=256 if fp8 else 128)
    out0, buf0 = layer.forward(x, train=True)
    out, buf = layer.forward(x, checkpoint=True)
    assert torch.equal(out, out0)
    assert buf["ac"] is None and buf["y"] is None and buf["x"] is None
    g0 = layer.backward(d_out, buf0)
    g = layer.backward(d_out, buf)
    names = ["dx", "dw_router", "dw13", "dw2"] + (["dnorm_weight"] if norm else []) + (["dnorm_bias"] if norm == "layer" else [])
    # what the checkpoints stand for, through the plain backward
    L = M()
    u = layer._checkpointed_x(buf)
    ac = L.fp8_ckpt_unpack(*buf["ac_ckpt"], out_dtype=torch.float32)
    rep = dict(buf0, x=u, y=L.fp8_ckpt_unpack(*buf["y_ckpt"]), ac=ac, checkpoint=False)
    if not fp8:
        rep["h"] = L.moe_swiglu_backward_ckpt(*buf["ac_ckpt"], torch.zeros((ac.shape[0], ac.shape[1] // 2), device=DEV))[1]
    if norm:
        rep["norm"] = buf["norm"]
    gr = layer.backward(d_out, rep)
    for n in names:
        say(f"  fp8={fp8} norm={norm} {n}: vs the checkpoints' values {rel_err(np64(g[n]), np64(gr[n])):.2e}")
        assert rel_err(np64(g[n]), np64(gr[n])) <= 2.0 ** -7 if not fp8 else rel_err(np64(g[n]), np64(gr[n])) <= 2.0 ** -4
        e, r = np64(g[n]) - np64(g0[n]), np64(g0[n])
        off = np.sqrt((e * e).sum() / (r * r).sum())
        say(f"    vs the plain step {off:.2e}")
        assert off <= 0.08, n


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("T", [1, 3])
def test_layer_checkpointed_few_tokens(fp8, T):
    """A checkpointed step of fewer tokens than experts, most experts without rows, against the plain backward run on
    what the checkpoints stand for, with the tolerances of the larger step; an expert without rows has a zero gradient."""
    cfg, layer, x, d_out = _layer(fp8, "rms", T=T, Inter=256 if fp8 else 128)
    out0, buf0 = layer.forward(x, train=True)
    out, buf = layer.forward(x, checkpoint=True)
    assert torch.equal(out, out0)
    ac = M().fp8_ckpt_unpack(*buf["ac_ckpt"], out_dtype=torch.float32)
    rep = dict(buf0, x=layer._checkpointed_x(buf), y=M().fp8_ckpt_unpack(*buf["y_ckpt"]), ac=ac, checkpoint=False,
               norm=buf["norm"])
    if not fp8:
        rep["h"] = M().moe_swiglu_backward_ckpt(*buf["ac_ckpt"], torch.zeros((ac.shape[0], ac.shape[1] // 2), device=DEV))[1]
    g, gr = layer.backward(d_out, buf), layer.backward(d_out, rep)
    for n in ("dx", "dw_router", "dw13", "dw2", "dnorm_weight"):
        say(f"  T={T} fp8={fp8} {n}: vs the checkpoints' values {rel_err(np64(g[n]), np64(gr[n])):.2e}")
        assert rel_err(np64(g[n]), np64(gr[n])) <= (2.0 ** -4 if fp8 else 2.0 ** -7), n
    empty = torch.nonzero(buf["expert_counts"] == 0).flatten()
    assert empty.numel() > 0 and not bool(g["dw13"][empty].any()) and not bool(g["dw2"][empty].any())


@pytest.mark.parametrize("norm", ["rms", "layer"])
def test_layer_with_norm_against_float64(norm):
    """The layer with a norm: the forward equals the layer on the norm's output, and the gradient of the rows before it
    is the norm's backward of the layer's dx, from float64 on the device's own upstream values."""
    cfg, layer, x, d_out = _layer(False, norm)
    bare = M().MoELayer(layer.w_router, layer.W13, layer.W2, layer.bias, layer.top_k)
    xin = (x.float() * 3.0 + 0.5)  # f32 input rows
    u, mean, rstd, _ = M().moe_norm(xin, layer.norm_weight, layer.norm_bias, rms=norm == "rms", out_dtype=torch.bfloat16,
                                    want_stats=True)
    assert torch.equal(layer.forward(xin), bare.forward(u))
    _, buf = layer.forward(xin, train=True)
    _, bufb = bare.forward(u, train=True)
    g, gb = layer.backward(d_out, buf), bare.backward(d_out, bufb)
    for n in ("dw13", "dw2", "dw_router"):
        assert torch.equal(g[n], gb[n])
    m64 = np.zeros(x.shape[0]) if mean is None else np64(mean)
    xhat = (np64(xin) - m64[:, None]) * np64(rstd)[:, None]
    du, w = np64(gb["dx"]), np64(layer.norm_weight)
    gy = du * w
    dx = np64(rstd)[:, None] * (gy - (0 if norm == "rms" else gy.mean(1, keepdims=True)) - xhat * (gy * xhat).mean(1, keepdims=True))
    assert rel_err(np64(g["dx"]), dx) <= 100 * U * 16
    assert rel_err(np64(g["dnorm_weight"]), (du * xhat).sum(0)) <= 100 * U * 16
    if norm == "layer":
        assert rel_err(np64(g["dnorm_bias"]), du.sum(0)) <= 100 * U * 16
    assert (g["dnorm_bias"] is None) == (norm == "rms")


def test_layer_checkpoint_memory():
    """What a checkpointed forward keeps of the activations: about a byte an element of x, a | c and y."""
    cfg, layer, x, _ = _layer(False, "rms", T=512)

    def kept(buf):
        n, seen = 0, set()
        def add(v):
            nonlocal n
            if isinstance(v, torch.Tensor) and v.is_cuda and v.data_ptr() not in seen:
                seen.add(v.data_ptr())
                n += v.numel() * v.element_size()
            elif isinstance(v, (tuple, list)):
                [add(i) for i in v]
            elif isinstance(v, dict):
                [add(i) for i in v.values()]
        add(buf)
        return n

    full = kept(layer.forward(x, train=True)[1])
    small = kept(layer.forward(x, checkpoint=True)[1])
    say(f"  kept: {full} -> {small} bytes")
    T, K, d, Inter = 512, 4, 256, 128
    rows = T * (K + 1)
    elems = T * d + rows * 2 * Inter + T * K * d
    rest = full - (x.numel() * 2 * 2 + rows * 2 * Inter * 4 + rows * Inter * 2 + T * K * d * 2 + T * d * 4)
    assert small <= elems * (1 + 1 / 128) + rest + 4096


def test_checkpointed_captured():
    """Pack, unpack and both backward kernels in one graph, replayed over changed inputs with eager work between."""
    T, K, N, d, Inter = 40, 4, 16, 256, 128
    idx, gate, scores = _route(330, T, K, N)
    _, _, pp = M().moe_permute(idx, N, 1)
    ac = I.gen_normal(331, (T * K, 2 * Inter), 1.0, torch.float32).to(DEV)
    y = I.gen_normal(332, (T * K, d), 1.0).to(DEV)
    dh = I.gen_normal(333, (T * K, Inter), 1.0, torch.float32).to(DEV)
    d_out = I.gen_normal(334, (T, d), 1.0).to(DEV)

    def go():
        ck = M().fp8_ckpt_pack(ac)
        yk = M().fp8_ckpt_pack(y)
        return (*ck, M().fp8_ckpt_unpack(*yk), *M().moe_swiglu_backward_ckpt(*ck, dh),
                *M().moe_combine_backward_ckpt(d_out, *yk, idx, gate, scores, pp))

    go()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = go()
    for k in range(4):
        ac.copy_(I.gen_normal(340 + k, ac.shape, 2.0, torch.float32))
        y.copy_(I.gen_normal(350 + k, y.shape, 0.5))
        g.replay()
        ref = go()
        torch.cuda.synchronize()
        for p, r in zip(out, ref):
            assert torch.equal(p, r), k


def test_rows_past_32_bit_offsets():
    """More than 2^31 elements (and bytes past 2^32): the last rows equal those of a call on them alone, to the bit."""
    rows, cols, last = 270_000, 8200, 3
    x = torch.empty((rows, cols), dtype=torch.bfloat16, device=DEV)
    x.fill_(1.5)
    x[-last:] = I.gen_normal(400, (last, cols), 1.0).to(DEV)
    tail = x[-last:].clone()
    q, s = M().fp8_ckpt_pack(x)
    q2, s2 = M().fp8_ckpt_pack(tail)
    assert torch.equal(q[-last:], q2) and torch.equal(s[-last:], s2)
    assert torch.equal(M().fp8_ckpt_unpack(q, s)[-last:], M().fp8_ckpt_unpack(q2, s2))
    y, mean, rstd, ck = M().moe_norm(x, want_stats=True, checkpoint=True)
    y2, mean2, rstd2, ck2 = M().moe_norm(tail, want_stats=True, checkpoint=True)
    # one chunk per lane for few rows, four for many: the sums' order differs, so not to the bit here
    assert rel_err(np64(y[-last:]), np64(y2)) <= 2.0 ** -7 and rel_err(np64(rstd[-last:]), np64(rstd2)) <= 100 * U
    assert torch.equal(y[:1], y[1:2]) and torch.equal(y[0], y[rows // 2])
    dx = M().moe_norm_backward(x, x, mean, rstd)[0]
    dx2 = M().moe_norm_backward(tail, tail, mean[-last:].contiguous(), rstd[-last:].contiguous())[0]
    assert torch.equal(dx[-last:], dx2)
    del y, dx, ck
    inter = cols // 2
    dh = torch.zeros((rows, inter), device=DEV)
    dh[-last:] = 1.0
    dac, h = M().moe_swiglu_backward_ckpt(q, s, dh)
    dac2, h2 = M().moe_swiglu_backward_ckpt(q2, s2, dh[-last:].clone())
    assert torch.equal(dac[-last:], dac2) and torch.equal(h[-last:], h2)
