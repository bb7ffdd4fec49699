"""GPU parity of moe_decode, the whole layer for a few tokens, against the layer's definition in float64 on the values that the
weights' codes stand for.

Two bounds.  Each output: sums of n products carry at most (n/4 + 16) 2^-23 of the sum of magnitudes (a matrix instruction adds
its products to a partial sum in at most 8 truncating steps; scales, gates and the waves' sums round a few times more), through
silu and the second product, whose h loses at most 2^-16 of itself between its two bf16 parts.  All outputs together: the
rounding of h is random, 2^-16 of the outputs' RMS for one output and 5 times that among thousands; 2e-4 holds 2.5 times that
much (silu and sums add 2^-20 or so).
"""
import numpy as np
import pytest
import torch

from oracle import moe_oracle as O
from sparse_moe_layer_sigmoid_amd import inputs as I
from tests.gpu_common import np64, rel_err, say

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=np.float64)
FORMATS = ["bf16", "e4m3", "e8m0", "i8", "w4"]


def M():
    import sparse_moe_layer_sigmoid_amd as m
    return m


def quantise(fmt, W):
    """(weights, scales) of bf16 weights [G, n, k] in a format."""
    m = M()
    q = {"bf16": lambda w: (w, None), "e4m3": m.fp8_quant_128x128, "e8m0": m.fp8_quant_128x128_e8m0, "i8": m.i8_quant,
         "w4": m.w4_quant}
    return q[fmt](W)


def values(fmt, W, s):
    """float64 weights that codes and scales stand for."""
    if fmt == "bf16":
        return np64(W)
    c, s = W.cpu().numpy(), s.cpu().numpy()
    if fmt == "i8":
        return c.astype(np.float64) * s.astype(np.float64)[..., None]
    if fmt == "w4":
        nib = np.stack([c & 15, c >> 4], -1).reshape(*c.shape[:-1], -1)
        return E2M1[nib & 7] * np.where(nib >= 8, -1.0, 1.0) * np.repeat(np.exp2(s.astype(np.float64) - 127), 32, axis=-1)
    s = np.exp2(s.astype(np.float64) - 127) if fmt == "e8m0" else s.astype(np.float64)
    return O.e4m3_decode(c) * np.repeat(np.repeat(s, 128, axis=-2), 128, axis=-1)


class Case:
    """A layer's weights and tokens on the device, and its definition in float64."""

    def __init__(self, fmt, T, d, inter, E, K, groups=(1, 1), norm=None, shared=1, seed=0, x_dtype=torch.bfloat16, pad=0,
                 same_tokens=False):
        self.fmt, self.T, self.d, self.inter, self.E, self.K, self.groups, self.norm = fmt, T, d, inter, E, K, groups, norm
        g = lambda i, shape, std, dt=torch.bfloat16: I.gen_normal(9000 + 100 * seed + i, shape, std, dt)  # noqa: E731
        x = g(0, (T, d + pad), 1.0, torch.float32) + (0.3 if norm else 0.0)
        if same_tokens:
            x = x[:1].repeat(T, 1)
        self.x = x.to(x_dtype).to(DEV)[:, :d]
        self.wr = g(1, (E, d), 0.5 / np.sqrt(d)).to(DEV)
        self.bias = (g(2, (E,), 0.01, torch.float32)).to(DEV)
        G = E + shared
        self.W13, self.s13 = quantise(fmt, g(3, (G, 2 * inter, d), 0.5 / np.sqrt(d)).to(DEV))
        self.W2, self.s2 = quantise(fmt, g(4, (G, d, inter), 0.5 / np.sqrt(inter)).to(DEV))
        self.nw = (1.0 + g(5, (d,), 0.1, torch.float32)).to(DEV) if norm else None
        self.nb = g(6, (d,), 0.1, torch.float32).to(DEV) if norm == "layer" else None
        self.shared = shared

    def run(self, out_dtype=torch.float32, x=None):
        return M().moe_decode(self.x if x is None else x, self.wr, self.bias, self.W13, self.W2, self.K, *self.groups,
                              W13_scale=self.s13, W2_scale=self.s2, norm=self.norm, norm_weight=self.nw, norm_bias=self.nb,
                              out_dtype=out_dtype)

    def rows(self):
        x = np64(self.x)
        if not self.norm:
            return x
        mean = x.mean(1, keepdims=True) if self.norm == "layer" else 0.0
        y = (x - mean) / np.sqrt(((x - mean) ** 2).mean(1, keepdims=True) + 1e-6) * np64(self.nw)
        return np64(torch.from_numpy(y + (np64(self.nb) if self.nb is not None else 0.0)).to(torch.bfloat16))

    def reference(self):
        """outputs, bound of each, routing."""
        x, n = self.rows(), self.inter
        r = O.route(x, np64(self.wr), np64(self.bias), self.K, *self.groups)
        w13, w2 = values(self.fmt, self.W13, self.s13), values(self.fmt, self.W2, self.s2)
        out, tol = np.zeros((self.T, self.d)), np.zeros((self.T, self.d))
        U = 2.0 ** -23
        for t in range(self.T):
            for k in range(self.K + self.shared):
                e, g = (r["idx"][t, k], r["gate"][t, k]) if k < self.K else (self.E, 1.0)
                v, tv = w13[e] @ x[t], (self.d / 4 + 16) * U * (np.abs(w13[e]) @ np.abs(x[t]))
                a, c, ta, tc = v[:n], v[n:], tv[:n], tv[n:]
                sg = 1.0 / (1.0 + np.exp(-a))
                h = a * sg * c
                # |silu'| <= 1.1; the device's silu itself is off by a relative (|a| + 8) 2^-24
                th = 1.1 * ta * (np.abs(c) + tc) + np.abs(a * sg) * tc + np.abs(h) * ((np.abs(a) + 10) * U + 2.0 ** -16)
                out[t] += g * (w2[e] @ h)
                tol[t] += g * (np.abs(w2[e]) @ (th + (n / 4 + self.K + 16) * U * (np.abs(h) + th)))
        return out, tol, r


def check(c, out_dtype=torch.float32):
    out, idx, gate, counts = c.run(out_dtype)
    want, tol, r = c.reference()
    assert np.all(r["margin"] > 1e-9) and np.all(r["group_margin"] > 1e-9)   # fp64 against fp64: no ties in these inputs
    assert np.array_equal(idx.cpu().numpy(), r["idx"])
    assert np.all(np.abs(np64(gate) - r["gate"]) <= 2.0 ** -24)
    assert np.array_equal(counts.cpu().numpy(), np.bincount(r["idx"].ravel(), minlength=c.E))
    got = np64(out)
    err = rel_err(got, want)
    say(f"  {c.fmt} T={c.T} d={c.d} I={c.inter} E={c.E} K={c.K}: {err:.2e}")
    half = 2.0 ** -8 if out_dtype == torch.bfloat16 else 2.0 ** -24
    assert np.all(np.abs(got - want) <= tol * (1 + half) + half * np.abs(want) + 1e-30)
    if out_dtype == torch.float32:
        assert err <= 2e-4
    return out


# T, d, inter, E, K, groups, norm, shared: one block of inputs for 8 waves, short last blocks, more than one slice of the inner
# width, the widest rows, one token and all columns, every expert chosen, no shared expert
CASES = [(1, 128, 128, 4, 1, (1, 1), None, 1), (16, 128, 128, 16, 2, (1, 1), None, 1), (5, 256, 128, 8, 8, (1, 1), "rms", 1),
         (3, 384, 384, 16, 4, (4, 2), "layer", 1), (1, 1152, 640, 8, 2, (1, 1), None, 0), (2, 2048, 2304, 4, 2, (1, 1), None, 1),
         (1, 7168, 256, 4, 1, (1, 1), "rms", 1), (7, 8192, 128, 4, 3, (1, 1), None, 1), (16, 640, 256, 64, 32, (1, 1), None, 1),
         (16, 896, 896, 256, 8, (8, 4), "rms", 1), (4, 128, 4480, 4, 2, (1, 1), None, 0), (9, 4096, 384, 8, 4, (2, 1), "layer", 1)]


@pytest.mark.parametrize("fmt", ["bf16", "e4m3", "i8", "w4"])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c[:5])))
def test_decode(fmt, case):
    T, d, inter, E, K, groups, norm, shared = case
    say(f"decode {fmt} {case}")
    check(Case(fmt, T, d, inter, E, K, groups, norm, shared))


@pytest.mark.parametrize("fmt", ["bf16", "i8", "w4"])
def test_decode_every_expert(fmt):
    """16 tokens that choose all 256 experts among them: more units than any token has."""
    c = Case(fmt, 16, 256, 256, 256, 32)
    out = check(c)
    assert len(torch.unique(c.run()[1])) > 200
    Case(fmt, 2, 512, 384, 8, 2).run()                      # another shape between, on the same stream
    assert torch.equal(c.run()[0], out)


@pytest.mark.parametrize("T,d,inter", [(1, 64, 64), (5, 256, 64), (3, 192, 320), (2, 8128, 64), (16, 64, 2112)])
def test_decode_bf16_blocks_of_64(T, d, inter):
    check(Case("bf16", T, d, inter, 8, 2))


@pytest.mark.parametrize("T,d,inter,norm", [(1, 512, 512, None), (6, 1024, 512, "rms"), (16, 512, 2560, None)])
def test_decode_e8m0(T, d, inter, norm):
    check(Case("e8m0", T, d, inter, 8, 2, norm=norm))


@pytest.mark.parametrize("fmt", FORMATS)
def test_decode_bf16_output_and_strides(fmt):
    """bf16 output; rows of x wider than d; f32 rows at an odd element behind a norm."""
    check(Case(fmt, 5, 512, 512, 8, 2, pad=8), torch.bfloat16)
    check(Case(fmt, 5, 512, 512, 8, 2, norm="layer", pad=3, x_dtype=torch.float32), torch.bfloat16)
    c = Case(fmt, 3, 512, 512, 8, 2, norm="rms", pad=3)
    c.x = c.x.as_strided((3, 512), (515, 1), 1)                            # bf16 rows that start at odd elements
    check(c)


@pytest.mark.parametrize("fmt", FORMATS)
def test_decode_token_by_itself(fmt):
    """A token's result has the same bits alone and among others, and with every token choosing the same experts."""
    c = Case(fmt, 16, 1024, 512, 16, 4, norm="rms")
    out, idx, gate, _ = c.run()
    for t in (0, 7, 15):
        o, i, g, _ = c.run(x=c.x[t:t + 1])
        assert torch.equal(o[0], out[t]) and torch.equal(i[0], idx[t]) and torch.equal(g[0], gate[t])
    o = c.run(x=c.x[3:10])[0]
    assert torch.equal(o, out[3:10])
    c = Case(fmt, 16, 1024, 512, 16, 4, same_tokens=True)
    out = check(c)
    assert bool((out == out[0]).all())


@pytest.mark.parametrize("fmt", FORMATS)
def test_decode_special_values(fmt):
    """A token with NaN or infinities leaves the others alone, an expert with NaN weights reaches only tokens that chose it."""
    c = Case(fmt, 6, 512, 512, 8, 2, shared=0)
    ref, idx, _, _ = c.run()
    x = c.x.clone()
    x[2, 7], x[4, 100] = float("nan"), float("inf")
    out, i2, _, counts = c.run(x=x)
    keep = [0, 1, 3, 5]
    assert torch.equal(out[keep], ref[keep]) and torch.equal(i2[keep], idx[keep])
    assert bool(torch.isnan(out[2]).all()) and not bool(torch.isfinite(out[4]).all())
    assert int(counts.sum()) == 12 and int(i2.min()) >= 0 and int(i2.max()) < 8
    e = int(idx[0, 0])
    if fmt in ("bf16",):
        c.W13[e, 3, 5] = float("nan")
    elif fmt in ("e4m3", "e8m0"):
        c.W13[e, 3, 5] = 0x7f
    elif fmt == "i8":
        c.s13[e, 3] = float("nan")
    else:
        c.s13[e, 3, 1] = 255
    out = c.run()[0]
    hit = (idx == e).any(1)
    assert bool(torch.isnan(out[hit]).all()) and torch.equal(out[~hit], ref[~hit]) and bool(hit.any())


def test_decode_norm_of_far_rows():
    """Rows far from zero and near the ends of the float range."""
    c = Case("bf16", 4, 512, 128, 8, 2, norm="layer", x_dtype=torch.float32)
    x = c.x.clone()
    x[0] = x[0] * 1e-3 + 1e3
    x[1] *= 2.0 ** 100
    x[2] *= 2.0 ** -5
    x[3] = x[3] * 2.0 ** 60 - 2.0 ** 63
    c.x = x
    check(c)


@pytest.mark.parametrize("fmt", FORMATS)
def test_decode_repeats_streams_and_capture(fmt):
    """The same bits on every call whatever workgroup takes what, on two streams at once, and from graphs replayed over changed
    tokens with eager calls between the replays."""
    c = Case(fmt, 4, 1024, 512, 32, 4, norm="rms")
    ref = c.run()
    for _ in range(20):
        for a, b in zip(c.run(), ref):
            assert torch.equal(a, b)
    c2 = Case(fmt, 9, 1024, 512, 32, 4, seed=1)
    ref2 = c2.run()
    st = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = []
    for _ in range(10):
        for s, k in zip(st, (c, c2)):
            with torch.cuda.stream(s):
                got.append((k, k.run()))
    torch.cuda.synchronize()
    for k, o in got:
        for a, b in zip(o, ref if k is c else ref2):
            assert torch.equal(a, b)
    g1, g2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g1):
        o1 = c.run()
    with torch.cuda.graph(g2):
        o2 = c2.run()
    for k in range(4):
        c.x.copy_(I.gen_normal(880 + k, tuple(c.x.shape), 1.0))
        c2.x.copy_(I.gen_normal(890 + k, tuple(c2.x.shape), 1.0))
        torch.cuda.synchronize()
        with torch.cuda.stream(st[0]):
            g1.replay()
        with torch.cuda.stream(st[1]):
            g2.replay()
        torch.cuda.synchronize()
        for got, want in ((o1, c.run()), (o2, c2.run())):
            for a, b in zip(got, want):
                assert torch.equal(a, b), k


def test_decode_beside_other_work():
    """Calls while another stream keeps the device full: workgroups that start late find their lists taken, or take what is
    left."""
    c = Case("bf16", 2, 1024, 1024, 16, 4)
    ref = c.run()[0]
    a = torch.randn(4096, 4096, device=DEV)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    outs = []
    for _ in range(10):
        with torch.cuda.stream(s):
            a = torch.mm(a, a) * 1e-2
        outs.append(c.run()[0])
    torch.cuda.synchronize()
    assert all(torch.equal(o, ref) for o in outs)


def test_decode_no_tokens_and_refusals():
    c = Case("i8", 2, 256, 128, 8, 2)
    out, idx, gate, counts = c.run(x=c.x[:0])
    assert out.shape == (0, 256) and idx.shape == (0, 2) and gate.shape == (0, 2) and not bool(counts.any())
    m = M()
    ok = dict(x=c.x, w_router=c.wr, bias=c.bias, W13=c.W13, W2=c.W2, top_k=2, W13_scale=c.s13, W2_scale=c.s2)
    m.moe_decode(**ok)
    bad = (dict(x=c.x.float()), dict(x=c.x.cpu()), dict(x=c.x.repeat(9, 1)), dict(x=c.x[:, :128]), dict(top_k=0), dict(top_k=9),
           dict(n_group=3), dict(topk_group=2), dict(W13_scale=None), dict(W2_scale=c.s2[:-1]), dict(W13=c.W13[:-1]),
           dict(W13=c.W13.view(torch.uint8)), dict(W13=c.W13[:, ::2]), dict(W2=c.W2.float()), dict(bias=c.bias[:-1]),
           dict(bias=c.bias.double()), dict(w_router=c.wr[:, :128]), dict(norm="batch"), dict(norm_weight=c.bias),
           dict(norm="rms", norm_weight=c.bias), dict(out_dtype=torch.float16), dict(x=c.x.t()), dict(x=c.x[0]))
    for kw in bad:
        with pytest.raises((ValueError, TypeError, m.MoeError)):
            m.moe_decode(**{**ok, **kw})
    w = Case("bf16", 2, 320, 64, 8, 2)
    with pytest.raises(m.MoeError):                                        # 4-bit rows are blocks of 128 inputs
        m.moe_decode(w.x, w.wr, w.bias, *(m.w4_quant(w.W13)[0], m.w4_quant(w.W2)[0]), 2, W13_scale=m.w4_quant(w.W13)[1],
                     W2_scale=m.w4_quant(w.W2)[1])


@pytest.mark.parametrize("kind", ["bf16", "fp8", "e8m0", "w4", "i8"])
@pytest.mark.parametrize("T,norm", [(1, None), (3, "rms"), (16, "layer")])
def test_layer_decode(kind, T, norm):
    """MoELayer.decode against its forward: the same experts and loads, and outputs apart by what forward rounds on the way
    (h to bf16: 1e-2 of the RMS; rows and h to 8 bits: 3 mantissa bits are 2^-4 of each, 7 bits of a row's largest 1/254)."""
    cfg = I.small(I.V3_BF16, name="decode_layer", T=T, d=512, n_experts=16, top_k=4, inter=512, w_std=0.03, router_std=0.05,
                  seed=21)
    ex = [I.gen_expert(cfg, e) for e in range(cfg.groups)]
    W13 = torch.stack([a for a, _ in ex]).to(torch.bfloat16).to(DEV)
    W2 = torch.stack([b for _, b in ex]).to(torch.bfloat16).to(DEV)
    kw = {"bf16": {}, "fp8": dict(fp8=True), "e8m0": dict(fp8=True, fp8_scales="e8m0"), "w4": dict(w4=True), "i8": dict(i8=True)}[kind]
    nw = (1.0 + I.gen_normal(11, (cfg.d,), 0.1, torch.float32)).to(DEV) if norm else None
    layer = M().MoELayer(I.gen_router(cfg).to(DEV), W13, W2, I.gen_bias(cfg).to(DEV), cfg.top_k, norm=norm, norm_weight=nw, **kw)
    x = I.gen_x(cfg).to(DEV)
    bias = layer.bias.clone()
    want = layer.forward(x, out_dtype=torch.float32, update_bias=True)
    after = layer.bias.clone()
    layer.bias.copy_(bias)
    got = layer.decode(x, out_dtype=torch.float32, update_bias=True)
    assert torch.equal(layer.bias, after)
    err = rel_err(np64(got), np64(want))
    say(f"  decode {kind} T={T} against forward: {err:.2e}")
    # E4M3: a value in [2^e, 2^(e+1)) is off by up to 2^(e-4), uniformly: 2^(e-4) / sqrt(3) of about 1.53 * 2^e, 0.0236 RMS.  x's
    # error enters h through gate and up (sqrt(2) times, and silu's slope times 1.2): 0.040; h's own 0.0236; together 0.046 of a
    # token's RMS.  Up to 16 * 512 outputs reach 4.5 sigma, and a token's RMS is up to 1.4 times all tokens': 0.29.
    # int8: x in steps of its largest (3.3 RMS of 512) / 127, 0.0075 RMS, 0.0127 in h; h in steps of 8 RMS / 127, 0.018; together
    # 0.022: 0.14.
    assert err <= {"bf16": 1e-2, "w4": 1e-2, "fp8": 0.29, "e8m0": 0.29, "i8": 0.14}[kind]
    layer.bias.copy_(bias)
    assert torch.equal(layer.decode(x), got.bfloat16())
