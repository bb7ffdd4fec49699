"""GPU parity of the 8-bit integer rows and products: i8_quant, i8_dequant, moe_i8_gemm and the layer that runs on them.

Sums of codes are exact integers below 2^31, so an output carries three roundings (the sum to f32, the product of the two
scales, their product), 3 * 2^-24 of its value; SwiGLU carries them into silu.
"""
import numpy as np
import pytest
import torch

from oracle import moe_oracle as O
from sparse_moe_layer_sigmoid_amd import inputs as I
from tests.gpu_common import check_permutation_properties, np64, rel_err, say

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
U = 2.0 ** -24
LEAST = np.float32(127.0) * np.float32(2.0 ** -126)


def M():
    import sparse_moe_layer_sigmoid_amd as m
    return m


def quant_reference(x):
    """Codes and scales by the rule, the codes in float64 (x: float32 array)."""
    bad = ~np.isfinite(x).all(-1)
    x = np.where(bad[..., None], np.float32(0), x)
    a = np.maximum(np.abs(x).max(-1), LEAST)
    q = np.rint(127.0 * x.astype(np.float64) / a.astype(np.float64)[..., None]).astype(np.int8)
    return q, np.where(bad, np.float32("nan"), a / np.float32(127.0)).astype(np.float32)


@pytest.mark.parametrize("rows,cols", [(1, 1), (3, 7), (5, 8), (2, 130), (7, 511), (6, 512), (4, 513), (3, 2048), (2, 2055),
                                       (2, 4097), (1, 7168), (3, 8193), (2, 16384), (2, 16385), (1, 40003), (300, 16)])
@pytest.mark.parametrize("pad", [0, 3])
def test_i8_quant_bf16_bitexact(rows, cols, pad):
    x = I.gen_normal(700 + cols, (rows, cols + pad), 1.0).float()
    x[0] *= 1e-20
    if rows > 2:
        x[1] = 0.0
        x[2] = x[2].abs().clamp(max=2.0)                              # ties: half the row's maximum stands in every other place
        x[2, ::2] = 1.0
        x[2, 0], x[2, -1 - pad] = 2.0, 2.0
    x = x.to(torch.bfloat16)
    q, s = M().i8_quant(x.to(DEV)[:, :cols])
    wq, ws = quant_reference(x[:, :cols].float().numpy())
    assert np.array_equal(s.cpu().numpy(), ws)
    assert np.array_equal(q.cpu().numpy(), wq)
    for dt in (torch.float32, torch.bfloat16):
        v = M().i8_dequant(q, s, dt)
        want = wq.astype(np.float32) * ws[:, None]
        assert torch.equal(v.cpu(), torch.from_numpy(want).to(dt))


@pytest.mark.parametrize("rows,cols", [(3, 5), (4, 1000), (2, 7168), (1, 20000)])
def test_i8_quant_f32(rows, cols):
    """f32 rows: 127 x and the quotient each round once, so a code may be one off where the exact quotient is within
    127 * 2^-23 of a midpoint."""
    x = (I.gen_normal(720 + cols, (rows, cols), 1.0, torch.float32) * 3.7).contiguous()
    x[0] *= 2.0 ** 120
    x[-1, 0] = 300.0
    q, s = M().i8_quant(x.to(DEV))
    wq, ws = quant_reference(x.numpy())
    assert np.array_equal(s.cpu().numpy(), ws)
    t = 127.0 * x.double().numpy() / np.abs(x.double().numpy()).max(1, keepdims=True)
    near = np.abs(np.abs(t - np.floor(t)) - 0.5) <= 127 * 2.0 ** -23
    d = np.abs(q.cpu().numpy().astype(int) - wq.astype(int))
    assert np.all(d[~near] == 0) and np.all(d <= 1)


def test_i8_quant_special_rows():
    """Infinities and NaN mark their row; the ends of the float range; a row at and below the least scale."""
    x = torch.ones((8, 24))
    x[0, 3], x[1, 23], x[2, 5] = float("inf"), float("nan"), float("-inf")
    x[3] = 3.3e38
    x[4] = 0.0
    x[5] = 127.0 * 2.0 ** -126
    x[5, 1] = 2.0 ** -126
    x[6] = 2.0 ** -130
    x[7] = -0.0
    for dt in (torch.float32, torch.bfloat16):
        y = x.to(dt)
        q, s = M().i8_quant(y.to(DEV))
        wq, ws = quant_reference(y.float().numpy())
        assert np.array_equal(s.cpu().numpy(), ws, equal_nan=True) and np.array_equal(q.cpu().numpy(), wq)
        assert np.isnan(M().i8_dequant(q, s).float().cpu().numpy()[:3]).all()
    q, s = M().i8_quant(torch.empty((0, 5), device=DEV))
    assert q.shape == (0, 5) and s.shape == (0,) and M().i8_dequant(q, s).shape == (0, 5)


def test_i8_quant_weights_and_refusals():
    w = I.gen_normal(730, (3, 5, 33), 0.02).to(DEV)
    q, s = M().i8_quant(w)
    q2, s2 = M().i8_quant(w.view(15, 33))
    assert q.shape == w.shape and s.shape == (3, 5) and torch.equal(q.view(15, 33), q2) and torch.equal(s.view(15), s2)
    assert M().i8_dequant(q, s).shape == w.shape
    for bad in (w.cpu(), w.half(), w[:, :, ::2], w.view(-1), w.view(15, 33).t()):
        with pytest.raises((TypeError, ValueError)):
            M().i8_quant(bad)
    for a in ((q.cpu(), s), (q, s.double()), (q, s[:2]), (q.view(torch.uint8), s)):
        with pytest.raises((TypeError, ValueError)):
            M().i8_dequant(*a)
    with pytest.raises(TypeError):
        M().i8_dequant(q, s, torch.float16)


def _operands(seed, G, N, K, src):
    r = np.random.default_rng(seed)
    w = torch.from_numpy(r.integers(-128, 128, (G, N, K), dtype=np.int8))
    ws = torch.from_numpy(r.uniform(0.5, 2.0, (G, N)).astype(np.float32) * np.float32(0.01))
    a = torch.from_numpy(r.integers(-128, 128, (src, K + 16), dtype=np.int8))
    as_ = torch.from_numpy(r.uniform(0.5, 2.0, src).astype(np.float32) * np.float32(1.0 / np.sqrt(K) / 40))
    return a.to(DEV)[:, :K], as_.to(DEV), w.to(DEV), ws.to(DEV)


def _reference(a, as_, w, ws, offs, rows, swiglu):
    """float64 outputs of every sorted row and their bound."""
    x, sx, w, ws = (t.cpu().numpy().astype(np.float64) for t in (a, as_, w, ws))
    out = [np.zeros((0, w.shape[1]))]
    for g in range(len(offs) - 1):
        r = rows[offs[g]:offs[g + 1]]
        out.append((x[r] @ w[g].T) * (sx[r][:, None] * ws[g]))  # the sums are exact in float64
    v = np.concatenate(out)
    if not swiglu:
        return v, 3.01 * U * np.abs(v)
    n = v.shape[1] // 2
    p, c = v[:, :n], v[:, n:]
    # |x silu'(x) / silu(x)| <= 1 + |x|; the device's silu itself is off by a relative (|x| + 8) u
    h = p / (1.0 + np.exp(-p)) * c
    return h, (4 * np.abs(p) + 16) * U * np.abs(h) + 1e-30


# lens of the groups (empty ones, one row, a block of 64 and of 128, one past it), N, K: whole and short last K steps and
# column blocks, one K step, more tiles than workgroups
CASES = [([1], 16, 16), ([0, 1, 0, 2], 32, 64), ([3, 16, 17, 0, 64, 65], 34, 160), ([70, 0, 0, 5], 100, 224),
         ([1, 1, 1, 1, 1], 130, 1056), ([0, 0, 129, 1], 64, 128), ([2] * 40, 48, 96), ([9, 0, 40], 258, 7168),
         ([1, 0, 1, 1], 7, 512), ([128, 127], 2, 32), ([129, 300], 1, 272), ([128], 256, 256), ([257, 100], 300, 384),
         ([500], 1100, 144), ([70] * 9, 640, 128), ([4] * 300, 520, 16), ([200, 0, 0, 90, 1], 512, 400)]


@pytest.mark.parametrize("swiglu", [False, True])
@pytest.mark.parametrize("lens,N,K", CASES)
def test_i8_gemm(lens, N, K, swiglu):
    if swiglu and N % 2:
        N += 1
    say(f"i8_gemm lens={lens[:8]} N={N} K={K} swiglu={swiglu}")
    G, src = len(lens), 50
    offs = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    rows = int(offs[-1])
    a, as_, w, ws = _operands(740 + K, G, N, K, src)
    gather = np.random.default_rng(741).integers(0, src, rows).astype(np.int32)
    cols = N // 2 if swiglu else N
    want, tol = _reference(a, as_, w, ws, offs, gather, swiglu)
    od, gd = torch.from_numpy(offs).to(DEV), torch.from_numpy(gather).to(DEV)
    for dt, half in ((torch.float32, 0.0), (torch.bfloat16, 2.0 ** -8)):
        out = torch.full((rows + 2, cols + 3), 9.0, dtype=dt, device=DEV)[:, :cols]
        M().moe_i8_gemm(a, as_, w, ws, od, 0, G, rows, out, a_rows=gd, swiglu=swiglu)
        got = np64(out)
        assert np.all(np.abs(got[:rows] - want) <= tol + half * np.abs(want) * 1.001)
        assert np.all(got[rows:] == 9.0)                                   # rows past the last one stay as they were
        assert bool((out.as_strided((rows + 2, 3), (cols + 3, 1), cols) == 9.0).all())
    # ungathered rows: row r of A
    i = torch.from_numpy(gather).long().to(DEV)
    out2 = torch.empty((rows, cols), dtype=torch.bfloat16, device=DEV)
    M().moe_i8_gemm(a[i].contiguous(), as_[i], w, ws, od, 0, G, rows, out2, swiglu=swiglu)
    assert torch.equal(out2, out[:rows])


@pytest.mark.parametrize("swiglu", [False, True])
@pytest.mark.parametrize("K", [16, 256, 288, 400])
def test_i8_gemm_tall_groups(K, swiglu):
    """Hundreds of rows to an expert and more tiles than workgroups: tiles that follow each other after two steps and more, in
    other experts and column blocks, and a last short one."""
    say(f"i8_gemm tall groups K={K} swiglu={swiglu}")
    lens, N = [6000, 90, 0, 3000, 193], 1606
    offs = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    rows = int(offs[-1])
    a, as_, w, ws = _operands(760 + K, len(lens), N, K, 700)
    gather = np.random.default_rng(761).integers(0, 700, rows).astype(np.int32)
    want, tol = _reference(a, as_, w, ws, offs, gather, swiglu)
    out = torch.full((rows + 1, want.shape[1]), 9.0, dtype=torch.float32, device=DEV)
    M().moe_i8_gemm(a, as_, w, ws, torch.from_numpy(offs).to(DEV), 0, len(lens), rows, out,
                    a_rows=torch.from_numpy(gather).to(DEV), swiglu=swiglu)
    got = np64(out)
    assert np.all(np.abs(got[:rows] - want) <= tol) and np.all(got[rows:] == 9.0)


def test_i8_gemm_group_range_and_tail():
    """A sub-range of the groups (rows relative to its first), and the last groups' f32 rows in their own output."""
    lens, N, K = [4, 0, 21, 3, 140, 6], 80, 192
    offs = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    rows = int(offs[-1])
    a, as_, w, ws = _operands(750, len(lens), N, K, rows)
    od = torch.from_numpy(offs).to(DEV)
    want, tol = _reference(a, as_, w, ws, offs, np.arange(rows), False)
    f, n = 2, 3
    m = int(offs[f + n] - offs[f])
    out = torch.empty((m, N), dtype=torch.float32, device=DEV)
    M().moe_i8_gemm(a, as_, w, ws, od, f, n, m, out)
    sl = slice(offs[f], offs[f + n])
    assert np.all(np.abs(np64(out) - want[sl]) <= tol[sl])
    for tails in (1, 2, 6):
        t0 = int(offs[len(lens) - tails])
        main = torch.full((max(t0, 1), N), 5.0, dtype=torch.bfloat16, device=DEV)
        tail = torch.empty((rows - t0, N), dtype=torch.float32, device=DEV)
        M().moe_i8_gemm(a, as_, w, ws, od, 0, len(lens), rows, main, out_tail=tail, tail_groups=tails)
        if t0:
            assert np.all(np.abs(np64(main) - want[:t0]) <= (tol + 2.0 ** -8 * 1.001 * np.abs(want))[:t0])
        assert np.all(np.abs(np64(tail) - want[t0:]) <= tol[t0:])


def test_i8_gemm_extremes():
    """Sums at the end of 32 bits (every code -128 over the longest K), NaN scales, scales whose product is subnormal."""
    K, N = 131072 - 16, 16
    a = torch.full((2, K), -128, dtype=torch.int8, device=DEV)
    a[1] = 127
    w = torch.full((1, N, K), -128, dtype=torch.int8, device=DEV)
    offs = torch.tensor([0, 2], dtype=torch.int32, device=DEV)
    one, out = torch.ones(2, device=DEV), torch.empty((2, N), device=DEV)
    M().moe_i8_gemm(a, one, w, torch.ones((1, N), device=DEV), offs, 0, 1, 2, out)
    assert bool((out[0] == np.float32(16384.0 * K)).all()) and bool((out[1] == np.float32(-16256.0 * K)).all())
    a, as_, w, ws = _operands(755, 1, 20, 64, 3)
    as_[1], ws[0, 4], ws[0, 5] = float("nan"), float("nan"), 1e-38
    out = torch.empty((3, 20), device=DEV)
    M().moe_i8_gemm(a, as_, w, ws, torch.tensor([0, 3], dtype=torch.int32, device=DEV), 0, 1, 3, out)
    o = np64(out)
    want, tol = _reference(a, as_, w, ws, [0, 3], np.arange(3), False)
    assert np.isnan(o[1]).all() and np.isnan(o[:, 4]).all()
    o, want, tol = (np.delete(np.delete(v, 1, 0), 4, 1) for v in (o, want, tol))
    assert np.all(np.abs(o - want) <= tol + 2.0 ** -149 * 64 * 16384)       # a scale product one subnormal step off


def test_i8_gemm_many_groups_and_no_rows():
    G, N, K = 1024, 32, 64
    lens = np.zeros(G, dtype=np.int64)
    lens[[0, 5, 511, 512, 1022, 1023]] = [1, 2, 40, 3, 1, 7]
    offs = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    rows = int(offs[-1])
    a, as_, w, ws = _operands(760, G, N, K, rows)
    out = torch.empty((rows, N), dtype=torch.float32, device=DEV)
    M().moe_i8_gemm(a, as_, w, ws, torch.from_numpy(offs).to(DEV), 0, G, rows, out)
    want, tol = _reference(a, as_, w, ws, offs, np.arange(rows), False)
    assert np.all(np.abs(np64(out) - want) <= tol)
    out.fill_(3.0)
    # offsets that claim more rows than m_total are held to it
    M().moe_i8_gemm(a, as_, w, ws, torch.from_numpy(offs).to(DEV), 0, G, 4, out)
    assert np.all(np.abs(np64(out[:4]) - want[:4]) <= tol[:4]) and bool((out[4:] == 3.0).all())
    out.fill_(3.0)
    zero = torch.zeros(G + 1, dtype=torch.int32, device=DEV)
    M().moe_i8_gemm(a, as_, w, ws, zero, 0, G, 5, out)
    M().moe_i8_gemm(a, as_, w, ws, zero, 0, G, 0, out)
    assert bool((out == 3.0).all())


def test_i8_gemm_repeats_streams_and_capture():
    """The same bits on every call, on another stream, and from a graph (quantiser, both products) replayed over changed
    inputs and offsets."""
    lens, N, K, src = [3, 0, 20, 1, 40], 64, 512, 30
    rows = sum(lens)
    offs = torch.from_numpy(np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)).to(DEV)
    _, _, w, ws = _operands(770, len(lens), 2 * N, K, src)
    _, _, w2, ws2 = _operands(771, len(lens), 48, N, src)
    x = I.gen_normal(772, (src, K), 1.0).to(DEV)
    gat = torch.from_numpy(np.random.default_rng(1).integers(0, src, rows).astype(np.int32)).to(DEV)

    def go():
        h = torch.empty((rows, N), dtype=torch.float32, device=DEV)
        M().moe_i8_gemm(*M().i8_quant(x), w, ws, offs, 0, len(lens), rows, h, a_rows=gat, swiglu=True)
        y = torch.empty((rows, 48), dtype=torch.bfloat16, device=DEV)
        return M().moe_i8_gemm(*M().i8_quant(h), w2, ws2, offs, 0, len(lens), rows, y)

    r0 = go()
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        r1 = go()
    torch.cuda.current_stream().wait_stream(st)
    assert torch.equal(r0, r1)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = go()
    for k, new in enumerate(([3, 0, 20, 1, 40], [0, 64, 0, 0, 0], [1, 1, 1, 1, 60], [64, 0, 0, 0, 0])):
        offs.copy_(torch.from_numpy(np.concatenate([[0], np.cumsum(new)]).astype(np.int32)))
        x.copy_(I.gen_normal(780 + k, (src, K), 1.0))
        g.replay()
        ref = go()
        torch.cuda.synchronize()
        assert torch.equal(out, ref), k


def test_i8_gemm_refuses_short_tensors():
    a, as_, w, ws = _operands(790, 2, 32, 64, 4)
    offs = torch.tensor([0, 2, 4], dtype=torch.int32, device=DEV)
    out = torch.empty((4, 32), device=DEV)
    bad = (dict(m_total=5), dict(out=out[:3]), dict(a_rows=offs[:3]), dict(n_groups=3), dict(offs=offs[:2]), dict(out=out[:, :31]),
           dict(a=a[:, :32]), dict(ws=ws[:, :1]), dict(tail_groups=1, out_tail=out[:0]), dict(out=out.double()),
           dict(a=a.float()), dict(a=a.t()), dict(as_=as_[:3]), dict(as_=as_.double()), dict(w=w.view(torch.uint8)))
    for kw in bad:
        c = dict(a=a, as_=as_, w=w, ws=ws, offs=offs, n_groups=2, m_total=4, out=out, a_rows=None, tail_groups=0, out_tail=None)
        c.update(kw)
        if "out_tail" in kw:
            c["out"] = out[:2]
        with pytest.raises((ValueError, TypeError)):
            M().moe_i8_gemm(c["a"], c["as_"], c["w"], c["ws"], c["offs"], 0, c["n_groups"], c["m_total"], c["out"],
                            a_rows=c["a_rows"], tail_groups=c["tail_groups"], out_tail=c["out_tail"])


@pytest.mark.parametrize("swiglu", [False, True])
def test_i8_gemm_holds_to_its_tensors(swiglu):
    """Rows that a_rows, a, out or out_tail does not hold are neither read nor written, whatever the offsets say.  Every
    tensor is the head of a longer one, whose rest has to stay as it was."""
    lens, N, K = [4, 0, 21, 3, 140, 6], 50, 192
    offs = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    rows, G, cols = int(offs[-1]), len(lens), N // 2 if swiglu else N
    a, as_, w, ws = _operands(800, G, N, K, rows)
    od, ident = torch.from_numpy(offs).to(DEV), torch.arange(rows, dtype=torch.int32, device=DEV)
    want, tol = _reference(a, as_, w, ws, offs, np.arange(rows), swiglu)

    def check(got, want, tol, n, half=0.0):
        g = np64(got)
        assert np.all(np.abs(g[:n] - want[:n]) <= (tol + half * 1.001 * np.abs(want))[:n] + 1e-30)
        assert np.all(g[n:] == 9.0)

    for have in (0, 3, 24, 27, 29, 169):  # sorted rows that are there; the range below is rows 4 to 168
        for kw in (dict(a_rows=ident[:have]), dict()):
            out = torch.full((164, cols), 9.0, device=DEV)
            M().moe_i8_gemm(a if kw else a[:have], as_ if kw else as_[:have], w, ws, od, 2, 3, 164, out, swiglu=swiglu, **kw)
            check(out, want[4:], tol[4:], min(max(have - 4, 0), 164))
    for tails in (1, 2, 6):
        t0 = int(offs[G - tails])
        for main in sorted({0, 1, t0 // 2, max(t0 - 1, 0), t0, t0 + 1, rows}):
            tail = rows - main
            out = torch.full((rows + 8, cols), 9.0, dtype=torch.bfloat16, device=DEV)
            rest = torch.full((rows + 8, cols), 9.0, device=DEV)
            M().moe_i8_gemm(a, as_, w, ws, od, 0, G, rows, out[:main], out_tail=rest[:tail], tail_groups=tails, swiglu=swiglu)
            check(out, want, tol, min(main, t0), 2.0 ** -8)
            check(rest, want[t0:], tol[t0:], 0 if main < t0 else min(tail, rows - t0))


def test_i8_gemm_two_streams_at_once():
    lens, N, K = [1, 0, 140, 3], 2048, 2048
    offs = torch.from_numpy(np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)).to(DEV)
    rows = sum(lens)
    ops = []
    for k in range(2):
        a, as_, w, ws = _operands(810 + k, len(lens), N, K, rows)
        ref = torch.empty((rows, N), device=DEV)
        M().moe_i8_gemm(a, as_, w, ws, offs, 0, len(lens), rows, ref)
        ops.append((a, as_, w, ws, ref, torch.empty((rows, N), device=DEV), torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(10):
        for a, as_, w, ws, ref, out, st in ops:
            with torch.cuda.stream(st):
                M().moe_i8_gemm(a, as_, w, ws, offs, 0, len(lens), rows, out)
    torch.cuda.synchronize()
    for a, as_, w, ws, ref, out, st in ops:
        assert torch.equal(ref, out)


def test_i8_gemm_row_by_itself():
    """A row's result has the same bits alone and among other rows, in any group size (both row blocks)."""
    a, as_, w, ws = _operands(820, 1, 300, 544, 200)
    for swiglu in (False, True):
        def go(n, first=0):
            out = torch.empty((n, 150 if swiglu else 300), device=DEV)
            return M().moe_i8_gemm(a[first:first + n], as_[first:first + n], w, ws,
                                   torch.tensor([0, n], dtype=torch.int32, device=DEV), 0, 1, n, out, swiglu=swiglu)
        full = go(200)
        for r in (0, 15, 16, 127, 128, 199):
            assert torch.equal(go(1, r)[0], full[r])
        assert torch.equal(go(63), full[:63])


@pytest.mark.parametrize("T,norm", [(1, None), (1, "rms"), (5, None), (64, "layer"), (300, "rms")])
def test_layer_i8(T, norm):
    """MoELayer(i8=True) stage by stage in float64 on what the device quantised: the bf16 path's bar (1e-2 of the RMS)."""
    cfg = I.small(I.V3_BF16, name="i8_layer", T=T, d=256, n_experts=16, top_k=4, inter=96, w_std=0.05, router_std=0.05, seed=9)
    ex = [I.gen_expert(cfg, e) for e in range(cfg.groups)]
    W13 = torch.stack([a for a, _ in ex]).to(torch.bfloat16)
    W2 = torch.stack([b for _, b in ex]).to(torch.bfloat16)
    wr, bias, x = I.gen_router(cfg), I.gen_bias(cfg), I.gen_x(cfg)
    nw = (1.0 + I.gen_normal(11, (cfg.d,), 0.1, torch.float32)).to(DEV) if norm else None
    layer = M().MoELayer(wr.to(DEV), W13.to(DEV), W2.to(DEV), bias.to(DEV), cfg.top_k, i8=True, norm=norm, norm_weight=nw)
    out, buf = layer.forward(x.to(DEV), out_dtype=torch.float32, keep=True)
    check_permutation_properties(buf["expert_offsets"], buf["sorted_token"], buf["pair_pos"], buf["topk_idx"], cfg.n_experts)
    u = x if norm is None else M().moe_norm(x.to(DEV), nw, rms=norm == "rms")[0].cpu()
    r = O.route(u.double().numpy(), wr.double().numpy(), bias.numpy(), cfg.top_k)
    ok = r["margin"] >= 1e-6
    xq, xs = quant_reference(u.float().numpy())
    assert np.array_equal(buf["xq"].cpu().numpy(), xq)
    xv = xq.astype(np.float64) * xs[:, None]
    val = lambda q, s: q.cpu().numpy().astype(np.float64) * s.cpu().numpy().astype(np.float64)[..., None]  # noqa: E731
    w13, w2 = val(layer.W13, layer.W13_s), val(layer.W2, layer.W2_s)
    assert np.all(np.abs(w13 - W13.double().numpy()) <= np.abs(W13.double().numpy()).max(-1, keepdims=True) / 253.9)
    hd = np64(buf["h"]) * np64(buf["hs"])[:, None]
    ref = np.zeros((T, cfg.d))
    pp = buf["pair_pos"].cpu().numpy()
    for t in range(T):
        for k in range(cfg.top_k + 1):
            e = int(buf["topk_idx"][t, k]) if k < cfg.top_k else cfg.n_experts
            g = float(buf["topk_gate"][t, k]) if k < cfg.top_k else 1.0
            row = pp[t, k] if k < cfg.top_k else T * cfg.top_k + t
            v = w13[e] @ xv[t]
            h = v[:cfg.inter] / (1.0 + np.exp(-v[:cfg.inter])) * v[cfg.inter:]
            step = np.abs(h).max() / 127.0
            assert np.all(np.abs(hd[row] - h) <= step * 0.51)                # the stored h is h rounded to its codes
            ref[t] += g * (w2[e] @ hd[row])
    err = rel_err(np64(out)[ok], ref[ok])
    say(f"  i8 layer T={T}: {err:.2e}")
    assert ok.any() and err <= 1e-2
    for call in (lambda: layer.forward(x.to(DEV), train=True), lambda: layer.forward(x.to(DEV), checkpoint=True),
                 lambda: layer.backward(out, buf)):
        with pytest.raises(NotImplementedError):
            call()


def test_layer_i8_no_tokens_and_formats():
    cfg = I.small(I.V3_BF16, name="i8_empty", T=1, d=64, n_experts=8, top_k=2, inter=64)
    ex = [I.gen_expert(cfg, e) for e in range(cfg.groups)]
    W13, W2 = (torch.stack([e[k] for e in ex]).to(torch.bfloat16).to(DEV) for k in (0, 1))
    args = (I.gen_router(cfg).to(DEV), W13, W2, I.gen_bias(cfg).to(DEV), 2)
    out = M().MoELayer(*args, i8=True, norm="layer").forward(torch.empty((0, 64), dtype=torch.bfloat16, device=DEV))
    assert out.shape == (0, 64)
    for kw in (dict(i8=True, w4=True), dict(i8=True, fp8=True)):
        with pytest.raises(ValueError):
            M().MoELayer(*args, **kw)
