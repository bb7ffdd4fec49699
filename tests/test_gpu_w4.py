"""GPU parity of the 4-bit expert weights: w4_quant, moe_w4_gemm and the layer that runs on them.

Products of a bf16 activation and a 4-bit weight (at most 10 significant bits) are exact in fp32, so only the sums
round: a wave adds K/128 matrix instructions of 32 products each, at most K/4 additions of a partial sum no larger
than sum|a w|, each off by at most 2^-23 of it (truncating adders included), and three more join the waves.
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
E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=np.float64)


def M():
    import sparse_moe_layer_sigmoid_amd as m
    return m


def decode(q, s):
    """Codes [.., K/2], scale codes [.., K/32] -> weights in float64."""
    q, s = q.cpu().numpy(), s.cpu().numpy()
    nib = np.stack([q & 15, q >> 4], -1).reshape(*q.shape[:-1], -1)
    v = E2M1[nib & 7] * np.where(nib >= 8, -1.0, 1.0)
    with np.errstate(over="ignore"):
        return v * np.repeat(np.where(s == 255, np.nan, np.exp2(s.astype(np.float64) - 127)), 32, axis=-1)


def quant_reference(w):
    """The quantiser's rule in float64: nearest code, ties to the even one; scale the least 2^k with amax <= 6 * 2^k."""
    g = w.reshape(-1, 32)
    amax = np.abs(g).max(1)
    k = np.zeros(len(g), dtype=np.int64)
    nz = amax > 0
    k[nz] = np.maximum(-127, np.ceil(np.log2(amax[nz] / 6.0)).astype(np.int64))
    for i in np.nonzero(nz)[0]:  # exact at the edges
        while amax[i] > 6.0 * 2.0 ** k[i]:
            k[i] += 1
        while k[i] > -127 and amax[i] <= 6.0 * 2.0 ** (k[i] - 1):
            k[i] -= 1
    v = np.abs(g) / np.exp2(k)[:, None]
    code = np.zeros(v.shape, dtype=np.int64)
    for c in range(7):
        mid = (E2M1[c] + E2M1[c + 1]) / 2
        code += (v > mid) | ((v == mid) & (c % 2 == 1))  # from odd c up to the even c + 1
    code |= np.where(np.signbit(g), 8, 0)
    code = code.reshape(w.shape)
    q = (code[..., 0::2] | (code[..., 1::2] << 4)).astype(np.uint8)
    return q, (k + 127).reshape(*w.shape[:-1], -1).astype(np.uint8)


@pytest.mark.parametrize("shape", [(1, 32), (3, 64), (5, 96), (2, 7, 224), (3, 16, 2048)])
def test_w4_quant_bitexact(shape):
    w = I.gen_normal(400 + shape[-1], shape, 0.02).float()
    f = w.view(-1, 32)
    f[0] = torch.linspace(-6, 6, 32)
    if len(f) > 3:
        f[1] = 0.0
        f[2, :8] = torch.tensor([6.0, 0.25, 0.75, 1.25, -1.75, 2.5, 3.5, 5.0])   # every midpoint at scale 1
        f[2, 8:] = 0.0
        f[3, 0], f[3, 1:] = 6.03125, 1e-3                                          # just past the edge of the scale
    w = w.to(torch.bfloat16)
    q, s = M().w4_quant(w.to(DEV))
    wq, ws = quant_reference(w.double().numpy())
    assert np.array_equal(s.cpu().numpy(), ws)
    assert np.array_equal(q.cpu().numpy(), wq)


def test_w4_quant_special():
    w = torch.full((5, 32), 0.01, dtype=torch.bfloat16)
    w[0, 3], w[1, 4], w[2] = float("inf"), float("nan"), -0.0
    w[3] = 1e-39
    w[4] = 3.3e38
    q, s = M().w4_quant(w.to(DEV))
    v = decode(q, s)
    assert s[0].item() == 255 and s[1].item() == 255 and np.isnan(v[:2]).all()
    assert not v[2].any() and s[2].item() == 127
    wq, ws = quant_reference(w[3:].double().numpy())
    assert np.array_equal(q[3:].cpu().numpy(), wq) and np.array_equal(s[3:].cpu().numpy(), ws)


def _weights(seed, G, N, K, uniform_scale=False):
    r = np.random.default_rng(seed)
    q = torch.from_numpy(r.integers(0, 256, (G, N, K // 2), dtype=np.uint8))
    s = torch.from_numpy(np.full((G, N, K // 32), 125, np.uint8) if uniform_scale
                         else r.integers(118, 124, (G, N, K // 32)).astype(np.uint8))
    return q.to(DEV), s.to(DEV)


def _reference(a, w, offs, rows, swiglu):
    """float64 outputs of every sorted row and the bound on the sums."""
    out, tol = [], []
    K = w.shape[2]
    for g in range(len(offs) - 1):
        r = rows[offs[g]:offs[g + 1]]
        if len(r) == 0:
            continue
        x = a[r]
        out.append(x @ w[g].T)
        tol.append((K / 4 + 3) * 2.0 ** -23 * (np.abs(x) @ np.abs(w[g]).T))
    v, t = np.concatenate(out), np.concatenate(tol)
    if not swiglu:
        return v, t
    n = v.shape[1] // 2
    x, c, tx, tc = v[:, :n], v[:, n:], t[:, :n], t[:, n:]
    sg = 1.0 / (1.0 + np.exp(-x))
    # |silu'| <= 1.1; the device's silu itself is off by a relative (|x| + 8) u
    return x * sg * c, 1.1 * tx * (np.abs(c) + tc) + np.abs(x * sg) * tc + np.abs(x * sg * c) * (np.abs(x) + 10) * 2 * U


# lens of the groups (empty ones, one row, a full tile of 16, one past it, a full block of 32, several blocks), N, K
CASES = [([1], 16, 32), ([0, 1, 0, 2], 32, 64), ([3, 16, 17, 0, 32, 33], 34, 160), ([70, 0, 0, 5], 100, 224),
         ([1, 1, 1, 1, 1], 130, 1056), ([0, 0, 129, 1], 64, 128), ([2] * 40, 48, 96), ([9, 0, 40], 258, 7168),
         ([1, 0, 1, 1], 7, 512), ([5, 31], 2, 32), ([16, 15], 1, 288),
         # each number of waves and K blocks, whole and short last blocks, more weight tiles than workgroups
         ([2, 0, 17], 48, 544), ([1, 20], 32, 992), ([0, 3], 64, 1184), ([40], 16, 2048), ([1, 1], 32, 2080),
         ([5], 80, 4064), ([17, 1], 32, 4128), ([2], 16, 6144), ([3], 32, 6176), ([1, 2], 16, 7136), ([33], 48, 7200),
         ([4], 32, 8192), ([4], 32, 8224), ([1, 1, 0, 16, 2], 12288, 64), ([60] * 9, 3200, 96)]


@pytest.mark.parametrize("swiglu", [False, True])
@pytest.mark.parametrize("lens,N,K", CASES)
def test_w4_gemm(lens, N, K, swiglu):
    if swiglu and N % 2:
        N += 1
    say(f"w4_gemm lens={lens} N={N} K={K} swiglu={swiglu}")
    G = len(lens)
    offs = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    rows = int(offs[-1])
    q, s = _weights(500 + K, G, N, K)
    w = decode(q, s)
    src = 50
    a = I.gen_normal(501, (src, K + 8), 1.0).to(DEV)[:, :K]                # rows wider than K
    gather = np.random.default_rng(502).integers(0, src, rows).astype(np.int32)
    cols = N // 2 if swiglu else N
    want, tol = _reference(np64(a), w, offs, gather, swiglu)
    od, gd = torch.from_numpy(offs).to(DEV), torch.from_numpy(gather).to(DEV)
    for dt, half in ((torch.float32, 0.0), (torch.bfloat16, 2.0 ** -8)):
        out = torch.full((rows + 2, cols + 3), 9.0, dtype=dt, device=DEV)[:, :cols]
        M().moe_w4_gemm(a, q, s, od, 0, G, rows, out, a_rows=gd, swiglu=swiglu)
        got = np64(out)
        assert np.all(np.abs(got[:rows] - want) <= tol * 1.01 + half * np.abs(want) + 1e-30)
        assert np.all(got[rows:] == 9.0)                                   # rows past the last one stay as they were
        assert bool((out.as_strided((rows + 2, 3), (cols + 3, 1), cols) == 9.0).all())
    # ungathered rows: row r of A
    a2 = a[torch.from_numpy(gather).long().to(DEV)].contiguous()
    out2 = torch.empty((rows, cols), dtype=torch.bfloat16, device=DEV)
    M().moe_w4_gemm(a2, q, s, od, 0, G, rows, out2, swiglu=swiglu)
    assert torch.equal(out2, out[:rows])


@pytest.mark.parametrize("swiglu", [False, True])
@pytest.mark.parametrize("lens,N,K", [
    ([1] * 40, 16, 2080), ([1, 0] * 35, 272, 2080), ([3] * 20 + [100] + [1] * 20, 48, 2112), ([30, 0, 70, 1, 17] * 4, 544, 2080),
    ([2] * 300, 160, 96), ([600, 0, 3900], 32, 64), ([5] * 130 + [40] * 20, 96, 1056), ([33] * 9, 272, 8192)])
def test_w4_gemm_many_row_blocks(lens, N, K, swiglu):
    """More row blocks than get workgroups of their own: few and many weight tiles, fewer and more blocks than groups,
    groups of many blocks between groups of one and empty ones."""
    G = len(lens)
    offs = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    rows = int(offs[-1])
    say(f"w4_gemm {rows} rows in {G} groups N={N} K={K} swiglu={swiglu}")
    q, s = _weights(600 + K, G, N, K)
    src = 50
    a = I.gen_normal(601, (src, K), 1.0).to(DEV)
    gather = np.random.default_rng(602).integers(0, src, rows).astype(np.int32)
    want, tol = _reference(np64(a), decode(q, s), offs, gather, swiglu)
    out = torch.full((rows + 1, want.shape[1]), 9.0, device=DEV)
    M().moe_w4_gemm(a, q, s, torch.from_numpy(offs).to(DEV), 0, G, rows, out, a_rows=torch.from_numpy(gather).to(DEV),
                    swiglu=swiglu)
    got = np64(out)
    assert np.all(np.abs(got[:rows] - want) <= tol * 1.01 + 1e-30) and np.all(got[rows:] == 9.0)


def test_w4_gemm_group_range_and_tail():
    """A sub-range of the groups (rows relative to its first), and the last groups' f32 rows in their own output."""
    lens, N, K = [4, 0, 21, 3, 40, 6], 80, 192
    offs = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    rows = int(offs[-1])
    q, s = _weights(510, len(lens), N, K)
    w = decode(q, s)
    a = I.gen_normal(511, (rows, K), 1.0).to(DEV)
    od = torch.from_numpy(offs).to(DEV)
    want, tol = _reference(np64(a), w, offs, np.arange(rows), False)
    f, n = 2, 3
    m = int(offs[f + n] - offs[f])
    out = torch.empty((m, N), dtype=torch.float32, device=DEV)
    M().moe_w4_gemm(a, q, s, od, f, n, m, out)
    sl = slice(offs[f], offs[f + n])
    assert np.all(np.abs(np64(out) - want[sl]) <= tol[sl])
    for tails in (1, 2, 6):
        t0 = int(offs[len(lens) - tails])
        main = torch.full((max(t0, 1), N), 5.0, dtype=torch.bfloat16, device=DEV)
        tail = torch.empty((rows - t0, N), dtype=torch.float32, device=DEV)
        M().moe_w4_gemm(a, q, s, od, 0, len(lens), rows, main, out_tail=tail, tail_groups=tails)
        if t0:
            assert np.all(np.abs(np64(main) - want[:t0]) <= tol[:t0] + 2.0 ** -8 * np.abs(want[:t0]))
        assert np.all(np.abs(np64(tail) - want[t0:]) <= tol[t0:])


def test_w4_gemm_special_values():
    """A NaN group scale reaches its own output column only; a NaN or infinite activation its own row only; scale codes
    at both ends of the range; weights of zero."""
    N, K = 48, 128
    offs = torch.tensor([0, 3, 8], dtype=torch.int32, device=DEV)
    q, s = _weights(520, 2, N, K, uniform_scale=True)
    s[0, 5, 2] = 255
    s[1, 7, 0] = 0
    s[1, 8, 1] = 250
    q[1, 9] = 0
    a = I.gen_normal(521, (8, K), 1.0).to(DEV)
    a[6, 3] = float("nan")
    a[7, 9] = float("inf")
    out = torch.empty((8, N), dtype=torch.float32, device=DEV)
    M().moe_w4_gemm(a, q, s, offs, 0, 2, 8, out)
    o = out.cpu().numpy()
    assert np.isnan(o[:3, 5]).all() and not np.isnan(np.delete(o[:3], 5, 1)).any()
    assert np.isnan(o[6]).all() and not np.isfinite(o[7]).any()
    w, x = decode(q, s)[1], np64(a)[3:6]
    tol = (K / 4 + 3) * 2.0 ** -23 * (np.abs(x) @ np.abs(w).T)
    want = x @ w.T
    # one product sum under the scale 2^123 is -3.64e38, beyond the largest f32: the output holds -inf there
    far = np.abs(want) > np.finfo(np.float32).max
    assert np.all(far == np.isinf(o[3:6])) and np.all(np.sign(o[3:6][far]) == np.sign(want[far]))
    assert np.all(np.abs(o[3:6] - want)[~far] <= tol[~far]) and not o[3:6, 9].any()


def test_w4_gemm_many_groups_and_no_rows():
    """1024 groups, most of them empty; a call without rows writes nothing."""
    G, N, K = 1024, 32, 64
    lens = np.zeros(G, dtype=np.int64)
    lens[[0, 5, 511, 512, 1022, 1023]] = [1, 2, 40, 3, 1, 7]
    offs = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    rows = int(offs[-1])
    q, s = _weights(530, G, N, K)
    a = I.gen_normal(531, (rows, K), 1.0).to(DEV)
    out = torch.empty((rows, N), dtype=torch.float32, device=DEV)
    M().moe_w4_gemm(a, q, s, torch.from_numpy(offs).to(DEV), 0, G, rows, out)
    want, tol = _reference(np64(a), decode(q, s), offs, np.arange(rows), False)
    assert np.all(np.abs(np64(out) - want) <= tol)
    out.fill_(3.0)
    # offsets that claim more rows than m_total are held to it
    M().moe_w4_gemm(a, q, s, torch.from_numpy(offs).to(DEV), 0, G, 4, out)
    assert np.all(np.abs(np64(out[:4]) - want[:4]) <= tol[:4]) and bool((out[4:] == 3.0).all())
    out.fill_(3.0)
    M().moe_w4_gemm(a, q, s, torch.zeros(G + 1, dtype=torch.int32, device=DEV), 0, G, 5, out)
    M().moe_w4_gemm(a, q, s, torch.zeros(G + 1, dtype=torch.int32, device=DEV), 0, G, 0, out)
    assert bool((out == 3.0).all())


def test_w4_gemm_repeats_streams_and_capture():
    """The same bits on every call, on another stream, and from a graph replayed over changed inputs and offsets."""
    lens, N, K, src = [3, 0, 20, 1, 40], 64, 512, 30
    rows = sum(lens)
    offs = torch.from_numpy(np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)).to(DEV)
    q, s = _weights(540, len(lens), 2 * N, K)
    a = I.gen_normal(541, (src, K), 1.0).to(DEV)
    gat = torch.from_numpy(np.random.default_rng(1).integers(0, src, rows).astype(np.int32)).to(DEV)

    def go():
        h = torch.empty((rows, N), dtype=torch.bfloat16, device=DEV)
        return M().moe_w4_gemm(a, q, s, offs, 0, len(lens), rows, h, a_rows=gat, swiglu=True)

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
        a.copy_(I.gen_normal(550 + k, (src, K), 1.0))
        g.replay()
        ref = go()
        torch.cuda.synchronize()
        assert torch.equal(out, ref), k


def test_w4_gemm_refuses_short_tensors():
    q, s = _weights(560, 2, 32, 64)
    a = I.gen_normal(561, (4, 64), 1.0).to(DEV)
    offs = torch.tensor([0, 2, 4], dtype=torch.int32, device=DEV)
    out = torch.empty((4, 32), device=DEV)
    bad = (dict(m_total=5), dict(out=out[:3]), dict(a_rows=offs[:3]), dict(n_groups=3), dict(offs=offs[:2]), dict(out=out[:, :31]),
           dict(a=a[:, :32]), dict(s=s[:, :, :1].contiguous()), dict(tail_groups=1, out_tail=out[:0]), dict(out=out.double()),
           dict(a=a.float()), dict(a=a.t()))
    for kw in bad:
        c = dict(a=a, q=q, s=s, offs=offs, n_groups=2, m_total=4, out=out, a_rows=None, tail_groups=0, out_tail=None)
        c.update(kw)
        if "out_tail" in kw:
            c["out"] = out[:2]
        with pytest.raises((ValueError, TypeError)):
            M().moe_w4_gemm(c["a"], c["q"], c["s"], c["offs"], 0, c["n_groups"], c["m_total"], c["out"], a_rows=c["a_rows"],
                            tail_groups=c["tail_groups"], out_tail=c["out_tail"])


@pytest.mark.parametrize("swiglu", [False, True])
@pytest.mark.parametrize("N", [48, 50])
def test_w4_gemm_holds_to_its_tensors(N, swiglu):
    """Rows that a_rows, a, out or out_tail does not hold are neither read nor written, whatever the offsets say
    (streaming and general kernel): a sub-range of the groups with too few rows before it, and outputs that are long
    enough together but not each.  Every tensor is the head of a longer one, whose rest has to stay as it was."""
    lens, K = [4, 0, 21, 3, 40, 6], 192
    offs = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    rows, G, cols = int(offs[-1]), len(lens), N // 2 if swiglu else N
    q, s = _weights(590, G, N, K)
    a = I.gen_normal(591, (rows, K), 1.0).to(DEV)
    od, ident = torch.from_numpy(offs).to(DEV), torch.arange(rows, dtype=torch.int32, device=DEV)
    want, tol = _reference(np64(a), decode(q, s), offs, np.arange(rows), swiglu)

    def check(got, want, tol, n, half=0.0):
        g = np64(got)
        assert np.all(np.abs(g[:n] - want[:n]) <= (tol * 1.01 + half * np.abs(want))[:n] + 1e-30)
        assert np.all(g[n:] == 9.0)

    for have in (0, 3, 24, 27, 29, 69):  # sorted rows that are there; the range below is rows 4 to 68
        for kw in (dict(a_rows=ident[:have]), dict()):
            out = torch.full((64, cols), 9.0, device=DEV)
            M().moe_w4_gemm(a if kw else a[:have], q, s, od, 2, 3, 64, out, swiglu=swiglu, **kw)
            check(out, want[4:], tol[4:], min(max(have - 4, 0), 64))
    for tails in (1, 2, 6):
        t0 = int(offs[G - tails])
        for main in sorted({0, 1, t0 // 2, max(t0 - 1, 0), t0, t0 + 1, rows}):
            tail = rows - main
            out = torch.full((rows + 8, cols), 9.0, dtype=torch.bfloat16, device=DEV)
            rest = torch.full((rows + 8, cols), 9.0, device=DEV)
            M().moe_w4_gemm(a, q, s, od, 0, G, rows, out[:main], out_tail=rest[:tail], tail_groups=tails, swiglu=swiglu)
            check(out, want, tol, min(main, t0), 2.0 ** -8)
            check(rest, want[t0:], tol[t0:], 0 if main < t0 else min(tail, rows - t0))


def test_w4_gemm_two_streams_at_once():
    """Calls that run at the same time keep to themselves (the operator has no workspace)."""
    lens, N, K = [1, 0, 40, 3], 2048, 2048
    offs = torch.from_numpy(np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)).to(DEV)
    rows = sum(lens)
    ops = []
    for k in range(2):
        q, s = _weights(570 + k, len(lens), N, K)
        a = I.gen_normal(572 + k, (rows, K), 1.0).to(DEV)
        ref = torch.empty((rows, N), device=DEV)
        M().moe_w4_gemm(a, q, s, offs, 0, len(lens), rows, ref)
        ops.append((a, q, s, ref, torch.empty((rows, N), device=DEV), torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(10):
        for a, q, s, ref, out, st in ops:
            with torch.cuda.stream(st):
                M().moe_w4_gemm(a, q, s, offs, 0, len(lens), rows, out)
    torch.cuda.synchronize()
    for a, q, s, ref, out, st in ops:
        assert torch.equal(ref, out)


@pytest.mark.parametrize("fill", [0, 1, 254])
def test_w4_gemm_scale_ends(fill):
    """Every group at an end of the scale range.  Weights below 2^-126 are subnormal bf16 numbers; the activations are
    scaled so that the exact sums are ordinary f32 numbers."""
    N, K = 16, 64
    q, s = _weights(580, 1, N, K)
    s.fill_(fill)
    a = (I.gen_normal(581, (3, K), 1.0).float() * 2.0 ** (100 if fill < 2 else -100)).to(torch.bfloat16).to(DEV)
    offs = torch.tensor([0, 3], dtype=torch.int32, device=DEV)
    out = torch.empty((3, N), device=DEV)
    M().moe_w4_gemm(a, q, s, offs, 0, 1, 3, out)
    w = decode(q, s)
    # a weight of 4 or 6 times 2^127 is beyond bf16: infinite
    big = np.abs(w[0]) > 3.4e38
    w[0][big] = np.sign(w[0][big]) * np.inf
    with np.errstate(invalid="ignore"):
        want, tol = _reference(np64(a), w, [0, 3], np.arange(3), False)
    o = np64(out)
    fine = np.isfinite(want)
    assert np.array_equal(fine, np.isfinite(o))
    assert np.all(np.abs(o - want)[fine] <= tol[fine])


@pytest.mark.parametrize("N,K", [(48, 544), (50, 544), (32, 8192), (34, 8224)])
def test_w4_gemm_row_by_itself(N, K):
    """A row's result has the same bits alone and among other rows, in any group size (streaming and general kernel)."""
    q, s = _weights(520, 1, N, K)
    a = I.gen_normal(521, (40, K), 1.0).to(DEV)

    def go(x, swiglu):
        out = torch.empty((x.shape[0], N // 2 if swiglu else N), device=DEV)
        M().moe_w4_gemm(x, q, s, torch.tensor([0, x.shape[0]], dtype=torch.int32, device=DEV), 0, 1, x.shape[0], out,
                        swiglu=swiglu)
        return out

    for swiglu in (False, True):
        full = go(a, swiglu)
        for r in (0, 15, 16, 39):
            assert torch.equal(go(a[r:r + 1], swiglu)[0], full[r])
        assert torch.equal(go(a[:17], swiglu), full[:17])


def test_w4_gemm_many_weight_rows():
    """One token against 2^25 weight rows: the tiles of all workgroups together pass 32 bits in the products that deal
    them out.  Weights 1, inputs 1, K = 32: every output is 32 exactly."""
    N, K = 1 << 25, 32
    q = torch.full((1, N, K // 2), 0x22, dtype=torch.uint8, device=DEV)
    s = torch.full((1, N, 1), 127, dtype=torch.uint8, device=DEV)
    out = torch.zeros((1, N), dtype=torch.bfloat16, device=DEV)
    M().moe_w4_gemm(torch.ones((1, K), dtype=torch.bfloat16, device=DEV), q, s,
                    torch.tensor([0, 1], dtype=torch.int32, device=DEV), 0, 1, 1, out)
    assert bool((out == 32.0).all())


def test_layer_w4_no_tokens():
    cfg = I.small(I.V3_BF16, name="w4_empty", T=1, d=64, n_experts=8, top_k=2, inter=64)
    ex = [I.gen_expert(cfg, e) for e in range(cfg.groups)]
    W13, W2 = (torch.stack([e[k] for e in ex]).to(torch.bfloat16).to(DEV) for k in (0, 1))
    layer = M().MoELayer(I.gen_router(cfg).to(DEV), W13, W2, I.gen_bias(cfg).to(DEV), 2, w4=True, norm="layer")
    out = layer.forward(torch.empty((0, 64), dtype=torch.bfloat16, device=DEV))
    assert out.shape == (0, 64)


@pytest.mark.parametrize("T,norm", [(1, None), (1, "rms"), (5, None), (64, "layer")])
def test_layer_w4(T, norm):
    """MoELayer(w4=True) against the oracle on the dequantised weights: the bf16 path's bar (1e-2 of the RMS)."""
    cfg = I.small(I.V3_BF16, name="w4_layer", T=T, d=256, n_experts=16, top_k=4, inter=96, w_std=0.05, router_std=0.05, seed=9)
    ex = [I.gen_expert(cfg, e) for e in range(cfg.groups)]
    W13 = torch.stack([a for a, _ in ex]).to(torch.bfloat16)
    W2 = torch.stack([b for _, b in ex]).to(torch.bfloat16)
    wr, bias, x = I.gen_router(cfg), I.gen_bias(cfg), I.gen_x(cfg)
    nw = (1.0 + I.gen_normal(11, (cfg.d,), 0.1, torch.float32)).to(DEV) if norm else None
    layer = M().MoELayer(wr.to(DEV), W13.to(DEV), W2.to(DEV), bias.to(DEV), cfg.top_k, w4=True, norm=norm, norm_weight=nw)
    out, buf = layer.forward(x.to(DEV), out_dtype=torch.float32, keep=True)
    check_permutation_properties(buf["expert_offsets"], buf["sorted_token"], buf["pair_pos"], buf["topk_idx"], cfg.n_experts)
    u = x if norm is None else M().moe_norm(x.to(DEV), nw, rms=norm == "rms")[0].cpu()
    w13, w2 = decode(layer.W13, layer.W13_s), decode(layer.W2, layer.W2_s)
    r = O.route(u.double().numpy(), wr.double().numpy(), bias.numpy(), cfg.top_k)
    ok = r["margin"] >= 1e-6
    ref, _ = O.forward_sparse(u.double().numpy(), r["idx"], r["gate"], cfg.n_experts, lambda e: (w13[e], w2[e]), "bf16")
    err = rel_err(np64(out)[ok], ref[ok])
    say(f"  w4 layer T={T}: {err:.2e}")
    assert ok.any() and err <= 1e-2
    with pytest.raises(NotImplementedError):
        layer.forward(x.to(DEV), train=True)
    with pytest.raises(NotImplementedError):
        layer.forward(x.to(DEV), checkpoint=True)
    with pytest.raises(NotImplementedError):
        layer.backward(out, buf)


@pytest.mark.parametrize("T", [1, 6])
def test_layer_w4_captured(T):
    """A decode step of the layer (norm, routing, both 4-bit products, combine) in one graph, replayed over changed tokens
    with eager steps between the replays."""
    cfg = I.small(I.V3_BF16, name="w4_graph", T=T, d=256, n_experts=16, top_k=4, inter=96, w_std=0.05, router_std=0.05, seed=12)
    ex = [I.gen_expert(cfg, e) for e in range(cfg.groups)]
    W13 = torch.stack([a for a, _ in ex]).to(torch.bfloat16).to(DEV)
    W2 = torch.stack([b for _, b in ex]).to(torch.bfloat16).to(DEV)
    layer = M().MoELayer(I.gen_router(cfg).to(DEV), W13, W2, I.gen_bias(cfg).to(DEV), cfg.top_k, w4=True, norm="rms")
    x = I.gen_x(cfg).to(DEV)
    layer.forward(x)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = layer.forward(x)
    for k in range(4):
        x.copy_(I.gen_normal(570 + k, (T, cfg.d), 1.0))
        g.replay()
        ref = layer.forward(x)
        torch.cuda.synchronize()
        assert torch.equal(out, ref), k
