"""GPU parity of moe_norm and moe_norm_backward with the formulas in float64.

Tolerances.  u = 2^-24 is half a step of fp32.  A sum of a row is taken as at most 32 terms in a
lane, 6 exchanges and at most 16 waves: 54 roundings, so a mean is off by at most 54 u mean|x|, and
with the rounding of the scaling by 1/d and of x - mean by at most 56 u (mean|x| + |x - mean|); the
variance is off by a relative (54 + 4) u plus that of its terms, half of which reaches rstd, plus the
division and the square root.  Together xhat is off by at most 100 u (|xhat| + mean|x| rstd), y adds
two roundings, and a bf16 result half a bf16 step, 2^-8 of the value.
"""
import numpy as np
import pytest
import torch

from oracle import moe_oracle as O
from sparse_moe_layer_sigmoid_amd import inputs as I
from tests.gpu_common import np64, say

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
U = 2.0 ** -24
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 0.0}


def M():
    import sparse_moe_layer_sigmoid_amd as m
    return m


def _rows(seed, T, d, dtype, pad=0, offset=0.3):
    x = I.gen_normal(seed, (T, d + pad), 1.0, torch.float32) + offset
    return x.to(dtype).to(DEV)[:, :d]


def _vec(seed, d, dtype, mean=0.0):
    return (I.gen_normal(seed, (d,), 0.2, torch.float32) + mean).to(dtype).to(DEV)


def _ref_norm(x, w, b, eps, rms):
    mean = np.zeros((x.shape[0], 1)) if rms else x.mean(1, keepdims=True)
    rstd = 1.0 / np.sqrt(((x - mean) ** 2).mean(1, keepdims=True) + eps)
    xhat = (x - mean) * rstd
    y = xhat * (1.0 if w is None else w) + (0.0 if b is None else b)
    return mean[:, 0], rstd[:, 0], xhat, y


# d: one element, below / at / past a chunk, a wave, four chunks a lane, several waves; the layer's 7168; the limit
DS = [1, 3, 8, 65, 512, 513, 1000, 1024, 1025, 2048, 2055, 4096, 7168, 8200, 16384]


@pytest.mark.parametrize("rms", [False, True])
@pytest.mark.parametrize("d", DS)
def test_norm_forward(d, rms):
    for k, (T, xt, yt, wt, pad) in enumerate([(1, torch.bfloat16, torch.bfloat16, torch.bfloat16, 0),
                                              (7, torch.float32, torch.float32, torch.float32, 3),
                                              (5, torch.bfloat16, torch.float32, torch.float32, 5),
                                              (130, torch.float32, torch.bfloat16, torch.bfloat16, 8),
                                              # over 256 rows a lane holds more chunks of a row
                                              (257, torch.bfloat16, torch.bfloat16, torch.float32, 0),
                                              (300, torch.float32, torch.float32, torch.float32, 1)]):
        say(f"norm d={d} rms={rms} T={T} {xt}->{yt} pad={pad}")
        x = _rows(10 + k, T, d, xt, pad)
        w = _vec(20, d, wt, 1.0) if k != 2 else None
        b = _vec(21, d, wt) if k % 2 == 0 else None
        y, mean, rstd, ck = M().moe_norm(x, w, b, eps=1e-5, rms=rms, out_dtype=yt, want_stats=True)
        assert ck is None and y.dtype == yt and (mean is None) == rms
        x64 = np64(x)
        w64 = None if w is None else np64(w)
        m, r, xhat, ref = _ref_norm(x64, w64, None if b is None else np64(b), 1e-5, rms)
        ax = np.abs(x64).mean(1)
        if not rms:
            assert np.all(np.abs(np64(mean) - m) <= 56 * U * ax)
        # rstd alone: the 58 u of the sum, the rounding of x - mean (its offset enters squared), the last two steps
        assert np.all(np.abs(np64(rstd) - r) <= r * 100 * U * (1 + ax * r))
        aw = 1.0 if w64 is None else np.abs(w64)
        tol = 100 * U * (np.abs(xhat) + (ax * r)[:, None]) * aw + 3 * U * np.abs(ref) + HALF[yt] * np.abs(ref)
        assert np.all(np.abs(np64(y) - ref) <= tol + 1e-30)


def _ckpt_reference(x64):
    """Codes' values and scale codes of the 8-bit checkpoint, from the oracle's quantiser on zero-padded columns."""
    rows, cols = x64.shape
    n = (cols + 127) // 128
    p = np.zeros((rows, n * 128))
    p[:, :cols] = x64
    q, s = O.quant_1x128_e8m0(p)
    v = O.e4m3_decode(q).reshape(rows, n, 128) * np.exp2(s.astype(np.float64) - 127)[:, :, None]
    return q[:, :cols], s, v.reshape(rows, n * 128)[:, :cols]


@pytest.mark.parametrize("d", [1, 9, 127, 128, 129, 1000, 2055, 7168])
@pytest.mark.parametrize("rms", [False, True])
def test_norm_checkpoint(d, rms):
    """The checkpoint the norm writes: scale codes by the rule, values within the E4M3 half step of xhat (the
    device's fp32 xhat differs from float64 by at most the bound above, so a code may sit at the other side of
    a midpoint); y does not depend on it."""
    T = 33
    x = _rows(31, T, d, torch.bfloat16)
    w = _vec(32, d, torch.float32, 1.0)
    y, _, rstd, (q, s) = M().moe_norm(x, w, rms=rms, checkpoint=True)
    y2, _, _, none = M().moe_norm(x, w, rms=rms)
    assert none is None and rstd is not None and torch.equal(y, y2)
    x64 = np64(x)
    _, r, xhat, _ = _ref_norm(x64, None, None, 1e-6, rms)
    slack = 100 * U * (np.abs(xhat) + (np.abs(x64).mean(1) * r)[:, None])
    n = (d + 127) // 128
    got = np64(M().fp8_ckpt_unpack(q, s, out_dtype=torch.float32))
    k = s.cpu().numpy().astype(np.int64) - 127
    step = np.repeat(np.exp2(k), 128, axis=1)[:, :d]
    # half a step of E4M3 at the device's scale: 2^-4 of the value, 2^-10 of the scale below 2^-6 of it
    half = np.maximum(2.0 ** -4 * np.abs(xhat), 2.0 ** -10 * step)
    assert np.all(np.abs(got - xhat) <= half * (1 + 2.0 ** -10) + slack)
    pad = np.zeros((T, n * 128))
    pad[:, :d] = np.abs(xhat)
    amax = pad.reshape(T, n, 128).max(2)
    rel = 100 * U * (1 + np.abs(x64).mean(1) * r)[:, None] + 1e-12
    lo, hi = O.e8m0_exponent(amax * (1 - rel)), O.e8m0_exponent(amax * (1 + rel))
    assert np.all((k >= np.minimum(lo, hi)) & (k <= np.maximum(lo, hi)))


def _ref_backward(dy, xhat, rstd, w, rms):
    g = dy * (1.0 if w is None else w)
    m1 = 0.0 if rms else g.mean(1, keepdims=True)
    m2 = (g * xhat).mean(1, keepdims=True)
    return g, rstd[:, None] * (g - m1 - xhat * m2), (dy * xhat).sum(0), dy.sum(0)


def _check_backward(got, dy, xhat, rstd, w, rms, odt, T, slack):
    """slack: what xhat may be off by.  dx: two sums of at most 38 roundings, four products and differences; dw: a
    chain of the rows of one workgroup (256 workgroups or more once T is: T / 256 + 1 rows), then of the partial rows
    (at most 512 for these T) in 16 strips, and of the strips.  Rows of up to 1024 columns: R = 64, 32, 16 or 8 rows to a
    workgroup, a lane's chain of T / (256 R) + 1 rows, then R sums, at most 512 partial rows and the strips."""
    dx, dw, db = got
    g, rdx, rdw, rdb = _ref_backward(dy, xhat, rstd, w, rms)
    s1 = np.abs(g).mean(1, keepdims=True)
    s2 = np.abs(g * xhat).mean(1, keepdims=True)
    sx = (np.abs(g) * slack).mean(1, keepdims=True)
    tol = rstd[:, None] * (48 * U * (np.abs(g) + s1 + np.abs(xhat) * s2) + np.abs(xhat) * sx + slack * s2)
    assert np.all(np.abs(np64(dx) - rdx) <= tol + HALF[odt] * np.abs(rdx) + 1e-30)
    d = dy.shape[1]
    R = 64 if d <= 128 else 32 if d <= 256 else 16 if d <= 512 else 8 if d <= 1024 else 1
    assert T <= 4096 or R > 1
    chain = (T / (256 * R) + 1) + (R if R > 1 else 0) + min(T, 512) / 16 + 1 + 16
    assert np.all(np.abs(np64(dw) - rdw) <= chain * U * np.abs(dy * xhat).sum(0) + (np.abs(dy) * slack).sum(0) + 1e-30)
    if db is not None:
        assert np.all(np.abs(np64(db) - rdb) <= chain * U * np.abs(dy).sum(0) + 1e-30)


@pytest.mark.parametrize("rms", [False, True])
@pytest.mark.parametrize("d", DS)
def test_norm_backward(d, rms):
    for k, (T, xt, gt, odt, pad) in enumerate([(1, torch.bfloat16, torch.bfloat16, torch.bfloat16, 0),
                                               (40, torch.float32, torch.float32, torch.float32, 3),
                                               (5, torch.bfloat16, torch.float32, torch.float32, 0),
                                               (600, torch.float32, torch.bfloat16, torch.float32, 1)]):
        if T * d > 4_000_000:
            T = 4_000_000 // d
        say(f"norm backward d={d} rms={rms} T={T} {xt} {gt}->{odt} pad={pad}")
        x = _rows(40 + k, T, d, xt, pad)
        dy = _rows(50 + k, T, d, gt, pad, offset=0.01)
        w = _vec(60, d, torch.float32, 1.0) if k != 2 else None
        _, mean, rstd, _ = M().moe_norm(x, w, rms=rms, want_stats=True)
        got = M().moe_norm_backward(dy, x, mean, rstd, w, rms=rms, want_dbias=k != 3, out_dtype=odt)
        r64 = np64(rstd)
        m64 = np.zeros(T) if rms else np64(mean)
        xhat = (np64(x) - m64[:, None]) * r64[:, None]
        slack = 2 * U * np.abs(xhat)  # the difference and the product
        _check_backward(got, np64(dy), xhat, r64, None if w is None else np64(w), rms, odt, T, slack)


@pytest.mark.parametrize("rms", [False, True])
@pytest.mark.parametrize("T,d", [(1, 128), (15, 64), (65, 120), (64, 129), (33, 256), (31, 250), (17, 257), (16, 511), (20001, 100),
                                 (16385, 128), (9000, 200), (8193, 256), (5000, 400), (4097, 512), (1, 513), (9, 1024), (25, 1000), (4100, 640), (4097, 1024),
                                 (4200, 1001)])
def test_norm_narrow(T, d, rms):
    """Rows of up to 512 (backward: 1024) columns, several to a workgroup: short last workgroups, more rows than the
    backward's workgroups take at once; the checkpoint is that of packing the f32 rows the norm gives without weights."""
    say(f"norm narrow T={T} d={d} rms={rms}")
    x = _rows(61, T, d, torch.bfloat16, 2)
    dy = _rows(62, T, d, torch.float32, 0, offset=0.01)
    w = _vec(63, d, torch.float32, 1.0)
    b = _vec(64, d, torch.float32)
    y, mean, rstd, _ = M().moe_norm(x, w, b, eps=1e-5, rms=rms, out_dtype=torch.float32, want_stats=True)
    xhat32, _, _, ck = M().moe_norm(x, eps=1e-5, rms=rms, out_dtype=torch.float32, checkpoint=True)
    x64, r64 = np64(x), np64(rstd)
    m, r, xhat, ref = _ref_norm(x64, np64(w), np64(b), 1e-5, rms)
    ax = np.abs(x64).mean(1)
    tol = 100 * U * (np.abs(xhat) + (ax * r)[:, None]) * np.abs(np64(w)) + 3 * U * np.abs(ref)
    assert np.all(np.abs(np64(y) - ref) <= tol + 1e-30)
    assert np.all(np.abs(r64 - r) <= r * 100 * U * (1 + ax * r))
    for got, want in zip(ck, M().fp8_ckpt_pack(xhat32)):
        assert torch.equal(got, want)
    got = M().moe_norm_backward(dy, x, mean, rstd, w, rms=rms, want_dbias=True)
    xh = (x64 - (0.0 if rms else np64(mean)[:, None])) * r64[:, None]
    _check_backward(got, np64(dy), xh, r64, np64(w), rms, torch.float32, T, 2 * U * np.abs(xh))
    got = M().moe_norm_backward(dy, None, None, rstd, w, rms=rms, checkpoint=ck, want_dbias=True)
    xh = np64(M().fp8_ckpt_unpack(*ck, out_dtype=torch.float32))
    _check_backward(got, np64(dy), xh, r64, np64(w), rms, torch.float32, T, 0.0 * xh)


@pytest.mark.parametrize("rms", [False, True])
@pytest.mark.parametrize("T,d", [(8208, 2048), (16384, 2048), (9001, 3001), (33000, 1025), (16400, 1500), (8192, 4100)])
def test_norm_backward_many_partial_rows(T, d, rms):
    """Rows wider than 1024 in batches whose workgroups walk 16 rows or more: up to 2048 partial rows of dw and db.  A
    lane's chain of T / n + 1 rows, then n / 16 + 1 partial rows to a strip and 16 strips; from x and from the checkpoint,
    against sums in float64 (of the stored statistics' xhat)."""
    n = M().lib().moe_norm_backward_workspace_size(T, d) // (8 * d)
    say(f"norm backward {T} x {d} rms={rms}: {n} partial rows")
    assert n > 256
    x = _rows(65, T, d, torch.bfloat16)
    dy = _rows(66, T, d, torch.float32, 0, offset=0.01)
    w = _vec(67, d, torch.float32, 1.0)
    _, mean, rstd, ck = M().moe_norm(x, w, rms=rms, want_stats=True, checkpoint=True)
    g64, r64, w64 = dy.double(), rstd.double()[:, None], w.double()
    chain = T / n + 1 + n / 16 + 1 + 16
    for kind in ("x", "checkpoint"):
        if kind == "x":
            got = M().moe_norm_backward(dy, x, mean, rstd, w, rms=rms, want_dbias=True)
            xh = (x.double() - (0.0 if rms else mean.double()[:, None])) * r64
            slack = 2 * U * xh.abs()  # the difference and the product
        else:
            got = M().moe_norm_backward(dy, None, None, rstd, w, rms=rms, checkpoint=ck, want_dbias=True)
            xh = M().fp8_ckpt_unpack(*ck, out_dtype=torch.float32).double()
            slack = 0.0 * xh
        dx, dw, db = (t.double() for t in got)
        assert bool(((dw - (g64 * xh).sum(0)).abs() <= chain * U * (g64 * xh).abs().sum(0) + (g64.abs() * slack).sum(0)).all())
        assert bool(((db - g64.sum(0)).abs() <= chain * U * g64.abs().sum(0)).all())
        g = g64 * w64
        s1, s2, sx = g.abs().mean(1, keepdim=True), (g * xh).abs().mean(1, keepdim=True), (g.abs() * slack).mean(1, keepdim=True)
        want = r64 * (g - (0.0 if rms else g.mean(1, keepdim=True)) - xh * (g * xh).mean(1, keepdim=True))
        tol = r64 * (48 * U * (g.abs() + s1 + xh.abs() * s2) + xh.abs() * sx + slack * s2)
        assert bool(((dx - want).abs() <= tol).all())


@pytest.mark.parametrize("d", [1, 9, 130, 1024, 7168, 8200])
@pytest.mark.parametrize("rms", [False, True])
def test_norm_backward_from_checkpoint(d, rms):
    T = 70
    x = _rows(71, T, d, torch.bfloat16)
    w = _vec(72, d, torch.bfloat16, 1.0)
    for gt in (torch.bfloat16, torch.float32):
        dy = _rows(73, T, d, gt, 0, offset=0.01)
        _, _, rstd, ck = M().moe_norm(x, w, rms=rms, checkpoint=True)
        got = M().moe_norm_backward(dy, None, None, rstd, w, rms=rms, checkpoint=ck, want_dbias=True, out_dtype=torch.float32)
        xhat = np64(M().fp8_ckpt_unpack(*ck, out_dtype=torch.float32))
        _check_backward(got, np64(dy), xhat, np64(rstd), np64(w), rms, torch.float32, T, 0.0 * xhat)


@pytest.mark.parametrize("rms", [False, True])
def test_norm_backward_against_differences(rms):
    """The analytic gradient against central differences of the float64 definition: L = sum(c * norm(x)); a step of
    2^-16 leaves a truncation below 1e-8 of the third derivative's scale, far under the fp32 bound used."""
    T, d = 3, 24
    x = _rows(81, T, d, torch.float32)
    w, b = _vec(82, d, torch.float32, 1.0), _vec(83, d, torch.float32)
    c = _rows(84, T, d, torch.float32)
    _, mean, rstd, _ = M().moe_norm(x, w, b, rms=rms, want_stats=True)
    dx, dw, db = M().moe_norm_backward(c, x, mean, rstd, w, rms=rms, want_dbias=True)
    x64, w64, b64, c64 = np64(x), np64(w), np64(b), np64(c)

    def loss(xx, ww, bb):
        return (c64 * _ref_norm(xx, ww, bb, 1e-6, rms)[3]).sum()

    h = 2.0 ** -16

    def diff(f, v):
        out = np.zeros_like(v)
        for i in np.ndindex(v.shape):
            p, n = v.copy(), v.copy()
            p[i] += h
            n[i] -= h
            out[i] = (f(p) - f(n)) / (2 * h)
        return out

    for got, want in ((dx, diff(lambda v: loss(v, w64, b64), x64)), (dw, diff(lambda v: loss(x64, v, b64), w64)),
                      (db, diff(lambda v: loss(x64, w64, v), b64))):
        assert np.max(np.abs(np64(got) - want)) <= 200 * U * np.abs(want).max() * d + 1e-8


def test_norm_constant_and_extreme_rows():
    """Constant rows (zero variance: rstd = eps^-1/2 and xhat of the size of the mean's rounding), zero rows, rows of
    1e18 (squares of 1e36 still finite), rows with an infinity or NaN, which stay in their row."""
    d = 1000
    x = torch.zeros((6, d))
    x[1] = 3.0
    x[2] = I.gen_normal(91, (d,), 1e18, torch.float32)
    x[3] = I.gen_normal(92, (d,), 1.0, torch.float32)
    x[4] = x[3]
    x[4, 17] = float("nan")
    x[5] = x[3]
    x[5, 999] = float("inf")
    y, mean, rstd, _ = M().moe_norm(x.to(DEV), eps=1e-6, want_stats=True)
    y, rstd = y.cpu(), rstd.cpu()
    assert torch.equal(y[0], torch.zeros(d))
    assert abs(float(rstd[0]) - 1e3) <= 1e3 * 4 * U
    assert y[1].abs().max() <= 56 * U * 3.0 * 1e3
    ref = _ref_norm(np64(x[2:4]), None, None, 1e-6, False)[3]
    assert np.all(np.abs(np64(y[2:4]) - ref) <= 100 * U * (np.abs(ref) + 1.0) + 3 * U * np.abs(ref))
    assert torch.isnan(y[4]).all() and torch.isnan(y[5]).all()


def test_norm_large_constant_rows():
    """Rows of 2^120: their sum passes the largest float although the mean does not (1024 columns), and the mean times
    rstd does too, which must not reach the chunk's lanes past the row (4 columns).  All exact: the mean is 2^120, xhat 0,
    rstd eps^-1/2, so dx = rstd (g - mean g) and dweight 0."""
    for d in (1024, 4):
        x = torch.full((3, d), 2.0 ** 120, device=DEV)
        dy = I.gen_normal(93, (3, d), 1.0, torch.float32).to(DEV)
        y, mean, rstd, _ = M().moe_norm(x, eps=1e-6, want_stats=True)
        assert torch.equal(y, torch.zeros_like(y)) and torch.equal(mean, x[:, 0])
        assert bool(((rstd - 1e3).abs() <= 1e3 * 4 * U).all())
        dx, dw, db = M().moe_norm_backward(dy, x, mean, rstd, want_dbias=True)
        g = np64(dy)
        want = np64(rstd)[:, None] * (g - g.mean(1, keepdims=True))
        assert np.all(np.abs(np64(dx) - want) <= 100 * U * 1e3 * (np.abs(g) + np.abs(g).mean(1, keepdims=True)))
        assert torch.equal(dw, torch.zeros(d, device=DEV))
        assert np.all(np.abs(np64(db) - g.sum(0)) <= 3 * U * np.abs(g).sum(0))


@pytest.mark.parametrize("eps", [0.0, 1e-6, 2.0 ** -100, 1e20])
@pytest.mark.parametrize("rms", [False, True])
@pytest.mark.parametrize("d", [4, 64, 129, 300, 512, 600, 1000, 1024, 2055, 7168, 16384])
def test_norm_rows_of_any_magnitude(d, rms, eps):
    """Rows of 2^e whose squares leave the float range, between ordinary ones: against float64 within the bounds above, to
    which come half steps of the smallest subnormal, 2^-150, for each of at most 54 roundings of a sum (of x where the row
    is taken as it is, of x / max|x| where it is scaled) and for the output.  rstd is held as f32, so a row of subnormals
    without eps has an infinite one, although its y does not; a row that rounds to zeros, without eps, is 0 / 0.  The ordinary rows' bits do not depend on the others."""
    exps = [-140, -127, -120, -100, -75, -70, -65, -60, -50, -45, -36, 30, 55, 59, 61, 63, 64, 66, 80, 100, 125]
    base = torch.clamp(I.gen_normal(85, (2 * len(exps), d), 1.0, torch.float32), -3.9, 3.9) + 0.05
    scale = torch.ones(2 * len(exps), dtype=torch.float64)
    scale[1::2] = torch.exp2(torch.tensor(exps, dtype=torch.float64))
    for times, xt in ((1, torch.float32), (1, torch.bfloat16), (7, torch.float32), (7, torch.bfloat16)):
        say(f"norm magnitudes d={d} rms={rms} eps={eps} rows={2 * len(exps) * times} {xt}")
        plain = base.repeat(times, 1).to(xt).to(DEV)
        x = (base.double() * scale[:, None]).float().repeat(times, 1).to(xt).to(DEV)
        y, mean, rstd, _ = M().moe_norm(x, eps=eps, rms=rms, out_dtype=torch.float32, want_stats=True)
        q, s = M().moe_norm(x, eps=eps, rms=rms, out_dtype=torch.bfloat16, checkpoint=True)[3]
        x64 = np64(x)
        e32 = float(np.float32(eps))
        with np.errstate(divide="ignore", invalid="ignore"):
            m, r, xhat, _ = _ref_norm(x64, None, None, e32, rms)
        ax, top = np.abs(x64).mean(1), np.abs(x64).max(1)
        small = 2.0 ** -142
        if not rms:
            assert np.all(np.abs(np64(mean) - m) <= 56 * U * ax + small * np.maximum(top, 1.0))
        r1, fine, held = np64(rstd), np.isfinite(r), r < 2.0 ** 127.9
        assert np.all(np.abs(r1[held] - r[held]) <= r[held] * 100 * U * (1 + (ax * r)[held]) + 2.0 ** -149)
        assert np.all(r1[~held] > 2.0 ** 127)
        y64 = np64(y)
        assert np.isnan(y64[~fine]).all() and not x64[~fine].any() and (~fine).sum() <= times
        y64, xhat, r, ax, top = y64[fine], xhat[fine], r[fine], ax[fine], top[fine]
        tol = 100 * U * (np.abs(xhat) + (ax * r)[:, None]) + (small * r * np.maximum(top, 1.0))[:, None] + 2.0 ** -148
        assert np.all(np.abs(y64 - xhat) <= tol)
        for got, want in zip((q, s), M().fp8_ckpt_pack(y)):
            assert torch.equal(got, want)
        y1, mean1, rstd1, _ = M().moe_norm(plain, eps=eps, rms=rms, out_dtype=torch.float32, want_stats=True)
        assert torch.equal(y[::2], y1[::2]) and torch.equal(rstd[::2], rstd1[::2])
        assert rms or torch.equal(mean[::2], mean1[::2])


@pytest.mark.parametrize("rms", [False, True])
@pytest.mark.parametrize("d", [300, 1000, 2055])
def test_norm_special_rows_without_eps(d, rms):
    """eps = 0: a row of zeros is 0 times infinity; an infinity makes NaN of itself (layer norm: of its row), NaN of its
    row; huge and tiny rows beside them are as by themselves."""
    x = I.gen_normal(86, (6, d), 1.0, torch.float32)
    x[1] = 0.0
    x[2, 3] = float("inf")
    x[3, d - 1] = float("nan")
    x[4] *= 1e30
    x[5] *= 1e-30
    y, _, rstd, _ = M().moe_norm(x.to(DEV), eps=0.0, rms=rms, want_stats=True)
    y, rstd = y.cpu(), rstd.cpu()
    assert torch.isnan(y[1]).all() and rstd[1] == float("inf") and torch.isnan(y[3]).all()
    if rms:
        assert rstd[2] == 0 and torch.isnan(y[2, 3]) and not y[2][torch.arange(d) != 3].any()
    else:
        assert torch.isnan(y[2]).all()
    rows = x[[0, 4, 5]]
    m, r, xhat, _ = _ref_norm(np64(rows), None, None, 0.0, rms)
    ax = np.abs(np64(rows)).mean(1)
    assert np.all(np.abs(np64(y[[0, 4, 5]]) - xhat) <= 100 * U * (np.abs(xhat) + (ax * r)[:, None]))


@pytest.mark.parametrize("rms", [False, True])
@pytest.mark.parametrize("e", [-100, -60, 61, 100])
def test_norm_backward_of_any_magnitude(e, rms):
    """The backward of such rows, from x and from the checkpoint (dw and db are of ordinary size; dx is about 2^-e)."""
    T, d = 20, 1000
    x = (I.gen_normal(87, (T, d), 1.0, torch.float32).double() * 2.0 ** e).float().to(DEV)
    dy = _rows(88, T, d, torch.float32, 0, offset=0.01)
    w = _vec(89, d, torch.float32, 1.0)
    _, mean, rstd, ck = M().moe_norm(x, w, eps=0.0, rms=rms, want_stats=True, checkpoint=True)
    r64 = np64(rstd)
    xh = (np64(x) - (0.0 if rms else np64(mean)[:, None])) * r64[:, None]
    got = M().moe_norm_backward(dy, x, mean, rstd, w, rms=rms, want_dbias=True)
    _check_backward(got, np64(dy), xh, r64, np64(w), rms, torch.float32, T, 2 * U * np.abs(xh))
    got = M().moe_norm_backward(dy, None, None, rstd, w, rms=rms, checkpoint=ck, want_dbias=True)
    xh = np64(M().fp8_ckpt_unpack(*ck, out_dtype=torch.float32))
    _check_backward(got, np64(dy), xh, r64, np64(w), rms, torch.float32, T, 0.0 * xh)


def test_norm_one_row_of_any_stride():
    """One row has no row stride: a transposed column and a row of an expanded tensor are taken like any other."""
    d = 72
    col = _vec(94, d, torch.float32).reshape(d, 1)
    row = col.t()                                                          # strides (1, 1)
    plain = col.reshape(1, d).clone()
    assert row.stride(0) == 1
    y, mean, rstd, ck = M().moe_norm(plain, want_stats=True, checkpoint=True)
    for x in (row, plain.expand(4, d)[:1]):
        y1, mean1, rstd1, ck1 = M().moe_norm(x, want_stats=True, checkpoint=True)
        assert torch.equal(y, y1) and torch.equal(ck[0], ck1[0]) and torch.equal(ck[1], ck1[1])
        for a, b in zip(M().moe_norm_backward(x, x, mean, rstd), M().moe_norm_backward(plain, plain, mean, rstd)):
            assert (a is None and b is None) or torch.equal(a, b)
        assert all(torch.equal(a, b) for a, b in zip(M().fp8_ckpt_pack(x), M().fp8_ckpt_pack(plain)))


def test_norm_no_rows_and_untouched_neighbours():
    d = 72
    x = torch.empty((0, d), device=DEV)
    y, mean, rstd, ck = M().moe_norm(x, want_stats=True, checkpoint=True)
    assert y.shape == (0, d) and ck[0].shape == (0, d) and mean.shape == (0,)
    dx, dw, db = M().moe_norm_backward(x, x, mean, rstd, want_dbias=True)
    assert dx.shape == (0, d) and torch.equal(dw, torch.zeros(d, device=DEV)) and torch.equal(db, torch.zeros(d, device=DEV))
    # a strided output of the C call leaves the columns between its rows as they were
    L = M()._lib
    T, wide = 5, 100
    x = _rows(95, T, d, torch.float32)
    out = torch.full((T, wide), 7.0, device=DEV)
    L._launch(x.device, "moe_norm", L._ptr(x), 1, d, None, None, 1, T, d, 1e-6, 0, L._ptr(out), 1, wide, None, None, None, None)
    assert torch.equal(out[:, d:], torch.full((T, wide - d), 7.0, device=DEV))
    assert torch.equal(out[:, :d], M().moe_norm(x)[0])


def test_norm_repeats_and_streams():
    """The same call twice gives the same bits (also dw, whose partial sums are added in a fixed order), on another
    stream too."""
    T, d = 1500, 1032
    x = _rows(96, T, d, torch.bfloat16)
    dy = _rows(97, T, d, torch.bfloat16, offset=0.0)
    w = _vec(98, d, torch.float32, 1.0)

    def go():
        y, mean, rstd, ck = M().moe_norm(x, w, want_stats=True, checkpoint=True)
        return (y, mean, rstd, *ck, *M().moe_norm_backward(dy, x, mean, rstd, w, want_dbias=True))

    a = go()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        b = go()
    torch.cuda.current_stream().wait_stream(s)
    c = go()
    for p, q, r in zip(a, b, c):
        assert torch.equal(p, q) and torch.equal(p, r)


def test_norm_captured():
    """Forward and backward in one graph, replayed over changed inputs with eager work between."""
    T, d = 300, 520
    x = _rows(99, T, d, torch.bfloat16).contiguous()
    dy = _rows(100, T, d, torch.float32, offset=0.0).contiguous()
    w = _vec(101, d, torch.float32, 1.0)

    def go():
        y, mean, rstd, ck = M().moe_norm(x, w, want_stats=True, checkpoint=True)
        return (y, mean, rstd, *ck, *M().moe_norm_backward(dy, None, None, rstd, w, checkpoint=ck, want_dbias=True))

    go()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = go()
    for k in range(4):
        x.copy_(_rows(110 + k, T, d, torch.bfloat16))
        dy.copy_(_rows(120 + k, T, d, torch.float32))
        g.replay()
        ref = go()
        torch.cuda.synchronize()
        for p, q in zip(out, ref):
            assert torch.equal(p, q), k
