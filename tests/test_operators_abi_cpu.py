"""Refusals of the norm, 8-bit checkpoint and 4-bit weight calls without a GPU: the C ABI checks its arguments before
anything is launched, the binding checks tensors before the C call."""
import ctypes
import os

import pytest
import torch


def _lib():
    from sparse_moe_layer_sigmoid_amd import _lib as L
    if not os.path.exists(L.LIB_PATH):
        pytest.skip("libmoe.so not built")
    return L


P = lambda v: None if v is None else ctypes.c_void_p(v)  # noqa: E731


def _expect(L, fn, args, code):
    st = getattr(L.lib(), fn)(*args)
    assert st == code, (fn, args, st, L.lib().moe_last_error())
    assert L.lib().moe_last_error().decode().startswith(fn)


def _norm(**kw):
    a = dict(x=16, xt=0, ldx=64, w=16, b=16, wt=1, rows=4, d=64, eps=1e-6, kind=0, y=16, yt=0, ldy=64, mean=16, rstd=16, q=16,
             s=16)
    a.update(kw)
    return (P(a["x"]), a["xt"], a["ldx"], P(a["w"]), P(a["b"]), a["wt"], a["rows"], a["d"], a["eps"], a["kind"], P(a["y"]),
            a["yt"], a["ldy"], P(a["mean"]), P(a["rstd"]), P(a["q"]), P(a["s"]), None)


@pytest.mark.parametrize("kw,code", [
    (dict(x=None), 1), (dict(y=None), 1), (dict(q=None), 1), (dict(s=None), 1), (dict(xt=2), 3), (dict(yt=2), 3),
    (dict(wt=5), 3), (dict(kind=2), 3), (dict(rows=-1), 2), (dict(d=0), 2), (dict(d=16385, ldx=16385, ldy=16385), 2),
    (dict(eps=-1.0), 2), (dict(eps=float("nan")), 2), (dict(eps=float("inf")), 2), (dict(ldx=63), 4), (dict(ldy=63), 4),
    (dict(x=17), 4), (dict(y=17), 4), (dict(w=18), 4), (dict(rstd=18), 4),
])
def test_norm_rejects(kw, code):
    L = _lib()
    _expect(L, "moe_norm", _norm(**kw), code)


def _norm_bwd(**kw):
    a = dict(dy=16, dyt=1, lddy=64, x=16, xt=0, ldx=64, q=None, s=None, mean=16, rstd=16, w=16, wt=1, rows=4, d=64, kind=0,
             dx=16, dxt=1, lddx=64, dw=16, db=16, ws=16, wsb=1 << 20)
    a.update(kw)
    return (P(a["dy"]), a["dyt"], a["lddy"], P(a["x"]), a["xt"], a["ldx"], P(a["q"]), P(a["s"]), P(a["mean"]), P(a["rstd"]),
            P(a["w"]), a["wt"], a["rows"], a["d"], a["kind"], P(a["dx"]), a["dxt"], a["lddx"], P(a["dw"]), P(a["db"]),
            P(a["ws"]), a["wsb"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(dy=None), 1), (dict(rstd=None), 1), (dict(dx=None), 1), (dict(x=None), 1), (dict(q=16), 1), (dict(q=16, s=16), 1),
    (dict(mean=None), 1), (dict(dyt=2), 3), (dict(xt=7), 3), (dict(dxt=2), 3), (dict(wt=2), 3), (dict(kind=-1), 3),
    (dict(rows=-2), 2), (dict(d=20000, lddy=20000, ldx=20000, lddx=20000), 2), (dict(lddy=60), 4), (dict(ldx=60), 4),
    (dict(lddx=60), 4), (dict(dy=18), 4), (dict(x=17), 4), (dict(dw=18), 4), (dict(rows=100, ws=None), 5),
    (dict(rows=100, wsb=100), 5), (dict(rows=100, ws=8), 5),
])
def test_norm_backward_rejects(kw, code):
    L = _lib()
    _expect(L, "moe_norm_backward", _norm_bwd(**kw), code)


def test_norm_backward_workspace_size():
    L = _lib()
    f = L.lib().moe_norm_backward_workspace_size
    assert f(0, 64) == 0 and f(-1, 64) == 0 and f(4, 0) == 0 and f(4, 16385) == 0
    assert f(1, 64) == 0 and f(1, 7168) == 0 and f(65, 64) == 2 * 2 * 64 * 4 and f(5, 2000) == 2 * 5 * 2000 * 4
    assert f(1 << 20, 7168) == f(1 << 21, 7168) > 0


def test_checkpoint_calls_reject():
    L = _lib()
    pk = lambda x=16, xt=1, rows=4, cols=100, ldx=100, q=16, s=16: (P(x), xt, rows, cols, ldx, P(q), P(s), None)  # noqa: E731
    for kw, code in ((dict(x=None), 1), (dict(s=None), 1), (dict(xt=2), 3), (dict(rows=-1), 2), (dict(cols=0), 2),
                     (dict(cols=(1 << 24) + 1, ldx=1 << 25), 2), (dict(ldx=99), 4), (dict(x=18), 4),
                     (dict(rows=1 << 40, cols=1), 2)):
        _expect(L, "fp8_ckpt_pack", pk(**kw), code)
    un = lambda q=16, s=16, rows=4, cols=100, w=None, b=None, wt=1, o=16, ot=0, ldo=100: (  # noqa: E731
        P(q), P(s), rows, cols, P(w), P(b), wt, P(o), ot, ldo, None)
    for kw, code in ((dict(q=None), 1), (dict(o=None), 1), (dict(ot=2), 3), (dict(wt=2), 3), (dict(cols=0), 2),
                     (dict(rows=-1), 2), (dict(ldo=50), 4), (dict(o=17), 4), (dict(w=18), 4), (dict(b=18), 4)):
        _expect(L, "fp8_ckpt_unpack", un(**kw), code)
    sw = lambda q=16, s=16, dh=16, rows=4, inter=64, dac=16, dq=None, ds=None, h=16: (  # noqa: E731
        P(q), P(s), P(dh), rows, inter, P(dac), P(dq), P(ds), P(h), None)
    for kw, code in ((dict(q=None), 1), (dict(s=None), 1), (dict(dh=None), 1), (dict(dac=None), 1), (dict(dq=16), 1),
                     (dict(rows=-1), 2), (dict(inter=6), 2), (dict(inter=0), 2), (dict(dq=16, ds=16), 2), (dict(q=8), 4),
                     (dict(dh=8), 4), (dict(dac=8), 4), (dict(h=8), 4)):
        _expect(L, "moe_swiglu_backward_ckpt", sw(**kw), code)
    cb = lambda o=16, q=16, s=16, T=4, K=2, d=16, N=8, dy=16, dq=None, ds=None: (  # noqa: E731
        P(o), P(q), P(s), P(16), P(16), P(16), P(16), T, K, d, N, P(dy), P(16), P(16), P(dq), P(ds), None)
    for kw, code in ((dict(o=None), 1), (dict(s=None), 1), (dict(dq=16), 1), (dict(T=-1), 2), (dict(K=0), 2),
                     (dict(K=33, N=64), 2), (dict(K=9), 2), (dict(d=12), 2), (dict(d=64, dq=16, ds=16), 2), (dict(q=4), 4),
                     (dict(dy=8), 4)):
        _expect(L, "moe_combine_backward_ckpt", cb(**kw), code)


def test_w4_quant_rejects():
    L = _lib()
    for args, code in (((None, 1, 4, 32, P(16), P(16)), 1), ((P(16), 1, 4, 33, P(16), P(16)), 2),
                       ((P(16), 1, 0, 32, P(16), P(16)), 2), ((P(16), -1, 4, 32, P(16), P(16)), 2),
                       ((P(8), 1, 4, 32, P(16), P(16)), 4), ((P(16), 1, 4, 0, P(16), P(16)), 2)):
        _expect(L, "w4_quant", (*args, None), code)


@pytest.mark.parametrize("kw,code", [
    (dict(a=None), 1), (dict(w_q=None), 1), (dict(w_scale=None), 1), (dict(group_offsets=None), 1), (dict(out=None), 1),
    (dict(epilogue=2), 3), (dict(out_dtype=2), 3), (dict(n_groups=0), 2), (dict(n_groups=1025), 2), (dict(first_group=-1), 2),
    (dict(m_total=-1), 2), (dict(m_total=1 << 31), 2), (dict(K=48), 2), (dict(K=0), 2), (dict(N=0), 2),
    (dict(N=31, epilogue=1), 2), (dict(tail_groups=5), 2), (dict(tail_groups=-1), 2), (dict(lda=32), 4), (dict(lda=68), 4),
    (dict(a=8), 4), (dict(w_q=8), 4), (dict(ldo=31), 4), (dict(out=18, out_dtype=1), 4), (dict(tail_groups=1), 1),
    (dict(tail_groups=1, out_tail=16, ldo_tail=31), 4), (dict(tail_groups=1, out_tail=18, ldo_tail=32), 4),
    (dict(N=1 << 20, K=1 << 13, lda=1 << 13, ldo=1 << 20), 2),
])
def test_w4_gemm_rejects(kw, code):
    L = _lib()
    d = dict(a=16, lda=64, w_q=16, w_scale=16, group_offsets=16, first_group=0, n_groups=4, m_total=10, N=32, K=64, epilogue=0,
             out=16, out_dtype=0, ldo=32)
    d.update(kw)
    st = L.lib().moe_w4_gemm(ctypes.byref(L.MoeW4Desc(**d)), None)
    assert st == code, L.lib().moe_last_error()
    assert L.lib().moe_last_error().decode().startswith("moe_w4_gemm")
    assert L.lib().moe_w4_gemm(None, None) == 1


def test_w4_gemm_needs_no_out_where_all_groups_are_tail_groups():
    """Without rows the call returns before a launch, so its checks are all that runs."""
    L = _lib()
    d = L.MoeW4Desc(a=16, lda=64, w_q=16, w_scale=16, group_offsets=16, n_groups=4, m_total=0, N=32, K=64, out_dtype=1,
                    tail_groups=4, out_tail=16, ldo_tail=32)
    assert L.lib().moe_w4_gemm(ctypes.byref(d), None) == 0, L.lib().moe_last_error()
    d.tail_groups = 3
    assert L.lib().moe_w4_gemm(ctypes.byref(d), None) == 4


@pytest.mark.parametrize("counts", [(-1, 4, 4), (4, -1, 4), (4, 4, -1)])
def test_w4_gemm_bounded_rejects(counts):
    """Negative counts of rows; the descriptor's own refusals are moe_w4_gemm's."""
    L = _lib()
    d = L.MoeW4Desc(a=16, lda=64, w_q=16, w_scale=16, group_offsets=16, n_groups=4, m_total=10, N=32, K=64, out=16, ldo=32)
    assert L.lib().moe_w4_gemm_bounded(ctypes.byref(d), *counts, None) == 2
    assert "negative" in L.lib().moe_last_error().decode()
    assert L.lib().moe_w4_gemm_bounded(None, 4, 4, 4, None) == 1
    d.K = 48
    assert L.lib().moe_w4_gemm_bounded(ctypes.byref(d), 4, 4, 4, None) == 2


def test_more_threads_than_a_launch_has():
    """A launch counts its threads in 32 bits: calls with more chunks of 8 elements than that are refused (workgroups of
    256 chunks; for the norms 16 lanes a row or more, for the combine 64)."""
    L = _lib()
    n = 1 << 32
    for fn, args in (
            ("fp8_ckpt_pack", (P(16), 1, n // 16, 128, 128, P(16), P(16), None)),
            ("fp8_ckpt_unpack", (P(16), P(16), n // 16, 128, None, None, 1, P(16), 0, 128, None)),
            ("moe_swiglu_backward_ckpt", (P(16), P(16), P(16), n // 16, 128, P(16), None, None, P(16), None)),
            ("w4_quant", (P(16), 1 << 10, 1 << 18, 128, P(16), P(16), None)),
            ("moe_combine_backward_ckpt", (P(16), P(16), P(16), P(16), P(16), P(16), P(16), n // 64, 1, 8, 8, P(16), P(16),
                                           P(16), None, None, None)),
            ("moe_norm", _norm(rows=n // 16, q=None, s=None))):
        _expect(L, fn, args, 2)


class _Sized(torch.Tensor):
    """A tensor of any size without memory, for the binding a GPU tensor."""
    is_cuda = True


def _sized(*shape, dtype=torch.float32):
    return torch.empty(shape, dtype=dtype, device="meta").as_subclass(_Sized)


def test_binding_refuses_sizes_past_32_bits():
    """The C calls take widths and counts as int: a size of 2^32 + n is refused and does not arrive there as n."""
    import sparse_moe_layer_sigmoid_amd as M
    n, u8, i32, b16 = (1 << 32) + 16, torch.uint8, torch.int32, torch.bfloat16
    many, wide = _sized(n, 8), _sized(1, n)
    q, s = _sized(1, n, dtype=u8), _sized(1, (n + 127) // 128, dtype=u8)
    offs, out = _sized(3, dtype=i32), _sized(4, 32)
    for call in (
            lambda: M.moe_norm(many), lambda: M.moe_norm(wide),
            lambda: M.moe_norm_backward(many, many, _sized(n), _sized(n)),
            lambda: M.moe_norm_backward(wide, wide, _sized(1), _sized(1)),
            lambda: M.fp8_ckpt_pack(wide), lambda: M.fp8_ckpt_unpack(q, s),
            lambda: M.moe_swiglu_backward_ckpt(q, s, _sized(1, n // 2)),
            lambda: M.moe_combine_backward_ckpt(
                _sized(n, 8, dtype=b16), _sized(n, 8, dtype=u8), _sized(n, 1, dtype=u8), _sized(n, 1, dtype=i32), _sized(n, 1),
                _sized(n, 4), _sized(n, 1, dtype=i32)),
            lambda: M.moe_combine_backward_ckpt(
                _sized(1, 8, dtype=b16), _sized(1, 8, dtype=u8), _sized(1, 1, dtype=u8), _sized(1, 1, dtype=i32), _sized(1, 1),
                _sized(1, n), _sized(1, 1, dtype=i32)),
            lambda: M.w4_quant(_sized(n, 32, dtype=b16)), lambda: M.w4_quant(_sized(n, 1, 32, dtype=b16)),
            lambda: M.w4_quant(_sized(1, n, dtype=b16)),
            lambda: M.moe_w4_gemm(_sized(4, 32, dtype=b16), _sized(1, n, 16, dtype=u8), _sized(1, n, 1, dtype=u8), offs, 0, 1, 4,
                                  _sized(4, n)),
            lambda: M.moe_w4_gemm(_sized(4, n, dtype=b16), _sized(1, 32, n // 2, dtype=u8), _sized(1, 32, n // 32, dtype=u8), offs,
                                  0, 1, 4, out)):
        with pytest.raises(ValueError, match="does not fit 32 bits"):
            call()
    a, wq, ws = _sized(4, 32, dtype=b16), _sized(2, 32, 16, dtype=u8), _sized(2, 32, 1, dtype=u8)
    for tails in (1 << 32, 3, -1):
        with pytest.raises(ValueError, match="tail_groups"):
            M.moe_w4_gemm(a, wq, ws, offs, 0, 2, 4, out, out_tail=out, tail_groups=tails)


def test_binding_refuses_cpu_tensors():
    import sparse_moe_layer_sigmoid_amd as M
    x = torch.zeros((4, 128))
    u8 = torch.zeros((4, 128), dtype=torch.uint8)
    i32 = torch.zeros((4, 2), dtype=torch.int32)
    for call in (lambda: M.moe_norm(x), lambda: M.moe_norm_backward(x, x, None, None), lambda: M.fp8_ckpt_pack(x),
                 lambda: M.fp8_ckpt_unpack(u8, u8), lambda: M.moe_swiglu_backward_ckpt(u8, u8, x),
                 lambda: M.moe_combine_backward_ckpt(x, u8, u8, i32, x, x, i32), lambda: M.w4_quant(x.bfloat16()),
                 lambda: M.moe_w4_gemm(x.bfloat16(), u8, u8, i32, 0, 1, 4, x)):
        with pytest.raises(TypeError, match="GPU tensor"):
            call()


def test_layer_refuses_arguments():
    import sparse_moe_layer_sigmoid_amd as M
    w = torch.zeros((8, 64))
    W13, W2 = torch.zeros((9, 64, 64)), torch.zeros((9, 64, 32))
    b = torch.zeros(8)
    with pytest.raises(ValueError, match="norm must be"):
        M.MoELayer(w, W13, W2, b, 2, norm="batch")
    with pytest.raises(ValueError, match="need norm"):
        M.MoELayer(w, W13, W2, b, 2, norm_weight=b)
    with pytest.raises(ValueError, match="either E4M3"):
        M.MoELayer(w, W13, W2, b, 2, fp8=True, w4=True)
