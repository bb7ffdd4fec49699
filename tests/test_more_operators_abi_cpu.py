"""Refusals of the 8-bit integer calls without a GPU: the C ABI checks its arguments before anything is launched, the binding
checks tensors before the C call."""
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


def test_i8_rows_reject():
    L = _lib()
    q = lambda x=16, xt=1, rows=4, cols=100, ldx=100, q=16, s=16: (P(x), xt, rows, cols, ldx, P(q), P(s), None)  # noqa: E731
    for kw, code in ((dict(x=None), 1), (dict(q=None), 1), (dict(s=None), 1), (dict(xt=2), 3), (dict(rows=-1), 2),
                     (dict(cols=0), 2), (dict(cols=(1 << 24) + 1, ldx=1 << 25), 2), (dict(ldx=99), 4), (dict(x=18), 4),
                     (dict(s=18), 4), (dict(rows=1 << 22), 2), (dict(x=17, xt=0), 4)):
        _expect(L, "i8_quant", q(**kw), code)
    d = lambda q=16, s=16, rows=4, cols=100, o=16, ot=0, ldo=100: (P(q), P(s), rows, cols, P(o), ot, ldo, None)  # noqa: E731
    for kw, code in ((dict(q=None), 1), (dict(s=None), 1), (dict(o=None), 1), (dict(ot=2), 3), (dict(rows=-1), 2),
                     (dict(cols=0), 2), (dict(ldo=99), 4), (dict(o=17), 4), (dict(s=17), 4), (dict(rows=1 << 40), 2)):
        _expect(L, "i8_dequant", d(**kw), code)


@pytest.mark.parametrize("kw,code", [
    (dict(a=None), 1), (dict(a_scale=None), 1), (dict(w_q=None), 1), (dict(w_scale=None), 1), (dict(group_offsets=None), 1),
    (dict(out=None), 1), (dict(epilogue=2), 3), (dict(out_dtype=2), 3), (dict(n_groups=0), 2), (dict(n_groups=1025), 2),
    (dict(first_group=-1), 2), (dict(m_total=-1), 2), (dict(m_total=1 << 31), 2), (dict(K=24), 2), (dict(K=0), 2),
    (dict(K=131072, lda=131072), 2), (dict(N=0), 2), (dict(N=31, epilogue=1), 2), (dict(tail_groups=5), 2),
    (dict(tail_groups=-1), 2), (dict(lda=48), 4), (dict(lda=72), 4), (dict(a=8), 4), (dict(w_q=8), 4), (dict(a_scale=18), 4),
    (dict(w_scale=18), 4), (dict(ldo=31), 4), (dict(out=18, out_dtype=1), 4), (dict(tail_groups=1), 1),
    (dict(tail_groups=1, out_tail=16, ldo_tail=31), 4), (dict(tail_groups=1, out_tail=18, ldo_tail=32), 4),
    (dict(N=1 << 18, K=1 << 13, lda=1 << 13, ldo=1 << 20), 2), (dict(sorted_rows=-1), 2), (dict(out_rows=-1), 2),
    (dict(tail_rows=-1), 2),
])
def test_i8_gemm_rejects(kw, code):
    L = _lib()
    d = dict(a=16, a_scale=16, lda=64, w_q=16, w_scale=16, group_offsets=16, first_group=0, n_groups=4, m_total=10, N=32, K=64,
             epilogue=0, out=16, out_dtype=0, ldo=32, sorted_rows=10, out_rows=10, tail_rows=10)
    d.update(kw)
    _expect(L, "moe_i8_gemm", (ctypes.byref(L.MoeI8Desc(**d)), None), code)


def test_i8_gemm_null_desc_and_no_rows():
    L = _lib()
    _expect(L, "moe_i8_gemm", (None, None), 1)
    d = dict(lda=64, w_q=16, w_scale=16, group_offsets=16, n_groups=4, N=32, K=64, ldo=32)
    for kw in (dict(m_total=0, sorted_rows=5, out_rows=5), dict(m_total=5, sorted_rows=0, out_rows=5)):
        assert L.lib().moe_i8_gemm(ctypes.byref(L.MoeI8Desc(**d, **kw)), None) == 0


def test_binding_refuses_cpu_tensors():
    L = _lib()
    z = torch.zeros
    for call in (lambda: L.i8_quant(z(2, 8)), lambda: L.i8_quant([1.0]),
                 lambda: L.i8_dequant(z(2, 8, dtype=torch.int8), z(2)),
                 lambda: L.moe_i8_gemm(z(2, 16, dtype=torch.int8), z(2), z(1, 4, 16, dtype=torch.int8), z(1, 4),
                                       z(2, dtype=torch.int32), 0, 1, 2, z(2, 4))):
        with pytest.raises(TypeError):
            call()


def _decode(**kw):
    a = dict(x=16, x_dtype=0, ldx=256, T=2, d=256, inter=128, n_experts=8, n_shared=1, top_k=2, n_group=1, topk_group=1, norm=-1,
             norm_dtype=1, norm_eps=1e-6, w_router=16, bias=16, w_dtype=0, scale_fmt=0, w13=16, w2=16, out=16, out_dtype=0, ldo=256,
             ws=256, ws_bytes=1 << 30)
    a.update(kw)
    return a


@pytest.mark.parametrize("kw,code", [
    (dict(x=None), 1), (dict(w_router=None), 1), (dict(bias=None), 1), (dict(w13=None), 1), (dict(w2=None), 1), (dict(out=None), 1),
    (dict(w_dtype=3), 1), (dict(w_dtype=3, w13_scale=16), 1), (dict(T=-1), 2), (dict(T=17), 2), (dict(n_experts=6), 2),
    (dict(n_experts=260), 2), (dict(n_shared=2), 2), (dict(n_shared=-1), 2), (dict(top_k=0), 2), (dict(top_k=9), 2),
    (dict(n_experts=64, top_k=33), 2), (dict(n_group=3), 2), (dict(n_group=0), 2), (dict(n_group=4), 2), (dict(topk_group=2), 2),
    (dict(n_experts=16, n_group=4, top_k=5), 2), (dict(w_dtype=1), 3), (dict(w_dtype=5), 3), (dict(scale_fmt=1), 3),
    (dict(norm=2), 3), (dict(norm=-2), 3), (dict(x_dtype=1), 3), (dict(x_dtype=2), 3), (dict(out_dtype=2), 3),
    (dict(norm=0, norm_dtype=2), 3), (dict(norm=0, norm_eps=-1.0), 2), (dict(norm=0, norm_eps=float("nan")), 2),
    (dict(d=96, ldx=96), 2), (dict(d=0), 2), (dict(d=8256, ldx=8256, ldo=8256), 2), (dict(inter=32), 2), (dict(inter=0), 2),
    (dict(w_dtype=3, d=320, ldx=320, ldo=320, w13_scale=16, w2_scale=16), 2), (dict(w_dtype=4, inter=192, w13_scale=16, w2_scale=16), 2),
    (dict(w_dtype=2, scale_fmt=1, w13_scale=16, w2_scale=16), 2), (dict(inter=1 << 17, d=8192, ldx=8192, ldo=8192), 2),
    (dict(T=16, n_experts=64, top_k=32, d=64, ldx=64, ldo=64, inter=1 << 21), 2),    # h of 4.1 GiB
    (dict(ldx=255), 4), (dict(ldx=260), 4), (dict(x=8), 4), (dict(ldo=255), 4), (dict(out=17), 4), (dict(out=18, out_dtype=1), 4),
    (dict(w_router=8), 4), (dict(w13=8), 4), (dict(w2=8), 4), (dict(bias=18), 4), (dict(w_dtype=4, w13_scale=18, w2_scale=16), 4),
    (dict(norm=0, x=17), 4), (dict(norm=0, norm_weight=18), 4), (dict(topk_idx=18), 4), (dict(ws=None), 5), (dict(ws_bytes=100), 5),
    (dict(ws=8), 5),
])
def test_decode_rejects(kw, code):
    L = _lib()
    _expect(L, "moe_decode", (ctypes.byref(L.MoeDecodeDesc(**_decode(**kw))), None), code)


def test_decode_null_desc_workspace_size():
    L = _lib()
    _expect(L, "moe_decode", (None, None), 1)
    f = L.lib().moe_decode_workspace_size
    assert f(-1, 256, 128, 8, 1, 2) == 0 and f(17, 256, 128, 8, 1, 2) == 0 and f(1, 8200, 128, 8, 1, 2) == 0
    assert f(1, 256, 128, 8, 2, 2) == 0 and f(1, 256, 128, 8, 1, 33) == 0
    assert f(16, 256, 128, 8, 1, 2) - f(16, 256, 128, 8, 0, 2) == 16 * 128 * 4 and f(0, 256, 128, 8, 1, 2) > 0
