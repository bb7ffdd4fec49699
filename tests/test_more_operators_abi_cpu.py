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
