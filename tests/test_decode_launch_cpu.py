"""moe_decode_shaped (the launch for tests of moe_decode) without a GPU: refusals, before anything is launched."""
import ctypes

import pytest

from tests.test_more_operators_abi_cpu import _decode, _expect, _lib


@pytest.mark.parametrize("workgroups,lists", [(0, 1), (-1, 4), (5, 4), (1, 1025), (1, 0)])
def test_launch_rejects(workgroups, lists):
    L = _lib()
    f = L.lib().moe_decode_shaped
    f.restype, f.argtypes = ctypes.c_int, [ctypes.POINTER(L.MoeDecodeDesc), ctypes.c_int, ctypes.c_int, ctypes.c_void_p]
    _expect(L, "moe_decode_shaped", (ctypes.byref(L.MoeDecodeDesc(**_decode())), workgroups, lists, None), 2)


def test_launch_checks_the_call_itself():
    L = _lib()
    f = L.lib().moe_decode_shaped
    f.restype, f.argtypes = ctypes.c_int, [ctypes.POINTER(L.MoeDecodeDesc), ctypes.c_int, ctypes.c_int, ctypes.c_void_p]
    assert f(ctypes.byref(L.MoeDecodeDesc(**_decode(T=17))), 4, 4, None) == 2 and f(None, 4, 4, None) == 1
