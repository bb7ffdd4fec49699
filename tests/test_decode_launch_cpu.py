"""moe_decode_shaped (the launch for tests of moe_decode) without a GPU: refusals, before anything is launched."""
import ctypes

import pytest

from tests.test_more_operators_abi_cpu import _decode, _expect, _lib


def _shaped(L):
    f = L.lib().moe_decode_shaped
    f.restype = ctypes.c_int
    f.argtypes = [ctypes.POINTER(L.MoeDecodeDesc), ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.c_void_p]
    return f


@pytest.mark.parametrize("workgroups,lists,looks", [(0, 1, 1), (-1, 4, 1), (5, 4, 1), (1, 1025, 1), (1, 0, 1), (4, 4, -1),
                                                    (4, 4, (1 << 22) + 1)])
def test_launch_rejects(workgroups, lists, looks):
    L = _lib()
    _shaped(L)
    _expect(L, "moe_decode_shaped", (ctypes.byref(L.MoeDecodeDesc(**_decode())), workgroups, lists, looks, None), 2)


def test_launch_checks_the_call_itself():
    L = _lib()
    assert _shaped(L)(ctypes.byref(L.MoeDecodeDesc(**_decode(T=17))), 4, 4, 1, None) == 2 and _shaped(L)(None, 4, 4, 1, None) == 1
