"""moe_decode launched as a smaller or a busy device runs it: fewer workgroups than CUs, so that each has several blocks of output
columns, and tiles of workgroups that never start, which the others take over.  Every result has to have the bits of the usual launch:
neither who takes a tile nor where a block of columns begins enters a sum."""
import ctypes

import pytest
import torch

from sparse_moe_layer_sigmoid_amd import _lib as L
from tests.gpu_common import say
from tests.test_gpu_decode import FORMATS, Case

pytestmark = pytest.mark.gpu

# workgroups, lists: one for everything, numbers that the 16 classes of started workgroups do not divide, many that never start, more
# than there are CUs
LAUNCHES = [(1, 1), (1, 7), (3, 64), (7, 7), (40, 41), (64, 64), (64, 256), (250, 256), (256, 300), (300, 300)]


def shaped(monkeypatch, workgroups, lists):
    """Calls of moe_decode go to moe_decode_shaped from here on."""
    f = L.lib().moe_decode_shaped
    f.restype, f.argtypes = ctypes.c_int, [ctypes.POINTER(L.MoeDecodeDesc), ctypes.c_int, ctypes.c_int, ctypes.c_void_p]

    def launch(dev, fn, desc):
        assert fn == "moe_decode"
        L._check("moe_decode_shaped", f(desc, workgroups, lists, torch.cuda.current_stream(dev).cuda_stream))

    monkeypatch.setattr(L, "_launch", launch)


# narrow rows, and 4 bits: a workgroup holds three tiles at once; the widest rows: two; more than 8 tokens: wide sums; one token
@pytest.mark.parametrize("T,d,inter,E,K", [(5, 512, 512, 16, 4), (12, 1024, 512, 32, 4), (7, 8192, 512, 4, 2), (1, 512, 512, 8, 1)])
@pytest.mark.parametrize("fmt", FORMATS)
def test_decode_launches(fmt, T, d, inter, E, K, monkeypatch):
    c = Case(fmt, T, d, inter, E, K, norm="rms", shared=0 if T == 1 else 1)
    want = c.run()
    for workgroups, lists in LAUNCHES:
        say(f"decode {fmt} T={T} d={d}: {workgroups} workgroups, {lists} lists")
        with monkeypatch.context() as m:
            shaped(m, workgroups, lists)
            got = c.run()
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)
    for a, b in zip(c.run(), want):
        assert torch.equal(a, b)
