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


def shaped(monkeypatch, workgroups, lists, looks=1 << 22):
    """Calls of moe_decode go to moe_decode_shaped from here on."""
    f = L.lib().moe_decode_shaped
    f.restype = ctypes.c_int
    f.argtypes = [ctypes.POINTER(L.MoeDecodeDesc), ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.c_void_p]

    def launch(dev, fn, desc):
        assert fn == "moe_decode"
        L._check("moe_decode_shaped", f(desc, workgroups, lists, looks, torch.cuda.current_stream(dev).cuda_stream))

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


@pytest.mark.parametrize("fmt", FORMATS)
def test_decode_gives_up_waiting(fmt, monkeypatch):
    """Workgroups that stop waiting for h write NaN to their columns, whole ones; without a look at the flag, all do.  The routing is
    right all the same, and so is the next call."""
    c = Case(fmt, 5, 2048, 512, 16, 4, norm="rms")
    want = c.run()
    for looks in (0, 1, 2, 8):
        say(f"decode {fmt}: {looks} looks")
        with monkeypatch.context() as m:
            shaped(m, 256, 256, looks)
            got = c.run()
        torch.cuda.synchronize()
        nan = torch.isnan(got[0])
        assert bool((nan.all(0) == nan.any(0)).all()) and torch.equal(got[0][~nan], want[0][~nan])
        assert bool((nan.view(5, 256, 8).all(2) == nan.view(5, 256, 8).any(2)).all())      # 2048 columns of 256 workgroups
        if looks == 0:
            assert bool(nan.all())
        for a, b in zip(got[1:], want[1:]):
            assert torch.equal(a, b)
        for a, b in zip(c.run(), want):
            assert torch.equal(a, b)
