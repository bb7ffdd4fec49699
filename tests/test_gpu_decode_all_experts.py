"""moe_decode where every expert is chosen: the longest list of active experts, 256 routed ones and the shared one."""
import numpy as np
import pytest
import torch

from tests.gpu_common import say
from tests.test_gpu_decode import Case, check

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("shared", [0, 1])
@pytest.mark.parametrize("fmt", ["bf16", "e4m3", "i8", "w4"])
def test_decode_all_experts(fmt, shared):
    """Token t of 16 prefers experts 16 t to 16 t + 15 by a router weight of 1 on its own input."""
    say(f"decode {fmt}: all experts, {shared} shared")
    c = Case(fmt, 16, 128, 128, 256, 16, shared=shared)
    c.x[:, :16] *= 0.1
    c.wr[:, :16] = 0
    for t in range(16):
        c.x[t, t] = 6.0
        c.wr[16 * t:16 * t + 16, t] = 1.0
    check(c)
    _, idx, _, counts = c.run()
    assert bool((counts == 1).all())
    assert np.array_equal(np.sort(idx.cpu().numpy(), axis=1), np.arange(256).reshape(16, 16))
