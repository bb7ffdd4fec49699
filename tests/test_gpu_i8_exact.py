"""i8_quant of f32 rows: the codes are RNE(127 x / A) of the exact quotient, also next to the midpoints between codes.

In float64 127 x is exact and the quotient off by 2^-53 of itself, while one that is not at a midpoint (c + 1/2) is at least 2^-40 away
from it (254 x and (2 c + 1) A are multiples of 2^-33 A where their difference is small): rint of it is the exact code."""
import numpy as np
import pytest
import torch

from sparse_moe_layer_sigmoid_amd import inputs as I
from tests.test_gpu_i8 import M, quant_reference

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def check(x):
    q, s = M().i8_quant(torch.from_numpy(x).to(DEV))
    wq, ws = quant_reference(x)
    assert np.array_equal(s.cpu().numpy(), ws)
    assert np.array_equal(q.cpu().numpy(), wq)


@pytest.mark.parametrize("scale", [1.0, 2.0 ** -100, 2.0 ** 120])
def test_i8_quant_f32_next_to_midpoints(scale):
    """The floats next to every midpoint of rows with random maxima, and the midpoints that are floats."""
    r = np.random.default_rng(31)
    rows = []
    for a in list(r.uniform(1.0, 2.0, 60).astype(np.float32)) + [np.float32(127.0 / 64), np.float32(1.0), np.float32(1.984375)]:
        mid = ((np.arange(127) + 0.5) * float(a) / 127.0).astype(np.float32)
        x = [mid]
        for _ in range(3):
            x.append(np.nextafter(x[-1], np.float32(0)))
        up = mid
        for _ in range(3):
            up = np.nextafter(up, np.float32(4))
            x.append(up)
        v = np.concatenate(x)
        rows.append(np.concatenate([v * r.choice(np.float32([-1, 1]), v.shape), [a]]).astype(np.float32) * np.float32(scale))
    check(np.stack(rows))


@pytest.mark.parametrize("rows,cols", [(4096, 2048), (1024, 512), (300, 4096), (200, 8192), (120, 16384), (60, 40000), (999, 1001)])
def test_i8_quant_f32_bitexact(rows, cols):
    """Every width's kernel over values that real rows have: products of normals (as the inner rows of an expert are)."""
    x = I.gen_normal(740 + cols, (rows, cols), 1.0, torch.float32)
    check((x * x.roll(1, 0)).numpy())


def test_i8_quant_f32_least_scale():
    """Rows at and below the least scale, whose values next to the midpoints are subnormal."""
    least = np.float32(127.0) * np.float32(2.0 ** -126)
    x = (np.arange(-508, 509) * 2.0 ** -128).astype(np.float32)          # quarter steps of the least scale
    x = np.concatenate([x, np.nextafter(x, np.float32(1)), np.nextafter(x, np.float32(-1))])
    assert np.abs(x).max() <= least * 1.01
    check(np.stack([x, x / 2]))
