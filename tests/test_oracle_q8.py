"""Pins of the fp64 oracle of the 8-bit operators: e4m3 against torch's conversion and every
code point, the scale rule by brute force, and the store's re-rounding by hand."""
import numpy as np
import torch

from oracle import q8_oracle as Q


def test_e4m3_agrees_with_torch_on_code_points_midpoints_and_neighbours():
    pts = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    pts = np.sort(pts[np.isfinite(pts)])
    assert np.array_equal(Q.e4m3(pts), pts)
    mid = (pts[1:] + pts[:-1]) / 2
    v = np.concatenate([mid, np.nextafter(mid, 1e9), np.nextafter(mid, -1e9)]).astype(np.float32)
    want = torch.tensor(v).to(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(Q.e4m3(v.astype(np.float64)), want)
    assert np.all(np.isnan(Q.e4m3([np.inf, -np.inf, np.nan])))


def test_scale_is_the_smallest_power_that_reaches_448():
    rng = np.random.default_rng(0)
    for a in list(np.exp(rng.uniform(-80, 80, 500))) + [448.0, 448.0 * 2 ** -20, 448.1, 2.0 ** 127]:
        s = Q.scale_of(a)
        assert a <= 448 * s and (s == 2.0 ** -126 or a > 448 * s / 2)
        assert np.log2(s) == np.round(np.log2(s))
    assert Q.scale_of(0.0) == 2.0 ** -126 and Q.scale_of(1e-45) == 2.0 ** -126


def test_store_re_rounds_earlier_rows_when_the_scale_grows():
    cache, scale = np.zeros((256, 1, 128)), np.zeros((2, 1))
    row = np.full((1, 1, 128), 1.0)
    row[0, 0, 0] = 2.0 ** -8
    Q.store(cache, scale, row, 0)          # amax 1: scale 2^-8, elements 256 and 1
    assert scale[0, 0] == 2.0 ** -8 and cache[0, 0, 0] == 1 and cache[0, 0, 1] == 256
    Q.store(cache, scale, np.full((1, 1, 128), 4096.0), 1)   # scale 2^4: a shift by 12
    assert scale[0, 0] == 2.0 ** 4 and cache[1, 0, 5] == 256
    assert cache[0, 0, 1] == 2.0 ** -4 and cache[0, 0, 0] == 0.0   # 2^-12 falls below 2^-10
    Q.store(cache, scale, np.full((1, 1, 128), 1.0), 128)    # a block of its own
    assert scale[1, 0] == 2.0 ** -8 and scale[0, 0] == 2.0 ** 4
