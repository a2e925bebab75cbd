"""Bytes of the norm with 8-bit output against 64-bit arithmetic.

Derivation. A row's sum of squares is a sum of fp32 values of one sign; with n roundings on the way
it is off by at most n 2^-24 of itself. Rows up to 8192 wide take 13 roundings (four squares and sums
in each half of a thread's eight columns, the two halves, five levels in the warp, three across the
warps; the last two levels keep their remainders), wider ones 25. 1 / rms is off by half of that, the
product behind it is rounded once more (2^-24): a value is off by at most 7.5 2^-24 < 2^-21 of itself
(13.5 2^-24 < 2^-20 where wider), besides 2^-40 for what the two-part 1 / rms leaves out. So each
byte is the one of the 64-bit value, or, where that value lies within this distance of the middle of
two e4m3 values (or the block's maximum of a border between two scales), the other one.

Rows of small whole numbers have exact sums. Then 1 / rms is good to 2^-40 and so is the value that a
middle is compared with: bytes have to be equal unless the value is that near to a middle. (Below 2^-6
of the scale, where e4m3 has fewer bits, a value that fp32 rounds onto a middle keeps that rounding:
one rounding, 2^-24, plus the small parts: 2^-23.9.)
"""
import numpy as np
import pytest
import torch

from gpu_common import q3
from oracle import q8_oracle as Q
from test_gpu_q8 import _e8, _gen

pytestmark = pytest.mark.gpu
EPS = 2.0 ** -20


def _cfg(H, dtype):
    return q3().config(H, 32, 8, 9728, dtype, rms_eps=EPS)


def _want(h, gain):
    """(values, scales of the blocks, e4m3 values) in 64 bits; h, gain float64."""
    y = h / np.sqrt(np.mean(h * h, 1, keepdims=True) + EPS) * gain
    q, s = Q.quantize(y, Q.edges(h.shape[1]))
    return y, s, q


def _middle_distance(v):
    """Relative distance of |v| (in units of the scale) from the nearest middle of e4m3 values."""
    a = np.abs(v)
    step = np.ldexp(1.0, np.maximum(np.frexp(np.maximum(a, 1e-300))[1] - 4, -9))
    mid = (np.floor(a / step) + 0.5) * step
    return np.abs(a - mid) / np.maximum(a, 1e-300)


def _differences(got_q, got_s, h, gain, delta):
    """Asserts that bytes and scales are those of 64 bits but for values within `delta` (relative) of
    a middle, or scales whose maximum is that near to a border; returns how many values differ."""
    y, s, q = _want(h, gain)
    bounds = Q.edges(h.shape[1])
    n = 0
    for i, (lo, hi) in enumerate(zip(bounds, bounds[1:])):
        part = y[:, lo:hi]
        amax = np.abs(part).max(1)
        other = np.vectorize(Q.scale_of, otypes=[float])(amax * (1 - delta))
        same = got_s[:, i] == s[:, i]
        assert np.all(same | (got_s[:, i] == other))
        near = _middle_distance(part / got_s[:, i:i + 1]) <= delta
        diff = (got_q[:, lo:hi] != q[:, lo:hi]) & same[:, None]
        assert np.all(~diff | near)
        n += int(diff.sum())
    return n


def _run(x, gain, dtype, delta=None):
    m = q3()
    cfg = _cfg(x.shape[1], dtype)
    h, q, s = m.add_rms_norm_q8(cfg, x.cuda(), gain.cuda(), None if delta is None else delta.cuda())
    m.check_device()
    return (h.double().cpu().numpy(), q.float().cpu().numpy().astype(np.float64), _e8(s))


@pytest.mark.parametrize("S,H,dtype,delta", [
    (3000, 64, "bf16", False), (2000, 256, "bf16", True), (1500, 512, "fp32", False),
    (1000, 2560, "bf16", True), (700, 5120, "fp32", True), (300, 8192, "bf16", True),
    (300, 8192 + 64, "bf16", False), (150, 32768, "fp32", True)])
def test_bytes_are_those_of_64_bits(S, H, dtype, delta):
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    x = torch.randn(S, H, generator=_gen(H)).to(dt)
    d = torch.randn(S, H, generator=_gen(H + 1)).to(dt) if delta else None
    gain = (1 + 0.1 * torch.randn(H, generator=_gen(H + 2))).to(dt)
    h, q, s = _run(x, gain, dtype, d)
    n = _differences(q, s, h, gain.double().numpy(), 2.0 ** -21 if H <= 8192 else 2.0 ** -20)
    # of values spread evenly, 16 middles a factor of two: less than 2 delta 16 / ln 2 can differ
    assert n <= 10 + S * H * 2.0 ** -14


def _whole(S, H, top, seed):
    """Rows of whole numbers up to `top` in magnitude: their sums of squares stay below 2^24."""
    assert H * top * top < 2 ** 24
    return torch.randint(-top, top + 1, (S, H), generator=_gen(seed)).float()


@pytest.mark.parametrize("H", [64, 256, 2560, 8192, 8192 + 128])
def test_fp32_values_that_round_onto_a_middle(H):
    # gains made so that h / rms * gain falls on a middle of e4m3 as nearly as fp32 can say it, and
    # the two neighbouring gains: true values on both sides
    x = _whole(1, H, 31, H)
    x[x == 0] = 1.0
    h = x.double().numpy()
    inv = 1 / np.sqrt(np.mean(h * h) + EPS)
    k = np.arange(H)
    mid = (8.5 + k % 8) * 2.0 ** (4 - k % 7)               # middles of seven binades
    g0 = (mid / (h[0] * inv)).astype(np.float32)
    g0[::64] = (440.0 / (h[0, ::64] * inv)).astype(np.float32)   # pins each block's scale at 1
    landed = [0, 0]
    for step in (-1, 0, 1):
        g = g0 if step == 0 else np.nextafter(g0, np.float32(np.inf if step > 0 else -np.inf))
        y = h[0] * inv * g.astype(np.float64)
        on = y.astype(np.float32).astype(np.float64) == np.where(k % 64 == 0, 0, mid)
        landed[0] += int((on & (y < mid)).sum())
        landed[1] += int((on & (y > mid)).sum())
        got_h, q, s = _run(x, torch.tensor(g), "fp32")
        assert np.all(s == 1) and np.array_equal(got_h, h)
        assert _differences(q, s, h, g.astype(np.float64), 2.0 ** -40) == 0
    assert min(landed) >= H // 16, landed                  # the case is met, on both sides


@pytest.mark.parametrize("H,top", [(2048, 63), (256, 127)])
def test_bf16_values_that_round_onto_a_middle(H, top):
    # rows picked from 2^25 random values for holding one that fp32 rounds onto a middle
    rows, gains, sides = [], [], [0, 0]
    gain = (1 + 0.3 * torch.rand(H, generator=_gen(1))).to(torch.bfloat16)
    g = gain.double()
    for seed in range(8):
        x = _whole(2 ** 22 // H, H, top, 10 + seed)
        h = x.double()
        y = h / torch.sqrt((h * h).mean(1, keepdim=True) + EPS) * g
        amax = y.abs().view(len(x), -1, 128).amax(2)
        s = torch.exp2(torch.ceil(torch.log2(amax / 448))).repeat_interleave(128, 1)
        v = y.abs() / s
        bits = v.float().view(torch.int32) & 0xfffff
        on = (bits == 0x80000) & (v >= 2.0 ** -6)
        keep = on.any(1)
        f = v.float().double()
        sides[0] += int((on & (v < f)).sum())
        sides[1] += int((on & (v > f)).sum())
        rows.append(x[keep])
    x = torch.cat(rows).to(torch.bfloat16)
    assert min(sides) >= 5, sides
    h, q, s = _run(x, gain, "bf16")
    assert np.array_equal(h, x.double().numpy())
    y, ws, wq = _want(h, g.numpy())
    assert np.array_equal(s, ws)
    v = np.abs(y / np.repeat(s, 128, 1))
    tiny = (v < 2.0 ** -6) & (_middle_distance(v) <= 2.0 ** -23.9)
    assert np.array_equal(np.where(tiny, 0, q), np.where(tiny, 0, wq))
