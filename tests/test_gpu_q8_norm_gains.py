"""Gains of the norm with 8-bit output at the ends of their range. Distances as derived in
test_gpu_q8_norm_bytes.py."""
import numpy as np
import pytest
import torch

from gpu_common import q3
from test_gpu_q8 import _gen
from test_gpu_q8_norm_bytes import _cfg, _differences, _run, _want, _whole

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,size,gain", [
    ("bf16", 2.0 ** 53, 1.8e19), ("bf16", 2.0 ** -100, 1.8e19), ("bf16", 1.0, 2.0 ** -80),
    ("fp32", 2.0 ** 50, 2.0 ** 90), ("fp32", 2.0 ** 53, 1e25), ("fp32", 1.0, 1e38)])
@pytest.mark.parametrize("H", [256, 8192 + 128])
def test_gains_at_the_ends_of_their_range(H, dtype, size, gain):
    # below 2^64 in bf16, any in fp32 whose h / rms * gain fits: the bytes of 64 bits up to the
    # derived distance
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    x = (size * _whole(4, H, 7, 3)).to(dt)
    g = (gain * (1 - 0.4 * torch.rand(H, generator=_gen(4)).double())).to(dt)
    h, q, s = _run(x, g, dtype)
    assert np.all(np.isfinite(q))
    assert np.abs(_want(h, g.double().numpy())[0]).max() < 3e38     # fits fp32
    _differences(q, s, h, g.double().numpy(), 2.0 ** -20)


@pytest.mark.parametrize("H", [256, 8192 + 128])
def test_a_far_bf16_gain_is_a_device_error(H):
    m = q3()
    cfg = _cfg(H, "bf16")
    x = (2.0 ** 50 * _whole(4, H, 7, 3)).to(torch.bfloat16).cuda()
    g = torch.ones(H, dtype=torch.bfloat16)
    g[H - 5] = 2.0 ** 64
    _, q, _ = m.add_rms_norm_q8(cfg, x, g.cuda())
    assert m.device_status()[0] == -2
    # other blocks are as they should be; an infinite gain is no error, its column NaN
    _, q1, _ = m.add_rms_norm_q8(cfg, x, torch.ones_like(g).cuda())
    assert torch.equal(q[:, :H - 128].view(torch.uint8), q1[:, :H - 128].view(torch.uint8))
    g[H - 5] = float("inf")
    _, q, _ = m.add_rms_norm_q8(cfg, x, g.cuda())
    m.check_device()
    assert bool(q[:, H - 5].float().isnan().all())
