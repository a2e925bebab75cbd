"""Starts of kv_store_q8 whose differences leave 32 bits: they fall, so nothing at all is stored."""
import numpy as np
import pytest
import torch

from gpu_common import q3
from test_gpu_q8 import HD, _cache, _cfg, _gen

pytestmark = pytest.mark.gpu
LOW, HIGH = -2 ** 31, 2 ** 31 - 1


# In 32-bit arithmetic every difference of the first two would be positive, and the last sequence
# would claim places on the grid that are the first one's.
@pytest.mark.parametrize("starts", [[0, 2000, LOW, -1, 0, 100], [0, 2000, LOW + 5, -3, 7, 90],
                                    [0, HIGH, LOW, LOW, 0, 10], [HIGH, LOW, 0, 1, 2, 3],
                                    [0, 10, 5, 20, 30, 40]])
def test_starts_that_fall_by_more_than_32_bits_hold(starts):
    m = q3()
    cfg = _cfg(nkv=2, nh=8)
    kv = _cache(cfg, 5, 2100, 1)
    held = (kv.k, kv.v, kv.k_scale, kv.v_scale)
    was = [t.clone().view(torch.uint8) for t in held]
    rows = torch.randn(2000, 2 * HD, generator=_gen(2)).to(torch.bfloat16).cuda()
    i32 = lambda v: torch.tensor(np.array(v, dtype=np.int32), device="cuda")  # noqa: E731
    m.kv_store_q8(cfg, rows, rows, kv, i32([0, 1, 2, 3, 4]), i32([0] * 5), i32(starts))
    assert m.device_status()[0] == -2
    for t, old in zip(held, was):
        assert torch.equal(t.view(torch.uint8), old)
