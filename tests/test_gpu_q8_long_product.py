"""A block-scaled product that keeps the GPU busy for longer than one device wait may last (1 s)."""
import pytest
import torch

from gpu_common import q3

pytestmark = pytest.mark.gpu


def test_a_product_of_more_than_a_second_reports_no_timeout():
    # 2 x 65536 x 65536 x 524288 operations, 4.5e15: 1.4 s at the highest rate that this kernel has
    # reached. Rows and weight are one tensor of ones, so every sum is 2^19, which bf16 holds.
    m = q3()
    n, k = 65536, 1 << 19
    ones = torch.full((n, k), 0x38, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    xs = torch.full((n, k // 128), 127, dtype=torch.uint8, device="cuda").view(torch.float8_e8m0fnu)
    lin = m.LinearQ8(ones, xs[:n // 128].clone())
    a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    a.record()
    out = m.linear_q8(ones, xs, lin)
    b.record()
    torch.cuda.synchronize()
    assert m.device_status()[0] == 0
    assert bool((out == 2.0 ** 19).all())
    assert a.elapsed_time(b) > 1000, "too short to show anything"
    del ones, xs, lin, out
    torch.cuda.empty_cache()
