"""Arguments of the 8-bit calls that are no tensors, or tensors of another number of dimensions: the
library's own error (no GPU)."""
import pytest
import torch

from test_abi import _cfg, lib  # noqa: F401  (fixture)


def _u8(*shape):
    return torch.zeros(shape, dtype=torch.uint8)


def test_what_is_no_tensor_or_of_other_dimensions_is_refused(lib):  # noqa: F811
    import qwen3_vl_decoder_b200 as q3
    c = _cfg()
    kv = q3.kv_caches(c, 1, 2, 200, "cpu", dtype="fp8")[0]
    i = torch.zeros(2, dtype=torch.int32)
    k = torch.zeros(2, 1024, dtype=torch.bfloat16)
    x = torch.zeros(2, 2560, dtype=torch.bfloat16)
    lin = q3.LinearQ8(_u8(256, 2560).view(torch.float8_e4m3fn),
                      _u8(2, 20).view(torch.float8_e8m0fnu))
    xq, xs = _u8(2, 2560).view(torch.float8_e4m3fn), _u8(2, 20).view(torch.float8_e8m0fnu)
    e4, e8 = kv.k, kv.k_scale
    calls = {
        "store k": lambda v: q3.kv_store_q8(c, v, k, kv, i, i),
        "store v": lambda v: q3.kv_store_q8(c, k, v, kv, i, i),
        "store seq": lambda v: q3.kv_store_q8(c, k, k, kv, v, i),
        "store lens": lambda v: q3.kv_store_q8(c, k, k, kv, i, v),
        "attention q": lambda v: q3.attention_q8(c, v, kv, i, i),
        "attention seq": lambda v: q3.attention_q8(c, torch.zeros(2, 4096, dtype=torch.bfloat16),
                                                   kv, v, i),
        "norm x": lambda v: q3.add_rms_norm_q8(c, v, None),
        "weight": lambda v: q3.quantize_weight_q8(v),
        "weight form": lambda v: q3.LinearQ8(v, xs),
        "weight scales": lambda v: q3.LinearQ8(xq, v),
        "product rows": lambda v: q3.linear_q8(v, xs, lin),
        "product scales": lambda v: q3.linear_q8(xq, v, lin),
        "head rows": lambda v: q3.lm_head(c, v, None, lin),
        "cache k": lambda v: q3.KvCacheQ8.of(c, v, e4, e8, e8),
        "cache v": lambda v: q3.KvCacheQ8.of(c, e4, v, e8, e8),
        "cache scales": lambda v: q3.KvCacheQ8.of(c, e4, e4, v, e8),
    }
    bad = [None, 3, [1, 2], torch.zeros((), dtype=torch.bfloat16), torch.zeros((), dtype=torch.int32),
           torch.zeros(4, dtype=torch.bfloat16), torch.zeros(1, 2, 3, 4, dtype=torch.bfloat16)]
    for name, call in calls.items():
        for v in bad:
            with pytest.raises(q3.Q3VLError):
                call(v)
                pytest.fail(f"{name} took {v!r}")
    with pytest.raises(q3.Q3VLError):
        q3.KvCacheQ8.of(c, e4.view(2, 200, 8, 128), e4, e8, e8)
    with pytest.raises(q3.Q3VLError):            # k alone on another device
        q3.KvCacheQ8.of(c, e4, e4.to("meta"), e8, e8)
    assert x.shape == (2, 2560)
