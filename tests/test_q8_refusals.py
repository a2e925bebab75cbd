"""Overlapping buffers of the 8-bit calls are refused before any CUDA call (no GPU)."""
import ctypes

import pytest
import torch

from test_abi import _cfg, lib  # noqa: F401  (fixture)


def _p(v):
    return ctypes.c_void_p(v)


def test_norm_refuses_outputs_over_inputs(lib):  # noqa: F811
    c = _cfg()
    S, row = 4, 2560
    x, d, h, q, s = (i << 30 for i in range(1, 6))

    def norm(x=x, d=d, h=h, q=q):
        return lib.q3vl_add_rms_norm_q8(ctypes.byref(c), _p(x), _p(d), S, None, _p(h), _p(q), _p(s),
                                        None)
    for kw in (dict(q=x), dict(q=x + S * row * 2 - 16), dict(q=d + 16), dict(q=h),
               dict(h=x + row * 2), dict(h=d + row * 2), dict(h=x - 16)):
        assert norm(**kw) == -1 and b"overlap" in lib.q3vl_last_error(), kw


def test_attention_refuses_an_output_that_starts_inside_its_query(lib):  # noqa: F811
    from qwen3_vl_decoder_b200 import _abi
    c = _cfg()
    kv = _abi.KvCacheQ8(1 << 32, 2 << 32, 3 << 32, 4 << 32, 64, 2)
    q, B, width = 5 << 32, 3, c.n_heads * 128

    def att(o):
        return lib.q3vl_attention_q8(ctypes.byref(c), _p(q), B, ctypes.byref(kv), _p(256), _p(256),
                                     _p(o), _p(256), 1, None)
    assert att(q + 2 * width) == -1 and b"overlap" in lib.q3vl_last_error()
    assert att(q - 16) == -1 and b"overlap" in lib.q3vl_last_error()
    # apart or the same: the next check answers (the workspace)
    assert att(q) == -5 and att(q + 2 * width * B) == -5


def test_binding_refuses_other_kinds_of_weights_caches_and_workspaces(lib):  # noqa: F811
    import qwen3_vl_decoder_b200 as q3
    c = _cfg()
    i = torch.zeros(2, dtype=torch.int32)
    k = torch.zeros(2, 1024, dtype=torch.bfloat16)
    q = torch.zeros(2, 4096, dtype=torch.bfloat16)
    w = torch.zeros(256, 2560, dtype=torch.uint8).view(torch.float8_e4m3fn)
    lin = q3.LinearQ8(w, torch.zeros(2, 20, dtype=torch.uint8).view(torch.float8_e8m0fnu))
    scales = torch.zeros(2, 20, dtype=torch.uint8).view(torch.float8_e8m0fnu)
    kv, kv8 = (q3.kv_caches(c, 1, 2, 200, "cpu", dtype=d)[0] for d in ("bf16", "fp8"))
    far = torch.empty(1 << 20, dtype=torch.uint8, device="meta")   # not the operands' device
    wide = torch.empty(1 << 20, dtype=torch.float32)
    for call, what in ((lambda: q3.linear_q8(w[:2], scales, w), "LinearQ8"),
                       (lambda: q3.kv_store_q8(c, k, k, kv, i, i), "KvCacheQ8"),
                       (lambda: q3.attention_q8(c, q, kv, i, i), "KvCacheQ8"),
                       (lambda: q3.attention_q8(c, q, kv8, i, i, ws=far), "ws is on"),
                       (lambda: q3.attention_q8(c, q, kv8, i, i, ws=wide), "ws must be"),
                       (lambda: q3.lm_head(c, k.new_zeros(2, 2560), None, lin, ws=far), "ws is on"),
                       (lambda: q3.lm_head(c, k.new_zeros(2, 2560), None, lin, ws=wide),
                        "ws must be")):
        with pytest.raises(q3.Q3VLError, match=what):
            call()
