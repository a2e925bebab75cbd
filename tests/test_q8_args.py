"""Refusals of the 8-bit operators (no GPU): they return before any CUDA call."""
import ctypes

import pytest
import torch

from test_abi import _cfg, lib  # noqa: F401  (fixture)

P = ctypes.c_void_p(256)


def _kv8(cap=64, n_seq=2, k=256):
    from qwen3_vl_decoder_b200 import _abi
    return _abi.KvCacheQ8(k, 512, 768, 1024, cap, n_seq)


def test_norm_arguments(lib):  # noqa: F811
    def norm(cfg=_cfg(), x=P, delta=None, S=4, gain=P, h=None, q=P, s=P):
        return lib.q3vl_add_rms_norm_q8(ctypes.byref(cfg), x, delta, S, gain, h, q, s, None)
    assert norm(S=0) == -1
    assert norm(x=None) == -1 and norm(q=None) == -1 and norm(s=None) == -1
    assert norm(x=ctypes.c_void_p(8)) == -1
    assert norm(delta=P) == -1 and b"h is NULL" in lib.q3vl_last_error()
    assert norm(cfg=_cfg(hidden=32768 + 64)) == -8
    assert norm(cfg=_cfg(head_dim=64)) == -8


def test_linear_arguments(lib):  # noqa: F811
    A = [ctypes.c_void_p((i + 1) << 30) for i in range(6)]

    def lin(M=4, N=100, K=128, resid=None, out=A[4], dt=1, xq=A[0], wq=A[2]):
        return lib.q3vl_linear_q8(xq, A[1], M, wq, A[3], N, K, resid, out, dt, None)
    assert lin(M=0) == -1 and lin(N=0) == -1 and lin(K=0) == -1
    assert lin(K=96) == -1 and lin(K=100) == -1
    assert lin(M=(1 << 30) + 1) == -1
    assert lin(dt=2) == -8
    assert lin(xq=None) == -1 and lin(wq=ctypes.c_void_p(8)) == -1
    assert lin(out=A[0]) == -1 and b"overlap" in lib.q3vl_last_error()
    assert lin(resid=ctypes.c_void_p(A[4].value + 16)) == -1
    c = _cfg()
    assert lib.q3vl_quantize_weight_q8(ctypes.byref(c), P, 8, 100, P, P, None) == -1
    assert lib.q3vl_quantize_weight_q8(ctypes.byref(c), P, 0, 128, P, P, None) == -1


def test_lm_head_arguments(lib):  # noqa: F811
    c = _cfg()
    assert lib.q3vl_lm_head_q8_workspace_bytes(ctypes.byref(c), 3) == 3 * 2560 + 256
    assert lib.q3vl_lm_head_q8_workspace_bytes(ctypes.byref(c), 0) == 0

    def head(cfg=c, B=1, n=1 << 20):
        return lib.q3vl_lm_head_q8(ctypes.byref(cfg), P, B, None, P, P, 1000, P, P, n, None)
    assert head(cfg=_cfg(dtype="fp32")) == -8
    assert head(B=0) == -1 and head(B=257) == -1 and head(n=100) == -5


def test_store_arguments(lib):  # noqa: F811
    c = _cfg()

    def store(cfg=c, k=P, ld=1024, T=2, starts=None, B=2, kv=_kv8(), seq=P, length=P):
        return lib.q3vl_kv_store_q8(ctypes.byref(cfg), k, P, ld, T, starts, B, ctypes.byref(kv),
                                    seq, length, None)
    assert store(cfg=_cfg(dtype="fp32")) == -8
    assert store(B=0) == -1 and store(B=257, T=257) == -1
    assert store(T=3) == -1                       # without starts one row per sequence
    assert store(T=0, starts=P) == -1
    assert store(ld=1016) == -1 and store(ld=1028) == -1
    assert store(k=ctypes.c_void_p(8)) == -1 and store(seq=None) == -1 and store(length=None) == -1
    assert store(kv=_kv8(cap=0)) == -1 and store(kv=_kv8(cap=131073)) == -8
    assert store(kv=_kv8(cap=131072, n_seq=1 << 15)) == -1 and store(kv=_kv8(k=8)) == -1


def test_attention_and_decode_arguments(lib):  # noqa: F811
    from qwen3_vl_decoder_b200 import _abi
    c = _cfg()
    size = lib.q3vl_attention_q8_workspace_bytes
    assert size(ctypes.byref(c), 4, 1000) > 0
    assert size(ctypes.byref(c), 0, 1000) == 0 and size(ctypes.byref(c), 4, 0) == 0
    assert size(ctypes.byref(_cfg(n_heads=24)), 4, 1000) == 0

    def att(cfg=c, B=2, kv=_kv8(), ws=P, n=1 << 40):
        return lib.q3vl_attention_q8(ctypes.byref(cfg), P, B, ctypes.byref(kv), P, P, P, ws, n,
                                     None)
    assert att(cfg=_cfg(dtype="fp32")) == -8 and att(cfg=_cfg(n_heads=24)) == -8
    assert att(B=0) == -1 and att(B=257) == -1 and att(kv=_kv8(cap=0)) == -1
    assert att(n=1) == -5 and att(ws=None) == -5 and att(ws=ctypes.c_void_p(264)) == -5
    lay = _abi.Layer(*[256] * 7)

    def dec(cfg=c, B=2, kv=_kv8(), n=1 << 40):
        return lib.q3vl_layer_decode_q8(ctypes.byref(cfg), ctypes.byref(lay), P, B, P,
                                        ctypes.byref(kv), P, P, P, n, None)
    assert dec(B=0) == -1 and dec(n=1024) == -5 and dec(kv=_kv8(cap=0)) == -1
    assert dec(cfg=_cfg(dtype="fp32")) == -8
    assert lib.q3vl_stack_decode_q8(ctypes.byref(c), 0, ctypes.byref(lay), None, P, 2, P,
                                    ctypes.byref(_kv8()), P, P, P, 1 << 40, None) == -1
    pk = lambda S, seq, kv: lib.q3vl_layer_prefill_kv_q8(  # noqa: E731
        ctypes.byref(c), ctypes.byref(lay), P, S, P, None, None, 0, ctypes.byref(kv), seq, P,
        1 << 40, None)
    assert pk(65, 0, _kv8()) == -2 and pk(8, 2, _kv8()) == -2 and pk(8, 0, _kv8(cap=0)) == -1


def test_binding_refuses_wrong_tensors(lib):  # noqa: F811
    import qwen3_vl_decoder_b200 as q3
    c = _cfg()
    with pytest.raises(q3.Q3VLError):            # CPU tensors
        q3.add_rms_norm_q8(c, torch.zeros(2, 2560, dtype=torch.bfloat16), None)
    bf = torch.zeros(2, 2560, dtype=torch.bfloat16)
    for x, kw in ((bf.float(), {}), (bf[:, :64], {}), (bf, dict(delta=bf[:1])),
                  (bf, dict(h=bf.clone())), (bf.t().contiguous().t(), {})):
        with pytest.raises(q3.Q3VLError):
            q3.add_rms_norm_q8(c, x, None, **kw)
    w = torch.zeros(256, 128, dtype=torch.uint8).view(torch.float8_e4m3fn)
    s = torch.zeros(2, 1, dtype=torch.uint8).view(torch.float8_e8m0fnu)
    lin = q3.LinearQ8(w, s)
    assert lin.shape == (256, 128)
    for bad in ((w, s[:1]), (w.view(torch.uint8), s), (w[:, :64], s)):
        with pytest.raises(q3.Q3VLError):
            q3.LinearQ8(*bad)
    xq = torch.zeros(3, 128, dtype=torch.uint8).view(torch.float8_e4m3fn)
    xs = torch.zeros(3, 1, dtype=torch.uint8).view(torch.float8_e8m0fnu)
    for args, kw in (((xq[:, :64].contiguous(), xs, lin), {}), ((xq, xs[:2], lin), {}),
                     ((xq, xs, lin), dict(out_dtype=torch.float16)),
                     ((xq, xs, lin), dict(resid=torch.zeros(3, 256)))):
        with pytest.raises(q3.Q3VLError):
            q3.linear_q8(*args, **kw)
    with pytest.raises(q3.Q3VLError):
        q3.kv_caches(c, 1, 1, 8, "cpu", dtype="int8")
    kv = q3.kv_caches(c, 1, 2, 200, "cpu", dtype="fp8")[0]
    assert kv.cap == 200 and kv.k_scale.shape == (2, 2, 8)
    with pytest.raises(q3.Q3VLError):            # one kind of cache per stack
        q3._kv_array([kv, q3.KvCache(c, 2, 200, "cpu")])
    k = torch.zeros(2, 1024, dtype=torch.bfloat16)
    i = torch.zeros(2, dtype=torch.int32)
    for args in ((k.float(), k, kv, i, i), (k[:, :512], k, kv, i, i), (k, k[:1], kv, i, i),
                 (k, k, kv, i.long(), i), (k, k, kv, i, i, i),
                 (k.expand(2, 1024)[:1].expand(2, 1024), k, kv, i, i)):
        with pytest.raises(q3.Q3VLError):
            q3.kv_store_q8(c, *args)
    q = torch.zeros(2, 4096, dtype=torch.bfloat16)
    for args in ((q.float(), kv, i, i), (q[:, :128], kv, i, i), (q, kv, i[:1], i),
                 (q, kv, i, i.long())):
        with pytest.raises(q3.Q3VLError):
            q3.attention_q8(c, *args)
