"""Buffers of the 8-bit calls that overlap where they must not: refused before any CUDA call (no
GPU). Addresses are made up; nothing is read."""
import ctypes

import pytest

from test_abi import _cfg, lib  # noqa: F401  (fixture)

G = 1 << 32     # spacing of buffers that lie apart


def _p(v):
    return ctypes.c_void_p(v)


def _refused(lib, rc):  # noqa: F811
    return rc == -1 and b"overlap" in lib.q3vl_last_error()


def _cases(base, **over):
    return {**base, **over}


NORM = dict(x=G, d=2 * G, g=3 * G, h=4 * G, q=5 * G, s=6 * G)
S, H = 4, 2560
SIZE = dict(x=S * H * 2, d=S * H * 2, g=H * 2, h=S * H * 2, q=S * H, s=S * H // 128)


@pytest.mark.parametrize("out", ["h", "q", "s"])
@pytest.mark.parametrize("other", list(NORM))
def test_norm(lib, out, other):  # noqa: F811
    if out == other:
        return
    c = _cfg()
    for at in (NORM[other], NORM[other] + SIZE[other] - 16, NORM[other] - SIZE[out] + 16):
        a = _cases(NORM, **{out: at})
        if out == "h" and at in (a["x"], a["d"]):
            continue                       # in place
        if at < 0 or (out != "s" and at % 16):
            continue
        rc = lib.q3vl_add_rms_norm_q8(ctypes.byref(c), _p(a["x"]), _p(a["d"]), S, _p(a["g"]),
                                      _p(a["h"]), _p(a["q"]), _p(a["s"]), None)
        assert _refused(lib, rc), (out, other, at)


@pytest.mark.parametrize("kw", [dict(wq=G), dict(ws=G), dict(wq=G + 256 * 128 * 2 - 16),
                                dict(ws=2 * G + 256 * 128 - 1), dict(wq=3 * G)])
def test_weight(lib, kw):  # noqa: F811
    c = _cfg()
    a = {**dict(w=G, wq=2 * G, ws=3 * G), **kw}
    rc = lib.q3vl_quantize_weight_q8(ctypes.byref(c), _p(a["w"]), 256, 128, _p(a["wq"]), _p(a["ws"]),
                                     None)
    assert _refused(lib, rc)


LIN = dict(xq=G, xs=2 * G, wq=3 * G, ws=4 * G, resid=5 * G)


@pytest.mark.parametrize("other", list(LIN))
def test_product(lib, other):  # noqa: F811
    M, N, K = 64, 256, 512
    size = dict(xq=M * K, xs=M * 4, wq=N * K, ws=8, resid=M * N * 2)[other]
    for at in (LIN[other] + (16 if other == "resid" else 0), LIN[other] - M * N * 2 + 16,
               (LIN[other] + size - 1) // 16 * 16):
        rc = lib.q3vl_linear_q8(_p(LIN["xq"]), _p(LIN["xs"]), M, _p(LIN["wq"]), _p(LIN["ws"]), N, K,
                                _p(LIN["resid"]), _p(at), 1, None)
        assert _refused(lib, rc), (other, at)


@pytest.mark.parametrize("kw", [dict(logits=1 * G), dict(logits=2 * G), dict(logits=3 * G),
                                dict(logits=4 * G), dict(logits=5 * G), dict(w=1 * G),
                                dict(w=2 * G), dict(w=3 * G), dict(w=4 * G)])
def test_lm_head(lib, kw):  # noqa: F811
    c = _cfg()
    a = {**dict(x=G, n=2 * G, wq=3 * G, ws=4 * G, w=5 * G, logits=6 * G), **kw}
    need = lib.q3vl_lm_head_q8_workspace_bytes(ctypes.byref(c), 3)
    rc = lib.q3vl_lm_head_q8(ctypes.byref(c), _p(a["x"]), 3, _p(a["n"]), _p(a["wq"]), _p(a["ws"]),
                             1000, _p(a["logits"]), _p(a["w"]), need, None)
    assert _refused(lib, rc), kw


def test_lm_head_checks_the_product_before_it_starts(lib):  # noqa: F811
    c = _cfg()
    need = lib.q3vl_lm_head_q8_workspace_bytes(ctypes.byref(c), 3)

    def head(vocab=1000, wq=3 * G, logits=6 * G):
        before = lib.q3vl_launch_count()
        rc = lib.q3vl_lm_head_q8(ctypes.byref(c), _p(G), 3, None, _p(wq), _p(4 * G), vocab,
                                 _p(logits), _p(5 * G), need, None)
        assert lib.q3vl_launch_count() == before
        return rc
    assert head(vocab=0) == -1 and head(wq=None) == -1 and head(logits=6 * G + 8) == -1


def _kv():
    from qwen3_vl_decoder_b200 import _abi
    return _abi.KvCacheQ8(10 * G, 11 * G, 12 * G, 13 * G, 200, 2)


@pytest.mark.parametrize("part", range(4))
@pytest.mark.parametrize("what", ["k", "v"])
def test_store(lib, what, part):  # noqa: F811
    c, kv = _cfg(), _kv()
    size = 2 * 200 * 1024 if part < 2 else 2 * 2 * 8
    for at in ((10 + part) * G, (10 + part) * G + size - 16, (10 + part) * G - 16):
        a = {**dict(k=G, v=2 * G), what: at}
        rc = lib.q3vl_kv_store_q8(ctypes.byref(c), _p(a["k"]), _p(a["v"]), 6144, 3, None, 3,
                                  ctypes.byref(kv), _p(3 * G), _p(4 * G), None)
        assert _refused(lib, rc), (what, part, at)


@pytest.mark.parametrize("kw", [dict(o=(10 + i) * G) for i in range(4)] +
                         [dict(w=(10 + i) * G) for i in range(4)] +
                         [dict(o=10 * G + 2 * 200 * 1024 - 16), dict(w=G), dict(w=4 * G),
                          dict(o=5 * G + 256)])
def test_attention(lib, kw):  # noqa: F811
    c, kv, B = _cfg(), _kv(), 3
    a = {**dict(q=G, o=4 * G, w=5 * G), **kw}
    need = lib.q3vl_attention_q8_workspace_bytes(ctypes.byref(c), B, 200)
    rc = lib.q3vl_attention_q8(ctypes.byref(c), _p(a["q"]), B, ctypes.byref(kv), _p(2 * G), _p(3 * G),
                               _p(a["o"]), _p(a["w"]), need, None)
    assert _refused(lib, rc), kw
