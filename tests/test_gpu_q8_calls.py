"""The 8-bit operators as a program may call them: several tiles per CTA, alignments, far cache
slots, calls on two streams, captured calls replayed with other data, every head layout, and the
bounds-checked build. Tolerances as in test_gpu_q8.py, which has their derivation."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

from gpu_common import host, layer_on_device, q3
from oracle import q8_oracle as Q
import q3vl_synth as syn
from test_gpu_q8 import (HD, _cache, _cfg, _check_attention, _check_linear, _e8, _fill, _gen,
                         _rows8, _weight)

pytestmark = pytest.mark.gpu


def _i32(*v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _shifted(t, elems):
    """A contiguous copy of t on the device that starts `elems` elements behind an allocation."""
    raw = t.contiguous().view(torch.uint8) if t.element_size() == 1 else t.contiguous()
    buf = torch.empty(raw.numel() + elems, dtype=raw.dtype, device="cuda")
    out = buf[elems:].view(raw.shape)
    out.copy_(raw)
    return out.view(t.dtype)


@pytest.mark.parametrize("M,N,K,out_dtype", [
    (2100, 7008, 128, torch.bfloat16),      # four tiles per pair of CTAs, whole 32-byte units
    (2100, 7001, 192, torch.bfloat16),      # ... and rows that start anywhere
    (1300, 4004, 320, torch.float32), (700, 9000, 64, torch.float32),
    (1, 40000, 512, torch.float32), (70, 30000, 576, torch.bfloat16),
    (128, 2560, 9728, torch.bfloat16), (640, 640, 25600, torch.bfloat16)])
def test_linear_over_many_tiles(M, N, K, out_dtype):
    m = q3()
    xq, xs, x, sx = _rows8(M, K, M + N + K)
    lin = m.quantize_weight_q8(_weight(N, K, 7).cuda())
    r = torch.randn(M, N, generator=_gen(8)).to(out_dtype)
    got = m.linear_q8(xq.cuda(), xs.cuda(), lin, r.cuda(), out_dtype)
    m.check_device()
    # scaled operands in fp32 are exact (a 4-bit value times a power of two), their product in
    # fp64; the scales of _rows8 span 2^13, far from fp32's range
    a = torch.tensor(x * np.repeat(sx, 128, 1)[:, :K], device="cuda")
    sw = np.repeat(np.repeat(_e8(lin.scales), 128, 0)[:N], 128, 1)[:, :K]
    w = lin.weight.float().double() * torch.tensor(sw, device="cuda")
    want = (a @ w.t() + r.cuda().double()).cpu().numpy()
    mag = (a.abs() @ w.abs().t() + r.cuda().double().abs()).cpu().numpy()
    _check_linear(host(got), want, mag, K, out_dtype)


@pytest.mark.parametrize("M,N,K", [(5, 256, 512), (300, 1008, 512), (513, 2560, 1024)])
def test_linear_at_the_least_alignment(M, N, K):
    # scales at any byte, the residual and the output 16 bytes behind a 32-byte border: the bits of
    # the aligned call
    m = q3()
    xq, xs, _, _ = _rows8(M, K, 3)
    lin = m.quantize_weight_q8(_weight(N, K, 4).cuda())
    r = torch.randn(M, N, generator=_gen(5)).to(torch.bfloat16)
    want = m.linear_q8(xq.cuda(), xs.cuda(), lin, r.cuda())
    odd = m.LinearQ8(_shifted(lin.weight, 16), _shifted(lin.scales, 3))
    out = _shifted(torch.zeros_like(r), 8)
    got = m.linear_q8(_shifted(xq, 16), _shifted(xs, 1), odd, _shifted(r, 8), out=out)
    m.check_device()
    assert got is out and torch.equal(got, want)
    assert out.data_ptr() % 32 == 16


def test_linear_and_norm_leave_what_is_behind_their_outputs():
    m = q3()
    for M, N in ((3, 130), (300, 1000), (300, 1001), (257, 224 * 3)):
        xq, xs, _, _ = _rows8(M, 192, 6)
        lin = m.quantize_weight_q8(_weight(N, 192, 7).cuda())
        for dt in (torch.bfloat16, torch.float32):
            buf = torch.full((M * N + 4096,), 7.0, dtype=dt, device="cuda")
            m.linear_q8(xq.cuda(), xs.cuda(), lin, out_dtype=dt, out=buf[:M * N].view(M, N))
            assert torch.equal(buf[M * N:], torch.full_like(buf[M * N:], 7.0)), (M, N, dt)
    m.check_device()


@pytest.mark.parametrize("S,H,dtype", [(3000, 2560, "bf16"), (2500, 192, "bf16"),
                                       (1500, 5120, "fp32"), (40, 16384, "bf16")])
@pytest.mark.parametrize("delta", [False, True], ids=["plain", "delta"])
def test_norm_over_many_rows_matches_single_rows(S, H, dtype, delta):
    # a block's later rows against the same rows alone: the same bits
    m = q3()
    cfg = _cfg(H, dtype=dtype)
    dt = m.torch_dtype(cfg)
    x = torch.randn(S, H, generator=_gen(S)).to(dt).cuda()
    d = torch.randn(S, H, generator=_gen(H)).to(dt).cuda() if delta else None
    g = (1 + 0.1 * torch.randn(H, generator=_gen(1))).to(dt).cuda()
    h, q, s = m.add_rms_norm_q8(cfg, x, g, d)
    for r in (0, 1, S // 2, S - 2, S - 1):
        h1, q1, s1 = m.add_rms_norm_q8(cfg, x[r:r + 1], g, None if d is None else d[r:r + 1])
        assert torch.equal(h1, h[r:r + 1])
        assert torch.equal(q1.view(torch.uint8), q[r:r + 1].view(torch.uint8)), r
        assert torch.equal(s1.view(torch.uint8), s[r:r + 1].view(torch.uint8)), r
    m.check_device()


def test_norm_of_zero_rows_and_infinite_sums():
    # a zero row stays zero; an overflowing sum of squares gives 1 / rms = 0
    m = q3()
    cfg = _cfg(256, dtype="fp32")
    x = torch.zeros(3, 256)
    x[1] = 1e30
    x[2, 5] = float("inf")
    h, q, s = m.add_rms_norm_q8(cfg, x.cuda(), torch.ones(256).cuda())
    m.check_device()
    q = host(q)
    assert not q[0].any() and not q[1].any()
    assert np.isnan(q[2, 5]) and not np.delete(q[2], 5).any()


LAYOUTS = [(nkv * G, nkv) for nkv in (1, 2, 3, 8, 16) for G in (1, 2, 4, 8)]


@pytest.mark.parametrize("nh,nkv", LAYOUTS, ids=[f"{a}-{b}" for a, b in LAYOUTS])
def test_attention_head_layouts(nh, nkv):
    m = q3()
    cfg = _cfg(nh=nh, nkv=nkv)
    lens = [1, 0, 640, 257, 31]
    kv = _cache(cfg, len(lens), 700, 60)
    ref = _fill(cfg, kv, lens, 61)
    q = torch.randn(len(lens), nh * HD, generator=_gen(62)).to(torch.bfloat16)
    o = m.attention_q8(cfg, q.cuda(), kv, _i32(*range(len(lens))), _i32(*lens))
    m.check_device()
    _check_attention(cfg, host(o), q, ref, range(len(lens)), lens)


def test_attention_over_the_longest_slot_and_the_most_sequences():
    m = q3()
    cfg = _cfg(nh=2, nkv=1)
    lens = [131072]
    kv = _cache(cfg, 1, 131072, 70)
    ref = _fill(cfg, kv, lens, 71, spread=1.0)
    q = (3 * torch.randn(1, 2 * HD, generator=_gen(72))).to(torch.bfloat16)
    o = m.attention_q8(cfg, q.cuda(), kv, _i32(0), _i32(*lens))
    m.check_device()
    _check_attention(cfg, host(o), q, ref, [0], lens)
    cfg = _cfg(nh=8, nkv=2)
    lens = [(37 * b) % 300 for b in range(256)]
    kv = _cache(cfg, 256, 300, 73)
    ref = _fill(cfg, kv, lens, 74)
    q = torch.randn(256, 8 * HD, generator=_gen(75)).to(torch.bfloat16)
    o = m.attention_q8(cfg, q.cuda(), kv, _i32(*range(256)), _i32(*lens))
    m.check_device()
    _check_attention(cfg, host(o), q, ref, range(256), lens)


def test_slots_beyond_the_reach_of_32_bits():
    # 20 slots of 131072 rows of 1024 bytes: the last ones start past 2^31 bytes; the same rows
    # stored and read in a small cache give the same bits
    m = q3()
    cfg = _cfg(nh=32, nkv=8)
    big, small = m.KvCacheQ8(cfg, 20, 131072), m.KvCacheQ8(cfg, 1, 700)
    k = torch.randn(600, 1024, generator=_gen(80)).to(torch.bfloat16).cuda()
    v = torch.randn(600, 1024, generator=_gen(81)).to(torch.bfloat16).cuda()
    q = torch.randn(1, 4096, generator=_gen(82)).to(torch.bfloat16).cuda()
    st, out = _i32(0, 600), []
    for kv, slot in ((big, 19), (small, 0)):
        m.kv_store_q8(cfg, k, v, kv, _i32(slot), _i32(0), st)
        out.append(m.attention_q8(cfg, q, kv, _i32(slot), _i32(600)))
        m.kv_store_q8(cfg, 40 * k[:1], v[:1], kv, _i32(slot), _i32(600))
        out.append(m.attention_q8(cfg, q, kv, _i32(slot), _i32(601)))
    m.check_device()
    assert torch.equal(out[0], out[2]) and torch.equal(out[1], out[3])
    for a, b in ((big.k, small.k), (big.v, small.v)):
        assert torch.equal(a[19, :601].view(torch.uint8), b[0, :601].view(torch.uint8))
        assert not a[0].view(torch.uint8).any() and not a[19, 601:1000].view(torch.uint8).any()


def test_calls_on_two_streams_at_once():
    m = q3()
    cfg = _cfg(nh=16, nkv=8)
    sides = []
    for i in range(2):
        lens = [3000 - 700 * i, 50, 1200]
        kv = _cache(cfg, 3, 3100, 90 + i)
        _fill(cfg, kv, lens, 92 + i)
        q = torch.randn(3, 16 * HD, generator=_gen(94 + i)).to(torch.bfloat16).cuda()
        x = torch.randn(600, 2560, generator=_gen(96 + i)).to(torch.bfloat16).cuda()
        lin = m.quantize_weight_q8(_weight(3000, 2560, 98 + i).cuda())
        sides.append((kv, q, _i32(0, 1, 2), _i32(*lens), x, lin))

    def run(side, stream=None):
        kv, q, seq, ln, x, lin = side
        out = []
        for _ in range(6):
            _, xq, xs = m.add_rms_norm_q8(cfg, x, None, stream=stream)
            out.append(m.linear_q8(xq, xs, lin, stream=stream))
            out.append(m.linear_q8(xq[:3], xs[:3], lin, stream=stream))
            out.append(m.attention_q8(cfg, q, kv, seq, ln, stream=stream))
        return out
    want = [run(s) for s in sides]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [run(s, st) for s, st in zip(sides, streams)]
    torch.cuda.synchronize()
    m.check_device()
    for w, g in zip(want, got):
        assert all(torch.equal(a, b) for a, b in zip(w, g))


def test_captured_calls_replayed_with_other_data():
    # norm, product, store and attention in one graph, two graphs of one workspace in turn: inputs,
    # lengths and cache change between replays
    m = q3()
    cfg = _cfg(256, nh=8, nkv=2)
    B, K = 3, 256
    kv = _cache(cfg, B, 500, 100, poison=False)
    lin = m.quantize_weight_q8(_weight(12 * HD, K, 101).cuda())
    x = torch.zeros(B, K, dtype=torch.bfloat16, device="cuda")
    gain = torch.ones(K, dtype=torch.bfloat16, device="cuda")
    ln, seq = _i32(0, 130, 400), _i32(2, 0, 1)
    ws = m.attention_q8_workspace(cfg, B, kv.cap)
    one = torch.ones(B, dtype=torch.int32, device="cuda")

    def step():
        _, xq, xs = m.add_rms_norm_q8(cfg, x, gain)
        qkv = m.linear_q8(xq, xs, lin)
        m.kv_store_q8(cfg, qkv[:, 8 * HD:10 * HD], qkv[:, 10 * HD:], kv, seq, ln)
        ln.add_(one)
        return m.attention_q8(cfg, qkv[:, :8 * HD].contiguous(), kv, seq, ln, ws=ws)
    rows = torch.randn(6, B, K, generator=_gen(102)).to(torch.bfloat16).cuda()
    keep = [t.clone() for t in (kv.k, kv.v, kv.k_scale, kv.v_scale, ln)]

    def reset():
        for t, old in zip((kv.k, kv.v, kv.k_scale, kv.v_scale, ln), keep):
            t.copy_(old)
    want = []
    for r in rows:
        x.copy_(r)
        want.append(step().clone())
    reset()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graphs, outs = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(step())
        graphs.append(g)
    reset()
    for i, r in enumerate(rows):
        x.copy_(r)
        graphs[i % 2].replay()
        assert torch.equal(outs[i % 2], want[i]), i
    m.check_device()


@pytest.mark.parametrize("level", [2.0 ** -9, 1.0, 300.0], ids=["grows", "even", "keeps"])
@pytest.mark.parametrize("lens", [[0, 1, 127, 128, 129, 255, 256, 700], [300], [7] * 70],
                         ids=["borders", "one", "b70"])
def test_decode_appends_the_row_that_the_store_would(lens, level):
    # the same layer step on a bf16 cache tells the row; the 8-bit cache gets it by the store's
    # rule: below, near and above the magnitude of what its blocks hold
    m = q3()
    w = syn.Q2B_LAYER
    cfg = m.config_of(w)
    _, packed = layer_on_device(w)
    B, nkv, cap = len(lens), w.n_kv_heads, max(lens) + 1
    kv8, kv = m.kv_caches(cfg, 1, B, cap, dtype="fp8")[0], m.kv_caches(cfg, 1, B, cap)[0]
    seq, ln = _i32(*reversed(range(B))), _i32(*lens)
    ref = []
    for b, n in enumerate(lens):
        rows = (level * torch.randn(2, max(n, 1), nkv * HD, generator=_gen(200 + b))).to(
            torch.bfloat16)
        slot = []
        for i in range(2):
            c, s = np.zeros((cap, nkv, HD)), np.ones((-(-cap // 128), nkv))
            if n:
                Q.store(c, s, rows[i, :n].double().numpy().reshape(n, nkv, HD), 0)
            slot.append((c, s))
        if n:
            r = rows.cuda()
            m.kv_store_q8(cfg, r[0], r[1], kv8, seq[b:b + 1].clone(), _i32(0), _i32(0, n))
        ref.append(slot)
    x = torch.randn(B, w.hidden, generator=_gen(300)).to(torch.bfloat16).cuda()
    pos = ln.repeat(3, 1).contiguous()
    m.layer_decode(cfg, packed, x.clone(), pos, kv, seq, ln)      # writes the bf16 rows alone
    m.layer_decode(cfg, packed, x.clone(), pos, kv8, seq, ln)
    m.check_device()
    for b, n in enumerate(lens):
        at = B - 1 - b
        for i, (t, sc, full) in enumerate(((kv8.k, kv8.k_scale, kv.k), (kv8.v, kv8.v_scale, kv.v))):
            c, s = ref[b][i]
            Q.store(c, s, host(full[at, n:n + 1]).reshape(1, nkv, HD), n)
            assert np.array_equal(host(t[at, :n + 1]).reshape(n + 1, nkv, HD), c[:n + 1]), (b, i)
            nb = n // 128 + 1
            assert np.array_equal(_e8(sc[at, :nb]), s[:nb]), (b, i)


DEBUG = r"""
import sys
sys.path[:0] = [{root!r}, {tests!r}]
import torch
import qwen3_vl_decoder_b200 as m
import test_gpu_q8 as T
assert m._abi.LIB_PATH.endswith("libq3vl_debug.so")
for M, N, K in ((1, 1, 64), (33, 2560, 1216), (129, 257, 320), (300, 1000, 2560), (513, 2049, 192)):
    for dt in (torch.bfloat16, torch.float32):
        T.test_linear_matches_the_oracle(M, N, K, dt, True)
for lens, new, cap in T.STORE:
    T.test_store_is_exact(lens, new, cap, 300.0)
for nh, nkv, lens in T.ATTEND[:4]:
    T.test_attention_matches_the_oracle(nh, nkv, lens)
T.test_layer_decode_over_the_8bit_cache(T.syn.Q2B_LAYER, [0, 1, 127, 128, 300])
T.test_norm_matches_the_oracle(700, 2560, "bf16", True, True)
m.check_device()
print("clean")
"""


def test_bounds_checked_build_finds_nothing():
    here = os.path.dirname(os.path.abspath(__file__))
    code = DEBUG.format(root=os.path.dirname(here), tests=here)
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=600,
                       env={**os.environ, "Q3VL_LIBRARY": "debug"}, cwd=os.path.dirname(here))
    assert r.returncode == 0 and r.stdout.strip().endswith("clean"), r.stderr[-2000:]
