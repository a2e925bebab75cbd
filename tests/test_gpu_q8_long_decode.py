"""Decode over 8-bit caches where it is used: parts of many chunks, batches of two, segments that
cross parts, tiles loaded ahead of the projection and then the appended row in the middle of a part.

The layer is made so that its output is the attention alone: the output projection is the identity,
the down projection zero, and the input is 2^-10 of what the attention gives. Its query, key and value
follow in 64 bits; positions are 0, where the rotation is none.

Tolerance. Gains are one, so that the packed weights are exact. The projections' bf16 results
(2^-8 of each element, after the norm of each head; the sums in fp32 are far better) move a score of
N(0, 1) by at most a few times 2^-8 / sqrt(3); the appended value row is rounded the same way before
its 8 bits, which are read back as they are. The output is rounded to bf16 twice. Errors of the scores
are independent, so each head's output is off by less than 2^-8 of itself on average over its 128
elements, times a few: 2^-6 is allowed. One chunk of 128 tokens left out of 4096, or read twice, is
off by sqrt(1 / 32) = 18%.
"""
import numpy as np
import pytest
import torch

from gpu_common import host, q3
from oracle import q8_oracle as Q
from test_gpu_q8 import HD, _e8, _gen

pytestmark = pytest.mark.gpu
NKV = 8


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _layer(G, seed):
    m = q3()
    nh = NKV * G
    H = nh * HD
    cfg = m.config(H, nh, NKV, 128, "bf16")
    g = torch.Generator(device="cuda").manual_seed(seed)

    def draw(*shape):
        return (0.02 * torch.randn(*shape, generator=g, device="cuda")).to(torch.bfloat16)

    def ones(n):
        return torch.ones(n, dtype=torch.bfloat16, device="cuda")
    raw = dict(attn_norm=ones(H), wq=draw(H, H), wk=draw(NKV * HD, H), wv=draw(NKV * HD, H),
               q_norm=ones(HD), k_norm=ones(HD),
               wo=torch.eye(H, dtype=torch.bfloat16, device="cuda"), ffn_norm=ones(H),
               wg=draw(128, H), wu=draw(128, H), wd=0 * draw(H, 128))
    return cfg, raw, m.pack_layer(cfg, raw)


def _caches(cfg, lens, extra, seed):
    """An 8-bit cache with lens[b] random rows in slot seq[b], stored in one call."""
    m = q3()
    kv = m.kv_caches(cfg, 1, len(lens), max(lens) + extra, dtype="fp8")[0]
    g = torch.Generator(device="cuda").manual_seed(seed)
    T = max(sum(lens), 1)
    k, v = (torch.randn(T, NKV * HD, generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    seq = torch.randperm(len(lens), generator=_gen(seed)).to(torch.int32)
    starts = _i32(np.cumsum([0] + list(lens)).tolist())
    m.kv_store_q8(cfg, k, v, kv, seq.cuda(), _i32([0] * len(lens)), starts)
    m.check_device()
    return kv, seq.cuda()


def _projected(raw, x, G):
    """q, k, v of rows x in 64 bits: [B, nh, 128], [B, nkv, 128], [B, nkv, 128]."""
    d = torch.float64
    xs = x.to(d)
    xs = xs / torch.sqrt(xs.square().mean(1, keepdim=True) + 1e-6)

    def heads(w):
        return (xs @ raw[w].to(d).t()).view(len(x), -1, HD)

    def unit(t):
        return t / torch.sqrt(t.square().mean(2, keepdim=True) + 1e-6)
    return unit(heads("wq")), unit(heads("wk")), heads("wv")


def _check(cfg, raw, x, got, kv, seq, lens, before):
    """The appended rows by the store's rule, and the output by 64-bit attention over the cache."""
    G = cfg.n_heads // NKV
    q, k, v = _projected(raw, x, G)
    d = torch.float64
    after = (kv.k, kv.v, kv.k_scale, kv.v_scale)
    out = (got.to(d) - x.to(d)).view(len(lens), NKV, G, HD)
    for b, n in enumerate(lens):
        s, nb = int(seq[b]), n // 128 + 1
        deq = []
        for i, new in ((0, k), (1, v)):
            c = after[i][s, :n + 1].float().to(d).view(n + 1, NKV, HD)
            u = torch.exp2(after[2 + i][s, :nb].view(torch.uint8).to(d) - 127)
            deq.append(c * u.repeat_interleave(128, 0)[:n + 1, :, None])
            # the new row within bf16 and then 8 bits of the projection
            row, want = deq[i][n], new[b]
            lim = (2.0 ** -4 + 2.0 ** -7) * want.abs() + 2.0 ** -7 * want.abs().amax(
                1, keepdim=True) + 2.0 ** -10 * u[-1][:, None]
            assert bool(((row - want).abs() <= lim).all()), (b, i)
            # earlier full blocks and what lies behind are as they were
            assert torch.equal(after[i][s, :(nb - 1) * 128].view(torch.uint8),
                               before[i][s, :(nb - 1) * 128].view(torch.uint8))
            assert torch.equal(after[i][s, n + 1:].view(torch.uint8),
                               before[i][s, n + 1:].view(torch.uint8))
        qb = q[b].view(NKV, G, HD)
        w = torch.softmax(torch.einsum("hgd,thd->hgt", qb, deq[0]) / HD ** 0.5, 2)
        want = torch.einsum("hgt,thd->hgd", w, deq[1])
        off = (out[b] - want).norm(dim=2) / want.norm(dim=2)
        assert float(off.max()) <= 2.0 ** -6, (b, n, float(off.max()))


LENS = {
    "long": [4096, 4095, 8191, 127, 0, 128, 2000, 6399],      # parts of 5 to 6 chunks
    "many": [(53 * b) % 390 for b in range(256)],             # parts of a dozen sequences
    "one": [5000],
    "even": [4096] * 32,
}


@pytest.mark.parametrize("which,G", [("long", 1), ("long", 2), ("long", 4), ("long", 8), ("many", 1),
                                     ("many", 4), ("many", 8), ("one", 8), ("one", 2), ("even", 4)])
def test_decode_over_many_chunks(which, G):
    m = q3()
    lens = LENS[which]
    cfg, raw, packed = _layer(G, 100 + G)
    kv, seq = _caches(cfg, lens, 3, 7 * G)
    before = [t.clone() for t in (kv.k, kv.v, kv.k_scale, kv.v_scale)]
    B = len(lens)
    x = (2.0 ** -10 * torch.randn(B, cfg.hidden, generator=_gen(G))).to(torch.bfloat16).cuda()
    pos = torch.zeros(3, B, dtype=torch.int32, device="cuda")
    outs = []
    for fill in (0, 0xFF):                    # the same bits, whatever the workspace held
        for t, old in zip((kv.k, kv.v, kv.k_scale, kv.v_scale), before):
            t.copy_(old)
        ws = m.decode_workspace(cfg, B, kv.cap, dtype="fp8").fill_(fill)
        xd = x.clone()
        m.layer_decode(cfg, packed, xd, pos, kv, seq, _i32(lens), ws)
        m.check_device()
        outs.append(xd)
    assert torch.equal(outs[0], outs[1])
    _check(cfg, raw, x, outs[0], kv, seq, lens, before)


@pytest.mark.parametrize("G", [4, 8])
def test_steps_of_a_captured_stack_over_many_chunks(G):
    # two layers, three steps across a block border, replayed from one graph: the bits of eager steps
    m = q3()
    lens = [4094, 1000, 127, 3000]
    B = len(lens)
    cfg, raw, packed = _layer(G, 200 + G)
    layers = [packed, _layer(G, 300 + G)[2]]
    pairs = [_caches(cfg, lens, 8, 9), _caches(cfg, lens, 8, 9)]
    kvs, seq = [p[0] for p in pairs], pairs[0][1]
    tensors = [t for kv in kvs for t in (kv.k, kv.v, kv.k_scale, kv.v_scale)]
    keep = [t.clone() for t in tensors]
    ln, pos = _i32(lens), torch.zeros(3, B, dtype=torch.int32, device="cuda")
    ws = m.decode_workspace(cfg, B, kvs[0].cap, dtype="fp8")
    xin = (2.0 ** -10 * torch.randn(3, B, cfg.hidden, generator=_gen(G))).to(torch.bfloat16).cuda()
    x = xin[0].clone()

    def step():
        m.stack_decode(cfg, layers, x, pos, kvs, seq, ln, ws=ws)
        m.decode_advance(pos, ln)

    def reset():
        for t, old in zip(tensors, keep):
            t.copy_(old)
        ln.copy_(_i32(lens))
        pos.zero_()
    want = []
    for r in xin:
        x.copy_(r)
        step()
        want.append(x.clone())
    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    with torch.cuda.graph(graph):
        step()
    reset()
    for r, w in zip(xin, want):
        x.copy_(r)
        graph.replay()
        assert torch.equal(x, w)
    m.check_device()


DEBUG = r"""
import sys
sys.path[:0] = [{root!r}, {tests!r}]
import qwen3_vl_decoder_b200 as m
import test_gpu_q8_long_decode as T
import test_gpu_q8_sinks as K
assert m._abi.LIB_PATH.endswith("libq3vl_debug.so")
for which, G in (("long", 1), ("long", 8), ("many", 4)):
    T.test_decode_over_many_chunks(which, G)
for G in (1, 8):
    K.test_attention_with_a_sink(G, [33, 128, 1000, 5000], [0, 127, 300, 4999], 16.0, 0.0)
m.check_device()
print("clean")
"""


def test_bounds_checked_build_finds_nothing_in_long_decodes():
    import os
    import subprocess
    import sys
    here = os.path.dirname(os.path.abspath(__file__))
    code = DEBUG.format(root=os.path.dirname(here), tests=here)
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=600,
                       env={**os.environ, "Q3VL_LIBRARY": "debug"}, cwd=os.path.dirname(here))
    assert r.returncode == 0 and r.stdout.strip().endswith("clean"), r.stderr[-2000:]
