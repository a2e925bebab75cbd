"""Attention over the 8-bit cache where one token's score stands far above the others' and its value
row is small: thousands of tokens of tiny probability then carry the output.

Tolerance. A probability is the sum of three e5m2 parts, each rounded by at most 2^-3 of what the
part before left over, so by 2^-9 of itself, down to 2^-28 of the largest among the tokens that share
its scale (below that by 2^-37 of that largest one). Scores here lie within 19.4 nats = 28 bits of the
sink's. Besides the probabilities: q to 2^-18 of its largest element and fp32 scores, which move a
score of at most 20 nats by less than 1e-3, so all probabilities by less than 2^-9.9; and the bf16
rounding of the output, 2^-8 of it. Together less than 2^-7 of the weighted mean of |v|, and 2^-8 of
the output.
"""
import math

import numpy as np
import pytest
import torch

from gpu_common import host, q3
from oracle import q8_oracle as Q
from test_gpu_q8 import HD, _cache, _cfg, _check_attention, _gen

pytestmark = pytest.mark.gpu


def _slots(cfg, q, lens, cap, gap, at, value, seed):
    """A cache whose slot b has lens[b] rows: scores of N(0, 0.3) nats, but `gap` at row at[b] for
    every head of a group; values N(0, 1), at row at[b] times `value`. Returns it and the oracle's
    copy."""
    nkv = cfg.n_kv_heads
    G = cfg.n_heads // nkv
    kv = _cache(cfg, len(lens), cap, seed)
    ref = []
    for b, n in enumerate(lens):
        base = q[b].double().view(nkv, G, HD).mean(1)
        sq = (base * base).sum(1, keepdim=True)
        slot = []
        for i, (t, sc) in enumerate(((kv.k, kv.k_scale), (kv.v, kv.v_scale))):
            rows = torch.randn(n, nkv, HD, generator=_gen(seed + 2 * b + i)).double()
            if i == 0:
                rows -= (rows * base).sum(2, keepdim=True) / sq * base      # no score at all
                rows *= 0.3
                rows += 0.3 * math.sqrt(HD) * torch.randn(n, nkv, 1, generator=_gen(seed + 77 + b)
                                                          ).double().clamp(-3, 3) * base / sq
                rows[at[b]] = gap * math.sqrt(HD) * base / sq
            else:
                rows[at[b]] *= value
            c, s = np.zeros((cap, nkv, HD)), np.zeros((-(-cap // 128), nkv))
            Q.store(c, s, rows.to(torch.bfloat16).double().numpy(), 0)
            t[b, :n] = torch.tensor(c[:n].reshape(n, -1)).float().to(torch.float8_e4m3fn).cuda()
            nb = -(-n // 128)
            sc[b, :nb] = torch.tensor(np.log2(s[:nb]) + 127).to(torch.uint8).view(
                torch.float8_e8m0fnu).cuda()
            slot += [c, s]
        ref.append(slot)
    return kv, ref


def _grouped_q(B, nkv, G, seed):
    """Query heads of a group near one another, so that one key row can face them all."""
    base = torch.randn(B, nkv, 1, HD, generator=_gen(seed))
    q = base + 0.02 * torch.randn(B, nkv, G, HD, generator=_gen(seed + 1))
    return q.reshape(B, nkv * G * HD).to(torch.bfloat16)


@pytest.mark.parametrize("value", [0.0, 0.01, 1.0])
@pytest.mark.parametrize("gap", [14.0, 16.0, 17.5])
@pytest.mark.parametrize("lens,at", [([40], [0]), ([200], [130]), ([2048], [0]), ([8192], [700]),
                                     ([33, 128, 1000, 5000], [0, 127, 300, 4999])],
                         ids=["40", "200", "2048", "8192", "four"])
@pytest.mark.parametrize("G", [1, 2, 4, 8])
def test_attention_with_a_sink(G, lens, at, gap, value):
    m = q3()
    nkv = 2
    cfg = _cfg(nh=nkv * G, nkv=nkv)
    B = len(lens)
    q = _grouped_q(B, nkv, G, 5)
    kv, ref = _slots(cfg, q, lens, max(lens) + 5, gap, at, value, 300)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    o = m.attention_q8(cfg, q.cuda(), kv, i32(list(range(B))), i32(lens))
    m.check_device()
    _check_attention(cfg, host(o), q, ref, range(B), lens)


def test_a_sequence_does_not_change_with_its_neighbours():
    # the same sequence alone (its parts a cluster) and among others (the list's parts): both within
    # the bound, wherever its segments end
    m = q3()
    cfg = _cfg(nh=8, nkv=2)
    n, gap = 6000, 16.5
    q1 = _grouped_q(1, 2, 4, 9)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    for others in ([], [100], [6000, 3, 2500], [777] * 40):
        q = q1.expand(1 + len(others), -1).contiguous()
        lens = [n] + others
        kv, ref = _slots(cfg, q, lens, n, gap, [0] * len(lens), 0.0, 400)
        o = m.attention_q8(cfg, q.cuda(), kv, i32(list(range(len(lens)))), i32(lens))
        m.check_device()
        _check_attention(cfg, host(o), q, ref, range(len(lens)), lens)


def test_a_sink_beyond_the_parts_range_keeps_the_absolute_bound():
    # 40 nats above the rest: what the parts drop is 2^-37 of the largest for each token
    m = q3()
    cfg = _cfg(nh=8, nkv=2)
    q = _grouped_q(2, 2, 4, 11)
    lens = [3000, 50]
    for value in (0.0, 1.0):
        kv, ref = _slots(cfg, q, lens, 3000, 40.0, [0, 49], value, 500)
        i32 = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
        o = host(m.attention_q8(cfg, q.cuda(), kv, i32, torch.tensor(lens, dtype=torch.int32).cuda()))
        m.check_device()
        for b, n in enumerate(lens):
            qb = q[b].double().numpy().reshape(-1, HD)
            kc, ks, vc, vs = ref[b]
            want = Q.attention(qb, kc, ks, vc, vs, n, 4)
            mean = Q.attention(qb, kc, ks, np.abs(vc), vs, n, 4)
            total = np.abs(vc[:n] * np.repeat(vs, 128, 0)[:n, :, None]).sum(0).repeat(4, 0)
            off = np.abs(o[b].reshape(-1, HD) - want)
            assert np.all(off <= 2.0 ** -7 * mean + 2.0 ** -8 * np.abs(want) + 2.0 ** -37 * total)
