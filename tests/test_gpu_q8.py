"""The 8-bit operators on the GPU against their fp64 oracle.

Tolerances. An e4m3 rounding is off by at most 2^-4 of the value, or half a subnormal step
(2^-10 of the scale); bf16 by 2^-8. The norm is computed in fp32: the sum over a row and the
few products behind it are good to 1e-5, by which a block's maximum may also land on the other
side of a power of two. A product of K terms summed in fp32 in any order is off by at most
2 K 2^-24 of the sum of the magnitudes (2^-23 a step where the adder truncates). The attention
rounds the probabilities of a block to 2^-8 of each, or 2^-18 of the block's largest, and q to
2^-18 of its largest element, so an output is off by at most 2^-7 of the weighted mean of |v|,
besides its own bf16 rounding. The store is exact.
"""
import math

import numpy as np
import pytest
import torch

from gpu_common import host, layer_on_device, positions, q3, rel_l2
from oracle import q3vl_oracle as O
from oracle import q8_oracle as Q
import q3vl_synth as syn

pytestmark = pytest.mark.gpu
HD = 128


def _cfg(hidden=2560, nh=32, nkv=8, dtype="bf16"):
    return q3().config(hidden, nh, nkv, 9728, dtype)


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _e8(t):
    return np.exp2(t.cpu().view(torch.uint8).numpy().astype(np.float64) - 127)


def _check_blocks(y, q, s, bounds):
    """Rows y (fp64) against elements q and scales s (fp64): each scale the rule's for the
    block's maximum up to 1e-5, each element within its rounding."""
    for i, (lo, hi) in enumerate(zip(bounds, bounds[1:])):
        part = y[:, lo:hi]
        amax = np.max(np.where(np.isfinite(part), np.abs(part), 0), axis=1)
        a = np.array([Q.scale_of(v * (1 - 1e-5)) for v in amax])
        b = np.array([Q.scale_of(v * (1 + 1e-5)) for v in amax])
        assert np.all((s[:, i] == a) | (s[:, i] == b))
        got = q[:, lo:hi] * s[:, i:i + 1]
        fin = np.isfinite(part)
        assert np.array_equal(np.isnan(got), ~fin)
        p = np.where(fin, part, 0)
        bound = np.abs(p) * (2.0 ** -4 + 2e-5) + s[:, i:i + 1] * 2.0 ** -10
        # a scale one step too small (by the 1e-5 above) saturates at 448
        assert np.all(np.abs(np.where(fin, got, 0) - p) <= bound)


@pytest.mark.parametrize("S,H,dtype,delta,gain", [
    (1, 2560, "bf16", True, True), (1, 64, "bf16", False, True), (3, 192, "fp32", True, True),
    (5, 2048, "bf16", True, False), (2, 5120, "fp32", False, True), (700, 2560, "bf16", True, True),
    (33, 64 * 37, "bf16", False, False), (2, 32768, "bf16", True, True),
    (3, 8192 + 64, "fp32", True, True), (17, 10240, "bf16", True, True)])
def test_norm_matches_the_oracle(S, H, dtype, delta, gain):
    m = q3()
    cfg = _cfg(H, dtype=dtype)
    g = _gen(S * 7919 + H)
    dt = m.torch_dtype(cfg)
    x = torch.randn(S, H, generator=g).to(dt)
    d = (0.3 * torch.randn(S, H, generator=g)).to(dt) if delta else None
    gn = (1 + 0.1 * torch.randn(H, generator=g)).to(dt) if gain else None
    dev = lambda t: None if t is None else t.cuda()  # noqa: E731
    h, q, s = m.add_rms_norm_q8(cfg, dev(x), dev(gn), dev(d))
    m.check_device()
    rnd = lambda v: torch.tensor(v).to(torch.float32).to(dt).double().numpy()  # noqa: E731
    np_ = lambda t: None if t is None else t.double().numpy()  # noqa: E731
    hw, _, _ = Q.add_rms_norm(np_(x), np_(d), np_(gn), 1e-6, rnd)
    assert np.array_equal(host(h), hw)
    y = hw if gn is None else hw / np.sqrt(np.mean(hw * hw, 1, keepdims=True) + 1e-6) * np_(gn)
    _check_blocks(y, host(q), _e8(s), Q.edges(H))
    if delta:   # in place: the same bits
        xd = x.cuda()
        h2, q2, s2 = m.add_rms_norm_q8(cfg, xd, dev(gn), dev(d), h=xd)
        assert h2 is xd and torch.equal(h2, h)
        assert torch.equal(q2.view(torch.uint8), q.view(torch.uint8))
        assert torch.equal(s2.view(torch.uint8), s.view(torch.uint8))


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_quantise_rows_at_the_ends_of_the_range(dtype):
    # zeros, infinities and NaN inside a block, the type's largest and smallest magnitudes,
    # exact powers and 448 on the border of two scales
    m = q3()
    cfg = _cfg(256, dtype=dtype)
    dt = m.torch_dtype(cfg)
    big = torch.finfo(dt).max
    x = torch.randn(8, 256, generator=_gen(3))
    x[0] = 0
    x[1, 5], x[1, 200], x[1, 201] = math.inf, -math.inf, math.nan
    x[2] *= 2.0 ** -130
    x[3, 0], x[3, 255] = big, -big
    x[4, :128], x[4, 128:] = 448.0, 449.0 if dtype == "fp32" else 450.0
    x[5, :128] = math.nan
    x[6] *= 2.0 ** 100
    x[7, :128] = torch.tensor([2.0 ** -(i % 24) for i in range(128)])
    x = x.to(dt)
    h, q, s = m.add_rms_norm_q8(cfg, x.cuda(), None)
    m.check_device()
    want_q, want_s = Q.quantize(x.double().numpy(), Q.edges(256))
    assert np.array_equal(_e8(s), want_s)
    assert np.array_equal(host(q), want_q, equal_nan=True)
    assert h.data_ptr() != q.data_ptr()


def _weight(N, K, seed, dtype=torch.bfloat16):
    return (0.02 * torch.randn(N, K, generator=_gen(seed))).to(dtype)


@pytest.mark.parametrize("N,K,dtype", [(1, 64, torch.bfloat16), (130, 192, torch.float32),
                                       (256, 2560, torch.bfloat16)])
def test_weight_form_is_the_oracles(N, K, dtype):
    m = q3()
    w = _weight(N, K, N + K, dtype)
    w[0, 3] = 1.0
    if N > 128:
        w[129] = 0
        w[:, 70] *= 100
    lin = m.quantize_weight_q8(w.cuda())
    wq, ws = Q.quantize_weight(w.double().numpy())
    assert np.array_equal(_e8(lin.scales), ws) and np.array_equal(host(lin.weight), wq)


def _rows8(M, K, seed, amp=None):
    """Random 8-bit rows with uneven block scales: (torch e4m3, E8M0, elements, scales)."""
    x = torch.randn(M, K, generator=_gen(seed)).double()
    x *= torch.exp2(torch.randint(-6, 7, (M, 1), generator=_gen(seed + 1)).double())
    if amp is not None:
        x *= amp
    q, s = Q.quantize(x.numpy(), Q.edges(K))
    return (torch.tensor(q).float().to(torch.float8_e4m3fn),
            torch.tensor(np.log2(s) + 127).to(torch.uint8).view(torch.float8_e8m0fnu), q, s)


def _check_linear(got, want, mag, K, out_dtype):
    bound = 2 * K * 2.0 ** -24 * mag + (2.0 ** -8 if out_dtype == torch.bfloat16 else
                                        2.0 ** -23) * np.abs(want) + 1e-37
    assert np.all(np.isfinite(got))
    assert np.all(np.abs(got - want) <= bound), np.max(np.abs(got - want) / bound)


LINEAR = [(1, 1, 64), (1, 128, 128), (1, 2560, 2560), (2, 129, 192), (15, 1000, 320),
          (16, 127, 2048), (17, 33, 192), (33, 2560, 1216), (64, 640, 4096), (127, 200, 640),
          (128, 256, 256), (129, 257, 320), (200, 384, 1088), (256, 1024, 512), (257, 130, 448),
          (300, 1000, 2560), (513, 2049, 192), (1064, 512, 1024)]


@pytest.mark.parametrize("resid", [False, True], ids=["plain", "resid"])
@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("M,N,K", LINEAR)
def test_linear_matches_the_oracle(M, N, K, out_dtype, resid):
    m = q3()
    xq, xs, x, sx = _rows8(M, K, M + 3 * N + K)
    lin = m.quantize_weight_q8(_weight(N, K, N * K + 1).cuda())
    w, sw = host(lin.weight), _e8(lin.scales)
    r = torch.randn(M, N, generator=_gen(5)).to(out_dtype) if resid else None
    out = torch.full((M, N), math.nan, dtype=out_dtype, device="cuda")
    got = m.linear_q8(xq.cuda(), xs.cuda(), lin, None if r is None else r.cuda(), out_dtype, out)
    m.check_device()
    assert got is out
    rn = None if r is None else r.double().numpy()
    want = Q.linear(x, sx, w, sw, rn)
    mag = Q.linear(np.abs(x), sx, np.abs(w), sw, None if rn is None else np.abs(rn))
    _check_linear(host(got), want, mag, K, out_dtype)
    again = m.linear_q8(xq.cuda(), xs.cuda(), lin, None if r is None else r.cuda(), out_dtype)
    assert torch.equal(again, got)          # the same bits each time
    if resid:                               # the residual updated in place
        rd = r.cuda()
        m.linear_q8(xq.cuda(), xs.cuda(), lin, rd, out_dtype, out=rd)
        assert torch.equal(rd, got)


@pytest.mark.parametrize("M", [3, 140])
def test_linear_keeps_extreme_scales_and_nan_to_their_rows(M):
    m = q3()
    K, N = 384, 300
    amp = torch.ones(M, K, dtype=torch.float64)
    amp[0], amp[1] = 2.0 ** 60, 2.0 ** -60
    amp[2, 128:256] = 2.0 ** 40              # one block far above its neighbours
    xq, xs, x, sx = _rows8(M, K, 11, amp)
    w = _weight(N, K, 12)
    w[130, 7] = math.inf                     # not finite: NaN, in this output column alone
    lin = m.quantize_weight_q8(w.cuda())
    xq = xq.view(torch.uint8)
    xq[M - 1, 300] = 0x7f
    got = host(m.linear_q8(xq.view(torch.float8_e4m3fn).cuda(), xs.cuda(), lin,
                           out_dtype=torch.float32))
    m.check_device()
    bad = np.zeros((M, N), bool)
    bad[M - 1] = bad[:, 130] = True
    assert np.array_equal(np.isnan(got), bad)
    wq, sw = np.nan_to_num(host(lin.weight)), _e8(lin.scales)
    want, mag = Q.linear(x, sx, wq, sw), Q.linear(np.abs(x), sx, np.abs(wq), sw)
    ok = ~bad
    assert np.all(np.abs(got - want)[ok] <= (2 * K * 2.0 ** -24 * mag)[ok])


def _cache(cfg, n_seq, cap, seed, poison=True):
    """An 8-bit cache of random rows, held as the kernel's and as the oracle's; every byte and
    scale random first (NaN among them) where `poison`."""
    m = q3()
    kv = m.KvCacheQ8(cfg, n_seq, cap)
    g = _gen(seed)
    for t in (kv.k, kv.v):
        b = torch.randint(0, 256, t.shape, generator=g, dtype=torch.int16).to(torch.uint8)
        t.view(torch.uint8).copy_(b if poison else b * 0)
    for t in (kv.k_scale, kv.v_scale):
        t.view(torch.uint8).copy_(torch.full(t.shape, 0xFF if poison else 1, dtype=torch.uint8))
    return kv


def _fill(cfg, kv, lens, seed, spread=0.4):
    """Writes lens[b] rows into slot b by the oracle's store; returns its copy of the slots."""
    nkv = cfg.n_kv_heads
    out = []
    for b, n in enumerate(lens):
        slot = []
        for t, sc, k in ((kv.k, kv.k_scale, 0), (kv.v, kv.v_scale, 1)):
            c = np.zeros((kv.cap, nkv, HD))
            s = np.zeros((-(-kv.cap // 128), nkv))
            g = _gen(seed + 10 * b + k)
            rows = torch.randn(n, nkv, HD, generator=g).double()
            rows *= torch.exp(spread * torch.randn(n, nkv, 1, generator=g).double())
            Q.store(c, s, rows.to(torch.bfloat16).double().numpy(), 0)
            t[b, :n] = torch.tensor(c[:n].reshape(n, nkv * HD)).float().to(torch.float8_e4m3fn).cuda()
            nb = -(-n // 128)
            if nb:
                sc[b, :nb] = torch.tensor(np.log2(s[:nb]) + 127).to(torch.uint8).view(
                    torch.float8_e8m0fnu).cuda()
            slot += [c, s]
        out.append(slot)
    return out


STORE = [  # lens, new rows per sequence (None: one each, without starts), cap
    ([0], [1], 1), ([0], [128], 128), ([0], [129], 200), ([127], [2], 200), ([128], [1], 300),
    ([5, 0, 300, 129], [300, 1, 0, 128], 700), ([1, 127, 128, 255, 640], None, 641),
    ([100] * 40, None, 128), ([0, 7, 256], [1000, 505, 77], 1024)]


@pytest.mark.parametrize("grow", [1.0, 300.0], ids=["even", "growing"])
@pytest.mark.parametrize("lens,new,cap", STORE)
def test_store_is_exact(lens, new, cap, grow):
    m = q3()
    cfg = _cfg(nkv=2, nh=8)
    B = len(lens)
    kv = _cache(cfg, B, cap, 1)
    perm = torch.randperm(B, generator=_gen(2))
    by_slot = [0] * B
    for b in range(B):
        by_slot[int(perm[b])] = lens[b]
    ref = _fill(cfg, kv, by_slot, 3)
    before = [t.clone() for t in (kv.k.view(torch.uint8), kv.v.view(torch.uint8),
                                  kv.k_scale.view(torch.uint8), kv.v_scale.view(torch.uint8))]
    counts = [1] * B if new is None else new
    T = sum(counts)
    qkv = (grow * torch.randn(max(T, 1), 4 * 2 * HD, generator=_gen(4))).to(torch.bfloat16)
    qkv[0, 2 * HD:] = 0                       # a row of zeros
    if T > 3:
        qkv[1, 2 * HD + 5], qkv[2, 6 * HD + 9] = math.inf, math.nan
    qd = qkv.cuda()
    k, v = qd[:, 2 * HD:4 * HD], qd[:, 6 * HD:]
    st = None if new is None else torch.tensor(np.cumsum([0] + new), dtype=torch.int32).cuda()
    seq, ln = perm.to(torch.int32).cuda(), torch.tensor(lens, dtype=torch.int32).cuda()
    m.kv_store_q8(cfg, k, v, kv, seq, ln, st)
    m.check_device()
    at = 0
    got = [t.clone() for t in (kv.k.view(torch.uint8), kv.v.view(torch.uint8),
                               kv.k_scale.view(torch.uint8), kv.v_scale.view(torch.uint8))]
    for b in range(B):
        n, L, slot = counts[b], lens[b], int(perm[b])
        rows = qkv[at:at + n].double().numpy()
        at += n
        for i, lo in ((0, 2 * HD), (1, 6 * HD)):
            c, s = ref[slot][2 * i], ref[slot][2 * i + 1]
            Q.store(c, s, rows[:, lo:lo + 2 * HD].reshape(n, 2, HD), L)
            e = L + n
            g8 = host((kv.k, kv.v)[i][slot, :e]).reshape(e, 2, HD)
            assert np.array_equal(g8, c[:e], equal_nan=True), (b, i)
            nb = -(-e // 128)
            assert np.array_equal(_e8((kv.k_scale, kv.v_scale)[i][slot, :nb]), s[:nb]), (b, i)
            # rows and scales behind the last one are left as they were
            assert torch.equal(got[i][slot, e:], before[i][slot, e:])
            assert torch.equal(got[2 + i][slot, nb:], before[2 + i][slot, nb:])


def test_store_skips_what_is_out_of_range_and_reports_it():
    m = q3()
    cfg = _cfg(nkv=2, nh=8)
    kv = _cache(cfg, 3, 150, 5, poison=False)   # lengths below claim rows of scale 2^-126
    was = kv.k.view(torch.uint8).clone()
    rows = torch.ones(4, 2 * HD, dtype=torch.bfloat16, device="cuda")
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    # slots -1 and 3, a length at the capacity, a negative length: none is written
    m.kv_store_q8(cfg, rows, rows, kv, i32(-1, 3, 1, 2), i32(0, 0, 150, -1))
    assert m.device_status()[0] == -2
    assert torch.equal(kv.k.view(torch.uint8), was)
    # one good sequence among bad ones is written
    m.kv_store_q8(cfg, rows[:2], rows[:2], kv, i32(0, 9), i32(149, 0))
    assert m.device_status()[0] == -2
    assert torch.equal(kv.k[0, 149].float(), torch.full((256,), 256.0, device="cuda"))
    # starts past the rows (the sequence is skipped), and starts that fall (nothing is stored)
    was = kv.k.view(torch.uint8).clone()
    m.kv_store_q8(cfg, rows, rows, kv, i32(1), i32(0), i32(2, 5))
    assert m.device_status()[0] == -2
    m.kv_store_q8(cfg, rows, rows, kv, i32(0, 1, 2), i32(0, 0, 0), i32(0, 3, 1, 4))
    assert m.device_status()[0] == -2
    assert torch.equal(kv.k.view(torch.uint8), was)


def _check_attention(cfg, got, q, ref, seq, lens):
    G, nkv = cfg.n_heads // cfg.n_kv_heads, cfg.n_kv_heads
    for b, (slot, n) in enumerate(zip(seq, lens)):
        qb = q[b].double().numpy().reshape(-1, HD)
        kc, ks, vc, vs = ref[slot]
        want = Q.attention(qb, kc, ks, vc, vs, n, G)
        mean = Q.attention(qb, kc, ks, np.abs(vc), vs, n, G)
        g = got[b].reshape(-1, HD)
        if n == 0:
            assert not g.any()
            continue
        assert np.all(np.isfinite(g)), b
        off = np.abs(g - want) / (2.0 ** -7 * mean + 2.0 ** -8 * np.abs(want) + 1e-30)
        assert off.max() <= 1, (b, n, off.max())


ATTEND = [  # heads, kv heads, lens
    (8, 8, [1, 127, 128, 129]), (4, 2, [0, 1, 300, 4000, 255]), (8, 2, [1000]),
    (32, 8, [4096, 5]), (16, 2, [2050, 0, 513]), (2, 2, [20000, 3]), (8, 2, [7 * i for i in range(100)])]


@pytest.mark.parametrize("nh,nkv,lens", ATTEND,
                         ids=[f"h{a}-{b}-{len(c)}x{max(c)}" for a, b, c in ATTEND])
def test_attention_matches_the_oracle(nh, nkv, lens):
    m = q3()
    cfg = _cfg(nh=nh, nkv=nkv)
    B = len(lens)
    kv = _cache(cfg, B, max(lens) + 3, 6)
    perm = torch.randperm(B, generator=_gen(7))
    by_slot = [0] * B
    for b in range(B):
        by_slot[int(perm[b])] = lens[b]
    ref = _fill(cfg, kv, by_slot, 8)
    q = torch.randn(B, nh * HD, generator=_gen(9)).to(torch.bfloat16)
    ws = m.attention_q8_workspace(cfg, B, kv.cap)
    outs = []
    for fill in (0, 0xFF):
        ws.fill_(fill)
        o = torch.full((B, nh * HD), math.nan, dtype=torch.bfloat16, device="cuda")
        m.attention_q8(cfg, q.cuda(), kv, perm.to(torch.int32).cuda(),
                       torch.tensor(lens, dtype=torch.int32).cuda(), o, ws)
        m.check_device()
        outs.append(o)
    assert torch.equal(outs[0], outs[1])
    _check_attention(cfg, host(outs[0]), q, ref, perm.tolist(), lens)


def test_attention_on_sharp_and_uneven_scores():
    # a sink token far above the rest, blocks of very different scales, large and tiny q
    m = q3()
    cfg = _cfg(nh=16, nkv=2)
    L = 1500
    kv = _cache(cfg, 4, L, 20)
    nkv = cfg.n_kv_heads
    ref = []
    q = torch.randn(4, 16 * HD, generator=_gen(21)).to(torch.bfloat16)
    q[1] *= 30
    q[2] *= 2.0 ** -20
    q[3, 5] = 3e4                              # one element far above its head's others
    for b in range(4):
        slot = []
        for i, (t, sc) in enumerate(((kv.k, kv.k_scale), (kv.v, kv.v_scale))):
            rows = torch.randn(L, nkv, HD, generator=_gen(22 + 2 * b + i))
            if i == 0:
                rows[3] = 4 * q[b].float().view(nkv, 8, HD)[:, 0] / (q[b].float().abs().max() + 1e-30)
            blk = torch.arange(L) // 128
            rows *= torch.exp2((blk % 5).float() * (-3 if i else -1))[:, None, None]
            c, s = np.zeros((L, nkv, HD)), np.zeros((-(-L // 128), nkv))
            Q.store(c, s, rows.to(torch.bfloat16).double().numpy(), 0)
            t[b] = torch.tensor(c.reshape(L, -1)).float().to(torch.float8_e4m3fn).cuda()
            sc[b] = torch.tensor(np.log2(s) + 127).to(torch.uint8).view(torch.float8_e8m0fnu).cuda()
            slot += [c, s]
        ref.append(slot)
    idx = torch.arange(4, dtype=torch.int32).cuda()
    lens = [L, 1400, 129, 700]
    o = m.attention_q8(cfg, q.cuda(), kv, idx, torch.tensor(lens, dtype=torch.int32).cuda())
    m.check_device()
    _check_attention(cfg, host(o), q, ref, range(4), lens)


def test_attention_rows_may_share_a_slot_and_bad_rows_are_zero():
    m = q3()
    cfg = _cfg(nh=8, nkv=2)
    kv = _cache(cfg, 2, 400, 30)
    ref = _fill(cfg, kv, [400, 10], 31)
    q = torch.randn(6, 8 * HD, generator=_gen(32)).to(torch.bfloat16)
    seq, lens = [0, 0, 1, 2, -1, 0], [400, 33, 10, 5, 5, 401]
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    o = m.attention_q8(cfg, q.cuda(), kv, i32(seq), i32(lens))
    assert m.device_status()[0] == -2
    got = host(o)
    assert not got[3:].any()
    _check_attention(cfg, got[:3], q[:3], ref, seq[:3], lens[:3])
    # a NaN in a row that is attended reaches the output of its head alone
    kv.v.view(torch.uint8)[1, 4, 7] = 0x7f
    o = host(m.attention_q8(cfg, q[:3].cuda(), kv, i32(seq[:3]), i32(lens[:3])))
    nan = np.isnan(o).reshape(3, 8, HD)
    assert nan[2, :4, 7].all() and nan.sum() == 4
    m.check_device()


def test_lm_head_with_an_8bit_weight():
    m = q3()
    w = syn.Q4B_LAYER
    cfg = m.config_of(w)
    vocab, B = 5000, 5
    g = _gen(40)
    table = (0.02 * torch.randn(vocab, w.hidden, generator=g)).to(torch.bfloat16)
    x = torch.randn(B, w.hidden, generator=g).to(torch.bfloat16)
    gain = (1 + 0.1 * torch.randn(w.hidden, generator=g)).to(torch.bfloat16)
    lin = m.quantize_weight_q8(table.cuda())
    got = m.lm_head(cfg, x.cuda(), gain.cuda(), lin)
    # the same steps, one by one
    _, q, s = m.add_rms_norm_q8(cfg, x.cuda(), gain.cuda())
    assert torch.equal(got, m.linear_q8(q, s, lin, out_dtype=torch.float32))
    m.check_device()
    # against the unquantised head: two e4m3 roundings of relative deviation
    # about 2^-4 / sqrt(3) each, independent over the sum
    want = O.lm_head(O.Config.of(w), x, gain, table)
    assert rel_l2(got.cpu().numpy(), want) <= 2 * 2.0 ** -4 / math.sqrt(3)


def test_ffn_of_8bit_products_on_a_side_stream():
    # a run of the operators as a layer's second half would use them, on a stream of its own:
    # norm -> gate/up product -> silu(g) u quantised -> down product onto the residual
    m = q3()
    cfg = _cfg(512)
    S, H, I = 77, 512, 768
    g = _gen(50)
    x = torch.randn(S, H, generator=g).to(torch.bfloat16).cuda()
    d = torch.randn(S, H, generator=g).to(torch.bfloat16).cuda()
    gain = (1 + 0.1 * torch.randn(H, generator=g)).to(torch.bfloat16).cuda()
    wgu = m.quantize_weight_q8(_weight(2 * I, H, 51).cuda())
    wd = m.quantize_weight_q8(_weight(H, I, 52).cuda())
    act_cfg = _cfg(I)

    def run(stream=None):
        h, q, s = m.add_rms_norm_q8(cfg, x, gain, d, stream=stream)
        gu = m.linear_q8(q, s, wgu, stream=stream)
        with torch.cuda.stream(stream or torch.cuda.current_stream()):
            act = (torch.nn.functional.silu(gu[:, :I].float()) * gu[:, I:].float()).bfloat16()
        _, aq, as_ = m.add_rms_norm_q8(act_cfg, act, None, stream=stream)
        return m.linear_q8(aq, as_, wd, h, stream=stream), (h, q, s, gu, aq, as_)
    want, _ = run()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got, (h, q, s, gu, aq, as_) = run(side)
    side.synchronize()
    m.check_device()
    assert torch.equal(got, want)
    y = Q.linear(host(aq), _e8(as_), host(wd.weight), _e8(wd.scales), host(h))
    mag = Q.linear(np.abs(host(aq)), _e8(as_), np.abs(host(wd.weight)), _e8(wd.scales), np.abs(host(h)))
    _check_linear(host(got), y, mag, I, torch.bfloat16)


# ---------------------------------------------------------------------------
# The decoder's own paths over 8-bit caches
# ---------------------------------------------------------------------------
def _text_pos(start, n):
    p = torch.arange(start, start + n, dtype=torch.int32)
    return torch.stack([p, p, p]).cuda().contiguous()


def _deq(kv, b, n, nkv):
    out = []
    for t, s in ((kv.k, kv.k_scale), (kv.v, kv.v_scale)):
        f = np.repeat(_e8(s[b]), 128, 0)[:n, :, None]
        out.append(host(t[b, :n]).reshape(n, nkv, HD) * f)
    return out


def test_prefill_writes_the_rows_that_the_bf16_cache_gets():
    m = q3()
    w = syn.Q4B_LAYER.with_seq(700, images=((100, 8, 12),))
    cfg = m.config_of(w)
    _, packed = layer_on_device(w)
    pos, _, _, _ = positions(w)
    x0 = syn.hidden_input(w).cuda()
    kv, kv8 = m.kv_caches(cfg, 1, 3, 705)[0], m.kv_caches(cfg, 1, 3, 705, dtype="fp8")[0]
    x1, x2 = x0.clone(), x0.clone()
    m.layer_prefill_kv(cfg, packed, x1, pos, kv, seq=1)
    m.layer_prefill_kv(cfg, packed, x2, pos, kv8, seq=1)
    m.check_device()
    assert torch.equal(x1, x2)
    nkv = w.n_kv_heads
    for src, t, s in ((kv.k, kv8.k, kv8.k_scale), (kv.v, kv8.v, kv8.v_scale)):
        c, sc = np.zeros((705, nkv, HD)), np.zeros((6, nkv))
        Q.store(c, sc, host(src[1, :700]).reshape(700, nkv, HD), 0)
        assert np.array_equal(host(t[1]).reshape(705, nkv, HD), c)
        assert np.array_equal(_e8(s[1]), sc)
        assert not t[0].view(torch.uint8).any() and not t[2].view(torch.uint8).any()


@pytest.mark.parametrize("w,lens", [
    (syn.Q2B_LAYER, [0, 1, 127, 128, 300]), (syn.Q4B_LAYER, [5, 256, 1000]),
    (syn.Q2B_LAYER, [3 * b + 1 for b in range(40)])], ids=["2b", "4b", "2b-b40"])
def test_layer_decode_over_the_8bit_cache(w, lens):
    m = q3()
    cfg = m.config_of(w)
    raw, packed = layer_on_device(w)
    B, nkv, G = len(lens), w.n_kv_heads, w.n_heads // w.n_kv_heads
    kv = m.kv_caches(cfg, 1, B, max(lens) + 1, dtype="fp8")[0]
    g = _gen(60)
    xs = []
    for b, L in enumerate(lens):
        x = torch.randn(L + 1, cfg.hidden, generator=g).to(torch.bfloat16)
        xs.append(x)
        if L:
            m.layer_prefill_kv(cfg, packed, x[:L].cuda().clone(), _text_pos(0, L), kv, seq=b)
    xn = torch.cat([x[-1:] for x in xs])
    pos = torch.tensor(lens, dtype=torch.int32).repeat(3, 1).cuda()
    seq = torch.arange(B, dtype=torch.int32).cuda()
    ln = torch.tensor(lens, dtype=torch.int32).cuda()
    outs = []
    keep = [t.clone() for t in (kv.k, kv.v, kv.k_scale, kv.v_scale)]
    for fill in (0, 0xFF):
        for t, old in zip((kv.k, kv.v, kv.k_scale, kv.v_scale), keep):
            t.copy_(old)
        ws = m.decode_workspace(cfg, B, kv.cap, dtype="fp8").fill_(fill)
        xd = xn.cuda().clone()
        m.layer_decode(cfg, packed, xd, pos, kv, seq, ln, ws)
        m.check_device()
        outs.append(xd)
    assert torch.equal(outs[0], outs[1])
    # teacher-forced: the oracle attends to the rows as the cache holds them
    oc = O.Config.of(w)
    ang = O.mrope_angles(pos.cpu().numpy().astype(np.int64), w.rope_theta)
    x64 = xn.double().numpy()
    q, k, v = O.qkv(oc, raw, x64, ang)
    got = host(outs[0])
    for b, L in enumerate(lens):
        kd, vd = _deq(kv, b, L + 1, nkv)
        for d, ref in ((kd, k), (vd, v)):     # the new row, within its rounding (bf16, then e4m3)
            r = np.asarray(ref).reshape(B, nkv, HD)[b]
            lim = 2.0 ** -4 * np.abs(r) + 0.02 * np.abs(r).max() + 2.0 ** -9 * np.abs(d).max()
            assert np.all(np.abs(d[L] - r) <= lim)
        one = np.ones((-(-(L + 1) // 128), nkv))
        o = Q.attention(np.asarray(q).reshape(B, -1, HD)[b], kd, one, vd, one, L + 1, G)
        h = O.o_residual(raw, o.reshape(1, -1), x64[b:b + 1])
        want = O.down_residual(raw, O.ffn_act(oc, raw, h), h)[0]
        assert rel_l2(got[b], want) <= 1e-2, b
        assert rel_l2(got[b] - x64[b], want - x64[b]) <= 2e-2, b


def test_stack_decode_steps_captured_in_a_graph_match_eager_steps():
    # two layers, three steps over a block border, then the head: eager, and one captured step
    # replayed; 8-bit weights for the head
    m = q3()
    w = syn.Q2B_LAYER
    cfg = m.config_of(w)
    layers = [layer_on_device(w, l)[1] for l in range(2)]
    lens = [126, 40, 255]
    B = len(lens)
    gain = torch.ones(w.hidden, dtype=torch.bfloat16, device="cuda")
    lin = m.quantize_weight_q8(_weight(1000, w.hidden, 70).cuda())
    xin = torch.randn(3, B, w.hidden, generator=_gen(71)).to(torch.bfloat16).cuda()

    def setup():
        kvs = m.kv_caches(cfg, 2, B, 260, dtype="fp8")
        for b, L in enumerate(lens):
            x = torch.randn(L, w.hidden, generator=_gen(72 + b)).to(torch.bfloat16).cuda()
            m.stack_prefill_kv(cfg, layers, x, _text_pos(0, L), kvs, seq=b)
        ln = torch.tensor(lens, dtype=torch.int32).cuda()
        return kvs, ln, ln.repeat(3, 1).contiguous(), torch.arange(B, dtype=torch.int32).cuda()

    kvs, ln, pos, seq = setup()
    want = []
    for i in range(3):
        x = xin[i].clone()
        m.stack_decode(cfg, layers, x, pos, kvs, seq, ln)
        want.append(m.lm_head(cfg, x, gain, lin))
        m.decode_advance(pos, ln)
    m.check_device()

    kvs, ln, pos, seq = setup()
    x = xin[0].clone()
    ws = m.decode_workspace(cfg, B, 260, dtype="fp8")
    logits = torch.empty(B, 1000, device="cuda")
    keep = [t.clone() for kv in kvs for t in (kv.k, kv.v, kv.k_scale, kv.v_scale)]

    def step():
        m.stack_decode(cfg, layers, x, pos, kvs, seq, ln, ws=ws)
        m.lm_head(cfg, x, gain, lin, logits=logits)
        m.decode_advance(pos, ln)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()                                    # warm-up
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    # back to the start
    ln.copy_(torch.tensor(lens, dtype=torch.int32))
    pos.copy_(ln.repeat(3, 1))
    for t, old in zip((t for kv in kvs for t in (kv.k, kv.v, kv.k_scale, kv.v_scale)), keep):
        t.copy_(old)
    for i in range(3):
        x.copy_(xin[i])
        graph.replay()
        assert torch.equal(logits, want[i]), i
    m.check_device()
