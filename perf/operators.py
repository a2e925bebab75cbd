"""Cases of the 8-bit serving operators: what each one computes in plain torch, and the calls.

Four operators of one path. A residual add with a root-mean-square norm whose output is
e4m3 with a scale for each 128 columns of a row ("norm"); the product of such rows with an
e4m3 weight that has a scale for each 128 x 128 block ("linear"); writing key and value rows
into a cache of e4m3 with a scale for each 128 tokens and head ("store"); the attention of
one query row per sequence over that cache ("attend"). Scales are powers of two held as
E8M0 bytes: byte u stands for 2^(u - 127).

The scale of a block is the smallest power of two, at least 2^-126, that brings the block's
largest finite magnitude to 448 or less; elements are divided by it and rounded to nearest
even. An element that is not finite is stored as NaN and takes no part in the maximum.

Shapes are those of the decoder's workloads: hidden 2048 / 2560 / 5120, heads 16 / 32 / 64
over 8 KV heads of 128, intermediate 6144 / 9728 / 25600, vocabulary 151936.
"""
import math
import random

import torch

own = False

BLK = 128          # columns, or tokens, that share a scale
HD = 128           # head dimension
EPS = 1e-6


# ---------------------------------------------------------------------------
# The cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # one decoded token before a projection: the shortest call
        dict(name="norm-token", op="norm", rows=1, hidden=2560, dtype="bf16", delta=True),
        # the 4096-row prompt of the 4B shape
        dict(name="norm-prompt", op="norm", rows=4096, hidden=2560, dtype="bf16", delta=True),
        # the 32B-shape prompt encoder's 1064 rows, doubled and odd, in the fp32 configuration
        dict(name="norm-encoder-fp32", op="norm", rows=2129, hidden=5120, dtype="fp32",
             delta=False),
        # one decoded token through the 4B QKV projection: weight streaming
        dict(name="linear-token", op="linear", rows=1, k=2560, n=6144, out="bf16", resid=False),
        # a decode batch of odd size through the 4B down projection, with the residual
        dict(name="linear-batch", op="linear", rows=33, k=9728, n=2560, out="bf16", resid=True),
        # the 4096-row prompt through the 4B gate/up projection: tensor-core bound
        dict(name="linear-prompt", op="linear", rows=4096, k=2560, n=19456, out="bf16",
             resid=False),
        # the LM head of four sequences: the largest weight, fp32 logits
        dict(name="linear-head", op="linear", rows=4, k=2560, n=151936, out="fp32", resid=False),
        # one decode step of 32 sequences: each appends a row to a block that is part full
        dict(name="store-step", op="store", batch=32, rows_each=0, cap=4608, kv_heads=8, pick=1),
        # prompts of uneven length packed in one call, appended behind earlier rows
        dict(name="store-prompts", op="store", batch=5, rows_each=4001, cap=8192, kv_heads=8,
             pick=2),
        # one sequence at the 4096-token context of the decode workload
        dict(name="attend-one", op="attend", batch=1, heads=32, kv_heads=8, longest=4096,
             shortest=4096, pick=3),
        # a decode batch of uneven contexts
        dict(name="attend-batch", op="attend", batch=32, heads=32, kv_heads=8, longest=8191,
             shortest=1, pick=4),
        # two sequences at the longest context that a cache slot holds, 2B shape
        dict(name="attend-long", op="attend", batch=2, heads=16, kv_heads=8, longest=131072,
             shortest=100003, pick=5),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "linear", "store", "attend"])
    if op == "norm":
        hidden = rng.choice([64 * rng.randint(2, 80), 2048, 2560, 5120])
        return dict(op=op, rows=_log(rng, 1, 8192), hidden=hidden,
                    dtype=rng.choice(["bf16", "bf16", "fp32"]), delta=rng.random() < 0.6)
    if op == "linear":
        k = rng.choice([64 * rng.randint(2, 152), 2048, 2560, 5120, 6144, 9728])
        n = rng.choice([_log(rng, 32, 19456), 2048, 2560, 6144, 12288])
        rows = _log(rng, 1, max(1, min(4096, int(4096 * 2560 * 19456 / (k * n)))))
        return dict(op=op, rows=rows, k=k, n=n, out=rng.choice(["bf16", "bf16", "fp32"]),
                    resid=rng.random() < 0.4)
    if op == "store":
        batch = _log(rng, 1, 64)
        step = rng.random() < 0.5
        return dict(op=op, batch=batch, rows_each=0 if step else _log(rng, 1, 16384 // batch),
                    cap=16384 // batch + rng.randint(200, 900), kv_heads=rng.choice([2, 8]),
                    pick=rng.randint(0, 10 ** 6))
    batch = _log(rng, 1, 64)
    longest = _log(rng, 1, min(131072, 262144 // batch))
    kv_heads = rng.choice([2, 8])
    return dict(op=op, batch=batch, heads=kv_heads * rng.choice([1, 2, 4, 8]), kv_heads=kv_heads,
                longest=longest, shortest=rng.randint(0, longest), pick=rng.randint(0, 10 ** 6))


def _store_plan(case):
    """(rows already cached, new rows) of each sequence: part of the case, not of its seed."""
    r = random.Random(case["pick"])
    each, cap = case["rows_each"], case["cap"]
    new = [1 if each == 0 else max(1, each - r.randint(0, each // 2)) for _ in range(case["batch"])]
    return [r.randint(0, cap - n) for n in new], new


def _attend_lens(case):
    r = random.Random(case["pick"])
    lens = [r.randint(case["shortest"], case["longest"]) for _ in range(case["batch"])]
    lens[0] = case["longest"]
    return lens


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------
def _exponent(amax):
    """E8M0 byte of the scale for a block maximum (float32, >= 0)."""
    m, e = torch.frexp(amax)
    s = e.to(torch.int32) - torch.where(m <= 0.875, 9, 8).to(torch.int32) + 127
    return torch.where(amax > 0, s.clamp(1, 254), 1).to(torch.uint8)


def _two_to(u):
    """2^(u - 127) in float32 of E8M0 bytes u in [1, 254]."""
    return (u.to(torch.int32) << 23).view(torch.float32)


def _inverse(u):
    """2^(127 - u) in float32 of E8M0 bytes u in [1, 253]; 2^-127 is not needed."""
    return ((254 - u.to(torch.int32)) << 23).view(torch.float32)


def _finite_amax(x, dim):
    return torch.where(torch.isfinite(x), x.abs(), torch.zeros((), device=x.device)).amax(dim)


def _to_e4m3(x):
    return torch.where(torch.isfinite(x), x, torch.full((), math.nan, device=x.device)).to(
        torch.float8_e4m3fn)


def _quantize_rows(x):
    """float32 [R, C] -> e4m3 [R, C], E8M0 [R, ceil(C / 128)]."""
    R, C = x.shape
    nb = -(-C // BLK)
    p = torch.nn.functional.pad(x, (0, nb * BLK - C)).view(R, nb, BLK)
    u = _exponent(_finite_amax(p, 2))
    q = _to_e4m3(p * _inverse(u)[:, :, None]).view(R, nb * BLK)[:, :C].contiguous()
    return q, u.view(torch.float8_e8m0fnu)


def _quantize_blocks(w):
    """float32 [N, K] -> e4m3 [N, K], E8M0 [ceil(N / 128), ceil(K / 128)]."""
    N, K = w.shape
    nb, kb = -(-N // BLK), -(-K // BLK)
    p = torch.nn.functional.pad(w, (0, kb * BLK - K, 0, nb * BLK - N)).view(nb, BLK, kb, BLK)
    u = _exponent(p.abs().amax((1, 3)))
    q = (p * _inverse(u)[:, None, :, None]).to(torch.float8_e4m3fn).view(nb * BLK, kb * BLK)
    return q[:N, :K].contiguous(), u.view(torch.float8_e8m0fnu)


def _quantize_cache(x):
    """bf16 [n_seq, cap, heads, 128] -> e4m3 [n_seq, cap, heads * 128], E8M0 [n_seq, blocks, heads]."""
    n, cap, h, _ = x.shape
    nb = -(-cap // BLK)
    q = torch.empty(n, cap, h * HD, dtype=torch.float8_e4m3fn, device=x.device)
    u = torch.empty(n, nb, h, dtype=torch.uint8, device=x.device)
    for s in range(n):  # a slot at a time keeps the temporaries small
        p = torch.nn.functional.pad(x[s].float(), (0, 0, 0, 0, 0, nb * BLK - cap))
        p = p.view(nb, BLK, h, HD)
        u[s] = _exponent(p.abs().amax((1, 3)))
        q[s] = (p * _inverse(u[s])[:, None, :, None]).to(torch.float8_e4m3fn).view(
            nb * BLK, h * HD)[:cap]
    return q, u.view(torch.float8_e8m0fnu)


def _kv_like(shape, g, spread):
    """Key or value rows: N(0, 1), each head's magnitude drifting slowly along the sequence."""
    x = torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16)
    amp = torch.exp(spread * torch.randn(shape[:-2] + (shape[-2], 1), generator=g, device="cuda",
                                         dtype=torch.float32)).to(torch.bfloat16)
    return x * amp


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, std=1.0, mean=0.0, dtype=torch.float32):
        return torch.randn(*shape, generator=g, device="cuda").mul_(std).add_(mean).to(dtype)

    op = case["op"]
    s = {"case": case}
    if op == "norm":
        dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
        s["x"] = normal(case["rows"], case["hidden"], dtype=dt)
        s["delta"] = normal(case["rows"], case["hidden"], std=0.3, dtype=dt) if case["delta"] else None
        s["gain"] = normal(case["hidden"], std=0.1, mean=1.0, dtype=dt)
    elif op == "linear":
        s["xq"], s["xs"] = _quantize_rows(normal(case["rows"], case["k"]))
        s["wq"], s["ws"] = _quantize_blocks(normal(case["n"], case["k"], std=0.02))
        dt = torch.bfloat16 if case["out"] == "bf16" else torch.float32
        s["resid"] = normal(case["rows"], case["n"], dtype=dt) if case["resid"] else None
        s["out_dtype"] = dt
    elif op == "store":
        lens, new = _store_plan(case)
        B, h = case["batch"], case["kv_heads"]
        T = sum(new)
        starts = [sum(new[:b]) for b in range(B + 1)]
        s["starts"] = torch.tensor(starts, dtype=torch.int32, device="cuda")
        s["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
        s["seq"] = torch.randperm(B, generator=g, device="cuda").to(torch.int32)
        # as column ranges of one QKV buffer, heads = 4 kv_heads
        qkv = normal(T, 6 * h * HD, dtype=torch.bfloat16)
        s["k"], s["v"] = qkv[:, 4 * h * HD:5 * h * HD], qkv[:, 5 * h * HD:]
        s["k"] *= torch.exp(0.7 * normal(T, 1)).to(torch.bfloat16)  # some rows outgrow the block
        for name in ("ck", "cv"):
            s[name], s[name + "s"] = _quantize_cache(
                normal(B, case["cap"], h, HD, dtype=torch.bfloat16))
        s["step"] = case["rows_each"] == 0
    else:
        lens = _attend_lens(case)
        B, h = case["batch"], case["kv_heads"]
        cap = max(1, case["longest"])
        s["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
        s["seq"] = torch.randperm(B, generator=g, device="cuda").to(torch.int32)
        s["q"] = normal(B, case["heads"] * HD, dtype=torch.bfloat16)
        for name in ("ck", "cv"):
            s[name], s[name + "s"] = _quantize_cache(_kv_like((B, cap, h, HD), g, 0.3))
    if own:
        import qwen3_vl_decoder_b200 as q3
        s["q3"] = q3
        heads = case.get("heads", 4 * case.get("kv_heads", 8))
        s["cfg"] = q3.config(hidden=case.get("hidden", 2560), n_heads=heads,
                             n_kv_heads=case.get("kv_heads", 8), intermediate=9728,
                             dtype=case.get("dtype", "bf16"), rms_eps=EPS)
        if op == "linear":
            s["lin"] = q3.LinearQ8(s["wq"], s["ws"])
        if op in ("store", "attend"):
            s["kv"] = q3.KvCacheQ8.of(s["cfg"], s["ck"], s["cv"], s["cks"], s["cvs"])
        if op == "attend":
            s["work"] = q3.attention_q8_workspace(s["cfg"], case["batch"], s["kv"].cap)
    return s


# ---------------------------------------------------------------------------
# The plain forms and the calls
# ---------------------------------------------------------------------------
def _plain_norm(s):
    x = s["x"]
    if s["delta"] is not None:
        x = (x.float() + s["delta"].float()).to(x.dtype)
    h = x.float()
    inv = 1.0 / torch.sqrt((h * h).mean(1, keepdim=True) + EPS)
    q, u = _quantize_rows(h * inv * s["gain"].float())
    return x, q, u


def _plain_linear(s):
    def spread(u, rows, cols):  # the scale of every element
        f = _two_to(u.view(torch.uint8))
        f = f.repeat_interleave(BLK, 1)[:, :cols]
        return f if rows is None else f.repeat_interleave(BLK, 0)[:rows]

    K = s["xq"].shape[1]
    a = s["xq"].float() * spread(s["xs"], None, K)
    w = s["wq"].float() * spread(s["ws"], s["wq"].shape[0], K)
    y = a @ w.t()
    if s["resid"] is not None:
        y = y + s["resid"].float()
    return y.to(s["out_dtype"])


def _plain_store(s):
    lens, starts, seq = (s[n].long() for n in ("lens", "starts", "seq"))
    T = s["k"].shape[0]
    row = torch.arange(T, device="cuda")
    b = torch.searchsorted(starts, row, right=True) - 1      # sequence of each new row
    at = lens[b] + row - starts[b]                           # its place in the slot
    slot = seq[b]
    out = []
    for src, name in ((s["k"], "ck"), (s["v"], "cv")):
        cache, scale = s[name], s[name + "s"].view(torch.uint8)
        n, cap, width = cache.shape
        nb, h = scale.shape[1], scale.shape[2]
        x = src.float().view(T, h, HD)
        # largest new magnitude of each (slot, block, head), and where new rows go
        blk = slot * nb + at // BLK
        amax = torch.zeros(n * nb, h, device="cuda").index_reduce_(
            0, blk, _finite_amax(x, 2), "amax").view(n, nb, h)
        touched = torch.zeros(n * nb, device="cuda").index_fill_(0, blk, 1.0).view(n, nb, 1) > 0
        first = torch.arange(nb, device="cuda") * BLK
        cached = torch.zeros(n, dtype=torch.long, device="cuda").index_copy_(0, seq, lens)
        keeps = (first[None, :] < cached[:, None])[:, :, None]     # the block holds earlier rows
        need = _exponent(amax)
        new = torch.where(touched, torch.where(keeps, torch.maximum(need, scale), need), scale)
        # earlier rows of the blocks whose scale grew are rounded again to it
        pos = torch.arange(nb * BLK, device="cuda")
        ratio = _two_to(scale) * _inverse(new)
        ratio = torch.where(touched & keeps, ratio, torch.ones((), device="cuda"))
        per_row = ratio.repeat_interleave(BLK, 1)[:, :cap, :, None]
        old = cache.view(n, cap, h, HD).float()
        earlier = (pos[None, :cap] < cached[:, None])[:, :, None, None]
        old = torch.where(earlier, old * per_row, old).to(torch.float8_e4m3fn).view(n * cap, width)
        rows = _to_e4m3(x * _inverse(new.view(n * nb, h)[blk])[:, :, None]).view(T, width)
        raw = old.view(torch.uint8)
        raw[slot * cap + at] = rows.view(torch.uint8)
        cache.view(torch.uint8).view(n * cap, width).copy_(raw)
        scale.copy_(new)
        out += [cache, s[name + "s"]]
    return out


def _plain_attend(s):
    q, lens, seq = s["q"].float(), s["lens"].long(), s["seq"].long()
    B, cap = q.shape[0], s["ck"].shape[1]
    h = s["cks"].shape[2]
    G = q.shape[1] // HD // h

    def rows(name):
        x = s[name].view(-1, cap, h, HD)[seq].float()
        return x.mul_(_two_to(s[name + "s"].view(torch.uint8)[seq]).repeat_interleave(BLK, 1)[
            :, :cap, :, None])

    k = rows("ck").permute(0, 2, 3, 1)                                 # [B, h, 128, cap]
    sc = (q.view(B, h, G, HD) @ k) / math.sqrt(HD)                      # [B, h, G, cap]
    del k
    sees = torch.arange(cap, device="cuda")[None, :] < lens[:, None]
    sc = sc.masked_fill(~sees[:, None, None, :], -math.inf)
    top = sc.amax(3, keepdim=True)
    p = torch.exp(sc - torch.where(top == -math.inf, torch.zeros_like(top), top))
    den = p.sum(3, keepdim=True)
    v = rows("cv").permute(0, 2, 1, 3)                                 # [B, h, cap, 128]
    v = v.masked_fill(~sees[:, None, :, None], 0.0)
    o = (p @ v) / torch.where(den == 0, torch.ones_like(den), den)     # nothing seen: zeros
    return o.reshape(B, -1).to(torch.bfloat16)


def run(state):
    s = state
    op = s["case"]["op"]
    if not own:
        return {"norm": _plain_norm, "linear": _plain_linear, "store": _plain_store,
                "attend": _plain_attend}[op](s)
    q3 = s["q3"]
    if op == "norm":
        return q3.add_rms_norm_q8(s["cfg"], s["x"], s["gain"], s["delta"])
    if op == "linear":
        return q3.linear_q8(s["xq"], s["xs"], s["lin"], s["resid"], out_dtype=s["out_dtype"])
    if op == "store":
        q3.kv_store_q8(s["cfg"], s["k"], s["v"], s["kv"], s["seq"], s["lens"],
                       None if s["step"] else s["starts"])
        return [s["ck"], s["cks"], s["cv"], s["cvs"]]
    return q3.attention_q8(s["cfg"], s["q"], s["kv"], s["seq"], s["lens"], ws=s["work"])


def work(case):
    op = case["op"]
    if op == "norm":
        e = 2 if case["dtype"] == "bf16" else 4
        n, C = case["rows"] * case["hidden"], case["hidden"]
        # x read; with a delta, delta read and the sum written; e4m3 and scales written
        return {"bytes": n * (e * (3 if case["delta"] else 1) + 1) + C * e + n / BLK,
                "flops": 6 * n}
    if op == "linear":
        m, k, n = case["rows"], case["k"], case["n"]
        e = 2 if case["out"] == "bf16" else 4
        return {"bytes": m * k + n * k + m * k / BLK + n * k / BLK / BLK +
                m * n * e * (2 if case["resid"] else 1), "flops": 2 * m * n * k}
    if op == "store":
        _, new = _store_plan(case)
        rows = 2 * sum(new) * case["kv_heads"]
        return {"bytes": rows * HD * 3 + rows / BLK, "flops": 3 * rows * HD}
    tokens = sum(_attend_lens(case))
    width = case["kv_heads"] * HD
    return {"bytes": 2 * tokens * width * (1 + 1 / BLK / HD) +
            case["batch"] * case["heads"] * HD * 4,
            "flops": 4 * tokens * case["heads"] * HD}


# ---------------------------------------------------------------------------
# The definitions, in 64 bits
# ---------------------------------------------------------------------------
def _e4m3_64(v):
    """v (float64) rounded to the nearest e4m3 value, ties to the even one."""
    mag = v.abs().clamp(min=2.0 ** -30)
    step = torch.exp2(torch.floor(torch.log2(mag)).clamp(min=-6) - 3)
    step = torch.where(mag >= 16 * step, 2 * step, torch.where(mag < 8 * step, step / 2, step))
    step = step.clamp(min=2.0 ** -9)
    return torch.round(v / step) * step


def _scale_64(amax):
    """Smallest 2^s, s >= -126, with amax <= 448 2^s (float64)."""
    s = torch.ceil(torch.log2(amax.clamp(min=1e-300) / 448))
    s = torch.where(amax <= 448 * torch.exp2(s - 1), s - 1, s)
    s = torch.where(amax > 448 * torch.exp2(s), s + 1, s)
    return torch.exp2(torch.where(amax > 0, s.clamp(min=-126), -126.0 * torch.ones_like(s)))


def exact(case, seed):
    global own
    kept, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = kept
    d = torch.float64
    op = case["op"]
    if op == "norm":
        h = s["x"].to(d)
        if s["delta"] is not None:   # the residual stream is kept in the input's type
            h = (h + s["delta"].to(d)).to(s["x"].dtype).to(d)
        y = h / torch.sqrt(h.square().sum(1, keepdim=True) / h.shape[1] + EPS) * s["gain"].to(d)
        qs, us = [], []
        for part in y.split(BLK, 1):
            f = _scale_64(part.abs().max(1, keepdim=True).values)
            qs.append(_e4m3_64(part / f))
            us.append(f)
        return h, torch.cat(qs, 1), torch.cat(us, 1)
    if op == "linear":
        K, N = case["k"], case["n"]
        y = s["resid"].to(d) if s["resid"] is not None else torch.zeros(
            case["rows"], N, dtype=d, device="cuda")
        xs = torch.exp2(s["xs"].view(torch.uint8).to(d) - 127)
        ws = torch.exp2(s["ws"].view(torch.uint8).to(d) - 127)
        for j in range(0, -(-K // BLK)):
            c = slice(j * BLK, min(K, (j + 1) * BLK))
            a = s["xq"][:, c].to(d) * xs[:, j:j + 1]
            b = s["wq"][:, c].to(d) * ws[:, j].repeat_interleave(BLK)[:N, None]
            y = y.addmm(a, b.t())
        return y
    if op == "store":
        lens, new = _store_plan(case)
        seq, h = s["seq"].tolist(), case["kv_heads"]
        out = []
        for src, name in ((s["k"], "ck"), (s["v"], "cv")):
            # whole cache in 64 bits would not fit the largest cases: float32 holds e4m3
            c = s[name].float().view(case["batch"], case["cap"], h, HD)
            u = torch.exp2(s[name + "s"].view(torch.uint8).to(d) - 127)
            at = 0
            for b, (n0, n) in enumerate(zip(lens, new)):
                x = src[at:at + n].to(d).view(n, h, HD)
                at += n
                for blk in range(n0 // BLK, (n0 + n - 1) // BLK + 1):
                    lo, hi = max(n0, blk * BLK), min(n0 + n, (blk + 1) * BLK)
                    part = x[lo - n0:hi - n0]
                    f = _scale_64(part.abs().amax((0, 2)))
                    if blk * BLK < n0:
                        was = u[seq[b], blk]
                        f = torch.maximum(f, was)
                        old = c[seq[b], blk * BLK:n0].to(d) * (was / f)[:, None]
                        c[seq[b], blk * BLK:n0] = _e4m3_64(old).float()
                    u[seq[b], blk] = f
                    c[seq[b], lo:hi] = _e4m3_64(part / f[:, None]).float()
            out += [c.view(s[name].shape).to(d), u]
        return out
    lens, seq = s["lens"].tolist(), s["seq"].tolist()
    B, h = case["batch"], case["kv_heads"]
    G = case["heads"] // h
    out = torch.zeros(B, h, G, HD, dtype=d, device="cuda")
    for b in range(B):
        n = lens[b]
        if n == 0:
            continue
        q = s["q"][b].to(d).view(h, G, HD)
        for j in range(h):
            def rows(name):
                f = torch.exp2(s[name + "s"][seq[b], :, j].view(torch.uint8).to(d) - 127)
                x = s[name][seq[b], :n, j * HD:(j + 1) * HD].to(d)
                return x * f.repeat_interleave(BLK)[:n, None]
            w = torch.softmax(q[j] @ rows("ck").t() / math.sqrt(HD), 1)
            out[b, j] = w @ rows("cv")
    return out.view(B, -1)
