"""8-bit calls behind one another on one stream, each launched before the one in front has ended,
with inputs that change in place."""
import ctypes

import pytest
import torch

from gpu_common import q3
from test_gpu_q8 import _cfg, _gen, _weight

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M,K,N", [(1, 512, 2560), (33, 2560, 2560), (130, 576, 640),
                                   (600, 1024, 2304)])
def test_rows_rewritten_between_products(M, K, N):
    # norm, product, norm, product ... over one buffer of rows and one of scales: each product sees
    # the rows and scales of the norm in front of it
    m = q3()
    cfg = _cfg(K)
    lin = m.quantize_weight_q8(_weight(N, K, 1).cuda())
    steps = 24
    xs = [(2.0 ** (5 * (i % 7) - 15) * torch.randn(M, K, generator=_gen(i))).to(torch.bfloat16).cuda()
          for i in range(steps)]
    want = []
    for x in xs:
        _, q, s = m.add_rms_norm_q8(cfg, x, None)
        torch.cuda.synchronize()
        want.append(m.linear_q8(q, s, lin, out_dtype=torch.float32))
        torch.cuda.synchronize()
    q, s = torch.empty_like(q), torch.empty_like(s)
    outs = [torch.empty_like(w) for w in want]
    lib, p = m.lib(), lambda t: ctypes.c_void_p(t.data_ptr())
    st = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    for _ in range(4):
        for x, o in zip(xs, outs):
            assert lib.q3vl_add_rms_norm_q8(ctypes.byref(cfg), p(x), None, M, None, None, p(q), p(s),
                                            st) == 0
            assert lib.q3vl_linear_q8(p(q), p(s), M, p(lin.weight), p(lin.scales), N, K, None, p(o),
                                      m._abi.DTYPE_FP32, st) == 0
    m.check_device()
    for i, (a, b) in enumerate(zip(outs, want)):
        assert torch.equal(a, b), i


def test_a_weight_made_between_products():
    m = q3()
    M, K, N = 40, 1024, 1280
    ws = [((10.0 ** i) * torch.randn(N, K, generator=_gen(40 + i))).to(torch.bfloat16).cuda()
          for i in range(4)]
    cfg = _cfg(K)
    _, q, s = m.add_rms_norm_q8(cfg, torch.randn(M, K, generator=_gen(50)).to(torch.bfloat16).cuda(),
                                None)
    want = []
    for w in ws:
        lin = m.quantize_weight_q8(w)
        torch.cuda.synchronize()
        want.append(m.linear_q8(q, s, lin, out_dtype=torch.float32))
        torch.cuda.synchronize()
    outs = [torch.empty_like(w) for w in want]
    lib, p = m.lib(), lambda t: ctypes.c_void_p(t.data_ptr())
    st = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    for _ in range(4):
        for w, o in zip(ws, outs):
            assert lib.q3vl_quantize_weight_q8(ctypes.byref(cfg), p(w), N, K, p(lin.weight),
                                               p(lin.scales), st) == 0
            assert lib.q3vl_linear_q8(p(q), p(s), M, p(lin.weight), p(lin.scales), N, K, None, p(o),
                                      m._abi.DTYPE_FP32, st) == 0
    m.check_device()
    for i, (a, b) in enumerate(zip(outs, want)):
        assert torch.equal(a, b), i


def test_split_products_on_two_streams_at_once():
    # wide row tiles of few k-blocks, split over clusters whose CTAs share SMs and their TMEM with
    # the other stream's
    m = q3()
    sides = []
    for i, (M, K, N) in enumerate(((128, 512, 4736), (125, 256, 9000))):
        cfg = _cfg(K)
        x = torch.randn(M, K, generator=_gen(60 + i)).to(torch.bfloat16).cuda()
        _, q, s = m.add_rms_norm_q8(cfg, x, None)
        lin = m.quantize_weight_q8(_weight(N, K, 62 + i).cuda())
        sides.append((q, s, lin, m.linear_q8(q, s, lin)))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [[], []]
    for _ in range(50):
        for i, (q, s, lin, _) in enumerate(sides):
            outs[i].append(m.linear_q8(q, s, lin, stream=streams[i]))
    torch.cuda.synchronize()
    m.check_device()
    for (_, _, _, want), got in zip(sides, outs):
        assert all(torch.equal(g, want) for g in got)
