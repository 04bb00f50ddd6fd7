"""The linear layer over NVFP4 weights against fp64: every shape within half
a step of the output type and the bar of the arithmetic (kv8_ref.linear_bar)."""
import math

import pytest
import torch

import kv8_ref as ref
from bit_quantization_b200 import ops

pytestmark = pytest.mark.gpu
BF16, FP16 = torch.bfloat16, torch.float16


def _weights(N, K, gen, dtype=BF16):
    w = torch.randn((N, K), generator=gen).to(dtype).cuda()
    c = max(c for c in range(16, 4097, 16) if K % c == 0)  # at most 4096 columns a call
    codes, scales, g = ops.nvfp4_quantize(w.view(-1, c))
    return codes.view(N, K // 2), scales.view(N, K // 16), g


def _check(x, codes, scales, g, y):
    w = ref.dequant(codes.cpu(), scales.cpu(), g)
    xd = x.cpu().double()
    want = xd @ w.T
    bar = torch.finfo(x.dtype).eps / 2 * want.abs() + ref.linear_bar(xd, w) + \
        torch.finfo(x.dtype).smallest_normal * torch.finfo(x.dtype).eps
    err = (y.cpu().double() - want).abs()
    assert (err <= bar).all(), (float((err - bar).max()), float((err / bar).max()))


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("M,K,N", [
    (1, 32, 1), (1, 64, 7), (2, 96, 128), (3, 256, 129), (1, 4096, 1024), (5, 2080, 300),
    (7, 1056, 1111), (8, 512, 2000), (16, 4096, 256), (15, 224, 513), (17, 320, 130),
    (33, 1024, 200), (64, 640, 384), (1, 16384, 257), (4, 14336, 128), (2, 4064, 5000),
    (1, 65536, 33), (18, 24544, 260), (2, 524288, 3),
])
def test_linear(M, K, N, dtype):
    gen = torch.Generator().manual_seed(M * 1000 + K + N)
    x = (torch.randn((M, K), generator=gen) * torch.exp(torch.randn(K, generator=gen))).to(dtype)
    args = _weights(N, K, gen)
    y = ops.nvfp4_linear(x.cuda(), *args)
    assert y.shape == (M, N) and y.dtype == dtype
    _check(x, *args, y)


@pytest.mark.parametrize("what", ["outlier", "tiny", "huge", "zero", "sparse", "one_row_zero"])
def test_linear_magnitudes(what):
    gen = torch.Generator().manual_seed(11)
    x = torch.randn((4, 1024), generator=gen)
    if what == "outlier":  # one channel a thousand times the others
        x[:, 77] *= 3000
    elif what == "tiny":
        x *= 2.0 ** -120
    elif what == "huge":
        x *= 2.0 ** 100
    elif what == "zero":
        x *= 0
    elif what == "sparse":
        x *= torch.rand(x.shape, generator=gen) < 0.01
    else:
        x[2] = 0
    x = x.to(BF16)
    args = _weights(300, 1024, gen)
    _check(x, *args, ops.nvfp4_linear(x.cuda(), *args))


def test_linear_not_finite_rows():
    gen = torch.Generator().manual_seed(12)
    x = torch.randn((5, 512), generator=gen).to(FP16).cuda()
    args = _weights(200, 512, gen)
    clean = ops.nvfp4_linear(x, *args)
    x[1, 500] = math.nan
    x[3, 0] = -math.inf
    y = ops.nvfp4_linear(x, *args)
    assert torch.isnan(y[[1, 3]]).all()
    assert torch.equal(y[[0, 2, 4]], clean[[0, 2, 4]])


def test_linear_all_codes_and_scales():
    """Every code under every UE4M3 scale byte but NaN, subnormal ones included."""
    scales = torch.arange(127, dtype=torch.uint8).repeat_interleave(2).reshape(127, 2)
    codes = torch.arange(16, dtype=torch.uint8)
    codes = (codes[::2] | codes[1::2] << 4).repeat(127, 2)
    x = torch.zeros((32, 32), dtype=FP16)
    x[torch.arange(32), torch.arange(32)] = 1.0  # one column of the weights a row
    g = torch.tensor([0.125], device="cuda")
    y = ops.nvfp4_linear(x.cuda(), codes.cuda(), scales.cuda(), g)
    assert torch.equal(y.cpu().double(), ref.dequant(codes, scales, 0.125).T.to(FP16).double())


def test_linear_repeats_across_streams_and_graphs():
    gen = torch.Generator().manual_seed(13)
    x = torch.randn((3, 4096), generator=gen).to(BF16).cuda()
    args = _weights(777, 4096, gen)
    first = ops.nvfp4_linear(x, *args)
    torch.cuda.synchronize()
    got = []
    for s in [torch.cuda.Stream() for _ in range(3)]:
        with torch.cuda.stream(s):
            got.append(ops.nvfp4_linear(x, *args))
    stream, graphs = torch.cuda.Stream(), []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=stream):
            got.append(ops.nvfp4_linear(x, *args))
        graphs.append(g)
    for g in graphs:
        g.replay()
    torch.cuda.synchronize()
    for y in got:
        assert torch.equal(y, first)
    x2 = x.flip(0).contiguous()
    want = ops.nvfp4_linear(x2, *args)
    x.copy_(x2)
    graphs[0].replay()
    torch.cuda.synchronize()
    assert torch.equal(got[3], want)
    assert ops.device_status() == ops.OK


def test_results_are_complete_for_the_call_that_follows():
    """The quantiser, whose first kernel reads its input as soon as it is
    scheduled, right behind the attention (split and in one launch) and the
    linear layer: the same codes as from their finished results."""
    gen = torch.Generator().manual_seed(15)
    args = _weights(4096, 4096, gen)
    x = torch.randn((16, 4096), generator=gen).to(BF16).cuda()
    caches = [ops.KV8Cache(B, 8, cap, d=128, blk=64) for B, cap in ((8, 8000), (2, 1000))]
    qs = []
    for c in caches:
        B, _, cap, _ = c.k.shape
        new = torch.randn((B, cap, 8, 128), generator=gen).to(BF16).cuda()
        c.append(new, -new)
        qs.append(torch.randn((B, 32, 128), generator=gen).to(BF16).cuda())
    for i in range(20):
        for call in [lambda: ops.nvfp4_linear(x, *args)] + [
                lambda c=c, q=q: c.decode(q, accumulate=bool(i % 2))[0].view(-1, 128)
                for c, q in zip(caches, qs)]:
            torch.cuda.synchronize()
            y = call()
            got = ops.nvfp4_quantize(y)
            torch.cuda.synchronize()
            want = ops.nvfp4_quantize(y)
            for a, b in zip(got, want):
                assert torch.equal(a, b)


def test_linear_empty():
    x = torch.zeros((0, 64), dtype=BF16, device="cuda")
    codes = torch.zeros((5, 32), dtype=torch.uint8, device="cuda")
    scales = torch.zeros((5, 4), dtype=torch.uint8, device="cuda")
    g = torch.ones(1, device="cuda")
    assert ops.nvfp4_linear(x, codes, scales, g).shape == (0, 5)
    x = torch.ones((2, 64), dtype=BF16, device="cuda")
    assert ops.nvfp4_linear(x, codes[:0], scales[:0], g).shape == (2, 0)
    assert not ops.nvfp4_linear(x, codes, scales, g).any()


def test_generation_step_layers():
    """One generation step of an attention layer by its operators: q, k, v
    projections by NVFP4 weights, the append, the attention with accumulated
    weights, the output projection; against fp64 of the same quantised
    weights and cache, each operator within its own bar."""
    gen = torch.Generator().manual_seed(14)
    B, H, Hkv, d, hidden = 4, 8, 2, 64, 512
    wq, wk, wv = (_weights(n * d, hidden, gen) for n in (H, Hkv, Hkv))
    wo = _weights(hidden, H * d, gen)
    cache = ops.KV8Cache(B, Hkv, 100, d=d, blk=16)
    prompt = torch.randn((B, 60, Hkv, d), generator=gen).to(BF16).cuda()
    cache.append(prompt, prompt.flip(1).contiguous(),
                 torch.tensor([60, 1, 33, 0], dtype=torch.int32, device="cuda"))
    lengths = [60, 1, 33, 0]
    for _ in range(3):
        x = torch.randn((B, hidden), generator=gen).to(BF16).cuda()
        q, k, v = (ops.nvfp4_linear(x, *w) for w in (wq, wk, wv))
        for w, y in ((wq, q), (wk, k), (wv, v)):
            _check(x, *w, y)
        cache.append(k.view(B, 1, Hkv, d), v.view(B, 1, Hkv, d))
        lengths = [n + 1 for n in lengths]
        out, lse = cache.decode(q.view(B, H, d), accumulate=True)
        for b in range(B):
            for h in range(Hkv):
                rows = slice(h * (H // Hkv), (h + 1) * (H // Hkv))
                o, l, _, bo, bl, _ = ref.decode(
                    q.view(B, H, d)[b, rows].cpu(), cache.k[b, h].cpu().view(torch.uint8),
                    cache.v[b, h].cpu().view(torch.uint8), cache.k_scale[b, h].cpu(),
                    cache.v_scale[b, h].cpu(), lengths[b], 16, d ** -0.5)
                err = (out[b, rows].cpu().double() - o).abs()
                assert (err <= torch.finfo(BF16).eps / 2 * o.abs() + bo).all()
                assert ((lse[b, rows].cpu().double() - l).abs() <= bl).all()
        flat = out.view(B, H * d)
        _check(flat, *wo, ops.nvfp4_linear(flat, *wo))
    assert cache.lengths.tolist() == lengths
    assert abs(float(cache.weight.sum()) - 3 * B * H) < 1e-3
