"""Calls that follow one another in a stream without a stop give what they give
with the GPU waited for after each: no kernel reads what the one before it is
still writing, however early it is scheduled."""
import pytest
import torch

from bit_quantization_b200 import ops

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


@pytest.mark.parametrize("M,K,N", [(1, 4096, 512), (16, 1024, 3000), (4, 256, 40)])
def test_weights_quantised_right_before_the_linear_layer(M, K, N):
    gen = torch.Generator(device="cuda").manual_seed(K + N)
    ws = [torch.randn((N, K), generator=gen, device="cuda").to(BF16) for _ in range(3)]
    xs = [torch.randn((M, K), generator=gen, device="cuda").to(BF16) for _ in range(3)]
    codes = torch.empty((N, K // 2), dtype=torch.uint8, device="cuda")
    scales = torch.empty((N, K // 16), dtype=torch.uint8, device="cuda")
    x = torch.empty_like(xs[0])

    def call(i, stop):
        x.copy_(xs[i % 3])
        g = ops.nvfp4_quantize(ws[i % 3], codes=codes, scales=scales)[2]
        if stop:
            torch.cuda.synchronize()
        return ops.nvfp4_linear(x, codes, scales, g)

    want = [call(i, True) for i in range(3)]
    torch.cuda.synchronize()
    got = [call(i, False) for i in range(150)]
    wrong = sum((y != want[i % 3]).sum() for i, y in enumerate(got))
    assert int(wrong) == 0


@pytest.mark.parametrize("B,Hkv,G,d,cap", [(1, 1, 1, 64, 500), (4, 8, 4, 128, 1000), (40, 2, 9, 64, 900)])
def test_generation_without_a_stop(B, Hkv, G, d, cap):
    """Steps of append and attention with weights, and an eviction whenever the
    longest sequence may not take the next one, into a spare cache."""
    def run(stop):
        gen = torch.Generator(device="cuda").manual_seed(cap)
        cache, spare = (ops.KV8Cache(B, Hkv, cap, d=d, blk=16) for _ in range(2))
        outs, longest = [], 0
        for i in range(120):
            T = 40 if i % 20 == 0 else 1 + i % 3
            kn, vn = (torch.randn((B, T, Hkv, d), generator=gen, device="cuda").to(BF16)
                      for _ in range(2))
            n = torch.randint(0, T + 1, (B,), generator=gen, device="cuda", dtype=torch.int32)
            q = torch.randn((B, Hkv * G, d), generator=gen, device="cuda").to(BF16)
            if longest + T > cap // 2:
                spare.lengths.fill_(3)
                cache, spare = cache.evict(cap // 4, recent=9, sink=2, out=spare), cache
                longest = cap // 4
                if stop:
                    torch.cuda.synchronize()
            cache.append(kn, vn, n)
            longest += T
            if stop:
                torch.cuda.synchronize()
            outs += cache.decode(q, accumulate=i % 2 == 0)
            if stop:
                torch.cuda.synchronize()
        return outs + [cache.lengths, cache.weight.clone().masked_fill_(
            torch.arange(cap, device="cuda") >= cache.lengths[:, None, None], 0.0)]

    want, got = run(True), run(False)
    for a, b in zip(want, got):
        assert torch.equal(a, b)
