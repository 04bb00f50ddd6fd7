"""The linear layer over NVFP4 weights at long contractions: sums that are
exact in fp32, bit for bit, and real values within the bar of the kernel's own
sums (kv8_bounds.linear)."""
import pytest
import torch

import kv8_bounds as bounds
import kv8_ref as ref
from bit_quantization_b200 import ops

pytestmark = pytest.mark.gpu
BF16, FP16 = torch.bfloat16, torch.float16


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("M,K,N", [
    (1, 32, 130), (1, 4096, 1024), (2, 14336, 513), (16, 14336, 200), (1, 65536, 129), (5, 65568, 64),
    (33, 16384, 140), (64, 4096, 300), (1, 524288, 5), (17, 524288, 3),
])
def test_integer_sums_are_exact(M, K, N, dtype):
    """x of integers up to 15 and weights that are multiples of 1/2 up to 6
    under scales 1/2, 1 and 2: a digit's products are multiples of 1/16 (a
    digit of 1/2 under a block's 1/2, a weight of 1/2 under 1/2) below 2^24
    times that, so no sum rounds."""
    gen = torch.Generator(device="cuda").manual_seed(K + N)
    x = torch.randint(-15, 16, (M, K), generator=gen, device="cuda")
    codes = torch.randint(0, 256, (N, K // 2), generator=gen, device="cuda", dtype=torch.uint8)
    # UE4M3 1/2, 1, 2: exponents 6, 7, 8 over the bias of 7
    scales = (torch.randint(6, 9, (N, K // 16), generator=gen, device="cuda") * 8).to(torch.uint8)
    g = torch.tensor([2.0 ** -10], device="cuda")
    w = torch.cat([_weights(c, s) for c, s in zip(codes.split(64), scales.split(64))])
    xd = x.double()
    # any stretch of columns is the difference of two of these, below 2^20
    for i, d in enumerate(bounds.digits(xd[:2])):
        assert (d[:, None] * w[None, :64]).cumsum(-1).abs().amax() * 8.0 ** i < 1 << 19
    want = (xd @ w.T).float() * g
    y = ops.nvfp4_linear(x.to(dtype), codes, scales, g)
    assert torch.equal(y, want.to(dtype))


def _weights(codes, scales):
    grid = ref.E2M1.to(codes.device)
    c = torch.stack((codes & 15, codes >> 4), -1).flatten(1).long()
    w = grid[c & 7] * (1 - 2 * (c >> 3)).double()
    return w * scales.view(torch.float8_e4m3fn).double().repeat_interleave(16, 1)


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("M,K,N", [
    (1, 96, 65), (1, 4096, 1024), (5, 2080, 300), (4, 14336, 128), (1, 16384, 257), (2, 4064, 500),
    (18, 24544, 130), (1, 65536, 33),
])
def test_real_values_within_the_bar_of_the_sums(M, K, N, dtype):
    gen = torch.Generator(device="cuda").manual_seed(M + K + N)
    x = torch.randn((M, K), generator=gen, device="cuda")
    x = (x * torch.exp(torch.randn(K, generator=gen, device="cuda"))).to(dtype)
    c = max(c for c in range(16, 4097, 16) if K % c == 0)  # at most 4096 columns a call
    codes, scales, g = ops.nvfp4_quantize(
        torch.randn((N * K // c, c), generator=gen, device="cuda").to(BF16))
    codes, scales = codes.view(N, K // 2), scales.view(N, K // 16)
    y = ops.nvfp4_linear(x, codes, scales, g)
    want, bar = bounds.linear(x.double(), _weights(codes, scales) * g.double())
    eps = torch.finfo(dtype).eps / 2
    err = (y.double() - want).abs()
    assert (err <= eps * (want.abs() + bar) + bar).all(), float((err / (bar + eps * want.abs())).max())
