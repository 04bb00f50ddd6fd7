"""Accuracy of the attention over the 8-bit cache where it is hardest to keep
(bars of kv8_bounds.py): a token that outweighs all others and has no value,
long contexts, and sums that are exact in fp32 and so pinned bit for bit."""
import math

import pytest
import torch

import kv8_bounds as bounds
from bit_quantization_b200 import ops

pytestmark = pytest.mark.gpu
F8 = torch.float8_e4m3fn
BF16, FP16 = torch.bfloat16, torch.float16


def _fill(kn, vn, blk, cap):
    """A cache of [B, n, Hkv, d] tokens, all of them there."""
    B, n, Hkv, d = kn.shape
    c = ops.KV8Cache(B, Hkv, cap, d=d, blk=blk, dtype=kn.dtype)
    c.append(kn.contiguous(), vn.contiguous())
    return c


def _check(c, q, n, out, lse, scale, weight=None):
    B, H, d = q.shape
    Hkv = c.k.shape[1]
    G = H // Hkv
    eps = torch.finfo(q.dtype).eps / 2
    tiny = torch.finfo(q.dtype).smallest_normal * torch.finfo(q.dtype).eps / 2
    for b in range(B):
        for h in range(Hkv):
            rows = slice(h * G, (h + 1) * G)
            o, l, p, bo, bl, bp = bounds.attention(
                q[b, rows], c.k[b, h].view(torch.uint8), c.v[b, h].view(torch.uint8),
                c.k_scale[b, h], c.v_scale[b, h], n, c.blk, scale, B * Hkv * -(-G // 16))
            err = (out[b, rows].double() - o).abs()
            assert (err <= eps * (o.abs() + bo) + bo + tiny).all(), (b, h, float((err / bo).max()))
            assert ((lse[b, rows].double() - l).abs() <= bl).all(), (b, h)
            if weight is not None:
                bar = bp.sum(0) + (2 * G + 4) * 2.0 ** -24 * p.sum(0)
                assert ((weight[b, h, :n].double() - p.sum(0)).abs() <= bar).all(), (b, h)


@pytest.mark.parametrize("gap", [10.0, 17.0, 18.0, 20.0, 24.0])
@pytest.mark.parametrize("n,at,G,d,dtype", [
    (1, 0, 1, 64, BF16), (500, 0, 4, 128, BF16), (1000, 999, 8, 64, FP16), (6000, 0, 4, 128, BF16),
    (6000, 3001, 12, 64, FP16), (40000, 0, 7, 64, BF16),
])
def test_sink(n, at, G, d, dtype, gap):
    """One token `gap` above the others' scores, with a value of zero: what is
    left of the output is the others' share, exp(-gap) each."""
    gen = torch.Generator(device="cuda").manual_seed(n + G)
    Hkv, scale = 2, d ** -0.5

    def randn(*shape):
        return torch.randn(shape, generator=gen, device="cuda")

    base = randn(1, Hkv, 1, d)
    q = (base + 0.05 * randn(1, Hkv, G, d)).flatten(1, 2)
    kn = 0.05 * randn(1, n, Hkv, d)
    vn = 64.0 + 8.0 * randn(1, n, Hkv, d)
    kn[0, at] = base[0, :, 0] * gap / (scale * (base[0, :, 0] ** 2).sum(-1, keepdim=True))
    vn[0, at] = 0.0
    c = _fill(kn.to(dtype), vn.to(dtype), 32, n if n > 1024 else 1024)
    q = q.to(dtype).contiguous()
    for accumulate in (False, True):
        c.weight.zero_()
        out, lse = c.decode(q, accumulate=accumulate)
        _check(c, q, n, out, lse, scale, c.weight if accumulate else None)


@pytest.mark.parametrize("n,Hkv,G,d,blk,dtype", [
    (131072, 2, 4, 128, 128, BF16), (131071, 1, 16, 64, 32, FP16), (30011, 3, 20, 128, 64, FP16),
])
def test_long(n, Hkv, G, d, blk, dtype):
    """Long contexts, with and without the accumulated weights; values with a
    mean, so that the output is not smaller than its bar."""
    gen = torch.Generator(device="cuda").manual_seed(n)
    kn, vn = (torch.randn((1, n, Hkv, d), generator=gen, device="cuda") for _ in range(2))
    kn += 3 * torch.randn((1, 1, Hkv, d), generator=gen, device="cuda")
    c = _fill(kn.to(dtype), (vn + 2).to(dtype), blk, n)
    q = torch.randn((1, Hkv * G, d), generator=gen, device="cuda").to(dtype)
    for accumulate in (False, True):
        out, lse = c.decode(q, accumulate=accumulate)
        _check(c, q, n, out, lse, d ** -0.5, c.weight if accumulate else None)


@pytest.mark.parametrize("n,G,d,dtype", [
    (1, 1, 64, BF16), (777, 8, 128, FP16), (1024, 3, 64, BF16), (5000, 16, 128, BF16),
    (100003, 4, 64, FP16), (131072, 9, 128, FP16), (131072, 2, 64, FP16),
])
def test_flat_rows_are_exact(n, G, d, dtype):
    """Equal scores and values that are small integers under scales that change
    from block to block: every sum is an integer below 2^24, so that the output
    is the integer sum over n, rounded as one division and the type."""
    gen = torch.Generator(device="cuda").manual_seed(n + d)
    Hkv, blk = 2, 32
    vn = torch.randint(-3, 4, (1, n, Hkv, d), generator=gen, device="cuda")
    block = torch.arange(n, device="cuda") // blk
    vn = vn * (2 ** (block * 7 % 5))[None, :, None, None]
    total = vn.double().sum(1).reshape(Hkv, 1, d)
    assert vn.abs().sum(1).max() < 1 << 24
    kn = torch.randn((1, n, Hkv, d), generator=gen, device="cuda")
    c = _fill(kn.to(dtype), vn.to(dtype), blk, n)
    q = torch.zeros((1, Hkv * G, d), dtype=dtype, device="cuda")
    want = (total.float() / n).to(dtype).expand(Hkv, G, d).reshape(1, Hkv * G, d)
    for accumulate in (False, True):
        out, lse = c.decode(q, accumulate=accumulate)
        assert torch.equal(out, want)
        assert ((lse.double() - math.log(n)).abs() <= 2.0 ** -22 * (math.log(n) + 1)).all()
    assert ((c.weight.double() * n / G - 1).abs() <= (2 * G + 4) * 2.0 ** -24).all()


@pytest.mark.parametrize("cap,B,Hkv,G,d", [
    (1024, 1, 8, 4, 128), (1025, 1, 8, 4, 128), (2048, 2, 2, 8, 64), (2049, 2, 2, 8, 64),
    (1024, 18, 8, 2, 128), (1024, 19, 8, 2, 128), (2048, 1, 1, 9, 64),
])
def test_one_launch_or_two(cap, B, Hkv, G, d):
    """Both sides of the rule that has a short cache attended to in one launch,
    full and at the edges of its steps."""
    gen = torch.Generator(device="cuda").manual_seed(cap + B)
    kn, vn = (torch.randn((B, cap, Hkv, d), generator=gen, device="cuda") for _ in range(2))
    c = _fill(kn.to(BF16), (vn + 2).to(BF16), 16, cap)
    q = torch.randn((B, Hkv * G, d), generator=gen, device="cuda").to(BF16)
    for n in (1, 255, 256, 513, 1023, cap):
        c.lengths.fill_(n)
        out, lse = c.decode(q)
        _check(c, q, n, out, lse, d ** -0.5)
