"""The bars of kv8_bounds.py can fail: what a kernel could lose is over them."""
import pytest
import torch

import kv8_bounds as bounds
import kv8_ref as ref

F16 = torch.float16


def _cache(n, d, blk, gen, sink_gap=None, scale=None):
    """Codes and scales of one head; with a sink, token 0 has a score `gap`
    above the others' and no value."""
    q = torch.randn((1, d), generator=gen) + 0.05 * torch.randn((4, d), generator=gen)
    k, v = 0.05 * torch.randn((n, d), generator=gen), 1 + 0.1 * torch.randn((n, d), generator=gen)
    if sink_gap is not None:
        k[0] = q[0] * sink_gap / (scale * float(q[0] @ q[0]))
        v[0] = 0
    got = []
    for x in (k, v):
        codes, s = torch.zeros((n, d), dtype=torch.uint8), torch.zeros(-(-n // blk))
        ref.append(codes, s, x, 0, n, blk)
        got += [codes, s]
    return q, got[0], got[2], got[1], got[3]


@pytest.mark.parametrize("gap", [17.0, 20.0])
def test_probabilities_rounded_below_the_smallest_fp16_number_are_over_the_bar(gap):
    gen = torch.Generator().manual_seed(1)
    n, d, blk = 3000, 64, 32
    q, k, v, ks, vs = _cache(n, d, blk, gen, gap, 0.125)
    o, _, p, bar, _, _ = bounds.attention(q, k, v, ks, vs, n, blk, 0.125, 1)
    values = ref.value(v) * vs.double().repeat_interleave(blk)[:n, None]
    # relative to the largest probability in (0, 1], and in (0, 2^15]
    top = p.amax(1, keepdim=True)
    for head, fine in ((0, False), (15, True)):
        held = (p / top * 2.0 ** head).to(F16).double() * 2.0 ** -head * top
        err = (held @ values - o).abs()
        assert (err <= bar).all() if fine else (err > bar).all()


@pytest.mark.parametrize("n,d", [(500, 64), (5999, 128)])
def test_lost_tokens_are_over_the_bar(n, d):
    gen = torch.Generator().manual_seed(2)
    q, k, v, ks, vs = _cache(n, d, 64, gen)
    o, lse, p, bar, bar_l, _ = bounds.attention(q, k, v, ks, vs, n, 64, d ** -0.5, 8)
    values = ref.value(v) * vs.double().repeat_interleave(64)[:n, None]
    assert (o.abs() > bar).all()
    lost = p.clone()
    lost[:, 100:132] = 0  # 32 tokens miss the product with V
    assert ((lost @ values - o).abs() > bar).all()
    assert (torch.log(lost.sum(1)).abs() > bar_l).all()


@pytest.mark.parametrize("M,K,N", [(1, 4096, 64), (4, 14336, 16), (1, 16384, 33), (2, 24544, 20),
                                   (1, 65536, 9)])
def test_a_lost_chunk_and_zeros_are_over_the_linear_bar(M, K, N):
    gen = torch.Generator().manual_seed(3)
    x = (torch.randn((M, K), generator=gen) * torch.exp(torch.randn(K, generator=gen))).double()
    w = torch.randn((N, K), generator=gen).double()
    y, bar = bounds.linear(x, w)
    assert (y.abs() > bar).float().mean() > 0.8
    lost, _ = bounds.linear(x, w, drop=(K // 512 * 256, K // 512 * 256 + 256))
    assert ((lost - y).abs() > bar + 2.0 ** -8 * y.abs()).any()


def test_digits_leave_what_six_of_them_may():
    gen = torch.Generator().manual_seed(4)
    x = (torch.randn((3, 640), generator=gen) * torch.exp(3 * torch.randn(640, generator=gen))).double()
    left = (x - bounds.digits(x).sum(0)).abs()
    top = x.abs().unflatten(1, (-1, 16)).amax(-1).repeat_interleave(16, 1)
    assert (left <= 2.0 ** -16 * top + 2.0 ** -33 * x.abs().amax(1, keepdim=True)).all()
    ints = torch.randint(-15, 16, (2, 512), generator=gen).double()
    assert torch.equal(bounds.digits(ints).sum(0), ints)
