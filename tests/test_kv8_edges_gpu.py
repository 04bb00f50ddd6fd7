"""Calls of the 8-bit cache at the ends of what they take."""
import pytest
import torch

import kv8_ref as ref
from bit_quantization_b200 import ops

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


def _u8(t):
    return t.cpu().view(torch.uint8)


def test_evict_of_empty_sequences_then_an_append():
    """Nothing to gather: the lengths that the eviction writes are what the
    append right behind it goes by, not those the spare cache held before."""
    gen = torch.Generator().manual_seed(1)
    B, Hkv, cap = 64, 8, 4096
    empty, spare = (ops.KV8Cache(B, Hkv, cap, d=64, blk=16) for _ in range(2))
    x = torch.randn((B, 1, Hkv, 64), generator=gen).to(BF16).cuda()
    want = ops.KV8Cache(B, Hkv, cap, d=64, blk=16)
    want.append(x, x)
    torch.cuda.synchronize()
    for i in range(50):
        spare.lengths.fill_(7 + i)  # of its previous contents
        empty.evict(100 + i, recent=3, out=spare).append(x, x)
        assert spare.lengths.tolist() == [1] * B
        assert torch.equal(_u8(spare.k)[:, :, 0], _u8(want.k)[:, :, 0])
        assert torch.equal(spare.k_scale[:, :, 0], want.k_scale[:, :, 0])


@pytest.mark.parametrize("blk", [16, 128])
def test_evict_keeps_codes_that_stand_for_two_to_the_128(blk):
    """The largest bf16 values round to a code 256 * 2^120: a number, although
    not one of fp32.  It counts for the new block's scale as it did for the
    old one's."""
    n = 2 * blk
    x = torch.ones((1, n, 1, 64), dtype=BF16, device="cuda")
    x[0, 3, 0, 5] = torch.finfo(BF16).max
    x[0, blk, 0, 7] = -torch.finfo(BF16).max
    c = ops.KV8Cache(1, 1, n, d=64, blk=blk)
    c.append(x, x)
    assert c.k_scale.tolist() == [[[2.0 ** 120] * 2]]
    c.weight.copy_(torch.arange(n, 0, -1.0))  # the first ones stay
    cut = c.evict(n - 1)
    assert cut.lengths.tolist() == [n - 1]
    assert cut.k_scale.tolist() == [[[2.0 ** 120] * 2]]
    assert torch.equal(_u8(cut.k)[0, 0, :n - 1], _u8(c.k)[0, 0, :n - 1])
    assert torch.equal(_u8(cut.v)[0, 0, :n - 1], _u8(c.v)[0, 0, :n - 1])


@pytest.mark.parametrize("budget,recent,sink", [
    ((1 << 32) + 5, 0, 0), (1 << 40, (1 << 33) + 7, 1 << 34), (40, 20, 20), (1 << 31, 3, 4),
])
def test_a_budget_beyond_the_cache_keeps_everything(budget, recent, sink):
    gen = torch.Generator().manual_seed(1)
    c = ops.KV8Cache(2, 1, 40, d=64, blk=16)
    x = torch.randn((2, 40, 1, 64), generator=gen).to(BF16).cuda()
    c.append(x, -x, torch.tensor([40, 13], dtype=torch.int32, device="cuda"))
    cut = c.evict(budget, recent=recent, sink=sink)
    assert cut.lengths.tolist() == [40, 13]
    for b, n in ((0, 40), (1, 13)):
        for i in (0, 1):  # encoded anew: a largest value that was rounded may need a smaller scale
            codes, scales = ref.reblock(_u8(c.tensors[i])[b, 0], c.tensors[2 + i][b, 0].cpu(),
                                        list(range(n)), 16)
            assert torch.equal(_u8(cut.tensors[i])[b, 0, :n], codes)
            assert torch.equal(cut.tensors[2 + i][b, 0, :len(scales)].cpu(), scales)


def test_captured_prompt_append_and_eviction_replay():
    """A prompt's append (two launches) and the eviction (a cluster launch and
    the gather), captured on one stream and replayed between eager calls that
    change lengths, weights and tokens."""
    gen = torch.Generator(device="cuda").manual_seed(9)
    B, Hkv, d, blk, cap, T = 3, 2, 64, 32, 20000, 9000
    c, spare, want = (ops.KV8Cache(B, Hkv, cap, d=d, blk=blk) for _ in range(3))
    x = torch.randn((B, T, Hkv, d), generator=gen, device="cuda").to(BF16)
    n = torch.full((B,), T, dtype=torch.int32, device="cuda")
    c.append(x, -x, n)  # warm
    c.evict(5000, recent=100, sink=4, out=spare)
    stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        c.append(x, -x, n)
        c.evict(5000, recent=100, sink=4, out=spare)
    for lengths, counts in (([0, 0, 0], [T, 1, 0]), ([7000, 20000, 31], [T, 5, 4970]),
                            ([0, 0, 0], [0, 0, 0]), ([19999, 12000, 5000], [1, T, 0])):
        x.copy_(torch.randn(x.shape, generator=gen, device="cuda"))
        n.copy_(torch.tensor(counts, dtype=torch.int32))
        c.lengths.copy_(torch.tensor(lengths, dtype=torch.int32))
        c.weight.copy_(torch.rand(c.weight.shape, generator=gen, device="cuda"))
        spare.lengths.fill_(77)
        before = [t.clone() for t in (*c.tensors, c.weight, c.lengths)]
        graph.replay()
        got = [t.clone() for t in (*spare.tensors, spare.weight, spare.lengths)]
        for t, old in zip((*c.tensors, c.weight, c.lengths), before):
            t.copy_(old)
        c.append(x, -x, n)
        c.evict(5000, recent=100, sink=4, out=want)
        torch.cuda.synchronize()
        kept = [min(5000, cap, a + b) for a, b in zip(lengths, counts)]
        assert got[5].tolist() == kept == want.lengths.tolist()
        for b, m in enumerate(kept):
            for g, w in zip(got[:2], want.tensors[:2]):
                assert torch.equal(_u8(g)[b, :, :m], _u8(w)[b, :, :m])
            for g, w in zip(got[2:4], want.tensors[2:]):
                assert torch.equal(g[b, :, :-(-m // blk)], w[b, :, :-(-m // blk)])
            assert torch.equal(got[4][b, :, :m], want.weight[b, :, :m])
