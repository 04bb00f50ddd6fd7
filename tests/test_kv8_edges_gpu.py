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
