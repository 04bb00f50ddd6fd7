"""The 8-bit KV cache on the GPU against the 64-bit forms of kv8_ref.py:
codes, scales, survivors and lengths bit for bit, attention within bars
derived from the kernel's arithmetic; what the documentation allows beside
the plain call: both memory orders, interleaved K and V, garbage behind the
lengths, streams, captured and replayed steps."""
import math

import numpy as np
import pytest
import torch

import kv8_ref as ref
from bit_quantization_b200 import ops

pytestmark = pytest.mark.gpu
F8 = torch.float8_e4m3fn
BF16, FP16 = torch.bfloat16, torch.float16


def _codes(shape, layout, gen, fill="random"):
    """Two code tensors [B, Hkv, cap, d] on the device, in one memory order;
    every byte value occurs, the NaN codes among them."""
    B, Hkv, cap, d = shape
    if layout == "head":
        full = [(B, Hkv, cap, d)] * 2
    elif layout == "token":
        full = [(B, cap, Hkv, d)] * 2
    else:  # K and V of a token side by side
        full = [(B, Hkv, cap, 2, d)]
    raw = [torch.randint(0, 256, f, generator=gen, dtype=torch.uint8).cuda() for f in full]
    if layout == "head":
        return raw[0].view(F8), raw[1].view(F8)
    if layout == "token":
        return tuple(r.transpose(1, 2).view(F8) for r in raw)
    return raw[0][..., 0, :].view(F8), raw[0][..., 1, :].view(F8)


def _scales(shape, blk, gen):
    B, Hkv, cap, _ = shape
    return [torch.randn((B, Hkv, -(-cap // blk)), generator=gen).cuda() for _ in range(2)]


def _u8(t):
    return t.cpu().view(torch.uint8)


def _values(shape, gen, dtype, wild=False):
    x = torch.randn(shape, generator=gen) + 3 * torch.randn((1, 1) + shape[2:], generator=gen)
    if wild:  # magnitudes over many octaves, zero rows, values that are not finite
        x *= torch.exp(3 * torch.randn(shape[:3] + (1,), generator=gen))
        x[:, ::7] = 0.0
        flat = x.view(-1)
        flat[torch.randint(0, flat.numel(), (3,), generator=gen)] = math.inf
        flat[torch.randint(0, flat.numel(), (3,), generator=gen)] = math.nan
    return x.to(dtype)


APPENDS = [
    # shape, blk, layout, dtype, (start lengths, pieces of at most T tokens each)
    ((1, 1, 1, 64), 16, "head", BF16, [0], [[1]]),
    ((1, 1, 40, 64), 16, "head", FP16, [0], [[1]] * 20),
    ((3, 2, 300, 128), 64, "token", BF16, [0, 63, 299], [[1, 1, 1], [0, 65, 9], [130, 1, 5]]),
    ((2, 3, 257, 128), 128, "pair", FP16, [128, 255], [[129, 1], [0, 1], [7, 7]]),
    ((4, 5, 100, 64), 32, "token", BF16, [0, 31, 32, 100], [[33, 1, 0, 4], [1, 1, 1, 1]]),
    ((2, 8, 1000, 128), 32, "head", BF16, [0, 500], [[999, 300], [1, 1], [1, 300]]),
    ((70, 1, 20, 64), 16, "head", FP16, [0] * 70, [[1] * 70, [18] * 70]),
]


@pytest.mark.parametrize("wild", [False, True])
@pytest.mark.parametrize("case", range(len(APPENDS)))
def test_append(case, wild):
    shape, blk, layout, dtype, start, pieces = APPENDS[case]
    B, Hkv, cap, d = shape
    gen = torch.Generator().manual_seed(100 + case)
    k, v = _codes(shape, layout, gen)
    ks, vs = _scales(shape, blk, gen)
    weight = torch.randn((B, Hkv, cap), generator=gen).cuda()
    lengths = torch.tensor(start, dtype=torch.int32, device="cuda")
    # rows already there are given scales the append rule can have left
    for s in (ks, vs):
        s.copy_(torch.exp2(torch.randint(-9, 3, s.shape, generator=gen).float()))
    want = [_u8(k).clone(), _u8(v).clone(), ks.cpu().clone(), vs.cpu().clone(), weight.cpu().clone()]
    at = list(start)
    for i, n in enumerate(pieces):
        T = max(n) + i % 2
        kn, vn = _values((B, T, Hkv, d), gen, dtype, wild), _values((B, T, Hkv, d), gen, dtype, wild)
        ops.thrift_kv8_append(kn.cuda(), vn.cuda(), k, v, ks, vs, lengths,
                              torch.tensor(n, dtype=torch.int32, device="cuda"), blk=blk,
                              weight=weight, new_len=lengths)
        for b in range(B):
            for h in range(Hkv):
                for c, s, x in ((0, 2, kn), (1, 3, vn)):
                    end = ref.append(want[c][b, h], want[s][b, h], x[b, :, h], at[b], n[b], blk)
            want[4][b, :, at[b]:end] = 0.0
            at[b] = end
        got = [_u8(k), _u8(v), ks.cpu(), vs.cpu(), weight.cpu()]
        for name, g, w in zip(("k", "v", "k_scale", "v_scale", "weight"), got, want):
            assert torch.equal(g, w), (name, i)
        assert lengths.tolist() == at


def test_append_default_count_and_out_of_place_length():
    gen = torch.Generator().manual_seed(7)
    c = ops.KV8Cache(2, 2, 50, d=64, blk=16, dtype=FP16)
    x = _values((2, 20, 2, 64), gen, FP16).cuda()
    new_len = torch.full((2,), -5, dtype=torch.int32, device="cuda")
    ops.thrift_kv8_append(x, x, *c.tensors, c.lengths, blk=16, new_len=new_len)
    assert new_len.tolist() == [20, 20] and c.lengths.tolist() == [0, 0]
    for _ in range(3):
        c.append(x, x)
    assert c.lengths.tolist() == [50, 50]
    before = _u8(c.k).clone()
    c.append(x[:, :0], x[:, :0])  # nothing to append
    c.append(x, x)                # full: all dropped
    assert c.lengths.tolist() == [50, 50] and torch.equal(_u8(c.k), before)


def test_append_lengths_outside_the_cache_are_clamped():
    gen = torch.Generator().manual_seed(8)
    c = ops.KV8Cache(2, 1, 32, d=64, blk=16)
    x = _values((2, 3, 1, 64), gen, BF16).cuda()
    c.lengths.copy_(torch.tensor([-4, 1000], dtype=torch.int32))
    c.append(x, x, torch.tensor([2, 3], dtype=torch.int32, device="cuda"))
    assert c.lengths.tolist() == [2, 32]
    want = torch.zeros((32, 64), dtype=torch.uint8)
    ref.append(want, torch.zeros(2), x[0, :, 0].cpu(), 0, 2, 16)
    assert torch.equal(_u8(c.k)[0, 0], want)
    assert not _u8(c.k)[1].any()


def _filled(shape, blk, layout, lengths, gen, dtype, offset=3.0):
    """A cache holding random tokens below the lengths and random bytes (NaN
    codes among them) behind; scales behind are NaN."""
    B, Hkv, cap, d = shape
    k, v = _codes(shape, layout, gen)
    ks, vs = (torch.full((B, Hkv, -(-cap // blk)), math.nan, device="cuda") for _ in range(2))
    T = max(max(lengths), 1)
    kn = (torch.randn((B, T, Hkv, d), generator=gen) +
          offset * torch.randn((1, 1, Hkv, d), generator=gen)).to(dtype).cuda()
    vn = torch.randn((B, T, Hkv, d), generator=gen).to(dtype).cuda()
    n = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    ops.thrift_kv8_append(kn, vn, k, v, ks, vs, torch.zeros_like(n), n, blk=blk)
    return k, v, ks, vs, n


def _check_decode(q, cache, lengths, blk, out, lse, scale=None, weight=None, weight0=None):
    B, H, d = q.shape
    k, v, ks, vs = _u8(cache[0]), _u8(cache[1]), cache[2].cpu(), cache[3].cpu()
    Hkv = k.shape[1]
    G = H // Hkv
    q, out, lse = q.cpu(), out.cpu(), lse.cpu()
    eps = torch.finfo(q.dtype).eps / 2
    tiny = torch.finfo(q.dtype).smallest_normal * torch.finfo(q.dtype).eps  # subnormal step
    for b in range(B):
        for h in range(Hkv):
            rows = slice(h * G, (h + 1) * G)
            o, l, p, bo, bl, bp = ref.decode(q[b, rows], k[b, h], v[b, h], ks[b, h], vs[b, h],
                                             lengths[b], blk, d ** -0.5 if scale is None else scale)
            err = (out[b, rows].double() - o).abs()
            assert (err <= eps * o.abs() + bo + tiny).all(), (b, h, float((err - bo).max()))
            if lengths[b] == 0:
                assert (lse[b, rows] == -math.inf).all()
            else:
                assert ((lse[b, rows].double() - l).abs() <= bl).all(), (b, h)
            if weight is not None:
                n = lengths[b]
                w, w0 = weight[b, h].cpu().double(), weight0[b, h].cpu().double()
                bar = bp.sum(0) + 2.0 ** -23 * (w0[:n].abs() + p.sum(0)) * 2
                assert ((w[:n] - w0[:n] - p.sum(0)).abs() <= bar).all(), (b, h)
                assert torch.equal(weight[b, h, n:].cpu(), weight0[b, h, n:].cpu())


DECODES = [
    # shape, H, blk, layout, dtype, lengths
    ((1, 1, 1, 64), 1, 16, "head", BF16, [1]),
    ((3, 1, 130, 128), 1, 128, "head", FP16, [0, 1, 130]),
    ((4, 2, 515, 128), 8, 64, "token", BF16, [127, 128, 129, 515]),
    ((2, 3, 700, 64), 21, 32, "pair", FP16, [700, 385]),
    ((2, 2, 300, 128), 32, 16, "head", BF16, [300, 257]),
    ((1, 1, 640, 64), 24, 64, "token", BF16, [640]),
    ((2, 1, 200, 128), 71, 32, "head", FP16, [200, 1]),
    ((1, 8, 6000, 128), 40, 64, "head", BF16, [5999]),
    ((40, 1, 260, 64), 5, 16, "pair", BF16, list(range(0, 260, 7))[:38] + [260, 259]),
    ((5, 4, 2100, 64), 16, 128, "token", FP16, [2048, 1, 0, 2100, 2049]),
    # more (sequence, kv head) pairs than the machine takes at once
    ((300, 8, 300, 64), 16, 32, "token", BF16, [(37 * i) % 301 for i in range(300)]),
    ((160, 4, 700, 128), 36, 64, "head", FP16, [(97 * i) % 701 for i in range(160)]),
]


@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("case", range(len(DECODES)))
def test_decode(case, accumulate):
    shape, H, blk, layout, dtype, lengths = DECODES[case]
    gen = torch.Generator().manual_seed(200 + case)
    *cache, n = _filled(shape, blk, layout, lengths, gen, dtype)
    q = torch.randn((shape[0], H, shape[3]), generator=gen).to(dtype).cuda()
    weight = torch.rand(shape[:3], generator=gen).cuda()
    w0 = weight.clone()
    out, lse = ops.thrift_kv8_decode(q, *cache, n, blk=blk, weight=weight if accumulate else None)
    _check_decode(q, cache, lengths, blk, out, lse, weight=weight if accumulate else None,
                  weight0=w0)
    if not accumulate:
        assert torch.equal(weight, w0)


@pytest.mark.parametrize("what", ["large", "tiny", "uneven", "zero", "flat", "negative"])
def test_decode_scales_and_magnitudes(what):
    """Queries and caches far from unit size, uneven channels, a scale of the
    caller's own."""
    gen = torch.Generator().manual_seed(300)
    shape, blk, lengths, scale = (2, 2, 300, 128), 32, [300, 131], None
    B, Hkv, cap, d = shape
    k, v = _codes(shape, "head", gen)
    ks, vs = (torch.zeros((B, Hkv, -(-cap // blk)), device="cuda") for _ in range(2))
    kn, vn = (torch.randn((B, cap, Hkv, d), generator=gen) for _ in range(2))
    q = torch.randn((B, 8, d), generator=gen)
    if what == "large":
        q, kn, vn, scale = q * 1e4, kn * 1e4, vn * 1e10, 1e-8 / 11
    elif what == "tiny":
        q, kn, vn, scale = q * 1e-6, kn * 1e-8, vn * 1e-20, 1e14 / 11
    elif what == "uneven":
        q = q * torch.exp(2 * torch.randn(d, generator=gen))
        vn = vn * torch.exp(3 * torch.randn((1, cap, 1, 1), generator=gen))
    elif what == "zero":
        q, vn = q * 0, vn * 0
    elif what == "flat":
        scale = 0.0
    else:
        scale = -0.3
    n = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    ops.thrift_kv8_append(kn.to(BF16).cuda(), vn.to(BF16).cuda(), k, v, ks, vs,
                          torch.zeros_like(n), n, blk=blk)
    q = q.to(BF16).cuda()
    weight = torch.zeros(shape[:3], device="cuda")
    out, lse = ops.thrift_kv8_decode(q, k, v, ks, vs, n, blk=blk, scale=scale, weight=weight)
    _check_decode(q, (k, v, ks, vs), lengths, blk, out, lse, scale, weight,
                  torch.zeros_like(weight))


def test_decode_nan_stays_in_its_rows():
    """A NaN or infinite key, value or query reaches the rows that attend to
    it and no other."""
    gen = torch.Generator().manual_seed(301)
    shape, blk, lengths = (3, 2, 200, 64), 16, [200, 150, 90]
    *cache, n = _filled(shape, blk, "head", lengths, gen, BF16)
    q = torch.randn((3, 8, 64), generator=gen).to(BF16).cuda()
    clean, clean_lse = ops.thrift_kv8_decode(q, *cache, n, blk=blk)
    cache[0].view(torch.uint8)[0, 1, 17, 3] = 0x7F   # a key of sequence 0, kv head 1
    cache[1].view(torch.uint8)[1, 0, 149, 5] = 0xFF  # a value channel of sequence 1, kv head 0
    q[2, 3, 0] = math.inf                            # one query row of sequence 2
    out, lse = ops.thrift_kv8_decode(q, *cache, n, blk=blk)
    nan = torch.zeros_like(out, dtype=torch.bool)
    nan[0, 4:] = True
    nan[1, :4, 5] = True
    nan[2, 3] = True
    assert torch.equal(torch.isnan(out), nan)
    assert torch.equal(out[~nan], clean[~nan])
    rows = nan.all(-1)
    assert torch.isnan(lse[rows]).all() and torch.equal(lse[~rows], clean_lse[~rows])


def test_decode_long_strided_offsets():
    """Code offsets past 2^32 bytes: two sequences far apart in one buffer."""
    gen = torch.Generator().manual_seed(302)
    far = (1 << 32) + 4096
    buf = torch.empty(2 * far, dtype=torch.uint8, device="cuda")
    k = buf.view(F8).as_strided((2, 1, 100, 64), (far, 64 * 100, 64, 1))
    v = buf.view(F8).as_strided((2, 1, 100, 64), (far, 64 * 100, 64, 1), far // 2)
    ks, vs = (torch.zeros((2, 1, 4), device="cuda") for _ in range(2))
    x = torch.randn((2, 100, 1, 64), generator=gen).to(BF16).cuda()
    n = torch.tensor([100, 77], dtype=torch.int32, device="cuda")
    ops.thrift_kv8_append(x, -x, k, v, ks, vs, torch.zeros_like(n), n, blk=32)
    q = torch.randn((2, 4, 64), generator=gen).to(BF16).cuda()
    out, lse = ops.thrift_kv8_decode(q, k, v, ks, vs, n, blk=32)
    _check_decode(q, (k, v, ks, vs), [100, 77], 32, out, lse)


def test_decode_repeats_bit_for_bit_and_across_streams():
    gen = torch.Generator().manual_seed(303)
    shape, blk, lengths = (6, 4, 3000, 128), 64, [3000, 2999, 1, 128, 1500, 700]
    *cache, n = _filled(shape, blk, "token", lengths, gen, BF16)
    q = torch.randn((6, 16, 128), generator=gen).to(BF16).cuda()
    weight = torch.zeros(shape[:3], device="cuda")
    first = ops.thrift_kv8_decode(q, *cache, n, blk=blk, weight=weight)
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in range(3)], []
    for s in streams:  # calls that overlap, each with its stream's workspace
        with torch.cuda.stream(s):
            w = torch.zeros_like(weight)
            got.append(ops.thrift_kv8_decode(q, *cache, n, blk=blk, weight=w) + (w,))
    torch.cuda.synchronize()
    for out, lse, w in got:
        assert torch.equal(out, first[0]) and torch.equal(lse, first[1]) and torch.equal(w, weight)


EVICTS = [
    # shape, blk, layout, lengths, budget, recent, sink, out capacity
    ((1, 1, 1, 64), 16, "head", [1], 1, 0, 0, 1),
    ((3, 2, 300, 128), 64, "token", [300, 100, 0], 100, 10, 4, 120),
    ((2, 3, 257, 64), 16, "pair", [257, 130], 129, 129, 0, 129),
    ((2, 1, 500, 128), 128, "head", [500, 499], 499, 0, 7, 600),
    ((1, 2, 3000, 64), 32, "token", [2999], 1, 0, 0, 33),
    ((1, 1, 5000, 64), 32, "head", [5000], 2500, 100, 4, 2500),
    ((2, 2, 70, 64), 16, "head", [70, 69], 1000, 3, 3, 70),
    # weights shared by a cluster, and more than its registers hold
    ((2, 1, 20000, 64), 32, "token", [20000, 11111], 9000, 64, 4, 9001),
    ((1, 1, 140001, 64), 128, "head", [140001], 70000, 5, 3, 70000),
]


@pytest.mark.parametrize("kind", ["random", "ties", "odd"])
@pytest.mark.parametrize("case", range(len(EVICTS)))
def test_evict(case, kind):
    shape, blk, layout, lengths, budget, recent, sink, cap_o = EVICTS[case]
    B, Hkv, cap, d = shape
    gen = torch.Generator().manual_seed(400 + case)
    *cache, n = _filled(shape, blk, layout, lengths, gen, BF16)
    weight = torch.exp(2 * torch.randn((B, Hkv, cap), generator=gen))
    if kind == "ties":
        weight = torch.round(weight)
    elif kind == "odd":
        pick = torch.randint(0, 6, weight.shape, generator=gen)
        for i, x in enumerate((math.nan, math.inf, -math.inf, 0.0, -0.0)):
            weight[pick == i] = x
    weight = weight.cuda()
    ko, vo = _codes((B, Hkv, cap_o, d), layout, gen)
    kso, vso = (torch.randn((B, Hkv, -(-cap_o // blk)), generator=gen).cuda() for _ in range(2))
    wo = torch.randn((B, Hkv, cap_o), generator=gen).cuda()
    lo = torch.full((B,), -1, dtype=torch.int32, device="cuda")
    want = [_u8(ko).clone(), _u8(vo).clone(), kso.cpu(), vso.cpu(), wo.cpu()]
    src = [_u8(cache[0]), _u8(cache[1]), cache[2].cpu(), cache[3].cpu()]
    before = [t.clone() for t in src]
    ops.thrift_kv8_evict(*cache, weight, n, budget, ko, vo, kso, vso, wo, lo, blk=blk,
                         recent=recent, sink=sink)
    for b in range(B):
        for h in range(Hkv):
            at = ref.keep(weight[b, h].cpu(), lengths[b], budget, sink, recent)
            for c in (0, 1):
                codes, sc = ref.reblock(src[c][b, h], src[2 + c][b, h], at, blk)
                want[c][b, h, :len(at)] = codes
                want[2 + c][b, h, :len(sc)] = sc
            want[4][b, h, :len(at)] = weight[b, h].cpu()[at]
    got = [_u8(ko), _u8(vo), kso.cpu(), vso.cpu(), wo.cpu()]
    for name, g, w in zip(("k", "v", "k_scale", "v_scale", "weight"), got, want):
        same = (g == w) | (torch.isnan(g) & torch.isnan(w)) if g.is_floating_point() else g == w
        assert same.all(), name
    assert lo.tolist() == [min(x, budget) for x in lengths]
    for g, w in zip([_u8(cache[0]), _u8(cache[1]), cache[2].cpu(), cache[3].cpu()], before):
        assert g.numpy().tobytes() == w.numpy().tobytes()  # the input is left alone


def test_evict_of_a_nan_value_keeps_it():
    gen = torch.Generator().manual_seed(450)
    shape = (1, 1, 64, 64)
    *cache, n = _filled(shape, 16, "head", [64], gen, BF16)
    cache[0].view(torch.uint8)[0, 0, 10, 7] = 0xFF
    weight = torch.zeros((1, 1, 64), device="cuda")
    weight[0, 0, 10] = 1.0
    c = ops.KV8Cache(1, 1, 64, d=64, blk=16)
    ops.thrift_kv8_evict(*cache, weight, n, 1, *c.tensors, c.weight, c.lengths, blk=16)
    row = _u8(c.k)[0, 0, 0]
    assert row[7] == 0x7F and (row[:7] & 0x7F != 0x7F).all() and c.lengths.tolist() == [1]


def test_generation_run():
    """The operators as a server uses them: a prompt appended, steps that
    append and attend with accumulated weights, a cut to the budget into a
    spare cache, and steps on the cut one."""
    gen = torch.Generator().manual_seed(500)
    B, Hkv, G, d, blk, cap = 3, 2, 4, 128, 32, 260
    cache, spare = (ops.KV8Cache(B, Hkv, cap, d=d, blk=blk) for _ in range(2))
    host = [[torch.zeros((cap, d), dtype=torch.uint8) for _ in range(2)] for _ in range(B * Hkv)]
    sc = [[torch.zeros(-(-cap // blk)) for _ in range(2)] for _ in range(B * Hkv)]
    w = [torch.zeros(cap, dtype=torch.float64) for _ in range(B * Hkv)]
    at = [0] * B

    def step(T, n, attend):
        kn, vn = (torch.randn((B, T, Hkv, d), generator=gen).to(BF16) for _ in range(2))
        cache.append(kn.cuda(), vn.cuda(), torch.tensor(n, dtype=torch.int32, device="cuda"))
        for b in range(B):
            for h in range(Hkv):
                i = b * Hkv + h
                for x, kv in ((kn, 0), (vn, 1)):
                    end = ref.append(host[i][kv], sc[i][kv], x[b, :, h], at[b], n[b], blk)
                w[i][at[b]:end] = 0.0
            at[b] = end
        if not attend:
            return
        q = torch.randn((B, Hkv * G, d), generator=gen).to(BF16).cuda()
        w0 = cache.weight.clone()
        out, lse = cache.decode(q, accumulate=True)
        _check_decode(q, cache.tensors, at, blk, out, lse, None, cache.weight, w0)
        for i in range(B * Hkv):
            w[i][:at[i // Hkv]] = cache.weight[i // Hkv, i % Hkv, :at[i // Hkv]].cpu().double()

    step(200, [200, 120, 3], False)
    for _ in range(5):
        step(1, [1, 1, 1], True)
    for budget in (100, 64):
        cut = cache.evict(budget, recent=16, sink=4, out=spare)
        assert cut is spare
        for i in range(B * Hkv):
            b, h = divmod(i, Hkv)
            kept = ref.keep(w[i], at[b], budget, 4, 16)
            for kv in (0, 1):
                codes, s = ref.reblock(host[i][kv], sc[i][kv], kept, blk)
                host[i][kv][:len(kept)] = codes
                sc[i][kv][:len(s)] = s
                assert torch.equal(_u8(cut.tensors[kv])[b, h, :len(kept)], codes), (budget, i, kv)
            w[i][:len(kept)] = w[i][kept]
        at[:] = [min(x, budget) for x in at]
        assert cut.lengths.tolist() == at
        cache, spare = cut, cache
        for i in range(4):
            step(1 + i, [1, i, 0], True)
    for i in range(B * Hkv):
        b, h = divmod(i, Hkv)
        for kv in (0, 1):
            assert torch.equal(_u8(cache.tensors[kv])[b, h, :at[b]], host[i][kv][:at[b]])


def test_captured_steps_replay():
    """Append and decode captured twice on one stream (each graph with its own
    scratch), replayed in turn while eager calls run, follow the lengths that
    the device holds."""
    gen = torch.Generator().manual_seed(501)
    B, Hkv, H, d, blk, cap = 2, 2, 8, 64, 16, 400
    caches = [ops.KV8Cache(B, Hkv, cap, d=d, blk=blk) for _ in range(3)]
    prompt = torch.randn((B, 50, Hkv, d), generator=gen).to(BF16).cuda()
    for c in caches:
        c.append(prompt, -prompt)
    x = torch.zeros((B, 1, Hkv, d), dtype=BF16, device="cuda")
    q = torch.zeros((B, H, d), dtype=BF16, device="cuda")
    caches[2].append(x, x)  # the library is warm before the capture
    caches[2].decode(q, accumulate=True)
    caches[2] = ops.KV8Cache(B, Hkv, cap, d=d, blk=blk)
    caches[2].append(prompt, -prompt)
    stream, graphs, outs = torch.cuda.Stream(), [], []
    for c in caches[:2]:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=stream):
            c.append(x, x)
            outs.append(c.decode(q, accumulate=True))
        graphs.append(g)
    for _ in range(20):
        x.copy_(torch.randn(x.shape, generator=gen))
        q.copy_(torch.randn(q.shape, generator=gen))
        for g in graphs:
            g.replay()
        caches[2].append(x, x)
        out, lse = caches[2].decode(q, accumulate=True)
        torch.cuda.synchronize()
        for o, l in outs:
            assert torch.equal(o, out) and torch.equal(l, lse)
    for c in caches[:2]:
        assert c.lengths.tolist() == [70, 70]
        assert torch.equal(c.weight, caches[2].weight)
        assert torch.equal(_u8(c.k), _u8(caches[2].k))
    assert ops.device_status() == ops.OK
