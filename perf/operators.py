"""What the operators of token-by-token generation are measured on.

Four operators that one generation step uses together: the projections by
NVFP4 weights (``linear``), the append to an 8-bit key/value cache
(``append``), the attention of one query token per sequence over that cache
(``decode``), and the eviction of its least attended tokens (``evict``).
``run`` computes each in plain torch, or calls the library where ``own`` is
set; ``exact`` computes it in 64 bits.

The 8-bit cache: E4M3 codes k, v [B, Hkv, capacity, d] and one fp32 scale per
(sequence, head, block of ``blk`` tokens), a power of two: the smallest 2^e,
e >= -120, with max|x| <= 448 * 2^e over the block's finite values.
"""
import math

import torch

own = False

E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ------------------------------------------------------------------- cases --

def listed():
    return [
        # one generated token for each of 64 running sequences, 8 kv heads
        dict(name="append_step_b64", op="append", B=64, Hkv=8, d=128, blk=64, T=1, cap=512, lo=1,
             hi=511, layout="head", dt="bf16"),
        # a prompt of 8000 tokens behind a short cached prefix, token-major cache
        dict(name="append_prompt_8000", op="append", B=1, Hkv=8, d=128, blk=32, T=8000, cap=8192,
             lo=77, hi=77, layout="token", dt="fp16"),
        # one short chat: the launch latency counts
        dict(name="decode_b1_500", op="decode", B=1, H=32, Hkv=8, d=128, blk=64, cap=1024, lo=500,
             hi=500, weight=False, layout="head", dt="bf16"),
        # small heads, an odd group of 7, ragged lengths from one token on
        dict(name="decode_b16_d64_g7", op="decode", B=16, H=14, Hkv=2, d=64, blk=32, cap=12345,
             lo=1, hi=12345, weight=False, layout="token", dt="fp16"),
        # a serving batch that also accumulates the weights that eviction goes by
        dict(name="decode_b32_8k_weight", op="decode", B=32, H=32, Hkv=8, d=128, blk=64, cap=8192,
             lo=4000, hi=8192, weight=True, layout="head", dt="bf16"),
        # the decode workload of the benchmark: four sequences of 131072 tokens
        dict(name="decode_b4_131k", op="decode", B=4, H=32, Hkv=8, d=128, blk=128, cap=131072,
             lo=131072, hi=131072, weight=False, layout="head", dt="bf16"),
        # a running batch falls back to its budget of 4096 tokens
        dict(name="evict_b8_4k", op="evict", B=8, Hkv=8, d=128, blk=64, cap=4352, budget=4096,
             recent=256, sink=4, lo=4200, hi=4352, layout="head"),
        # one long context cut to a quarter
        dict(name="evict_b1_131k", op="evict", B=1, Hkv=8, d=128, blk=32, cap=131072, budget=32768,
             recent=1024, sink=16, lo=130001, hi=130001, layout="head"),
        # key projection of one token
        dict(name="linear_m1_4096x1024", op="linear", M=1, K=4096, N=1024, dt="bf16"),
        # feed-forward projection of one token
        dict(name="linear_m1_4096x14336", op="linear", M=1, K=4096, N=14336, dt="bf16"),
        # feed-forward projection back, a batch of 16 tokens
        dict(name="linear_m16_14336x4096", op="linear", M=16, K=14336, N=4096, dt="bf16"),
        # logits of four tokens over a large vocabulary
        dict(name="linear_m4_4096x128256", op="linear", M=4, K=4096, N=128256, dt="fp16"),
    ]


def _between(rng, lo, hi):
    """An integer of [lo, hi], uniform over the logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("append", "decode", "decode", "evict", "linear", "linear"))
    d, blk = rng.choice((64, 128)), rng.choice((16, 32, 64, 128))
    layout, dt = rng.choice(("head", "token")), rng.choice(("bf16", "fp16"))
    Hkv = rng.choice((1, 2, 3, 4, 5, 8, 8))
    if op == "append":
        T = _between(rng, 1, 8000)
        B = _between(rng, 1, max(1, min(64, 16000 // T)))
        hi = _between(rng, 1, 512)
        cap = hi + T + rng.randrange(0, 64)
        return dict(op=op, B=B, Hkv=Hkv, d=d, blk=blk, T=T, cap=cap, lo=rng.randrange(0, hi + 1),
                    hi=hi, layout=layout, dt=dt)
    if op == "decode":
        B, G = _between(rng, 1, 64), rng.randrange(1, 17)
        hi = _between(rng, 1, min(131072, 4 * 8 * 131072 // (B * Hkv)))
        return dict(op=op, B=B, H=Hkv * G, Hkv=Hkv, d=d, blk=blk, cap=hi + rng.randrange(0, 200),
                    lo=rng.randrange(0, hi + 1), hi=hi, weight=rng.random() < 0.5, layout=layout,
                    dt=dt)
    if op == "evict":
        B = _between(rng, 1, 16)
        hi = _between(rng, 64, min(131072, 8 * 131072 // (B * Hkv)))
        budget = rng.randrange(16, hi + 1)
        recent = rng.randrange(0, budget // 2 + 1)
        return dict(op=op, B=B, Hkv=Hkv, d=d, blk=blk, cap=hi + rng.randrange(0, 100),
                    budget=budget, recent=recent, sink=rng.randrange(0, min(16, budget - recent) + 1),
                    lo=rng.randrange(0, hi + 1), hi=hi, layout=layout)
    M, K = _between(rng, 1, 16), 32 * _between(rng, 2, 512)
    return dict(op=op, M=M, K=K, N=_between(rng, 1, min(131072, 4096 * 128256 // K)), dt=dt)


def _lengths(case):
    """The batch's lengths, spread evenly over [lo, hi]; the seed only orders them."""
    B, lo, hi = case["B"], case["lo"], case["hi"]
    return [hi - (hi - lo) * i // max(1, B - 1) for i in range(B)] if B > 1 else [hi]


def _news(case):
    """Tokens appended to each sequence: the whole step, or ragged pieces of it."""
    return [case["T"] - (case["T"] * (i % 4)) // 5 for i in range(case["B"])]


# ------------------------------------------------------------------ inputs --

def _dtype(case):
    return torch.bfloat16 if case["dt"] == "bf16" else torch.float16


def _pow2_scale(amax):
    """Smallest 2^e, e >= -120, with amax <= 448 * 2^e = 1.75 * 2^(e + 8)."""
    m, x = torch.frexp(amax)  # amax = m * 2^x, 0.5 <= m < 1
    e = x - 9 + (m > 0.875).to(x.dtype)
    e = torch.where(amax > 0, e, torch.full_like(e, -120)).clamp(min=-120)
    return torch.ldexp(torch.ones_like(amax), e)


def _encode(x, scale):
    """E4M3 codes of x / scale, round to nearest even; what is not finite becomes NaN."""
    y = torch.where(torch.isfinite(x), x / scale, torch.full_like(x, math.nan))
    return y.to(torch.float8_e4m3fn)


def _blocks(x, blk):
    """[B, Hkv, T, d] -> [B, Hkv, nblk, blk, d], zero-padded."""
    n = -(-x.shape[2] // blk)
    x = torch.nn.functional.pad(x, (0, 0, 0, n * blk - x.shape[2]))
    return x.unflatten(2, (n, blk))


def _amax(x):
    return torch.where(torch.isfinite(x), x, torch.zeros_like(x)).abs().amax(dim=(-1, -2))


def _cache(shape, layout, blk, gen):
    """A filled cache: codes [B, Hkv, cap, d] in the given memory order, and
    scales.  Keys carry channel offsets as in trained models."""
    B, Hkv, cap, d = shape
    got = []
    for offset in (3.0, 0.0):
        x = torch.randn(shape, generator=gen, device="cuda")
        x += offset * torch.randn((1, Hkv, 1, d), generator=gen, device="cuda")
        x = _blocks(x, blk)
        scale = _pow2_scale(_amax(x))
        codes = _encode(x, scale[..., None, None]).flatten(2, 3)[:, :, :cap]
        if layout == "token":
            codes = codes.transpose(1, 2).contiguous().transpose(1, 2)
        else:
            codes = codes.contiguous()
        got += [codes, scale]
    return got


def _empty_cache(shape, layout, blk):
    B, Hkv, cap, d = shape
    got = []
    for _ in range(2):
        codes = torch.zeros((B, cap, Hkv, d) if layout == "token" else shape, dtype=torch.uint8,
                            device="cuda").view(torch.float8_e4m3fn)
        got += [codes.transpose(1, 2) if layout == "token" else codes,
                torch.zeros((B, Hkv, -(-cap // blk)), device="cuda")]
    return got


def _int32(values, order):
    return torch.tensor([values[i] for i in order], dtype=torch.int32, device="cuda")


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    if case["op"] == "linear":
        M, K, N = case["M"], case["K"], case["N"]
        x = torch.randn((M, K), generator=gen, device="cuda")
        x *= torch.exp(torch.randn((1, K), generator=gen, device="cuda"))  # uneven channels
        w = torch.randn((N, K // 16, 16), generator=gen, device="cuda")
        g = w.abs().amax() / 2688.0
        s = (w.abs().amax(-1) / (6.0 * g)).to(torch.float8_e4m3fn)
        w /= (s.float() * g)[..., None]
        edges = torch.tensor([(a + b) / 2 for a, b in zip(E2M1, E2M1[1:])], device="cuda")
        mag = torch.bucketize(w.abs(), edges, out_int32=True).to(torch.uint8)
        code = (mag | ((w < 0).to(torch.uint8) << 3)).reshape(N, K // 2, 2)
        codes = code[..., 0] | (code[..., 1] << 4)
        del w, mag, code
        return dict(case=case, x=x.to(_dtype(case)), codes=codes.contiguous(),
                    scales=s.view(torch.uint8), g=g.reshape(1))
    B, Hkv, cap, d, blk = (case[n] for n in ("B", "Hkv", "cap", "d", "blk"))
    order = torch.randperm(B, generator=torch.Generator().manual_seed(seed)).tolist()
    lengths = _int32(_lengths(case), order)
    k, ks, v, vs = _cache((B, Hkv, cap, d), case["layout"], blk, gen)
    st = dict(case=case, k=k, v=v, k_scale=ks, v_scale=vs, lengths=lengths)
    if case["op"] == "append":
        T = case["T"]
        kn = torch.randn((B, T, Hkv, d), generator=gen, device="cuda")
        kn += 3.0 * torch.randn((1, 1, Hkv, d), generator=gen, device="cuda")
        vn = torch.randn((B, T, Hkv, d), generator=gen, device="cuda")
        return dict(st, k_new=kn.to(_dtype(case)), v_new=vn.to(_dtype(case)),
                    n_new=_int32(_news(case), order),
                    new_len=torch.zeros(B, dtype=torch.int32, device="cuda"))
    weight = torch.exp(2.0 * torch.randn((B, Hkv, cap), generator=gen, device="cuda"))
    weight[torch.rand((B, Hkv, cap), generator=gen, device="cuda") < 0.1] = 0.0
    st["weight"] = weight
    if case["op"] == "decode":
        st["q"] = torch.randn((B, case["H"], d), generator=gen, device="cuda").to(_dtype(case))
        return st
    out_cap = case["budget"] + 13
    ko, kso, vo, vso = _empty_cache((B, Hkv, out_cap, d), case["layout"], blk)
    return dict(st, k_out=ko, v_out=vo, k_scale_out=kso, v_scale_out=vso,
                weight_out=torch.zeros((B, Hkv, out_cap), device="cuda"),
                len_out=torch.zeros(B, dtype=torch.int32, device="cuda"))


# ------------------------------------------------------------- plain forms --

def _append_one(codes, scales, new, lengths, n_new, blk):
    """Writes the new tokens of one cache tensor ([B, Hkv, cap, d])."""
    B, Hkv, cap, d = codes.shape
    T = new.shape[1]
    nb = (T + blk - 2) // blk + 1  # blocks that T tokens can touch
    row = torch.arange(nb * blk, device="cuda")
    base = lengths.long() // blk * blk
    pos = base[:, None] + row  # [B, R]
    end = torch.clamp(lengths.long() + n_new, max=cap)
    is_new = ((pos >= lengths[:, None]) & (pos < end[:, None]))[:, None, :, None]
    is_old = (pos < lengths[:, None])[:, None, :, None]
    at = torch.clamp(pos - lengths[:, None], 0, T - 1)
    x = torch.gather(new.float(), 1, at[:, :, None, None].expand(-1, -1, Hkv, d)).transpose(1, 2)
    x = torch.where(is_new, x, torch.zeros_like(x))
    rows = torch.clamp(pos, max=cap - 1)[:, None, :, None].expand(-1, Hkv, -1, d)
    old = torch.gather(codes.view(torch.uint8), 2, rows).view(torch.float8_e4m3fn).float()
    blocks = torch.clamp(base[:, None] // blk + torch.arange(nb, device="cuda"),
                         max=scales.shape[2] - 1)[:, None].expand(-1, Hkv, -1)
    had = torch.gather(scales, 2, blocks)
    has_old = is_old.unflatten(2, (nb, blk)).any(dim=(-1, -2))
    touched = is_new.unflatten(2, (nb, blk)).any(dim=(-1, -2))
    now = _pow2_scale(_amax(x.unflatten(2, (nb, blk))))
    now = torch.where(has_old, torch.maximum(now, had), now)
    per_row = now.repeat_interleave(blk, dim=2)[..., None]
    ratio = (had / now).repeat_interleave(blk, dim=2)[..., None]
    val = torch.where(is_new, _encode(x, per_row).float(), _encode(old * ratio, 1.0).float())
    write = ((is_new | is_old) & touched.repeat_interleave(blk, dim=2)[..., None])
    b, h, r, _ = write.expand(-1, Hkv, -1, 1).nonzero(as_tuple=True)
    codes.view(torch.uint8)[b, h, pos[b, r]] = val[b, h, r].to(torch.float8_e4m3fn).view(torch.uint8)
    b, h, j = touched.expand(-1, Hkv, -1).nonzero(as_tuple=True)
    scales[b, h, base[b] // blk + j] = now[b, h, j]


def _values(codes, scales, blk):
    """What the codes of a cache stand for, fp32 [B, Hkv, cap, d]."""
    s = scales.repeat_interleave(blk, dim=2)[:, :, :codes.shape[2], None]
    return codes.float() * s


def _decode(st):
    c, q, blk = st["case"], st["q"], st["case"]["blk"]
    B, H, d = q.shape
    Hkv, cap = c["Hkv"], c["cap"]
    live = torch.arange(cap, device="cuda") < st["lengths"][:, None]
    s = q.float().reshape(B, Hkv, H // Hkv, d) @ _values(st["k"], st["k_scale"], blk).mT
    s = torch.where(live[:, None, None], s / math.sqrt(d), torch.full_like(s, -math.inf))
    m = s.amax(-1, keepdim=True)
    p = torch.where(live[:, None, None], torch.exp(s - m), torch.zeros_like(s))
    l = p.sum(-1, keepdim=True)
    p = torch.where(l > 0, p / l, torch.zeros_like(p))
    v = _values(st["v"], st["v_scale"], blk)
    o = p @ torch.where(live[:, None, :, None], v, torch.zeros_like(v))
    lse = (m + torch.log(l)).reshape(B, H)
    lse = torch.where((st["lengths"] > 0)[:, None], lse, torch.full_like(lse, -math.inf))
    out = o.reshape(B, H, d).to(q.dtype)
    if not c["weight"]:
        return out, lse
    st["weight"].add_(p.sum(2))
    return out, lse, st["weight"]


def _evict(st):
    c, w, L = st["case"], st["weight"], st["lengths"].long()[:, None, None]
    blk, budget = c["blk"], c["budget"]
    t = torch.arange(c["cap"], device="cuda")
    key = torch.where(torch.isnan(w), torch.full_like(w, -math.inf), w)
    key = torch.where((t < c["sink"]) | (t >= L - c["recent"]), torch.full_like(w, math.inf), key)
    key = torch.where(t < L, key, torch.full_like(w, -math.inf))
    n = min(budget, c["cap"])
    kept = torch.sort(key, dim=-1, descending=True, stable=True)[1][..., :n].sort(dim=-1)[0]
    live = (torch.arange(n, device="cuda") < L)[..., None]
    for name in ("k", "v"):
        x = _values(st[name], st[name + "_scale"], blk)
        x = torch.gather(x, 2, kept[..., None].expand(-1, -1, -1, c["d"]))
        x = _blocks(torch.where(live, x, torch.zeros_like(x)), blk)
        s = _pow2_scale(_amax(x))
        x = _encode(x, s[..., None, None]).flatten(2, 3)[:, :, :n].view(torch.uint8)
        to, so = st[name + "_out"][:, :, :n].view(torch.uint8), st[name + "_scale_out"]
        to.copy_(torch.where(live, x, to))
        has = torch.arange(s.shape[2], device="cuda") * blk < L
        so[:, :, :s.shape[2]] = torch.where(has, s, so[:, :, :s.shape[2]])
    wo = st["weight_out"][:, :, :n]
    wo.copy_(torch.where(live[..., 0], torch.gather(w, 2, kept), wo))
    st["len_out"].copy_(torch.clamp(st["lengths"], max=budget))


def _linear(st):
    x = st["x"]
    pair = torch.tensor([[(1 - 2 * (c >> 3 & 1)) * E2M1[c & 7] for c in (b & 15, b >> 4)]
                         for b in range(256)], device="cuda")
    w = pair[st["codes"].int()].flatten(1).unflatten(1, (-1, 16))
    w = w * (st["scales"].view(torch.float8_e4m3fn).float() * st["g"])[..., None]
    return (x.float() @ w.flatten(1).T).to(x.dtype)


def run(state):
    c = state["case"]
    if own:
        return _run_own(state)
    if c["op"] == "linear":
        return _linear(state)
    if c["op"] == "decode":
        return _decode(state)
    if c["op"] == "append":
        for name in ("k", "v"):
            _append_one(state[name], state[name + "_scale"], state[name + "_new"],
                        state["lengths"], state["n_new"], c["blk"])
        state["new_len"].copy_(torch.clamp(state["lengths"] + state["n_new"], max=c["cap"]))
        return tuple(state[n] for n in ("k", "v", "k_scale", "v_scale", "new_len"))
    _evict(state)
    return tuple(state[n] for n in ("k_out", "v_out", "k_scale_out", "v_scale_out", "weight_out",
                                    "len_out"))


def _run_own(st):
    from bit_quantization_b200 import ops

    c = st["case"]
    if c["op"] == "linear":
        return ops.nvfp4_linear(st["x"], st["codes"], st["scales"], st["g"])
    cache = (st["k"], st["v"], st["k_scale"], st["v_scale"])
    if c["op"] == "decode":
        weight = st["weight"] if c["weight"] else None
        out, lse = ops.thrift_kv8_decode(st["q"], *cache, st["lengths"], blk=c["blk"],
                                         weight=weight)
        return (out, lse, weight) if c["weight"] else (out, lse)
    if c["op"] == "append":
        ops.thrift_kv8_append(st["k_new"], st["v_new"], *cache, st["lengths"], st["n_new"],
                              blk=c["blk"], new_len=st["new_len"])
        return (*cache, st["new_len"])
    outs = tuple(st[n] for n in ("k_out", "v_out", "k_scale_out", "v_scale_out", "weight_out",
                                 "len_out"))
    ops.thrift_kv8_evict(*cache, st["weight"], st["lengths"], c["budget"], *outs, blk=c["blk"],
                         recent=c["recent"], sink=c["sink"])
    return outs


# -------------------------------------------------------------------- work --

def work(case):
    if case["op"] == "linear":
        M, K, N = case["M"], case["K"], case["N"]
        return dict(bytes=N * K // 2 + N * K // 16 + 2 * M * (K + N), flops=2 * M * K * N)
    Hkv, d, blk = case["Hkv"], case["d"], case["blk"]
    if case["op"] == "append":
        # 16-bit rows in, 8-bit rows out
        n = sum(_news(case))
        return dict(bytes=n * Hkv * 2 * (2 * d + d), flops=n * Hkv * 2 * d)
    lens = _lengths(case)
    scales = sum(-(-x // blk) for x in lens) * 8 * Hkv
    if case["op"] == "decode":
        n = sum(lens) * Hkv
        G = case["H"] // Hkv
        io = case["B"] * case["H"] * (4 * d + 4)
        return dict(bytes=n * (2 * d + (8 if case["weight"] else 0)) + scales + io,
                    flops=4 * n * G * d)
    kept = sum(min(x, case["budget"]) for x in lens) * Hkv
    return dict(bytes=sum(lens) * Hkv * 4 + kept * (4 * d + 4) + 2 * scales, flops=kept * 2 * d)


# ------------------------------------------------------------------- exact --

def _scale64(amax):
    e = max(-120, math.ceil(math.log2(amax / 448.0))) if amax > 0 else -120
    e += amax > math.ldexp(448.0, e)
    if e > -120 and amax <= math.ldexp(448.0, e - 1):
        e -= 1
    return math.ldexp(1.0, e)


def _e4m3_64(x):
    """x rounded to E4M3 (to nearest even, |x| <= 448) as fp64 values, by its
    spacing: 2^(floor(log2|x|) - 3), 2^-9 at the least."""
    _, e = torch.frexp(x)
    step = torch.ldexp(torch.ones_like(x), torch.clamp(e - 4, min=-9))
    return torch.round(x / step) * step


def _exact_decode(case, st):
    B, H, d = st["q"].shape
    Hkv, blk = case["Hkv"], case["blk"]
    G = H // Hkv
    out = torch.zeros((B, H, d), dtype=torch.float64, device="cuda")
    lse = torch.full((B, H), -math.inf, dtype=torch.float64, device="cuda")
    weight = st["weight"].double()
    for b, n in enumerate(st["lengths"].tolist()):
        block = torch.arange(n, device="cuda") // blk
        for h in range(Hkv):
            if n == 0:
                continue
            k = st["k"][b, h, :n].double() * st["k_scale"][b, h, block].double()[:, None]
            v = st["v"][b, h, :n].double() * st["v_scale"][b, h, block].double()[:, None]
            s = (st["q"][b, h * G:(h + 1) * G].double() @ k.T) * d ** -0.5
            lse[b, h * G:(h + 1) * G] = torch.logsumexp(s, 1)
            p = torch.softmax(s, 1)
            out[b, h * G:(h + 1) * G] = p @ v
            weight[b, h, :n] += p.sum(0)
    return (out, lse, weight) if case["weight"] else (out, lse)


def _exact_linear(case, st):
    M, K, N = case["M"], case["K"], case["N"]
    x = st["x"].double()
    out = torch.empty((M, N), dtype=torch.float64, device="cuda")
    grid = torch.tensor([(-1.0) ** (c >> 3) * E2M1[c & 7] for c in range(16)],
                        dtype=torch.float64, device="cuda")
    for n in range(0, N, 8192):
        c = st["codes"][n:n + 8192].long()
        w = torch.stack((grid[c & 15], grid[c >> 4]), -1).reshape(len(c), K)
        s = st["scales"][n:n + 8192].long()
        e, f = s >> 3, (s & 7).double()
        s = torch.where(e > 0, (8 + f) * torch.exp2(e.double() - 10), f * 2.0 ** -9)
        w *= s.repeat_interleave(16, 1)
        out[:, n:n + 8192] = (x @ w.T) * st["g"].double()
    return out


def _exact_blocks(x, blk):
    """Codes' values and scales of the tokens x [n, d] (fp64, finite) of one head."""
    val = torch.empty_like(x)
    tops = torch.stack([x[i:i + blk].abs().max() for i in range(0, len(x), blk)]).tolist()
    scales = [_scale64(a) for a in tops]
    for j, s in enumerate(scales):
        val[j * blk:(j + 1) * blk] = _e4m3_64(x[j * blk:(j + 1) * blk] / s)
    return val, torch.tensor(scales, dtype=torch.float64, device="cuda")


def _exact_append(case, st):
    blk, cap, got = case["blk"], case["cap"], []
    ends = [min(cap, a + b) for a, b in zip(st["lengths"].tolist(), st["n_new"].tolist())]
    for name in ("k", "v"):
        codes, scales = st[name].double(), st[name + "_scale"].double()
        for b, end in enumerate(ends):
            at = int(st["lengths"][b])
            j0 = at // blk
            for h in range(case["Hkv"] if end > at else 0):
                new = st[name + "_new"][b, :end - at, h].double()
                first = min(end, (j0 + 1) * blk) - at  # tokens that join the open block
                top = _scale64(float(new[:first].abs().max()))
                if at > j0 * blk:
                    was = float(scales[b, h, j0])
                    top = max(top, was)
                    codes[b, h, j0 * blk:at] = _e4m3_64(codes[b, h, j0 * blk:at] * (was / top))
                scales[b, h, j0] = top
                codes[b, h, at:at + first] = _e4m3_64(new[:first] / top)
                if first < end - at:
                    val, s = _exact_blocks(new[first:], blk)
                    codes[b, h, at + first:end] = val
                    scales[b, h, j0 + 1:j0 + 1 + len(s)] = s
        got += [codes, scales]
    return got[0], got[2], got[1], got[3], torch.tensor(ends, dtype=torch.int32, device="cuda")


def _exact_evict(case, st):
    blk = case["blk"]
    outs = {n: st[n].double() for n in ("k_out", "v_out", "k_scale_out", "v_scale_out",
                                        "weight_out")}
    lens = st["lengths"].tolist()
    for b, n in enumerate(lens):
        for h in range(case["Hkv"] if n else 0):
            w = st["weight"][b, h, :n].double().cpu()
            keep = torch.ones(n, dtype=torch.bool)
            if n > case["budget"]:
                keep[case["sink"]:n - case["recent"]] = False
                rank = sorted(range(case["sink"], n - case["recent"]), key=(-w).tolist().__getitem__)
                keep[rank[:case["budget"] - case["sink"] - case["recent"]]] = True
            at = keep.nonzero()[:, 0].cuda()
            for name in ("k", "v"):
                s = st[name + "_scale"][b, h, at // blk].double()
                val, scale = _exact_blocks(st[name][b, h, at].double() * s[:, None], blk)
                outs[name + "_out"][b, h, :len(at)] = val
                outs[name + "_scale_out"][b, h, :len(scale)] = scale
            outs["weight_out"][b, h, :len(at)] = st["weight"][b, h, at].double()
    return (*(outs[n] for n in ("k_out", "v_out", "k_scale_out", "v_scale_out", "weight_out")),
            torch.tensor([min(n, case["budget"]) for n in lens], dtype=torch.int32, device="cuda"))


def exact(case, seed):
    st = prepare(case, seed)
    return {"append": _exact_append, "decode": _exact_decode, "evict": _exact_evict,
            "linear": _exact_linear}[case["op"]](case, st)
