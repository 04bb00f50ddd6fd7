"""Plain 64-bit forms of the 8-bit cache and of the NVFP4 linear layer, and
the error bars their kernels are held to."""
import math

import torch

E2M1 = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64)
F8 = torch.float8_e4m3fn


def scale_of(x):
    """The smallest 2^e, e >= -120, with max|x| <= 448 * 2^e over the finite x."""
    x = x[torch.isfinite(x)].abs()
    a = float(x.max()) if x.numel() else 0.0
    e = -120
    if a > 0:
        e = max(-120, math.frexp(a)[1] - 10)
        while math.ldexp(448.0, e) < a:
            e += 1
    return math.ldexp(1.0, e)


def e4m3(x):
    """E4M3 bytes of fp64 values of at most 448, to nearest even, by the
    format's spacing; what is not finite becomes NaN (0x7F)."""
    bad = ~torch.isfinite(x)
    x = torch.where(bad, torch.zeros_like(x), x)
    _, e = torch.frexp(x)
    step = torch.ldexp(torch.ones_like(x), torch.clamp(e - 4, min=-9))
    code = (torch.round(x / step) * step).to(torch.float32).to(F8).view(torch.uint8)  # exact
    return torch.where(bad, torch.full_like(code, 0x7F), code)


def value(code):
    return code.view(F8).to(torch.float64)


def append(codes, scales, new, length, n, blk):
    """codes u8 [cap, d], scales f32 [nblk] of one (sequence, head), in place."""
    cap = codes.shape[0]
    length = min(cap, max(0, length))
    end = min(cap, length + n)
    for j in range(length // blk, -(-end // blk) if end > length else 0):
        a, b = max(length, j * blk), min(end, (j + 1) * blk)
        x = new[a - length:b - length].to(torch.float64)
        s = scale_of(x)
        if a > j * blk:
            was = float(scales[j])
            s = max(s, was)
            if s != was:
                codes[j * blk:a] = e4m3(value(codes[j * blk:a]) * (was / s))
        codes[a:b] = e4m3(x / s)
        scales[j] = s
    return end


def decode(q, codes_k, codes_v, ks, vs, n, blk, scale):
    """One sequence and kv head: q [G, d]; returns out [G, d], lse [G], the
    probabilities [G, n], and bars for the three."""
    G, d = q.shape
    if n == 0:
        z = torch.zeros((G, d), dtype=torch.float64)
        return z, torch.full((G,), -math.inf, dtype=torch.float64), z[:, :0], z, z[:, 0], z[:, :0]
    block = torch.arange(n) // blk
    k = value(codes_k[:n]) * ks[block].to(torch.float64)[:, None]
    v = value(codes_v[:n]) * vs[block].to(torch.float64)[:, None]
    q = q.to(torch.float64)
    s = (q @ k.T) * scale
    lse, p = torch.logsumexp(s, 1), torch.softmax(s, 1)
    # A score: fp32 accumulation of d products (at most one ulp an addition,
    # truncating allowed), q held to 2^-20 of its row's largest, and the
    # exponent's argument rounded at its own size.
    ds = abs(scale) * (2 * d * 2.0 ** -23 * (q.abs() @ k.abs().T) +
                       2.0 ** -20 * q.abs().amax(1, keepdim=True) * k.abs().sum(1)[None])
    ds = ds.amax(1, keepdim=True) + 2.0 ** -22 * (s.abs().amax(1, keepdim=True) + 1)
    # A probability that enters the product with V carries 12 bits, and 2^-18
    # of the row's largest one at the least; fp32 sums below that.
    vmax = v.abs().amax(0)[None]
    bar_o = vmax * (2 * ds + 2.0 ** -11 + 2.0 ** -20 * math.sqrt(n)) + \
        2.0 ** -18 * p.amax(1, keepdim=True) * v.abs().sum(0)[None]
    # lse and weights come from unrounded fp32 probabilities.
    bar_l = ds[:, 0] + 2.0 ** -21 * (lse.abs() + 4)
    bar_p = p * (2 * ds + 2.0 ** -20)
    return p @ v, lse, p, bar_o, bar_l, bar_p


def keep(w, n, budget, sink, recent):
    """Indices of the tokens that stay, ascending."""
    if n <= budget:
        return list(range(n))
    key = [-math.inf if math.isnan(x) else x for x in w[:n].tolist()]
    middle = sorted(range(sink, n - recent), key=lambda t: (-key[t], t))
    return sorted(list(range(sink)) + middle[:budget - sink - recent] + list(range(n - recent, n)))


def reblock(codes, scales, at, blk):
    """Codes and scales of the tokens `at` of one (sequence, head), as a cache
    of their own; their fp32 values are what is encoded."""
    at = torch.tensor(at, dtype=torch.int64)
    x = (codes[at].view(F8).float() * scales[at // blk][:, None]).to(torch.float64)
    out, sc = torch.zeros_like(codes[at]), []
    for j in range(0, len(at), blk):
        s = scale_of(x[j:j + blk])
        sc.append(s)
        out[j:j + blk] = e4m3(x[j:j + blk] / s)
    return out, torch.tensor(sc)


def dequant(codes, scales, g):
    """NVFP4 weights [N, K] in fp64."""
    c = torch.stack((codes & 15, codes >> 4), -1).reshape(codes.shape[0], -1).long()
    w = E2M1[c & 7] * (1 - 2 * (c >> 3)).to(torch.float64)
    return w * value(scales).repeat_interleave(16, 1) * float(g)


def linear_bar(x, w):
    """What a product may be off before its last rounding: x held to 2^-16 of
    its 16-block's largest value and 2^-33 of its row's, fp32 accumulation
    (at most one ulp an addition, truncating allowed)."""
    M, K = x.shape
    a = x.abs().unflatten(1, (-1, 16)).amax(-1).repeat_interleave(16, 1)
    a = 2.0 ** -16 * a + 2.0 ** -33 * x.abs().amax(1, keepdim=True)
    return a @ w.abs().T + 2 * K * 2.0 ** -23 * (x.abs() @ w.abs().T)
