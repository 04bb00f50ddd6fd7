"""Bars for the 8-bit cache's attention and the NVFP4 linear layer that follow
the kernels' arithmetic term by term, so that a lost token, chunk or partial
sum is over them; 64-bit forms on any device.

Both kernels sum in fp32 on the tensor cores.  What one instruction with n
products may be off is bounded by n + 1 addends, each cut at 2^-23 of the
largest magnitude at hand (rounded or truncated)."""
import torch

from kv8_ref import E2M1, value

ULP = 2.0 ** -23
SMS = 148


def attention_steps(n, pairs, d):
    """Instructions of 16 tokens that follow one another in one warp, at most:
    its share of the units of `pairs` sequences and heads of n tokens over two
    CTAs an SM, or an eighth of one sequence in one launch."""
    tokens = 4096 // d  # of a warp in a step
    units = pairs * (-(-n // (4 * tokens)) + 1)
    return tokens // 16 * max(-(-units // (2 * SMS)) + 1, -(-n // (8 * tokens)))


def attention(q, codes_k, codes_v, ks, vs, n, blk, scale, pairs):
    """One sequence and kv head: q [G, d]; out [G, d], lse [G], probabilities
    [G, n] in 64 bits, and bars for the three (n > 0), before the rounding to
    the output's type."""
    G, d = q.shape
    block = torch.arange(n, device=q.device) // blk
    k = value(codes_k[:n]) * ks[block].to(torch.float64)[:, None]
    v = value(codes_v[:n]) * vs[block].to(torch.float64)[:, None]
    q = q.to(torch.float64)
    s = (q @ k.T) * scale
    lse, p = torch.logsumexp(s, 1), torch.softmax(s, 1)
    # a score: d / 16 instructions of 16 products; q within 2^-39 of its row's
    # largest value; four roundings of the factor and the product
    ds = abs(scale) * (17 * d / 16 * ULP * (q.abs() @ k.abs().T) +
                       2.0 ** -39 * q.abs().amax(1, keepdim=True) * k.abs().sum(1)[None]) + \
        4 * 2.0 ** -24 * s.abs() + 2.0 ** -22
    shift = ds + (p * ds).sum(1, keepdim=True)  # of a probability's exponent
    steps = attention_steps(n, pairs, d)
    join = 64 * ULP + steps * ULP  # rescaling in the loop, and the parts' joins
    # a probability enters the product with V as fp16 in (0, 2^15]: half a step
    # is 2^-11 of it, or 2^-25 in those units
    rel = 1.01 * shift + 2.0 ** -11 + 17 * steps * ULP + join
    bar_o = (p * rel) @ v.abs() + 2.0 ** -40 * p.amax(1, keepdim=True) * v.abs().sum(0)[None]
    bar_l = 1.01 * (p * ds).sum(1) + join + 2.0 ** -22 * (lse.abs() + 1)
    return p @ v, lse, p, bar_o, bar_l, p * (1.01 * shift + join)


# ----------------------------------------------------------------- linear --

def e2m1(x):
    """Nearest E2M1 value of |x| <= 5."""
    grid = E2M1.to(x.device)
    edges = (grid[1:] + grid[:-1]) / 2
    return grid[torch.bucketize(x.abs(), edges)] * torch.sign(x)


def digits(x, count=6):
    """x [M, K] -> [count, M, K] whose sum is x but for the residual: base-8
    digits in E2M1 under a power of two per 16 elements."""
    b = x.unflatten(1, (-1, 16))
    top = b.abs().amax(-1, keepdim=True)
    row = x.abs().amax(1)[:, None, None]
    s = torch.exp2(torch.floor(torch.log2(torch.where(top > 0, top, torch.ones_like(top)))) - 1)
    low = torch.exp2(torch.floor(torch.log2(torch.where(row > 0, row, torch.ones_like(row)))) - 18)
    s = torch.maximum(s, low)  # the scale's range: 2^-18 of the row's largest
    r, out = b / s, []
    for i in range(count):
        d = e2m1(r)
        out.append((d * s * 8.0 ** -i).flatten(1))
        r = (r - d) * 8
    return torch.stack(out)


def linear(x, w, drop=None):
    """y [M, N] and its bar before the last rounding; `drop` columns [a, b)
    are left out of y."""
    K = x.shape[1]
    dig = digits(x)
    bar = (x - dig.sum(0)).abs() @ w.abs().T
    pad = -K % 64
    dig = torch.nn.functional.pad(dig, (0, pad)).unflatten(2, (-1, 64))
    wg = torch.nn.functional.pad(w, (0, pad)).unflatten(1, (-1, 64))
    for d in dig:
        part = torch.einsum("mgk,ngk->gmn", d, wg)
        # any stretch of columns sums to the difference of two of these
        top = 2 * part.cumsum(0).abs().amax(0)
        largest = d.abs().amax((1, 2))[:, None] * w.abs().amax(1)[None]
        bar += (wg.shape[1] * 65 + SMS + 8) * ULP * (top + largest)
    if drop:
        x = x.clone()
        x[:, drop[0]:drop[1]] = 0
    y = x @ w.T
    return y, bar
