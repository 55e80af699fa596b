"""Plain 64-bit forms of the head norm and rotation, and the paged-cache layouts of the tests."""
import torch


def f64(x):
    return x.detach().double().cpu()


def norm(x, g, eps):
    """RMS norm of the last dim; x and the weight in 64 bits."""
    return x if g is None else x / torch.sqrt(x.pow(2).mean(-1, keepdim=True) + eps) * g


def rotate(x, pos, inv_freq, interleaved, sign=1.0):
    """Pair rotation of the first 2 * len(inv_freq) dims of x [T, H, d] by sign * pos * inv_freq."""
    if inv_freq is None:
        return x
    n = inv_freq.numel()
    a = sign * pos.double()[:, None, None] * inv_freq
    c, s = torch.cos(a), torch.sin(a)
    u, v = (x[..., 0:2 * n:2], x[..., 1:2 * n:2]) if interleaved else (x[..., :n], x[..., n:2 * n])
    p, q = u * c - v * s, u * s + v * c
    y = torch.stack([p, q], -1).flatten(-2) if interleaved else torch.cat([p, q], -1)
    return torch.cat([y, x[..., 2 * n:]], -1)


def norm_rope(x, g, eps, pos, inv_freq, interleaved):
    return rotate(norm(x, g, eps), pos, inv_freq, interleaved)


def norm_rope_tolerance(x, g, eps, y):
    """How far a bf16 output may be from the 64-bit one.

    The output's rounding is at most 2^-8 |y| (half a bf16 step).  Before it, in fp32: the sum of
    128 squares, in chains of 16 joined by 3, is off by (16 + 3) 2^-24 relative, half of which
    enters the root; rsqrtf by 2^-22; two products and the pair's two by 2^-24 each: below 1.1e-6 of
    |n|.  cos and sin: the angle, at most pi / 4 after its quarter turns, is off by 2^-23 of itself,
    9.4e-8 rad; the polynomials' remainders are below 3e-8 and their last roundings 2^-23.  Over
    both members of a pair that is 1.4e-6 (|u| + |v|), at most 3e-6 times the row's largest |n|."""
    return 2.0 ** -8 * y.abs() + 3e-6 * norm(x, g, eps).abs().amax(-1, keepdim=True)


def frequencies(rotary, base=10000.0):
    return base ** (-torch.arange(0, rotary, 2, dtype=torch.float64) / rotary)


def page_table(lens, page, pool, gen, width=None):
    """int32 [B, width] over a shuffled pool of `pool` pages, -1 in the unused entries."""
    need = [(max(n, 0) + page - 1) // page for n in lens]
    assert sum(need) <= pool
    perm = torch.randperm(pool, generator=gen)
    table = torch.full((len(lens), max(max(need), 1) if width is None else width), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = perm[at:at + n].to(torch.int32)
        at += n
    return table


def cached(cache, table, b, n, page):
    """Positions 0 .. n-1 of sequence b: [n, ...] from cache [pages, page, ...] (same device)."""
    s = torch.arange(n)
    return cache[table[b].long()[s // page], s % page]
