"""Inputs of the dense-page attention whose scores are single products.

A query has one non-zero entry, so a score is one product and carries no error of a sum: what is left between the
kernel and 64 bits is the softmax and the weighted sum, and a bound on them can be tight.  Used by the GPU tests and,
with the weights' arithmetic done on the CPU, by the test that the tight bound sees a lost part.
"""
import torch

U = 2.0 ** -24  # half a step of fp32


def single_term(seed, lengths, hq, hkv, d, dtype, weight_log2, size_log2, heavy=True):
    """(q [batch][hq][d], k, v [tokens][hkv][d]) of `dtype`, the sequences' tokens one behind another.

    Position weights of a row are about 2^x, x spread over [weight_log2, 0], and a token's values are normal entries
    (within 3.9 of 0) times 2^y, y spread over size_log2 = (lo, hi).  With `heavy` one token of each sequence has x = 0 and y = lo, and
    all others x <= weight_log2 / 2: the token that has the weight is the one with the smallest values."""
    gen = torch.Generator().manual_seed(seed)
    n = sum(lengths)
    x = torch.rand(n, generator=gen) * weight_log2
    y = torch.randint(size_log2[0], size_log2[1] + 1, (n,), generator=gen).float()
    if heavy:
        x = weight_log2 / 2 + x / 2
        at = 0
        for m in lengths:
            if m:
                i = at + int(torch.randint(0, m, (1,), generator=gen))
                x[i], y[i] = 0.0, float(size_log2[0])
            at += m
    # key entries differ by up to an eighth from one dim to the next, so that the heads' weights do too
    k = (x * 0.6931471805599453)[:, None, None] * (1 + torch.rand(1, hkv, d, generator=gen) / 8)
    v = torch.randn(n, hkv, d, generator=gen).clamp(-3.9, 3.9) * torch.exp2(y)[:, None, None]
    q = torch.zeros(len(lengths), hq, d)
    j = torch.randint(0, d, (len(lengths), hq, 1), generator=gen)
    q.scatter_(2, j, d ** 0.5)
    return q.to(dtype), k.to(dtype), v.to(dtype)


def one_token(seed, n, hq, hkv, d, dtype):
    """n sequences of one token: the result is its values, whatever its weight; weights are anywhere in (1/2, 1]."""
    gen = torch.Generator().manual_seed(seed)
    q = torch.zeros(n, hq, d)
    q.scatter_(2, torch.randint(0, d, (n, hq, 1), generator=gen), 1 + torch.rand(n, hq, 1, generator=gen))
    k, v = torch.randn(n, hkv, d, generator=gen) * 3, torch.randn(n, hkv, d, generator=gen)
    return q.to(dtype), k.to(dtype), v.to(dtype)


# What one token's result may be off by, in u relative: the weight's parts 4 (two of 11 bits; 16-bit parts less), the cut
# of their sum 2, the division and the product 1 each.
ONE_TOKEN = 8


def light_tokens(key_values, query_values, d):
    """(query, key): a one-entry query and a key whose weight is as near to 3/8 u as their types allow, beside a
    token of weight 1 (key 0); and how far off it is, relative.

    With values of 1, a page of 16 such tokens adds 6 u = 3 steps to a sum of 1 in fp32, without a rounding; two of them,
    3/4 u, add nothing to a total of 1 unless what they lose is kept."""
    import math

    want = math.log(3 / 8 * U) * math.sqrt(d)
    best = min(((q, -k) for q in query_values for k in key_values), key=lambda x: abs(x[0] * x[1] - want))
    return best[0], best[1], abs(math.expm1((best[0] * best[1] - want) / math.sqrt(d)))


LIGHT_PAGES = 256


def light_tolerance(off):
    """|result - 1| in u: the sum of 256 pages is off by their additions' share of `off`, the rest as ONE_TOKEN with the
    joining of a sequence's pieces (weights 2^x of their references: 2^-22, 4 u) and of the lanes' totals (3 u)."""
    return 2 * (ONE_TOKEN + 4 + 3) + LIGHT_PAGES * 6 * off
