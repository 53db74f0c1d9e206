"""Dense-page attention over the range of its types: weights and values of very different sizes in one page, values and
queries near the ends of their types.

Tolerance.  Scores are single products (paged_cases.single_term), so a score s (in powers of two) is exact up to the
roundings of its factors and of s - m: at most 6 u (|s| + 1) with u = 2^-24, and a weight is off by as much, relative.
The exponential, the split of a weight and the division add 2^-19, and the sum over the positions 2 u for each of its at
most n / 16 + 64 partial sums.  Each enters numerator and total once:
  |out - ref| <= (2 * 6 u (S + 1) + 2^-19 + (n / 8 + 128) u) sum p |v|,  S = max |s|,
element by element: nothing is said about the size of a vector's other entries or of other tokens' values.
8-bit pages hold a weight times its value exponent in two fp16 parts, whose last step is 2^-24, with the row's
largest product at 2^12 or more: a token is off by at most 2^-25 times a code of at most 448, and the token of the
largest product has an entry whose code is at least 224 (its exponent is the least that fits).  So n tokens add at
most n 2^-25 448 / (2^12 224) = n 2^-36 of the row's largest entry of sum p |v|, which is more where an entry's code is 0 in
every token that weighs.
"""
import numpy as np
import pytest
import torch

from oracle import paged
from paged_cases import U, single_term

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from kv_cache_quantization_tq_gb300.build import build

    build()
    import kv_cache_quantization_tq_gb300 as tq
    from test_gpu_paged import attend, elem, make_case

FORMS = [(16, False), (16, True), (8, False), (8, True)]


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def fill(e, q, k, v):
    """Stores k and v of the case's sequences, one behind another, and takes q as its queries."""
    slots = np.concatenate([e["bt"][b, np.arange(n) // 16].astype(np.int64) * 16 + np.arange(n) % 16
                            for b, n in enumerate(e["lengths"])])
    e["ctx"].paged_store(k.cuda(), v.cuda(), torch.from_numpy(slots).cuda(), e["pool"])
    e["q"] = q


def check(e, out, lse, scale=None):
    assert e["ctx"].device_errors() == 0
    ref, rlse, (a, vabs), _ = paged.attention(e["q"].double().numpy(), e["pool"].cpu().numpy(), e["bt"], e["lengths"], e["d"],
                                              e["bits"], e["bf16"], 0, scale)
    rel = 12 * U * (a * 1.4427 + 1) + 2.0 ** -19 + (e["lengths"].max() / 8 + 128) * U
    bound = rel[..., None] * vabs
    if e["bits"] == 8:
        bound = bound + e["lengths"].max() * 2.0 ** -36 * vabs.max(-1, keepdims=True)
    err = np.abs(out.cpu().numpy().astype(np.float64) - ref)
    assert np.all(err <= bound), f"worst {np.nanmax(err / (bound + 1e-300)):.3g} of the bound"
    got = lse.cpu().numpy().astype(np.float64)
    assert np.all(np.abs(got - rlse) <= rel + 2 * U * np.abs(rlse))


# how far the weights fall and the sizes of the values: the light tokens' share of the result goes from nothing to
# everything.  fp16 values are kept within fp16's normal numbers; bf16 ones go further.
RANGES = [(-10, (-6, 12)), (-24, (-12, 14)), (-34, (-14, 13)), (-50, (-14, 13))]
WIDE = [(-10, (-20, 20)), (-24, (-30, 30)), (-60, (-30, 30)), (-30, (-60, 60)), (-80, (-30, 30))]


@pytest.mark.parametrize("bits,bf16,weight_log2,size_log2", [(*f, *r) for f in FORMS for r in RANGES + (WIDE if f[1] else [])])
@pytest.mark.parametrize("hq,hkv,d", [(4, 2, 64), (8, 1, 128), (24, 2, 128), (2, 1, 256), (3, 1, 512)])
def test_weights_and_values_of_different_sizes(bits, bf16, hq, hkv, d, weight_log2, size_log2):
    lengths = [2, 16, 5, 40, 300]
    e = make_case(d + hq, lengths, hq, hkv, d, bits, bf16)
    fill(e, *single_term(hq - weight_log2, lengths, hq, hkv, d, elem(bf16), weight_log2, size_log2))
    check(e, *attend(e))


@pytest.mark.parametrize("bits", [16, 8])
@pytest.mark.parametrize("hq,d", [(4, 64), (16, 128), (2, 512)])
def test_values_near_the_largest(bits, hq, d):
    """bf16 values of up to 3.9 x 2^118, all positive: 100 of them with weights of at most 1 stay below 2^127."""
    lengths = [100, 17]
    e = make_case(d, lengths, hq, 1, d, bits, True)
    q, k, v = single_term(d, lengths, hq, 1, d, torch.bfloat16, -2, (117, 118), heavy=False)
    fill(e, q, k, v.abs())
    check(e, *attend(e))


@pytest.mark.parametrize("bits,size_log2", [(16, (-100, -98)), (8, (-78, -76))])
@pytest.mark.parametrize("hq,d", [(4, 64), (16, 128), (2, 512)])
def test_values_near_the_smallest(bits, size_log2, hq, d):
    """bf16 values down to where the range that is kept ends."""
    lengths = [100, 17, 1]
    e = make_case(d, lengths, hq, 1, d, bits, True)
    fill(e, *single_term(d, lengths, hq, 1, d, torch.bfloat16, -12, size_log2, heavy=False))
    check(e, *attend(e))


@pytest.mark.parametrize("power", [-118, -90, 90, 118])
def test_queries_against_keys_of_the_opposite_size(power):
    """8-bit pages: bf16 queries times 2^power, keys times 2^-power (8-bit keys go down to about 2^-120)."""
    lengths = [60, 33]
    e = make_case(power + 200, lengths, 4, 2, 64, 8, True)
    q, k, v = single_term(power + 200, lengths, 4, 2, 64, torch.bfloat16, -12, (-1, 1))
    fill(e, (q.double() * 2.0 ** power).bfloat16(), (k.double() * 2.0 ** -power).bfloat16(), v)
    check(e, *attend(e))


@pytest.mark.parametrize("bf16", [False, True])
def test_scores_that_are_all_minus_infinity(bf16):
    """A sequence whose keys are all -inf (its queries are positive) has no weight anywhere; its neighbours keep theirs."""
    lengths = [33, 40, 700]
    e = make_case(3, lengths, 4, 2, 64, 16, bf16)
    q, k, v = single_term(3, lengths, 4, 2, 64, elem(bf16), -5, (0, 1))
    q[1], k[33:73] = 1.0, float("-inf")
    fill(e, q, k, v)
    out, lse = attend(e)
    assert (out[1] == 0).all() and (lse[1] == float("-inf")).all()
    assert torch.isfinite(out[::2]).all() and torch.isfinite(lse[::2]).all() and out[::2].any(-1).all()
    assert e["ctx"].device_errors() == 0
