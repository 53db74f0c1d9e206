"""4-bit pages over the range of their types, and light tokens of large values beside a heavy one of small values.

Tolerance of the first part: the bound of test_gpu_paged_range.py (single-product scores)
  |out - ref| <= (12 u (S + 1) + 2^-19 + (n / 8 + 128) u) sum p |v|,  u = 2^-24, S = max |s| in powers of two,
and what the two fp16 parts of a weight times its value exponent leave out: their last step is 2^-24 and the row's largest product is at
2^12 or more, so a token is off by at most 2^-25 times a code times scale of at most 2688.  The token of the largest product
has an entry of more than 1344 before it is rounded; its block's scale is within 2^-4 and its code is 6, so that it is held as at
least 1344 (1 - 2^-4) = 1260.  n tokens add at most n 2^-25 2688 / (2^12 1260) = 2.14 n 2^-37 of the row's largest entry of sum p |v|.
"""
import numpy as np
import pytest
import torch

from oracle import paged
from paged_cases import U, single_term
from test_gpu_paged_range import RANGES, WIDE, fill

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from kv_cache_quantization_tq_gb300.build import build

    build()
    from test_gpu_paged import attend, elem, make_case


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def check(e, out, lse, scale=None, optional=0.0):
    """optional: weights below this share of a row's largest may be missing."""
    assert e["ctx"].device_errors() == 0
    seen = []
    ref, rlse, (a, vabs), _ = paged.attention(e["q"].double().numpy(), e["pool"].cpu().numpy(), e["bt"], e["lengths"], e["d"],
                                              e["bits"], e["bf16"], 0, scale, weights=seen)
    rel = 12 * U * (a * 1.4427 + 1) + 2.0 ** -19 + (e["lengths"].max() / 8 + 128) * U
    bound = rel[..., None] * vabs
    if e["bits"] < 16:
        share = 2.14 * 2.0 ** -37 if e["bits"] == 4 else 2.0 ** -36
        bound = bound + e["lengths"].max() * share * vabs.max(-1, keepdims=True)
    pool, rep = e["pool"].cpu().numpy(), e["q"].shape[1] // e["pool"].shape[1]
    for b, h, p, s, _ in seen:
        w = np.exp(s - rlse[b, h])
        for at in p[w < optional * w.max()]:
            tile = paged.tile_rows(pool[e["bt"][b, at // 16], h // rep], e["d"], e["bits"], e["bf16"])
            bound[b, h] += w[at] * np.abs(tile[1][at % 16])
    err = np.abs(out.cpu().numpy().astype(np.float64) - ref)
    assert np.all(err <= bound), f"worst {np.max(err / (bound + 1e-300)):.3g} of the bound"
    got = lse.cpu().numpy().astype(np.float64)
    assert np.all(np.abs(got - rlse) <= rel + 2 * U * np.abs(rlse))


# the forms of 4-bit attention: 4 heads, 8 and 16 in a product's columns, one and two pages a step
HEADS = [(4, 2, 64), (8, 1, 64), (8, 2, 128), (8, 1, 128), (24, 2, 128), (2, 1, 256), (6, 1, 256), (9, 1, 256), (3, 1, 512), (8, 1, 512)]


@pytest.mark.parametrize("bf16,weight_log2,size_log2", [(False, *r) for r in RANGES] + [(True, *r) for r in RANGES + WIDE])
@pytest.mark.parametrize("hq,hkv,d", HEADS)
def test_weights_and_values_of_different_sizes(bf16, hq, hkv, d, weight_log2, size_log2):
    lengths = [2, 16, 5, 40, 300]
    e = make_case(d + hq, lengths, hq, hkv, d, 4, bf16)
    fill(e, *single_term(hq - weight_log2, lengths, hq, hkv, d, elem(bf16), weight_log2, size_log2))
    check(e, *attend(e))


@pytest.mark.parametrize("hq,hkv,d", HEADS)
def test_values_near_the_largest(hq, hkv, d):
    """bf16 values of up to 3.9 x 2^118, all positive: 100 of them with weights of at most 1 stay below 2^127."""
    lengths = [100, 17]
    e = make_case(d, lengths, hq, hkv, d, 4, True)
    q, k, v = single_term(d, lengths, hq, hkv, d, torch.bfloat16, -2, (117, 118), heavy=False)
    fill(e, q, k, v.abs())
    check(e, *attend(e))


@pytest.mark.parametrize("hq,hkv,d", HEADS)
def test_values_near_the_smallest(hq, hkv, d):
    """bf16 values down to where the range that is kept ends."""
    lengths = [100, 17, 1]
    e = make_case(d, lengths, hq, hkv, d, 4, True)
    fill(e, *single_term(d, lengths, hq, hkv, d, torch.bfloat16, -12, (-75, -73), heavy=False))
    check(e, *attend(e))


@pytest.mark.parametrize("power", [-112, -90, 90, 112])
def test_queries_against_keys_of_the_opposite_size(power):
    """bf16 queries times 2^power, keys times 2^-power."""
    lengths = [60, 33]
    e = make_case(power + 200, lengths, 4, 2, 64, 4, True)
    q, k, v = single_term(power + 200, lengths, 4, 2, 64, torch.bfloat16, -12, (-1, 1))
    fill(e, (q.double() * 2.0 ** power).bfloat16(), (k.double() * 2.0 ** -power).bfloat16(), v)
    check(e, *attend(e))


@pytest.mark.parametrize("bits", [16, 8, 4])
@pytest.mark.parametrize("hq,hkv,d", HEADS)
@pytest.mark.parametrize("heavy,light,nats", [(0, 116, -97), (0, 116, -200), (-49, 71, -87), (None, 60, -84), (-30, 60, -96), (-20, 80, -64)])
def test_light_tokens_of_large_values(heavy, light, nats, hq, hkv, d, bits):
    """One token has the weight and values of 2^heavy (None: zeros), another a weight of e^nats and values of 2^light, beside it or
    pages behind it.  Weights below 2^-100 of the largest may be left out, but nothing is infinite or NaN."""
    lengths = [2, 40, 70]
    e = make_case(d + hq, lengths, hq, hkv, d, bits, True)
    n = sum(lengths)
    q, k, v = torch.zeros(3, hq, d), torch.full((n, hkv, d), -30.0), torch.zeros(n, hkv, d)
    q[:, :, 3] = 1.0
    gen = torch.Generator().manual_seed(d)
    for b, (heavy_at, light_at) in enumerate([(0, 1), (1, 37), (60, 2)]):
        at = sum(lengths[:b])
        k[at + heavy_at] = 0.0
        k[at + light_at] = nats
        v[at:at + lengths[b]] = 0.0 if heavy is None else 2.0 ** heavy * torch.randn(lengths[b], hkv, d, generator=gen).clamp(-3.9, 3.9)
        v[at + light_at] = 2.0 ** light * (1 + torch.rand(hkv, d, generator=gen))
    fill(e, q.bfloat16(), k.bfloat16(), v.bfloat16())
    check(e, *attend(e, scale=1.0), scale=1.0, optional=2.0 ** -100)
