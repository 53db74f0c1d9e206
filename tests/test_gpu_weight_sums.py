"""Weight sums: what gets no weight keeps its sum, also where a log-sum-exp is NaN or -inf; the roundings of a score."""
import pytest
import torch

from oracle import paged
from test_gpu_small_cache import ALL

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from kv_cache_quantization_tq_gb300.build import build

    build()
    from test_gpu_paged import attend
    from test_gpu_small_cache import add_weights, rewrite, slopes_of, weights_case


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


@pytest.mark.parametrize("bits,bf16", ALL)
@pytest.mark.parametrize("hq,hkv,d", [(4, 2, 64), (8, 1, 128), (20, 1, 128), (3, 1, 256), (9, 1, 512)])
@pytest.mark.parametrize("cap", [0.0, 20.0])
def test_a_nan_reaches_only_tokens_that_count(hq, hkv, d, bits, bf16, cap):
    """In front of the window, on its first page and before it, and on pages with a bad id, sums fade and nothing else."""
    e = weights_case(d + hq, [100, 61, 16, 33], hq, hkv, d, bits, bf16)
    window = 41
    e["bt"][0, 4], e["bt"][3, 1] = -1, e["pool"].shape[0]  # positions 64 .. 79 of the first, 16 .. 31 of the last
    _, lse = attend(e, window=window)
    assert e["ctx"].device_errors() == paged.ERR_BLOCK_ID
    ref = add_weights(e, lse, decay=0.5, window=window, cap=cap)
    e["ctx"].device_errors()
    rep, before = hq // hkv, e["before"].cuda()
    for h in {0, hq - 1}:
        bad = lse.clone()
        bad[:, h] = float("nan")
        for in_place in (False, True):
            got = add_weights(e, bad, decay=0.5, window=window, cap=cap, in_place=in_place)
            assert e["ctx"].device_errors() == paged.ERR_BLOCK_ID
            for b, n in enumerate(e["lengths"]):
                p = torch.arange(n, device="cuda")
                id = torch.from_numpy(e["bt"][b]).cuda()[p // 16]
                counts = (p >= n - window) & (id >= 0) & (id < e["pool"].shape[0])
                row = got[b, h // rep, :n]
                assert torch.isnan(row[counts]).all()
                assert torch.equal(row[~counts], 0.5 * before[b, h // rep, :n][~counts])
            others = [x for x in range(hkv) if x != h // rep]
            for b, n in enumerate(e["lengths"]):
                assert torch.equal(got[b, others, :n], ref[b, others, :n])


@pytest.mark.parametrize("bits,bf16", ALL)
@pytest.mark.parametrize("cap,biased", [(0.0, False), (20.0, True)])
def test_a_row_without_weights_adds_nothing_whatever_its_keys_hold(cap, biased, bits, bf16):
    """A log-sum-exp of -inf against keys that are NaN and infinite (8- and 4-bit pages: as large as they get)."""
    e = weights_case(17, [50, 20], 6, 2, 64, bits, bf16)
    s = slopes_of(6) if biased else None
    k = torch.randn(50, 2, 64)
    k[3, 0, 5], k[20, 0], k[21, 0], k[40, 1, 1] = float("nan"), float("inf"), float("-inf"), float("inf")
    rewrite(e, 0, k, torch.randn(50, 2, 64))
    lse = torch.zeros(2, 6, device="cuda")
    lse[0, :3] = -float("inf")
    got = add_weights(e, lse, decay=0.5, cap=cap, slopes=s)
    assert e["ctx"].device_errors() == 0
    assert torch.equal(got[0, 0, :50], 0.5 * e["before"][0, 0, :50].cuda())
    # beside a head that has weights the others still add nothing
    lse[0, :3] = torch.tensor([-float("inf"), 0.0, -float("inf")])
    one = add_weights(e, lse, decay=0.5, cap=cap, slopes=s, before=False)
    lse[0, :3] = torch.tensor([float("inf"), 0.0, float("inf")])
    ref = add_weights(e, lse, decay=0.5, cap=cap, slopes=s, before=False)
    finite = torch.isfinite(ref[0, 0, :50])
    assert int(finite.sum()) >= 45 and torch.equal(one[0, 0, :50][finite], ref[0, 0, :50][finite])


@pytest.mark.parametrize("d", [64, 128, 256, 512])
def test_fp16_scores_are_rounded_once(d):
    """A score of 1024 and two small parts, each less than half a step of it: one in a product of its own, one in the bits behind a
    query entry's first five.  Together they count: the score is off by half a step of 1024 (2^-14), the exponential by 2^-21."""
    gen = torch.Generator().manual_seed(d)
    n, step = 96, 2.0 ** -13
    a, b = 0.3 + 0.19 * torch.rand(n, generator=gen), 0.3 + 0.19 * torch.rand(n, generator=gen)
    sign = torch.where(torch.arange(n) % 2 == 0, 1.0, -1.0)
    k = torch.zeros(n, 1, d)
    k[:, 0, 0] = 32.0
    k[:, 0, 16] = sign * a * step * 128
    k[:, 0, 17] = k[:, 0, 18] = sign * b * step * 128
    e = weights_case(d, [n], 1, 1, d, 16, False)
    rewrite(e, 0, k, torch.zeros(n, 1, d))
    e["q"][:] = 0
    e["q"][0, 0, 0], e["q"][0, 0, 16], e["q"][0, 0, 17], e["q"][0, 0, 18] = 32.0, 2.0 ** -7, 1 + 2.0 ** -7, -1.0
    got = add_weights(e, torch.full((1, 1), 1024.0, device="cuda"), before=False, scale=1.0)[0, 0, :n].double().cpu()
    z = (k[:, 0].half().double() * e["q"][0, 0].double()).sum(1) - 1024
    assert (z.abs() > 0.6 * step).all()
    assert ((got - torch.exp(z)).abs() <= 2.0 ** -14 * (1 + 2.0 ** -10) + 2.0 ** -21).all()
