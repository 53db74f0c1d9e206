"""Weight sums where a log-sum-exp is NaN: what gets no weight keeps its sum."""
import pytest
import torch

from oracle import paged
from test_gpu_small_cache import ALL

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from kv_cache_quantization_tq_gb300.build import build

    build()
    from test_gpu_paged import attend
    from test_gpu_small_cache import add_weights, weights_case


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
