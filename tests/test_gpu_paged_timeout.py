"""The end of the dense-page attention's bounded waits: with a limit of 0 a warp's second copy counts as late (where
keys and values are copied apart these are its first values, with the next keys on their way), and the call must still
return, say so, give NaN in place of numbers, and leave the context, its buffers and the next call as they were."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from kv_cache_quantization_tq_gb300.build import build

    build()
    import kv_cache_quantization_tq_gb300 as tq
    from test_gpu_paged import attend, make_case

FORMS = [(16, False), (16, True), (8, False), (8, True)]


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


@pytest.mark.parametrize("hq,hkv,d", [(2, 2, 64), (24, 2, 64), (8, 2, 128), (32, 2, 128), (4, 2, 256), (4, 1, 512)])
@pytest.mark.parametrize("bits,bf16", FORMS)
def test_waits_that_run_out(bits, bf16, hq, hkv, d):
    e = make_case(d + hq, [200, 130], hq, hkv, d, bits, bf16)  # 21 pages, named again and again by long sequences
    ctx, held = e["ctx"], np.concatenate([e["bt"][0, :12], e["bt"][1, :8]])  # the whole ones
    e["lengths"] = np.array([60000, 0, 17, 20000, 31000, 16, 60000], np.int32)
    e["bt"] = np.resize(held, (7, 60000 // 16)).astype(np.int32)
    e["q"] = torch.randn(7, hq, d, generator=torch.Generator().manual_seed(d)).to(e["q"].dtype)
    ref, ref_lse = attend(e)
    assert ctx.device_errors() == 0 and torch.isfinite(ref).all()
    pool = e["pool"].clone()
    ctx.set_wait_limit(0)
    out, lse = attend(e)
    assert ctx.device_errors() == tq.binding.TQ_DEVERR_TIMEOUT
    late = torch.isnan(lse)
    assert late.any() and not late[1].any()  # an empty sequence waits for nothing
    assert torch.isnan(out[late]).all()
    assert torch.equal(out[~late], ref[~late]) and torch.equal(lse[~late], ref_lse[~late])
    assert torch.equal(e["pool"], pool)
    ctx.set_wait_limit(10 ** 9)
    again, again_lse = attend(e)
    assert ctx.device_errors() == 0 and torch.equal(again, ref) and torch.equal(again_lse, ref_lse)


def test_the_limit_is_checked():
    ctx = tq.Context(tq.TQ_LAYOUT_DENSE, 64, 2, 2)
    for ns in (-1, 2 ** 32):
        with pytest.raises(ValueError):
            ctx.set_wait_limit(ns)
    assert tq.lib.tq_set_wait_limit(None, 5) == tq.binding.TQ_ERR_INVALID_ARG
