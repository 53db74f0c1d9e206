"""Dense-page store: a pool without blocks, as a program has before its first page is made."""
import pytest
import torch

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from kv_cache_quantization_tq_gb300.build import build

    build()
    import kv_cache_quantization_tq_gb300 as tq
    from test_gpu_paged import dense


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


@pytest.mark.parametrize("bits", [16, 8])
def test_a_pool_without_blocks(bits):
    ctx = dense(64, 2, 2, bits)
    pool = torch.empty(0, 2, ctx.page_bytes, dtype=torch.uint8, device="cuda")
    k = torch.ones(3, 2, 64, dtype=torch.float16, device="cuda")
    ctx.paged_store(k, k, torch.full((3,), -1, dtype=torch.int64, device="cuda"), pool)  # no token has a page
    assert ctx.device_errors() == 0
    ctx.paged_store(k, k, torch.tensor([-1, 0, 1 << 40], device="cuda"), pool)
    assert ctx.device_errors() == tq.binding.TQ_DEVERR_BLOCK_ID
