"""Page plan: table entries that are no blocks, from the step that meets them to the one that gets them again."""
import numpy as np
import pytest
import torch

from oracle import paged

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from kv_cache_quantization_tq_gb300.build import build

    build()
    from test_gpu_paged import check_plan, dense


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


@pytest.mark.parametrize("entry", [-1, -7, 10, 2 ** 31 - 1])
def test_an_entry_that_is_no_block_is_flagged_when_it_is_given_back(entry):
    ctx = dense(64, 1, 1)
    table, queue = np.array([[4, entry, 6], [7, -1, -1]], np.int32), np.array([1, 2, -1, -1, -1, -1], np.int32)
    r = check_plan(ctx, [40, 3], [-1, 1], table, queue, [0, 2], 10, 4, 0)
    assert r["flags"] == paged.ERR_BLOCK_ID and r["queue"].tolist() == [1, 2, 4, entry, 6, -1]
    # the next step hands the pages out again, in order
    r = check_plan(ctx, r["lengths"], [48, 13], r["block_table"], r["queue"], r["queue_state"], 10, 70, 0)
    assert r["flags"] == paged.ERR_BLOCK_ID and r["block_table"].tolist() == [[1, 2, 4], [7, -1, -1]]
    assert (r["slots"][:48] >= 0).all() and r["slots"][48:61].max() == 7 * 16 + 15 and r["slots"][60] == -1


def test_many_pages_given_back():
    """More pages than one CTA has threads, one of them no block: the others keep their places."""
    ctx = dense(64, 1, 1)
    batch, held = 40, 200
    table = np.arange(batch * held, dtype=np.int32).reshape(batch, held)
    table[17, 33] = -1
    queue = np.full(batch * held + 5, -1, np.int32)
    queue[:3] = [8000, 8001, 8002]
    new = np.where(np.arange(batch) % 3 == 2, -1, 0)
    r = check_plan(ctx, np.full(batch, held * 16), new, table, queue, [0, 3], 8003, 1, 0)
    assert r["flags"] == paged.ERR_BLOCK_ID and r["queue_state"].tolist() == [0, 3 + 13 * held]
    table[17, 33] = 33
    assert check_plan(ctx, np.full(batch, held * 16), new, table, queue, [0, 3], 8003, 1, 0)["flags"] == 0
