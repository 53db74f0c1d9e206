"""A cache held small over many steps, with intervals between evictions that shrink and grow, a second prompt and a new request in a
row: what a token has not reached yet has no weight, and every page is accounted for.  Sums within the bound of
test_gpu_small_cache.py (check_weights)."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from kv_cache_quantization_tq_gb300.build import build

    build()
    from test_gpu_paged import dense, elem
    from test_gpu_small_cache import check_weights, i32


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


@pytest.mark.parametrize("bits,bf16", [(16, True), (8, False), (4, False)])
def test_new_tokens_begin_without_weight(bits, bf16):
    hq, hkv, d, bsz, keep, maxb, nb = 4, 2, 64, 3, 24, 10, 40
    ctx, dt, gen = dense(d, hq, hkv, bits, bf16), elem(bf16), torch.Generator().manual_seed(bits)
    pool = torch.zeros(nb, hkv, ctx.page_bytes, dtype=torch.uint8, device="cuda")
    bt, queue = torch.full((bsz, maxb), -1, dtype=torch.int32, device="cuda"), torch.arange(nb, dtype=torch.int32, device="cuda")
    state, state_out = i32([0, nb]), i32([0, 0])
    lengths, shorter, keeps = i32([0] * bsz), i32([0] * bsz), i32([keep] * bsz)
    start, slots = i32([0] * (bsz + 1)), torch.zeros(300, dtype=torch.int64, device="cuda")
    out, lse = torch.zeros(bsz, hq, d, device="cuda"), torch.zeros(bsz, hq, device="cuda")
    ws = torch.zeros(ctx.paged_workspace_size(bsz), dtype=torch.uint8, device="cuda")
    w, w2 = torch.zeros(2, bsz, hkv, maxb * 16, device="cuda")
    kept = torch.zeros(bsz, hkv, maxb * 16, dtype=torch.int32, device="cuda")
    ctx_len, had = i32([0] * bsz), [0] * bsz  # tokens in the cache, and how many of them have sums

    def step(new):
        nonlocal ctx_len, state, state_out, lengths, had
        ctx.plan_pages(ctx_len, i32(new), bt, queue, state, lengths, start, slots, state_out, num_blocks=nb)
        k, v = (torch.randn(300, hkv, d, generator=gen).to(dt).cuda() for _ in range(2))
        ctx.paged_store(k, v, slots, pool)
        q = torch.randn(bsz, hq, d, generator=gen).to(dt)
        ctx.paged_attention(q.cuda(), pool, bt, lengths, out, ws, lse=lse)
        before = w.cpu()
        for b in range(bsz):
            before[b, :, had[b]:] = 0.0
        ctx.paged_weights(q.cuda(), pool, bt, lengths, lse, w, weights=w, decay=0.9)
        e = dict(ctx=ctx, q=q, pool=pool, bt=bt.cpu().numpy(), lengths=lengths.cpu().numpy(), before=before, d=d, bits=bits, bf16=bf16)
        check_weights(e, w, lse, decay=0.9, in_place=True)
        ctx_len, state, state_out = lengths.clone(), state_out, state
        had = lengths.tolist()

    def evict():
        nonlocal w, w2, ctx_len, state, state_out, had
        ctx.paged_evict(w, pool, bt, lengths, keeps, w2, shorter, kept, sinks=2, recent=4)
        ctx.release_pages(lengths, shorter, bt, queue, state, state_out, num_blocks=nb)
        w, w2 = w2, w
        w2.zero_()
        ctx_len, state, state_out = shorter.clone(), state_out, state
        had = shorter.tolist()
        assert had == [min(keep, x) for x in lengths.tolist()]

    def accounted():
        held = [bt[b, :-(-n // 16)].tolist() for b, n in enumerate(ctx_len.tolist())]
        head, count = state.tolist()
        free = queue.tolist()
        assert sorted(sum(held, []) + [free[(head + j) % nb] for j in range(count)]) == list(range(nb))

    step([100, 7, 64])
    evict()
    for _ in range(3):
        step([1, 1, 1])
    evict()
    accounted()
    step([60, 50, 1])  # a second prompt
    for _ in range(9):
        step([1, 0, 1])
    evict()
    accounted()
    step([-1, 1, 1])  # the first request has ended, and another one takes its row
    w[0].zero_()
    had[0] = 0
    step([90, 1, 20])
    evict()
    accounted()
    assert ctx.device_errors() == 0
    assert np.isfinite(w.cpu().numpy()).all()
