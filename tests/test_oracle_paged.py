"""Pins of the dense-page oracle (CPU): number formats against torch's casts, the attention against a direct
softmax, the plan's bookkeeping, bad pages and refused requests; the binding's own argument checks."""
import numpy as np
import pytest
import torch

from oracle import paged

from kv_cache_quantization_tq_gb300.build import build

build()
from kv_cache_quantization_tq_gb300 import binding as B  # noqa: E402


def test_e4m3_codes_match_the_cast():
    every = np.arange(256, dtype=np.uint8)
    ref = torch.from_numpy(every.copy()).view(torch.float8_e4m3fn).double().numpy()
    got = paged.e4m3_value(every)
    assert np.array_equal(np.isnan(got), np.isnan(ref)) and np.array_equal(got[~np.isnan(ref)], ref[~np.isnan(ref)])
    x = np.concatenate([np.linspace(-448, 448, 40001), 2.0 ** np.arange(-14, 9.0), 17 * 2.0 ** np.arange(-14, 4.0)])
    x = x.astype(np.float32)
    ref = torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(paged.e4m3_code(x.astype(np.float64)), ref)
    assert paged.e4m3_code(np.array([np.inf, -np.inf, 1e9, np.nan])).tolist() == [0x7E, 0xFE, 0x7E, 0x7F]


def test_exponent_is_the_least_that_fits():
    top = np.array([0.0, 448.0, 448.1, 1.0, 1.75, 1.7500001, 65504.0, 3e38, 1e-45])
    e = paged.exponent(top[:, None])
    assert e.tolist() == [-120, 0, 1, -8, -8, -7, 8, 120, -120]
    for t, k in zip(top, e):
        assert t <= 448 * 2.0 ** k and (k == -120 or t > 448 * 2.0 ** (k - 1))
    assert paged.exponent(np.array([np.inf, -2.0, np.nan])) == paged.exponent(np.array([2.0]))


@pytest.mark.parametrize("bits,bf16", [(16, False), (16, True), (8, False), (8, True)])
def test_store_then_attend_is_a_softmax(bits, bf16):
    rng = np.random.default_rng(5)
    d, hkv, n, nb = 64, 2, 37, 7
    dt = torch.bfloat16 if bf16 else torch.float16
    k = torch.from_numpy(rng.standard_normal((n, hkv, d))).to(dt)
    v = torch.from_numpy(rng.standard_normal((n, hkv, d))).to(dt)
    bt = np.array([[4, 0, 6]], np.int32)
    pos = np.arange(n)
    slots = bt[0, pos // 16].astype(np.int64) * 16 + pos % 16
    pool = np.full((nb, hkv, paged.tile_bytes(d, bits)), 0xFF, np.uint8)  # NaN wherever nothing is stored
    pool, flags = paged.store(pool, k.view(torch.int16).numpy().view(np.uint16), v.view(torch.int16).numpy().view(np.uint16),
                              slots, d, bits, bf16)
    assert flags == 0
    q = rng.standard_normal((1, 4, d))
    for window in (0, 1, 20, 100):
        out, lse, _, flags = paged.attention(q, pool, bt, [n], d, bits, bf16, window)
        assert flags == 0
        lo = max(0, n - window) if window else 0
        kk, vv = k.double()[lo:], v.double()[lo:]
        s = torch.einsum("hgd,nhd->hgn", torch.from_numpy(q.reshape(2, 2, d)), kk) / 8.0
        ref = torch.einsum("hgn,nhd->hgd", torch.softmax(s, -1), vv).reshape(4, d).numpy()
        # 8-bit entries are off by half a step of 3 fraction bits, 2^-4 relative: the values directly, the scores
        # through the weights
        tol = 1e-12 if bits == 16 else 0.6
        assert np.max(np.abs(out[0] - ref)) < tol
        if bits == 16:
            assert np.allclose(lse[0], torch.logsumexp(s, -1).flatten().numpy(), atol=1e-12)


def test_attention_leaves_bad_pages_and_lengths_out():
    d, rng = 64, np.random.default_rng(6)
    pool = rng.standard_normal((3, 1, 32 * d)).astype(np.float16).view(np.uint8).reshape(3, 1, -1)
    q = rng.standard_normal((4, 1, d))
    bt = np.array([[0, 9], [1, 2], [0, 1], [-1, -1]], np.int32)
    out, lse, _, flags = paged.attention(q, pool, bt, [20, 33, -1, 5], d, 16, False)
    assert flags == paged.ERR_BLOCK_ID | paged.ERR_POSITION
    only, _, _, _ = paged.attention(q[:1], pool, bt[:1, :1], [16], d, 16, False)
    assert np.array_equal(out[0], only[0])
    assert not out[1:].any() and np.all(lse[1:] == -np.inf)


@pytest.mark.parametrize("ring", [0, 128])
def test_plan_keeps_every_page_once(ring):
    """Over random steps: each block is in exactly one place (a row's held pages or the queue)."""
    rng = np.random.default_rng(7 + ring)
    bsz, maxb, nb = 9, 40, 150
    table = np.full((bsz, maxb), -1, np.int32)
    queue, state = rng.permutation(nb).astype(np.int32), np.array([0, nb], np.int32)
    ctx = np.zeros(bsz, np.int32)
    for step in range(60):
        new = rng.integers(0, 60, bsz).astype(np.int32)
        new[rng.random(bsz) < 0.1] = -1
        r = paged.plan(ctx, new, table, queue, state, nb, 400, ring)
        assert r["flags"] & ~(paged.ERR_PAGES | paged.ERR_POSITION) == 0
        table, queue, state, ctx = r["block_table"], r["queue"], r["queue_state"], r["lengths"]
        held = [table[b, :paged.pages_of(int(ctx[b]), ring)] for b in range(bsz)]
        free = queue[(state[0] + np.arange(state[1])) % nb]
        assert np.array_equal(np.sort(np.concatenate(held + [free])), np.arange(nb))
        real = r["slots"][r["slots"] >= 0]
        assert len(np.unique(real)) == len(real)
        assert np.all(r["n_paged"] % 16 == 0) or not ring


def test_plan_refusals():
    table = np.full((4, 4), -1, np.int32)
    queue = np.arange(5, dtype=np.int32)
    r = paged.plan([0, 0, 3, 0], [40, 33, 2, 1], np.where(np.arange(4)[:, None] == 2, 9, table), queue, [3, 5], 10, 100)
    # 3 pages for the first; the second wants 3 of the 2 left; the third needs none; the fourth wants one but stands
    # behind a refused one
    assert r["flags"] == paged.ERR_PAGES and r["lengths"].tolist() == [40, 0, 5, 0]
    assert r["block_table"][0].tolist() == [3, 4, 0, -1] and r["queue_state"].tolist() == [1, 2]
    assert r["slots"][73:76].tolist() == [9 * 16 + 3, 9 * 16 + 4, -1] and (r["slots"][40:73] == -1).all()
    r = paged.plan([0, -4], [65, 1], table[:2], queue, [0, 5], 10, 100)
    assert r["flags"] == paged.ERR_POSITION and r["lengths"].tolist() == [0, 0] and r["queue_state"].tolist() == [0, 5]
    r = paged.plan([0], [1], table[:1], queue, [0, 6], 10, 100)
    assert r["flags"] == paged.ERR_PAGES and r["queue_state"].tolist() == [0, 6]


# ---------------------------------------------------------------- host checks of the library (no GPU)
@pytest.mark.parametrize("d", [64, 128, 256, 512])
def test_dense_config_sizes(d):
    for bits in (16, 8):
        cfg = B.tq_config_init(B.TQ_LAYOUT_DENSE, d, 14, 2)
        cfg.key_bits = cfg.value_bits = bits
        assert 16 * B.tq_config_check(cfg) == paged.tile_bytes(d, bits)
        cfg.key_format = B.TQ_ELEM_BF16
        assert 16 * B.tq_config_check(cfg) == paged.tile_bytes(d, bits)
    assert B.tq_config_init(B.TQ_LAYOUT_DENSE, d, 36, 4).key_bits == 16  # any ratio of heads


def test_dense_config_refusals():
    for field, value in (("key_bits", 8), ("value_bits", 4), ("key_format", 2), ("qjl_m", 64), ("page_size", 32)):
        cfg = B.tq_config_init(B.TQ_LAYOUT_DENSE, 128, 8, 8)
        setattr(cfg, field, value)
        with pytest.raises(B.TQError) as e:
            B.tq_config_check(cfg)
        assert e.value.status == B.TQ_ERR_UNSUPPORTED, field
    with pytest.raises(B.TQError):
        B.tq_config_init(B.TQ_LAYOUT_DENSE, 96, 8, 8)
    with pytest.raises(B.TQError) as e:
        B.tq_config_init(B.TQ_LAYOUT_DENSE, 128, 9, 8)
    assert e.value.status == B.TQ_ERR_INVALID_ARG


def test_null_context_is_refused():
    n = None
    assert B.lib.tq_plan_pages(n, n, n, 1, 0, n, 1, 1, n, 1, n, n, n, n, n, n, n, n, 1, n, n) == B.TQ_ERR_INVALID_ARG
    assert B.lib.tq_paged_store(n, n, n, 0, 0, n, 1, n, 1, n) == B.TQ_ERR_INVALID_ARG
    assert B.lib.tq_paged_workspace_size(n, 1, n) == B.TQ_ERR_INVALID_ARG
    assert B.lib.tq_paged_attention(n, n, 0, 1, n, 1, n, 1, n, 0, 0.0, n, n, n, 0, n) == B.TQ_ERR_INVALID_ARG


def test_binding_checks_shapes_before_the_library():
    ctx = object.__new__(B.Context)
    ctx.ptr = None
    ctx.cfg = B.tq_config_init(B.TQ_LAYOUT_DENSE, 64, 4, 2)
    ctx.head_dim, ctx.num_q_heads, ctx.num_kv_heads, ctx._device = 64, 4, 2, 0
    ctx._elem, ctx._types = torch.float16, (torch.int32, torch.int64, torch.float32, torch.uint8)
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    q = torch.zeros(3, 4, 64, dtype=torch.float16)
    with pytest.raises(ValueError, match="CUDA"):
        ctx.paged_attention(q, None, i32(3, 1), i32(3), torch.zeros(3, 4, 64), None)
    with pytest.raises(ValueError, match="float16"):
        ctx.paged_attention(q.bfloat16(), None, i32(3, 1), i32(3), torch.zeros(3, 4, 64), None)
    with pytest.raises(ValueError, match=r"\[n, 2, 64\]"):
        ctx.paged_store(q, q, torch.zeros(3, dtype=torch.int64), None)
    ok = dict(ctx_len=i32(3), new_len=i32(3), block_table=i32(3, 2), queue=i32(4), queue_state=i32(2), lengths=i32(3),
              token_start=i32(4), slots=torch.zeros(5, dtype=torch.int64), queue_state_out=i32(2), num_blocks=4)
    with pytest.raises(ValueError, match="must be a CUDA tensor"):
        ctx.plan_pages(**ok)
    for name, bad in (("new_len", i32(2)), ("token_start", i32(3)), ("queue_state", i32(1)), ("block_table", i32(2, 2)),
                      ("positions", i32(4)), ("n_ring", i32(4)), ("num_blocks", 2 ** 32 + 4), ("num_blocks", -1)):
        with pytest.raises(ValueError):
            ctx.plan_pages(**{**ok, name: bad})
