"""Page plan, dense-page store and single-token attention on the GPU against oracle/paged.py.

Tolerances (derived, not fitted).  The plan gives whole numbers and the store exact codes: both must match
bit for bit.  Attention: with u = 2^-24 (half a step of fp32) and A = max_p sum_i |scale q_i k_pi|, a score
is a sum of d exact products in fp32 whose order is the kernel's, each addition off by at most 2 u (the
tensor cores cut instead of rounding), so |ds| <= 2 (d + 4) u A; a weight exp(s - m) is then off by
2 |ds| relative, plus 2^-20 for the exponential (2^-22), the split of the weight into 16-bit parts (2^-21)
and the final division; the sum over the positions adds 2 u for each of its at most n / 16 + 64 partial
sums.  Each of these enters numerator and denominator once, hence
  |out - ref| <= (4 (d + 4) 2 u A + 2^-19 + (n / 8 + 128) u) sum p |v|,   |lse - ref| the same without |v|.
"""
import ctypes as C

import numpy as np
import pytest
import torch

from oracle import paged

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from kv_cache_quantization_tq_gb300.build import build

    build()
    import kv_cache_quantization_tq_gb300 as tq
else:
    tq = None

U = 2.0 ** -24
FORMS = [(16, False), (16, True), (8, False), (8, True)]


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def dense(d, hq, hkv, bits=16, bf16=False):
    return tq.Context(tq.TQ_LAYOUT_DENSE, d, hq, hkv, key_bits=bits, value_bits=bits,
                      key_format=tq.TQ_ELEM_BF16 if bf16 else tq.TQ_ELEM_F16)


def bits_of(t):
    return t.detach().contiguous().view(torch.int16).cpu().numpy().view(np.uint16)


def elem(bf16):
    return torch.bfloat16 if bf16 else torch.float16


# ---------------------------------------------------------------- store
@pytest.mark.parametrize("bits,bf16", FORMS)
@pytest.mark.parametrize("d,hkv,n", [(64, 1, 1), (64, 3, 37), (128, 4, 33), (128, 8, 5), (256, 2, 19), (512, 1, 7), (512, 3, 18)])
def test_store_matches_the_oracle(d, hkv, n, bits, bf16):
    gen = torch.Generator(device="cuda").manual_seed(d + n)
    nb = n // 16 + 5
    wide = torch.randn(n, 3 * hkv * d + 8, generator=gen, device="cuda") * torch.exp(
        4 * torch.randn(n, 1, generator=gen, device="cuda"))
    wide = wide.to(elem(bf16))
    k = wide[:, hkv * d:2 * hkv * d].view(n, hkv, d)  # rows cut out of a wider tensor
    v = wide[:, 2 * hkv * d:3 * hkv * d].view(n, hkv, d)
    if n > 4:
        k[0, 0] = 0.0
        k[1, 0, :3] = torch.tensor([float("inf"), float("-inf"), float("nan")])
        v[2, -1] = float("inf")
        v[3, 0] = 448.0 * 2.0 ** -6
        v[4, 0] = torch.finfo(elem(bf16)).tiny / 4  # a vector of subnormals
    ctx = dense(d, hkv, hkv, bits, bf16)
    pool = torch.randint(0, 256, (nb, hkv, ctx.page_bytes), generator=gen, device="cuda", dtype=torch.uint8)
    slots = torch.randperm(nb * 16, generator=gen, device="cuda")[:n]
    if n > 6:
        slots[5] = -1
        slots[6] = -(1 << 40)
    ref, flags = paged.store(pool.cpu().numpy(), bits_of(k), bits_of(v), slots.cpu().numpy(), d, bits, bf16)
    ctx.paged_store(k, v, slots, pool)
    assert ctx.device_errors() == 0 == flags
    assert np.array_equal(pool.cpu().numpy(), ref)


def test_store_skips_slots_outside_the_pool():
    ctx = dense(64, 2, 2)
    pool = torch.zeros(3, 2, ctx.page_bytes, dtype=torch.uint8, device="cuda")
    k = torch.ones(4, 2, 64, dtype=torch.float16, device="cuda")
    slots = torch.tensor([48, 1 << 40, 47, (1 << 62)], device="cuda")
    ctx.paged_store(k, k, slots, pool)
    assert ctx.device_errors() == tq.binding.TQ_DEVERR_BLOCK_ID
    rows = pool.view(torch.float16).view(3, 2, 2, 16, 64)
    assert (rows[2, :, :, 15] == 1).all() and int((rows != 0).sum()) == 2 * 2 * 64


# ---------------------------------------------------------------- attention
def make_case(seed, lengths, hq, hkv, d, bits, bf16, max_blocks=None, extra=3, spread=1.0):
    """Shuffled pages; everything that no sequence holds (free pages, rows behind a last token) is NaN."""
    rng = np.random.default_rng(seed)
    gen = torch.Generator().manual_seed(seed)
    used = [-(-n // 16) for n in lengths]
    max_blocks = max_blocks or max(max(used), 1)
    nb = sum(used) + extra
    ids = rng.permutation(nb).astype(np.int32)
    bt = np.full((len(lengths), max_blocks), -1, np.int32)
    at = 0
    for b, u in enumerate(used):
        bt[b, :u] = ids[at:at + u]
        at += u
    slots = np.concatenate([bt[b, np.arange(n) // 16].astype(np.int64) * 16 + np.arange(n) % 16
                            for b, n in enumerate(lengths)] + [np.zeros(0, np.int64)])
    dt = elem(bf16)
    n = len(slots)
    k = (torch.randn(n, hkv, d, generator=gen) * spread).to(dt)
    v = (torch.randn(n, hkv, d, generator=gen) * torch.exp(torch.randn(n, 1, 1, generator=gen))).to(dt)
    q = torch.randn(len(lengths), hq, d, generator=gen).to(dt)
    ctx = dense(d, hq, hkv, bits, bf16)
    pool = torch.full((nb, hkv, ctx.page_bytes), 0xFF, dtype=torch.uint8, device="cuda")
    if n:
        ctx.paged_store(k.cuda(), v.cuda(), torch.from_numpy(slots).cuda(), pool)
        assert ctx.device_errors() == 0
    return dict(ctx=ctx, q=q, pool=pool, bt=bt, lengths=np.array(lengths, np.int32), d=d, bits=bits, bf16=bf16)


def attend(e, window=0, scale=0.0, want_lse=True, q=None, stream=None):
    ctx, bsz = e["ctx"], len(e["lengths"])
    q = e["q"].cuda() if q is None else q
    out = torch.full((bsz, ctx.num_q_heads, e["d"]), float("nan"), dtype=torch.float32, device="cuda")
    lse = torch.full((bsz, ctx.num_q_heads), float("nan"), dtype=torch.float32, device="cuda") if want_lse else None
    ws = torch.full((ctx.paged_workspace_size(bsz),), 0xFF, dtype=torch.uint8, device="cuda")
    ctx.paged_attention(q, e["pool"], torch.from_numpy(e["bt"]).cuda(), torch.from_numpy(e["lengths"]).cuda(), out, ws,
                        lse=lse, window=window, scale=scale, stream=stream)
    return out, lse


def check(e, out, lse, window=0, scale=None, flags=0):
    ctx = e["ctx"]
    assert ctx.device_errors() == flags
    q64 = e["q"].double().numpy()
    ref, rlse, (a, vabs), rflags = paged.attention(q64, e["pool"].cpu().numpy(), e["bt"], e["lengths"], e["d"], e["bits"],
                                                   e["bf16"], window, scale)
    assert rflags == flags
    rel = 8 * (e["d"] + 4) * U * a + 2.0 ** -19 + (max(e["lengths"].max(), 0) / 8 + 128) * U
    got = out.cpu().numpy().astype(np.float64)
    err = np.abs(got - ref)
    assert np.all(err <= rel[..., None] * vabs), f"worst {np.nanmax(err / np.maximum(rel[..., None] * vabs, 1e-300)):.3g} of the bound"
    if lse is not None:
        g = lse.cpu().numpy().astype(np.float64)
        empty = np.isneginf(rlse)
        assert np.array_equal(np.isneginf(g), empty)
        g, r, t = g[~empty], rlse[~empty], rel[~empty]
        assert np.all(np.abs(g - r) <= t + 2 * U * np.abs(r))


SHAPES = [
    (1, 1, 64, [1]), (4, 4, 64, [1, 15, 16, 17, 0, 100]), (8, 2, 64, [500, 3]), (14, 2, 64, [129, 64]),
    (16, 4, 128, [1000]), (28, 4, 128, [37, 0, 400, 16]), (5, 1, 128, [257, 31]), (16, 1, 128, [90, 333]), (33, 3, 128, [70]),
    (24, 1, 128, [64, 130]), (8, 8, 256, [50, 200]), (10, 1, 256, [77]), (16, 2, 256, [300, 1, 0]), (4, 2, 512, [33, 250]),
    (12, 1, 512, [100]), (17, 1, 64, [47, 160]),
]


@pytest.mark.parametrize("bits,bf16", FORMS)
@pytest.mark.parametrize("hq,hkv,d,lengths", SHAPES)
def test_attention_matches_the_oracle(hq, hkv, d, lengths, bits, bf16):
    e = make_case(hq * 7 + d, lengths, hq, hkv, d, bits, bf16)
    check(e, *attend(e))


@pytest.mark.parametrize("bits,bf16", FORMS)
@pytest.mark.parametrize("window", [1, 2, 15, 16, 17, 33, 64, 1000])
def test_attention_window(window, bits, bf16):
    e = make_case(window, [1, 16, 40, 65, 300, 0], 6, 2, 64, bits, bf16)
    check(e, *attend(e, window=window), window=window)


@pytest.mark.parametrize("bits,bf16", FORMS)
def test_attention_long(bits, bf16):
    """Many pages, several parts per sequence, beside short and empty neighbours."""
    e = make_case(11, [9001, 1, 0, 2048, 4095], 8, 1, 128, bits, bf16)
    check(e, *attend(e))


@pytest.mark.parametrize("bits,bf16", FORMS)
@pytest.mark.parametrize("d", [64, 128])
def test_attention_many_sequences(d, bits, bf16):
    """More sequences than the GPU has multiprocessors, of every length around a page's."""
    lengths = [(i * 37) % 83 for i in range(700)]
    e = make_case(13, lengths, 4, 2, d, bits, bf16)
    check(e, *attend(e))


@pytest.mark.parametrize("batch", [1023, 1024, 1025, 2500])
def test_attention_batches_beyond_one_scan(batch):
    lengths = [(i * 7) % 19 for i in range(batch)]
    e = make_case(batch, lengths, 1, 1, 64, 16, False)
    check(e, *attend(e))


@pytest.mark.parametrize("bits,bf16", FORMS)
def test_attention_peaked_and_large_scores(bits, bf16):
    """Keys times 20: scores of hundreds, weights of one position and exact zeros beside it."""
    e = make_case(17, [700, 130], 8, 2, 128, bits, bf16, spread=20.0)
    check(e, *attend(e))


@pytest.mark.parametrize("scale", [0.03, 1.0, -0.2])
def test_attention_scale(scale):
    e = make_case(19, [100, 33], 8, 2, 64, 16, False)
    check(e, *attend(e, scale=scale), scale=scale)


def test_attention_strided_queries_and_no_lse():
    e = make_case(23, [100, 33, 5], 8, 2, 64, 16, True)
    wide = torch.zeros(3, 8 * 64 + 40, dtype=torch.bfloat16, device="cuda")
    wide[:, 16:16 + 512] = e["q"].cuda().view(3, -1)
    q = wide[:, 16:16 + 512].view(3, 8, 64)
    assert q.stride(0) == 552
    out, lse = attend(e, q=q, want_lse=False)
    check(e, out, None)


def test_attention_wide_range_of_value_exponents():
    """8-bit values whose vectors differ by up to 2^60 in size from token to token."""
    gen = torch.Generator().manual_seed(29)
    e = make_case(29, [200, 48], 4, 2, 128, 8, True)
    ctx = e["ctx"]
    k = torch.randn(200, 2, 128, generator=gen).bfloat16().cuda()
    v = (torch.randn(200, 2, 128, generator=gen) * torch.exp2(torch.randint(-30, 31, (200, 1, 1), generator=gen).float())).bfloat16().cuda()
    pos = np.arange(200)
    slots = torch.from_numpy(e["bt"][0, pos // 16].astype(np.int64) * 16 + pos % 16).cuda()
    ctx.paged_store(k, v, slots, e["pool"])
    check(e, *attend(e))


def test_attention_large_and_small_queries_on_8_bit_pages():
    """bf16 queries of 2^60 and 2^-60 against 8-bit keys of the opposite size."""
    e = make_case(31, [90, 90], 4, 2, 64, 8, True)
    ctx = e["ctx"]
    gen = torch.Generator().manual_seed(31)
    pos = np.arange(90)
    for b, f in ((0, 2.0 ** -60), (1, 2.0 ** 60)):
        k = (torch.randn(90, 2, 64, generator=gen) * f).bfloat16().cuda()
        v = torch.randn(90, 2, 64, generator=gen).bfloat16().cuda()
        slots = torch.from_numpy(e["bt"][b, pos // 16].astype(np.int64) * 16 + pos % 16).cuda()
        ctx.paged_store(k, v, slots, e["pool"])
        e["q"][b] = (e["q"][b].float() / f).bfloat16()
    check(e, *attend(e))


def test_attention_nan_of_a_position_stays_in_its_row():
    e = make_case(37, [60, 60, 60], 4, 2, 64, 16, False)
    rows = e["pool"].view(torch.float16).view(-1, 2, 2, 16, 64)
    rows[int(e["bt"][1, 1]), 0, 0, 3, 5] = float("nan")  # a key of sequence 1, KV head 0
    out, lse = attend(e)
    nan = torch.isnan(out).all(-1).cpu()
    assert nan.tolist() == [[False] * 4, [True, True, False, False], [False] * 4]
    assert torch.isfinite(out[nan.cuda().logical_not()]).all()


def test_attention_bad_device_values_are_flagged():
    e = make_case(41, [100, 50, 30, 20], 4, 2, 64, 16, False)
    e["bt"] = e["bt"].copy()
    e["bt"][0, 2], e["bt"][1, 0] = e["pool"].shape[0], -7
    e["lengths"] = np.array([100, 50, -3, 16 * e["bt"].shape[1] + 1], np.int32)
    check(e, *attend(e), flags=paged.ERR_BLOCK_ID | paged.ERR_POSITION)


def test_attention_of_a_pool_without_blocks():
    ctx = dense(64, 4, 2)
    pool = torch.empty(0, 2, ctx.page_bytes, dtype=torch.uint8, device="cuda")
    e = dict(ctx=ctx, q=torch.randn(2, 4, 64).half(), pool=pool, bt=np.zeros((2, 2), np.int32), lengths=np.array([0, 20], np.int32),
             d=64, bits=16, bf16=False)
    check(e, *attend(e), flags=paged.ERR_BLOCK_ID)


def test_attention_refuses_counts_beyond_31_bits():
    e = make_case(42, [5], 4, 2, 64, 16, False)
    for window in (-1, 2 ** 31, 2 ** 32 + 5):
        with pytest.raises(ValueError):
            attend(e, window=window)
    check(e, *attend(e, window=2 ** 31 - 1), window=2 ** 31 - 1)


def test_attention_shared_pages_and_repeated_calls():
    """Two sequences that name the same pages; the same call ten times gives the same bits."""
    e = make_case(43, [400, 400, 333], 8, 2, 128, 16, True)
    e["bt"][1] = e["bt"][0]
    first, lse = attend(e)
    check(e, first, lse)
    for _ in range(9):
        again, lse2 = attend(e)
        assert torch.equal(again, first) and torch.equal(lse2, lse)


def test_attention_keeps_rows_it_does_not_own():
    """Guard bytes behind the workspace and the outputs stay as they were."""
    e = make_case(47, [300, 7], 8, 2, 64, 16, False)
    ctx = e["ctx"]
    n = ctx.paged_workspace_size(2)
    ws = torch.full((n + 256,), 0xAB, dtype=torch.uint8, device="cuda")
    out = torch.full((4, 8, 64), 7.0, device="cuda")
    lse = torch.full((4, 8), 7.0, device="cuda")
    ctx.paged_attention(e["q"].cuda(), e["pool"], torch.from_numpy(e["bt"]).cuda(), torch.from_numpy(e["lengths"]).cuda(), out[:2],
                        ws[:n], lse=lse[:2])
    check(e, out[:2], lse[:2])
    assert (out[2:] == 7).all() and (lse[2:] == 7).all() and (ws[n:] == 0xAB).all()


def test_attention_in_a_graph_and_on_another_stream():
    """One captured call replayed after its inputs changed in place; two streams with a workspace each."""
    e = make_case(53, [300, 7, 0, 64], 8, 2, 128, 16, False)
    ctx, q = e["ctx"], e["q"].cuda()
    bt, ln = torch.from_numpy(e["bt"]).cuda(), torch.from_numpy(e["lengths"]).cuda()
    out, lse = torch.zeros(4, 8, 128, device="cuda"), torch.zeros(4, 8, device="cuda")
    ws = torch.empty(ctx.paged_workspace_size(4), dtype=torch.uint8, device="cuda")
    ctx.paged_attention(q, e["pool"], bt, ln, out, ws, lse=lse)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        ctx.paged_attention(q, e["pool"], bt, ln, out, ws, lse=lse)
    for lengths in ([300, 7, 0, 64], [12, 0, 0, 33], [160, 7, 0, 1]):
        e["lengths"] = np.array(lengths, np.int32)
        ln.copy_(torch.from_numpy(e["lengths"]))
        e["q"] = torch.randn(4, 8, 128).half()
        q.copy_(e["q"])
        out.fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        check(e, out, lse)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [attend(e, stream=s, q=q) for s in streams]
    torch.cuda.synchronize()
    for o, l in got:
        check(e, o, l)


def test_attention_line_beyond_31_bits():
    """A block table so long that the work line of all pages it allows counts two pages as one."""
    hkv, d, maxb = 64, 64, 2_200_000
    e = make_case(59, [3000 - 177 * i for i in range(16)], hkv, hkv, d, 16, False, max_blocks=maxb)
    assert 16 * hkv * maxb > 2 ** 31
    check(e, *attend(e))
    check(e, *attend(e, window=70), window=70)


def test_page_offsets_beyond_32_bits():
    """Pages behind the first 4 GiB of the pool."""
    d, hkv = 512, 2
    ctx = dense(d, 4, hkv)
    nb = (5 << 30) // (hkv * ctx.page_bytes)
    pool = torch.empty(nb, hkv, ctx.page_bytes, dtype=torch.uint8, device="cuda")
    bt = np.array([[nb - 1, 3, nb - 2], [nb // 2, nb - 5, 0]], np.int32)
    lengths = np.array([40, 33], np.int32)
    pos = [np.arange(n) for n in lengths]
    slots = torch.from_numpy(np.concatenate([bt[b, p // 16].astype(np.int64) * 16 + p % 16 for b, p in enumerate(pos)])).cuda()
    k = torch.randn(73, hkv, d).half()
    v = torch.randn(73, hkv, d).half()
    ctx.paged_store(k.cuda(), v.cuda(), slots, pool)
    ids = sorted(set(bt.flatten().tolist()))
    small = {i: j for j, i in enumerate(ids)}
    e = dict(ctx=ctx, q=torch.randn(2, 4, d).half(), pool=pool, bt=bt, lengths=lengths, d=d, bits=16, bf16=False)
    out, lse = attend(e)
    e["bt"] = np.vectorize(small.get)(bt).astype(np.int32)
    e["pool"] = pool[torch.tensor(ids, device="cuda")]
    check(e, out, lse)


# ---------------------------------------------------------------- plan
def run_plan(ctx, ctx_len, new_len, table, queue, state, num_blocks, max_tokens, ring, optional=True):
    bsz = len(ctx_len)
    dev = lambda x: torch.from_numpy(np.array(x)).cuda()  # noqa: E731
    i32 = lambda n: torch.full((n,), 77, dtype=torch.int32, device="cuda")  # noqa: E731
    r = dict(block_table=dev(np.asarray(table, np.int32)), queue=dev(np.asarray(queue, np.int32)), lengths=i32(bsz),
             token_start=i32(bsz + 1), slots=torch.full((max_tokens,), 77, dtype=torch.int64, device="cuda"), queue_state=i32(2))
    if optional:
        r.update(positions=i32(max_tokens), rows=i32(max_tokens), n_paged=i32(bsz), n_ring=i32(bsz))
    ctx.plan_pages(dev(np.asarray(ctx_len, np.int32)), dev(np.asarray(new_len, np.int32)), r["block_table"], r["queue"],
                   dev(np.asarray(state, np.int32)), r["lengths"], r["token_start"], r["slots"], r["queue_state"],
                   num_blocks=num_blocks, ring_capacity=ring, **{k: r[k] for k in ("positions", "rows", "n_paged", "n_ring") if k in r})
    return r


def check_plan(ctx, *args, optional=True):
    args = [np.asarray(a, np.int32) if i < 5 else a for i, a in enumerate(args)]
    ref = paged.plan(*args)
    got = run_plan(ctx, *args, optional=optional)
    assert ctx.device_errors() == ref["flags"]
    for name, t in got.items():
        assert np.array_equal(t.cpu().numpy(), ref[name]), name
    return ref


@pytest.mark.parametrize("ring", [0, 128])
@pytest.mark.parametrize("batch,most,maxb,nb,max_tokens", [
    (1, 1, 4, 10, 1), (3, 40, 8, 30, 100), (9, 60, 40, 150, 400), (64, 1, 20, 900, 64), (300, 200, 30, 3000, 40000),
    (1500, 20, 12, 9000, 20000), (2100, 3, 12, 9000, 5000),
])
def test_plan_steps(batch, most, maxb, nb, max_tokens, ring):
    """A run of steps, each from the last one's outputs, with ended requests and, now and then, refusals."""
    rng = np.random.default_rng(batch + ring)
    ctx = dense(64, 1, 1)
    table, queue, state = np.full((batch, maxb), -1, np.int32), rng.permutation(nb).astype(np.int32), [nb // 3, nb]
    lens = np.zeros(batch, np.int32)
    for step in range(12):
        new = rng.integers(0, most + 1, batch).astype(np.int32)
        new[rng.random(batch) < 0.08] = -1
        r = check_plan(ctx, lens, new, table, queue, state, nb, max_tokens, ring)
        table, queue, state, lens = r["block_table"], r["queue"], r["queue_state"], r["lengths"]


@pytest.mark.parametrize("skew", [0, 1])
def test_plan_large_prefill(skew):
    """More tokens than the grid has threads, the token buffers 16-byte aligned and not."""
    ctx = dense(64, 1, 1)
    ctx_len, new = np.array([5, 0, 700, 31], np.int32), np.array([200001, 3, -1, 199990], np.int32)
    nb, maxb, cap, n = 30000, 13000, 30000, 400003
    held = np.full((4, maxb), -1, np.int32)
    held[0, 0], held[2, :44], held[3, :2] = 29000, np.arange(29001, 29045), [29100, 29101]
    queue, state = np.arange(cap, dtype=np.int32) % 28000, np.array([3000, 26000], np.int32)
    ref = paged.plan(ctx_len, new, held, queue, state, nb, n)
    dev = lambda x: torch.from_numpy(x.copy()).cuda()  # noqa: E731
    at = lambda dt: torch.full((n + skew,), 77, dtype=dt, device="cuda")[skew:]  # noqa: E731
    r = dict(block_table=dev(held), queue=dev(queue), lengths=torch.zeros(4, dtype=torch.int32, device="cuda"),
             token_start=torch.zeros(5, dtype=torch.int32, device="cuda"), slots=at(torch.int64), positions=at(torch.int32),
             rows=at(torch.int32), queue_state=torch.zeros(2, dtype=torch.int32, device="cuda"))
    ctx.plan_pages(dev(ctx_len), dev(new), r["block_table"], r["queue"], dev(state), r["lengths"], r["token_start"], r["slots"],
                   r["queue_state"], num_blocks=nb, positions=r["positions"], rows=r["rows"])
    assert ctx.device_errors() == ref["flags"]
    for name, t in r.items():
        assert np.array_equal(t.cpu().numpy(), ref[name]), name


def test_plan_sums_beyond_31_bits():
    """Lengths whose sums pass 2^31: what lies behind is refused, what lies in front is served."""
    ctx = dense(64, 1, 1)
    big = 2 ** 31 - 1
    check_plan(ctx, [0, 0, 0, 4], [20, 10 ** 9, 10 ** 9, 3], np.full((4, 4), 2, np.int32), np.arange(8), [0, 8], 10, 50, 0)
    r = run_plan(ctx, [0, 0, 0, 0], [20, big, big, big], np.full((4, 4), 2, np.int32), np.arange(8), [0, 8], 10, 50, 0)
    assert r["lengths"].tolist() == [20, 0, 0, 0] and r["slots"][:20].tolist() == list(range(20)) and (r["slots"][20:] == -1).all()
    assert ctx.device_errors() == paged.ERR_POSITION
    # pages of rows that are all sound: 6 x 2^27 / 16 ... more than the queue has, more than 2^31 tokens in all
    lens = run_plan(ctx, [0] * 5, [2 ** 29] * 5, np.zeros((5, 1), np.int32), np.arange(8), [0, 8], 10, 50, 0)["lengths"]
    assert lens.tolist() == [0] * 5 and ctx.device_errors() == paged.ERR_POSITION


def test_plan_refusals_and_bad_values():
    ctx = dense(64, 1, 1)
    none = np.full((4, 4), -1, np.int32)
    held = np.where(np.arange(4)[:, None] == 2, 9, none)
    check_plan(ctx, [0, 0, 3, 0], [40, 33, 2, 1], held, np.arange(5), [3, 5], 10, 100, 0)     # too few pages
    check_plan(ctx, [0, -4], [65, 1], none[:2], np.arange(5), [0, 5], 10, 100, 0)             # beyond the row, negative
    check_plan(ctx, [0], [1], none[:1], np.arange(5), [0, 6], 10, 100, 0)                     # a state that is none
    check_plan(ctx, [0], [1], none[:1], np.arange(5), [5, 1], 10, 100, 0)
    check_plan(ctx, [0, 0, 0], [10, 10, 0], none[:3], np.arange(5), [0, 5], 10, 15, 0)        # too few token rows
    check_plan(ctx, [0, 20], [20, 5], [[-1, -1], [7, 12]], [3, 99, -2, 4], [0, 4], 10, 30, 0)  # ids that are no blocks
    check_plan(ctx, [64, 10], [-1, 3], held[:2] * 0 + 1, np.arange(5), [1, 3], 10, 30, 0)     # no room for pages given back
    check_plan(ctx, [2 ** 31 - 1], [5], none[:1], np.arange(5), [1, 3], 10, 30, 0)
    check_plan(ctx, [5, 3], [0, 0], none[:2], np.arange(5), [1, 3], 10, 0, 0)                 # no tokens at all
    check_plan(ctx, [5, 3], [1, 1], none[:2] + 3, np.arange(5), [1, 3], 10, 9, 0, )
    got = run_plan(ctx, [5, 3], [1, 1], none[:2] + 3, np.arange(5), [1, 3], 10, 9, 0, optional=False)
    assert got["slots"].tolist() == [37, 35] + [-1] * 7 and ctx.device_errors() == 0
    empty = run_plan(ctx, [], [], np.zeros((0, 4)), np.arange(5), [1, 3], 10, 9, 0)
    assert empty["token_start"].tolist() == [0] and empty["queue_state"].tolist() == [1, 3]
    assert (empty["slots"] == -1).all() and (empty["rows"] == -1).all()


def test_refused_calls():
    ctx = dense(64, 4, 2)
    lib, B = tq.lib, tq.binding
    buf = torch.zeros(1 << 16, dtype=torch.uint8, device="cuda")
    p, odd = C.c_void_p(buf.data_ptr()), C.c_void_p(buf.data_ptr() + 8)
    n, bad = None, B.TQ_ERR_INVALID_ARG
    att = lambda **k: lib.tq_paged_attention(  # noqa: E731
        k.get("ctx", ctx).ptr, k.get("q", p), k.get("qs", 256), k.get("batch", 1), k.get("pool", p), k.get("nb", 1), k.get("bt", p),
        k.get("mb", 1), k.get("len", p), k.get("window", 0), k.get("scale", 0.0), k.get("out", p), n, k.get("ws", p),
        k.get("size", 1 << 30), n)
    assert att(batch=0) == B.TQ_OK
    for k in (dict(batch=-1), dict(nb=-1), dict(mb=-1), dict(window=-1), dict(q=n), dict(q=odd), dict(qs=255), dict(qs=248), dict(qs=-256),
              dict(pool=n), dict(pool=odd), dict(bt=n), dict(len=n), dict(out=n), dict(out=odd), dict(scale=float("nan")),
              dict(scale=float("inf")), dict(ws=odd), dict(nb=2 ** 31 - 1), dict(mb=2 ** 31 - 1)):
        assert att(**k) == bad, k
    assert att(size=16) == att(ws=n) == B.TQ_ERR_WORKSPACE
    main = tq.Context(tq.TQ_LAYOUT_MAIN, 64, 4, 2)
    assert att(ctx=main) == B.TQ_ERR_UNSUPPORTED
    sto = lambda **k: lib.tq_paged_store(  # noqa: E731
        k.get("ctx", ctx).ptr, k.get("k", p), k.get("v", p), k.get("ks", 128), k.get("vs", 128), k.get("slots", p), k.get("n", 1),
        k.get("pool", p), k.get("nb", 1), n)
    assert sto(n=0) == B.TQ_OK and sto(ctx=main) == B.TQ_ERR_UNSUPPORTED
    for k in (dict(n=-1), dict(nb=-1), dict(k=n), dict(v=odd), dict(ks=120), dict(vs=132), dict(slots=n), dict(pool=odd)):
        assert sto(**k) == bad, k
    pln = lambda **k: lib.tq_plan_pages(  # noqa: E731
        ctx.ptr, k.get("c", p), p, k.get("batch", 1), k.get("ring", 0), k.get("bt", p), k.get("mb", 1), k.get("nb", 1), k.get("q", p),
        k.get("cap", 1), k.get("st", p), k.get("len", odd), n, n, k.get("ts", odd), k.get("slots", odd), n, n, k.get("mt", 1),
        k.get("so", odd), n)
    assert pln(ring=64) == B.TQ_ERR_UNSUPPORTED
    for k in (dict(batch=-1), dict(mb=-1), dict(nb=-1), dict(cap=-1), dict(mt=-1), dict(c=n), dict(bt=n), dict(q=n), dict(st=n), dict(len=n),
              dict(len=p), dict(ts=n), dict(slots=n), dict(so=n), dict(so=p), dict(mb=2 ** 31 - 1)):
        assert pln(**k) == bad, k
    # the compressed caches' calls do not take dense contexts
    size = C.c_size_t()
    assert lib.tq_workspace_size(ctx.ptr, 1, 16, C.byref(size)) == B.TQ_ERR_UNSUPPORTED
    assert lib.tq_encode_flush(ctx.ptr, p, p, 1, 16, 16, p, p, 1, p, 1, n) == B.TQ_ERR_UNSUPPORTED
    assert lib.tq_append_token(ctx.ptr, p, p, p, 1, p, p, p, 1, p, 1, n) == B.TQ_ERR_UNSUPPORTED
    assert lib.tq_decode_attention(ctx.ptr, p, 1, p, 1, p, 1, p, n, n, n, 16, p, p, 1 << 20, n) == B.TQ_ERR_UNSUPPORTED
    assert lib.tq_decode_attention_static(ctx.ptr, p, 1, p, 1, p, 1, p, n, n, n, 16, p, n) == B.TQ_ERR_UNSUPPORTED
    assert lib.tq_dequantize(ctx.ptr, p, 1, p, 1, p, n, n, n, 1, 16, p, p, n) == B.TQ_ERR_UNSUPPORTED
    assert lib.tq_get_tables(ctx.ptr, n, n, n, n) == B.TQ_ERR_UNSUPPORTED
    assert main.paged_workspace_size is not None
    with pytest.raises(tq.TQError):
        main.paged_workspace_size(1)
    assert ctx.device_errors() == 0 and ctx.launch_count == 0


# ---------------------------------------------------------------- together
@pytest.mark.parametrize("bits,bf16", FORMS)
def test_a_run_of_steps(bits, bf16):
    """Prefill, decode steps, an ended request whose pages another takes: plan, store and attend in a row, the stored
    history held on the host beside it."""
    d, hq, hkv, bsz, nb, maxb = 128, 8, 2, 4, 30, 8
    gen = torch.Generator().manual_seed(61)
    ctx = dense(d, hq, hkv, bits, bf16)
    dt = elem(bf16)
    pool = torch.full((nb, hkv, ctx.page_bytes), 0xFF, dtype=torch.uint8, device="cuda")
    table, queue, state, lens = np.full((bsz, maxb), -1, np.int32), np.arange(nb, dtype=np.int32)[::-1].copy(), [4, nb], np.zeros(bsz, np.int32)
    steps = [[30, 1, 0, 17], [1, 1, 60, 1], [1, -1, 1, 1], [1, 33, 1, 1], [1, 1, 1, -1], [0, 1, 1, 90]]
    for new in steps:
        n = sum(max(x, 0) for x in new)
        r = run_plan(ctx, lens, new, table, queue, state, nb, n + 3, 0)
        assert ctx.device_errors() == 0
        k = torch.randn(n + 3, hkv, d, generator=gen).to(dt).cuda()
        v = torch.randn(n + 3, hkv, d, generator=gen).to(dt).cuda()
        ctx.paged_store(k, v, r["slots"], pool)
        table, queue, state, lens = (r[x].cpu().numpy() for x in ("block_table", "queue", "queue_state", "lengths"))
        e = dict(ctx=ctx, q=torch.randn(bsz, hq, d, generator=gen).to(dt), pool=pool, bt=table, lengths=lens, d=d, bits=bits, bf16=bf16)
        check(e, *attend(e))
        live = np.concatenate([table[b, :-(-int(lens[b]) // 16)] for b in range(bsz)])
        assert len(np.unique(live)) == len(live)


@pytest.mark.parametrize("bits,bf16", FORMS)
def test_captured_decode_steps(bits, bf16):
    """Two decode steps (plan, store, attend; lengths and queue state handed from one to the other and back) in one
    graph, replayed without a synchronisation between its kernels, against the pages as they then stand."""
    d, hq, hkv, bsz, nb, maxb = 64, 6, 3, 5, 60, 10
    gen = torch.Generator().manual_seed(67)
    ctx, dt = dense(d, hq, hkv, bits, bf16), elem(bf16)
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    pool = torch.full((nb, hkv, ctx.page_bytes), 0xFF, dtype=torch.uint8, device="cuda")
    table = torch.full((bsz, maxb), -1, dtype=torch.int32, device="cuda")
    queue, states = torch.randperm(nb, generator=gen).int().cuda(), [i32(7, nb), i32(0, 0)]
    # the two lengths share a line of memory, as slices of one buffer do
    both = torch.zeros(2 * bsz, dtype=torch.int32, device="cuda")
    lens, new = [both[:bsz], both[bsz:]], torch.ones(bsz, dtype=torch.int32, device="cuda")
    starts, slots = torch.zeros(bsz + 1, dtype=torch.int32, device="cuda"), torch.zeros(bsz, dtype=torch.int64, device="cuda")
    kv = [torch.zeros(bsz, 2 * hkv * d, dtype=dt, device="cuda") for _ in range(2)]
    q = [torch.zeros(bsz, hq, d, dtype=dt, device="cuda") for _ in range(2)]
    out = [torch.zeros(bsz, hq, d, device="cuda") for _ in range(2)]
    lse = [torch.zeros(bsz, hq, device="cuda") for _ in range(2)]
    ws = torch.full((ctx.paged_workspace_size(bsz),), 0xFF, dtype=torch.uint8, device="cuda")
    snap = torch.zeros_like(pool)

    def step(i):
        ctx.plan_pages(lens[i], new, table, queue, states[i], lens[1 - i], starts, slots, states[1 - i], num_blocks=nb)
        k, v = kv[i][:, :hkv * d].view(bsz, hkv, d), kv[i][:, hkv * d:].view(bsz, hkv, d)
        ctx.paged_store(k, v, slots, pool)
        ctx.paged_attention(q[i], pool, table, lens[1 - i], out[i], ws, lse=lse[i])

    warm = torch.zeros_like(pool)  # the first calls outside the capture, on a pool of their own
    ctx.paged_attention(q[0], warm, table, lens[0], out[0], ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step(0)
        snap.copy_(pool)
        step(1)
    host = 0
    for _ in range(24):
        for t in kv + q:
            t.copy_(torch.randn(t.shape, generator=gen).to(dt))
        g.replay()
        torch.cuda.synchronize()
        assert ctx.device_errors() == 0
        for i, pages in ((0, snap), (1, pool)):
            host += 1
            e = dict(ctx=ctx, q=q[i].cpu(), pool=pages, bt=table.cpu().numpy(), lengths=np.full(bsz, host, np.int32), d=d, bits=bits, bf16=bf16)
            check(e, out[i], lse[i])
    assert states[0].tolist() == [(7 + bsz * 3) % nb, nb - bsz * 3] and lens[0].tolist() == [48] * bsz


def test_plan_feeds_the_compressed_cache():
    """The ring form of the plan beside tq_append_token and tq_decode_attention of the main layout: 140 decode steps
    from an empty cache, block tables, n_compressed and n_buf all from the plan."""
    from gpu_cases import allclose_report, make_ctx
    from oracle import attention

    d, hq, hkv, bsz, nb, maxb, seed = 64, 4, 2, 2, 20, 10, 3
    cctx, c, s, sk = make_ctx(tq, True, d, hq, hkv, seed)
    gen = torch.Generator().manual_seed(seed)
    pool = torch.zeros(nb, hkv, cctx.page_bytes, dtype=torch.uint8, device="cuda")
    ring_k = torch.zeros(bsz, hkv, 128, d, dtype=torch.float16, device="cuda")
    ring_v = torch.zeros_like(ring_k)
    table, queue, state, lens = np.full((bsz, maxb), -1, np.int32), np.arange(nb, dtype=np.int32), [7, nb], np.zeros(bsz, np.int32)
    for step in range(140):
        r = run_plan(cctx, lens, [1, 1], table, queue, state, nb, 2, 128)
        k, v = (torch.randn(bsz, hkv, d, generator=gen).half().cuda() for _ in range(2))
        cctx.append_token(k, v, torch.from_numpy(lens.copy()).cuda(), ring_k, ring_v, r["block_table"], pool)
        table, queue, state, lens = (r[x].cpu().numpy() for x in ("block_table", "queue", "queue_state", "lengths"))
        if step in (0, 127, 128, 139):
            q = torch.randn(bsz, hq, d, generator=gen).half()
            out = torch.empty(bsz, hq, d, device="cuda")
            ws = torch.empty(cctx.workspace_size(bsz, 256), dtype=torch.uint8, device="cuda")
            cctx.decode_attention(q.cuda(), pool, r["block_table"], r["n_paged"], ring_k, ring_v, r["n_ring"], 256, out, ws)
            assert cctx.device_errors() == 0
            ref = attention.decode_main(q.numpy(), pool.cpu().numpy(), table, r["n_paged"].cpu().numpy(), ring_k.cpu().numpy(),
                                        ring_v.cpu().numpy(), r["n_ring"].cpu().numpy(), s, c, sk, hkv)
            ok, worst, nbad = allclose_report(out.cpu().numpy(), ref)
            assert ok, f"step {step}: max abs err {worst}, {nbad} off"
