"""4-bit pages, capped and biased attention, weight sums and eviction on the GPU against oracle/paged.py.

Tolerances (derived, not fitted).  Store, eviction and the return of pages give whole numbers and copies: equal byte for byte.
Attention: the bound of test_gpu_paged.py, |out - ref| <= rel sum p |v| with rel = 8 (d + 4) u A + 2^-19 + (n / 8 + 128) u,
u = 2^-24, A the largest sum of a score's magnitudes.  4-bit elements are code x scale, 6 bits, exact in fp16, so nothing is added
for them.  A cap's tanh is within 4e-7 < 7 u of the result and the slopes' products, the constants and the sum within 5 u of the
magnitudes, all of which A holds (tanh x <= x): with the factor 2 of numerator and denominator 24 u A more.
Weight sums: a score is off by ds = (2 (d + 4) + 12) u A, the log-sum-exp it is taken from by 2 u |lse| in its split and the
difference, the exponential by 2^-22, the sum over h heads and the fading by (h + 3) u of the result:
  |got - ref| <= added (2 ds + 4 u |lse| + 2^-20) + (h + 3) u |ref|.
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
    from test_gpu_paged import attend, bits_of, check, dense, elem, make_case
else:
    tq = None

U = 2.0 ** -24
ALL = [(16, False), (16, True), (8, False), (8, True), (4, False), (4, True)]


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


# ---------------------------------------------------------------- store
@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("d,hkv,n", [(64, 1, 1), (64, 3, 37), (128, 4, 33), (128, 8, 700), (256, 2, 19), (512, 1, 7), (512, 3, 18)])
def test_store4_matches_the_oracle(d, hkv, n, bf16):
    gen = torch.Generator(device="cuda").manual_seed(d + n)
    nb = n // 16 + 5
    wide = torch.randn(n, 3 * hkv * d + 8, generator=gen, device="cuda") * torch.exp(4 * torch.randn(n, 1, generator=gen, device="cuda"))
    wide = wide.to(elem(bf16))
    k = wide[:, hkv * d:2 * hkv * d].view(n, hkv, d)  # rows cut out of a wider tensor
    v = wide[:, 2 * hkv * d:3 * hkv * d].view(n, hkv, d)
    if n > 4:
        k[0, 0] = 0.0
        k[1, 0, :3] = torch.tensor([float("inf"), float("-inf"), float("nan")])
        k[1, 0, 16:18] = torch.tensor([float("inf"), -1.0])
        k[2, -1, 40:48] = -0.0
        v[2, -1] = float("inf")
        v[2, 0] = float("nan")
        v[3, 0] = 2688.0 * 2.0 ** -6
        v[4, 0] = torch.finfo(elem(bf16)).tiny / 4  # a vector of subnormals
        v[1, 0, 16:] *= 2.0 ** -20  # blocks whose scale is 0 beside a large one
    ctx = dense(d, hkv, hkv, 4, bf16)
    pool = torch.randint(0, 256, (nb, hkv, ctx.page_bytes), generator=gen, device="cuda", dtype=torch.uint8)
    slots = torch.randperm(nb * 16, generator=gen, device="cuda")[:n]
    if n > 6:
        slots[5] = -1
        slots[6] = -(1 << 40)
    ref, flags = paged.store(pool.cpu().numpy(), bits_of(k), bits_of(v), slots.cpu().numpy(), d, 4, bf16)
    ctx.paged_store(k, v, slots, pool)
    assert ctx.device_errors() == 0 == flags
    assert np.array_equal(pool.cpu().numpy(), ref)


@pytest.mark.parametrize("bf16", [False, True])
def test_store4_where_rounding_is_decided(bf16):
    """Entries on the middles between two magnitudes, for every scale, and their neighbours on both sides; block maxima on the
    middles between two scales."""
    d, rows = 64, []
    mids = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0])
    scales = paged.e4m3_value(np.arange(1, 0x7F))
    step = 2.0 ** -7 if bf16 else 2.0 ** -10
    for s in scales:
        for f in (1.0, 1 - step, 1 + step, 1 - 2 * step):
            x = np.zeros(64)
            x[0] = 2688.0  # e = 0, so that the other blocks' scales are what they are set to
            x[16], x[17:24] = 6 * s, mids * s * f
            x[32], x[33:40] = -6 * s, -mids * s * f
            x[48] = 6 * s * (1 + 2.0 ** -4) * f
            rows.append(x)
    x = torch.from_numpy(np.array(rows)).to(elem(bf16))[:, None]
    n = x.shape[0]
    ctx = dense(d, 1, 1, 4, bf16)
    pool = torch.zeros(n // 16 + 1, 1, ctx.page_bytes, dtype=torch.uint8, device="cuda")
    slots = torch.arange(n, device="cuda")
    ref, _ = paged.store(pool.cpu().numpy(), bits_of(x), bits_of(-x), slots.cpu().numpy(), d, 4, bf16)
    ctx.paged_store(x.cuda(), (-x).cuda(), slots, pool)
    assert np.array_equal(pool.cpu().numpy(), ref)


@pytest.mark.parametrize("bf16", [False, True])
def test_store4_every_finite_value(bf16):
    """All finite 16-bit patterns, in vectors beside entries of other sizes."""
    bits = np.arange(65536, dtype=np.uint16)
    f = paged.to_f64(bits, bf16)
    bits = bits[np.isfinite(f)]
    rng = np.random.default_rng(5)
    near = np.concatenate([bits[:bits.size // 64 * 64], rng.permutation(bits)[:bits.size // 64 * 64]]).reshape(-1, 1, 64)
    x = torch.from_numpy(near.view(np.int16).copy()).view(elem(bf16))
    n = x.shape[0]
    ctx = dense(64, 1, 1, 4, bf16)
    pool = torch.zeros(n // 16 + 1, 1, ctx.page_bytes, dtype=torch.uint8, device="cuda")
    slots = torch.arange(n, device="cuda")
    ref, _ = paged.store(pool.cpu().numpy(), near, near, slots.cpu().numpy(), 64, 4, bf16)
    ctx.paged_store(x.cuda(), x.cuda(), slots, pool)
    assert np.array_equal(pool.cpu().numpy(), ref)


# ---------------------------------------------------------------- attention from 4-bit pages
SHAPES = [
    (1, 1, 64, [1]), (4, 4, 64, [1, 15, 16, 17, 0, 100]), (8, 2, 64, [500, 3]), (14, 2, 64, [129, 64]),
    (16, 4, 128, [1000]), (28, 4, 128, [37, 0, 400, 16]), (5, 1, 128, [257, 31]), (16, 1, 128, [90, 333]), (33, 3, 128, [70]),
    (24, 1, 128, [64, 130]), (8, 8, 256, [50, 200]), (10, 1, 256, [77]), (16, 2, 256, [300, 1, 0]), (4, 2, 512, [33, 250]),
    (12, 1, 512, [100]), (17, 1, 64, [47, 160]),
]


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("hq,hkv,d,lengths", SHAPES)
def test_attention4_matches_the_oracle(hq, hkv, d, lengths, bf16):
    e = make_case(hq * 7 + d, lengths, hq, hkv, d, 4, bf16)
    check(e, *attend(e))


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("window", [1, 2, 15, 16, 17, 33, 64, 1000])
def test_attention4_window(window, bf16):
    e = make_case(window, [1, 16, 40, 65, 300, 0], 6, 2, 64, 4, bf16)
    check(e, *attend(e, window=window), window=window)


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("d,rep", [(64, 8), (64, 16), (128, 8), (128, 16), (256, 4), (256, 9), (512, 3)])
def test_attention4_long(d, rep, bf16):
    e = make_case(11, [9001, 1, 0, 2048, 4095], rep, 1, d, 4, bf16)
    check(e, *attend(e))


def test_attention4_many_sequences():
    e = make_case(13, [(i * 37) % 83 for i in range(1100)], 4, 2, 64, 4, False)
    check(e, *attend(e))


@pytest.mark.parametrize("bf16", [False, True])
def test_attention4_peaked_and_large_scores(bf16):
    e = make_case(17, [700, 130], 8, 2, 128, 4, bf16, spread=20.0)
    check(e, *attend(e))


def rewrite(e, b, k, v):
    """New keys and values of sequence b."""
    pos = np.arange(k.shape[0])
    slots = torch.from_numpy(e["bt"][b, pos // 16].astype(np.int64) * 16 + pos % 16).cuda()
    e["ctx"].paged_store(k.to(elem(e["bf16"])).cuda(), v.to(elem(e["bf16"])).cuda(), slots, e["pool"])


def test_attention4_wide_range_of_values():
    """Vectors that differ by up to 2^60 in size from token to token, blocks by up to 2^12 within one."""
    gen = torch.Generator().manual_seed(29)
    e = make_case(29, [200, 48], 4, 2, 128, 4, True)
    v = torch.randn(200, 2, 128, generator=gen) * torch.exp2(torch.randint(-30, 31, (200, 1, 1), generator=gen).float())
    v = (v.view(200, 2, 8, 16) * torch.exp2(-torch.randint(0, 13, (200, 2, 8, 1), generator=gen).float())).view(200, 2, 128)
    rewrite(e, 0, torch.randn(200, 2, 128, generator=gen), v)
    check(e, *attend(e))


def test_attention4_large_and_small_queries():
    e = make_case(31, [90, 90], 4, 2, 64, 4, True)
    gen = torch.Generator().manual_seed(31)
    for b, f in ((0, 2.0 ** -60), (1, 2.0 ** 60)):
        rewrite(e, b, torch.randn(90, 2, 64, generator=gen) * f, torch.randn(90, 2, 64, generator=gen))
    e["q"] = (torch.randn(2, 4, 64, generator=gen) * torch.tensor([2.0 ** 60, 2.0 ** -60])[:, None, None]).bfloat16()
    check(e, *attend(e))


def test_attention4_a_nan_stays_where_it_counts():
    """A NaN in a key makes its head's rows NaN, one in a value 16 dims of them; other heads and sequences keep theirs."""
    e = make_case(37, [40, 40, 40], 4, 2, 64, 4, False)
    ref, _ = attend(e)
    k, v = torch.randn(40, 2, 64), torch.randn(40, 2, 64)
    k[7, 1, 3] = float("nan")
    rewrite(e, 1, k, v)
    k[7, 1, 3] = 0.0
    v[9, 0, 35] = float("nan")
    rewrite(e, 2, k, v)
    out, lse = attend(e)
    assert torch.equal(out[0], ref[0])
    assert torch.isnan(out[1, 2:]).all() and torch.isfinite(out[1, :2]).all() and torch.isnan(lse[1, 2:]).all()
    assert torch.isnan(out[2, :2, 32:48]).all() and torch.isfinite(out[2, 2:]).all() and torch.isfinite(lse[2]).all()
    assert torch.isfinite(out[2, :2, :32]).all() and torch.isfinite(out[2, :2, 48:]).all()


def test_attention4_bad_pages_and_lengths():
    e = make_case(41, [100, 50, 33], 4, 2, 128, 4, False)
    e["bt"][0, 2], e["bt"][2, 0] = e["pool"].shape[0], -7
    e["lengths"][1] = e["bt"].shape[1] * 16 + 1
    check(e, *attend(e), flags=paged.ERR_BLOCK_ID | paged.ERR_POSITION)


def test_attention4_pool_beyond_31_bits():
    """Tiles whose place in the pool passes 2^31 and 2^32 bytes."""
    d, hkv = 128, 8
    ctx = dense(d, 8, hkv, 4)
    nb = (5 << 30) // (hkv * ctx.page_bytes)
    pool = torch.zeros(nb, hkv, ctx.page_bytes, dtype=torch.uint8, device="cuda")
    gen = torch.Generator().manual_seed(43)
    k, v = torch.randn(48, hkv, d, generator=gen).half(), torch.randn(48, hkv, d, generator=gen).half()
    blocks = np.array([nb - 1, 3 * nb // 5, nb // 2], np.int32)
    slots = torch.from_numpy(np.repeat(blocks.astype(np.int64) * 16, 16) + np.tile(np.arange(16), 3)).cuda()
    ctx.paged_store(k.cuda(), v.cuda(), slots, pool)
    small = make_case(43, [48], 8, hkv, d, 4, False)
    rewrite(small, 0, k, v)
    ref = attend(small)
    big = dict(small, ctx=ctx, pool=pool, bt=blocks[None])
    got = attend(big)
    assert ctx.device_errors() == 0 and torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1])


# ---------------------------------------------------------------- capped and biased scores
def attend_scored(e, cap=0.0, slopes=None, window=0, scale=0.0, stream=None):
    ctx, bsz = e["ctx"], len(e["lengths"])
    out = torch.full((bsz, ctx.num_q_heads, e["d"]), float("nan"), dtype=torch.float32, device="cuda")
    lse = torch.full((bsz, ctx.num_q_heads), float("nan"), dtype=torch.float32, device="cuda")
    ws = torch.full((ctx.paged_workspace_size(bsz),), 0xFF, dtype=torch.uint8, device="cuda")
    ctx.paged_attention(e["q"].cuda(), e["pool"], i32(e["bt"]), i32(e["lengths"]), out, ws, lse=lse, window=window, scale=scale,
                        cap=cap, slopes=slopes if slopes is None else slopes.cuda(), stream=stream)
    return out, lse


def check_scored(e, out, lse, cap=0.0, slopes=None, window=0, scale=None):
    assert e["ctx"].device_errors() == 0
    ref, rlse, (a, vabs), _ = paged.attention(e["q"].double().numpy(), e["pool"].cpu().numpy(), e["bt"], e["lengths"], e["d"],
                                              e["bits"], e["bf16"], window, scale, cap, None if slopes is None else slopes.double().numpy())
    rel = (8 * (e["d"] + 4) + 24) * U * a + 2.0 ** -19 + (max(e["lengths"].max(), 0) / 8 + 128) * U
    got, g = out.cpu().numpy().astype(np.float64), lse.cpu().numpy().astype(np.float64)
    assert np.all(np.abs(got - ref) <= rel[..., None] * vabs)
    empty = np.isneginf(rlse)
    assert np.array_equal(np.isneginf(g), empty)
    assert np.all(np.abs(g[~empty] - rlse[~empty]) <= rel[~empty] + 2 * U * np.abs(rlse[~empty]))


def slopes_of(hq, seed=0):
    gen = torch.Generator().manual_seed(seed)
    return torch.exp2(-8.0 * torch.rand(hq, generator=gen)) * torch.where(torch.rand(hq, generator=gen) < 0.2, -1.0, 1.0)


@pytest.mark.parametrize("bits,bf16", ALL)
@pytest.mark.parametrize("cap,biased", [(30.0, False), (1.5, False), (0.0, True), (50.0, True)])
@pytest.mark.parametrize("hq,hkv,d,lengths", [(4, 4, 64, [1, 15, 16, 17, 0, 100]), (28, 4, 128, [37, 0, 400, 16]), (33, 3, 128, [70]),
                                              (16, 1, 64, [90, 333]), (10, 1, 256, [77]), (12, 1, 512, [100])])
def test_scored_matches_the_oracle(hq, hkv, d, lengths, cap, biased, bits, bf16):
    e = make_case(hq * 7 + d, lengths, hq, hkv, d, bits, bf16, spread=4.0)
    s = slopes_of(hq) if biased else None
    check_scored(e, *attend_scored(e, cap, s), cap, s)


@pytest.mark.parametrize("bits,bf16", ALL)
def test_scored_long_with_a_window(bits, bf16):
    e = make_case(53, [5001, 1, 0, 2048], 8, 1, 128, bits, bf16)
    s = slopes_of(8, 1)
    for window in (0, 1000):
        check_scored(e, *attend_scored(e, 20.0, s, window=window), 20.0, s, window=window)


@pytest.mark.parametrize("bits", [16, 4])
def test_scored_small_scores_keep_their_bits(bits):
    """Scores far below the cap: as without one, to the rounding of the scores themselves."""
    e = make_case(59, [300, 44], 8, 2, 64, bits, False, spread=0.01)
    check_scored(e, *attend_scored(e, 2.0 ** 20), 2.0 ** 20)
    check_scored(e, *attend_scored(e, 0.25), 0.25)


def test_scored_infinite_scores_are_capped():
    e = make_case(61, [40], 2, 1, 64, 16, False)
    k, v = torch.zeros(40, 1, 64), torch.randn(40, 1, 64)
    k[3, 0, 0], k[5, 0, 0] = float("inf"), float("-inf")
    e["q"][:] = 0
    e["q"][:, :, 0] = 1.0
    k[:, :, 1:] = 0.0
    rewrite(e, 0, k, v)
    # inf * 1 + 0 * 0: scores inf, -inf and 0
    out, _ = attend_scored(e, 2.0)
    z = np.zeros(40)
    z[3], z[5] = 2.0, -2.0
    w = np.exp(z)
    ref = (w[:, None] * v[:, 0].half().double().numpy()).sum(0) / w.sum()
    assert np.all(np.abs(out[0].cpu().numpy() - ref) <= 2.0 ** -18 * (w[:, None] * np.abs(v[:, 0].numpy())).sum(0) / w.sum())


def test_scored_without_cap_and_slopes_is_plain():
    e = make_case(67, [100, 33], 8, 2, 128, 16, True)
    a, b = attend(e), attend_scored(e)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


# ---------------------------------------------------------------- weight sums
def weights_case(seed, lengths, hq, hkv, d, bits, bf16, n=None, **kw):
    e = make_case(seed, lengths, hq, hkv, d, bits, bf16, **kw)
    n = n or e["bt"].shape[1] * 16
    e["before"] = torch.randn(len(lengths), hkv, n, generator=torch.Generator().manual_seed(seed)).abs()
    return e


def add_weights(e, lse, decay=1.0, window=0, scale=0.0, cap=0.0, slopes=None, before=True, in_place=False, q=None, bt=None, stream=None):
    w = e["before"].cuda() if before else None
    out = w if in_place else torch.full(e["before"].shape, 77.0, device="cuda")
    e["ctx"].paged_weights(e["q"].cuda() if q is None else q, e["pool"], i32(e["bt"]) if bt is None else bt, i32(e["lengths"]), lse, out,
                           weights=w, decay=decay, window=window, scale=scale, cap=cap, slopes=slopes if slopes is None else slopes.cuda(),
                           stream=stream)
    return out


def check_weights(e, got, lse, decay=1.0, window=0, scale=None, cap=0.0, slopes=None, before=True, in_place=False, flags=0):
    assert e["ctx"].device_errors() == flags
    b4 = e["before"].double().numpy() if before else np.zeros(e["before"].shape)
    l64 = lse.double().cpu().numpy()
    ref, a, f = paged.weight_sums(e["q"].double().numpy(), e["pool"].cpu().numpy(), e["bt"], e["lengths"], l64, b4, decay, e["d"],
                                  e["bits"], e["bf16"], window, scale, cap, None if slopes is None else slopes.double().numpy())
    assert f == flags
    rep = e["ctx"].num_q_heads // e["ctx"].num_kv_heads
    lmax = np.where(np.isfinite(l64), np.abs(l64), 0).reshape(len(b4), -1, rep).max(-1)[..., None]
    got = got.cpu().numpy().astype(np.float64)
    lim = min(e["bt"].shape[1] * 16, b4.shape[2])
    for b, n in enumerate(e["lengths"]):
        n = n if 0 <= n <= lim else 0
        r = ref[b, :, :n]
        added = r - decay * b4[b, :, :n]
        tol = added * ((4 * (e["d"] + 4) + 24) * U * a[b, :, :n] + 4 * U * lmax[b] + 2.0 ** -20) + (rep + 3) * U * np.abs(r)
        tol = tol + U * np.abs(decay * b4[b, :, :n]) + 2.0 ** -126  # fp32's subnormal weights are 0
        err = np.abs(got[b, :, :n] - r)
        assert np.all(err <= tol), (b, np.nanmax(err / tol))
        rest = b4[b, :, n:] if in_place else 77.0
        assert np.all(got[b, :, n:] == rest)  # what is behind the last token stays


@pytest.mark.parametrize("bits,bf16", ALL)
@pytest.mark.parametrize("hq,hkv,d,lengths", SHAPES)
def test_weights_match_the_oracle(hq, hkv, d, lengths, bits, bf16):
    e = weights_case(hq * 7 + d, lengths, hq, hkv, d, bits, bf16)
    _, lse = attend(e)
    check_weights(e, add_weights(e, lse, decay=0.75), lse, decay=0.75)


@pytest.mark.parametrize("bits,bf16", ALL)
@pytest.mark.parametrize("window", [1, 15, 16, 17, 64, 1000])
def test_weights_window_cap_and_slopes(window, bits, bf16):
    e = weights_case(window, [1, 16, 40, 65, 300, 0], 6, 2, 64, bits, bf16, spread=3.0)
    s = slopes_of(6, window)
    _, lse = attend_scored(e, 20.0, s, window=window)
    for kw in (dict(decay=0.5), dict(decay=1.0, in_place=True), dict(decay=-0.5, in_place=True), dict(before=False)):
        got = add_weights(e, lse, window=window, cap=20.0, slopes=s, **kw)
        check_weights(e, got, lse, window=window, cap=20.0, slopes=s, **kw)


@pytest.mark.parametrize("bits", [16, 8, 4])
@pytest.mark.parametrize("scale", [0.03, 1.0, -0.2, -1.0])
def test_weights_scale(scale, bits):
    """Any factor, with tokens in front of the window that must get nothing whatever its sign."""
    e = weights_case(103, [100, 33, 7], 8, 2, 64, bits, False)
    for window, cap, s in ((0, 0.0, None), (21, 0.0, None), (21, 10.0, None), (21, 0.0, slopes_of(8))):
        _, lse = attend_scored(e, cap, s, window=window, scale=scale)
        got = add_weights(e, lse, decay=0.5, window=window, scale=scale, cap=cap, slopes=s)
        check_weights(e, got, lse, decay=0.5, window=window, scale=scale, cap=cap, slopes=s)


@pytest.mark.parametrize("bits,bf16", ALL)
@pytest.mark.parametrize("d,rep", [(128, 8), (64, 16), (128, 20)])
def test_weights_long(d, rep, bits, bf16):
    e = weights_case(71, [9001, 1, 0, 2048, 4095], rep, 1, d, bits, bf16)
    _, lse = attend(e)
    got = add_weights(e, lse, before=False)
    check_weights(e, got, lse, before=False)
    sums = got.cpu().numpy().astype(np.float64)
    for b, n in enumerate(e["lengths"]):
        if n:  # the weights of a head add up to 1
            assert abs(sums[b, 0, :n].sum() - rep) <= rep * 1e-4


def test_weights_many_sequences_and_strided_queries():
    e = weights_case(73, [(i * 37) % 83 for i in range(1100)], 4, 2, 64, 16, False)
    _, lse = attend(e)
    wide = torch.zeros(1100, 4 * 64 + 24, dtype=torch.float16, device="cuda")
    wide[:, 8:264] = e["q"].cuda().view(1100, -1)
    check_weights(e, add_weights(e, lse, q=wide[:, 8:264].view(1100, 4, 64)), lse)


def test_weights_rows_longer_and_shorter_than_the_table():
    for n in (40, 1000):
        e = weights_case(79, [100, 37, 40], 4, 2, 64, 16, False, n=n)
        _, lse = attend(e)
        check_weights(e, add_weights(e, lse), lse, flags=paged.ERR_POSITION if n == 40 else 0)


def test_weights_bad_pages_lengths_and_empty_rows():
    e = weights_case(83, [100, 50, 33, 20], 4, 2, 128, 4, False)
    _, lse = attend(e)
    lse[3, 1] = -float("inf")  # no weight
    e["bt"][0, 2], e["bt"][2, 0] = e["pool"].shape[0], -7
    e["lengths"][1] = -3
    check_weights(e, add_weights(e, lse, decay=0.5), lse, decay=0.5, flags=paged.ERR_BLOCK_ID | paged.ERR_POSITION)


def test_weights_of_infinite_keys():
    """An infinite key that one head scores -inf and that heads which are none (of 8) must not turn into NaN."""
    e = weights_case(89, [20], 2, 1, 64, 16, False)
    k = torch.randn(20, 1, 64)
    k[4, 0, 0] = float("-inf")
    rewrite(e, 0, k, torch.randn(20, 1, 64))
    e["q"] = e["q"].abs() + 0.125
    _, lse = attend(e)
    got = add_weights(e, lse, before=False)
    assert torch.isfinite(got[0, 0, :20]).all() and got[0, 0, 4] == 0 and abs(float(got[0, 0, :20].sum()) - 2) < 1e-5


@pytest.mark.parametrize("bits,d,rep", [(4, 64, 4), (4, 128, 8), (4, 256, 16), (4, 512, 4), (16, 128, 8), (8, 512, 4)])
def test_the_wait_limit_is_for_other_pages(bits, d, rep):
    """Long sequences over the same few pages, many rounds of copies a warp: weight sums, and attention from 4-bit pages, wait by
    counting their copies and know no limit."""
    e = weights_case(d + rep, [200, 130], rep, 1, d, bits, False)
    ctx, held = e["ctx"], np.concatenate([e["bt"][0, :12], e["bt"][1, :8]])
    e["lengths"] = np.array([60000, 0, 17, 20000, 31000], np.int32)
    e["bt"] = np.resize(held, (5, 60000 // 16)).astype(np.int32)
    e["q"] = torch.randn(5, rep, d, generator=torch.Generator().manual_seed(d)).half()
    e["before"] = torch.zeros(5, 1, 60000)
    ref = attend(e)
    sums = add_weights(e, ref[1])
    assert ctx.device_errors() == 0 and torch.isfinite(sums).all() and torch.isfinite(ref[0]).all()
    ctx.set_wait_limit(0)
    assert torch.equal(add_weights(e, ref[1]), sums)
    if bits == 4:
        again = attend(e)
        assert torch.equal(again[0], ref[0]) and torch.equal(again[1], ref[1])
    assert ctx.device_errors() == 0


# ---------------------------------------------------------------- eviction
def evict_case(seed, lengths, hkv, d, bits, max_blocks=None, n=None, kind="mixed"):
    rng = np.random.default_rng(seed)
    used = [-(-max(x, 0) // 16) for x in lengths]
    max_blocks = max_blocks or max(max(used), 1)
    nb = sum(used) + 3
    ids, at = rng.permutation(nb).astype(np.int32), 0
    bt = np.full((len(lengths), max_blocks), -1, np.int32)
    for b, u in enumerate(used):
        bt[b, :u] = ids[at:at + u]
        at += u
    n = n or max_blocks * 16
    w = np.exp(2 * rng.standard_normal((len(lengths), hkv, n)))
    if kind == "mixed":
        u = rng.random(w.shape)
        w = np.where(u < 0.2, 0.0, np.where(u < 0.5, np.round(w * 4) / 4, w))
        w = np.where(u > 0.99, -w, w)
    elif kind == "equal":
        w[:] = 0.25
    w = w.astype(np.float32)
    if kind == "mixed":
        u = rng.random(w.shape)
        w[u < 0.01] = np.nan
        w[(u > 0.01) & (u < 0.02)] = -0.0
        w[(u > 0.02) & (u < 0.025)] = np.inf
        w[(u > 0.025) & (u < 0.03)] = -np.inf
    ctx = dense(d, hkv, hkv, bits)
    pool = rng.integers(0, 256, (nb, hkv, ctx.page_bytes), dtype=np.uint8)
    return dict(ctx=ctx, pool=pool, bt=bt, lengths=np.array(lengths, np.int32), w=w, d=d, bits=bits)


def run_evict(e, keep, sinks, recent, stream=None):
    pool, w = torch.from_numpy(e["pool"]).cuda(), torch.from_numpy(e["w"]).cuda()
    out, kept = torch.full_like(w, 77.0), torch.full(w.shape, -5, dtype=torch.int32, device="cuda")
    lens = torch.full((len(e["lengths"]),), -9, dtype=torch.int32, device="cuda")
    e["ctx"].paged_evict(w, pool, i32(e["bt"]), i32(e["lengths"]), i32(np.broadcast_to(np.asarray(keep, np.int32), e["lengths"].shape).copy()),
                         out, lens, kept, sinks=sinks, recent=recent, stream=stream)
    return pool, out, lens, kept


def check_evict(e, got, keep, sinks, recent, flags=0):
    assert e["ctx"].device_errors() == flags
    keep = np.broadcast_to(np.asarray(keep, np.int32), e["lengths"].shape)
    r = paged.evict(e["w"], e["pool"], e["bt"], e["lengths"], keep, sinks, recent, e["d"], e["bits"])
    assert r["flags"] == flags
    pool, out, lens, kept = (x.cpu().numpy() for x in got)
    assert np.array_equal(lens, r["lengths"])
    for b in range(len(lens)):
        for h in range(out.shape[1]):
            k, s = r["kept"][b][h], r["weights"][b][h]
            assert np.array_equal(kept[b, h, :len(k)], k) and np.all(kept[b, h, len(k):] == -5)
            assert np.array_equal(out[b, h, :len(s)].view(np.int32), s.view(np.int32)) and np.all(out[b, h, len(s):] == 77.0)
    assert np.array_equal(pool, r["pool"])


EVICT = [([100], 1, 40, 0, 0), ([1, 0, 17, 300], 2, 16, 4, 8), ([500, 3, 64], 3, 100, 0, 100), ([200], 2, 0, 4, 4), ([77, 90], 1, 1000, 1, 1),
         ([333, 16, 15], 2, 5, 10, 2), ([48], 4, 47, 0, 1), ([48, 31], 1, -3, 1, 0), ([640], 1, 639, 0, 0)]


@pytest.mark.parametrize("d", [64, 128, 256, 512])
@pytest.mark.parametrize("bits", [16, 8, 4])
@pytest.mark.parametrize("lengths,hkv,keep,sinks,recent", EVICT)
def test_evict_matches_the_oracle(lengths, hkv, keep, sinks, recent, bits, d):
    e = evict_case(d + keep, lengths, hkv, d, bits)
    check_evict(e, run_evict(e, keep, sinks, recent), keep, sinks, recent)


@pytest.mark.parametrize("bits", [16, 8, 4])
@pytest.mark.parametrize("kind", ["mixed", "equal", "plain"])
def test_evict_long_rows(kind, bits):
    """Slices beyond what a CTA holds of keys, several rounds of moves."""
    e = evict_case(3, [120001, 9000, 31], 1, 64, bits, kind=kind)
    for keep, sinks, recent in ((9000, 4, 100), (70000, 0, 0)):
        check_evict(e, run_evict(e, keep, sinks, recent), keep, sinks, recent)


@pytest.mark.parametrize("rows,hkv", [(19, 4), (40, 4), (100, 4), (350, 2)])
def test_evict_batches_of_every_cluster_size(rows, hkv):
    lengths = [(i * 53) % 401 for i in range(rows)]
    keep = [(i * 29) % 300 for i in range(rows)]
    e = evict_case(rows, lengths, hkv, 64, 16)
    check_evict(e, run_evict(e, keep, 2, 16), keep, 2, 16)


def test_evict_many_rows_with_long_ones_among_them():
    """More rows than the GPU has room for at once, some longer than a CTA holds."""
    lengths = [(i * 37) % 90 for i in range(160)]
    lengths[3], lengths[77], lengths[159] = 11003, 20001, 10241
    e = evict_case(17, lengths, 2, 64, 4)
    keep = [40] * 160
    keep[3], keep[77], keep[159] = 5000, 19990, 1
    check_evict(e, run_evict(e, keep, 3, 9), keep, 3, 9)


@pytest.mark.parametrize("bits", [16, 4])
def test_evict_and_weights_in_a_pool_beyond_32_bits(bits):
    """Tiles whose place in the pool passes 2^31 and 2^32 bytes: the same as in a small pool."""
    hkv, d = 4, 128
    small = evict_case(19, [100, 70], hkv, d, bits, kind="plain")
    ctx = small["ctx"]
    nb = (5 << 30) // (hkv * ctx.page_bytes)
    rng = np.random.default_rng(3)
    # pages of real keys and values, for the weights
    gen = torch.Generator().manual_seed(3)
    k, v = torch.randn(170, hkv, d, generator=gen).half().cuda(), torch.randn(170, hkv, d, generator=gen).half().cuda()
    slots = np.concatenate([small["bt"][b, np.arange(n) // 16].astype(np.int64) * 16 + np.arange(n) % 16 for b, n in enumerate([100, 70])])
    pool = torch.from_numpy(small["pool"]).cuda()
    ctx.paged_store(k, v, torch.from_numpy(slots).cuda(), pool)
    small["pool"] = pool.cpu().numpy()
    far = np.concatenate([np.linspace(0, nb - 1, len(small["pool"]), dtype=np.int64)])
    far = rng.permutation(far).astype(np.int32)
    big_pool = torch.zeros(nb, hkv, ctx.page_bytes, dtype=torch.uint8, device="cuda")
    big_pool[torch.from_numpy(far).long().cuda()] = pool
    bt = np.where(small["bt"] >= 0, far[small["bt"]], -1).astype(np.int32)
    q = torch.randn(2, hkv, d, generator=gen).half().cuda()
    lens, n = i32(small["lengths"]), small["w"].shape[2]
    got = []
    for p, t in ((pool, small["bt"]), (big_pool, bt)):
        out, lse = torch.zeros(2, hkv, d, device="cuda"), torch.zeros(2, hkv, device="cuda")
        ws = torch.zeros(ctx.paged_workspace_size(2), dtype=torch.uint8, device="cuda")
        ctx.paged_attention(q, p, i32(t), lens, out, ws, lse=lse)
        w, w2 = torch.zeros(2, hkv, n, device="cuda"), torch.zeros(2, hkv, n, device="cuda")
        ctx.paged_weights(q, p, i32(t), lens, lse, w)
        kept, new = torch.zeros(2, hkv, n, dtype=torch.int32, device="cuda"), i32([0, 0])
        ctx.paged_evict(w, p, i32(t), lens, i32([50, 33]), w2, new, kept, sinks=2, recent=10)
        ctx.paged_attention(q, p, i32(t), new, out, ws, lse=lse)
        got.append((out, lse, w, w2, kept, new))
    assert ctx.device_errors() == 0
    for x, y in zip(*got):
        assert torch.equal(x, y)


def test_two_calls_at_once():
    """The same context on two streams: calls that share only what they read."""
    e = weights_case(101, [3000, 130, 9, 2000], 8, 2, 128, 4, False)
    f = evict_case(23, [700, 90, 300], 4, 128, 8, kind="plain")
    ref, lse = attend_scored(e, 10.0, slopes_of(8))
    sums = add_weights(e, lse)
    gone = run_evict(f, 60, 1, 8)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    got = []
    for _ in range(10):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got.append((attend_scored(e, 10.0, slopes_of(8))[0], add_weights(e, lse), *run_evict(f, 60, 1, 8)))
    torch.cuda.synchronize()
    for out, w, *rest in got:
        assert torch.equal(out, ref) and torch.equal(w, sums)
        assert all(torch.equal(x, y) for x, y in zip(rest, gone))


def test_evict_rows_longer_and_shorter_than_the_table():
    e = evict_case(5, [100, 37], 2, 64, 16, max_blocks=9, n=300)
    check_evict(e, run_evict(e, 30, 0, 5), 30, 0, 5)
    e = evict_case(5, [100, 37], 2, 64, 16, n=60)
    check_evict(e, run_evict(e, 30, 0, 5), 30, 0, 5, flags=paged.ERR_POSITION)


def test_evict_bad_pages_and_lengths():
    e = evict_case(7, [200, 100, 90, 60], 2, 128, 4)
    e["bt"][0, 1], e["bt"][1, 6] = e["pool"].shape[0], -1
    e["lengths"][2], e["lengths"][3] = -1, e["bt"].shape[1] * 16 + 1
    check_evict(e, run_evict(e, 50, 2, 8), 50, 2, 8, flags=paged.ERR_BLOCK_ID | paged.ERR_POSITION)


def test_evict_again_and_again():
    """One token at a time out of a full cache: what is kept of what was kept."""
    e = evict_case(9, [64], 2, 64, 8, kind="plain")
    for _ in range(5):
        got = run_evict(e, int(e["lengths"][0]) - 1, 1, 4)
        check_evict(e, got, int(e["lengths"][0]) - 1, 1, 4)
        e["pool"], e["w"], e["lengths"] = got[0].cpu().numpy(), got[1].cpu().numpy(), got[2].cpu().numpy()


# ---------------------------------------------------------------- pages given back
def run_release(lengths, new, bt, queue, state, nb):
    ctx = tq.Context(tq.TQ_LAYOUT_DENSE, 64, 1, 1)
    q, out = i32(queue), i32([-4, -4])
    ctx.release_pages(i32(lengths), i32(new), i32(bt), q, i32(state), out, num_blocks=nb)
    return q.cpu().numpy(), out.cpu().numpy(), ctx.device_errors()


@pytest.mark.parametrize("batch", [1, 3, 150, 1000])
def test_release_matches_the_oracle(batch):
    rng = np.random.default_rng(batch)
    maxb = 20
    lengths = rng.integers(0, maxb * 16 + 1, batch)
    new = (lengths * rng.random(batch)).astype(np.int64)
    bt = rng.permutation(batch * maxb).astype(np.int32).reshape(batch, maxb)
    if batch > 2:
        new[1], lengths[2] = lengths[1] + 1, maxb * 16 + 1  # two that give nothing back
        bt[0, :] = -1                                       # pages that are none
    for cap, head, count in ((batch * maxb + 7, batch * maxb - 3, 7), (batch * 2 + 1, 1, batch)):  # the second has too little room
        queue = rng.integers(0, 100, cap).astype(np.int32)
        ref = paged.release(lengths, new, bt, queue, np.array([head, count], np.int32), batch * maxb)
        got = run_release(lengths, new, bt, queue, [head, count], batch * maxb)
        assert got[2] == ref[2] and np.array_equal(got[0], ref[0]) and np.array_equal(got[1], ref[1])


def test_release_with_a_state_that_is_none():
    bt = np.arange(4, dtype=np.int32)[None]
    for state in ([-1, 0], [0, 9], [8, 0], [0, -1]):
        q, s, f = run_release([64], [0], bt, np.arange(8), state, 4)
        assert f == paged.ERR_PAGES and s.tolist() == state and np.array_equal(q, np.arange(8))
    q, s, f = run_release([], [], np.zeros((0, 4), np.int32), np.arange(8), [3, 2], 4)
    assert f == 0 and s.tolist() == [3, 2]


# ---------------------------------------------------------------- a run of them together
@pytest.mark.parametrize("bits,bf16,d,captured", [(16, False, 64, False), (4, True, 128, False), (8, True, 128, True), (4, False, 64, True)])
def test_a_cache_held_small(bits, bf16, d, captured):
    """Prompt, then steps of store, attention, weight sums, eviction and return of the pages, with the pages planned by
    plan_pages; at the end attention over what is left equals the oracle's over the pool, and every page is accounted for."""
    hq, hkv, bsz, keep, maxb, nb = 8, 2, 3, 48, 8, 26
    ctx, gen = dense(d, hq, hkv, bits, bf16), torch.Generator().manual_seed(d)
    dt = elem(bf16)
    pool = torch.zeros(nb, hkv, ctx.page_bytes, dtype=torch.uint8, device="cuda")
    bt, queue = torch.full((bsz, maxb), -1, dtype=torch.int32, device="cuda"), torch.arange(nb, dtype=torch.int32, device="cuda")
    state, state2, state3 = i32([0, nb]), i32([0, 0]), i32([0, 0])
    ctx_len, new_len, lengths, shorter = i32([0] * bsz), i32([100, 7, 64]), i32([0] * bsz), i32([0] * bsz)
    start, rows = torch.zeros(bsz + 1, dtype=torch.int32, device="cuda"), 171
    slots = torch.zeros(rows, dtype=torch.int64, device="cuda")
    k, v = (torch.randn(rows, hkv, d, generator=gen).to(dt).cuda() for _ in range(2))
    q = torch.randn(bsz, hq, d, generator=gen).to(dt).cuda()
    slopes, kp = slopes_of(hq).abs().cuda() / 8, i32([keep] * bsz)
    out = torch.zeros(bsz, hq, d, device="cuda")
    lse, ws = torch.zeros(bsz, hq, device="cuda"), torch.zeros(ctx.paged_workspace_size(bsz), dtype=torch.uint8, device="cuda")
    w1, w2 = torch.zeros(bsz, hkv, maxb * 16, device="cuda"), torch.zeros(bsz, hkv, maxb * 16, device="cuda")
    kept = torch.zeros(bsz, hkv, maxb * 16, dtype=torch.int32, device="cuda")

    def step():
        ctx.plan_pages(ctx_len, new_len, bt, queue, state, lengths, start, slots, state2, num_blocks=nb)
        ctx.paged_store(k, v, slots, pool)
        ctx.paged_attention(q, pool, bt, lengths, out, ws, lse=lse, cap=20.0, slopes=slopes)
        ctx.paged_weights(q, pool, bt, lengths, lse, w1, weights=w1, decay=0.9, cap=20.0, slopes=slopes)
        ctx.paged_evict(w1, pool, bt, lengths, kp, w2, shorter, kept, sinks=2, recent=8)
        ctx.release_pages(lengths, shorter, bt, queue, state2, state3, num_blocks=nb)
        w1.copy_(w2)
        ctx_len.copy_(shorter)
        state.copy_(state3)

    step()  # the prompt
    new_len.fill_(1)
    if captured:
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            step()
    for i in range(40):
        k.copy_(torch.randn(rows, hkv, d, generator=gen).to(dt))
        v.copy_(torch.randn(rows, hkv, d, generator=gen).to(dt))
        q.copy_(torch.randn(bsz, hq, d, generator=gen).to(dt))
        graph.replay() if captured else step()
        if i in (0, 13, 39):
            lens = shorter.cpu().numpy()
            assert np.array_equal(lens, np.minimum([keep, 8 + i, keep], keep))
            held = [bt[b, :-(-int(n) // 16)].cpu().tolist() for b, n in enumerate(lens)]
            head, count = state.cpu().tolist()
            free = queue.cpu().tolist()
            free = [free[(head + j) % nb] for j in range(count)]
            assert sorted(sum(held, []) + free) == list(range(nb))
            ctx.paged_attention(q, pool, bt, shorter, out, ws, lse=lse, cap=20.0, slopes=slopes)
            e = dict(ctx=ctx, q=q.cpu(), pool=pool, bt=bt.cpu().numpy(), lengths=lens, d=d, bits=bits, bf16=bf16)
            check_scored(e, out, lse, 20.0, slopes.cpu())
    assert ctx.device_errors() == 0


def test_a_side_stream_and_repeated_calls_agree():
    e = weights_case(97, [700, 130, 9], 8, 2, 128, 4, False)
    ref = attend_scored(e, 10.0, slopes_of(8))
    sums = add_weights(e, ref[1], cap=10.0, slopes=slopes_of(8))
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(3):
        with torch.cuda.stream(side):
            got = attend_scored(e, 10.0, slopes_of(8))
            more = add_weights(e, got[1], cap=10.0, slopes=slopes_of(8))
        side.synchronize()
        assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1]) and torch.equal(more, sums)


def test_the_profile_counts_attention_alone():
    e = weights_case(107, [300, 20], 8, 2, 64, 16, False)
    ctx = e["ctx"]
    _, lse = attend_scored(e, 5.0)
    ctx.profile_begin()
    attend_scored(e, 5.0)
    for _ in range(3):
        add_weights(e, lse, cap=5.0)
    p = ctx.profile_end()
    assert p["decode_launches"] == 1 and p["merge_launches"] == 1 and p["decode_kernel"] == "paged_kernel"


# ---------------------------------------------------------------- refusals
def test_refusals():
    ctx = dense(64, 4, 2, 4)
    bad, lib, p = tq.binding.TQ_ERR_INVALID_ARG, tq.lib, ctx.ptr
    pool = torch.zeros(4, 2, ctx.page_bytes, dtype=torch.uint8, device="cuda")
    bt, lens = i32([[0, 1]]), i32([20])
    q, out, lse = torch.zeros(1, 4, 64, dtype=torch.float16, device="cuda"), torch.zeros(1, 4, 64, device="cuda"), torch.zeros(1, 4, device="cuda")
    ws, w = torch.zeros(ctx.paged_workspace_size(1), dtype=torch.uint8, device="cuda"), torch.zeros(1, 2, 32, device="cuda")
    for cap in (-1.0, float("inf"), float("nan"), 1e-30, 1e30):
        with pytest.raises(tq.TQError) as x:
            ctx.paged_attention(q, pool, bt, lens, out, ws, cap=cap)
        assert x.value.status == bad
        with pytest.raises(tq.TQError) as x:
            ctx.paged_weights(q, pool, bt, lens, lse, w, cap=cap)
        assert x.value.status == bad
    with pytest.raises(tq.TQError):
        ctx.paged_weights(q, pool, bt, lens, lse, w, decay=float("nan"))
    with pytest.raises(tq.TQError):
        ctx.paged_attention(q, pool, bt, lens, out, ws, cap=2.0 ** -60, scale=2.0 ** 100)
    for call in (lambda: ctx.paged_attention(q, pool, bt, lens, out, ws, slopes=torch.zeros(3, device="cuda")),
                 lambda: ctx.paged_attention(q, pool, bt, lens, out, ws, slopes=torch.zeros(4, dtype=torch.float64, device="cuda")),
                 lambda: ctx.paged_attention(q, pool, bt, lens, out, ws, slopes=torch.zeros(4)),
                 lambda: ctx.paged_weights(q, pool, bt, lens, lse, w[:, :1]),
                 lambda: ctx.paged_weights(q, pool, bt, lens, lse, w, weights=torch.zeros(1, 2, 16, device="cuda")),
                 lambda: ctx.paged_weights(q, pool, bt, lens, lse[:, :2], w),
                 lambda: ctx.paged_weights(q, pool, bt, lens, lse, w.transpose(0, 1)),
                 lambda: ctx.paged_weights(q.bfloat16(), pool, bt, lens, lse, w),
                 lambda: ctx.paged_weights(q, pool[:, :, :-16], bt, lens, lse, w)):
        with pytest.raises(ValueError):
            call()
    kept, lo, w2 = torch.zeros(1, 2, 32, dtype=torch.int32, device="cuda"), i32([0]), torch.zeros(1, 2, 32, device="cuda")
    with pytest.raises(tq.TQError):
        ctx.paged_evict(w, pool, bt, lens, i32([4]), w, lo, kept)
    with pytest.raises(tq.TQError):
        ctx.paged_evict(w, pool, bt, lens, lo, w2, lo, kept)
    for call in (lambda: ctx.paged_evict(w, pool, bt, lens, i32([4]), w2, lo, kept.long()),
                 lambda: ctx.paged_evict(w, pool, bt, lens, i32([4, 4]), w2, lo, kept),
                 lambda: ctx.paged_evict(w, pool, bt, lens, i32([4]), w2, lo, kept[:, :, :16]),
                 lambda: ctx.paged_evict(w, pool, bt, lens, i32([4]), w2, lo, kept, sinks=-1),
                 lambda: ctx.paged_evict(w, pool, bt, lens, i32([4]), w2, lo, kept, recent=1 << 31)):
        with pytest.raises(ValueError):
            call()
    a = lambda t: t.data_ptr()  # noqa: E731
    assert lib.tq_paged_evict(p, a(w), (1 << 30) + 1, 1, a(pool), 4, a(bt), 2, a(lens), a(i32([4])), 0, 0, a(w2), a(lo), a(kept), None) == bad
    assert lib.tq_paged_evict(p, a(w), 32, 1 << 27, a(pool), 4, a(bt), 2, a(lens), a(i32([4])), 0, 0, a(w2), a(lo), a(kept), None) == bad
    assert lib.tq_paged_evict(p, a(w), 32, 0, None, 0, None, 0, None, None, 0, 0, None, None, None, None) == 0
    assert lib.tq_paged_weights(p, a(q), 256, 1, a(pool), 4, a(bt), 2, a(lens), 0, 0.0, 0.0, None, None, None, 1.0, a(w), 32, None) == bad
    state = i32([0, 0])
    with pytest.raises(tq.TQError):
        ctx.release_pages(lens, i32([3]), bt, i32([0] * 4), state, state, num_blocks=4)
    main = tq.Context(tq.TQ_LAYOUT_MAIN, 64, 4, 2)
    n = tq.binding.TQ_ERR_UNSUPPORTED
    assert lib.tq_paged_evict(main.ptr, a(w), 32, 1, a(pool), 4, a(bt), 2, a(lens), a(i32([4])), 0, 0, a(w2), a(lo), a(kept), None) == n
    assert lib.tq_paged_weights(main.ptr, a(q), 256, 1, a(pool), 4, a(bt), 2, a(lens), 0, 0.0, 0.0, None, a(lse), None, 1.0, a(w), 32, None) == n
    size = C.c_size_t()
    assert lib.tq_paged_workspace_size(main.ptr, 1, C.byref(size)) == n
    assert ctx.device_errors() == 0
