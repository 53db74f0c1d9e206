"""The cap of scores where it bends and beyond, with nothing else that is inexact.

Sequences of one token and one query head per KV head, queries and keys of one non-zero entry and a cap that is a power of two:
x = scale q k / cap is exact, and z = cap tanh x is off by the tanh's own error alone, at most E = 2.7e-7 of it (u = 2^-24).
  From 0.9 on, 1 - 2 r with r = 1 / (y + 1), y = e^2x: y is off by 2^-22 (exponential) and 2 |x| u twice (the argument's constant and
product), of which 1 / (1 + e^-2x) reaches r; the sum adds u and the reciprocal 2^-23.  2 r is at most 0.397 of the result, at
0.9, and falls faster than |x| grows; the result's own rounding is at most 0.7 u:
0.397 (0.858 (2^-22 + 3.6 u) + u + 2^-23) + 0.7 u = 2.7e-7.
  Below 0.9 the fit is off by 1.6e-8, the last multiply-add by u, its first factor (at most 0.2 of the result) by 4 u: 1.3e-7.
Weight sums: exp(z - lse) with lse the exact z rounded to fp32: the exponent is near 0, and beside z's error there is the
exponential's 2^-22 and less than that of everything else: |got - exp(z - lse)| <= |z| E + 2^-21.
Attention: the log-sum-exp is z: cap log2 e (constant, product), its product with the tanh, the sum with the logarithm, and ln 2
(constant, product) round once each, the exponential and its logarithm add 2^-21: |got - z| <= |z| (E + 6 u) + 2^-21.
"""
import numpy as np
import pytest
import torch

from test_gpu_small_cache import ALL

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from kv_cache_quantization_tq_gb300.build import build

    build()
    from test_gpu_paged import dense, elem
    from test_gpu_small_cache import i32

U, E = 2.0 ** -24, 2.7e-7


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


@pytest.mark.parametrize("bits,bf16", ALL)
@pytest.mark.parametrize("cap,scale", [(32.0, 1.0), (1.0, 0.25), (64.0, -0.5), (2.0 ** 20, 2.0 ** 18), (2.0 ** 60, 2.0 ** 40), (2.0 ** -60, 2.0 ** -60)])
def test_capped_scores_are_exact_to_the_tanh(cap, scale, bits, bf16):
    """|x| from 2^-10 to 10, every size between alike, and dense around 0.9 where the form changes."""
    rng = np.random.default_rng(bits + bf16)
    n, hkv, d = 4000, 4, 64
    want = np.concatenate([np.exp(rng.uniform(np.log(2.0 ** -10), np.log(10.0), n * hkv // 2)), rng.uniform(0.85, 0.95, n * hkv // 4),
                           rng.uniform(0.0, 10.0, n * hkv // 4)]) * np.where(rng.random(n * hkv) < 0.5, -1.0, 1.0)
    # the key's entry is the largest of its vector and, from 4-bit pages, 6 times a scale; the query takes the rest
    key = rng.choice([6.0, 6.5, 7.0, 3.75, 4.5] if bits > 4 else [6.0, 6.75, 7.5, 5.25, 4.5], n * hkv)
    key_t = torch.from_numpy(key).view(n, hkv)
    unit = 2.0 ** (round(np.log2(cap / abs(scale))) // 2)  # cap / scale is shared by query and key
    q = torch.from_numpy(want / key * (cap / scale) / unit).view(n, hkv).to(elem(bf16))
    k = torch.zeros(n, hkv, d, dtype=elem(bf16))
    k[:, :, 7] = (key_t * unit).to(elem(bf16))
    qq = torch.zeros(n, hkv, d, dtype=elem(bf16))
    qq[:, :, 7] = q
    ctx = dense(d, hkv, hkv, bits, bf16)
    pool = torch.zeros(n, hkv, ctx.page_bytes, dtype=torch.uint8, device="cuda")
    ctx.paged_store(k.cuda(), k.cuda(), torch.arange(n, device="cuda") * 16, pool)
    table, lens = torch.arange(n, dtype=torch.int32, device="cuda")[:, None].contiguous(), i32([1] * n)
    z = cap * np.tanh(scale * q.double().numpy() * k[:, :, 7].double().numpy() / cap)
    assert np.isfinite(z).all() and np.abs(z).max() > 0.99 * cap
    out, lse = torch.zeros(n, hkv, d, device="cuda"), torch.zeros(n, hkv, device="cuda")
    ws = torch.zeros(ctx.paged_workspace_size(n), dtype=torch.uint8, device="cuda")
    ctx.paged_attention(qq.cuda(), pool, table, lens, out, ws, lse=lse, scale=scale, cap=cap)
    err = np.abs(lse.double().cpu().numpy() - z)
    tol = np.abs(z) * (E + 6 * U) + 2.0 ** -21
    assert np.all(err <= tol), f"attention: {np.max(err / tol):.3g} of the bound"
    if cap <= 2.0 ** 10:  # beyond that exp(z - lse) is not near 1
        near = torch.from_numpy(z).float().cuda()
        w = torch.zeros(n, hkv, 16, device="cuda")
        ctx.paged_weights(qq.cuda(), pool, table, lens, near, w, scale=scale, cap=cap)
        ref = np.exp(z - near.double().cpu().numpy())
        err, tol = np.abs(w[:, :, 0].double().cpu().numpy() - ref), np.abs(z) * E + 2.0 ** -21
        assert np.all(err <= tol), f"weight sums: {np.max(err / tol):.3g} of the bound"
    assert ctx.device_errors() == 0


@pytest.mark.parametrize("bits,bf16", ALL)
def test_factors_far_from_the_cap_are_refused(bits, bf16):
    """Where scale / cap has no bits left in fp32 every score would be 0, or 0 times infinity."""
    import kv_cache_quantization_tq_gb300 as tq

    ctx = dense(64, 2, 1, bits, bf16)
    pool = torch.zeros(1, 1, ctx.page_bytes, dtype=torch.uint8, device="cuda")
    table, lens = i32([[0]]), i32([5])
    q, out, lse = torch.ones(1, 2, 64, dtype=elem(bf16), device="cuda"), torch.zeros(1, 2, 64, device="cuda"), torch.zeros(1, 2, device="cuda")
    ws, w = torch.zeros(ctx.paged_workspace_size(1), dtype=torch.uint8, device="cuda"), torch.zeros(1, 1, 16, device="cuda")
    for cap, scale, ok in ((2.0 ** 60, 2.0 ** -90, False), (2.0 ** 60, -2.0 ** -90, False), (2.0 ** 60, 2.0 ** -7, False), (2.0 ** 60, 2.0 ** -6, True),
                           (2.0 ** -60, 2.0 ** 7, False), (2.0 ** -60, -2.0 ** 80, False), (2.0 ** -60, 2.0 ** 6, True), (1.0, 2.0 ** -66, True),
                           (1.0, 2.0 ** 66, True), (1.0, 2.0 ** 67, False)):
        for call in (lambda: ctx.paged_attention(q, pool, table, lens, out, ws, lse=lse, scale=scale, cap=cap),
                     lambda: ctx.paged_weights(q, pool, table, lens, lse, w, scale=scale, cap=cap)):
            if ok:
                call()
            else:
                with pytest.raises(tq.TQError) as x:
                    call()
                assert x.value.status == tq.binding.TQ_ERR_INVALID_ARG
    assert ctx.device_errors() == 0 and torch.isfinite(out).all() and torch.isfinite(w).all()
