"""What the dense-page attention is built to keep: every part of a weight, and the weights' total of long sequences.  The
bounds (paged_cases) are a few units of fp32, tight enough to see either lost; test_paged_precision.py shows on the CPU
that they do."""
import numpy as np
import pytest
import torch

from paged_cases import LIGHT_PAGES, ONE_TOKEN, U, light_tokens, light_tolerance, one_token
from oracle import paged

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from kv_cache_quantization_tq_gb300.build import build

    build()
    from test_gpu_paged import attend, dense, elem, make_case
    from test_gpu_paged_range import fill

FORMS = [(16, False), (16, True), (8, False), (8, True)]


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


@pytest.mark.parametrize("hq,hkv,d", [(4, 2, 64), (24, 1, 64), (8, 2, 128), (32, 2, 128), (3, 1, 256), (12, 1, 256), (5, 1, 512)])
@pytest.mark.parametrize("bits,bf16", FORMS)
def test_one_token_gives_its_values(bits, bf16, hq, hkv, d):
    n = 64
    e = make_case(d + hq, [1] * n, hq, hkv, d, bits, bf16)
    fill(e, *one_token(d + hq, n, hq, hkv, d, elem(bf16)))
    out, _ = attend(e)
    assert e["ctx"].device_errors() == 0
    pool = e["pool"].cpu().numpy()
    v = np.stack([[paged.tile_rows(pool[e["bt"][b, 0], h], d, bits, bf16)[1][0] for h in range(hkv)] for b in range(n)])
    ref = np.repeat(v, hq // hkv, 1)
    err = np.abs(out.cpu().numpy().astype(np.float64) - ref)
    assert np.all(err <= ONE_TOKEN * U * np.abs(ref)), f"{np.nanmax(err / (np.abs(ref) * U + 1e-300)):.3g} u"


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("bits,bf16", FORMS)
def test_total_of_many_light_tokens(bits, bf16, d):
    """4096 sequences of the same 256 pages: one token of weight 1 and 4095 of 3/8 u, all values 1."""
    dt = elem(bf16)
    every = torch.arange(1 << 16, dtype=torch.int32).to(torch.int16).view(dt).float()
    some = every[(every >= 8) & (every < 16)].tolist()
    keys = [float(x) for x in range(8, 16)] if bits == 8 else some
    x, k, off = light_tokens(keys, [float(v) * 2 for v in some][::max(1, len(some) // 128)], d)
    batch, n = 4096, LIGHT_PAGES * 16
    ctx = dense(d, 1, 1, bits, bf16)
    pool = torch.zeros(LIGHT_PAGES, 1, ctx.page_bytes, dtype=torch.uint8, device="cuda")
    kk, vv = torch.full((n, 1, d), k, dtype=dt, device="cuda"), torch.ones(n, 1, d, dtype=dt, device="cuda")
    kk[0] = 0
    ctx.paged_store(kk, vv, torch.arange(n, device="cuda"), pool)
    q = torch.zeros(batch, 1, d, dtype=dt)
    q[:, 0, 5] = x
    bt = np.broadcast_to(np.arange(LIGHT_PAGES, dtype=np.int32), (batch, LIGHT_PAGES)).copy()
    e = dict(ctx=ctx, q=q, pool=pool, bt=bt, lengths=np.full(batch, n, np.int32), d=d, bits=bits, bf16=bf16)
    out, lse = attend(e)
    assert ctx.device_errors() == 0
    tol = light_tolerance(off) * U
    assert float((out.double() - 1).abs().max()) <= tol
    weight = np.exp(x * k / np.sqrt(d))
    assert float((lse.double() - np.log1p((n - 1) * weight)).abs().max()) <= tol
