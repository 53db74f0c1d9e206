"""The oracle of 4-bit pages, capped and biased scores, weight sums and eviction, against brute force and closed forms, and
what the library refuses without a GPU."""
import numpy as np
import pytest

from kv_cache_quantization_tq_gb300 import build

build.build()
import kv_cache_quantization_tq_gb300 as tq  # noqa: E402
from oracle import paged  # noqa: E402

B = tq.binding


def test_e2m1_values_and_codes():
    v = paged.e2m1_value(np.arange(16))
    for c in range(16):  # sign, two exponent bits with bias 1, one fraction bit
        e, f = c >> 1 & 3, c & 1
        x = f * 0.5 if e == 0 else (1 + f / 2) * 2.0 ** (e - 1)
        assert v[c] == (-x if c & 8 else x)
    assert np.array_equal(paged.e2m1_code(v), np.arange(16))
    x = np.linspace(-8, 8, 40001)
    got = paged.e2m1_value(paged.e2m1_code(x))
    assert np.all(np.abs(got - x) <= np.abs(paged.E2M1[None] - np.minimum(np.abs(x), 1e9)[:, None]).min(-1) + 1e-15)
    mid = (paged.E2M1[1:] + paged.E2M1[:-1]) / 2
    assert np.array_equal(paged.e2m1_code(mid), [0, 2, 2, 4, 4, 6, 6]) and np.array_equal(paged.e2m1_code(-mid), [8, 10, 10, 12, 12, 14, 14])
    assert paged.e2m1_code(np.array([-0.0]))[0] == 8 and paged.e2m1_code(np.array([np.inf]))[0] == 7


def test_quantised_vectors_are_near_and_use_the_range():
    rng = np.random.default_rng(1)
    for size in (1e-30, 1e-3, 1.0, 1e6):
        x = rng.standard_normal(128) * size * np.exp(rng.standard_normal(128))
        c, s, e = paged.quantise4(x)
        top = np.abs(x).max()
        assert top <= 2688 * 2.0 ** e and top > 2688 * 2.0 ** (e - 1)
        y = paged.e2m1_value(c) * np.repeat(paged.e4m3_value(s), 16) * 2.0 ** e
        blk = np.repeat(np.abs(x).reshape(-1, 16).max(-1), 16)
        # half of the widest step (4 .. 6) of a scale that is at most 2^-4 off, or the saturation beyond 6
        assert np.all(np.abs(y - x) <= blk / 6 * (1 + 2.0 ** -4) + 2.0 ** (e - 10) * 6)
    c, s, e = paged.quantise4(np.zeros(64))
    assert e == -120 and not c.any() and not s.any()
    x = np.ones(64)
    x[3], x[20], x[40] = np.nan, np.inf, -np.inf
    c, s, e = paged.quantise4(x)
    assert s[0] == 0x7F and not c[:16].any() and s[1] == s[2] == 0x7E and c[20] == 7 and c[40] == 15 and e == -11


def test_capped_and_biased_scores():
    rng = np.random.default_rng(2)
    d, n = 64, 37
    pool = rng.standard_normal((3, 1, 2 * 16 * d)).astype(np.float16).view(np.uint8)
    bt = np.array([[2, 0, 1]], np.int32)
    q, slopes = rng.standard_normal((1, 2, d)) * 3, np.array([0.5, 0.0])
    k = np.concatenate([paged.tile_rows(pool[b, 0], d, 16, False)[0] for b in bt[0]])[:n]
    v = np.concatenate([paged.tile_rows(pool[b, 0], d, 16, False)[1] for b in bt[0]])[:n]
    out, lse, _, flags = paged.attention(q, pool, bt, [n], d, 16, False, cap=2.0, slopes=slopes)
    assert flags == 0
    for h in range(2):
        z = [2.0 * np.tanh(sum(k[p] * q[0, h]) / 8 / 2.0) + slopes[h] * (p - 36) for p in range(n)]
        w = np.exp(z)
        assert np.allclose(out[0, h], (w[:, None] * v).sum(0) / w.sum(), rtol=1e-12) and np.isclose(lse[0, h], np.log(w.sum()))
    # a cap far above the scores is none
    far = paged.attention(q, pool, bt, [n], d, 16, False, cap=1e9)[0]
    assert np.allclose(far, paged.attention(q, pool, bt, [n], d, 16, False)[0], rtol=1e-6)


def test_weight_sums_add_up_to_the_heads():
    rng = np.random.default_rng(3)
    d, lens = 64, [40, 0, 17]
    pool = rng.standard_normal((6, 2, 2 * 16 * d)).astype(np.float16).view(np.uint8)
    bt = np.array([[0, 1, 2], [0, 0, 0], [3, 4, 5]], np.int32)
    q = rng.standard_normal((3, 6, d))
    _, lse, _, _ = paged.attention(q, pool, bt, lens, d, 16, False)
    before = np.ones((3, 2, 48))
    got, _, flags = paged.weight_sums(q, pool, bt, lens, lse, before, 0.25, d, 16, False)
    assert flags == 0
    for b, n in enumerate(lens):
        assert np.allclose(got[b, :, :n].sum(-1), 0.25 * n + (3 if n else 0)) and np.all(got[b, :, n:] == 1)
    assert paged.weight_sums(q, pool, bt, [49, -1, 17], lse, before, 1.0, d, 16, False)[2] == paged.ERR_POSITION


def test_choice_of_what_stays():
    w = np.array([0.5, 0.0, 3.0, 0.5, -0.0, 0.5, np.nan, 9.0, 0.1])
    assert paged.choose(w, 9, 0, 0) == list(range(9)) and paged.choose(w, 99, 5, 5) == list(range(9))
    assert paged.choose(w, 0, 3, 3) == [] and paged.choose(w, -4, 3, 3) == []
    assert paged.choose(w, 3, 0, 0) == [2, 6, 7]            # NaN before all
    assert paged.choose(w, 4, 0, 0) == [0, 2, 6, 7]         # the older of equal ones
    assert paged.choose(w, 4, 2, 1) == [0, 1, 6, 8]
    assert paged.choose(w, 2, 2, 2) == [7, 8]               # the newest before the oldest
    assert paged.choose(w, 3, 2, 2) == [0, 7, 8]
    assert paged.choose(w, 8, 0, 0) == [0, 1, 2, 3, 5, 6, 7, 8]  # -0 counts as 0


def test_eviction_moves_whole_tokens():
    rng = np.random.default_rng(4)
    d = 64
    for bits in (16, 8, 4):
        pool = rng.integers(0, 256, (5, 2, paged.tile_bytes(d, bits)), dtype=np.uint8)
        bt = np.array([[4, 1, 2]], np.int32)
        w = rng.random((1, 2, 48)).astype(np.float32)
        r = paged.evict(w, pool, bt, [45], [20], 1, 3, d, bits)
        assert r["lengths"][0] == 20 and r["flags"] == 0
        for h in range(2):
            kept = r["kept"][0][h]
            assert len(kept) == 20 and kept[0] == 0 and kept[-3:] == [42, 43, 44] and kept == sorted(kept)
            for i, p in enumerate(kept):
                a = paged.token_bytes(r["pool"][bt[0, i // 16], h], i % 16, d, bits)
                b = paged.token_bytes(pool[bt[0, p // 16], h], p % 16, d, bits)
                assert sum(len(x) for x in a) * 16 == paged.tile_bytes(d, bits)
                assert all(np.array_equal(x, y) for x, y in zip(a, b))
        assert np.array_equal(r["pool"][[0, 3]], pool[[0, 3]])


def test_pages_given_back():
    bt = np.arange(12, dtype=np.int32).reshape(3, 4)
    q, s, f = paged.release([64, 33, 16], [17, 33, 0], bt, np.full(8, -1, np.int32), np.array([6, 1], np.int32), 12)
    assert f == 0 and s.tolist() == [6, 4] and q.tolist() == [3, 8, -1, -1, -1, -1, -1, 2]
    assert paged.release([64], [0], bt, np.zeros(3, np.int32), np.array([0, 0], np.int32), 12)[2] == paged.ERR_PAGES
    assert paged.release([16], [17], bt, np.zeros(3, np.int32), np.array([0, 0], np.int32), 12)[2] == paged.ERR_POSITION


@pytest.mark.parametrize("d", [64, 128, 256, 512])
def test_4_bit_configuration(d):
    cfg = B.tq_config_init(B.TQ_LAYOUT_DENSE, d, 8, 2)
    cfg.key_bits = cfg.value_bits = 4
    assert 16 * B.tq_config_check(cfg) == paged.tile_bytes(d, 4) == 18 * d + 32
    for kb, vb in ((4, 8), (16, 4), (5, 5), (2, 2)):
        cfg.key_bits, cfg.value_bits = kb, vb
        with pytest.raises(B.TQError) as e:
            B.tq_config_check(cfg)
        assert e.value.status == B.TQ_ERR_UNSUPPORTED


def test_calls_without_a_context_are_refused():
    lib, bad = B.lib, B.TQ_ERR_INVALID_ARG
    assert lib.tq_paged_attention_scored(None, None, 0, 1, None, 0, None, 0, None, 0, 0.0, 5.0, None, None, None, None, 0, None) == bad
    assert lib.tq_paged_weights(None, None, 0, 1, None, 0, None, 0, None, 0, 0.0, 0.0, None, None, None, 1.0, None, 0, None) == bad
    assert lib.tq_paged_evict(None, None, 0, 1, None, 0, None, 0, None, None, 0, 0, None, None, None, None) == bad
    assert lib.tq_release_pages(None, None, None, 1, None, 0, 0, None, 0, None, None, None) == bad
