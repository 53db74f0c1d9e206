"""The tight bounds of paged_cases on the CPU: the weights' parts and totals as the dense-page attention holds them keep
within them, and with a part or the compensation left out they do not."""
import numpy as np
import pytest
import torch

from paged_cases import LIGHT_PAGES, ONE_TOKEN, U, light_tokens, light_tolerance


def parts_of(w, form, parts):
    """The first `parts` parts of fp32 weights, summed in 64 bits."""
    left, total = w.clone(), torch.zeros_like(w, dtype=torch.float64)
    for i in range(parts):
        if form == "tf32":
            bits = left.view(torch.int32)
            part = ((bits + (0x1000 if i else 0)) & ~0x1FFF).view(torch.float32)
        else:
            part = left.to(torch.bfloat16 if form == "bf16" else torch.float16).float()
        total += part.double()
        left = left - part
    return total


@pytest.mark.parametrize("form,parts,scale", [("tf32", 2, 2.0 ** -8), ("bf16", 3, 2.0 ** -8), ("f16", 2, 2.0 ** 12)])
def test_a_lost_part_passes_the_bound_of_one_token(form, parts, scale):
    gen = torch.Generator().manual_seed(1)
    w = torch.exp2(-torch.rand(256, generator=gen)) * scale
    off = lambda n: float(((parts_of(w, form, n) - w.double()).abs() / w.double()).max()) / U  # noqa: E731
    assert off(parts) <= 4
    assert off(parts - 1) > 2 * ONE_TOKEN


@pytest.mark.parametrize("bits", [16, 8])
def test_a_plain_total_passes_the_bound_of_light_tokens(bits):
    d = 64
    every = torch.arange(1 << 16, dtype=torch.int32).to(torch.int16).view(torch.bfloat16).float()
    some = every[(every >= 8) & (every < 16)].tolist()
    x, k, off = light_tokens([float(v) for v in range(8, 16)] if bits == 8 else some, [2 * v for v in some], d)
    w = np.float32(np.exp(x * k / np.sqrt(d)))
    assert abs(w / (0.375 * U) - 1) <= 1.01 * off + 1e-6
    page = np.float32(16 * w)
    plain, kept, lost, total = np.float32(1) + w, np.float32(1) + w, np.float32(0), np.float32(1 + 15 * np.float64(w))
    for _ in range(LIGHT_PAGES - 1):
        plain = np.float32(plain + np.float32(2 * w))
        y = np.float32(np.float32(2 * w) - lost)
        s = np.float32(kept + y)
        kept, lost = s, np.float32(np.float32(s - kept) - y)
        total = np.float32(total + page)
    others = 14 * np.float64(w) * LIGHT_PAGES  # the other seven lanes' totals are sums of equal light weights
    tol = light_tolerance(off) * U
    assert abs(total / (kept + others) - 1) <= tol
    assert abs(total / (plain + others) - 1) > 1.5 * tol
