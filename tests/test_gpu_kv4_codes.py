"""The 4-bit cache's codes are rint((x - min) r) of the exact difference and product, r = fp32(1 / scale), also where
numbers of very different size make the difference longer than fp32 (or fp64), next to a tie above all. Checked against
fractions, which are exact."""

from fractions import Fraction

import numpy as np
import pytest
import torch

import blockwise_attn_ffn_bpt_b200 as bpt

pytestmark = pytest.mark.gpu


def stored(rows):
    """K's and V's codes [n, 64] that a cache holds of rows [n, 64] (bf16), and their scales and minimums."""
    n = len(rows)
    cache = bpt.kv4_cache(1, 1, n, 64)
    x = rows.view(1, n, 64).cuda()
    bpt.kv4_store(cache, x, x, torch.zeros(1, dtype=torch.int32, device="cuda"))
    assert bpt.stream_status() == 0
    data = cache.data[0, 0].cpu().numpy()
    out = []
    for which in "kv":
        codes, params = [], []
        for t in range(n):
            block, r = data[t // 64], t % 64
            at = (0 if which == "k" else 2304) + r * 32
            words = np.frombuffer(block[at:at + 32].tobytes(), np.uint32)
            if which == "k":
                words = np.array([words[(u % 4) * 2 + u // 4] for u in range(8)], np.uint64)
                words = ((words >> 3) | (words << 29)) & 0xFFFFFFFF
            codes.append([(int(w) >> (4 * i)) & 15 for w in words for i in range(8)])
            at = (2048 if which == "k" else 4352) + r * 4
            params.append(np.frombuffer(block[at:at + 4].tobytes(), np.uint16).astype(np.uint32) << 16)
        params = np.array(params, np.uint32).view(np.float32)
        out.append((np.array(codes), params[:, 0], params[:, 1]))
    return out


def groups():
    rng = np.random.default_rng(0)
    out = []
    tiny = [s * 2.0 ** e for e in (-18, -24, -25, -40, -60, -100, -133) for s in (1, -1)]
    for scale in (0.125, 1.0, 2.0 ** 40, 0.109375):
        # numbers next to 0 on a tie between two codes, below and above it
        for low in (-6.5, -7.5, -0.5, -3.5):
            out.append([low * scale, (low + 15) * scale, 0.0, -0.0, *(t * scale for t in tiny)])
        # half steps from a minimum next to 0
        for low in tiny:
            out.append([low * scale, 15 * scale, *((k + 0.5) * scale for k in range(15))])
    for _ in range(200):
        out.append(rng.standard_normal(64) * 2.0 ** rng.integers(-70, 3, 64))
    for _ in range(100):  # half steps and numbers of every size
        s = 2.0 ** rng.integers(-30, 30)
        out.append([-s * rng.integers(0, 15) - s / 2, *(s * rng.integers(-15, 16, 30) / 2),
                    *(s * rng.choice((1, -1), 30) * 2.0 ** rng.integers(-120, 4, 30))])
    rows = torch.zeros(len(out), 64)
    for i, x in enumerate(out):
        x = torch.tensor(np.asarray(x, np.float64)).float()
        rows[i] = x[torch.arange(64) % len(x)]
        rows[i] = rows[i, torch.randperm(64, generator=torch.Generator().manual_seed(i))]
    return rows.bfloat16()


def test_codes_of_numbers_of_very_different_size():
    rows = groups()
    left = 0
    for codes, scale, low in stored(rows):
        for i, row in enumerate(rows.double().tolist()):
            lo = min(Fraction(x) for x in row)
            assert Fraction(float(low[i])) == lo
            r = Fraction(float(np.float32(1) / scale[i]))
            for d, x in enumerate(row):
                exact = (Fraction(x) - lo) * r
                want = min(max(round(exact), 0), 15)  # Python rounds ties to even
                assert codes[i, d] == want, f"group {i}, x = {x!r}, min = {float(lo)!r}: {codes[i, d]}, not {want}"
                left += abs(exact - int(exact) - Fraction(1, 2)) < Fraction(1, 2 ** 30)
    assert left > 1000  # numbers next to a tie
