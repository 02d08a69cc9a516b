"""How exact the 4-bit attention's output is where errors of its weights could add up over a long cache.

Per head, in the 2-norm over its dimensions, relative to o:
* o's rounding to bf16: at most 2^-8;
* the weights' products with V's scale enter as fp16, off by at most 2^-11 of themselves. An error e of a product meets
  the token's code less 7.5 (the kernel takes off 7.5 of the same rounded product), which is of either sign; with values
  that are independent of the weights the sum of the e (code - 7.5) is to the sum of the products times (code - 7.5) at
  most as their sizes, 2^-11, and that sum is to o about as one to one: within 2^-10.
Both fall with o as the cache grows. A sum of errors of one sign does not: 2^-11 of 7.5 scale is far above o then.
"""

import numpy as np
import pytest
import torch

import blockwise_attn_ffn_bpt_b200 as bpt
from oracle import serving_oracle as so

pytestmark = pytest.mark.gpu

NORM = 2.0 ** -8 + 2.0 ** -10


def heads_of(x, heads):
    return x.double().cpu().numpy().reshape(x.shape[0], x.shape[1], heads, x.shape[2] // heads)


@pytest.mark.parametrize("dh", [64, 128])
@pytest.mark.parametrize("b,kv,group,length", [(1, 2, 1, 20000), (1, 2, 4, 20000), (1, 1, 16, 20000), (3, 32, 1, 3000)])
@pytest.mark.parametrize("kind", ["scores within 1e-4", "every 64th token above equal ones"])
def test_nearly_equal_weights_over_a_long_cache(kind, b, kv, group, length, dh):
    # the split over the device with 1, 4 and 16 queries a head, and a thread block a head
    g = torch.Generator().manual_seed(length + dh)
    heads, c = kv * group, np.log2(np.e) / np.sqrt(dh)
    v = torch.randn((b, length, kv * dh), generator=g).bfloat16()
    if kind == "scores within 1e-4":
        k = torch.randn((b, length, kv * dh), generator=g).bfloat16()
        q = (torch.randn((b, 1, heads * dh), generator=g) * (1e-4 / (c * dh ** 0.5))).bfloat16()
    else:
        k = torch.zeros((b, length, kv * dh), dtype=torch.bfloat16)
        k[:, ::64] = 3.3 / (c * dh)
        q = torch.ones((b, 1, heads * dh), dtype=torch.bfloat16)
    cache = bpt.kv4_cache(b, kv, length, dh)
    zero = torch.zeros(b, dtype=torch.int32, device="cuda")
    bpt.kv4_store(cache, k.cuda(), v.cuda(), zero)
    o = heads_of(bpt.kv4_attention(q.cuda(), cache, zero + length, heads), heads)
    assert bpt.stream_status() == 0
    qn = heads_of(q, heads)
    for i in range(b):
        for h in sorted({0, kv - 1}):
            kn, vn = (so.values(*so.quantise(heads_of(x[i:i + 1], kv)[0, :, h])) for x in (k, v))
            for x in range(h * group, (h + 1) * group):
                ref, _, _ = so.attention(qn[i, :, x:x + 1], kn[None], vn[None], True)
                err = np.linalg.norm(o[i, 0, x] - ref[0, 0]) / np.linalg.norm(ref)
                assert err <= NORM, f"sequence {i}, head {x}: o is {err:.2e} off"


@pytest.mark.parametrize("dh", [64, 128])
@pytest.mark.parametrize("group", [1, 4, 8, 12])
def test_values_that_cancel_over_a_very_long_cache(group, dh):
    # Tokens in pairs of the same key and opposite values, both exact in the cache: o is 0, a pair's weights are rounded
    # alike, and what is left is what the sums of weight times code lose. These grow for 16 blocks at most until their
    # mean is taken off: to 15 times the products of 1024 tokens, or of the half or quarter of them that each of 2 or 4
    # copies of the queries meets (up to 4 and 2 queries a head). Each product of 16 tokens loses at most a last place of
    # the sum, 2^-23 of it. Relative to the sum of the weights, with scales below 2, that is 2^-23 15 (1024 / copies) / 16 2.
    # 256 heads of 131072 tokens, the same 64 over and over, are 200 blocks and more for every warp.
    b, kv, blocks = 8, 32, 2048
    g = torch.Generator().manual_seed(dh)
    x = torch.randint(0, 16, (b, 32, kv, dh // 64, 64), generator=g) - 7.5
    x[..., 0], x[..., 1] = -7.5, 7.5
    x = (x * (1 + torch.randint(0, 8, (b, 32, kv, dh // 64, 1), generator=g) / 8)).reshape(b, 32, 1, kv * dh)
    v = torch.cat((x, -x), 2).view(b, 64, kv * dh)
    assert torch.equal(v, v.bfloat16().float())
    k = torch.randn((b, 32, kv * dh), generator=g).bfloat16().repeat_interleave(2, 1)
    small = bpt.kv4_cache(b, kv, 64, dh)
    zero = torch.zeros(b, dtype=torch.int32, device="cuda")
    bpt.kv4_store(small, k.cuda(), v.bfloat16().cuda(), zero)
    cache = bpt.KV4Cache(small.data.repeat(1, 1, blocks, 1), dh)
    q = torch.randn((b, 1, kv * group * dh), generator=g).bfloat16().cuda()
    o = bpt.kv4_attention(q, cache, zero + 64 * blocks, kv * group)
    assert bpt.stream_status() == 0
    copies = 4 if group <= 2 else 2 if group <= 4 else 1
    most = o.float().abs().max().item()
    assert most <= 2.0 ** -23 * 15 * (1024 / copies) / 16 * 2, f"{most:.2e}"


@pytest.mark.parametrize("capacity", [512, 20032])
@pytest.mark.parametrize("size", [-95, -108, -116, -121])
@pytest.mark.parametrize("low", [-13, -20])
def test_values_near_the_smallest_scale(size, low, capacity):
    # one token of score 0 and no value, and many `low` (log2) below it, with V's scales down to the smallest that the
    # cache keeps.
    # Bounds: o's rounding, where it may be subnormal (half a step is 2^-134 then); the products' fp16 rounding, 2^-11 of
    # 15 p scale; scores and exponentials 2^-18; and 2^-31 of the largest product, or 2^-150, lost of each token's.
    n, dh = 400, 128
    g = np.random.default_rng(-size)
    v = torch.tensor(g.standard_normal((1, n, dh)) * 2.0 ** size).float().bfloat16()
    v[:, 130] = 0
    score = np.where(np.arange(n) == 130, 0.0, low) * np.log(2) / np.sqrt(dh)  # times a query of ones
    k = torch.tensor(np.broadcast_to(score[:, None], (n, dh))[None].copy()).float().bfloat16()
    cache = bpt.kv4_cache(1, 1, capacity, dh)
    zero = torch.zeros(1, dtype=torch.int32, device="cuda")
    bpt.kv4_store(cache, k.cuda(), v.cuda(), zero)
    q = torch.ones((1, 1, dh), dtype=torch.bfloat16, device="cuda")
    o = heads_of(bpt.kv4_attention(q, cache, zero + n, 1), 1)[0, 0, 0]
    (kc, ks, km), (vc, vs, vm) = (so.quantise(heads_of(x, 1)[0, :, 0]) for x in (k, v))
    assert (np.delete(vs, 130, 0) >= 2.0 ** -126).all()
    s = so.values(kc, ks, km) @ np.ones(dh) / np.sqrt(dh)
    p = np.exp(s - s.max())
    p /= p.sum()
    step, mid = np.repeat(vs, 64, -1), np.repeat(np.abs(vm), 64, -1)
    ref = p @ so.values(vc, vs, vm)
    tol = (2.0 ** -8 * np.abs(ref) + 2.0 ** -134 + 2.0 ** -11 * (p @ (15 * step)) + 2.0 ** -18 * (p @ (mid + 15 * step))
           + n * 15 * np.maximum(2.0 ** -31 * (p[:, None] * step).max(0), 2.0 ** -150))
    err = np.abs(o - ref)
    assert (err <= tol).all(), f"{(err / tol).max():.2f} times the bound"
    assert bpt.stream_status() == 0
