"""The 4-bit cache's operators over many sequences: more than a warp finds at once, and more rows than a grid has."""

import pytest
import torch

import blockwise_attn_ffn_bpt_b200 as bpt
from tests.test_gpu_kv4 import bf16, check_attention, filled

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dh", [64, 128])
@pytest.mark.parametrize("heads,kv,n", [(2, 1, 1), (4, 2, 3), (10, 1, 1)])
@pytest.mark.parametrize("capacity", [256, 20032])
def test_attention_over_70_sequences(heads, kv, n, dh, capacity):
    # the split finds a warp's first sequence 32 at a time; here in the first, second and third of them, behind whole
    # groups of empty ones too
    lens = [(i * 37) % 250 if i % 3 else 0 for i in range(30)] + [0] * 36 + [1, 200, 64, 65]
    cache, held = filled(len(lens), kv, dh, lens, capacity, seed=91)
    q = bf16((len(lens), n, heads * dh), 92)
    w = torch.rand((len(lens), kv, capacity), generator=torch.Generator().manual_seed(2)).cuda()
    check_attention(q, cache, held, lens, heads)
    check_attention(q, cache, held, lens, heads, weights=w)


def test_66000_sequences():
    # rows past 65535 are a block's second turn in the store, the load, the weights and the eviction's move
    b, dh = 66000, 64
    x = bf16((b, 1, 2 * dh), 1)
    k, v = x[..., :dh], x[..., dh:]
    cache, out = bpt.kv4_cache(b, 1, 64, dh), bpt.kv4_cache(b, 1, 64, dh)
    at = torch.arange(b, dtype=torch.int32, device="cuda")
    start, counts = at % 64, (at % 5 != 0).int()
    bpt.kv4_store(cache, k, v, start, counts=counts)
    got = bpt.kv4_load(cache, start + counts, 1, start=start)
    for x, y in zip(got, (k, v)):
        # half a step of 1/15 of the range, the scale's rounding, and that of the value
        y = y * counts[:, None, None]
        step = (y.float().amax(-1) - y.float().amin(-1))[..., None] / 15
        assert ((x.float() - y.float()).abs() <= (0.5 + 15 * 2.0 ** -8) * step + 2.0 ** -8 * y.float().abs()).all()
    # one token of each sequence that has any: o is its value, and its weight 1
    first = torch.zeros_like(start)
    bpt.kv4_store(cache, k, v, first, counts=counts)
    k1, v1 = bpt.kv4_load(cache, counts, 1)
    w = torch.full((b, 1, 64), 0.25, device="cuda")
    o, lse2 = bpt.kv4_attention(k.contiguous(), cache, counts, 1, weights=w, return_lse=True)
    # the value is within 2^-11 of 15 steps, and rounded to bf16 as v1 is
    step = (v.float().amax(-1) - v.float().amin(-1))[..., None] / 15
    assert ((o.float() - v1.float()).abs() <= 2.0 ** -7 * v1.float().abs() + 2.0 ** -11 * 15 * 1.01 * step).all()
    assert torch.equal(lse2.isinf().flatten(), counts == 0)
    assert ((w[:, 0, 0] - 0.25 - counts).abs() <= 2.0 ** -17).all() and (w[:, :, 1:] == 0.25).all()
    kept, lens, moved = bpt.kv4_evict(cache, w, counts, 1, 0, out)
    assert torch.equal(lens, counts) and torch.equal(kept.flatten(), counts - 1)
    assert torch.equal(moved[:, 0, 0], w[:, 0, 0] * counts) and (moved[:, :, 1:] == 0).all()
    for x, y in zip(bpt.kv4_load(out, lens, 1), (k1, v1)):
        assert torch.equal(x, y)
    assert bpt.stream_status() == 0
