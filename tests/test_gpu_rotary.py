"""Rotary positions on the GPU against the 64-bit oracle.

Tolerance, per element, with x0, x1 the pair's inputs and m the magnitude: the
output's rounding (half a step: 2^-8 of its value for bf16, 2^-24 for fp32),
and 1.5e-6 m (|x0| + |x1|) for the angle and the fp32 products. The angle: the
turn's remainder in fp32 is off by at most 2^-26 turns, 9.4e-8 rad, the fp64
turn of positions up to 2^31 by 2^-52 of at most 3.4e8 turns, 4.8e-7 rad; sine
and cosine to 2 ulp, 2.4e-7, their product with m 6e-8, and the two products
and their sum 1.8e-7: together below 1.1e-6.
"""

import numpy as np
import pytest
import torch

import blockwise_attn_ffn_bpt_b200 as bpt
from oracle import serving_oracle as so

pytestmark = pytest.mark.gpu

HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def rand(shape, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(shape, generator=g).to(dtype).cuda()


def check(got, x, positions, freq, heads, magnitude, interleaved, inverse):
    b, s, width = x.shape
    dh, rot = width // heads, 2 * len(freq)
    xn = x.double().cpu().numpy().reshape(b, s, heads, dh)
    ref = so.rotary(xn, positions, freq.numpy(), magnitude, interleaved, inverse)
    pair = np.zeros(rot, int)
    for j in range(rot // 2):
        pair[[2 * j, 2 * j + 1] if interleaved else [j, j + rot // 2]] = j
    mass = np.zeros_like(xn)
    for j in range(rot // 2):
        mass[..., :rot][..., pair == j] = np.abs(xn[..., :rot][..., pair == j]).sum(-1, keepdims=True)
    tol = HALF_STEP[x.dtype] * np.abs(ref) + 1.5e-6 * magnitude * mass + 1e-37
    err = np.abs(got.double().cpu().numpy().reshape(ref.shape) - ref)
    assert (err <= tol).all(), f"{(err / tol).max():.2f} times the tolerance"
    rest = got.view(b, s, heads, dh)[..., rot:]
    assert torch.equal(rest, x.reshape(b, s, heads, dh)[..., rot:])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("b,s,heads,kv,dh,rot", [
    (1, 1, 1, 1, 64, 64), (3, 1, 32, 4, 128, 128), (2, 37, 5, 1, 64, 32), (1, 129, 4, 2, 128, 24),
    (2, 5, 80, 40, 128, 2), (1, 1000, 3, 3, 64, 48),
    (2, 700, 3, 1, 128, 20), (1, 300, 2, 2, 64, 56), (1, 33, 2, 1, 64, 6),
])
def test_against_the_oracle(b, s, heads, kv, dh, rot, interleaved, dtype):
    q, k = rand((b, s, heads * dh), dtype, 1), rand((b, s, kv * dh), dtype, 2)
    freq, m = bpt.rotary_frequencies(rot, scaling="base" if rot > 2 else "plain", factor=4.0 if rot > 2 else 1.0)
    for inverse, offset in ((False, 0), (True, 4093)):
        pos = np.broadcast_to(offset + np.arange(s), (b, s))
        qo, ko = bpt.rotary(q, k, heads, kv, freq, offset=offset, interleaved=interleaved, magnitude=m, inverse=inverse)
        check(qo, q, pos, freq, heads, m, interleaved, inverse)
        check(ko, k, pos, freq, kv, m, interleaved, inverse)
    assert bpt.stream_status() == 0


@pytest.mark.parametrize("dtype", [torch.int32, torch.int64])
def test_positions_of_their_own_far_away_and_scaled(dtype):
    b, s, heads, dh = 3, 7, 2, 64
    q = rand((b, s, heads * dh), torch.float32, 3)
    freq, m = bpt.rotary_frequencies(dh, scaling="ramp", factor=32.0, original=4096)
    assert m > 1.3
    pos = torch.randint(0, 2 ** 31 - 1, (b, s), generator=torch.Generator().manual_seed(0)).to(dtype)
    pos[0, :3] = torch.tensor([0, 2 ** 31 - 1, -5], dtype=dtype)
    qo, ko = bpt.rotary(q, None, heads, 0, freq, positions=pos.cuda(), magnitude=m)
    assert ko is None
    check(qo, q, pos.numpy(), freq, heads, m, False, False)
    # one row of positions for every sequence; a view with a stride between sequences
    qo, _ = bpt.rotary(q, None, heads, 0, freq, positions=pos[1].cuda(), magnitude=m)
    check(qo, q, np.broadcast_to(pos[1].numpy(), (b, s)), freq, heads, m, False, False)
    wide = torch.zeros((b, s + 3), dtype=dtype, device="cuda")
    wide[:, :s] = pos.cuda()
    qo, _ = bpt.rotary(q, None, heads, 0, freq, positions=wide[:, :s], magnitude=m)
    check(qo, q, pos.numpy(), freq, heads, m, False, False)


@pytest.mark.parametrize("shift", [0, 1, 2, 4])
@pytest.mark.parametrize("layout", ["sequences", "tokens"])
def test_strided_rows_in_place_leave_their_neighbours(layout, shift):
    # q and k as columns of one fused buffer, turned in place; shifted by 1, 2
    # or 4 elements the rows are aligned to 2, 4 or 8 bytes
    b, s, heads, kv, dh = 2, 9, 3, 1, 64
    wide = (heads + 2 * kv) * dh + 8
    x = rand((b, s, wide) if layout == "sequences" else (s, b, wide), torch.bfloat16, 4)
    rows = x if layout == "sequences" else x.transpose(0, 1)
    before = rows.clone()
    q, k = rows[..., shift:shift + heads * dh], rows[..., shift + heads * dh:shift + (heads + kv) * dh]
    freq, _ = bpt.rotary_frequencies(dh)
    qo, ko = bpt.rotary(q, k, heads, kv, freq, offset=5, q_out=q, k_out=k)
    assert qo is q and ko is k
    pos = np.broadcast_to(5 + np.arange(s), (b, s))
    end = shift + (heads + kv) * dh
    check(qo, before[..., shift:shift + heads * dh], pos, freq, heads, 1.0, False, False)
    check(ko, before[..., shift + heads * dh:end], pos, freq, kv, 1.0, False, False)
    assert torch.equal(rows[..., end:], before[..., end:]) and torch.equal(rows[..., :shift], before[..., :shift])


def test_inverse_is_the_gradient():
    # against torch's autograd of the formula in fp64, and a difference quotient
    b, s, heads, dh = 2, 6, 2, 64
    freq, m = bpt.rotary_frequencies(32)
    x, g = rand((b, s, heads * dh), torch.float32, 5), rand((b, s, heads * dh), torch.float32, 6)
    got, _ = bpt.rotary(g, None, heads, 0, freq, offset=3, magnitude=m, inverse=True)
    leaf = x.double().requires_grad_()
    ang = (3 + torch.arange(s, device="cuda"))[:, None].double() * freq.cuda()
    h = leaf.view(b, s, heads, dh)
    c, sn = ang.cos()[:, None], ang.sin()[:, None]
    lo, hi = h[..., :16], h[..., 16:32]
    y = torch.cat((lo * c - hi * sn, hi * c + lo * sn, h[..., 32:]), -1).flatten(2)
    (y * g.double()).sum().backward()
    assert (got.double() - leaf.grad).abs().max() <= 2.0 ** -24 * 8 + 1.5e-6 * 10
    e = torch.zeros_like(x)
    e[1, 4, 70] = 0.5
    up, _ = bpt.rotary(x + e, None, heads, 0, freq, offset=3)
    down, _ = bpt.rotary(x - e, None, heads, 0, freq, offset=3)
    diff = ((up.double() - down.double()) * g.double()).sum()
    assert abs(diff.item() - got[1, 4, 70].item()) <= 1.5e-6 * 10 * 8


def test_more_tokens_than_one_grid_row_and_a_wide_token():
    freq, _ = bpt.rotary_frequencies(64)
    q = rand((1, 70001, 64), torch.bfloat16, 7)
    qo, _ = bpt.rotary(q, None, 1, 0, freq)
    check(qo, q, np.arange(70001)[None], freq, 1, 1.0, False, False)
    q = rand((1, 2, 300 * 64), torch.float32, 8)
    qo, _ = bpt.rotary(q, None, 300, 0, freq)
    check(qo, q, np.arange(2)[None], freq, 300, 1.0, False, False)


def test_another_stream_a_graph_and_nothing():
    freq, _ = bpt.rotary_frequencies(64)
    q = rand((2, 8, 128), torch.bfloat16, 9)
    ref, _ = bpt.rotary(q, None, 2, 0, freq)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out, _ = bpt.rotary(q, None, 2, 0, freq, stream=side)
    side.synchronize()
    assert torch.equal(out, ref)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, _ = bpt.rotary(q, None, 2, 0, freq)
    q.mul_(2)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, bpt.rotary(q, None, 2, 0, freq)[0])
    empty, _ = bpt.rotary(q[:, :0], None, 2, 0, freq)
    assert empty.shape == (2, 0, 128)


def test_the_binding_refuses():
    freq, _ = bpt.rotary_frequencies(64)
    q = rand((2, 4, 128), torch.bfloat16, 1)
    for bad in (dict(inv_freq=freq.float()), dict(inv_freq=freq.cuda()), dict(positions=torch.zeros(2, 4).cuda()),
                dict(q=q.half())):
        with pytest.raises(TypeError):
            bpt.rotary(**(dict(q=q, k=None, heads=2, kv_heads=0, inv_freq=freq) | bad))
    for bad in (dict(heads=3), dict(k=q[:1], kv_heads=2), dict(q=q.transpose(1, 2)[:, :, :4].contiguous(), heads=2),
                dict(positions=torch.zeros(4, 2, dtype=torch.int64).cuda()), dict(k=q.float(), kv_heads=2)):
        with pytest.raises((ValueError, bpt.BPTError)):
            bpt.rotary(**(dict(q=q, k=None, heads=2, kv_heads=0, inv_freq=freq) | bad))
    with pytest.raises(bpt.BPTError, match="ALIAS"):
        bpt.rotary(q[:, :3], None, 2, 0, freq, q_out=q[:, 1:])
