"""The serving oracle against independent statements: complex rotation and
orthogonality for rotary positions, torch's softmax attention, the quantisation
error's bound, and closed forms."""

import numpy as np
import pytest
import torch

import blockwise_attn_ffn_bpt_b200 as bpt
from oracle import serving_oracle as so


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rot", [2, 24, 64])
def test_rotary_is_a_complex_rotation_and_inverse_is_its_transpose(rot, interleaved):
    rng = np.random.default_rng(rot)
    x = rng.standard_normal((2, 3, 2, 64))
    pos = rng.integers(0, 10**6, (2, 3))
    f = 10000.0 ** (-np.arange(0, rot, 2) / rot)
    y = so.rotary(x, pos, f, 1.25, interleaved)
    lo, hi = (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else (slice(0, rot // 2), slice(rot // 2, rot))
    z = (x[..., lo] + 1j * x[..., hi]) * 1.25 * np.exp(1j * pos[..., None, None] * f)
    assert np.allclose(y[..., lo], z.real, atol=1e-9) and np.allclose(y[..., hi], z.imag, atol=1e-9)
    assert np.array_equal(y[..., rot:], x[..., rot:])
    # <g, R x> = <R^T g, x>, and a central difference in one element
    g = rng.standard_normal(x.shape)
    back = so.rotary(g, pos, f, 1.25, interleaved, inverse=True)
    assert np.isclose((g * y).sum(), (back * x).sum(), rtol=1e-12)
    e = np.zeros_like(x)
    e[1, 2, 1, 1] = 1e-3
    diff = (g * (so.rotary(x + e, pos, f, 1.25, interleaved) - so.rotary(x - e, pos, f, 1.25, interleaved))).sum()
    assert np.isclose(diff / 2e-3, back[1, 2, 1, 1], rtol=1e-8)


def test_rotary_scores_depend_on_distance_alone():
    rng = np.random.default_rng(1)
    q, k = rng.standard_normal((2, 1, 1, 1, 64))
    f = 10000.0 ** (-np.arange(0, 64, 2) / 64)
    near = (so.rotary(q, [[7]], f) * so.rotary(k, [[3]], f)).sum()
    far = (so.rotary(q, [[70007]], f) * so.rotary(k, [[70003]], f)).sum()
    assert np.isclose(near, far, atol=1e-9)


def test_frequencies_follow_their_formulas():
    rot, base, factor, original = 64, 10000.0, 8.0, 4096
    f = base ** (-np.arange(0, rot, 2) / rot)
    got, m = bpt.rotary_frequencies(rot, base)
    assert np.allclose(got.numpy(), f, rtol=1e-15) and m == 1.0
    got, m = bpt.rotary_frequencies(rot, base, "linear", factor)
    assert np.allclose(got.numpy(), f / factor, rtol=1e-15) and m == 1.0
    got, m = bpt.rotary_frequencies(rot, base, "base", factor)
    assert np.isclose(got[0].item(), 1.0) and np.isclose(got[-1].item(), f[-1] / factor, rtol=1e-12) and m == 1.0
    got, m = bpt.rotary_frequencies(rot, base, "ramp", factor, original, 1.0, 32.0)
    turns = original * f / (2 * np.pi)
    g = got.numpy()
    assert np.allclose(g[turns >= 32], f[turns >= 32]) and np.allclose(g[turns <= 1], f[turns <= 1] / factor)
    between = (turns > 1) & (turns < 32)
    assert between.any() and (g[between] < f[between]).all() and (g[between] > f[between] / factor).all()
    assert np.isclose(m, 0.1 * np.log(8.0) + 1, rtol=1e-7)


@pytest.mark.parametrize("args", [
    dict(rot=0), dict(rot=3), dict(rot=130), dict(rot=64, base=0.0), dict(rot=64, base=float("inf")),
    dict(rot=64, scaling="linear", factor=0.5), dict(rot=64, scaling="linear", factor=float("nan")),
    dict(rot=2, scaling="base", factor=2.0), dict(rot=64, scaling="ramp", factor=2.0),
    dict(rot=64, scaling="ramp", factor=2.0, original=8, low_turns=3.0, high_turns=3.0),
])
def test_frequencies_refuse(args):
    with pytest.raises(bpt.BPTError, match="SHAPE"):
        bpt.rotary_frequencies(**args)


def test_frequencies_refuse_an_unknown_scaling():
    with pytest.raises(ValueError):
        bpt.rotary_frequencies(64, scaling="other")


@pytest.mark.parametrize("dh", [64, 128])
def test_quantisation_error_is_at_most_half_a_step(dh):
    rng = np.random.default_rng(dh)
    x = so.to_bf16(rng.standard_normal((9, dh)) * 3 + 1)
    codes, scale, low = so.quantise(x)
    err = np.abs(so.values(codes, scale, low) - x).reshape(9, -1, 64)
    # half a step, and at the top the scale's rounding: 15 steps of 2^-8 of it
    assert (err <= (0.5 + 15 * 2.0 ** -8) * scale[..., None]).all()
    flat = np.full((2, dh), 3.5)
    assert np.array_equal(so.values(*so.quantise(flat)), flat)


def test_pack_writes_every_byte_of_full_blocks_once():
    rng = np.random.default_rng(2)
    for dh in (64, 128):
        x = so.to_bf16(rng.standard_normal((64, dh)))
        data, used = so.pack(x, x)
        assert data.shape == (1, 72 * dh) and used.all()
        _, used = so.pack(x[:5], x[:5])
        assert used.sum() == 5 * 2 * (dh // 2 + dh // 16)


def test_attention_is_torchs_on_the_visible_prefix():
    rng = np.random.default_rng(3)
    q, k, v = rng.standard_normal((5, 4, 64)), rng.standard_normal((2, 9, 64)), rng.standard_normal((2, 9, 64))
    o, lse2, w = so.attention(q, k, v, True)
    tq = torch.tensor(q).transpose(0, 1)
    tk, tv = (torch.tensor(x).repeat_interleave(2, 0) for x in (k, v))
    mask = torch.ones(5, 9, dtype=torch.bool).tril(4)
    ref = torch.nn.functional.scaled_dot_product_attention(tq, tk, tv, attn_mask=mask)
    assert np.allclose(o, ref.transpose(0, 1).numpy(), atol=1e-12)
    s = (tq @ tk.transpose(-1, -2) / 8).masked_fill(~mask, -torch.inf)
    assert np.allclose(lse2, torch.logsumexp(s, -1).numpy() / np.log(2), atol=1e-12)
    assert np.allclose(w, torch.softmax(s, -1).sum(1).view(2, 2, 9).sum(1).numpy(), atol=1e-12)
    o, lse2, w = so.attention(q, k[:, :3], v[:, :3], True)  # the first tokens see nothing
    assert (o[:2] == 0).all() and np.isneginf(lse2[:, :2]).all() and np.isfinite(lse2[:, 2:]).all()


def test_kept_tokens_by_hand():
    w = np.array([5, 1, 9, 1, 0, 9, 2, 3], np.float32)
    assert so.kept_tokens(w, 8, 4, 1) == [0, 2, 5, 7]
    assert so.kept_tokens(w, 8, 5, 0) == [0, 2, 5, 6, 7]
    assert so.kept_tokens(w, 5, 3, 1) == [0, 2, 4]
    assert so.kept_tokens(w, 4, 3, 0) == [0, 1, 2]  # of two equal ones the first
    assert so.kept_tokens(w, 2, 3, 2) == [0, 1]
    assert so.kept_tokens(w, 0, 3, 2) == []
    w[3] = np.nan
    assert so.kept_tokens(w, 8, 2, 0) == [2, 3]
