"""The sines and cosines of rotary positions, to fp32's last places."""

import numpy as np
import pytest
import torch

import blockwise_attn_ffn_bpt_b200 as bpt

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("magnitude,inverse", [(1.0, False), (1.0, True), (1.3465, False)])
def test_sine_and_cosine_to_the_last_places(magnitude, inverse, interleaved):
    # A pair (1, 0) comes out as (m cos, +-m sin), without a rounding of its own. Sine and cosine are within 2 units of
    # their last place, and half a unit is their product with m: 2.5 2^-23 of the value. The fp64 angle of a position
    # below 2^14 is within 2^14 2^-53 turns and as much in the reference, 4e-11 rad in all.
    s, dh = 16384, 64
    freq, _ = bpt.rotary_frequencies(dh)
    m = float(np.float32(magnitude))
    x = torch.zeros((1, s, dh // 2, 2), dtype=torch.float32, device="cuda")
    x[..., 0] = 1
    x = (x if interleaved else x.transpose(-1, -2)).reshape(1, s, dh)
    y, _ = bpt.rotary(x, None, 1, 0, freq, interleaved=interleaved, magnitude=m, inverse=inverse)
    y = y.double().cpu().numpy()[0]
    cos, sin = (y[:, 0::2], y[:, 1::2]) if interleaved else (y[:, :dh // 2], y[:, dh // 2:])
    angle = np.arange(s)[:, None] * freq.numpy()
    for got, ref in ((cos, m * np.cos(angle)), (sin, m * np.sin(angle) * (-1 if inverse else 1))):
        off = np.abs(got - ref) / (2.5 * 2.0 ** -23 * np.abs(ref) + 4e-11 * m)
        assert off.max() <= 1, f"{off.max():.2f} times the bound"
