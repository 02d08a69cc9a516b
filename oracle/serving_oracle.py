"""Plain 64-bit definitions of rotary positions and of the 4-bit key/value
cache: its quantisation and layout, attention over it, and the choice of the
tokens that an eviction keeps. Test infrastructure only; it shares no code with
the library."""

import numpy as np

BLOCK = 64
GROUP = 64


def rotary(x, positions, inv_freq, magnitude=1.0, interleaved=False, inverse=False):
    """x [b, s, heads, dh] turned by positions [b, s]; 2 len(inv_freq) dimensions of each head."""
    x = np.asarray(x, np.float64)
    y = x.copy()
    half = len(inv_freq)
    for j, f in enumerate(inv_freq):
        lo, hi = (2 * j, 2 * j + 1) if interleaved else (j, j + half)
        a = (np.asarray(positions, np.float64) * float(f))[..., None] * (-1 if inverse else 1)
        c, s = np.cos(a) * magnitude, np.sin(a) * magnitude
        y[..., lo] = x[..., lo] * c - x[..., hi] * s
        y[..., hi] = x[..., hi] * c + x[..., lo] * s
    return y


def to_bf16(x):
    """Rounded to bf16 (nearest, ties to even), as fp64; x is representable in fp32 or is rounded to it first."""
    bits = np.asarray(x, np.float32).view(np.uint32).astype(np.uint64)
    bits = (bits + 0x7FFF + ((bits >> 16) & 1)) & 0xFFFF0000
    return bits.astype(np.uint32).view(np.float32).astype(np.float64)


def bf16_bits(x):
    return (np.asarray(x, np.float32).view(np.uint32) >> 16).astype(np.uint32)


def quantise(x):
    """x [..., dh] (bf16 values): codes [..., dh], scale and minimum [..., dh / 64]."""
    g = np.asarray(x, np.float64).reshape(*x.shape[:-1], x.shape[-1] // GROUP, GROUP)
    low = g.min(-1)
    scale = to_bf16((g.max(-1) - low) / 15)
    live = scale >= 2.0 ** -126
    scale = np.where(live, scale, 0.0)
    r = np.where(live, 1 / np.where(live, scale, 1), 0.0).astype(np.float32).astype(np.float64)
    codes = np.clip(np.rint((g - low[..., None]) * r[..., None]), 0, 15).astype(np.uint32)
    return codes.reshape(x.shape), scale, low


def values(codes, scale, low):
    g = codes.reshape(*codes.shape[:-1], codes.shape[-1] // GROUP, GROUP)
    return (low[..., None] + scale[..., None] * g).reshape(codes.shape)


def pack(k, v):
    """The bytes [blocks, block bytes] that tokens k, v [tokens, dh] of one head at places 0 .. occupy, and a mask of
    the bytes that they write."""
    tokens, dh = k.shape
    codes_bytes, params_bytes = BLOCK * dh // 2, BLOCK * (dh // GROUP) * 4
    blocks = (tokens + BLOCK - 1) // BLOCK
    data = np.zeros((blocks, 2 * (codes_bytes + params_bytes)), np.uint8)
    used = np.zeros(data.shape, bool)
    for which, x, base in (("k", k, 0), ("v", v, codes_bytes + params_bytes)):
        codes, scale, low = quantise(x)
        sb, lb = bf16_bits(scale), bf16_bits(low)
        for t in range(tokens):
            blk, r = divmod(t, BLOCK)
            for u in range(dh // 8):
                word = 0
                for i in range(8):
                    word |= int(codes[t, 8 * u + i]) << (4 * i)
                if which == "k":
                    word = ((word << 3) | (word >> 29)) & 0xFFFFFFFF
                    place = (u % 4) * (dh // 32) + u // 4
                elif dh == 64:
                    place = u
                else:
                    pair = u % 8
                    if r & 2:
                        pair = (pair + 4) % 8
                    place = pair * 2 + u // 8
                at = base + r * (dh // 2) + 4 * place
                data[blk, at:at + 4] = np.frombuffer(np.uint32(word).tobytes(), np.uint8)
                used[blk, at:at + 4] = True
            for g in range(dh // GROUP):
                at = base + codes_bytes + (r * (dh // GROUP) + g) * 4
                word = int(sb[t, g]) | (int(lb[t, g]) << 16)
                data[blk, at:at + 4] = np.frombuffer(np.uint32(word).tobytes(), np.uint8)
                used[blk, at:at + 4] = True
    return data, used


def attention(q, k, v, causal):
    """q [n, heads, dh] over k, v [kv_heads, len, dh]: o [n, heads, dh], lse2 [heads, n], weights [kv_heads, len]."""
    n, heads, dh = q.shape
    kv_heads, length, _ = k.shape
    group = heads // kv_heads
    o = np.zeros((n, heads, dh))
    lse2 = np.full((heads, n), -np.inf)
    weights = np.zeros((kv_heads, length))
    for i in range(heads):
        for t in range(n):
            seen = length - n + 1 + t if causal else length
            if seen <= 0:
                continue
            s = k[i // group, :seen] @ q[t, i] / np.sqrt(dh)
            e = np.exp(s - s.max())
            p = e / e.sum()
            o[t, i] = p @ v[i // group, :seen]
            lse2[i, t] = (s.max() + np.log(e.sum())) / np.log(2)
            weights[i // group, :seen] += p
    return o, lse2, weights


def kept_tokens(weights, length, keep, recent):
    """The places, in order, that one head keeps of its `length` tokens."""
    left = min(length, keep)
    recent = min(recent, left)
    old = length - recent
    def order(i):
        w = float(weights[i])
        return (0, 0.0, i) if np.isnan(w) else (1, -w, i)
    return sorted(sorted(range(old), key=order)[:left - recent]) + list(range(old, length))
