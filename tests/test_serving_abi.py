"""Refusals of the rotary and 4-bit cache entry points, without a GPU: the
argument checks run before any CUDA call, so fake addresses do."""

import ctypes

import pytest
import torch

import blockwise_attn_ffn_bpt_b200 as bpt

OK, NULL, SHAPE, ALIGN, ALIAS, NOMEM, DTYPE = 0, -1, -2, -4, -5, -6, -10
BASE, STEP = 1 << 40, 1 << 36
FREQ = (ctypes.c_double * 64)()


def at(i):
    return BASE + i * STEP


def call_rotary(dtype=0, q=at(0), bs_q=2048, ld_q=256, k=at(1), bs_k=1024, ld_k=128, b=2, s=8, heads=4, kv_heads=2,
                dh=64, rot=64, inter=0, freq=ctypes.addressof(FREQ), pos=None, size=8, step=0, q_out=at(2), bs_qo=2048,
                ld_qo=256, k_out=at(3), bs_ko=1024, ld_ko=128):
    return bpt.lib().bpt_rotary(dtype, q, bs_q, ld_q, k, bs_k, ld_k, b, s, heads, kv_heads, dh, rot, inter, freq, 1.0,
                                pos, size, step, 0, 0, q_out, bs_qo, ld_qo, k_out, bs_ko, ld_ko, None)


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=2), DTYPE), (dict(pos=at(5), size=2), DTYPE),
    (dict(b=-1), SHAPE), (dict(s=-1), SHAPE), (dict(heads=0), SHAPE), (dict(kv_heads=-1), SHAPE),
    (dict(dh=32), SHAPE), (dict(rot=0), SHAPE), (dict(rot=63), SHAPE), (dict(rot=66), SHAPE),
    (dict(b=1 << 16, s=1 << 16), SHAPE), (dict(pos=at(5), step=-1), SHAPE),
    (dict(ld_q=-256), SHAPE), (dict(bs_q=1 << 62), SHAPE),
    (dict(ld_qo=255), SHAPE), (dict(bs_qo=2047), SHAPE), (dict(bs_ko=0), SHAPE),   # rows of an output overlap
    (dict(q=None), NULL), (dict(k=None), NULL), (dict(q_out=None), NULL), (dict(k_out=None), NULL),
    (dict(freq=None), NULL),
    (dict(q=at(0) + 1), ALIGN), (dict(dtype=1, k=at(1) + 2), ALIGN), (dict(pos=at(5) + 4), ALIGN),
    (dict(q_out=at(0) + 512), ALIAS),                       # its own input, shifted
    (dict(q_out=at(0), bs_qo=4096), ALIAS),                 # its own input, other strides
    (dict(q_out=at(1)), ALIAS), (dict(k_out=at(0)), ALIAS), (dict(k_out=at(2)), ALIAS),
    (dict(pos=at(2) + 64), ALIAS),
    (dict(b=0), OK), (dict(s=0, q=None), OK),
])
def test_rotary_refuses(kw, code):
    assert call_rotary(**kw) == code


def fused(**kw):
    """q and k as columns of one buffer of rows of 512 elements, turned in place."""
    base = dict(q=at(0), bs_q=4096, ld_q=512, k=at(0) + 512, bs_k=4096, ld_k=512, q_out=at(0), bs_qo=4096, ld_qo=512,
                k_out=at(0) + 512, bs_ko=4096, ld_ko=512)
    return call_rotary(**(base | kw))


def test_rotary_takes_columns_of_one_buffer():
    if torch.cuda.is_available():
        pytest.skip("the addresses are fake, and past the checks the call would use them")
    assert fused() not in (NULL, SHAPE, ALIGN, ALIAS, DTYPE)
    assert fused(k=at(0) + 510, k_out=at(0) + 510) == ALIAS     # one element of q's
    assert fused(k=at(0) + 1024 - 254, k_out=at(0) + 1024 - 254) == ALIAS  # into the next row
    # tokens first: sequences 512 elements apart, tokens 1024
    swapped = dict(bs_q=512, ld_q=1024, bs_k=512, ld_k=1024, bs_qo=512, ld_qo=1024, bs_ko=512, ld_ko=1024)
    assert fused(**swapped) not in (NULL, SHAPE, ALIGN, ALIAS, DTYPE)


def store(cache=at(0), b=2, kv=2, cap=128, dh=64, k=at(1), bs_k=1024, ld_k=128, v=at(2), bs_v=1024, ld_v=128, n=8,
          start=at(3), counts=None):
    return bpt.lib().bpt_kv4_store(cache, b, kv, cap, dh, k, bs_k, ld_k, v, bs_v, ld_v, n, start, counts, None)


@pytest.mark.parametrize("kw,code", [
    (dict(b=-1), SHAPE), (dict(kv=0), SHAPE), (dict(cap=0), SHAPE), (dict(cap=100), SHAPE), (dict(dh=96), SHAPE),
    (dict(n=-1), SHAPE), (dict(n=1 << 30), SHAPE), (dict(b=1 << 20, kv=1 << 12), SHAPE), (dict(ld_k=-8), SHAPE),
    (dict(cache=None), NULL), (dict(k=None), NULL), (dict(v=None), NULL), (dict(start=None), NULL),
    (dict(cache=at(0) + 8), ALIGN), (dict(k=at(1) + 8), ALIGN), (dict(ld_v=132), ALIGN), (dict(bs_k=1028), ALIGN),
    (dict(start=at(3) + 2), ALIGN), (dict(counts=at(4) + 1), ALIGN),
    (dict(k=at(0) + 4608), ALIAS), (dict(v=at(0)), ALIAS), (dict(start=at(0)), ALIAS), (dict(counts=at(0)), ALIAS),
    (dict(b=0), OK), (dict(n=0, k=None), OK),
])
def test_store_refuses(kw, code):
    assert store(**kw) == code


def load(cache=at(0), b=2, kv=2, cap=128, dh=64, start=None, lens=at(1), n=8, k=at(2), v=at(3)):
    return bpt.lib().bpt_kv4_load(cache, b, kv, cap, dh, start, lens, n, k, v, None)


@pytest.mark.parametrize("kw,code", [
    (dict(cap=63), SHAPE), (dict(n=-1), SHAPE), (dict(lens=None), NULL), (dict(k=None), NULL),
    (dict(v=at(3) + 8), ALIGN), (dict(lens=at(1) + 2), ALIGN), (dict(start=at(5) + 2), ALIGN),
    (dict(k=at(0)), ALIAS), (dict(v=at(2) + 16), ALIAS), (dict(k=at(1) - 16), ALIAS), (dict(start=at(3)), ALIAS),
    (dict(n=0), OK), (dict(b=0), OK),
])
def test_load_refuses(kw, code):
    assert load(**kw) == code


def attend(q=at(0), bs=256, ld=256, cache=at(1), lens=at(2), b=2, n=1, heads=4, kv=2, cap=1 << 16, dh=64, o=at(3),
           lse=None, weights=None, ws=at(6), nbytes=1 << 30):
    return bpt.lib().bpt_kv4_attention(q, bs, ld, cache, lens, b, n, heads, kv, cap, dh, 1, o, lse, weights, ws,
                                       nbytes, None)


@pytest.mark.parametrize("kw,code", [
    (dict(heads=3), SHAPE), (dict(heads=0), SHAPE), (dict(dh=80), SHAPE), (dict(cap=65), SHAPE), (dict(n=-1), SHAPE),
    (dict(b=1 << 16, n=1 << 16), SHAPE), (dict(ld=-8), SHAPE),
    (dict(q=None), NULL), (dict(cache=None), NULL), (dict(lens=None), NULL), (dict(o=None), NULL),
    (dict(ws=None), NULL),
    (dict(q=at(0) + 8), ALIGN), (dict(bs=260), ALIGN), (dict(ws=at(6) + 64), ALIGN), (dict(lse=at(4) + 4), ALIGN),
    (dict(weights=at(5) + 8), ALIGN), (dict(lens=at(2) + 1), ALIGN),
    (dict(nbytes=0), NOMEM),
    (dict(o=at(0)), ALIAS), (dict(ws=at(1)), ALIAS), (dict(weights=at(3)), ALIAS), (dict(lse=at(2) - 16), ALIAS),
    (dict(ws=at(3)), ALIAS),
    (dict(b=0), OK), (dict(n=0), OK),
])
def test_attention_refuses(kw, code):
    assert attend(**kw) == code


def test_attention_workspace():
    f = bpt.lib().bpt_kv4_attention_workspace_bytes
    small, big = f(2, 1, 4, 2, 1 << 16, 64, 0), f(2, 1, 4, 2, 1 << 16, 64, 1)
    assert 0 < small < big and big - small >= 2 * 4 * (1 << 16) * 4  # the scores
    # a short cache without weights needs none, and then takes none
    assert f(2, 1, 4, 2, 128, 64, 0) == 0 and f(2, 1, 4, 2, 128, 64, 1) >= 2 * 4 * 128 * 4
    if not torch.cuda.is_available():  # the addresses are fake
        assert attend(cap=128, ws=None, nbytes=0) not in (NULL, NOMEM)
    assert f(2, 1, 3, 2, 128, 64, 0) == 0 and f(0, 1, 4, 2, 128, 64, 0) == 0 and f(2, 1, 4, 2, 100, 64, 0) == 0
    assert attend(nbytes=small - 1) == NOMEM
    assert attend(weights=at(5), nbytes=big - 1) == NOMEM


def evict(cache=at(0), weights=at(1), lens=at(2), b=2, kv=2, cap=256, dh=64, keep=100, recent=10, out=at(3), cap_out=128,
          w_out=at(4), l_out=at(5), kept=at(6)):
    return bpt.lib().bpt_kv4_evict(cache, weights, lens, b, kv, cap, dh, keep, recent, out, cap_out, w_out, l_out, kept,
                                   None)


@pytest.mark.parametrize("kw,code", [
    (dict(keep=0), SHAPE), (dict(keep=129), SHAPE), (dict(recent=-1), SHAPE), (dict(recent=101), SHAPE),
    (dict(cap_out=120), SHAPE), (dict(cap=1), SHAPE), (dict(dh=1), SHAPE), (dict(b=-2), SHAPE),
    (dict(cache=None), NULL), (dict(weights=None), NULL), (dict(lens=None), NULL), (dict(out=None), NULL),
    (dict(w_out=None), NULL), (dict(l_out=None), NULL), (dict(kept=None), NULL),
    (dict(out=at(3) + 8), ALIGN), (dict(weights=at(1) + 4), ALIGN), (dict(kept=at(6) + 2), ALIGN),
    (dict(out=at(0)), ALIAS), (dict(w_out=at(1)), ALIAS), (dict(l_out=at(2)), ALIAS), (dict(kept=at(5)), ALIAS),
    (dict(b=0), OK),
])
def test_evict_refuses(kw, code):
    assert evict(**kw) == code


def test_cache_bytes():
    f = bpt.lib().bpt_kv4_cache_bytes
    assert f(1, 1, 64, 128) == 9216 and f(3, 5, 192, 64) == 3 * 5 * 3 * 4608
    assert f(64, 32, 1 << 17, 128) == 64 * 32 * 2048 * 9216  # past 32 bits
    assert f(1, 1, 63, 128) == 0 and f(1, 1, 64, 127) == 0 and f(1, 0, 64, 128) == 0 and f(-1, 1, 64, 128) == 0


def test_status_string():
    assert bpt.status_string(-11).startswith("BPT_ERR_RANGE")


def test_the_binding_refuses_host_tensors():
    x = torch.zeros(1, 1, 64, dtype=torch.bfloat16)
    freq, _ = bpt.rotary_frequencies(64)
    with pytest.raises(ValueError):
        bpt.rotary(x, None, 1, 0, freq)
    with pytest.raises(TypeError):
        bpt.KV4Cache(torch.zeros(1, 1, 1, 9216, dtype=torch.uint8), 128)
    with pytest.raises(ValueError):
        bpt.KV4Cache(torch.zeros(1, 1, 1, 9216, dtype=torch.uint8), 96)
    with pytest.raises(ValueError):
        bpt.kv4_cache(1, 1, 64, 96, device="cpu")


def test_the_binding_refuses_before_it_touches_a_gpu():
    # messages with numbers in them, raised from C++
    freq, _ = bpt.rotary_frequencies(64)
    q = torch.zeros(2, 4, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="q's last dimension 128 does not hold 3 heads"):
        bpt.rotary(q, None, 3, 0, freq)
    with pytest.raises(ValueError, match="q must be a CUDA tensor"):
        bpt.rotary(q, None, 2, 0, freq)
    with pytest.raises(ValueError, match="heads = 4294967296 is out of range"):
        bpt.rotary(q, None, 1 << 32, 0, freq)
