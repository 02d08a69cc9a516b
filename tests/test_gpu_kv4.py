"""The 4-bit key/value cache on the GPU against the 64-bit oracle: the stored
bytes and the moved bytes exactly, the attention within bounds that follow from
its roundings.

Attention, per query (c = log2(e) / sqrt(dh)):
* a score in log2 units is a sum of dh products in fp32 and a few more fp32
  operations on values of at most B = c sum_d |q_d| (|min| + 31 scale), so it is
  off by at most E = (dh + 16) 2^-24 B; lse2 by E and 2^-20 for exponentials
  and logarithm, in relation to its size 2^-23;
* a weight p by p (2 ln2 E + 2^-19), and their sum over the queries by an
  fp32 rounding each;
* o: each p's product with V's scale is rounded to fp16, 2^-11 of p scale code,
  at most 15 p scale, the result to bf16, 2^-8 of |o|, and the weights' error
  shows as (2 ln2 E + 2^-18) sum p (|min| + 15 scale).
"""

import numpy as np
import pytest
import torch

import blockwise_attn_ffn_bpt_b200 as bpt
from oracle import serving_oracle as so

pytestmark = pytest.mark.gpu

RANGE = -11


def bf16(shape, seed, scale=1.0, offset=0.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale + offset).bfloat16().cuda()


def ints(*v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def heads_of(x, heads):
    """[b, n, heads * dh] on the GPU to fp64 [b, n, heads, dh]."""
    return x.double().cpu().numpy().reshape(x.shape[0], x.shape[1], heads, x.shape[2] // heads)


def filled(b, kv, dh, lens, capacity, seed=0):
    """A cache that holds lens[beta] tokens of each sequence, and the oracle's K, V values [b][kv, len, dh], with the
    scales [b][kv, len, groups] and minimums of both."""
    cache = bpt.kv4_cache(b, kv, capacity, dh)
    # bytes that no stored token defines: parameters among them that are NaN
    cache.data.fill_(0xFF)
    n = max(max(lens), 1)
    k, v = bf16((b, n, kv * dh), seed, 1.0, 0.3), bf16((b, n, kv * dh), seed + 1)
    bpt.kv4_store(cache, k, v, ints(*[0] * b), counts=ints(*lens))
    out = []
    for i in range(b):
        one = {}
        for name, x in (("k", k), ("v", v)):
            codes, scale, low = so.quantise(heads_of(x[i:i + 1, :lens[i]], kv)[0].transpose(1, 0, 2))
            one[name], one[name + "s"], one[name + "m"] = so.values(codes, scale, low), scale, low
        out.append(one)
    return cache, out


@pytest.mark.parametrize("dh", [64, 128])
@pytest.mark.parametrize("kv,n", [(1, 1), (3, 5), (2, 130)])
def test_store_writes_the_oracles_bytes_and_no_others(kv, n, dh):
    b, capacity = 3, 256
    cache = bpt.kv4_cache(b, kv, capacity, dh)
    cache.data.fill_(0xA5)
    rows = bf16((b, n, 2 * kv * dh), n, 2.0, -0.5)  # k and v as columns of one buffer
    rows[0, 0, :64] = 1.25                       # a group without a range
    k, v = rows[..., :kv * dh], rows[..., kv * dh:]
    start, counts = [0, 61, 126], [n, max(n - 2, 0), min(n, 3)]
    bpt.kv4_store(cache, k, v, ints(*start), counts=ints(*counts))
    assert bpt.stream_status() == 0
    got = cache.data.cpu().numpy()
    for i in range(b):
        for h in range(kv):
            pad = np.zeros((start[i], dh))
            kn = np.concatenate((pad, heads_of(k[i:i + 1, :counts[i]], kv)[0, :, h]))
            vn = np.concatenate((pad, heads_of(v[i:i + 1, :counts[i]], kv)[0, :, h]))
            ref, used = so.pack(kn, vn)
            _, old = so.pack(pad, pad) if start[i] else (None, np.zeros((0, used.shape[1]), bool))
            mine = used.copy()
            mine[:old.shape[0]] &= ~old
            block = got[i, h]
            assert np.array_equal(block[:len(ref)][mine], ref[mine])
            rest = np.ones(block.shape, bool)
            rest[:len(ref)] = ~mine
            assert (block[rest] == 0xA5).all()


def test_store_at_every_scale():
    # down to where the scale is no normal number, and whole numbers, whose quotients tie
    rng = np.random.default_rng(0)
    for e in [*range(-133, 120, 9), -126, -125, -122, -120]:
        for x in (rng.standard_normal((1, 64, 128)) * 2.0 ** e, rng.integers(-16, 17, (1, 64, 128)) * 2.0 ** e):
            k = torch.tensor(x).float().bfloat16().cuda()
            cache = bpt.kv4_cache(1, 1, 64, 128)
            bpt.kv4_store(cache, k, k, ints(0))
            kn = heads_of(k, 1)[0, :, 0]
            assert np.array_equal(cache.data[0, 0].cpu().numpy(), so.pack(kn, kn)[0])


def test_load_returns_the_values_and_zeros_past_the_length():
    for dh in (64, 128):
        lens = [70, 3, 0]
        cache, held = filled(3, 2, dh, lens, 128)
        start, n = [65, 0, 0], 8
        k, v = bpt.kv4_load(cache, ints(*lens), n, start=ints(*start))
        for name, got in (("k", k), ("v", v)):
            g = heads_of(got, 2)
            for i in range(3):
                m = max(min(lens[i] - start[i], n), 0)
                ref = held[i][name][:, start[i]:start[i] + m].transpose(1, 0, 2)
                assert (np.abs(g[i, :m] - ref) <= (2.0 ** -8 + 2.0 ** -23) * np.abs(ref) + 2.0 ** -24 * 4).all()
                assert (g[i, m:] == 0).all()
        whole, _ = bpt.kv4_load(cache, ints(*lens), 70)
        assert torch.equal(whole[0, 65:], k[0, :5])
    assert bpt.stream_status() == 0


def test_a_group_with_infinities_or_nans_reads_back_as_nan():
    cache = bpt.kv4_cache(1, 1, 64, 128)
    x = bf16((1, 5, 128), 3)
    x[0, 0, 5], x[0, 1, 70], x[0, 2, 64] = float("inf"), float("nan"), float("-inf")
    x[0, 3, 0], x[0, 3, 1] = 3e38, -3e38  # its range overflows
    x[0, 4, 7] = 3e38
    bpt.kv4_store(cache, x, x, ints(0))
    for got in bpt.kv4_load(cache, ints(5), 5):
        bad = got[0].view(5, 2, 64).isnan()
        assert bad[0].all(1).tolist() == [True, False] and bad[1].all(1).tolist() == [False, True]
        assert bad[2].all(1).tolist() == [False, True] and bad[3].all(1).tolist() == [True, False]
        assert bad.any(2).sum() == 4 and not bad[4].any()


def test_places_outside_the_cache_are_dropped_and_reported():
    cache = bpt.kv4_cache(3, 1, 64, 64)
    cache.data.fill_(0x11)
    x = bf16((3, 4, 64), 1)
    assert bpt.stream_status() == 0
    bpt.kv4_store(cache, x, x, ints(62, -1, 70))
    assert bpt.stream_status() == RANGE and bpt.stream_status() == 0
    ref = bpt.kv4_cache(3, 1, 64, 64)
    ref.data.fill_(0x11)
    bpt.kv4_store(ref, x[:, :2], x[:, :2], ints(62, 0, 0), counts=ints(2, 0, 0))
    bpt.kv4_store(ref, x[:, 1:], x[:, 1:], ints(0, 0, 0), counts=ints(0, 3, 0))
    assert torch.equal(cache.data, ref.data) and bpt.stream_status() == 0
    bpt.kv4_store(ref, x, x, ints(0, 0, 0), counts=ints(5, -1, 0))
    assert bpt.stream_status() == RANGE
    k, _ = bpt.kv4_load(cache, ints(64, 64, 65), 2, start=ints(63, -1, 2 ** 31 - 1))
    assert bpt.stream_status() == RANGE
    assert (k[0, 1] == 0).all() and (k[1, 0] == 0).all() and (k[2] == 0).all() and (k[1, 1] != 0).any()
    bpt.kv4_load(cache, ints(64, 64, 64), 2, start=ints(0, 65, 0))
    assert bpt.stream_status() == RANGE
    bpt.kv4_load(cache, ints(64, 64, 64), 2, start=ints(0, 64, 63))  # past the length, but inside
    assert bpt.stream_status() == 0
    o, lse2 = bpt.kv4_attention(x[:, :1].contiguous(), cache, ints(65, -3, 64), 1, return_lse=True)
    assert bpt.stream_status() == RANGE
    full, _ = bpt.kv4_attention(x[:, :1].contiguous(), cache, ints(64, 0, 64), 1, return_lse=True)
    assert torch.equal(o, full) and bpt.stream_status() == 0


def check_attention(q, cache, held, lens, heads, causal=True, weights=None, **kw):
    b, n, _ = q.shape
    kv, dh = cache.kv_heads, cache.dh
    before = None if weights is None else weights.clone()
    o, lse2 = bpt.kv4_attention(q, cache, ints(*lens), heads, causal=causal, weights=weights, return_lse=True, **kw)
    assert o.shape == (b, n, heads * dh) and lse2.shape == (b, heads, n)
    qn = heads_of(q, heads)
    on, ln = heads_of(o, heads), lse2.double().cpu().numpy()
    group, c = heads // kv, np.log2(np.e) / np.sqrt(dh)
    for i in range(b):
        one = held[i]
        ro, rl, rw = so.attention(qn[i], one["k"], one["v"], causal)
        assert np.array_equal(np.isneginf(ln[i]), np.isneginf(rl))
        live = ~np.isneginf(rl)
        if lens[i] == 0:
            assert (on[i] == 0).all()
            continue
        hh = np.arange(heads) // group
        # the bounds of the module's comment
        big = np.repeat(np.abs(one["km"]) + 31 * one["ks"], 64, -1)              # [kv, len, dh]
        E = (dh + 16) * 2.0 ** -24 * c * np.einsum("nhd,hud->hnu", np.abs(qn[i]), big[hh]).max(-1)  # [heads, n]
        assert (np.abs(ln[i][live] - rl[live]) <= (E + 2.0 ** -20 + 2.0 ** -23 * np.abs(rl))[live]).all()
        s = np.einsum("nhd,hud->hnu", qn[i], one["k"][hh]) / np.sqrt(dh)
        seen = np.arange(lens[i]) < (lens[i] - n + 1 + np.arange(n) if causal else np.full(n, lens[i]))[:, None]
        p = np.where(seen, np.exp2(s * np.log2(np.e) - np.where(live, rl, 0)[..., None]), 0)  # [heads, n, len]
        step = np.repeat(one["vs"], 64, -1)[hh]
        most = np.repeat(np.abs(one["vm"]) + 15 * one["vs"], 64, -1)[hh]
        tol = (2.0 ** -11 * np.einsum("hnu,hud->nhd", p, 15 * step) + 2.0 ** -8 * np.abs(ro)
               + (2 * np.log(2) * E.T[..., None] + 2.0 ** -18) * np.einsum("hnu,hud->nhd", p, most) + 1e-30)
        err = np.abs(on[i] - ro)
        assert (err <= tol).all(), f"o is {(err / tol).max():.2f} times its bound off"
        if weights is not None:
            add = (weights[i] - 0).double().cpu().numpy()[:, :lens[i]]
            base = before[i].double().cpu().numpy()[:, :lens[i]]
            rel = (2 * np.log(2) * E.max() + 2.0 ** -19) * rw + (group * n + 1) * 2.0 ** -24 * (base + rw)
            assert (np.abs(add - base - rw) <= rel + 1e-30).all()
    if weights is not None:
        for i in range(b):
            assert torch.equal(weights[i, :, lens[i]:], before[i, :, lens[i]:])
    assert bpt.stream_status() == 0
    return o


@pytest.mark.parametrize("dh", [64, 128])
@pytest.mark.parametrize("heads,kv,n", [(1, 1, 1), (4, 4, 1), (8, 1, 1), (6, 2, 1), (5, 5, 3), (20, 4, 2), (2, 2, 17),
                                        (40, 1, 1), (9, 3, 12)])
@pytest.mark.parametrize("capacity", [256, 20032])
def test_attention_over_odd_lengths(heads, kv, n, dh, capacity):
    # in a short cache a thread block takes a head; in a long one the blocks of
    # all heads are split over the device
    lens = [1, 64, 0, 65, 200, 63, 127]
    cache, held = filled(len(lens), kv, dh, lens, capacity, seed=heads)
    q = bf16((len(lens), n, heads * dh), 7)
    w = torch.rand((len(lens), kv, capacity), generator=torch.Generator().manual_seed(0)).cuda()
    check_attention(q, cache, held, lens, heads)
    check_attention(q, cache, held, lens, heads, weights=w)
    check_attention(q, cache, held, lens, heads, causal=False, weights=w)


@pytest.mark.parametrize("dh,heads,kv,n,lens,capacity", [
    (128, 2, 2, 1, [5000, 1, 4096], 8192), (64, 4, 1, 4, [9001], 9024), (128, 8, 8, 1, [777] * 5, 832),
    (64, 1, 1, 1, [20000], 20032), (128, 16, 2, 1, [3001, 12], 3008),
])
def test_attention_over_long_caches(dh, heads, kv, n, lens, capacity):
    cache, held = filled(len(lens), kv, dh, lens, capacity, seed=5)
    q = bf16((len(lens), n, heads * dh), 8, 2.0)
    w = torch.zeros((len(lens), kv, capacity), device="cuda")
    o = check_attention(q, cache, held, lens, heads, weights=w)
    again = bpt.kv4_attention(q, cache, ints(*lens), heads)
    assert torch.equal(o, again)  # the order of its sums does not change from call to call
    assert torch.allclose(w.sum((1, 2)).double(), torch.full((len(lens),), float(heads * n), dtype=torch.float64,
                                                                 device="cuda"), rtol=1e-4)


@pytest.mark.parametrize("dh,heads,kv,n", [(64, 9, 3, 25), (128, 80, 16, 8), (64, 96, 96, 1), (128, 20, 20, 3)])
def test_attention_of_many_queries_over_short_contexts(dh, heads, kv, n):
    # more results than the device has blocks: a warp joins a column, several a block, the last ones of a sequence not a
    # whole block's; some columns' heads have no token
    lens = [93, 1, 0, 64, 65, 300, 7, 128, 0, 33, 90, 2, 5]
    cache, held = filled(len(lens), kv, dh, lens, 320, seed=81)
    q = bf16((len(lens), n, heads * dh), 82)
    w = torch.rand((len(lens), kv, 320), generator=torch.Generator().manual_seed(1)).cuda()
    check_attention(q, cache, held, lens, heads)
    check_attention(q, cache, held, lens, heads, weights=w)


def test_attention_with_large_and_equal_scores():
    # scores of about a thousand, whose exponentials overflow without the maximum, and equal ones: o is V's mean
    for dh in (64, 128):
        cache, held = filled(1, 1, dh, [150], 192, seed=11)
        q = bf16((1, 2, 2 * dh), 12, 60.0)
        q[:, :, dh:] = 0
        o = check_attention(q, cache, held, [150], 2, causal=False)
        mean = held[0]["v"][0].mean(0)
        assert (np.abs(heads_of(o, 2)[0, 0, 1] - mean) <= 2.0 ** -8 * np.abs(mean) + 2.0 ** -11 * 15 * held[0]["vs"].max()).all()


@pytest.mark.parametrize("capacity", [512, 20032])
@pytest.mark.parametrize("pattern", ["alternating", "large and unseen first", "large and unseen last", "rising", "falling",
                                     "tiny", "huge"])
def test_values_of_very_different_size(pattern, capacity):
    # V's rows scaled by powers of two, and scores (K's rows are constant) that
    # raise the small ones. What lies 2^-31 below the largest product of weight
    # and scale may be lost.
    n, dh = 400, 128
    t = np.arange(n)
    size, score = {"alternating": (np.where(t % 2, 30, -30), 0 * t),
                   "large and unseen first": (np.where(t < 70, 60, 0), np.where(t < 70, -150, 0)),
                   "large and unseen last": (np.where(t < 330, 0, 60), np.where(t < 330, 0, -150)),
                   "rising": (t // 8, -t // 16), "falling": (-(t // 8), t // 16),
                   "tiny": (0 * t - 90, 0 * t), "huge": (0 * t + 100, 0 * t)}[pattern]
    g = np.random.default_rng(5)
    v = torch.tensor(g.standard_normal((1, n, dh)) * 2.0 ** size[:, None]).float().bfloat16().cuda()
    k = torch.tensor(np.broadcast_to(score[:, None] / np.sqrt(dh), (n, dh))[None].copy()).float().bfloat16().cuda()
    q = torch.ones((1, 1, dh), dtype=torch.bfloat16, device="cuda")
    cache = bpt.kv4_cache(1, 1, capacity, dh)
    bpt.kv4_store(cache, k, v, ints(0))
    o = heads_of(bpt.kv4_attention(q, cache, ints(n), 1), 1)[0, 0, 0]
    kc, vc = (so.quantise(heads_of(x, 1)[0, :, 0]) for x in (k, v))
    s = so.values(*kc) @ np.ones(dh) / np.sqrt(dh)
    p = np.exp(s - s.max())
    p /= p.sum()
    step, low = np.repeat(vc[1], 64, -1), np.repeat(vc[2], 64, -1)
    ref = p @ so.values(*vc)
    E = (dh + 16) * 2.0 ** -24 * np.log2(np.e) / np.sqrt(dh) * dh * np.abs(so.values(*kc)).max()
    tol = (2.0 ** -8 * np.abs(ref) + (2.0 ** -11 + 2 * np.log(2) * E + 2.0 ** -18) * (p @ (np.abs(low) + 15 * step))
           + n * 2.0 ** -31 * 15 * (p[:, None] * step).max(0))
    assert (np.abs(o - ref) <= tol).all(), f"{(np.abs(o - ref) / tol).max():.2f} times the bound"
    assert bpt.stream_status() == 0


@pytest.mark.parametrize("dh", [64, 128])
@pytest.mark.parametrize("size", [-120, -60, 60, 110])
def test_queries_of_any_size(size, dh):
    # scores of the usual size from very large or small queries on keys of the inverse size
    cache = bpt.kv4_cache(1, 1, 256, dh)
    g = np.random.default_rng(6)
    k = torch.tensor(g.standard_normal((1, 150, dh)) * 2.0 ** -size).float().bfloat16().cuda()
    q = torch.tensor(g.standard_normal((1, 1, dh)) * 2.0 ** size).float().bfloat16().cuda()
    v = bf16((1, 150, dh), 7)
    bpt.kv4_store(cache, k, v, ints(0))
    one = {}
    for name, x in (("k", k), ("v", v)):
        codes, scale, low = so.quantise(heads_of(x, 1)[0].transpose(1, 0, 2))
        one[name], one[name + "s"], one[name + "m"] = so.values(codes, scale, low), scale, low
    check_attention(q, cache, [one], [150], 1)


@pytest.mark.parametrize("dh", [64, 128])
def test_the_mean_of_a_long_cache_keeps_its_accuracy(dh):
    # Zero queries: every weight is the same and P' is V's scale, without a
    # rounding; o is V's mean. 128 heads of 131072 tokens, the same 64 over and
    # over, are long runs for every warp. What is left beside o's rounding are
    # the fp32 sums of at most 31 scale a token: 2^-20 of that.
    b, kv, blocks = 4, 32, 2048
    small, held = filled(b, kv, dh, [64] * b, 64, seed=21)
    cache = bpt.KV4Cache(small.data.repeat(1, 1, blocks, 1), dh)
    q = torch.zeros((b, 1, kv * dh), dtype=torch.bfloat16, device="cuda")
    n = 64 * blocks
    o, lse2 = bpt.kv4_attention(q, cache, ints(*[n] * b), kv, return_lse=True)
    assert ((lse2 - np.log2(n)).abs() <= 2.0 ** -20 + 2.0 ** -19).all()
    got = heads_of(o, kv)[:, 0]
    mean = np.stack([x["v"].mean(1) for x in held])
    step = np.stack([x["vs"].max() for x in held])[:, None, None]
    assert (np.abs(got - mean) <= 2.0 ** -8 * np.abs(mean) + 2.0 ** -20 * 31 * step).all()


def test_what_lies_past_the_length_does_not_matter_and_nan_inside_shows():
    cache, held = filled(2, 2, 128, [100, 30], 192, seed=13)
    q = bf16((2, 1, 4 * 128), 14)
    o = check_attention(q, cache, held, [100, 30], 4)
    x = torch.full((2, 60, 2 * 128), float("nan"), dtype=torch.bfloat16, device="cuda")
    bpt.kv4_store(cache, x, x, ints(100, 30))
    assert torch.equal(o, bpt.kv4_attention(q, cache, ints(100, 30), 4))
    o = bpt.kv4_attention(q, cache, ints(101, 30), 4)
    assert o[0].isnan().all() and not o[1].isnan().any()


def test_strided_queries_streams_and_graphs():
    dh, heads, kv, lens = 128, 4, 2, [90, 17]
    cache, held = filled(2, kv, dh, lens, 128, seed=15)
    rows = bf16((2, 3, (heads + 2 * kv) * dh), 16)
    q = rows[..., :heads * dh]
    o = check_attention(q, cache, held, lens, heads)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    check_attention(q, cache, held, lens, heads, stream=side)
    # two graphs captured one after the other share a memory pool; replayed in turn, on new lengths and queries
    ln, graphs, outs = ints(*lens), [], []
    w = torch.zeros((2, kv, 128), device="cuda")
    pool = torch.cuda.graph_pool_handle()
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, pool=pool):
            outs.append(bpt.kv4_attention(q, cache, ln, heads, weights=w))
        graphs.append(g)
    ln.copy_(ints(60, 3))
    rows.mul_(0.5)
    w.zero_()
    for g in graphs:
        g.replay()
    torch.cuda.synchronize()
    w2 = torch.zeros_like(w)
    ref = bpt.kv4_attention(q, cache, ln, heads, weights=w2)
    bpt.kv4_attention(q, cache, ln, heads, weights=w2)
    assert torch.equal(outs[0], ref) and torch.equal(outs[1], ref) and torch.equal(w, w2)


@pytest.mark.parametrize("capacity", [256, 20032])
def test_a_captured_step_and_eviction(capacity):
    # one decoded token (positions, store, attention with weights, the new length) and an eviction, captured and
    # replayed on new queries, against the same calls made one by one
    b, heads, kv, dh, keep = 2, 4, 2, 64, 40
    lens = [130, 77]
    base, _ = filled(b, kv, dh, lens, capacity, seed=31)
    freq, _ = bpt.rotary_frequencies(dh)
    rows = bf16((b, 1, (heads + 2 * kv) * dh), 32)

    def step(cache, small, ln, w):
        q, k = bpt.rotary(rows[..., :heads * dh], rows[..., heads * dh:(heads + kv) * dh], heads, kv, freq,
                          positions=ln.view(b, 1))
        bpt.kv4_store(cache, k, rows[..., (heads + kv) * dh:], ln)
        ln += 1
        o, lse2 = bpt.kv4_attention(q, cache, ln, heads, weights=w, return_lse=True)
        return (o, lse2, *bpt.kv4_evict(cache, w, ln, keep, 7, small), *bpt.kv4_load(small, ln.clamp(max=keep), keep))

    def state():
        return (bpt.KV4Cache(base.data.clone(), dh), bpt.kv4_cache(b, kv, keep, dh), ints(*lens),
                torch.zeros((b, kv, capacity), device="cuda"))

    step(*state())  # loads what a capture must not load
    one, two = state(), state()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(*one)
    for new in range(3):
        rows.copy_(bf16(rows.shape, 40 + new))
        graph.replay()
        ref = step(*two)
        torch.cuda.synchronize()
        for x, y in zip((*out, *one[2:]), (*ref, *two[2:])):
            assert torch.equal(x, y)
        assert torch.equal(one[0].data, two[0].data) and torch.equal(one[1].data, two[1].data)
    assert bpt.stream_status() == 0


@pytest.mark.parametrize("heads,kv,dh,start", [(4, 2, 64, 300), (16, 8, 128, 9000)])
def test_calls_that_follow_closely_wait_for_each_other(heads, kv, dh, start):
    # each call reads what the one ahead writes, or writes what that one reads, with nothing between them; the same
    # calls with the device idle before each give the same bits
    b, steps, keep, width = 4, 12, 128, kv * dh
    capacity = start + 100
    base, _ = filled(b, kv, dh, [start - 11 * i for i in range(b)], capacity, seed=61)
    rows = bf16((b, 1, heads * dh + 2 * width), 62)
    freq, _ = bpt.rotary_frequencies(dh)

    def run(between):
        cache, small = bpt.KV4Cache(base.data.clone(), dh), bpt.kv4_cache(b, kv, keep, dh)
        lens = ints(*[start - 11 * i for i in range(b)])
        at = [lens + i for i in range(steps + 1)]
        w = torch.zeros((b, kv, cache.capacity), device="cuda")
        q, k, v = rows[..., :heads * dh].clone(), rows[..., heads * dh:-width].clone(), rows[..., -width:].clone()
        out = []
        for i in range(steps):
            between()
            bpt.rotary(q, k, heads, kv, freq, positions=at[i].view(b, 1), q_out=q, k_out=k)
            between()
            bpt.kv4_store(cache, k, v, at[i])
            between()
            out.append(bpt.kv4_attention(q, cache, at[i + 1], heads, weights=w))
            between()
            out.extend(bpt.kv4_evict(cache, w, at[i + 1], keep, 7, small))  # reads the weights, rewrites `small`
            between()
            out.extend(bpt.kv4_load(small, out[-2], keep))
            between()
            out.append(bpt.kv4_attention(q, small, out[-4], heads, weights=out[-3]))
            between()
            bpt.kv4_store(small, k, v, ints_zero)  # rewrites what the attention ahead reads
        return [*out, q, k, w, cache.data, small.data]

    ints_zero = ints(*[0] * b)
    ref = run(torch.cuda.synchronize)
    for _ in range(3):
        for x, y in zip(run(lambda: None), ref, strict=True):
            assert torch.equal(x, y)
    assert bpt.stream_status() == 0


def test_captured_behind_copies_fills_and_other_streams():
    # what a captured call follows is a copy, a fill, a kernel of torch's and another stream's call
    lens, capacity = [500, 333], 512
    base, _ = filled(2, 2, 64, lens, capacity, seed=71)
    x, y = bf16((2, 1, 4 * 64), 72), torch.empty((2, 1, 4 * 64), dtype=torch.bfloat16, device="cuda")
    kv = bf16((2, 1, 2 * 64), 73)
    n, freq = ints(*lens), bpt.rotary_frequencies(64)[0]
    w = torch.zeros((2, 2, capacity), device="cuda")
    cache = bpt.KV4Cache(base.data.clone(), 64)
    side = torch.cuda.Stream()

    def step():
        cache.data.copy_(base.data)
        bpt.kv4_store(cache, kv, kv, n)
        y.copy_(x)
        bpt.rotary(y, None, 4, 0, freq, offset=5, q_out=y)
        w.zero_()
        o = bpt.kv4_attention(y, cache, n, 4, weights=w)
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            k, v = bpt.kv4_load(cache, n, 500)
        bpt.rotary(y, None, 4, 0, freq, offset=6, q_out=y)
        torch.cuda.current_stream().wait_stream(side)
        bpt.kv4_store(cache, kv, kv, n - 1)
        return o, k, v, bpt.kv4_attention(y, cache, n, 4, weights=w)

    ref = [t.clone() for t in step()] + [w.clone(), y.clone(), cache.data.clone()]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for _ in range(3):
        graph.replay()
        torch.cuda.synchronize()
        for a, e in zip((*out, w, y, cache.data), ref, strict=True):
            assert torch.equal(a, e)
    assert bpt.stream_status() == 0


def test_a_cache_that_is_not_what_it_says_is_refused():
    cache, other = bpt.kv4_cache(1, 2, 64, 64), bpt.kv4_cache(1, 2, 64, 128)
    k, n = bf16((1, 1, 2 * 64), 0), ints(0)
    wide = bf16((1, 1, 2 * 128), 0)
    cache.dh = 128
    for call in (lambda: bpt.kv4_store(cache, wide, wide, n), lambda: bpt.kv4_load(cache, n, 1),
                 lambda: bpt.kv4_attention(wide, cache, n, 2),
                 lambda: bpt.kv4_evict(other, torch.zeros((1, 2, 64), device="cuda"), n, 8, 1, cache)):
        with pytest.raises(ValueError, match="blocks are 4608 bytes"):
            call()
    cache.dh, cache.data = 64, cache.data[..., :64]
    with pytest.raises(ValueError, match="contiguous uint8"):
        bpt.kv4_store(cache, k, k, n)
    assert bpt.stream_status() == 0


def test_two_streams_at_once():
    lens = [1000, 400]
    cache, _ = filled(2, 4, 64, lens, 1024, seed=17)
    q = [bf16((2, 1, 8 * 64), 18 + i) for i in range(2)]
    ln = ints(*lens)
    ref = [bpt.kv4_attention(x, cache, ln, 8) for x in q]
    streams = [torch.cuda.Stream() for _ in q]
    torch.cuda.synchronize()
    got = [[bpt.kv4_attention(x, cache, ln, 8, stream=s) for x, s in zip(q, streams)] for _ in range(20)]
    torch.cuda.synchronize()
    for pair in got:
        assert torch.equal(pair[0], ref[0]) and torch.equal(pair[1], ref[1])
    assert all(bpt.stream_status(s) == 0 for s in streams)


def check_evict(dh, kv, lens, capacity, keep, recent, out_capacity, weights, rows=True):
    b = len(lens)
    cache = bpt.kv4_cache(b, kv, capacity, dh)
    cache.data.random_(0, 256, generator=torch.Generator(device="cuda").manual_seed(3))
    out = bpt.kv4_cache(b, kv, out_capacity, dh)
    out.data.fill_(0x5A)
    kept, new, moved = bpt.kv4_evict(cache, weights, ints(*lens), keep, recent, out)
    assert bpt.stream_status() == 0
    assert new.tolist() == [min(x, keep) for x in lens]
    wn, mn, kn = weights.cpu().numpy(), moved.cpu().numpy(), kept.cpu().numpy()
    src, dst = (cache.data.cpu().numpy(), out.data.cpu().numpy()) if rows else (None, None)
    half, par = dh // 2, dh // 64 * 4
    v_at = 64 * (half + par)

    def row(data, r):  # a row's bytes in the order of its dimensions
        blk, r = data[r // 64], r % 64
        words = blk[v_at + r * half:v_at + (r + 1) * half].reshape(-1, 4)
        if dh == 128:
            words = words.reshape(8, 2, 4)[[p ^ (4 if r & 2 else 0) for p in range(8)]].reshape(-1, 4)
        return np.concatenate((blk[r * half:(r + 1) * half], blk[64 * half + r * par:64 * half + (r + 1) * par],
                               words.reshape(-1), blk[v_at + 64 * half + r * par:v_at + 64 * half + (r + 1) * par]))

    for i in range(b):
        for h in range(kv):
            ref = so.kept_tokens(wn[i, h], lens[i], keep, recent)
            assert kn[i, h].tolist() == ref + [-1] * (keep - len(ref))
            assert np.array_equal(mn[i, h, :len(ref)], wn[i, h, ref], equal_nan=True) and (mn[i, h, len(ref):] == 0).all()
            if not rows:
                continue
            for j, r in enumerate(ref):
                assert np.array_equal(row(dst[i, h], j), row(src[i, h], r))
            for j in range(len(ref), out_capacity):
                assert (row(dst[i, h], j) == 0x5A).all()


@pytest.mark.parametrize("dh", [64, 128])
@pytest.mark.parametrize("keep,recent", [(1, 0), (1, 1), (50, 0), (64, 64), (65, 10), (128, 1)])
def test_evict_keeps_the_newest_and_the_heaviest(keep, recent, dh):
    lens = [0, 1, 50, 129, 256, 70]
    g = torch.Generator().manual_seed(keep)
    w = torch.randn((len(lens), 2, 256), generator=g).exp().cuda()
    check_evict(dh, 2, lens, 256, keep, recent, 128, w)


def test_evict_ties_signs_infinities_and_nan():
    g = torch.Generator().manual_seed(1)
    w = torch.randint(0, 4, (3, 1, 320), generator=g).float() - 1  # many ties, zeros, negative ones
    w[w == 0] *= torch.where(torch.rand((w == 0).sum(), generator=g) < 0.5, -1.0, 1.0)  # both zeros
    w[1] = 0
    w[2, 0, ::7], w[2, 0, 3::50], w[2, 0, 5::90] = float("inf"), float("nan"), float("-inf")
    for keep in (3, 100, 300):
        check_evict(64, 1, [320, 300, 317], 320, keep, 2, 320, w.cuda())


@pytest.mark.parametrize("kind", ["spread", "ties", "equal", "odd values"])
@pytest.mark.parametrize("capacity,keep", [(64, 1), (512, 200), (4096, 1500)])
def test_evict_from_many_short_rows(capacity, keep, kind):
    # more rows than two blocks an SM
    lens = [capacity - 7 * i for i in range(8)] + [0, 1]
    g = torch.Generator().manual_seed(capacity)
    w = torch.randn((len(lens), 31, capacity), generator=g)
    w = {"spread": w.mul(3).exp(), "ties": w.mul(2).round(), "equal": torch.zeros_like(w), "odd values": w}[kind]
    if kind == "odd values":
        w[:, :, ::5], w[:, 3, 1::5], w[:, 4, 2::7] = -0.0, float("nan"), -float("inf")
    check_evict(64, 31, lens, capacity, keep, keep // 9, capacity, w.cuda(), rows=False)


@pytest.mark.parametrize("length,heads", [(1023, 2), (1025, 2), (5000, 2), (33333, 2), (16390, 40), (16390, 80),
                                          (200001, 1)])
@pytest.mark.parametrize("ties", [False, True])
def test_evict_from_long_caches(length, heads, ties):
    # one, two and four blocks a row, keys in shared memory or not; few values let ties reach across every part
    g = torch.Generator().manual_seed(length)
    capacity = (length + 63) // 64 * 64
    w = torch.rand((1, heads, capacity), generator=g) * 50
    w = (w.round() if ties else w).cuda()
    check_evict(64, heads, [length], capacity, 300, 33, 320, w, rows=ties)


def test_evict_without_shared_memory_for_the_keys():
    # 150 rows fill the device with one block each; 45000 tokens are more than a block keeps
    g = torch.Generator().manual_seed(3)
    w = (torch.rand((1, 150, 45056), generator=g) * 50).cuda()
    check_evict(64, 150, [45001], 45056, 100, 3, 128, w, rows=False)


def test_a_run_of_them_together():
    """Prompt: projection, positions, dense attention, store. Then tokens one by one (positions, store, attention with
    weights), an eviction, and tokens again; the last attention against the oracle on what the cache should hold."""
    b, s, heads, dh = 2, 70, 4, 64
    h = heads * dh
    g = torch.Generator().manual_seed(0)
    x = torch.randn((b, s + 6, h), generator=g).bfloat16().cuda()
    Wqkv = (torch.randn((h, 3 * h), generator=g) / h ** 0.5).bfloat16().cuda()
    bqkv = torch.zeros(3 * h, dtype=torch.bfloat16, device="cuda")
    freq, m = bpt.rotary_frequencies(dh)
    cache, small = bpt.kv4_cache(b, heads, 100, dh), bpt.kv4_cache(b, heads, 40, dh)
    weights = torch.zeros((b, heads, cache.capacity), device="cuda")
    q, k, v = bpt.qkv_projection(x[:, :s].contiguous(), Wqkv, bqkv)
    q, k = bpt.rotary(q, k, heads, heads, freq)
    dense = bpt.attention(q, k, v, heads, s, s, True)
    assert torch.isfinite(dense).all()
    bpt.kv4_store(cache, k, v, ints(0, 0))
    held = {"k": k, "v": v}
    lens = torch.full((b,), s, dtype=torch.int32, device="cuda")
    for t in range(6):
        q1, k1, v1 = bpt.qkv_projection(x[:, s + t:s + t + 1].contiguous(), Wqkv, bqkv)
        at = torch.full((b, 1), s + t, dtype=torch.int64, device="cuda")
        q1, k1 = bpt.rotary(q1, k1, heads, heads, freq, positions=at)
        bpt.kv4_store(cache, k1, v1, lens)
        lens += 1
        held = {"k": torch.cat((held["k"], k1), 1), "v": torch.cat((held["v"], v1), 1)}
        o = bpt.kv4_attention(q1, cache, lens, heads, weights=weights)
        if t == 2:
            kept, lens, weights = bpt.kv4_evict(cache, weights, lens, 40, 8, small)
            cache, length = small, s + t + 1
            places = kept.long().transpose(1, 2)[..., None].expand(-1, -1, -1, dh)
            held = {n: torch.gather(z.view(b, length, heads, dh), 1, places).flatten(2) for n, z in held.items()}
    assert lens.tolist() == [43, 43] and bpt.stream_status() == 0
    one = [{n: so.values(*so.quantise(heads_of(z[i:i + 1], heads)[0].transpose(1, 0, 2))) for n, z in held.items()}
           for i in range(b)]
    for i in range(b):
        ro, _, _ = so.attention(heads_of(q1, heads)[i], one[i]["k"], one[i]["v"], True)
        err = np.abs(heads_of(o, heads)[i] - ro)
        assert (err <= 2.0 ** -8 * (np.abs(ro) + np.abs(one[i]["v"]).max() + 1e-3)).all()
