"""Cases that measure rotary positions, the 4-bit key/value cache, attention over it, and eviction from it.

`run` computes each operator in elementary torch operations where `own` is false, and by the framework's calls where
it is true. `exact` computes the same results in 64 bits.

The cache's layout (one uint8 tensor [b, kv_heads, capacity / 64, block bytes]): a block holds 64 tokens of one
key/value head, as [K codes | K parameters | V codes | V parameters]. Each token's row of codes has dh / 2 bytes: a
32-bit word holds 8 consecutive dimensions (dimension 8u + i in bits 4i .. 4i + 3 of word u; the words of K are rotated
left by 3 bits), and the words of a row are permuted (`_word_order`). The parameters are two bf16, scale then minimum, per token and 64 dimensions; a code c stands
for minimum + scale c.
"""

import math

import torch

own = False

BLOCK = 64
GROUP = 64


# ------------------------------------------------------------------ the cache's layout

def _sections(dh):
    """Byte offsets of K codes, K parameters, V codes, V parameters in a block, and the block's bytes."""
    codes, params = BLOCK * dh // 2, BLOCK * (dh // GROUP) * 4
    return 0, codes, codes + params, 2 * codes + params, 2 * (codes + params)


def _word_order(dh, which, device):
    """[64, dh / 8]: the word u (dimensions 8u .. 8u + 7) that a block's row r holds at each place."""
    place = torch.arange(dh // 8, device=device)
    if which == "k":
        per = dh // 32
        return ((place % per) * 4 + place // per).expand(BLOCK, -1)
    if dh == 64:
        return place.expand(BLOCK, -1)
    row = torch.arange(BLOCK, device=device)[:, None]
    return (place % 2) * 8 + ((place // 2) ^ (4 * ((row >> 1) & 1)))


def _quantise(x):
    """Codes (0 .. 15, in 64 bits), scale and minimum (in 32 bits) of x [..., dh], per 64 dimensions."""
    g = x.float().unflatten(-1, (-1, GROUP))
    low, high = g.amin(-1, keepdim=True), g.amax(-1, keepdim=True)
    scale = ((high - low) / 15).bfloat16().float()
    live = scale >= 2.0 ** -126
    scale = torch.where(live, scale, torch.zeros_like(scale))
    inverse = torch.where(live, 1 / scale, torch.zeros_like(scale))
    codes = ((g.double() - low.double()) * inverse.double()).round().clamp(0, 15)
    return codes, scale, low


def _rotate(words, by):
    """32-bit words rotated left by `by` bits."""
    return (words << by) | ((words >> (32 - by)) & ((1 << by) - 1))


def _pack(x, which):
    """Code bytes [..., blocks, 32 dh] and parameter bytes of x [..., capacity, dh] (capacity a multiple of 64)."""
    dh = x.shape[-1]
    codes, scale, low = _quantise(x)
    codes = codes.to(torch.uint8).flatten(-2)
    data = codes[..., 0::2] | (codes[..., 1::2] << 4)
    if which == "k":
        data = _rotate(data.view(torch.int32), 3).view(torch.uint8)
    data = data.unflatten(-1, (dh // 8, 4)).unflatten(-3, (-1, BLOCK))
    order = _word_order(dh, which, x.device)[..., None].expand(data.shape)
    data = torch.gather(data, -2, order)
    params = torch.cat((scale, low), -1).bfloat16().view(torch.uint8).flatten(-2).unflatten(-2, (-1, BLOCK))
    return data.flatten(-3), params.flatten(-2)


def _unpack(data, dh, which):
    """The values [b, kv_heads, capacity, dh] that a cache holds, in 32 bits."""
    k_codes, k_params, v_codes, v_params, end = _sections(dh)
    at, params, stop = (k_codes, k_params, v_codes) if which == "k" else (v_codes, v_params, end)
    words = data[..., at:params].unflatten(-1, (BLOCK, dh // 8, 4))
    back = torch.argsort(_word_order(dh, which, data.device), -1)[..., None].expand(words.shape)
    words = torch.gather(words, -2, back)
    if which == "k":
        words = _rotate(words.view(torch.int32), 29).view(torch.uint8)
    codes = torch.stack((words & 15, words >> 4), -1).flatten(-3).float().unflatten(-1, (-1, GROUP))
    pair = data[..., params:stop].unflatten(-1, (BLOCK, dh // GROUP, 4)).contiguous().view(torch.bfloat16).float()
    return (pair[..., 1:] + pair[..., :1] * codes).flatten(-2).flatten(2, 3)


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # one new token of each of 32 sequences, far into a long context
        dict(name="rotary token", op="rotary", dtype="bf16", b=32, s=1, heads=32, kv_heads=32, dh=128, rot=128,
             interleaved=False, inverse=False, own_positions=True, far=900001, factor=32.0, fused=False),
        # the whole sequence of the 7B-class layer, in training or as a prompt
        dict(name="rotary 32k tokens", op="rotary", dtype="bf16", b=1, s=32768, heads=32, kv_heads=32, dh=128, rot=128,
             interleaved=False, inverse=False, own_positions=False, far=0, factor=1.0, fused=False),
        # the gradient on its way back to the projection, fp32, half of each head rotated, rows of one fused buffer
        dict(name="rotary backward", op="rotary", dtype="fp32", b=2, s=2047, heads=16, kv_heads=16, dh=64, rot=32,
             interleaved=True, inverse=True, own_positions=False, far=0, factor=1.0, fused=True),
        # one decoded token a sequence, each at its own place
        dict(name="store token", op="store", b=64, n=1, heads=32, dh=128, capacity=1024),
        # prompts of different lengths in a padded batch
        dict(name="store prompts", op="store", b=4, n=8191, heads=16, dh=128, capacity=8256),
        # the smallest call: a short context of one sequence
        dict(name="attend short", op="attend", b=1, n=1, heads=4, kv_heads=4, dh=64, longest=200, spread=0,
             weights=False, empty=False),
        # a serving batch with ragged lengths and a slot that is not in use
        dict(name="attend batch", op="attend", b=16, n=1, heads=32, kv_heads=32, dh=128, longest=4096, spread=3500,
             weights=False, empty=True),
        # a few drafted tokens at once, shared heads, an odd length
        dict(name="attend 7 tokens", op="attend", b=4, n=7, heads=16, kv_heads=4, dh=64, longest=8191, spread=1000,
             weights=False, empty=False),
        # shared heads over a long context, with the weights that an eviction goes by
        dict(name="attend 32k weights", op="attend", b=8, n=1, heads=32, kv_heads=8, dh=128, longest=32768,
             spread=12000, weights=True, empty=False),
        # the largest: sixteen contexts of about 32k tokens, every head its own
        dict(name="attend 32k batch", op="attend", b=16, n=1, heads=32, kv_heads=32, dh=128, longest=32768,
             spread=8000, weights=False, empty=False),
        # a short context cut in half
        dict(name="evict short", op="evict", b=1, kv_heads=4, dh=64, longest=500, spread=0, keep=250, recent=30),
        # long contexts cut to an eighth
        dict(name="evict 32k", op="evict", b=4, kv_heads=16, dh=128, longest=32768, spread=9000, keep=4096, recent=1024),
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    most = [max(work(c)[x] for c in listed()) for x in ("bytes", "flops")]
    while True:
        op = rng.choice(("rotary", "store", "attend", "attend", "evict"))
        dh = rng.choice((64, 128))
        kv_heads = rng.choice((1, 2, 4, 8, 16, 32))
        b = _log(rng, 1, 48)
        if op == "rotary":
            case = dict(op=op, dtype=rng.choice(("bf16", "bf16", "fp32")), b=b, s=_log(rng, 1, 16384),
                        heads=kv_heads * rng.choice((1, 1, 2, 4)), kv_heads=kv_heads, dh=dh,
                        rot=rng.choice((dh, dh, dh // 2, dh // 4, 24)), interleaved=rng.random() < 0.5,
                        inverse=rng.random() < 0.4, own_positions=rng.random() < 0.5,
                        far=rng.choice((0, _log(rng, 1, 1 << 21))), factor=rng.choice((1.0, 4.0, 32.0)),
                        fused=rng.random() < 0.5)
        elif op == "store":
            n = rng.choice((1, _log(rng, 1, 8192)))
            case = dict(op=op, b=b, n=n, heads=kv_heads, dh=dh, capacity=64 * ((n + rng.randrange(1, 2000) + 63) // 64))
        elif op == "attend":
            longest = _log(rng, 1, 60000)
            n = rng.choice((1, 1, 1, rng.randrange(2, 17)))
            case = dict(op=op, b=b, n=n, heads=kv_heads * rng.choice((1, 1, 2, 4, 5, 8)), kv_heads=kv_heads, dh=dh,
                        longest=longest, spread=int(longest * rng.random()), weights=rng.random() < 0.4,
                        empty=b > 1 and rng.random() < 0.3)
        else:
            longest = _log(rng, 8, 60000)
            keep = max(1, int(longest * rng.uniform(0.05, 1.0)))
            case = dict(op=op, b=b, kv_heads=kv_heads, dh=dh, longest=longest, spread=int(longest * 0.5 * rng.random()),
                        keep=keep, recent=int(keep * rng.random() * 0.6))
        if work(case)["bytes"] <= 0.5 * most[0] and work(case)["flops"] <= most[1]:
            return case


def _lengths(case):
    """Cached tokens of each sequence: `longest` less a scattered part of `spread`; the last one none where `empty`."""
    n = [case["longest"] - (i * 40503 % (case["spread"] + 1)) for i in range(case["b"])]
    return n[:-1] + [0] if case.get("empty") else n


def _counts(case):
    """New tokens of each sequence of a padded batch, and where they go."""
    n = [max(1, case["n"] - (i * 1237 % (case["n"] // 3 + 1))) for i in range(case["b"])]
    start = [(i * 40503 + 17) % (case["capacity"] - case["n"] + 1) for i in range(case["b"])]
    return n, start


def _row_bytes(dh):
    return 2 * (dh // 2 + dh // GROUP * 4)


def work(case):
    op, b, dh = case["op"], case["b"], case["dh"]
    if op == "rotary":
        rows = b * case["s"]
        per = (case["heads"] + case["kv_heads"])
        size = 4 if case["dtype"] == "fp32" else 2
        return {"bytes": rows * per * dh * size * 2 + (rows * 8 if case["own_positions"] else 0),
                "flops": rows * per * case["rot"] * 3}
    if op == "store":  # the new rows in, the cache's bytes written and read back, the values out
        rows = sum(_counts(case)[0]) * case["heads"]
        return {"bytes": rows * (2 * dh * 2 + 2 * _row_bytes(dh)) + b * case["n"] * case["heads"] * 2 * dh * 2,
                "flops": rows * 2 * dh * 6}
    if op == "attend":
        rows = sum(_lengths(case)) * case["kv_heads"]
        q = b * case["n"] * case["heads"]
        group = case["heads"] // case["kv_heads"] * case["n"]
        return {"bytes": rows * (_row_bytes(dh) + (8 if case["weights"] else 0)) + q * (dh * 4 + 4),
                "flops": 4 * rows * group * dh}
    kept = sum(min(n, case["keep"]) for n in _lengths(case)) * case["kv_heads"]
    seen = sum(_lengths(case)) * case["kv_heads"]
    # every weight read; the kept rows, their weights and their places written; the rows read back, the values out
    return {"bytes": seen * 4 + kept * (3 * _row_bytes(dh) + 8)
            + b * case["keep"] * case["kv_heads"] * 2 * dh * 2, "flops": seen + kept * 2 * dh * 2}


# ------------------------------------------------------------------ what a program has in hand

def _frequencies(rot, factor, original=4096, base=10000.0, low=1.0, high=32.0):
    """Radians per position of each pair, in 64 bits, and the magnitude: plain for factor 1; otherwise those that turn
    less than `low` times over the original length divided by `factor`, those over `high` left, the others between."""
    f = base ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    if factor == 1.0:
        return f, 1.0
    w = ((original * f / (2 * math.pi) - low) / (high - low)).clamp(0, 1)
    return f * (w + (1 - w) / factor), 0.1 * math.log(factor) + 1


def _cache(case, capacity, gen, dev):
    """A cache of `capacity` tokens a sequence: keys with an offset of their own in each dimension, values without."""
    b, h, dh = case["b"], case["kv_heads"], case["dh"]
    data = torch.empty((b, h, capacity // BLOCK, _sections(dh)[-1]), dtype=torch.uint8, device=dev)
    k_codes, k_params, v_codes, v_params, end = _sections(dh)
    offset = torch.randn((h, 1, dh), device=dev, generator=gen)
    for i in range(b):
        k = torch.randn((h, capacity, dh), device=dev, generator=gen).add_(offset).bfloat16()
        v = torch.randn((h, capacity, dh), device=dev, generator=gen).bfloat16()
        data[i, ..., k_codes:k_params], data[i, ..., k_params:v_codes] = _pack(k, "k")
        data[i, ..., v_codes:v_params], data[i, ..., v_params:end] = _pack(v, "v")
    return data


def _ints(values, dev, dtype=torch.int32):
    return torch.tensor(values, dtype=dtype, device=dev)


def _up(n):
    return max(BLOCK, (n + BLOCK - 1) // BLOCK * BLOCK)


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    op, b, dh = case["op"], case["b"], case["dh"]
    state = {"case": case}
    if op == "rotary":
        dtype = torch.float32 if case["dtype"] == "fp32" else torch.bfloat16
        s, wq, wk = case["s"], case["heads"] * dh, case["kv_heads"] * dh
        rows = torch.randn((b, s, wq + 2 * wk), device=dev, generator=gen).to(dtype)
        q, k = rows[..., :wq], rows[..., wq:wq + wk]
        state |= {"q": q, "k": k} if case["fused"] else {"q": q.contiguous(), "k": k.contiguous()}
        state["freq"], state["magnitude"] = _frequencies(case["rot"], case["factor"])
        state["freq_there"] = state["freq"].to(dev)
        state["positions"] = None
        if case["own_positions"]:
            first = [case["far"] + 7919 * i for i in range(b)]
            state["positions"] = _ints(first, dev, torch.int64)[:, None] + torch.arange(s, device=dev)
    elif op == "store":
        n, start = _counts(case)
        state["k"], state["v"] = (torch.randn((b, case["n"], case["heads"] * dh), device=dev, generator=gen).bfloat16()
                                  for _ in range(2))
        shape = (b, case["heads"], case["capacity"] // BLOCK, _sections(dh)[-1])
        state["cache"] = torch.zeros(shape, dtype=torch.uint8, device=dev)
        state["start"], state["counts"] = _ints(start, dev), _ints(n, dev)
        state["ends"] = _ints([x + y for x, y in zip(start, n)], dev)
    else:
        lengths = _lengths(case)
        capacity = _up(case["longest"])
        state["cache"] = _cache(case, capacity, gen, dev)
        state["lens"] = _ints(lengths, dev)
        live = torch.arange(capacity, device=dev) < state["lens"][:, None, None]
        if op == "attend":
            state["q"] = torch.randn((b, case["n"], case["heads"] * dh), device=dev, generator=gen).bfloat16()
            if case["weights"]:
                state["weights"] = torch.rand((b, case["kv_heads"], capacity), device=dev, generator=gen) * live
        else:
            heavy = torch.randn((b, case["kv_heads"], capacity), device=dev, generator=gen).mul(2).exp()
            state["weights"] = heavy * live
            out = (b, case["kv_heads"], _up(case["keep"]) // BLOCK, _sections(dh)[-1])
            state["out"] = torch.zeros(out, dtype=torch.uint8, device=dev)
    return state


# ------------------------------------------------------------------ one pass

def run(state):
    if own:
        return _run_own(state)
    return {"rotary": _rotary, "store": _store, "attend": _attend, "evict": _evict}[state["case"]["op"]](state)


def _run_own(state):
    import blockwise_attn_ffn_bpt_b200 as bpt
    case = state["case"]
    op = case["op"]
    if op == "rotary":
        q, k = bpt.rotary(state["q"], state["k"], case["heads"], case["kv_heads"], state["freq"],
                          positions=state["positions"], offset=case["far"], interleaved=case["interleaved"],
                          magnitude=state["magnitude"], inverse=case["inverse"])
        return {"q": q, "k": k}
    cache = bpt.KV4Cache(state["cache"], case["dh"])
    if op == "store":
        bpt.kv4_store(cache, state["k"], state["v"], state["start"], counts=state["counts"])
        k, v = bpt.kv4_load(cache, state["ends"], case["n"], start=state["start"])
        return {"k": k, "v": v}
    if op == "attend":
        o, lse2 = bpt.kv4_attention(state["q"], cache, state["lens"], case["heads"], causal=True,
                                    weights=state.get("weights"), return_lse=True)
        return {"o": o, "lse2": lse2} | ({"weights": state["weights"]} if case["weights"] else {})
    out = bpt.KV4Cache(state["out"], case["dh"])
    kept, lens, weights = bpt.kv4_evict(cache, state["weights"], state["lens"], case["keep"], case["recent"], out)
    k, v = bpt.kv4_load(out, lens, case["keep"])
    return {"kept": kept, "lens": lens, "weights": weights, "k": k, "v": v}


def _rotary(state):
    case = state["case"]
    q, rot, s = state["q"], case["rot"], case["s"]
    at = state["positions"]
    if at is None:
        at = (case["far"] + torch.arange(s, device=q.device)).expand(case["b"], s)
    angle = at.double()[..., None] * state["freq_there"]
    cos = (angle.cos() * state["magnitude"]).float()[:, :, None]
    sin = (angle.sin() * state["magnitude"]).float()[:, :, None]
    sin = -sin if case["inverse"] else sin

    def turn(x, heads):
        y = x.float().unflatten(-1, (heads, case["dh"]))
        head, rest = y[..., :rot], y[..., rot:]
        a, c = (head[..., 0::2], head[..., 1::2]) if case["interleaved"] else head.chunk(2, -1)
        a, c = a * cos - c * sin, c * cos + a * sin
        head = torch.stack((a, c), -1).flatten(-2) if case["interleaved"] else torch.cat((a, c), -1)
        return torch.cat((head, rest), -1).flatten(-2).to(x.dtype)

    return {"q": turn(q, case["heads"]), "k": turn(state["k"], case["kv_heads"])}


def _store(state):
    case = state["case"]
    live = (torch.arange(case["n"], device=state["k"].device) < state["counts"][:, None])[..., None]

    def keep(x):
        codes, scale, low = _quantise(x)
        return ((low + scale * codes.float()).flatten(-2) * live).bfloat16()

    return {"k": keep(state["k"]), "v": keep(state["v"])}


def _attend(state):
    case = state["case"]
    dh, h, n = case["dh"], case["kv_heads"], case["n"]
    b, group = case["b"], case["heads"] // h
    q = state["q"].float().view(b, n, h, group, dh).permute(0, 2, 3, 1, 4).reshape(b, h, group * n, dh)
    k = _unpack(state["cache"], dh, "k")
    score = (q @ k.transpose(-1, -2)) * dh ** -0.5
    del k
    capacity = score.shape[-1]
    last = state["lens"][:, None] - n + torch.arange(n, device=q.device)  # the last key that each token sees
    seen = torch.arange(capacity, device=q.device) <= last[..., None]
    seen = seen[:, None, None].expand(b, h, group, n, capacity).reshape(b, h, group * n, capacity)
    score = torch.where(seen, score, torch.full_like(score, -math.inf))
    top = score.amax(-1, keepdim=True)
    p = torch.where(seen, torch.exp(score - top), torch.zeros_like(score))
    total = p.sum(-1, keepdim=True)
    some = total > 0
    p = torch.where(some, p / total, torch.zeros_like(p))
    o = p @ _unpack(state["cache"], dh, "v")
    lse2 = torch.where(some, (top + total.log()) / math.log(2), torch.full_like(top, -math.inf))
    out = {"o": o.view(b, h, group, n, dh).permute(0, 3, 1, 2, 4).reshape(b, n, -1).bfloat16(),
           "lse2": lse2.view(b, h * group, n)}
    if case["weights"]:
        out["weights"] = state["weights"].add_(p.sum(2))
    return out


def _evict(state):
    case = state["case"]
    weights, lens, keep = state["weights"], state["lens"][:, None, None], case["keep"]
    at = torch.arange(weights.shape[-1], device=weights.device)
    newest = (at >= lens - min(case["recent"], keep)) & (at < lens)
    order = torch.where(newest, torch.full_like(weights, math.inf), weights)
    order = torch.where(at < lens, order, torch.full_like(weights, -math.inf))
    kept = torch.sort(order, dim=-1, descending=True, stable=True)[1][..., :keep]
    kept = torch.where(kept < lens, kept, torch.full_like(kept, weights.shape[-1])).sort(-1)[0]
    left = torch.minimum(state["lens"], torch.full_like(state["lens"], keep))
    live = torch.arange(kept.shape[-1], device=kept.device) < left[:, None, None]
    at = torch.where(live, kept, torch.zeros_like(kept))
    pad = (0, state["out"].shape[2] * BLOCK - kept.shape[-1])
    moved = torch.nn.functional.pad(weights.gather(-1, at) * live, pad)

    def values(which):
        x = _unpack(state["cache"], case["dh"], which)
        x = x.gather(2, at[..., None].expand(-1, -1, -1, case["dh"])) * live[..., None]
        x = torch.nn.functional.pad(x, (0, 0, 0, keep - x.shape[2]))
        return x.transpose(1, 2).flatten(-2).bfloat16()

    kept = torch.nn.functional.pad(torch.where(live, kept, torch.full_like(kept, -1)), (0, keep - kept.shape[-1]), value=-1)
    return {"kept": kept.int(), "lens": left, "weights": moved, "k": values("k"), "v": values("v")}


# ------------------------------------------------------------------ the same in 64 bits

def _exact_rows(data, dh, which):
    """The values [heads, capacity, dh] of one sequence's blocks in 64 bits, each dimension looked up in its byte."""
    h, blocks, _ = data.shape
    dim, row = torch.meshgrid(torch.arange(dh), torch.arange(BLOCK), indexing="xy")  # [64, dh]
    u = dim // 8
    if which == "k":
        place, first = (u % 4) * (dh // 32) + u // 4, 0
    elif dh == 64:
        place, first = u, _sections(dh)[2]
    else:
        place, first = ((u % 8) ^ (4 * ((row // 2) % 2))) * 2 + u // 8, _sections(dh)[2]
    byte = (first + row * (dh // 2) + place * 4).to(data.device)  # of the dimension's word
    word = sum(data[..., (byte + i).flatten()].long() << (8 * i) for i in range(4))
    shift = (4 * (dim % 8) + (3 if which == "k" else 0)).to(data.device).flatten()
    code = (((word | (word << 32)) >> shift) & 15).view(h, blocks, BLOCK, dh)
    at = first + BLOCK * dh // 2
    par = (at + (row * (dh // GROUP) + dim // GROUP) * 4).to(data.device)

    def number(place):  # two bytes as a bf16, whose bits are a float's upper half
        low, high = data[..., place.flatten()].int(), data[..., (place + 1).flatten()].int()
        return ((low << 16) | (high << 24)).view(torch.float32).double().view(h, blocks, BLOCK, dh)

    return (number(par + 2) + number(par) * code.double()).flatten(1, 2)


def exact(case, seed):
    state = prepare(case, seed)
    return {"rotary": _exact_rotary, "store": _exact_store, "attend": _exact_attend,
            "evict": _exact_evict}[case["op"]](case, state)


def _exact_rotary(case, state):
    dh, rot, out = case["dh"], case["rot"], {}
    dim = torch.arange(rot, device=state["q"].device)
    if case["interleaved"]:
        pair, other, sign = dim // 2, dim ^ 1, (dim % 2) * 2 - 1
    else:
        pair, other, sign = dim % (rot // 2), (dim + rot // 2) % rot, torch.where(dim < rot // 2, -1, 1)
    freq = state["freq_there"][pair]
    for name, heads in (("q", case["heads"]), ("k", case["kv_heads"])):
        rows = []
        for i in range(case["b"]):
            first = 7919 * i if case["own_positions"] else 0
            angle = (case["far"] + first + torch.arange(case["s"], device=dim.device)).double()[:, None, None] * freq
            x = state[name][i].double().view(case["s"], heads, dh)
            y = x.clone()
            turned = x[..., other] * sign * torch.sin(angle) * (-1 if case["inverse"] else 1)
            y[..., :rot] = (x[..., :rot] * torch.cos(angle) + turned) * state["magnitude"]
            rows.append(y.flatten(1))
        out[name] = torch.stack(rows)
    return out


def _exact_store(case, state):
    out, n = {}, state["counts"].tolist()
    for name in ("k", "v"):
        y = torch.zeros(state[name].shape, dtype=torch.float64, device=state[name].device)
        for i in range(case["b"]):
            x = state[name][i, :n[i]].double().view(n[i], -1, GROUP)
            low = x.min(-1, keepdim=True).values
            scale = ((x.max(-1, keepdim=True).values - low) / 15).to(torch.bfloat16)
            inverse = (1 / scale.double()).float().double()  # the stored format's inverse has 24 bits
            code = torch.round((x - low) * inverse).clamp(0, 15)
            y[i, :n[i]] = torch.where(scale > 0, low + scale.double() * code, low).view(n[i], -1)
        out[name] = y
    return out


def _exact_attend(case, state):
    dh, h, n, b = case["dh"], case["kv_heads"], case["n"], case["b"]
    group = case["heads"] // h
    dev = state["q"].device
    o = torch.zeros((b, n, h, group, dh), dtype=torch.float64, device=dev)
    lse2 = torch.full((b, h, group, n), -math.inf, dtype=torch.float64, device=dev)
    weights = state["weights"].double() if case["weights"] else None
    for i, length in enumerate(_lengths(case)):
        if not length:
            continue
        blocks = (length + BLOCK - 1) // BLOCK
        k = _exact_rows(state["cache"][i, :, :blocks], dh, "k")[:, :length]
        v = _exact_rows(state["cache"][i, :, :blocks], dh, "v")[:, :length]
        q = state["q"][i].double().view(n, h, group, dh)
        for t in range(n):
            seen = length - n + 1 + t
            if seen <= 0:
                continue
            s = torch.einsum("hgd,hud->hgu", q[t], k[:, :seen]) / math.sqrt(dh)
            lse = torch.logsumexp(s, -1)
            p = torch.exp(s - lse[..., None])
            o[i, t] = torch.einsum("hgu,hud->hgd", p, v[:, :seen])
            lse2[i, :, :, t] = lse / math.log(2)
            if weights is not None:
                weights[i, :, :seen] += p.sum(1)
    out = {"o": o.flatten(2), "lse2": lse2.flatten(1, 2)}
    return out | ({"weights": weights} if case["weights"] else {})


def _exact_evict(case, state):
    b, h, dh, keep = case["b"], case["kv_heads"], case["dh"], case["keep"]
    dev = state["weights"].device
    values = {x: torch.zeros((b, keep, h * dh), dtype=torch.float64, device=dev) for x in ("k", "v")}
    moved = torch.zeros((b, h, state["out"].shape[2] * BLOCK), dtype=torch.float64, device=dev)
    kept_all = torch.full((b, h, keep), -1, dtype=torch.int32, device=dev)
    for i, length in enumerate(_lengths(case)):
        left = min(length, keep)
        recent = min(case["recent"], left)
        old = state["weights"][i, :, :length - recent].double()
        heavy = torch.argsort(-old, dim=-1, stable=True)[:, :left - recent]
        late = torch.arange(length - recent, length, device=dev).expand(h, recent)
        kept = torch.cat((heavy, late), -1).sort(-1).values
        kept_all[i, :, :left] = kept.int()
        moved[i, :, :left] = state["weights"][i].double().gather(-1, kept)
        for x in ("k", "v"):
            rows = _exact_rows(state["cache"][i], dh, x)
            rows = rows.gather(1, kept[..., None].expand(h, left, dh))
            values[x][i, :left] = rows.transpose(0, 1).reshape(left, h * dh)
    return {"kept": kept_all, "lens": torch.tensor([min(n, keep) for n in _lengths(case)], dtype=torch.int32, device=dev),
            "weights": moved, **values}
