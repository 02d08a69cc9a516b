"""README's example of decoding over the 4-bit cache runs, and gives every new token the position after the last one's,
behind an eviction too (where the cache's length has fallen)."""

import os

import pytest
import torch

import blockwise_attn_ffn_bpt_b200 as bpt

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_the_decoding_example(monkeypatch):
    with open(os.path.join(ROOT, "README.md")) as f:
        blocks = [x.split("```")[0] for x in f.read().split("```python\n")[1:]]
    (code,) = [x for x in blocks if "kv4_evict" in x]
    evicted, positions, evict, rotary = [], [], bpt.kv4_evict, bpt.rotary

    def watched_evict(*args, **kw):
        evicted.append(len(positions))
        return evict(*args, **kw)

    def watched_rotary(*args, **kw):
        if kw.get("positions") is not None:
            positions.append(kw["positions"].flatten().tolist())
        return rotary(*args, **kw)

    monkeypatch.setattr(bpt, "kv4_evict", watched_evict)
    monkeypatch.setattr(bpt, "rotary", watched_rotary)
    h, heads = 512, 8
    bf = dict(device="cuda", dtype=torch.bfloat16)
    space = {"torch": torch, "bpt": bpt, "bf": bf, "h": h, "heads": heads,
             "params": {"Wqkv": torch.randn(h, 3 * h, **bf) / h ** 0.5, "bqkv": torch.zeros(3 * h, **bf)}}
    exec(code, space)
    assert bpt.stream_status() == 0
    assert torch.isfinite(space["o"]).all()
    assert evicted and 0 < evicted[0] < len(positions), "a step before the eviction and one after it"
    for i, p in enumerate(positions):
        assert p == [1000 + i] * space["b"]
    assert space["lens"].tolist() == [513] * space["b"]
