"""Which path the 4-bit attention's host side takes, seen (without a GPU) by the workspace that it asks for: none where a
thread block takes a head."""

import pytest

import blockwise_attn_ffn_bpt_b200 as bpt


def workspace(b, heads, kv_heads, capacity, dh, n=1):
    return bpt.lib().bpt_kv4_attention_workspace_bytes(b, n, heads, kv_heads, capacity, dh, 0)


@pytest.mark.parametrize("dh,heads,short,long", [(128, 4, 2944, 3200), (64, 4, 4096, 4160), (128, 40, 2048, 2112),
                                                 (64, 40, 2944, 3200)])
def test_a_thread_block_takes_a_head_of_a_short_cache_only(dh, heads, short, long):
    # 148 heads are as many as the device has SMs: each would have a thread block, but the call would last as long as
    # the longest sequence. A warp is to take 4 blocks of 64 tokens at most.
    assert workspace(37, heads, 4, short, dh) == 0
    assert workspace(37, heads, 4, long, dh) > 0
    assert workspace(36, heads, 4, 45440, dh) > 0 and workspace(37, heads, 4, 1 << 20, dh) > 0
    # fewer heads leave SMs idle
    assert workspace(1, heads, 4, 512, dh) == 0 and workspace(1, heads, 4, 4096, dh) > 0
