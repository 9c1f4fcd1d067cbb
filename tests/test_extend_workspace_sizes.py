"""What an extend workspace is asked to hold, per slab format and kind of call (host only)."""
import pytest

FORMATS = {"bf16": 0, "int8": 1, "fp8": 2, "fp4": 3}


@pytest.fixture
def fa():
    import __graft_entry__
    __graft_entry__.build()
    import full_attention_gb300 as fa
    return fa


def make(fa, kv, D, hq, hkv, window=0):
    lay = dict(kind=fa.SLIDING if window else fa.FULL, head_dim=D, num_q_heads=hq, num_kv_heads=hkv, window=window,
               kv_source=fa.KV_OWN, sm_scale=0.0625)
    return fa.Cache([lay], 64, 16, FORMATS[kv])


# sequences, new tokens, prefix, head_dim, query and KV heads, window
SIZES = [(8, 512, 32768, 512, 16, 2, 0), (8, 512, 32768, 256, 16, 8, 0), (64, 512, 8192, 512, 16, 2, 0), (8, 1, 131072, 256, 8, 8, 0),
         (64, 4, 131072, 512, 8, 1, 0), (16, 2048, 65536, 256, 16, 8, 4096)]


@pytest.mark.parametrize("kv", ["int8", "fp8"])
@pytest.mark.parametrize("size", SIZES)
def test_plain_calls_over_8_bit_caches_ask_for_the_split_alone(fa, kv, size):
    """Plain extend and multi-token decode over 8-bit slabs read nothing but the split
    workspace: a program that sizes its buffer for them is not asked for gigabytes of rows
    that only differential extend writes."""
    B, new, prefix, D, hq, hkv, window = size
    c = make(fa, kv, D, hq, hkv, window)
    split = fa.extend_workspace_bytes()
    assert c.extend_workspace_bytes(0, B, new, prefix) == split
    seen = min(prefix, window + new + 15) // 16 * 16 if window else prefix
    rows = 4 * D * hkv * B * (seen + new)   # K and V in f16
    assert c.extend_diff_workspace_bytes(0, B, new, prefix) >= split + rows >= split + (128 << 20)


@pytest.mark.parametrize("kv", list(FORMATS))
def test_sizes_of_the_two_kinds_of_call(fa, kv):
    split = fa.extend_workspace_bytes()
    for B, new, prefix, D, hq, hkv, window in SIZES + [(1, 1, 0, 256, 1, 1, 0), (2, 150, 300, 512, 8, 2, 0), (5, 1500, 4096, 512, 16, 2, 0)]:
        c = make(fa, kv, D, hq, hkv, window)
        plain, diff = c.extend_workspace_bytes(0, B, new, prefix), c.extend_diff_workspace_bytes(0, B, new, prefix)
        if kv == "bf16":
            assert plain == diff == split
        elif kv == "fp4":
            assert plain == diff and (diff > split) == (prefix > 0)
        else:
            assert diff > split and plain == (diff if diff - split <= 128 << 20 else split)
    with pytest.raises(fa.FAError):
        c.extend_diff_workspace_bytes(1, 1, 1, 1)
    assert int(fa.lib().fa_extend_diff_unpack_bytes(c._h, 1, 1, 1, 1)) == int(fa.lib().fa_extend_diff_unpack_bytes(None, 0, 1, 1, 1)) == 0
    assert c.extend_diff_workspace_bytes(0, 0, 5, 5) == c.extend_diff_workspace_bytes(0, 1, -1, 5) == split
