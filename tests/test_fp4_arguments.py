"""The binding's checks of a 4-bit cache's tensors, without a GPU: host tensors
stand for device ones, and what passes the checks meets the library's own refusal
of a slab that is not bound."""
from types import SimpleNamespace

import pytest
import torch

STREAM = SimpleNamespace(cuda_stream=0)
B, D, HQ, HKV, LEN = 3, 256, 8, 2, 32


@pytest.fixture
def fa(monkeypatch):
    import __graft_entry__
    __graft_entry__.build()
    import full_attention_gb300 as fa
    monkeypatch.setattr(fa, "_device", lambda: -1)   # where host tensors are
    return fa


def i32(*shape):
    return torch.zeros(shape, dtype=torch.int32)


def bf16(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16)


@pytest.fixture
def cache(fa):
    lay = dict(kind=fa.FULL, head_dim=D, num_q_heads=HQ, num_kv_heads=HKV, window=0, kv_source=fa.KV_OWN, sm_scale=0.0625)
    return fa.Cache([lay, lay], 8, 16, fa.KV_FP4)


def status(fa, call, *args, **kw):
    with pytest.raises(fa.FAError) as e:
        call(*args, stream=STREAM, **kw)
    return e.value.status


def decode_args(**m):
    return {**dict(layer=0, q=bf16(B, HQ, D), block_table=i32(B, LEN // 16), seq_lens=i32(B), max_seq_len=LEN,
                   out=bf16(B, HQ, D), lse=torch.zeros(B, HQ)), **m}


def store_args(**m):
    return decode_args(k_new=bf16(B, HKV, D), v_new=bf16(B, HKV, D), slot_mapping=i32(B), **m)


def test_what_fits_is_taken(fa, cache):
    assert status(fa, cache.decode, **decode_args()) == fa.ERR_NOT_BOUND
    assert status(fa, cache.decode_store, **store_args()) == fa.ERR_NOT_BOUND
    assert status(fa, cache.store, 0, bf16(B, HKV, D), bf16(B, HKV, D), i32(B)) == fa.ERR_NOT_BOUND


@pytest.mark.parametrize("rows", [0, 1, B - 1])
def test_a_fused_store_needs_a_slot_and_rows_for_each_sequence(fa, cache, rows):
    """The kernel reads slot_mapping[b] of every sequence of the batch."""
    bad = dict(slot_mapping=i32(rows), k_new=bf16(rows, HKV, D), v_new=bf16(rows, HKV, D))
    assert status(fa, cache.decode_store, **{**store_args(), **bad}) == fa.ERR_INVALID_ARG
    for name in bad:
        assert status(fa, cache.decode_store, **{**store_args(), name: bad[name]}) == fa.ERR_INVALID_ARG


def layers_args(**m):
    return {**dict(layers=[0, 1], qs=[bf16(B, HQ, D)] * 2, block_tables=[i32(B, LEN // 16)] * 2, seq_lens=i32(B),
                   max_seq_len=LEN, outs=[bf16(B, HQ, D)] * 2, lses=[torch.zeros(B, HQ)] * 2), **m}


TAKEN = ("ERR_NOT_BOUND", "ERR_WORKSPACE")   # the library's, past the binding's checks


def test_block_tables_of_one_launch_are_alike(fa, cache):
    """All layers' tables are read with one row length, the first one's."""
    assert status(fa, cache.decode_layers, **layers_args()) in [getattr(fa, s) for s in TAKEN]
    for narrow in (i32(B, 1), i32(2 * B, 1), i32(B, LEN // 16 + 1)):
        bad = layers_args(block_tables=[i32(B, LEN // 16), narrow])
        assert status(fa, cache.decode_layers, **bad) == fa.ERR_INVALID_ARG


@pytest.mark.parametrize("kv_dtype", ["KV_BF16", "KV_INT8", "KV_FP8", "KV_FP4"])
def test_lists_of_a_launch_have_an_entry_for_each_layer(fa, kv_dtype):
    """The library reads n pointers from each list."""
    lay = dict(kind=fa.FULL, head_dim=D, num_q_heads=HQ, num_kv_heads=HKV, window=0, kv_source=fa.KV_OWN, sm_scale=0.0625)
    cache = fa.Cache([lay, lay], 8, 16, getattr(fa, kv_dtype))
    for name in ("qs", "block_tables", "outs", "lses"):
        for n in (0, 1):
            bad = layers_args(**{name: (layers_args()[name] * 2)[:n]})
            assert status(fa, cache.decode_layers, **bad) == fa.ERR_INVALID_ARG, (name, n)
    rows = lambda n: [bf16(B, HKV, D)] * n
    for k, v, s in ((1, 2, 2), (2, 1, 2), (2, 2, 1), (0, 0, 0)):
        assert status(fa, cache.store_layers, [0, 1], rows(k), rows(v), [i32(B)] * s) == fa.ERR_INVALID_ARG, (k, v, s)
    assert status(fa, cache.store_layers, [0, 1], rows(2), rows(2), [i32(B)] * 2) != fa.ERR_INVALID_ARG


def test_buffers_with_rows_to_spare_are_taken(fa, cache):
    """Tables, lengths and outputs kept for a larger batch, as a captured graph's are."""
    spare = dict(seq_lens=i32(B + 5), block_table=i32(B + 5, LEN // 16), out=bf16(B + 5, HQ, D), lse=torch.zeros(B + 5, HQ))
    slots = dict(slot_mapping=i32(B + 5), k_new=bf16(B + 5, HKV, D), v_new=bf16(B + 5, HKV, D))
    for name in spare:
        assert status(fa, cache.decode, **decode_args(**{name: spare[name]})) == fa.ERR_NOT_BOUND, name
    assert status(fa, cache.decode, **decode_args(**spare)) == fa.ERR_NOT_BOUND
    assert status(fa, cache.decode_noalloc, **decode_args(**spare)) != fa.ERR_INVALID_ARG
    assert status(fa, cache.decode_store, **{**store_args(**spare), **slots}) == fa.ERR_NOT_BOUND
    assert status(fa, cache.store, 0, bf16(B + 5, HKV, D), bf16(B + 5, HKV, D), i32(B)) == fa.ERR_NOT_BOUND
    wide = layers_args(seq_lens=i32(B + 5), block_tables=[i32(B + 1, 2), i32(B + 5, 2)], outs=[bf16(B + 5, HQ, D)] * 2)
    assert status(fa, cache.decode_layers, **wide) in [getattr(fa, s) for s in TAKEN]
    for kv in (fa.KV_BF16, fa.KV_FP4):
        c = fa.Cache(cache.layers, 8, 16, kv)
        assert status(fa, c.load, 0, i32(B), bf16(B + 5, HKV, D), bf16(B + 5, HKV, D)) == fa.ERR_NOT_BOUND
    N = 7
    ext = dict(layer=0, q=bf16(N, HQ, D), qo_indptr=i32(B + 9), block_table=i32(B + 5, 2), max_q_len=4, out=bf16(N + 5, HQ, D),
               lse=torch.zeros(N + 5, HQ))
    assert status(fa, cache.extend, **ext, k_ext=bf16(N + 5, HKV, D), v_ext=bf16(N + 5, HKV, D), prefix_lens=i32(B),
                  max_prefix_len=LEN) == fa.ERR_NOT_BOUND
    assert status(fa, cache.decode_multi, **ext, seq_lens=i32(B), max_seq_len=LEN) == fa.ERR_NOT_BOUND


def test_buffers_too_small_or_not_dense_are_refused(fa, cache):
    for bad in (dict(seq_lens=i32(B - 1)), dict(block_table=i32(B - 1, 2)), dict(out=bf16(B - 1, HQ, D)),
                dict(lse=torch.zeros(B - 1, HQ)), dict(block_table=i32(B, 4)[:, :2]), dict(seq_lens=i32(2 * B)[::2]),
                dict(q=bf16(B, HQ, 2 * D)[..., ::2]), dict(seq_lens=i32(B).long()), dict(q=bf16(B, HQ, D).half()),
                dict(q=bf16(B, HQ, D - 16))):
        assert status(fa, cache.decode, **decode_args(**bad)) == fa.ERR_INVALID_ARG, bad.keys()


@pytest.mark.parametrize("kv_dtype", ["KV_BF16", "KV_FP4"])
def test_a_missing_tensor_is_refused_as_in_the_other_formats(fa, kv_dtype):
    """(Past the layer and the slab, which the library looks at first.)"""
    lay = dict(kind=fa.FULL, head_dim=D, num_q_heads=HQ, num_kv_heads=HKV, window=0, kv_source=fa.KV_OWN, sm_scale=0.0625)
    cache = fa.Cache([lay, lay], 8, 16, getattr(fa, kv_dtype))
    refused = (fa.ERR_INVALID_ARG, fa.ERR_NOT_BOUND)
    assert status(fa, cache.store, 0, None, bf16(B, HKV, D), i32(B)) in refused
    assert status(fa, cache.store, 0, bf16(B, HKV, D), None, i32(B)) in refused
    for name in ("k_new", "v_new", "slot_mapping", "seq_lens", "out"):
        assert status(fa, cache.decode_store, **{**store_args(), name: None}) in refused, name


@pytest.mark.parametrize("kv_dtype", ["KV_BF16", "KV_INT8", "KV_FP8", "KV_FP4"])
def test_a_window_of_any_size_is_planned(fa, kv_dtype):
    """A window past every length plans as a full layer does, up to the largest int."""
    def need(window, n):
        lay = dict(kind=fa.SLIDING if window else fa.FULL, head_dim=D, num_q_heads=HQ, num_kv_heads=HKV, window=window,
                   kv_source=fa.KV_OWN, sm_scale=0.0625)
        c = fa.Cache([lay, lay], 8, 16, getattr(fa, kv_dtype))
        return c.decode_workspace_bytes(0, B, n), c.decode_layers_workspace_bytes([0, 1], B, n)
    for n in (5000, 100_000, 2**31 - 1):
        full = need(0, n)
        assert full[0] > 0
        for window in (2**31 - 17, 2**31 - 16, 2**31 - 15, 2**31 - 1):
            assert need(window, n) == full
