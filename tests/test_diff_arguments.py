"""Refusals of the differential attention calls, without a GPU: host tensors stand
for device ones, and what passes the checks meets the library's refusal of a slab
that is not bound."""
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


def make(fa, hq=HQ, kv=0):
    lay = dict(kind=fa.FULL, head_dim=D, num_q_heads=hq, num_kv_heads=HKV, window=0, kv_source=fa.KV_OWN, sm_scale=0.0625)
    return fa.Cache([lay], 8, 16, kv)


def status(call, *args, **kw):
    import full_attention_gb300 as fa
    with pytest.raises(fa.FAError) as e:
        call(*args, stream=STREAM, **kw)
    return e.value.status


def decode(**m):
    return {**dict(layer=0, q=bf16(B, HQ, D), lam=torch.zeros(HQ), block_table=i32(B, LEN // 16), seq_lens=i32(B), max_seq_len=LEN,
                   out=bf16(B, HQ, D), lse=torch.zeros(B, HQ, 2)), **m}


def extend(**m):
    return {**dict(layer=0, q=bf16(9, HQ, D), lam=torch.zeros(HQ), k_ext=bf16(9, HKV, D), v_ext=bf16(9, HKV, D), qo_indptr=i32(B + 1),
                   prefix_lens=i32(B), block_table=i32(B, 2), max_q_len=4, max_prefix_len=LEN, out=bf16(9, HQ, D),
                   lse=torch.zeros(9, HQ, 2)), **m}


NEW = dict(k_new=bf16(B, HKV, D), v_new=bf16(B, HKV, D), slot_mapping=i32(B))


def test_what_fits_is_taken(fa):
    c = make(fa)
    for a in (decode(), decode(lse=None), decode(**NEW)):
        assert status(c.decode_diff, **a) == fa.ERR_NOT_BOUND
    for a in (extend(), extend(lse=None)):
        assert status(c.extend_diff, **a) == fa.ERR_NOT_BOUND


@pytest.mark.parametrize("bad", [
    dict(lam=None), dict(lam=torch.zeros(HQ - 1)), dict(lam=torch.zeros(HQ, dtype=torch.float64)), dict(lse=torch.zeros(B, HQ)),
    dict(lse=bf16(B, HQ, 2)), dict(q=bf16(B, HQ, D // 2)), dict(out=bf16(B, HQ - 1, D)), dict(seq_lens=i32(B - 1)), dict(block_table=i32(B - 1, 2)),
    dict(k_new=bf16(B, HKV, D)), dict(NEW, slot_mapping=i32(B - 1)), dict(NEW, v_new=None), dict(NEW, k_new=bf16(B, HQ, D)), dict(layer=1),
])
def test_decodes_the_kernel_would_misread(fa, bad):
    assert status(make(fa).decode_diff, **decode(**bad)) == fa.ERR_INVALID_ARG


@pytest.mark.parametrize("bad", [
    dict(lam=None), dict(lam=torch.zeros(2 * HQ)[::2]), dict(lse=torch.zeros(9, HQ)), dict(k_ext=None), dict(v_ext=bf16(8, HKV, D)),
    dict(q=bf16(9, HQ, 2 * D)), dict(qo_indptr=i32(B)), dict(out=bf16(8, HQ, D)), dict(layer=-1),
])
def test_extends_the_kernel_would_misread(fa, bad):
    assert status(make(fa).extend_diff, **extend(**bad)) == fa.ERR_INVALID_ARG


def test_what_is_not_served(fa):
    assert status(make(fa, kv=fa.KV_FP4).decode_diff, **decode()) == fa.ERR_UNSUPPORTED
    assert make(fa, kv=fa.KV_FP4).decode_diff_workspace_bytes(0, B, LEN) == 0
    for hq, want in ((256, fa.ERR_UNSUPPORTED), (128, fa.ERR_NOT_BOUND), (6, fa.ERR_UNSUPPORTED), (2, fa.ERR_NOT_BOUND)):   # 2 hq / 2 halves a tile of 128
        a = extend(q=bf16(9, hq, D), lam=torch.zeros(hq), out=bf16(9, hq, D), lse=None)
        assert status(make(fa, hq).extend_diff, **a) == want


def test_the_workspace_holds_both_maps(fa):
    c = make(fa)
    for b, n in ((1, 5000), (64, 4096), (3, 100000)):
        plain, both = c.decode_workspace_bytes(0, b, n), c.decode_diff_workspace_bytes(0, b, n)
        assert plain > 0 and both - fa.DECODE_COUNTER_BYTES >= 2 * (plain - fa.DECODE_COUNTER_BYTES) - 4096
    assert c.decode_diff_workspace_bytes(0, 0, 10) == c.decode_diff_workspace_bytes(3, 1, 10) == 0


@pytest.mark.parametrize("kv,each", [(0, None), (1, 4), (2, 4)])
def test_room_for_f16_rows(fa, kv, each):
    """8-bit: K and V rows of what the queries see and of the chunk, a scale a row, a table."""
    lays = [dict(kind=fa.FULL, head_dim=512, num_q_heads=8, num_kv_heads=2, window=0, kv_source=fa.KV_OWN, sm_scale=0.1),
            dict(kind=fa.SLIDING, head_dim=256, num_q_heads=8, num_kv_heads=1, window=100, kv_source=fa.KV_OWN, sm_scale=0.1)]
    c = fa.Cache(lays, 8, 16, kv)
    room = lambda *a: int(fa._lib.fa_extend_unpack_bytes(c._h, *a))
    up = lambda n: (n + 255) // 256 * 256
    if each is None:
        assert room(0, 2, 150, 300) == room(1, 2, 150, 300) == 0
        return
    full = 2 * (2 * 2 * 304 * 512 * 2) + 256 + 2 * (2 * 150 * 2 * 512 * 2) + 2 * up(2 * 2 * 304 * each)
    assert room(0, 2, 150, 300) == full
    slid = 2 * (2 * 272 * 256 * 2) + 256 + 2 * (2 * 150 * 256 * 2) + 2 * up(2 * 272 * each)   # 100 + 150 + 15 rows at most
    assert room(1, 2, 150, 300) == slid
    assert room(0, 2, 150, 0) == 2 * (2 * 2 * 16 * 512 * 2) + 256 + 2 * (2 * 150 * 2 * 512 * 2) + 2 * up(2 * 2 * 16 * each)
    assert room(0, 2, 0, 300) == room(0, 0, 150, 300) == room(0, 1, -1, 300) == room(0, 70000, 1, 1) == 0
