"""Refusals of the step's calls (fa_plan_step, fa_norm_rope_store), without a GPU:
host tensors stand for device ones, and what passes the checks meets the library's
own refusal of a call that has no device or no slab."""
import ctypes
from types import SimpleNamespace

import pytest
import torch

STREAM = SimpleNamespace(cuda_stream=0)
T, D, HQ, HKV, B = 5, 256, 4, 2, 3


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


def layer(fa, kind=0, src=-1):
    return dict(kind=kind, head_dim=D, num_q_heads=HQ, num_kv_heads=HKV, window=20, kv_source=src, sm_scale=0.0625)


@pytest.fixture
def cache(fa):
    return fa.Cache([layer(fa), layer(fa, 0, fa.KV_AUTO)], 8, 16)


def status(fa, call, *args, **kw):
    with pytest.raises(fa.FAError) as e:
        call(*args, stream=STREAM, **kw)
    return e.value.status


def rows(fa, **m):
    return {**dict(layer=0, how=fa.NormRope(D, [0.5] * (D // 2), device="cpu"), q=bf16(T, HQ, D), k=bf16(T, HKV, D), v=bf16(T, HKV, D),
                   positions=i32(T), slot_mapping=i32(T), q_out=bf16(T, HQ, D)), **m}


def test_rows_that_fit_are_taken(fa, cache):
    x = bf16(T, (HQ + 2 * HKV) * D)
    ok = [rows(fa), rows(fa, k_out=bf16(T, HKV, D)), rows(fa, q=x[:, : HQ * D], k=x[:, HQ * D: (HQ + HKV) * D], v=x[:, (HQ + HKV) * D:]),
          rows(fa, q=None, q_out=None), rows(fa, positions=i32(T + 3), slot_mapping=i32(T + 1), q_out=bf16(T + 2, HQ, D))]
    for a in ok:
        assert status(fa, cache.norm_rope_store, **a) == fa.ERR_NOT_BOUND
    cache.norm_rope_store(**rows(fa, q=bf16(0, HQ, D), k=bf16(0, HKV, D), v=bf16(0, HKV, D)), stream=STREAM)   # no rows: nothing to do


BAD_ROWS = {
    "q type": lambda fa: dict(q=torch.zeros(T, HQ, D)),
    "q shape": lambda fa: dict(q=bf16(T, HQ + 1, D)),
    "k rows": lambda fa: dict(k=bf16(T - 1, HKV, D)),
    "v missing": lambda fa: dict(v=None),
    "q not dense in a token": lambda fa: dict(q=bf16(T, HQ, 2 * D)[..., ::2]),
    "heads apart": lambda fa: dict(q=bf16(T, HQ, 2 * D)[..., :D]),
    "stride 4": lambda fa: dict(q=bf16(T * (HQ * D + 4)).as_strided((T, HQ, D), (HQ * D + 4, D, 1))),
    "overlapping tokens": lambda fa: dict(q=bf16(T * HQ * D).as_strided((T, HQ, D), (8, D, 1))),
    "q misaligned": lambda fa: dict(q=bf16(T * HQ * D + 4)[4:].view(T, HQ, D)),
    "no q_out": lambda fa: dict(q_out=None),
    "q_out short": lambda fa: dict(q_out=bf16(T - 1, HQ, D)),
    "k_out type": lambda fa: dict(k_out=torch.zeros(T, HKV, D)),
    "positions missing": lambda fa: dict(positions=None),
    "positions short": lambda fa: dict(positions=i32(T - 1)),
    "positions 64-bit": lambda fa: dict(positions=torch.zeros(T, dtype=torch.int64)),
    "slots short": lambda fa: dict(slot_mapping=i32(T - 1)),
    "keys nowhere": lambda fa: dict(slot_mapping=None),
    "nothing": lambda fa: dict(q=None, k=None, v=None),
    "another head_dim": lambda fa: dict(how=fa.NormRope(512, device="cpu")),
    "eps 0": lambda fa: dict(how=fa.NormRope(D, eps=0.0, device="cpu")),
    "eps NaN": lambda fa: dict(how=fa.NormRope(D, eps=float("nan"), device="cpu")),
    "offset infinite": lambda fa: dict(how=fa.NormRope(D, weight_offset=float("inf"), device="cpu")),
    "layer": lambda fa: dict(layer=2),
}


@pytest.mark.parametrize("what", BAD_ROWS)
def test_rows_the_kernel_would_misread(fa, cache, what):
    want = fa.OK if what == "nothing" else fa.ERR_INVALID_ARG
    if what == "nothing":
        cache.norm_rope_store(**rows(fa, **BAD_ROWS[what](fa)), stream=STREAM)   # T = 0
        return
    assert status(fa, cache.norm_rope_store, **rows(fa, **BAD_ROWS[what](fa))) == want


@pytest.mark.parametrize("R", [2, 24, 257 * 2, 512])
def test_rotations_that_are_not_served(fa, cache, R):
    how = fa.NormRope(D, [0.1] * (R // 2), device="cpu")
    assert status(fa, cache.norm_rope_store, **rows(fa, how=how)) == fa.ERR_UNSUPPORTED


def test_a_shared_layer_ignores_keys(fa, cache):
    # past every check: refused only for want of a device
    assert status(fa, cache.norm_rope_store, **rows(fa, layer=1, k="ignored", v=None, slot_mapping="ignored")) == fa.ERR_CUDA


def test_weights_are_checked_where_they_are_given(fa):
    for w in (torch.zeros(D), bf16(D + 1), bf16(2 * D)[::2]):
        with pytest.raises(fa.FAError):
            fa.NormRope(D, q_weight=w, device="cpu")


def test_steps_are_exact(fa):
    """Against the frequency's own fraction of a turn, in integers."""
    from decimal import Decimal, getcontext
    getcontext().prec = 60
    two_pi = Decimal("6.28318530717958647692528676655900576839433879875021164194988918461563281257")
    f = [1.0, 0.1, 1e-4, 3.0, 7.123456789, 0.0, -0.5, 1e6]
    for got, x in zip(fa.rope_steps(f), f):
        want = (Decimal(x) / two_pi * 2 ** 64).to_integral_value() % 2 ** 64
        assert got == int(want) % 2 ** 64


def plan(fa, cache, **m):
    t = fa.PageTable(cache, m.pop("kind", fa.FULL), m.pop("block_table", i32(B, 4)), m.pop("free_pages", i32(8)), m.pop("state", i32(4 + 2 * B)))
    a = {**dict(new_lens=i32(B), qo_indptr=i32(B + 1), prefix_lens=i32(B), positions=i32(T), slot_mapping=i32(T)), **m}
    return status(fa, t.step, **a)


def test_a_plan_that_fits_is_taken(fa, cache):
    assert plan(fa, cache) == fa.ERR_CUDA   # past every check: refused only for want of a device
    assert plan(fa, cache, positions=i32(0), slot_mapping=i32(0)) == fa.ERR_CUDA
    assert plan(fa, cache, state_out=i32(4 + 2 * B)) == fa.ERR_CUDA


@pytest.mark.parametrize("bad", [
    dict(new_lens=i32(B - 1)), dict(new_lens=torch.zeros(B)), dict(qo_indptr=i32(B)), dict(prefix_lens=i32(B - 1)), dict(positions=i32(T - 1)),
    dict(free_pages=i32(7)), dict(state=i32(3 + 2 * B)), dict(state_out=i32(3 + 2 * B)), dict(block_table=i32(B, 8)[:, ::2]), dict(kind=1),
    dict(kind=2), dict(block_table=i32(B, 0)), dict(positions=i32(4 * T)[3: 3 + T], slot_mapping=i32(T)), dict(new_lens=None),
])
def test_plans_the_kernel_would_misread(fa, cache, bad):
    assert plan(fa, cache, **bad) == fa.ERR_INVALID_ARG


def test_batches_past_the_limit(fa, cache):
    n = fa.MAX_STEP_BATCH + 1
    m = dict(block_table=i32(n, 1), state=i32(4 + 2 * n), new_lens=i32(n), qo_indptr=i32(n + 1), prefix_lens=i32(n))
    assert plan(fa, cache, **m) == fa.ERR_INVALID_ARG
    assert fa.lib().fa_plan_step(None, 0, *[None] * 1, 1, *[None] * 4, 1, *[None] * 4, 0, None) == fa.ERR_INVALID_ARG


def test_rows_of_positions_past_32_bits(fa, cache):
    t = i32(1)
    p = t.data_ptr() + (-t.data_ptr()) % 16
    call = fa.lib().fa_plan_step
    for cols, want in ((((1 << 31) - 256) // 16, fa.ERR_INVALID_ARG), (((1 << 31) - 256) // 16 - 1, fa.ERR_CUDA), (0, fa.ERR_INVALID_ARG)):
        assert call(cache._h, 0, p, 1, p, p, p, p, cols, p, p, p, p, 4, None) == want
