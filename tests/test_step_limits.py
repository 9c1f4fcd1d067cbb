"""Limits and missing tensors of the step's and of differential attention's calls, without
a GPU (as in test_step_arguments.py and test_diff_arguments.py: host tensors stand for device ones)."""
import pytest

import test_diff_arguments as diff
from test_step_arguments import STREAM, cache, fa, i32, rows  # noqa: F401  (fixtures among them)


def test_tokens_past_32_bits(fa, cache):  # noqa: F811
    """The kernel walks tokens in runs of 128 with 32-bit counters: a run that would end
    past 2^31 - 1 is refused before it is launched."""
    t = i32(1)
    p = t.data_ptr() + (-t.data_ptr()) % 16
    call = fa.lib().fa_plan_step
    for n, want in ((0, fa.ERR_CUDA), (2 ** 31 - 256, fa.ERR_CUDA), (2 ** 31 - 255, fa.ERR_INVALID_ARG), (2 ** 31 - 128, fa.ERR_INVALID_ARG),
                    (2 ** 31 - 2, fa.ERR_INVALID_ARG), (2 ** 31 - 1, fa.ERR_INVALID_ARG), (-1, fa.ERR_INVALID_ARG)):
        assert call(cache._h, 0, p, 1, p, p, p, p, 4, p, p, p, p, n, None) == want


def refused(fa, call, *args, **kw):  # noqa: F811
    with pytest.raises(fa.FAError) as e:
        call(*args, **kw)
    return e.value.status


@pytest.mark.parametrize("what", ["new_lens", "qo_indptr", "prefix_lens", "positions", "slot_mapping", "free_pages", "state", "block_table"])
def test_a_plan_without_one_of_its_tensors(fa, cache, what):  # noqa: F811
    made = dict(block_table=i32(3, 4), free_pages=i32(8), state=i32(10))
    a = dict(new_lens=i32(3), qo_indptr=i32(4), prefix_lens=i32(3), positions=i32(5), slot_mapping=i32(5))
    (made if what in made else a)[what] = None

    def call():
        fa.PageTable(cache, fa.FULL, **made).step(**a, stream=STREAM)

    assert refused(fa, call) == fa.ERR_INVALID_ARG


@pytest.mark.parametrize("kv", [0, 1])
@pytest.mark.parametrize("what", ["q", "lam", "block_table", "seq_lens", "out"])
def test_a_differential_decode_without_one_of_its_tensors(fa, what, kv):  # noqa: F811
    c = diff.make(fa, kv=kv)
    assert refused(fa, c.decode_diff, **diff.decode(**{what: None}), stream=STREAM) == fa.ERR_INVALID_ARG


@pytest.mark.parametrize("what", ["q", "lam", "k_ext", "v_ext", "qo_indptr", "prefix_lens", "out"])
def test_a_differential_extend_without_one_of_its_tensors(fa, what):  # noqa: F811
    c = diff.make(fa)
    assert refused(fa, c.extend_diff, **diff.extend(**{what: None}), stream=STREAM) == fa.ERR_INVALID_ARG


def test_rows_without_a_norm_and_rotation(fa, cache):  # noqa: F811
    assert refused(fa, cache.norm_rope_store, **rows(fa, how=None), stream=STREAM) == fa.ERR_INVALID_ARG


@pytest.mark.parametrize("what", ["q", "block_table"])
def test_a_4_bit_decode_without_one_of_its_tensors(fa, what):  # noqa: F811
    c = diff.make(fa, kv=fa.KV_FP4)
    a = {k: v for k, v in diff.decode(**{what: None}).items() if k not in ("lam", "lse")}
    assert refused(fa, c.decode, **a, stream=STREAM) == fa.ERR_INVALID_ARG
