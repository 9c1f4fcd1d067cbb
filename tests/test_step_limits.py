"""Limits and missing tensors of the step's and of differential attention's calls, without
a GPU (as in test_step_arguments.py and test_diff_arguments.py: host tensors stand for device ones)."""
import pytest
import torch

from test_step_arguments import cache, fa, i32  # noqa: F401  (fixtures)


def test_tokens_past_32_bits(fa, cache):  # noqa: F811
    """The kernel walks tokens in runs of 128 with 32-bit counters: a run that would end
    past 2^31 - 1 is refused before it is launched."""
    t = i32(1)
    p = t.data_ptr() + (-t.data_ptr()) % 16
    call = fa.lib().fa_plan_step
    for n, want in ((0, fa.ERR_CUDA), (2 ** 31 - 256, fa.ERR_CUDA), (2 ** 31 - 255, fa.ERR_INVALID_ARG), (2 ** 31 - 128, fa.ERR_INVALID_ARG),
                    (2 ** 31 - 2, fa.ERR_INVALID_ARG), (2 ** 31 - 1, fa.ERR_INVALID_ARG), (-1, fa.ERR_INVALID_ARG)):
        assert call(cache._h, 0, p, 1, p, p, p, p, 4, p, p, p, p, n, None) == want
