"""Extend and multi-token decode over fp4 slabs read only pages that some query sees."""
import pytest
import torch

import workloads as W
from fp4_case import ExtendCase4

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("stored", [False, True], ids=["extend", "multi-token decode"])
@pytest.mark.parametrize("layer", [W.layer(W.FULL, 512, 8, 1), W.layer(W.SLIDING, 256, 8, 2, 300)], ids=["full", "sliding"])
def test_a_sequence_without_new_tokens_reads_no_pages(layer, stored):
    """No query sees its rows, so its block table may hold anything, with a
    workspace for unpacked rows as without."""
    for split in (None, "unpack"):
        c = ExtendCase4([layer], [700, 900, 640], [40, 0, 25], 16, seed=61, stored=stored, split=split)
        c.bt[1] = -1
        out, lse = c.run(0)
        assert c.cache.device_error() == 0, split
        c.check(0, out, lse)


def test_a_window_of_one_reads_no_prefix_pages():
    layer = W.layer(W.SLIDING, 512, 8, 2, 1)
    for split in (None, "unpack"):
        c = ExtendCase4([layer], [700, 37, 640], [40, 3, 25], 16, seed=62, split=split)
        c.bt.fill_(-1)
        out, lse = c.run(0)
        assert c.cache.device_error() == 0, split
        c.check(0, out, lse)
