"""Batches padded with sequences that have nothing to do, and buffers with rows
to spare, over fp4 slabs."""
import pytest
import torch

import workloads as W
from fp4_case import DecodeCase4, ExtendCase4

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("stored", [False, True], ids=["extend", "multi-token decode"])
@pytest.mark.parametrize("layer", [W.layer(W.FULL, 512, 8, 1), W.layer(W.SLIDING, 256, 8, 2, 300)], ids=["full", "sliding"])
def test_a_sequence_without_new_tokens_reads_no_pages(layer, stored):
    """No query sees its rows, so its block table may hold anything, with a
    workspace for unpacked rows as without."""
    res = []
    for split in (None, "unpack"):
        c = ExtendCase4([layer], [700, 900, 640], [40, 0, 25], 16, seed=61, stored=stored, split=split)
        c.bt[1] = -1
        out, lse = c.run(0)
        assert c.cache.device_error() == 0, split
        c.check(0, out, lse)
        res.append(out)
