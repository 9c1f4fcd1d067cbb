"""Differential extend over 8-bit slabs through f16 rows, with proof that the rows were made:
the smallest and oddest calls, which by their own bounds would convert in the kernel."""
import pytest
import torch

import workloads as W
from diff_case import DiffCase
from test_gpu_diff import EXTEND

pytestmark = pytest.mark.gpu

MORE = [(256, 16, 8, 16, 100, [0, 0, 0], [0, 1, 0]), (512, 8, 1, 16, 1, [64, 1], [64, 1]), (256, 64, 1, 16, 17, [333], [129])]


@pytest.mark.parametrize("kv", [W.KV_INT8, W.KV_FP8])
@pytest.mark.parametrize("D,hq,hkv,ps,window,prefix,new", EXTEND + MORE)
@pytest.mark.parametrize("split", [False, True])
def test_f16_rows_of_every_shape(D, hq, hkv, ps, window, prefix, new, split, kv):
    """A bound on the new tokens far above them lets any call take the rows: bit for bit the
    converting call of the same bound, and the room of the rows was written."""
    c = DiffCase(D, hq, hkv, ps, prefix, kv, window, new, seed=D + hq + len(new))
    fa, most = c.fa, max(new) + 4096
    base = fa.extend_workspace_bytes()
    room = c.cache.extend_diff_workspace_bytes(0, c.B, most, max(prefix))
    ws = fa.workspace(room)
    if split:
        c.cache.set_flags(fa.FLAG_EXTEND_SPLIT_ALL)
    res = []
    for n in (base, room):
        c.cache.bind_extend_workspace(ws[:n])
        ws[base:] = 0xFF
        c.out.fill_(float("nan")), c.lse.fill_(float("nan"))
        c.cache.extend_diff(0, c.q, c.lam, c.k_ext, c.v_ext, c.indptr, c.lens_dev, c.bt, most, max(prefix), c.out, c.lse)
        assert bool((ws[base:] != 0xFF).any()) == (n == room)
        res.append((c.out.clone(), c.lse.clone()))
    c.check(*res[0])
    for a, b in zip(*res):
        assert torch.equal(a, b)
