"""Decode over fp4 slabs where every 16-key tile shows in the result, so that one
left out or counted twice where shares meet cannot pass.

Zero queries give all keys the same weight: lse = log n, and the output is the
mean of the values.  The rows of tile t hold 1.3125 = 6 * 448 / 2^11 (exact in the
format) in column (t + an offset) mod D alone.  Weights, products and sums are
powers of two, multiples of 1.3125 and whole numbers: exact.  What is left:
  out: one quotient, two products (2^-24 each) and the rounding to bf16 (2^-8 at
  most in all);
  lse: __log2f (2 units in the last place of its result), the constant ln 2 and a
  product (2^-24 each): 3 * 2^-23 of its value, and 2^-22 near 0.
A tile left out moves lse by 16 / n and its column by D / (n / 16)."""
import numpy as np
import pytest
import torch

import workloads as W
from fp4_case import DecodeCase4

pytestmark = pytest.mark.gpu

ONE = 1.3125


def tile_case(kind, D, hq, hkv, Wn, lens, ps):
    layer = W.layer(kind, D, hq, hkv, Wn)
    cols = []
    for b, L in enumerate(lens):
        pos = np.arange(max(0, L - Wn) if kind == W.SLIDING else 0, L)
        cols.append((pos // 16 + 37 * b) % D)
    at = np.concatenate(cols)

    def edit(i, k, v):
        v.zero_()
        for h in range(hkv):
            v[torch.arange(len(at)), h, torch.from_numpy((at + 11 * h) % D)] = ONE

    case = DecodeCase4([layer], lens, ps, seed=1, edit=edit)
    case.q[0].zero_()
    want = np.zeros((len(lens), hkv, D))
    for b, c in enumerate(cols):
        for h in range(hkv):
            want[b, h] = ONE * np.bincount((c + 11 * h) % D, minlength=D) / max(1, len(c))
    return case, want, np.array([len(c) for c in cols])


def check(case, want, n, out, lse):
    out, lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
    g = out.shape[1] // want.shape[1]
    for b in range(len(n)):
        if n[b] == 0:
            assert (out[b] == 0).all() and (lse[b] == -np.inf).all()
            continue
        assert np.all(np.abs(lse[b] - np.log(n[b])) <= 3 * 2.0 ** -23 * np.log(n[b]) + 2.0 ** -22), (b, n[b], lse[b])
        w = np.repeat(want[b], g, axis=0)
        assert np.all(np.abs(out[b] - w) <= 2.0 ** -8 * w), (b, n[b])


CASES = [
    *[(W.FULL, D, 8, 1, 0, [n], 16) for D in (256, 512) for n in (512, 1000, 3328, 20_011, 60_001)],
    (W.FULL, 512, 16, 1, 0, [30_000], 16),                                    # two chunks of heads
    (W.FULL, 256, 8, 2, 0, [30_000, 17, 0, 9_000], 64),                       # whole units, several shares each
    (W.FULL, 512, 2, 1, 0, [4000, 900, 5000, 100, 2500, 3000, 1, 700, 6000, 2222], 16),
    (W.SLIDING, 256, 8, 1, 1000, [1024, 5000, 3000, 1023, 2048, 1500, 7], 16),
    (W.FULL, 512, 8, 1, 0, [700 + i for i in range(152)], 16),                # laid end to end, cut evenly
    # laid end to end: the units in the middle take hundreds of shares, whose last goes on to the next unit
    (W.FULL, 512, 8, 1, 0, [20] * 300 + [30_003] + [20] * 300, 16),
    (W.FULL, 256, 8, 2, 0, [33] * 200 + [16_001, 5, 12_000] + [17] * 150, 16),
    (W.FULL, 256, 4, 2, 0, [(53 * i) % 97 for i in range(333)], 16),          # units unsplit
]


@pytest.mark.parametrize("kind,D,hq,hkv,Wn,lens,ps", CASES, ids=[f"{'FS'[c[0]]}{c[1]}-{c[2]}q{c[3]}kv-{len(c[5])}-{max(c[5])}"
                                                                   for c in CASES])
def test_every_tile_counts_once(kind, D, hq, hkv, Wn, lens, ps):
    case, want, n = tile_case(kind, D, hq, hkv, Wn, lens, ps)
    fused, ws = case.decode(0, fused=True), case.workspace(0)
    check(case, want, n, *fused)
    for _ in range(10):
        out, lse = case.decode(0, ws)
        assert torch.equal(out, fused[0]) and torch.equal(lse, fused[1])
    if case.cache.decode_workspace_bytes(0, case.B, case.max_len) <= case.fa.NOALLOC_SCRATCH_BYTES:
        out, lse = case.outs(0)
        case.cache.decode_noalloc(0, case.q[0], case.bt[0], case.lens_dev, case.max_len, out, lse)
        assert torch.equal(out, fused[0]) and torch.equal(lse, fused[1])
    assert case.cache.device_error() == 0


def test_every_tile_counts_once_in_a_launch_of_several_layers():
    lens, heads = [9000, 40, 0, 20_000, 16, 700], [(8, 1), (8, 2), (16, 1)]
    cases = [tile_case(W.FULL, 512, hq, hkv, 0, lens, 16) for hq, hkv in heads]
    a = cases[0][0]
    cache = a.fa.Cache([W.layer(W.FULL, 512, hq, hkv) for hq, hkv in heads], a.cache.num_pages, 16, a.fa.KV_FP4)
    slabs = cache.allocate("cuda")
    for i, (c, _, _) in enumerate(cases):
        c.store_current()
        for x, y in zip(slabs[i], c.slabs[0]):
            x.copy_(y)
    for ids in ([0, 1, 2], [2, 0], [1]):
        ws = a.fa.workspace(cache.decode_layers_workspace_bytes(ids, a.B, a.max_len))
        outs = [cases[i][0].outs(0) for i in ids]
        for _ in range(2):
            cache.decode_layers(ids, [cases[i][0].q[0] for i in ids], [cases[i][0].bt[0] for i in ids], a.lens_dev,
                                a.max_len, [o for o, _ in outs], [l for _, l in outs], ws)
            for i, (o, l) in zip(ids, outs):
                check(*cases[i], o, l)
    assert cache.device_error() == 0


@pytest.mark.parametrize("D", [256, 512])
def test_joins_of_shares_that_go_on_to_the_next_unit(D):
    """Long units between short ones, laid end to end: the share that ends a long
    unit joins several levels of its parts with its next unit's rows already
    landing in the ring.  Random values, the same bits on every one of many runs."""
    rng = np.random.default_rng(3)
    lens = [int(n) for n in rng.integers(1, 40, 460)]
    for b, n in ((40, 5003), (41, 9001), (222, 12_345), (300, 3000), (459, 7007)):
        lens[b] = n
    case = DecodeCase4([W.layer(W.FULL, D, 8, 1)], lens, 16, seed=21)
    case.store_current()
    ws = case.workspace(0)
    out, lse = case.decode(0, ws)
    case.check(0, out, lse, [0, 39, 40, 41, 42, 222, 223, 300, 301, 459])
    for _ in range(200):
        o, l = case.decode(0, ws)
        assert torch.equal(o.view(torch.int16), out.view(torch.int16)) and torch.equal(l, lse)
    assert case.cache.device_error() == 0
