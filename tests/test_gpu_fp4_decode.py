"""Decode attention over fp4 slabs against float64 (fp4_case.py: inputs, reference, bounds)."""
import numpy as np
import pytest
import torch

import workloads as W
from fp4_case import DecodeCase4

pytestmark = pytest.mark.gpu


def lay(kind, D, hq, hkv, Wn=0, src=W.KV_OWN):
    return W.layer(kind, D, hq, hkv, Wn, src)


EDGES = [1, 15, 16, 17, 63, 64, 65, 0, 127, 128, 129, 200, 257, 31]

CASES = [
    (W.FULL, 512, 8, 1, 0, EDGES, 16),
    (W.FULL, 256, 8, 1, 0, EDGES, 16),
    (W.SLIDING, 256, 4, 1, 64, EDGES, 16),
    (W.SLIDING, 512, 4, 1, 64, EDGES, 32),
    (W.SLIDING, 256, 8, 2, 1, [1, 2, 16, 17, 300], 48),
    (W.SLIDING, 256, 8, 2, 17, [1, 2, 16, 17, 18, 33, 300], 256),
    (W.SLIDING, 512, 6, 3, 100, [99, 100, 101, 1000], 64),
    (W.FULL, 512, 12, 2, 0, [700, 3, 0, 1025], 48),          # six heads per KV head
    (W.FULL, 256, 16, 1, 0, [513, 64, 1], 16),               # two chunks of heads
    (W.FULL, 512, 17, 1, 0, [200, 0, 90], 16),               # three chunks, the last of one head
    (W.FULL, 256, 9, 9, 0, [333, 10], 16),                   # one head per KV head
    (W.FULL, 512, 8, 1, 0, [6001], 16),                      # one sequence, split
    (W.FULL, 256, 8, 1, 0, [9001, 5], 128),
    (W.SLIDING, 256, 8, 1, 1024, [1024, 5000, 3000, 1023, 2048, 1500], 16),   # equal units: cut into equal parts
    (W.FULL, 512, 8, 1, 0, list(range(0, 400, 2)), 16),      # more units than threads
    (W.FULL, 256, 2, 2, 0, [0, 0], 16),                      # nothing visible
    # partials joined: 4 to 7 and 26 CTAs of one share, then CTAs of two and of three shares
    *[(W.FULL, D, 8, 1, 0, [n], 16) for D in (256, 512) for n in (512, 640, 768, 896, 3328, 20_011)],
    (W.FULL, 512, 8, 1, 0, [60_001], 64),
    (W.FULL, 256, 8, 2, 0, [30_000, 17, 0, 9_000], 16),
    (W.FULL, 512, 2, 1, 0, [4000, 900, 5000, 100, 2500, 3000, 1, 700, 6000, 2222], 16),
    # more short units than parts of full length: a share each
    (W.SLIDING, 256, 24, 8, 1450, [2, 3, 4, 0, 3, 4, 2, 1, 17, 4], 32),
    (W.FULL, 512, 13, 1, 0, [81, 83], 128),
    # sequences past a warp's registers, in a whole-unit cut and with more units than shares
    (W.FULL, 256, 4, 1, 0, [(37 * i) % 90 if i % 50 else 1700 for i in range(200)], 16),
    (W.FULL, 256, 4, 2, 0, [(53 * i) % 97 for i in range(333)], 16),
    (W.SLIDING, 512, 8, 1, 40, [(29 * i) % 75 for i in range(1025)], 32),
    (W.FULL, 512, 10, 1, 0, [(31 * i) % 260 for i in range(255)], 16),    # units of up to 17 tiles
    (W.FULL, 512, 10, 1, 0, [(31 * i) % 257 for i in range(255)], 16),    # and of up to 16
]


@pytest.mark.parametrize("kind,D,hq,hkv,Wn,lens,ps", CASES, ids=[f"{'FS'[c[0]]}{c[1]}-{c[2]}q{c[3]}kv-W{c[4]}-{i}"
                                                                   for i, c in enumerate(CASES)])
def test_decode(kind, D, hq, hkv, Wn, lens, ps):
    case = DecodeCase4([lay(kind, D, hq, hkv, Wn)], lens, ps, seed=len(lens))
    case.store_current()
    ws = case.workspace(0)
    out, lse = case.decode(0, ws)
    assert case.cache.device_error() == 0
    case.check(0, out, lse, None if len(lens) < 50 else range(0, len(lens), 23))
    for _ in range(3):   # the same bits each time, through the same workspace
        o2, l2 = case.decode(0, ws)
        assert torch.equal(out.view(torch.int16), o2.view(torch.int16)) and torch.equal(lse, l2)


STACK = [lay(W.SLIDING, 256, 8, 1, 64), lay(W.FULL, 512, 8, 1), lay(W.SLIDING, 256, 4, 1, 64, W.KV_AUTO),
         lay(W.FULL, 512, 16, 1, 0, W.KV_AUTO), lay(W.SLIDING, 256, 8, 1, 64)]


@pytest.mark.parametrize("window_pool", [False, True])
def test_layer_stack_fused_layers_and_noalloc_agree(window_pool):
    """Shared layers, the fused store, the multi-layer launch and the
    allocation-free call: the same bits as store, then decode."""
    lens = [1, 40, 700, 64, 0, 2001, 333]
    a = DecodeCase4(STACK, lens, 16, seed=3, window_pool=window_pool)
    b = DecodeCase4(STACK, lens, 16, seed=3, window_pool=window_pool)
    a.store_current()
    ref = {i: a.decode(i) for i in range(len(STACK))}
    for i, (o, l) in ref.items():
        a.check(i, o, l)
    same = lambda x, y: torch.equal(x[0].view(torch.int16), y[0].view(torch.int16)) and torch.equal(x[1], y[1])
    for i in range(len(STACK)):
        assert same(b.decode(i, fused=True), ref[i])
    for i in a.slabs:   # the fused store wrote the same rows (unwritten slots hold the same junk)
        for x, y in zip(a.slabs[i], b.slabs[i]):
            assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))
    for ids in ([0, 2, 4], [1, 3]):
        outs = [a.outs(i) for i in ids]
        ws = a.fa.workspace(a.cache.decode_layers_workspace_bytes(ids, a.B, a.max_len))
        for _ in range(2):
            a.cache.decode_layers(ids, [a.q[i] for i in ids], [a.bt[i] for i in ids], a.lens_dev, a.max_len,
                                  [o for o, _ in outs], [l for _, l in outs], ws)
        for i, (o, l) in zip(ids, outs):
            a.check(i, o, l)
    for i in range(len(STACK)):
        o, l = a.outs(i)
        a.cache.decode_noalloc(i, a.q[i], a.bt[i], a.lens_dev, a.max_len, o, l)
        assert same((o, l), ref[i])
    assert a.cache.device_error() == 0 and b.cache.device_error() == 0


@pytest.mark.parametrize("D,hkv,lens", [(512, 1, [(97 * i) % 700 for i in range(128)]), (256, 2, [(53 * i) % 97 for i in range(333)]),
                                        (256, 1, [9000, 0, 40]), (512, 2, [(41 * i) % 350 for i in range(130)]),
                                        (512, 1, [700 + i for i in range(152)])],
                         ids=["batch 128", "unsplit", "split", "end to end", "equal"])
def test_fused_store_and_noalloc_in_every_cut(D, hkv, lens):
    """The fused store and the allocation-free call, the same bits as store, then decode."""
    layer = [lay(W.FULL, D, 4 * hkv, hkv)]
    a, b = (DecodeCase4(layer, lens, 16, seed=13) for _ in range(2))
    a.store_current()
    ref = a.decode(0)
    assert a.cache.device_error() == 0
    a.check(0, *ref, range(0, len(lens), 41))
    got = b.decode(0, fused=True)
    for x, y in zip(a.slabs[0], b.slabs[0]):
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))
    out, lse = a.outs(0)
    noalloc = lambda: a.cache.decode_noalloc(0, a.q[0], a.bt[0], a.lens_dev, a.max_len, out, lse)
    if a.cache.decode_workspace_bytes(0, a.B, a.max_len) > 8 << 20:   # more than the library's fixed scratch
        with pytest.raises(a.fa.FAError) as e:
            noalloc()
        assert e.value.status == a.fa.ERR_WORKSPACE and lens != [(97 * i) % 700 for i in range(128)]
        out, lse = got
    else:
        noalloc()
    for o, l in (got, (out, lse)):
        assert torch.equal(o.view(torch.int16), ref[0].view(torch.int16)) and torch.equal(l, ref[1])
    assert a.cache.device_error() == 0 and b.cache.device_error() == 0


def test_value_scales_far_apart():
    """Zero V rows under large weights, and V rows 2^110 apart in magnitude: the
    weights follow score + value scale, the denominator the scores alone."""
    def edit(i, k, v):
        v[0] = 0.0                                   # a sink token: large key, no value
        k[0] = k[0] * 8
        v[1:40] = v[1:40] * 2.0 ** -60
        v[100:120] = v[100:120] * 2.0 ** 50
        v[333] = 0.0
    for D in (256, 512):
        case = DecodeCase4([lay(W.FULL, D, 8, 1)], [40, 300, 77], 16, seed=9, edit=edit)
        case.store_current()
        out, lse = case.decode(0)
        assert case.cache.device_error() == 0
        case.check(0, out, lse)


def test_one_key_gives_its_value():
    """A window of 1: the output is the current row's kept value, bit for bit."""
    for D in (256, 512):
        case = DecodeCase4([lay(W.SLIDING, D, 8, 2, 1)], [1, 5, 16, 33, 100], 16, seed=2)
        out, lse = case.decode(0, fused=True)
        assert case.cache.device_error() == 0
        for b in range(case.B):
            V = case.vals[0][b][1][-1]
            got = out[b].double().cpu().numpy()
            for j in range(8):
                assert np.array_equal(got[j], V[j // 4])


def test_graph_replays_with_new_lengths_and_rows():
    case = DecodeCase4([lay(W.FULL, 512, 8, 1)], [600, 33, 128, 2000], 16, seed=5)
    case.cache.set_flags(case.fa.FLAG_EARLY_METADATA)
    ws = case.workspace(0)
    out, lse = case.outs(0)
    lens = case.lens_dev.clone()
    q = case.q[0].clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    k, v = case.new[0]
    with torch.cuda.stream(s):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            case.cache.store(0, k, v, case.slots[0])
            case.cache.decode(0, q, case.bt[0], lens, case.max_len, out, lse, ws)
    for cut in (0, 5, 30):
        n = np.maximum(case.lens - cut, 1)
        lens.copy_(torch.from_numpy(n.astype(np.int32)))
        g.replay()
        torch.cuda.synchronize()
        keep, case.lens = case.lens, n.astype(np.int32)
        vals = case.vals[0]
        case.vals[0] = [[x[: int(m)] for x in kv] for kv, m in zip(vals, n)]
        case.check(0, out, lse)
        case.vals[0], case.lens = vals, keep
    assert case.cache.device_error() == 0


def test_rows_past_two_gigabytes():
    """Slab offsets beyond 32 bits: the last pages of a slab of 2.8 GB."""
    import full_attention_gb300 as fa
    pages = 600_000
    cache = fa.Cache([lay(W.FULL, 512, 8, 1)], pages, 16, fa.KV_FP4)
    slab = cache.allocate("cuda")[0]
    assert slab[0].numel() > 1 << 31
    small = DecodeCase4([lay(W.FULL, 512, 8, 1)], [100, 37], 16, seed=6)
    small.store_current()
    ref = small.decode(0)
    bt = torch.where(small.bt[0] >= 0, pages - 1 - small.bt[0], -1).int()
    n = small.slabs[0][0].shape[0]
    for x, y in zip(slab, small.slabs[0]):
        x[pages - n:].copy_(y.flip(0))
    out, lse = small.outs(0)
    cache.decode(0, small.q[0], bt, small.lens_dev, small.max_len, out, lse, small.workspace(0))
    assert cache.device_error() == 0
    assert torch.equal(out.view(torch.int16), ref[0].view(torch.int16)) and torch.equal(lse, ref[1])


def test_bad_pages_lengths_queries_and_workspaces_are_reported():
    case = DecodeCase4([lay(W.FULL, 512, 8, 1)], [300, 40], 16, seed=7)
    case.store_current()
    fa, c = case.fa, case.cache
    good = case.decode(0)
    for bad in (-1, case.cache.num_pages, 1 << 30):
        bt = case.bt[0].clone()
        bt[0, 3] = bad
        out, lse = case.outs(0)
        c.decode(0, case.q[0], bt, case.lens_dev, case.max_len, out, lse, case.workspace(0))
        assert c.device_error() == fa.DEV_ERR_PAGE
        assert torch.isfinite(out.float()).all()
        assert torch.equal(out[1].view(torch.int16), good[0][1].view(torch.int16))   # the other sequence is untouched
    out, lse = case.outs(0)
    c.decode(0, case.q[0], case.bt[0], case.lens_dev, 299, out, lse, case.workspace(0))
    assert c.device_error() == fa.DEV_ERR_BOUND
    big = case.q[0].clone()
    big[1, 3, 5] = 1e30
    c.decode(0, big, case.bt[0], case.lens_dev, case.max_len, out, lse, case.workspace(0))
    assert c.device_error() == fa.DEV_ERR_RANGE
    ws = case.workspace(0)
    with pytest.raises(fa.FAError) as e:
        c.decode(0, case.q[0], case.bt[0], case.lens_dev, case.max_len, out, lse, ws[:-1])
    assert e.value.status == fa.ERR_WORKSPACE
    # 33 sequences of up to 2^26 tiles: more than the kernel counts (all empty, were it to run)
    q33, none = torch.zeros((33, 8, 512), dtype=torch.bfloat16, device="cuda"), torch.zeros(33, dtype=torch.int32, device="cuda")
    big_ws, o33 = fa.workspace(c.decode_workspace_bytes(0, 33, 1 << 30)), torch.empty_like(q33)
    for n, st in ((1 << 30, fa.ERR_UNSUPPORTED), (1 << 29, fa.OK)):
        assert fa.lib().fa_paged_decode_attn(c._h, 0, q33.data_ptr(), none.data_ptr(), 1 << 26, none.data_ptr(), 33, n,
                                             o33.data_ptr(), None, big_ws.data_ptr(), big_ws.numel(), None) == st
    assert (o33 == 0).all()
    for q, o in ((case.q[0].float(), out), (case.q[0].transpose(1, 2), out), (case.q[0], out[:, ::2])):
        with pytest.raises(fa.FAError) as e:
            c.decode(0, q, case.bt[0], case.lens_dev, case.max_len, o, lse, ws)
        assert e.value.status == fa.ERR_INVALID_ARG


def test_two_streams_with_their_own_workspaces():
    a = DecodeCase4([lay(W.FULL, 512, 8, 1)], [3000, 40, 900], 16, seed=11)
    a.store_current()
    ref = a.decode(0)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    res = []
    for s in streams:
        out, lse = a.outs(0)
        ws = a.workspace(0)
        torch.cuda.synchronize()
        for _ in range(20):
            a.cache.decode(0, a.q[0], a.bt[0], a.lens_dev, a.max_len, out, lse, ws, stream=s)
        res.append((out, lse))
    torch.cuda.synchronize()
    for out, lse in res:
        assert torch.equal(out.view(torch.int16), ref[0].view(torch.int16)) and torch.equal(lse, ref[1])


@pytest.mark.parametrize("D", [256, 512])
@pytest.mark.parametrize("grow", [1.0, 30.0, 1000.0, 2.0 ** 30])
def test_one_key_gives_its_value_whatever_its_score(D, grow):
    """Scores of tens of thousands to past 2^23.  The value's exponent joins the
    score in the weight's exponent, which must not round at the score's own scale.
    Past 2^23 in log2 units, where that cannot be had, the call reports its range."""
    def edit(i, k, v):
        k.mul_(grow)
    case = DecodeCase4([lay(W.SLIDING, D, 8, 2, 1)], [1, 5, 16, 33, 100], 16, seed=2, edit=edit)
    case.q[0].mul_(10_000.0)
    out, lse = case.decode(0, fused=True)
    q = case.q[0].double().cpu().numpy()
    score = np.array([[case.layers[0]["sm_scale"] * (case.vals[0][b][0][-1, j // 4] @ q[b, j]) for j in range(8)]
                      for b in range(case.B)])
    err = np.array([[np.abs(case.vals[0][b][0][-1, j // 4]) @ np.abs(q[b, j]) for j in range(8)] for b in range(case.B)])
    err *= case.layers[0]["sm_scale"] * 600 * 2.0 ** -24      # fp32 sums of 512 products, a few roundings more
    log2 = np.abs(score) * np.log2(np.e)
    inside = log2 < 2.0 ** 23 * 0.99
    assert case.cache.device_error() == (0 if inside.all() else case.fa.DEV_ERR_RANGE)
    assert inside.all() == (grow <= 30.0) and (grow < 2.0 ** 30 or not inside.any())
    assert (np.abs(lse.double().cpu().numpy() - score) <= err + 2.0 ** -22 * np.abs(score))[inside].all()
    got = out.double().cpu().numpy()
    for b, j in zip(*np.nonzero(inside)):
        assert np.array_equal(got[b, j], case.vals[0][b][1][-1, j // 4]), (b, j, score[b, j])
