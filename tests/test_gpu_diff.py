"""Differential attention over the paged cache, decode and extend, against 64 bits
(bounds in diff_case.py)."""
import pytest
import torch

import workloads as W
from diff_case import DiffCase

pytestmark = pytest.mark.gpu

FORMATS = [W.KV_BF16, W.KV_INT8, W.KV_FP8]

DECODE = [  # D, hq, hkv, page, window, lens
    (256, 1, 1, 16, 0, [1]), (512, 8, 1, 16, 0, [1, 2, 15, 16, 17, 0, 33]), (256, 4, 1, 16, 64, [200]),
    (512, 8, 1, 16, 0, [4096, 513, 70]), (256, 16, 8, 16, 100, [900, 99, 100, 101, 1, 0, 3000]),
    (512, 12, 2, 48, 0, [1000, 5, 0, 2500, 31]), (256, 9, 1, 32, 1, [50, 1, 16, 17]), (512, 24, 1, 64, 33, [700, 20]),
    (256, 34, 2, 256, 0, [2222, 300, 1, 0]), (512, 16, 2, 16, 1024, [5000, 1023, 1024, 1025]),
    (256, 8, 1, 16, 0, [0, 0]), (512, 8, 8, 16, 0, [20000]), (256, 8, 1, 16, 0, list(range(1, 200))), (512, 4, 4, 16, 300, [299 + i for i in range(90)]),
]


@pytest.mark.parametrize("kv", FORMATS)
@pytest.mark.parametrize("D,hq,hkv,ps,window,lens", DECODE)
def test_decode(D, hq, hkv, ps, window, lens, kv):
    c = DiffCase(D, hq, hkv, ps, lens, kv, window, seed=D + hq + len(lens))
    c.check(*c.decode())


@pytest.mark.parametrize("kv", FORMATS)
@pytest.mark.parametrize("D,early", [(256, True), (512, False)])
def test_decode_stores_the_current_rows(D, early, kv):
    """One launch equals the store and the decode; the slab's bytes are the store's."""
    lens = [1, 40, 0, 700, 16, 17, 3000]
    c = DiffCase(D, 8, 2, 16, lens, kv, seed=D, early=early)
    new = [torch.zeros((c.B, 2, D), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    slots = torch.full((c.B,), -1, dtype=torch.int32, device="cuda")
    for b, n in enumerate(lens):
        if n > 0:
            slots[b] = int(c.bt[b, (n - 1) // 16]) * 16 + (n - 1) % 16
            for i in range(2):
                new[i][b] = c.raw[b][1][i][-1]
    c.cache.store(0, *new, slots)
    want = [t.clone() for t in c.decode()]
    slab = [None if t is None else t.clone() for t in c.slabs]
    for slot in slots[slots >= 0].tolist():
        for i in range(2):
            c.slabs[i][slot // 16, :, slot % 16] = 0x55 if kv else 3.0
            if kv:
                c.slabs[2 + i][slot // 16, :, slot % 16] = float("nan")
    got = c.decode(k_new=new[0], v_new=new[1], slot_mapping=slots)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert all(a is None or torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(slab, c.slabs))
    c.check(*got)


@pytest.mark.parametrize("lam", [0.0, 1.0, -2.5, 1e3])
def test_lambda(lam):
    c = DiffCase(512, 8, 1, 16, [300, 7], seed=3, lam=lam, offset=4.0)
    c.check(*c.decode())
    e = DiffCase(256, 4, 2, 16, [300, 0], new=[9, 130], seed=3, lam=lam, offset=4.0)
    e.check(*e.extend())


def test_equal_maps_leave_one_minus_lambda():
    """The same halves give the same weights: (1 - lambda) softmax(..) v, and 0 at lambda 1 exactly."""
    for kv in FORMATS:
        c = DiffCase(256, 8, 1, 16, [1200, 50], kv, seed=4, lam=1.0)
        h = c.D // 2
        c.q[..., h:] = c.q[..., :h]
        c.slabs[0][..., h:] = c.slabs[0][..., :h]
        out, lse = c.decode()
        assert torch.equal(lse[..., 0], lse[..., 1])
        assert float(out.float().abs().max()) <= 2.0 ** -20


def test_shared_layers_read_their_source():
    c = DiffCase(512, 8, 2, 16, [400, 33], seed=5, shared=True)
    c.check(*c.decode(k_new=None, v_new=None, slot_mapping=None))
    e = DiffCase(256, 8, 2, 32, [400, 33], W.KV_INT8, new=[5, 60], seed=5, shared=True)
    e.check(*e.extend())


EXTEND = [  # D, hq, hkv, page, window, prefix, new
    (256, 1, 1, 16, 0, [0], [1]), (512, 4, 2, 16, 0, [0, 5], [3, 1]), (256, 16, 8, 16, 100, [900, 99, 0], [64, 63, 130]),
    (512, 16, 2, 32, 0, [1000, 0, 70, 16], [1, 300, 64, 0]), (256, 64, 1, 16, 0, [130], [40]), (512, 32, 1, 64, 40, [500, 39], [77, 2]),
    (256, 8, 8, 48, 1, [100, 0], [33, 65]), (512, 2, 1, 16, 700, [3000, 699], [200, 5]), (256, 2, 1, 256, 0, [2047], [513]),
]


@pytest.mark.parametrize("kv", FORMATS + [W.KV_FP4])
@pytest.mark.parametrize("D,hq,hkv,ps,window,prefix,new", EXTEND)
@pytest.mark.parametrize("split", [None, "all"])
def test_extend(D, hq, hkv, ps, window, prefix, new, split, kv):
    if kv == W.KV_FP4:   # rows that the 4-bit cache keeps exactly: its own, read back
        c = _fp4(D, hq, hkv, ps, window, prefix, new)
    else:
        c = DiffCase(D, hq, hkv, ps, prefix, kv, window, new, seed=D + hq + len(new))
    if split:
        fa = c.fa
        ws = fa.workspace(c.cache.extend_workspace_bytes(c.layer, c.B, max(new), max(prefix)))
        c.cache.bind_extend_workspace(ws)
        c.cache.set_flags(fa.FLAG_EXTEND_SPLIT_ALL)
    c.check(*c.extend())


@pytest.mark.parametrize("kv", [W.KV_INT8, W.KV_FP8])
@pytest.mark.parametrize("D,hq,hkv,ps,window,prefix,new", EXTEND + [
    (256, 16, 8, 16, 1024, [3584, 1, 0, 1500], [512, 300, 64, 0]), (512, 16, 2, 32, 0, [0, 2100, 3814, 16], [400, 1, 513, 1000]),
    (512, 8, 1, 64, 0, [0, 0, 0], [700, 63, 65])])
def test_extend_over_f16_rows_is_the_same(D, hq, hkv, ps, window, prefix, new, kv):
    """With room in the workspace the codes and the chunk become f16 rows before the
    kernel: the same operands, so the same bits; nothing of what lay in the room, of
    another sequence's chunk or of rows that nobody sees gets into a result."""
    c = DiffCase(D, hq, hkv, ps, prefix, kv, window, new, seed=D + hq + len(new))
    fa = c.fa
    base = fa.extend_workspace_bytes()
    full = c.cache.extend_workspace_bytes(c.layer, c.B, max(new), max(prefix))
    assert full > base
    ws = torch.full((full,), 0xFF, dtype=torch.uint8, device="cuda")
    res = []
    for n in (base, full, full - 256 * 64):   # (the last has not the room)
        ws[base:] = 0xFF
        c.cache.bind_extend_workspace(ws[:n])
        c.out.fill_(float("nan")), c.lse.fill_(float("nan"))
        res.append([t.clone() for t in c.extend()])
    c.check(*res[0])
    for out, lse in res[1:]:
        assert torch.equal(out, res[0][0]) and torch.equal(lse, res[0][1])


@pytest.mark.parametrize("kv", [W.KV_INT8, W.KV_FP8])
@pytest.mark.parametrize("D", [256, 512])
def test_f16_rows_keep_sequences_apart(D, kv):
    """Sequences of NaN in rows and chunk beside others; a page that is none; a chunk
    beyond f16's range: as without the workspace, and reported."""
    c = DiffCase(D, 16, 2, 16, [700, 200, 900], kv, 0, [330, 70, 280], seed=D)
    fa = c.fa
    ws = fa.workspace(c.cache.extend_workspace_bytes(0, c.B, 330, 900))
    c.cache.bind_extend_workspace(ws)
    want = [t.clone() for t in c.extend()]
    c.check(*want)
    page = c.bt[1, : 200 // 16].long()
    keep = [t[page].clone() for t in c.slabs[2:]], c.k_ext.clone(), c.v_ext.clone()
    for t in c.slabs[2:]:
        t[page] = float("nan")
    c.v_ext[330:400] = float("nan")
    got = c.extend()
    assert c.cache.device_error() == fa.DEV_ERR_RANGE
    for a, b in zip(got, want):
        assert torch.equal(a[:330], b[:330]) and torch.equal(a[400:], b[400:])
    c.v_ext.copy_(keep[2])
    for t, k in zip(c.slabs[2:], keep[0]):
        t[page] = k
    bt = c.bt.clone()
    results = []
    for n in (fa.extend_workspace_bytes(), ws.numel()):
        c.cache.bind_extend_workspace(ws[:n])
        c.bt = bt.clone()
        c.bt[0, 3] = c.cache.num_pages
        c.k_ext[5] = 1e5
        results.append([t.clone() for t in c.extend()])
        assert c.cache.device_error() == fa.DEV_ERR_PAGE | fa.DEV_ERR_RANGE
        c.bt, c.k_ext = bt, keep[1].clone()
    for a, b in zip(*results):   # bits: scores beyond the softmax's range may leave NaN
        assert torch.equal(a.view(torch.int16), b.view(torch.int16))


def test_f16_rows_in_a_graph_and_between_other_calls():
    """One workspace: calls of other sizes, layers and plain attention between, and a replay."""
    import full_attention_gb300 as fa
    a = DiffCase(512, 8, 2, 16, [800, 90], W.KV_FP8, 0, [260, 300], seed=1)
    b = DiffCase(256, 8, 4, 32, [1500, 0, 70], W.KV_INT8, 200, [64, 130, 1], seed=2)
    ws = fa.workspace(max(c.cache.extend_workspace_bytes(0, c.B, max(c.new), max(c.lens)) for c in (a, b)))
    want = [[t.clone() for t in c.extend()] for c in (a, b)]
    for c in (a, b):
        c.cache.bind_extend_workspace(ws)
    for c, w in zip((a, b, a, b), want * 2):
        c.out.zero_(), c.lse.zero_()
        got = c.extend()
        assert all(torch.equal(x, y) for x, y in zip(got, w))
    plain = torch.empty_like(a.out)
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        a.extend()
        b.extend()
        a.cache.extend(0, a.q, a.k_ext, a.v_ext, a.indptr, a.lens_dev, a.bt, 300, 800, plain)
    for _ in range(3):
        for c in (a, b):
            c.out.zero_(), c.lse.zero_()
        ws[fa.extend_workspace_bytes():] = 0xFF
        g.replay()
        for c, w in zip((a, b), want):
            assert torch.equal(c.out, w[0]) and torch.equal(c.lse, w[1])
    assert a.cache.device_error() == b.cache.device_error() == 0


@pytest.mark.parametrize("kv", FORMATS)
@pytest.mark.parametrize("D", [256, 512])
@pytest.mark.parametrize("early", [False, True])
def test_shared_layers_padded_batches_and_plain_calls(kv, D, early):
    """A layer that reads its source; token rows behind the last sequence, NaN, get into
    no result or report and their outputs stay; in 8 bits with and without f16 rows, and
    plain attention with the same workspace is as without."""
    c = DiffCase(D, 16, 2, 64, [1200, 0, 640], kv, 0, [200, 170, 33], seed=9, shared=True, early=early)
    fa, N, more = c.fa, 403, 61
    pad = lambda t, x: torch.cat((t, torch.full((more,) + t.shape[1:], x, dtype=t.dtype, device="cuda")))
    q, k, v = (pad(t, float("nan")) for t in (c.q, c.k_ext, c.v_ext))
    ws = fa.workspace(c.cache.extend_workspace_bytes(1, c.B, 200, 1200))
    base = fa.extend_workspace_bytes()
    got, plain = [], []
    for n in (base, ws.numel()):
        c.cache.bind_extend_workspace(ws[:n])
        out, lse = pad(c.out, 7.0), pad(c.lse, 7.0)
        c.cache.extend_diff(1, q, c.lam, k, v, c.indptr, c.lens_dev, c.bt, 200, 1200, out, lse)
        got.append((out, lse))
        c.check(out[:N], lse[:N])
        out = pad(c.out, 7.0)
        c.cache.extend(1, pad(c.q, 0.0), pad(c.k_ext, 0.0), pad(c.v_ext, 0.0), c.indptr, c.lens_dev, c.bt, 200, 1200, out)
        plain.append(out)
    for (a, b) in zip(*got):
        assert torch.equal(a, b) and bool((a[N:] == 7.0).all())
    assert torch.equal(*plain) and bool((plain[0][N:] == 7.0).all())


def _fp4(D, hq, hkv, ps, window, prefix, new):
    import full_attention_gb300 as fa
    c = DiffCase(D, hq, hkv, ps, prefix, W.KV_BF16, window, new, seed=D + hq + len(new))
    lay = dict(c.cache.layers[0])
    cache = fa.Cache([lay], c.cache.num_pages, ps, fa.KV_FP4)
    c.slabs = cache.allocate("cuda")[0]
    for t in c.slabs:
        t.fill_(float("nan") if t.is_floating_point() else 0x7F)
    rows = []
    for b, n in enumerate(prefix):
        lo, (k, v) = c.raw[b]
        pos = torch.arange(lo, n, device="cuda")
        if len(pos):
            slots = (c.bt[b][pos // ps].long() * ps + pos % ps).int()
            cache.store(0, k, v, slots)
            kb, vb = torch.empty_like(k), torch.empty_like(v)
            cache.load(0, slots, kb, vb)
            k, v = kb, vb
        rows.append((lo, k.double(), v.double()))
    c.cache, c.rows, c.kv = cache, rows, W.KV_FP4
    return c


def test_one_workspace_serves_plain_and_differential_calls():
    c = DiffCase(512, 8, 1, 16, [3000, 2000, 77], seed=6)
    d = DiffCase(512, 8, 1, 16, [9000, 40], seed=7)
    ws = c.fa.workspace(max(x.cache.decode_diff_workspace_bytes(0, x.B, x.max_len()) for x in (c, d)))
    first = None
    for _ in range(2):
        c.check(*c.decode(ws))
        plain = torch.empty_like(d.out)
        d.cache.decode(0, d.q, d.bt, d.lens_dev, d.max_len(), plain, None, ws)
        d.check(*d.decode(ws))
        first = plain.clone() if first is None else first
        assert torch.equal(first, plain)
    assert int(ws[: c.fa.DECODE_COUNTER_BYTES].any()) == 0


def test_captured_calls_and_another_stream():
    c = DiffCase(256, 8, 2, 16, [3000, 1, 250], W.KV_FP8, seed=8)
    e = DiffCase(512, 8, 2, 16, [300, 0], new=[40, 130], seed=8)
    ws = c.fa.workspace(c.cache.decode_diff_workspace_bytes(0, c.B, c.max_len()))
    want = [t.clone() for t in c.decode(ws) + e.extend()]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.decode(ws)
        e.extend()
    for t in (c.out, c.lse, e.out, e.lse):
        t.fill_(7.0)
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip((c.out, c.lse, e.out, e.lse), want))
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        c.decode(ws)
        e.extend()
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip((c.out, c.lse, e.out, e.lse), want))


def test_faults_are_reported_not_followed():
    fa = DiffCase(256, 2, 1, 16, [40], seed=1).fa
    c = DiffCase(256, 2, 1, 16, [40, 40], seed=1)
    c.bt[0, 1] = c.cache.num_pages
    out, _ = c.decode()
    assert c.cache.device_error() == fa.DEV_ERR_PAGE
    ref, _, room = c.reference()
    assert bool(((out[1].double() - ref[1]).abs() <= room[1]).all())
    c = DiffCase(256, 2, 1, 16, [40, 40], seed=1)
    ws = fa.workspace(c.cache.decode_diff_workspace_bytes(0, 2, 39))
    c.cache.decode_diff(0, c.q, c.lam, c.bt, c.lens_dev, 39, c.out, c.lse, ws)
    assert c.cache.device_error() == fa.DEV_ERR_BOUND
    c = DiffCase(512, 2, 1, 16, [40], W.KV_INT8, seed=1)
    c.q[0, 1, 300] = 1e5
    c.decode()
    assert c.cache.device_error() == fa.DEV_ERR_RANGE
