"""Extend and multi-token decode over fp4 slabs against float64 (fp4_case.py:
inputs, reference, bounds; chunk rows stay bf16, exact in f16 at these sizes)."""
import numpy as np
import pytest
import torch

import workloads as W
from fp4_case import ExtendCase4

pytestmark = pytest.mark.gpu


def lay(kind, D, hq, hkv, Wn=0, src=W.KV_OWN):
    return W.layer(kind, D, hq, hkv, Wn, src)


CASES = [
    # layer, prefix, chunk, page size
    (lay(W.SLIDING, 256, 4, 2, 48), [40, 0, 100, 17], [37, 20, 130, 1], 16),
    (lay(W.FULL, 512, 8, 1), [40, 0, 100, 17], [37, 20, 130, 1], 16),
    (lay(W.FULL, 256, 16, 8), [64, 3], [64, 200], 16),
    (lay(W.SLIDING, 512, 16, 2, 100), [300, 33], [90, 160], 48),
    (lay(W.SLIDING, 256, 8, 1, 1), [20, 0], [45, 16], 16),            # W = 1: only the current token
    (lay(W.FULL, 256, 2, 2), [0, 129], [257, 1], 256),                # an empty prefix, a single new token
    (lay(W.SLIDING, 512, 8, 2, 40), [95, 33, 64, 15, 16], [33, 96, 1, 16, 0], 32),   # a sequence with nothing new
    (lay(W.FULL, 512, 16, 1), [1000], [17], 64),
    (lay(W.FULL, 256, 128, 1), [130, 5], [3, 2], 16),                 # 128 query heads to one KV head
    (lay(W.SLIDING, 256, 8, 2, 300), [900, 299, 300, 301, 17], [40, 70, 16, 1, 200], 16),   # a window's ring that wraps
    (lay(W.FULL, 256, 8, 1), [700, 0], [5, 300], 128),
]
IDS = [f"{'FS'[c[0]['kind']]}{c[0]['head_dim']}-{c[0]['num_q_heads']}q{c[0]['num_kv_heads']}kv-W{c[0]['window']}" for c in CASES]


@pytest.mark.parametrize("layer,prefix,chunk,ps", CASES, ids=IDS)
@pytest.mark.parametrize("split", [None, "all", "unpack", "unpack all"])
def test_extend(layer, prefix, chunk, ps, split):
    c = ExtendCase4([layer], prefix, chunk, ps, seed=31, split=split)
    out, lse = c.run(0)
    assert c.cache.device_error() == 0
    c.check(0, out, lse)
    o2, l2 = c.run(0)
    assert torch.equal(out.view(torch.int16), o2.view(torch.int16)) and torch.equal(lse, l2)


@pytest.mark.parametrize("layer,prefix,chunk,ps", CASES, ids=IDS)
@pytest.mark.parametrize("split", [None, "unpack"])
def test_multi_token_decode(layer, prefix, chunk, ps, split):
    c = ExtendCase4([layer], prefix, chunk, ps, seed=32, stored=True, split=split)
    out, lse = c.run(0)
    assert c.cache.device_error() == 0
    c.check(0, out, lse)


@pytest.mark.parametrize("split", ["tail", "unpack"])
def test_shared_layers_and_long_prefixes(split):
    layers = [lay(W.SLIDING, 256, 8, 2, 512), lay(W.FULL, 512, 8, 1), lay(W.SLIDING, 256, 16, 2, 512, W.KV_AUTO),
              lay(W.FULL, 512, 4, 1, 0, W.KV_AUTO)]
    c = ExtendCase4(layers, [1500, 700], [300, 513], 16, seed=33, split=split)
    assert c.src == [0, 1, 0, 1]
    for i in range(4):
        out, lse = c.run(i)
        c.check(i, out, lse, most=40)
    assert c.cache.device_error() == 0


def test_prefill_then_decode_as_a_server_runs_them():
    """Two prompts chunk by chunk: extend, then store the chunk; then one token by
    the fused decode.  The last chunk's first row and the decode agree with the
    reference over everything kept."""
    layers = [lay(W.SLIDING, 256, 8, 2, 100), lay(W.FULL, 512, 8, 1)]
    for i in range(2):
        d = layers[i]
        c = ExtendCase4([d], [0, 0], [150, 90], 16, seed=34)
        k, v = c.ext[0]
        out, lse = c.run(0)
        c.check(0, out, lse)
        slots = []
        bt = torch.arange(2 * 12, dtype=torch.int32).view(2, 12)
        cache = c.fa.Cache([d], 24, 16, c.fa.KV_FP4)
        cache.allocate("cuda")
        for b, n in enumerate((150, 90)):
            slots.append(W.slots_for_positions(bt[b].numpy(), np.arange(n), 16))
        cache.store(0, k, v, torch.from_numpy(np.concatenate(slots).astype(np.int32)).cuda())
        from fp4_case import DecodeCase4
        one = DecodeCase4([d], [151, 91], 16, seed=35)   # its own rows: replaced by the cache's below
        one.cache, one.bt[0] = cache, bt.cuda()
        one.slots[0] = torch.tensor([bt[0, 150 // 16] * 16 + 150 % 16, bt[1, 90 // 16] * 16 + 90 % 16],
                                    dtype=torch.int32, device="cuda")
        import oracle
        from paged_case import bits
        kept = [oracle.fp4_value(*oracle.quantize_fp4(bits(x))) for x in (k, v)]
        new = [oracle.fp4_value(*oracle.quantize_fp4(bits(x))) for x in one.new[0]]
        one.vals[0] = [[np.concatenate([x[a:a + n], y[b:b + 1]]) for x, y in zip(kept, new)]
                       for b, (a, n) in enumerate(((0, 150), (150, 90)))]
        out, lse = one.decode(0, fused=True)
        assert cache.device_error() == 0
        one.check(0, out, lse)


def test_value_scales_far_apart():
    def edit(i, kp, vp, kn, vn):
        vp[1] = 0.0                      # zero rows
        vp[5:30] = vp[5:30] * 2.0 ** -20
        vp[50:60] = vp[50:60] * 2.0 ** 20
    for d in (lay(W.FULL, 256, 8, 1), lay(W.FULL, 512, 8, 1)):
        c = ExtendCase4([d], [100, 64], [30, 10], 16, seed=36, edit=edit)
        out, lse = c.run(0)
        assert c.cache.device_error() == 0
        c.check(0, out, lse)


def test_unpacked_prefixes_over_many_calls_and_a_graph():
    """One workspace for two layers and several calls, the prefixes growing: the
    window's ring wraps, rows of earlier calls are left in it, and a captured call
    replays with new lengths."""
    layers = [lay(W.SLIDING, 256, 8, 2, 40), lay(W.FULL, 512, 16, 1)]
    ws = None
    for n, prefix in enumerate(([0, 0], [130, 33], [500, 90], [517, 480])):
        c = ExtendCase4(layers, prefix, [140, 70], 16, seed=40 + n)
        if ws is None:
            ws = torch.zeros(max(c.cache.extend_workspace_bytes(i, 2, 140, 600) for i in range(2)), dtype=torch.uint8, device="cuda")
        c.cache.bind_extend_workspace(ws)
        c.unpacked = True
        for i in (0, 1, 0):
            out, lse = c.run(i)
            c.check(i, out, lse, most=60)
        assert c.cache.device_error() == 0
    want = [c.run(i) for i in range(2)]
    outs = [c.outs(i) for i in range(2)]
    pre = c.prefix_dev.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for i in range(2):
            k, v = c.ext[i]
            c.cache.extend(i, c.q[i], k, v, c.indptr_dev, pre, c.bt, 140, 517, *outs[i])
    for cut in (0, 100):
        pre.copy_(c.prefix_dev - cut)
        g.replay()
        torch.cuda.synchronize()
        if cut == 0:
            for (o, l), (wo, wl) in zip(outs, want):
                assert torch.equal(o.view(torch.int16), wo.view(torch.int16)) and torch.equal(l, wl)
        else:
            vals = {i: [[np.concatenate([x[:int(P) - cut], x[int(P):]]) for x in c.vals[i][b]]
                        for b, P in enumerate(c.prefix)] for i in range(2)}
            keep, c.prefix, c.vals = (c.prefix, c.vals), c.prefix - cut, vals
            for i in range(2):
                c.check(i, *outs[i], most=60)
            c.prefix, c.vals = keep
    assert c.cache.device_error() == 0


def test_unpack_sizes_and_fallback():
    """fa_extend_unpack_bytes: K and V rows of the visible prefix and a table; a
    workspace too small for a call leaves it on the direct path."""
    import full_attention_gb300 as fa
    layers = [lay(W.SLIDING, 256, 8, 2, 100), lay(W.FULL, 512, 8, 1)]
    c = ExtendCase4(layers, [300, 20], [150, 20], 16, seed=50, split="unpack")
    full = c.cache.extend_workspace_bytes(1, 2, 150, 300) - fa.extend_workspace_bytes()
    assert full == 2 * (2 * 304 * 512 * 2) + 256
    n = c.cache.extend_workspace_bytes(0, 2, 150, 300) - fa.extend_workspace_bytes()
    assert n == 2 * (2 * 2 * 272 * 256 * 2) + 256      # 100 + 150 + 15 rows at most, 272 in the ring
    assert c.cache.extend_workspace_bytes(1, 2, 150, 0) == fa.extend_workspace_bytes()
    big = c.run(1)
    c.check(1, *big)
    for cut in (1, full):
        c.cache.bind_extend_workspace(c.ws[: fa.extend_workspace_bytes() + full - cut])
        c.check(1, *c.run(1))
    bt = c.bt.clone()
    bt[0, 1] = -1
    c.cache.bind_extend_workspace(c.ws)
    out, lse = c.outs(1)
    c.cache.extend(1, c.q[1], *c.ext[1], c.indptr_dev, c.prefix_dev, bt, 150, 300, out, lse)
    assert c.cache.device_error() == fa.DEV_ERR_PAGE


def test_refusals_and_reports():
    c = ExtendCase4([lay(W.FULL, 256, 8, 1)], [40, 20], [30, 10], 16, seed=37)
    fa, cache = c.fa, c.cache
    k, v = c.ext[0]
    out, lse = c.outs(0)
    args = lambda **m: {**dict(q=c.q[0], k_ext=k, v_ext=v, qo_indptr=c.indptr_dev, prefix_lens=c.prefix_dev,
                               block_table=c.bt, max_q_len=30, max_prefix_len=40, out=out, lse=lse), **m}
    for bad in (dict(q=c.q[0].float()), dict(q=c.q[0].transpose(0, 1)), dict(k_ext=k[:, :, ::2]), dict(v_ext=v.half()),
                dict(prefix_lens=c.prefix_dev.long()), dict(out=out[:5]), dict(lse=lse.half())):
        with pytest.raises(fa.FAError) as e:
            cache.extend(0, **args(**bad))
        assert e.value.status == fa.ERR_INVALID_ARG
    multi = lambda **m: cache.decode_multi(**{**dict(layer=0, q=c.q[0], qo_indptr=c.indptr_dev, seq_lens=c.prefix_dev,
                                                     block_table=c.bt, max_q_len=30, max_seq_len=40, out=out, lse=lse), **m})
    for bad in (dict(q=c.q[0].float()), dict(q=c.q[0].transpose(0, 1)), dict(seq_lens=c.prefix_dev.long()),
                dict(qo_indptr=c.indptr_dev[:2]), dict(block_table=c.bt[:1]), dict(out=out[:5]), dict(lse=lse.half())):
        with pytest.raises(fa.FAError) as e:
            multi(**bad)
        assert e.value.status == fa.ERR_INVALID_ARG
    bt = c.bt.clone()
    bt[0, 1] = cache.num_pages
    cache.extend(0, **args(block_table=bt))
    assert cache.device_error() == fa.DEV_ERR_PAGE
    q = c.q[0].clone()
    q[3, 1, 7] = 65536.0
    cache.extend(0, **args(q=q))
    assert cache.device_error() == fa.DEV_ERR_RANGE
