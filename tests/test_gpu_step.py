"""Serving steps as a program makes them, with nothing but the numbers of new tokens from
the host: the step's plan, each layer's rows normed, rotated and stored, and differential
attention over what the steps before stored, while sequences start, grow and end.  A full layer and
a sliding one with a pool of its own, whose plan gives pages up as its window moves.

The reference keeps each sequence's raw rows: the rows out are held to the 64-bit formula
(test_gpu_norm_rope.py), and attention, in 64 bits over those rows, to diff_case.py's bounds."""
import math

import numpy as np
import pytest
import torch

import workloads as W
from diff_case import kept
from test_gpu_norm_rope import formula, freqs, near

pytestmark = pytest.mark.gpu

PS, WINDOW = 16, 70


class Layer:
    def __init__(self, fa, cache, i, d, g, B):
        D = d["head_dim"]
        self.cache, self.i, self.d, self.D = cache, i, d, D
        self.qw, self.kw = (torch.randn(D, generator=g).bfloat16().cuda() for _ in range(2))
        self.how = fa.NormRope(D, freqs(D), self.qw, self.kw, eps=1e-6, norm_v=True)
        self.lam = torch.rand(d["num_q_heads"], generator=g).cuda()
        self.rows = [[] for _ in range(B)]   # per sequence: (k, v) rows as they came out, a step's at a time


def attention(layer, q, rows, P, kv):
    """out, lse and the bound of one sequence's new rows q at positions P .. over its rows; the
    new tokens' own rows unquantised where new > 1 (extend), all as kept otherwise."""
    d, D = layer.d, layer.D
    n = q.shape[0]
    k = torch.cat([r[0] for r in rows])
    v = torch.cat([r[1] for r in rows])
    kd, vd = kept(k, kv)[2], kept(v, kv)[2]
    if layer.extend:
        kd[P:], vd[P:] = k[P:].double(), v[P:].double()
    kpos = torch.arange(P + n, device="cuda")
    qpos = P + torch.arange(n, device="cuda")[:, None]
    seen = kpos <= qpos
    if d["window"]:
        seen &= qpos - kpos < d["window"]
    g, half = d["num_q_heads"] // d["num_kv_heads"], D // 2
    out = torch.zeros(n, d["num_q_heads"], D, dtype=torch.float64, device="cuda")
    room = torch.zeros_like(out)
    lam = layer.lam.double()
    for j in range(d["num_q_heads"]):
        h = j // g
        for m, w in ((0, 1.0), (1, -lam[j])):
            c = slice(m * half, (m + 1) * half)
            s = torch.where(seen, (q[:, j, c].double() @ kd[:, h, c].T) * d["sm_scale"], -math.inf)
            p = torch.softmax(s, -1)
            out[:, j] += w * (p @ vd[:, h])
            room[:, j] += abs(w) * ((2.0 ** -7 + 2.0 ** -12) * (p @ vd[:, h].abs()) + (P + n) * 2.0 ** -24 * float(vd.abs().max()))
    return out, room + 2.0 ** -8 * out.abs()


@pytest.mark.parametrize("kv", [W.KV_BF16, W.KV_INT8, W.KV_FP8])
@pytest.mark.parametrize("early", [False, True])
def test_steps_of_a_changing_batch(kv, early):
    import full_attention_gb300 as fa
    B, N = 6, 256
    sm = {D: float(np.float32(1 / math.sqrt(D // 2))) for D in (256, 512)}
    layers = [dict(W.layer(W.FULL, 512, 8, 2), sm_scale=sm[512]), dict(W.layer(W.SLIDING, 256, 4, 1, WINDOW), sm_scale=sm[256])]
    cache = fa.Cache(layers, 90, PS, kv)
    cache.set_window_pool(60)
    slabs = cache.allocate("cuda")
    for s in slabs.values():
        for t in s:
            if t is not None:
                t.fill_(float("nan") if t.is_floating_point() else 0x7F)
    if early:
        cache.set_flags(fa.FLAG_EARLY_METADATA)
    g = torch.Generator().manual_seed(kv + 10 * early)
    ls = [Layer(fa, cache, i, d, g, B) for i, d in enumerate(layers)]
    tables = [cache.page_table(W.FULL, B, 24), cache.page_table(W.SLIDING, B, 24)]
    i32 = lambda *n: torch.full(n, 7, dtype=torch.int32, device="cuda")  # noqa: E731
    plans = [(i32(B + 1), i32(B), i32(N), i32(N)) for _ in tables]
    ws = fa.workspace(max(cache.decode_diff_workspace_bytes(i, B, 24 * PS) for i in range(2)))
    lens = [0] * B
    steps = [[100, 0, 30, 1, 0, 5], [1] * B, [1, 90, 1, 1, 0, 1], [1, 1, 1, 1, 1, 1], [-1, 1, 60, 1, 1, -1], [120, 1, 1, 1, 1, 33]] + [[1] * B] * 3 + [[-1] * B, [20, 0, 0, 0, 0, 17]]
    for new in steps:
        for t, pl in zip(tables, plans):
            t.step(torch.tensor(new, dtype=torch.int32, device="cuda"), *pl)
        decode = all(n == 1 for n in new)
        for layer, t, (indptr, prefix, pos, slots) in zip(ls, tables, plans):
            d, D = layer.d, layer.D
            hq, hkv = d["num_q_heads"], d["num_kv_heads"]
            rows = B if decode else N          # the buffers of a step are padded
            x = torch.randn(rows, (hq + 2 * hkv) * D, generator=g).bfloat16().cuda()
            q, k, v = x[:, : hq * D], x[:, hq * D: (hq + hkv) * D], x[:, (hq + hkv) * D:]
            qo, ko, vo = (torch.empty(rows, h, D, dtype=torch.bfloat16, device="cuda") for h in (hq, hkv, hkv))
            cache.norm_rope_store(layer.i, layer.how, q, k, v, pos[:rows], slots[:rows], qo, ko, vo)
            out = torch.full((rows, hq, D), 5.0, dtype=torch.bfloat16, device="cuda")
            if decode:
                cache.decode_diff(layer.i, qo, layer.lam, t.block_table, t.seq_lens, max(lens) + 1, out, None, ws)
            else:
                cache.extend_diff(layer.i, qo, layer.lam, ko, vo, indptr, prefix, t.block_table, max(new + [0]), max(lens + [1]), out)
            assert cache.device_error() == 0
            at = 0
            layer.extend = not decode
            for b, n in enumerate(new):
                if n < 0:
                    layer.rows[b] = []
                    continue
                P = lens[b]
                where = torch.arange(P, P + n)
                cut = slice(at, at + n)
                if n:
                    assert pos[cut].tolist() == where.tolist()
                    near(qo[cut], *formula(q[cut].view(n, hq, D), True, layer.qw, 0, 1e-6, freqs(D), where))
                    near(ko[cut], *formula(k[cut].reshape(n, hkv, D), True, layer.kw, 0, 1e-6, freqs(D), where))
                    near(vo[cut], *formula(v[cut].reshape(n, hkv, D), True, None, 0, 1e-6, [], where))
                    layer.rows[b].append((ko[cut].clone(), vo[cut].clone()))
                    ref, room = attention(layer, qo[cut], layer.rows[b], P, kv)
                    assert bool(((out[cut].double() - ref).abs() <= room).all()), (new, b, layer.i)
                at += n
            if not decode:
                assert bool((out[at:] == 5.0).all())   # rows behind the last sequence
        lens = [0 if n < 0 else a + n for a, n in zip(lens, new)]
        assert all(t.seq_lens.tolist() == lens for t in tables)
    assert int(tables[0].state[1]) == 90 - sum(-(-n // PS) for n in lens)   # every page is free or held


def test_a_captured_decode_step_goes_on_by_itself():
    """Plan, rows and attention in one graph: each replay is the next token."""
    import full_attention_gb300 as fa
    B, D, hq, hkv = 3, 256, 4, 1
    lay = dict(W.layer(W.FULL, D, hq, hkv), sm_scale=float(np.float32(1 / math.sqrt(D // 2))))

    def make():
        cache = fa.Cache([lay], 30, PS)
        for t in cache.allocate("cuda")[0][:2]:
            t.zero_()
        return cache, cache.page_table(W.FULL, B, 8)

    g = torch.Generator().manual_seed(1)
    how = fa.NormRope(D, freqs(D))
    lam = torch.tensor([0.3, 0.8, 0.0, -1.0]).cuda()
    x = torch.randn(9, B, (hq + 2 * hkv) * D, generator=g).bfloat16().cuda()
    runs = []
    for captured in (False, True):
        cache, table = make()
        ws = fa.workspace(cache.decode_diff_workspace_bytes(0, B, 8 * PS))
        ones = torch.ones(B, dtype=torch.int32, device="cuda")
        pl = [torch.zeros(n, dtype=torch.int32, device="cuda") for n in (B + 1, B, B, B)]
        inp, q, out = torch.empty_like(x[0]), torch.empty(B, hq, D, dtype=torch.bfloat16, device="cuda"), torch.empty(B, hq, D, dtype=torch.bfloat16, device="cuda")

        def step():
            table.step(ones, *pl)
            cache.norm_rope_store(0, how, inp[:, : hq * D], inp[:, hq * D: (hq + hkv) * D], inp[:, (hq + hkv) * D:], pl[2], pl[3], q)
            cache.decode_diff(0, q, lam, table.block_table, table.seq_lens, 8 * PS, out, None, ws)

        graph = None
        if captured:
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                step()
        outs = []
        for i in range(len(x)):
            inp.copy_(x[i])
            graph.replay() if captured else step()
            torch.cuda.synchronize()
            outs.append(out.clone())
        assert cache.device_error() == 0 and table.seq_lens.tolist() == [len(x)] * B
        runs.append(outs)
    assert all(torch.equal(a, b) for a, b in zip(*runs))
