"""One decode workspace, zeroed once, behind calls of many sizes: every call's
bits against the same call on a workspace of its own."""
import pytest
import torch

import workloads as W

pytestmark = pytest.mark.gpu

FORMATS = [W.KV_BF16, W.KV_INT8, W.KV_FP8, W.KV_FP4]
IDS = ["bf16", "int8", "fp8", "fp4"]
TOKENS = 20_480
LAYERS = [W.layer(W.FULL, 512, 8, 1), W.layer(W.SLIDING, 256, 8, 1, 2000), W.layer(W.FULL, 512, 16, 1),
          W.layer(W.SLIDING, 256, 4, 2, 700), W.layer(W.FULL, 512, 4, 1)]


class Calls:
    """A cache whose sequences all read the first rows of one page list."""

    def __init__(self, kv_dtype):
        import full_attention_gb300 as fa
        self.fa = fa
        self.cache = fa.Cache(LAYERS, TOKENS // 16, 16, kv_dtype)
        self.cache.allocate("cuda")
        g = torch.Generator(device="cuda").manual_seed(7)
        slots = torch.arange(TOKENS, dtype=torch.int32, device="cuda")
        for i, d in enumerate(LAYERS):
            k, v = (torch.randn((TOKENS, d["num_kv_heads"], d["head_dim"]), generator=g, device="cuda").to(torch.bfloat16)
                    for _ in range(2))
            self.cache.store(i, k, v, slots)
        self.pages = torch.arange(TOKENS // 16, dtype=torch.int32, device="cuda")

    def args(self, i, B, bound):
        d = LAYERS[i]
        g = torch.Generator(device="cuda").manual_seed(B * 31 + bound + i)
        q = torch.randn((B, d["num_q_heads"], d["head_dim"]), generator=g, device="cuda").to(torch.bfloat16)
        lens = torch.tensor([max(1, bound - 13 * b % bound) for b in range(B)], dtype=torch.int32, device="cuda")
        bt = self.pages[None, : -(-bound // 16)].expand(B, -1).contiguous()
        return q, bt, lens, torch.full_like(q, float("nan")), torch.full(q.shape[:2], float("nan"), device="cuda")

    def one(self, i, B, bound, ws):
        q, bt, lens, out, lse = self.args(i, B, bound)
        self.cache.decode(i, q, bt, lens, bound, out, lse, ws)
        return out, lse

    def many(self, ids, B, bound, ws):
        a = [self.args(i, B, bound) for i in ids]
        self.cache.decode_layers(ids, [x[0] for x in a], [x[1] for x in a], a[0][2], bound, [x[3] for x in a],
                                 [x[4] for x in a], ws)
        return [t for x in a for t in x[3:]]

    def run(self, what, B, bound, ws=None):
        if isinstance(what, int):
            need = self.cache.decode_workspace_bytes(what, B, bound)
            return need, lambda w: self.one(what, B, bound, w)
        need = self.cache.decode_layers_workspace_bytes(what, B, bound)
        return need, lambda w: self.many(what, B, bound, w)


# layers of both kinds, bounds and batches that grow and shrink, several layers in one launch
SEQUENCE = [(0, 8, 1000), (0, 8, 4096), (1, 8, 4096), (0, 1, 20_000), (0, 1, 1000), (2, 8, 1000), (2, 70, 4096),
            ([0, 2, 4], 8, 4096), ([1, 3], 8, 1000), ([0, 4], 8, 20_000), (3, 33, 300), (0, 200, 300), ([2, 0], 70, 1000),
            (4, 1, 100), (0, 8, 20_000), (1, 130, 20_000), (0, 8, 1000), ([0, 2, 4], 1, 20_000), (2, 1, 20_000)]


@pytest.mark.parametrize("kv_dtype", FORMATS, ids=IDS)
def test_one_workspace_serves_calls_of_every_size(kv_dtype):
    c = Calls(kv_dtype)
    calls = [c.run(*s) for s in SEQUENCE]
    shared = c.fa.workspace(max(n for n, _ in calls))
    for s, (n, call) in zip(SEQUENCE + SEQUENCE, calls + calls):
        want = call(c.fa.workspace(n))
        assert c.cache.device_error() == 0
        got = call(shared)
        assert c.cache.device_error() == 0, s
        for g, w in zip(got, want):
            assert torch.isfinite(w).all() and torch.equal(g, w), s


def test_one_workspace_serves_caches_of_every_format():
    caches = [Calls(kv) for kv in FORMATS]
    shared = caches[0].fa.workspace(max(c.run(*s)[0] for s in SEQUENCE for c in caches))
    for s in SEQUENCE:
        for c in caches:
            n, call = c.run(*s)
            want = call(c.fa.workspace(n))
            got = call(shared)
            assert c.cache.device_error() == 0, s
            for g, w in zip(got, want):
                assert torch.equal(g, w), s


@pytest.mark.parametrize("word", [3, -7], ids=["positive", "negative"])
@pytest.mark.parametrize("kv_dtype", FORMATS, ids=IDS)
def test_a_workspace_that_was_not_zeroed_is_reported(kv_dtype, word):
    """Counters that did not start at zero: reported whatever they hold, and a
    workspace zeroed again serves the next call."""
    c = Calls(kv_dtype)
    n, call = c.run(0, 1, 20_000)
    want = call(c.fa.workspace(n))
    ws = c.fa.workspace(n)
    ws[: 1024].view(torch.int32).fill_(word * 1000)
    call(ws)
    assert c.cache.device_error() == c.fa.DEV_ERR_WORKSPACE
    ws.zero_()
    for g, w in zip(call(ws), want):
        assert torch.equal(g, w)
    assert c.cache.device_error() == 0


@pytest.mark.parametrize("kv_dtype", FORMATS, ids=IDS)
def test_captured_graphs_of_different_sizes_share_a_workspace(kv_dtype):
    c = Calls(kv_dtype)
    steps = [(0, 8, 4096), ([0, 2, 4], 8, 1000), (1, 70, 4096), (0, 1, 20_000)]
    calls = [c.run(*s) for s in steps]
    want = [call(c.fa.workspace(n)) for n, call in calls]
    ws = c.fa.workspace(max(n for n, _ in calls))
    graphs = []
    for what, B, bound in steps:
        ids = [what] if isinstance(what, int) else what
        a = [c.args(i, B, bound) for i in ids]
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            if isinstance(what, int):
                c.cache.decode(what, *a[0][:3], bound, *a[0][3:], ws)
            else:
                c.cache.decode_layers(ids, [x[0] for x in a], [x[1] for x in a], a[0][2], bound, [x[3] for x in a],
                                      [x[4] for x in a], ws)
        graphs.append((g, [t for x in a for t in x[3:]], a))
    for i in (0, 1, 2, 3, 0, 3, 1, 2, 0):
        g, outs, _ = graphs[i]
        for t in outs:
            t.fill_(float("nan"))
        g.replay()
        for got, w in zip(outs, want[i]):
            assert torch.equal(got, w), (i, steps[i])
    assert c.cache.device_error() == 0
