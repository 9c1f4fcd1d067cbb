"""Block tables and slot maps built on the GPU (fa_plan_step) against a plain Python
page allocator: every array equal, over runs of steps in which sequences start, grow
and end, and in which a window's pages are given up."""
import random

import numpy as np
import pytest
import torch

import workloads as W

pytestmark = pytest.mark.gpu

FULL, SLIDING = W.FULL, W.SLIDING


class Model:
    """The same state with Python's lists."""

    def __init__(self, B, pages, ps, cols, window):
        self.ring, self.head, self.count = list(range(pages)), 0, pages
        self.len, self.first = [0] * B, [0] * B
        self.table = [[-1] * cols for _ in range(B)]
        self.ps, self.cols, self.window = ps, cols, window

    def step(self, new, N):
        """(offsets, prefixes, positions, slots); None: the step cannot be made."""
        ps, P = self.ps, len(self.ring)
        have = [-(-n // ps) for n in self.len]
        want = [h if n < 0 else -(-(l + n) // ps) for h, l, n in zip(have, self.len, new)]
        need = sum(w - h for w, h in zip(want, have))
        if need > self.count or any(w > self.cols for w in want) or sum(max(n, 0) for n in new) > N:
            return None
        at, gone = self.head + self.count, 0
        pushed = []
        for b, n in enumerate(new):
            keep = have[b] if n < 0 else max(self.first[b], max(0, self.len[b] - self.window + 1) // ps) if self.window else self.first[b]
            pushed += self.table[b][self.first[b]: keep]
            self.first[b] = 0 if n < 0 else keep
        popped = [self.ring[(self.head + i) % P] for i in range(need)]
        for i, page in enumerate(pushed):
            self.ring[(at + i) % P] = page
        self.head, self.count = (self.head + need) % P, self.count - need + len(pushed)
        ptr, prefix, pos, slots = [0], [], [], []
        for b, n in enumerate(new):
            prefix.append(0 if n < 0 else self.len[b])
            for j in range(have[b], want[b]):
                self.table[b][j] = popped.pop(0)
            for p in range(self.len[b], self.len[b] + max(n, 0)):
                pos.append(p)
                slots.append(self.table[b][p // ps] * ps + p % ps)
            self.len[b] = 0 if n < 0 else self.len[b] + n
            ptr.append(len(pos))
        return ptr, prefix, pos + [0] * (N - len(pos)), slots + [-1] * (N - len(slots))

    def state(self):
        return [self.head, self.count, 0, 0] + self.len + self.first


def make(fa, kind, pages, ps, window=0, pool=0):
    layers = [W.layer(FULL, 256, 2, 1)] + ([W.layer(SLIDING, 256, 2, 1, window), W.layer(SLIDING, 256, 2, 1, max(1, window // 2))] if window else [])
    cache = fa.Cache(layers, pages if not pool else pool, ps)
    if pool:
        cache.set_window_pool(pages)
    cache.bind(0, *[torch.zeros((pages if not pool else pool, 1, ps, 256), dtype=torch.bfloat16, device="cuda") for _ in range(2)])
    return cache


def buffers(B, N):
    return [torch.full((n,), 77, dtype=torch.int32, device="cuda") for n in (B + 1, B, N, N)]


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def check(table, out, model, want):
    assert table.cache.device_error() == 0
    for t, w in zip(out, want):
        assert t.tolist() == w
    same_state(table, model)


def same_state(table, model):
    assert table.state.tolist() == model.state()
    assert table.free_pages.tolist() == model.ring
    assert table.block_table.tolist() == model.table


@pytest.mark.parametrize("B,ps,window,pool,N,seed", [
    (1, 16, 0, 0, 40, 0), (1, 16, 1, 0, 33, 1), (5, 16, 0, 0, 200, 2), (5, 48, 100, 7, 203, 3), (64, 16, 70, 0, 1501, 4),
    (300, 32, 0, 0, 6000, 5), (257, 16, 16, 3, 9001, 6), (700, 256, 300, 0, 20011, 7),
])
def test_runs_of_steps(B, ps, window, pool, N, seed):
    import full_attention_gb300 as fa
    r = random.Random(seed)
    cols = 3 * N // (B * ps) + 4
    pages = B * min(cols, 2 * N // (B * ps) + 3)
    kind = SLIDING if window else FULL
    cache = make(fa, kind, pages, ps, window, pool)
    table, model = cache.page_table(kind, B, cols), Model(B, pages, ps, cols, window)
    most = max(1, min(2 * N // B, cols * ps // 3))
    made = 0
    for step in range(12):
        new = [r.choice((-1, 0, 1, 1, 1, r.randint(0, most))) for _ in range(B)]
        while sum(max(n, 0) for n in new) > N:
            new[r.randrange(B)] = -1
        out = buffers(B, N)
        before = [model.len[:], model.state()]
        want = model.step(new, N)
        table.step(i32(new), *out)
        if want is None:
            assert cache.device_error() in (fa.DEV_ERR_POOL, fa.DEV_ERR_BOUND, fa.DEV_ERR_POOL | fa.DEV_ERR_BOUND)
            want = ([0] * (B + 1), before[0], [0] * N, [-1] * N)
        else:
            made += 1
        check(table, out, model, want)
        assert table.seq_lens.tolist() == model.len
    assert made >= 6


@pytest.mark.parametrize("B,N", [(3, 100), (400, 30000)])
def test_a_step_into_another_state_can_be_made_again(B, N):
    import full_attention_gb300 as fa
    ps, r = 16, random.Random(B)
    cache = make(fa, SLIDING, 4 * B * (N // B // ps + 2), ps, 50)
    pages = cache.num_pages
    table, model = cache.page_table(SLIDING, B, 4 * (N // B // ps + 2)), Model(B, pages, ps, 4 * (N // B // ps + 2), 50)
    for new in ([r.randint(0, N // B) for _ in range(B)], [r.choice((-1, 0, 5, N // B)) for _ in range(B)]):
        first = table.state.clone()
        want = model.step(new, N)
        state_out = torch.zeros_like(table.state)
        for _ in range(3):
            out = buffers(B, N)
            table.step(i32(new), *out, state_out=state_out)
            assert torch.equal(table.state, first) and state_out.tolist() == model.state()
            assert [t.tolist() for t in out] == list(want)
            assert table.free_pages.tolist() == model.ring and table.block_table.tolist() == model.table
        table.state.copy_(state_out)


def test_refused_steps_change_nothing():
    import full_attention_gb300 as fa
    B, ps, pages, cols, N = 4, 16, 10, 6, 128
    cache = make(fa, FULL, pages, ps)
    table, model = cache.page_table(FULL, B, cols), Model(B, pages, ps, cols, 0)
    out = buffers(B, N)
    check_ok = model.step([20, 30, 0, 16], N)
    table.step(i32([20, 30, 0, 16]), *out)
    check(table, out, model, check_ok)
    for new, bits in (([13, 40, 32, 0], fa.DEV_ERR_POOL), ([0, 0, 0, 81], fa.DEV_ERR_BOUND), ([60, 30, 30, 9], fa.DEV_ERR_BOUND | fa.DEV_ERR_POOL),
                      ([2 ** 31 - 1] * 4, fa.DEV_ERR_BOUND), ([-1, 60, 60, 0], fa.DEV_ERR_POOL)):
        table.step(i32(new), *out)
        assert cache.device_error() & bits
        assert out[0].tolist() == [0] * (B + 1) and out[1].tolist() == model.len
        assert out[2].tolist() == [0] * N and out[3].tolist() == [-1] * N
        same_state(table, model)
    new = [12, 34, 16, -1]   # the pool's last page too
    want = model.step(new, N)
    table.step(i32(new), *out)
    check(table, out, model, want)
    for at, value in ((0, pages), (0, -1), (1, pages + 1), (1, -1), (4, -1), (5, cols * ps + 1), (4 + B, 7), (4 + B, -2), (1, pages)):
        keep = table.state.clone()
        table.state[at] = value
        odd = table.state.clone()
        table.step(i32([0, 0, 0, -1] if value != pages else [-1] * B), *out)
        assert cache.device_error() & fa.DEV_ERR_WORKSPACE
        assert torch.equal(table.state, odd) and out[3].tolist() == [-1] * N
        table.state.copy_(keep)


def test_bad_pages_are_reported():
    import full_attention_gb300 as fa
    B, ps, pages = 3, 16, 20
    cache = make(fa, FULL, pages, ps)
    table = cache.page_table(FULL, B, 4)
    table.free_pages[1], table.free_pages[2] = pages, -3
    out = buffers(B, 60)
    table.step(i32([16, 20, 10]), *out)
    assert cache.device_error() == fa.DEV_ERR_PAGE
    assert out[3].tolist() == list(range(16)) + [-1] * 20 + list(range(48, 58)) + [-1] * 14


def test_no_tokens_at_all():
    import full_attention_gb300 as fa
    cache = make(fa, FULL, 8, 16)
    table = cache.page_table(FULL, 2, 4)
    out = buffers(2, 4)
    table.step(i32([3, 0]), *out)
    none = torch.empty(0, dtype=torch.int32, device="cuda")
    table.step(i32([-1, 0]), out[0], out[1], none, none)
    assert cache.device_error() == 0
    assert out[0].tolist() == [0, 0, 0] and out[1].tolist() == [0, 0] and table.state.tolist() == [1, 8, 0, 0, 0, 0, 0, 0]


def test_the_largest_batch_and_captured_steps():
    """8192 sequences; replays of one captured step go on from each other."""
    import full_attention_gb300 as fa
    B, ps, N = fa.MAX_STEP_BATCH, 16, 3 * fa.MAX_STEP_BATCH + 5
    cache = make(fa, FULL, 2 * B, ps)
    table, model = cache.page_table(FULL, B, 2), Model(B, 2 * B, ps, 2, 0)
    new = [(-1, 0, 3, 1, 7, 1, 0)[b % 7] for b in range(B)]
    dev, out = i32(new), buffers(B, N)
    table.step(dev, *out)
    want = model.step(new, N)
    check(table, out, model, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        table.step(dev, *out)
    for _ in range(3):
        want = model.step(new, N)
        graph.replay()
        torch.cuda.synchronize()
        check(table, out, model, want)
