"""Step plans: the lengths after a step into another state, states that no step leaves, and
runs of more tokens than a warp takes at once."""
import random

import pytest
import torch

import workloads as W
from test_gpu_plan import FULL, Model, buffers, i32, make

pytestmark = pytest.mark.gpu


def test_lengths_follow_the_state_that_the_last_step_wrote():
    """seq_lens is what decode of the step reads: with state_out, too, the new tokens are in it."""
    import full_attention_gb300 as fa
    B, ps, N = 3, 16, 64
    cache = make(fa, FULL, 30, ps)
    table, model = cache.page_table(FULL, B, 8), Model(B, 30, ps, 8, 0)
    assert table.seq_lens.tolist() == [0] * B
    out, spare = buffers(B, N), torch.zeros_like(table.state)

    def step(new, **kw):
        model.step(new, N)
        table.step(i32(new), *out, **kw)
        assert cache.device_error() == 0 and table.seq_lens.tolist() == model.len

    step([5, 0, 20])
    step([1, 17, 1], state_out=spare)
    table.step(i32([1, 17, 1]), *out, state_out=spare)      # made again: the same lengths
    assert table.seq_lens.tolist() == model.len and table.state[4: 4 + B].tolist() == [5, 0, 20]
    table.state.copy_(spare)                                  # going on by a copy ...
    assert table.seq_lens.tolist() == model.len
    step([1, 1, -1])
    step([2, 1, 9], state_out=spare)
    table.state, spare = spare, table.state                   # ... or by taking the other buffer's place
    assert table.seq_lens.tolist() == model.len
    spare.zero_()
    step([1, 1, 1], state_out=spare)
    table.state.copy_(spare)
    step([1, 1, 1])
    assert table.state.tolist() == model.state()
    snapshot = table.state.clone()
    step([1, 0, 3])
    table.state = snapshot                                    # an earlier state put back
    assert table.seq_lens.tolist() == snapshot[4: 4 + B].tolist()


def test_a_decode_after_a_step_into_another_state_sees_the_new_token():
    """A captured step into another state and the decode behind it, fed by table.seq_lens."""
    import full_attention_gb300 as fa
    cache = fa.Cache([W.layer(FULL, 256, 2, 1)], 8, 16)
    for t in cache.allocate("cuda")[0][:2]:
        t.zero_()
    table = cache.page_table(FULL, 1, 4)
    out, spare = buffers(1, 1), torch.zeros_like(table.state)
    q = torch.zeros(1, 2, 256, dtype=torch.bfloat16, device="cuda")
    att, lse = torch.empty_like(q), torch.empty(1, 2, device="cuda")
    one, ws = i32([1]), fa.workspace(cache.decode_workspace_bytes(0, 1, 64))
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        table.step(one, *out, state_out=spare)
        cache.decode(0, q, table.block_table, table.seq_lens, 64, att, lse, ws)
    for n in range(1, 4):
        graph.replay()
        assert torch.allclose(lse, torch.full_like(lse, float(n)).log())   # n keys of score 0
        table.state.copy_(spare)
    assert cache.device_error() == 0


@pytest.mark.parametrize("N", [64, 30000])   # one CTA, and several
def test_the_states_words_of_0(N):
    """A state whose third or fourth word is not 0 is one that no step leaves."""
    import full_attention_gb300 as fa
    B, ps = 4, 16
    cache = make(fa, FULL, 2 * (N // ps + B), ps)
    table, model = cache.page_table(FULL, B, N // ps + 2), Model(B, cache.num_pages, ps, N // ps + 2, 0)
    out, spare = buffers(B, N), torch.zeros_like(table.state)
    new = [N // 4 - 1, 0, N // 2, 7]
    model.step(new, N)
    table.step(i32(new), *out)
    assert cache.device_error() == 0
    for into in (None, spare):
        for at, value in ((3, 1), (3, -5), (2, 1000), (2, -1000)):
            table.state[at] = value
            odd = table.state.clone()
            table.step(i32([1, 1, -1, 1]), *out, state_out=into)
            assert cache.device_error() == fa.DEV_ERR_WORKSPACE
            if at == 3 or into is not None or N == 64:   # else: CTAs count their arrivals there
                assert out[0].tolist() == [0] * (B + 1) and out[3].tolist() == [-1] * N
                assert table.free_pages.tolist() == model.ring and table.block_table.tolist() == model.table
                if at == 3 or into is not None:
                    assert torch.equal(table.state, odd)
            table.state.copy_(i32(model.state()))
            table.free_pages.copy_(i32(model.ring)), table.block_table.copy_(i32(model.table))
    want = model.step([1, 1, -1, 1], N)
    table.step(i32([1, 1, -1, 1]), *out)
    assert cache.device_error() == 0
    assert [t.tolist() for t in out] == list(want) and table.state.tolist() == model.state()


@pytest.mark.parametrize("window", [0, 1000])
def test_more_tokens_than_one_run_a_warp(window):
    """Enough tokens for every warp to take several runs of 128: long and short prompts,
    sequences without new tokens and ended ones in between, a prompt longer than a warp's
    share, and padding that begins inside a run; in place and into another state."""
    import full_attention_gb300 as fa
    B, ps, most, seed = 300, 64, 120_000, window
    r = random.Random(seed)
    kind = W.SLIDING if window else FULL
    cols = 2 * most // ps + 2
    cache = make(fa, kind, 60_000, ps, window)
    table, model = cache.page_table(kind, B, cols), Model(B, 60_000, ps, cols, window)
    spare = torch.zeros_like(table.state)
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    for step in range(3):
        new = [r.choice((0, 0, 1, 1, 3, 127, 128, 130, r.randint(1, 30_000), r.randint(1, 30_000)) + ((-1,) if step else ())) for _ in range(B)]
        new[40 + step] = most // 2 + step          # longer than a warp's share
        new[100: 180] = [1] * 40 + [0] * 40        # many short ones in a run, and none
        N = sum(max(n, 0) for n in new) + 250_001 + 13 * step
        assert N > 2 * 128 * 16 * sms
        want = model.step(new, N)
        into = spare if step == 1 else None
        out = buffers(B, N)
        table.step(i32(new), *out, state_out=into)
        assert cache.device_error() == 0 and want is not None
        for t, w in zip(out, want):
            assert t.tolist() == w
        assert table.free_pages.tolist() == model.ring and table.block_table.tolist() == model.table
        if into is not None:
            table.state.copy_(into)
        assert table.state.tolist() == model.state()
