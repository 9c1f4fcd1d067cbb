"""Extend and multi-token decode over fp4 slabs read only pages that some query sees."""
import pytest
import torch

import workloads as W
from fp4_case import ExtendCase4

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("stored", [False, True], ids=["extend", "multi-token decode"])
@pytest.mark.parametrize("layer", [W.layer(W.FULL, 512, 8, 1), W.layer(W.SLIDING, 256, 8, 2, 300)], ids=["full", "sliding"])
def test_a_sequence_without_new_tokens_reads_no_pages(layer, stored):
    """No query sees its rows, so its block table may hold anything, with a
    workspace for unpacked rows as without."""
    for split in (None, "unpack"):
        c = ExtendCase4([layer], [700, 900, 640], [40, 0, 25], 16, seed=61, stored=stored, split=split)
        c.bt[1] = -1
        out, lse = c.run(0)
        assert c.cache.device_error() == 0, split
        c.check(0, out, lse)


def test_a_window_of_one_reads_no_prefix_pages():
    layer = W.layer(W.SLIDING, 512, 8, 2, 1)
    for split in (None, "unpack"):
        c = ExtendCase4([layer], [700, 37, 640], [40, 3, 25], 16, seed=62, split=split)
        c.bt.fill_(-1)
        out, lse = c.run(0)
        assert c.cache.device_error() == 0, split
        c.check(0, out, lse)


def test_padded_buffers_as_kept_for_a_captured_graph():
    """Tables, lengths and outputs with rows to spare: the rows past the batch stay as they are."""
    from fp4_case import DecodeCase4
    case = DecodeCase4([W.layer(W.FULL, 512, 8, 1)], [300, 40, 0, 1000], 16, seed=63)
    case.store_current()
    want = case.decode(0)
    pad = lambda t, fill: torch.cat([t, torch.full((3, *t.shape[1:]), fill, dtype=t.dtype, device="cuda")])
    out, lse = (torch.full((7, *t.shape[1:]), 9.0, dtype=t.dtype, device="cuda") for t in want)
    case.cache.decode(0, case.q[0], pad(case.bt[0], 1 << 30), pad(case.lens_dev, 1 << 30), case.max_len, out, lse, case.workspace(0))
    assert case.cache.device_error() == 0
    for got, w in zip((out, lse), want):
        assert torch.equal(got[:4], w) and (got[4:] == 9.0).all()


@pytest.mark.parametrize("kv_dtype", [W.KV_BF16, W.KV_INT8, W.KV_FP8, W.KV_FP4], ids=["bf16", "int8", "fp8", "fp4"])
def test_tables_too_narrow_for_the_largest_bounds_are_refused(kv_dtype):
    """Refused on the host, before any launch."""
    import full_attention_gb300 as fa
    cache = fa.Cache([W.layer(W.FULL, 256, 8, 1)], 8, 16, kv_dtype)
    cache.allocate("cuda")
    q, kv = torch.zeros((2, 8, 256), dtype=torch.bfloat16, device="cuda"), torch.zeros((2, 1, 256), dtype=torch.bfloat16, device="cuda")
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")
    bt = torch.zeros((2, 4), dtype=torch.int32, device="cuda")
    for bound in (65, 2**31 - 20, 2**31 - 1):
        for call in (lambda: cache.extend(0, q, kv, kv, i32(0, 1, 2), i32(3, 3), bt, 1, bound, torch.empty_like(q)),
                     lambda: cache.decode_multi(0, q, i32(0, 1, 2), i32(3, 3), bt, 1, bound, torch.empty_like(q)),
                     lambda: cache.decode(0, q, bt, i32(3, 3), bound, torch.empty_like(q))):
            with pytest.raises(fa.FAError) as e:
                call()
            assert e.value.status == fa.ERR_INVALID_ARG, bound


def test_a_length_below_its_new_tokens_under_the_widest_window():
    """Reported; what the call still computes is the same with and without unpacked rows."""
    layer = W.layer(W.SLIDING, 512, 8, 1, 2**31 - 1)
    outs = []
    for split in (None, "unpack"):
        c = ExtendCase4([layer], [700, 300], [40, 6], 16, seed=64, stored=True, split=split)
        c.check(0, *c.run(0))
        c.lens_dev[1] = 1
        out, lse = c.run(0)
        assert c.cache.device_error() == c.fa.DEV_ERR_BOUND
        outs.append(out)
    assert torch.equal(outs[0][40], outs[1][40])   # one key: its value, exact on both paths


@pytest.mark.parametrize("stored", [False, True], ids=["extend", "multi-token decode"])
def test_unpacking_more_rows_than_one_sweep_of_its_blocks(stored):
    """256 sequences over one page list, prefixes up to 3000 rows, a bound past that:
    each block of the unpacking kernel takes several stretches of rows."""
    import full_attention_gb300 as fa
    B, T, D, hq = 256, 3000, 512, 8
    layer = W.layer(W.FULL, D, hq, 1)
    cache = fa.Cache([layer], 200, 16, fa.KV_FP4)
    cache.allocate("cuda")
    g = torch.Generator(device="cuda").manual_seed(5)
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda").to(torch.bfloat16)
    slots = torch.arange(T, dtype=torch.int32, device="cuda")
    cache.store(0, rnd(T, 1, D), rnd(T, 1, D), slots)
    K, V = rnd(T, 1, D), rnd(T, 1, D)
    cache.load(0, slots, K, V)
    K, V = K[:, 0].double(), V[:, 0].double()
    lens = (torch.arange(B, device="cuda") * 97 % (T - 1) + 1).int()
    q, kx, vx = rnd(B, hq, D), rnd(B, 1, D), rnd(B, 1, D)
    bt = torch.arange(200, dtype=torch.int32, device="cuda").expand(B, -1).contiguous()
    ptr = torch.arange(B + 1, dtype=torch.int32, device="cuda")
    bound = 3200
    ws = fa.workspace(cache.extend_workspace_bytes(0, B, 1, bound))
    ws.fill_(255)
    cache.bind_extend_workspace(ws)
    out = torch.empty_like(q)
    if stored:
        cache.decode_multi(0, q, ptr, lens, bt, 1, bound, out)
    else:
        cache.extend(0, q, kx, vx, ptr, lens, bt, 1, bound, out)
    assert cache.device_error() == 0
    s = layer["sm_scale"] * q.double() @ K.T
    s = torch.where(torch.arange(T, device="cuda") < lens[:, None, None], s, -torch.inf)
    if not stored:
        s = torch.cat([s, layer["sm_scale"] * (q.double() * kx.double()).sum(-1, keepdim=True)], -1)
    p = torch.softmax(s, -1)
    ref, mag = p[..., :T] @ V, p[..., :T] @ V.abs()
    if not stored:
        ref, mag = ref + p[..., T:] * vx.double(), mag + p[..., T:] * vx.double().abs()
    assert ((out.double() - ref).abs() <= 2.0 ** -7 * ref.abs() + 1.5 * 2.0 ** -8 * mag).all()
