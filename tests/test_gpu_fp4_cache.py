"""The fp4 slab written and read back, and fa_kv_load over every format, against the oracle.

The store is bit-exact; reading back is exact in bf16 and fp4 and one rounding
of an fp32 product in the 8-bit formats, which numpy repeats.
"""
import numpy as np
import pytest
import torch

import oracle
import workloads as W
from paged_case import bits
from test_fp4_format import rows as special_rows

pytestmark = pytest.mark.gpu

FORMATS = [W.KV_BF16, W.KV_INT8, W.KV_FP8, W.KV_FP4]
IDS = ["bf16", "int8", "fp8", "fp4"]


def _x(T, H, D, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((T, H, D), generator=g).to(torch.bfloat16)
    sp = torch.from_numpy(special_rows(seed, D).view(np.int16)).view(torch.bfloat16)
    n = min(T, len(sp))
    x[:n, seed % H] = sp[:n]
    if T > 20:
        x[14, 0, 3], x[15, 0, 4], x[16, 0, 5] = float("nan"), float("inf"), -float("inf")
        x[17, 0] = -0.0
    return x


def _cache(fa, D, H, ps, pool, kv):
    cache = fa.Cache([W.layer(W.FULL, D, 2 * H, H)], pool, ps, kv)
    return cache, cache.allocate("cuda")[0]


@pytest.mark.parametrize("D,H,ps,T", [(256, 1, 16, 40), (512, 1, 16, 40), (256, 8, 48, 61), (512, 2, 256, 1),
                                      (256, 3, 32, 517)])
def test_store_bit_for_bit(D, H, ps, T):
    import full_attention_gb300 as fa
    pool = -(-T // ps) + 3
    cache, (k_s, v_s, ks_s, vs_s) = _cache(fa, D, H, ps, pool, fa.KV_FP4)
    for t in (k_s, v_s):
        t.random_(0, 256)
    ks_s.fill_(0.25), vs_s.fill_(0.5)
    k, v = _x(T, H, D, 1), _x(T, H, D, 2)
    slots = np.random.default_rng(4).permutation(pool * ps)[:T].astype(np.int32)
    slots[T // 2:: 7] = -1
    want = [t.cpu().numpy().copy() for t in (k_s, v_s, ks_s, vs_s)]
    oracle.store_fp4(*want, bits(k), bits(v), slots, ps)
    cache.store(0, k.cuda(), v.cuda(), torch.from_numpy(slots).cuda())
    assert cache.device_error() == 0
    for got, w in zip((k_s, v_s, ks_s, vs_s), want):
        assert np.array_equal(got.cpu().numpy(), w)


@pytest.mark.parametrize("D", [256, 512])
def test_every_quotient_of_a_value_by_a_block_scale(D):
    """Each block scale with every bf16 magnitude from its largest code's value down to
    1/128 of that: the store decides each quotient, ties included, as the oracle."""
    import full_attention_gb300 as fa
    blocks = []
    for b in oracle.e4m3_value(np.arange(1, 0x7F, dtype=np.uint8)):
        top = 6.0 * b                                     # the block's largest magnitude: scale b exactly
        x = np.ldexp(np.arange(128, 256)[None], np.floor(np.log2(top)).astype(int) - np.arange(7)[:, None] - 7).ravel()
        x = x[x <= top] * np.where(np.arange((x <= top).sum()) % 3 == 1, -1.0, 1.0)
        x = np.concatenate([x, np.zeros(-len(x) % 15)]).reshape(-1, 15)
        blocks.append(np.concatenate([np.full((len(x), 1), top), x], axis=1))
    blocks = np.concatenate(blocks)
    per = D // 16 - 1                                     # and a block of 2688, so that the row scale is 1
    blocks = np.concatenate([blocks, np.zeros((-len(blocks) % per, 16))]).reshape(-1, per, 16)
    x = np.concatenate([np.full((len(blocks), 1, 16), 2688.0), blocks], axis=1).reshape(len(blocks), 1, D)
    k = torch.from_numpy(x).to(torch.bfloat16)
    assert np.array_equal(k.double().numpy(), x)
    pool = -(-len(x) // 16)
    cache, slab = _cache(fa, D, 1, 16, pool, fa.KV_FP4)
    want = [np.zeros(t.shape, t.cpu().numpy().dtype) for t in slab]
    for t in slab:
        t.zero_()
    slots = np.arange(len(x), dtype=np.int32)
    oracle.store_fp4(*want, bits(k), bits(-k), slots, 16)
    cache.store(0, k.cuda(), (-k).cuda(), torch.from_numpy(slots).cuda())
    assert cache.device_error() == 0
    for got, w in zip(slab, want):
        assert np.array_equal(got.cpu().numpy(), w)
    assert set(np.unique(want[0][..., D // 2:])) >= set(range(1, 0x7F)) and (want[2].ravel()[: len(x)] == 1).all()


def test_store_layers_and_slot_past_the_pool():
    import full_attention_gb300 as fa
    layers = [W.layer(W.SLIDING, 256, 8, 2, 64), W.layer(W.FULL, 512, 8, 1), W.layer(W.FULL, 512, 8, 1, 0, W.KV_AUTO)]
    ps, pool, T = 16, 4, 33
    cache = fa.Cache(layers, pool, ps, fa.KV_FP4)
    slabs = cache.allocate("cuda")
    slots = torch.arange(T, dtype=torch.int32)
    slots[7] = pool * ps
    slots[9] = -5
    ks, vs, want = [], [], {}
    for i, d in enumerate(layers):
        k, v = _x(T, d["num_kv_heads"], d["head_dim"], 5 + i), _x(T, d["num_kv_heads"], d["head_dim"], 9 + i)
        ks.append(k.cuda()), vs.append(v.cuda())
        if i in slabs:
            for t in slabs[i]:
                t.zero_()
            w = [t.cpu().numpy().copy() for t in slabs[i]]
            s = slots.numpy().copy()
            s[7] = -1
            oracle.store_fp4(*w, bits(k), bits(v), s, ps)
            want[i] = w
    sl = slots.cuda()
    cache.store_layers([0, 1, 2], ks, vs, [sl] * 3)
    assert cache.device_error() == fa.DEV_ERR_SLOT
    for i, w in want.items():
        for got, x in zip(slabs[i], w):
            assert np.array_equal(got.cpu().numpy(), x)


@pytest.mark.parametrize("kv", FORMATS, ids=IDS)
@pytest.mark.parametrize("D,H,ps,T", [(256, 1, 16, 1), (512, 2, 32, 77), (256, 8, 48, 300)])
def test_load_reads_rows_back(kv, D, H, ps, T):
    import full_attention_gb300 as fa
    pool = -(-T // ps) + 2
    cache, slab = _cache(fa, D, H, ps, pool, kv)
    k, v = _x(T, H, D, 1), _x(T, H, D, 2)
    k, v = torch.nan_to_num(k, 0, 1e30, -1e30), torch.nan_to_num(v, 0, 1e30, -1e30)
    slots = torch.from_numpy(np.random.default_rng(3).permutation(pool * ps)[:T].astype(np.int32))
    cache.store(0, k.cuda(), v.cuda(), slots.cuda())
    # read in another order, with repeats, padding and a slot past the pool
    pick = torch.from_numpy(np.random.default_rng(5).integers(0, T, 2 * T + 3))
    back = slots[pick].clone()
    back[1::5] = -1
    back[2] = pool * ps + 1
    ko = torch.full((len(pick), H, D), 7.0, dtype=torch.bfloat16, device="cuda")
    vo = ko.clone()
    cache.load(0, back.cuda(), ko, vo)
    assert cache.device_error() == fa.DEV_ERR_SLOT
    live = (back >= 0) & (back < pool * ps)
    for x, got in ((k, ko), (v, vo)):
        if kv == W.KV_BF16:
            want = bits(x)
        elif kv == W.KV_FP4:
            want = bits(torch.from_numpy(oracle.fp4_value(*oracle.quantize_fp4(bits(x)))).to(torch.bfloat16))
        else:
            q = oracle.quantize_fp8_per_token_head if kv == W.KV_FP8 else oracle.quantize_int8_per_token_head
            c, s = q(bits(x))
            c = oracle.e4m3_value(c) if kv == W.KV_FP8 else c
            want = bits(torch.from_numpy((c.astype(np.float32) * s[..., None]).astype(np.float32)).to(torch.bfloat16))
        want = want[pick.numpy()].copy()
        want[~live.numpy()] = bits(torch.tensor([7.0], dtype=torch.bfloat16))[0]
        assert np.array_equal(bits(got), want)
    one = torch.empty_like(ko)
    cache.load(0, back.cuda().clamp(0, pool * ps - 1), None, one)   # V alone
    ref = torch.empty_like(ko)
    cache.load(0, back.cuda().clamp(0, pool * ps - 1), ref, vo)
    assert torch.equal(one.view(torch.int16), vo.view(torch.int16))
    cache.load(0, back.cuda().clamp(0, pool * ps - 1), one, None)   # K alone
    assert torch.equal(one.view(torch.int16), ref.view(torch.int16))
    cache.load(0, back[:0].cuda(), ko[:0], vo[:0])                  # nothing to read


def test_load_through_a_shared_layer_in_a_graph_and_refusals():
    import full_attention_gb300 as fa
    layers = [W.layer(W.SLIDING, 256, 8, 2, 64), W.layer(W.SLIDING, 256, 8, 2, 64, W.KV_AUTO)]
    cache = fa.Cache(layers, 4, 16, fa.KV_FP4)
    cache.allocate("cuda")
    k, v = _x(20, 2, 256, 1).cuda(), _x(20, 2, 256, 2).cuda()
    slots = torch.arange(20, dtype=torch.int32, device="cuda")
    ko, vo = torch.empty_like(k), torch.empty_like(v)
    cache.store(0, k, v, slots)
    cache.load(1, slots, ko, vo)
    want = ko.clone()
    g = torch.cuda.CUDAGraph()
    k2 = k.clone()
    with torch.cuda.graph(g):
        cache.store(0, k2, v, slots)
        cache.load(0, slots, ko, vo)
    for scale in (1.0, 4.0, 0.5):   # powers of two scale every kept value (but the infinities' 2^127)
        k2.copy_(torch.nan_to_num(k, 0, 0, 0) * scale)
        g.replay()
        torch.cuda.synchronize()
        ref = oracle.fp4_value(*oracle.quantize_fp4(bits(k2)))
        assert np.array_equal(ko.double().cpu().numpy(), ref)
    assert want.shape == ko.shape
    for bad in (dict(k=k.float()), dict(k=k[:, :, ::2]), dict(k=k[:10]), dict(k=k.transpose(0, 1))):
        with pytest.raises(fa.FAError) as e:
            cache.load(0, slots, **bad)
        assert e.value.status == fa.ERR_INVALID_ARG
        with pytest.raises(fa.FAError) as e:
            cache.store(0, bad["k"], v, slots)
        assert e.value.status == fa.ERR_INVALID_ARG
    with pytest.raises(fa.FAError):
        cache.load(0, slots.long(), ko, vo)
    with pytest.raises(fa.FAError):
        cache.load(0, slots)                       # neither K nor V
    slab = cache.slab(0)
    with pytest.raises(fa.FAError):
        cache.bind(0, slab[0][:2], slab[1], slab[2], slab[3])
