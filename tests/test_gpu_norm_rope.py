"""Norms, rotation and store in one launch (fa_norm_rope_store) against 64-bit rows.

Bound on a value z with its partner (normed values y, y'): half a bf16 step, 2^-8 |z|, plus the fp32
arithmetic's 2^-18 (|y| + |y'|): the sum of 512 squares and its root at most 2^-19.8
relative, the hardware's sine and cosine 2^-21.2 and their angle 2^-21.5 absolute, a
few roundings of 2^-24.
"""
import math

import numpy as np
import pytest
import torch

import workloads as W

pytestmark = pytest.mark.gpu

FORMATS = [W.KV_BF16, W.KV_INT8, W.KV_FP8, W.KV_FP4]


def make(fa, D, hq, hkv, kv=W.KV_BF16, ps=16, pool=12, layers=None):
    cache = fa.Cache(layers or [W.layer(W.FULL, D, hq, hkv)], pool, ps, kv)
    slabs = cache.allocate("cuda")
    for t in slabs[0]:
        if t is not None:
            t.copy_(torch.ones_like(t))
    return cache, slabs[0]


def inputs(T, hq, hkv, D, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(T, hq + 2 * hkv, D, generator=g) * torch.exp(torch.randn(T, hq + 2 * hkv, 1, generator=g)) * scale
    pos = torch.randint(-5, 1 << 20, (T,), generator=g)
    pos[0] = 2 ** 31 - 1
    if T > 1:
        pos[1] = -2 ** 31
    w = torch.randn(2, D, generator=g)
    return x.bfloat16().cuda(), pos.int().cuda(), w[0].bfloat16().cuda(), w[1].bfloat16().cuda()


def freqs(R, base=1e4):
    return (base ** (-np.arange(R // 2, dtype=np.float64) / max(1, R // 2))).tolist()


def turns(pos, f):
    """cos and sin of position * frequency, the product reduced in integers."""
    import full_attention_gb300 as fa
    ph = np.array([[(int(p) * s) % (1 << 64) for s in fa.rope_steps(f)] for p in pos], dtype=np.float64).reshape(len(pos), len(f))
    a = torch.from_numpy(ph * (2 * math.pi / 2.0 ** 64))
    return torch.cos(a)[:, None], torch.sin(a)[:, None]


def formula(x, norm, w, offset, eps, f, pos):
    """Rows z [T][H][D] in 64 bits, and the bound's |y| + |y'|."""
    y = x.double().cpu()
    if norm:
        y = y / torch.sqrt((y * y).mean(-1, keepdim=True) + eps)
        if w is not None:
            y = y * (w.double().cpu() + offset)
    size = y.abs()
    if f:
        h = len(f)
        c, s = turns(pos.tolist(), f)
        a, b = y[..., :h], y[..., h: 2 * h]
        y = torch.cat((a * c - b * s, b * c + a * s, y[..., 2 * h:]), -1)
        both = size[..., :h] + size[..., h: 2 * h]
        size = torch.cat((both, both, size[..., 2 * h:]), -1)
    return y, size


def near(got, z, size):
    err = (got.double().cpu() - z).abs()
    room = 2.0 ** -8 * z.abs() + 2.0 ** -18 * size
    assert bool((err <= room).all()), f"{float((err / room.clamp(min=1e-300)).max()):.3f} of the bound"


CASES = [  # D, hq, hkv, T, R, page
    (256, 4, 1, 1, 256, 16), (512, 4, 1, 1, 512, 16), (256, 7, 1, 3, 256, 48), (512, 6, 2, 5, 256, 32),
    (256, 16, 8, 700, 256, 16), (512, 16, 2, 900, 512, 64), (512, 8, 8, 700, 16, 16), (256, 24, 3, 501, 240, 16),
    (512, 5, 5, 1203, 496, 16), (256, 8, 2, 1500, 0, 16), (512, 33, 1, 400, 480, 16),
]


@pytest.mark.parametrize("kv", FORMATS)
@pytest.mark.parametrize("D,hq,hkv,T,R,ps", CASES)
def test_rows_and_slab(D, hq, hkv, T, R, ps, kv):
    import full_attention_gb300 as fa
    pool = -(-T // ps) + 2
    x, pos, qw, kw = inputs(T, hq, hkv, D, T + R + kv)
    offset, norm_v = float(T % 2), bool(hq % 2)
    how = fa.NormRope(D, freqs(R) if R else None, qw, kw, eps=1e-6, weight_offset=offset, norm_v=norm_v)
    slots = np.random.default_rng(T).permutation(pool * ps)[:T].astype(np.int32)
    slots[T // 2:: 7] = -1
    slots = torch.from_numpy(slots).cuda()
    outs = [torch.full((T, h, D), 9.0, dtype=torch.bfloat16, device="cuda") for h in (hq, hkv, hkv)]
    cache, slab = make(fa, D, hq, hkv, kv, ps, pool)
    q, k, v = x[:, :hq], x[:, hq: hq + hkv], x[:, hq + hkv:]       # strided: one projection's rows
    cache.norm_rope_store(0, how, q, k, v, pos, slots, *outs)
    assert cache.device_error() == 0
    f = freqs(R) if R else []
    near(outs[0], *formula(q, True, qw, offset, 1e-6, f, pos))
    near(outs[1], *formula(k, True, kw, offset, 1e-6, f, pos))
    if norm_v:
        near(outs[2], *formula(v, True, None, 0, 1e-6, [], pos))
    else:
        assert torch.equal(outs[2], v)
    # the slab holds what the store of those rows writes, bit for bit, and nothing else
    other, want = make(fa, D, hq, hkv, kv, ps, pool)
    other.store(0, outs[1], outs[2], slots)
    for a, b in zip(slab, want):
        assert a is None or torch.equal(a, b)
    # the same from dense inputs, in their own place and without rows out
    cache2, slab2 = make(fa, D, hq, hkv, kv, ps, pool)
    qd, kd, vd = q.contiguous(), k.contiguous(), v.contiguous()
    cache2.norm_rope_store(0, how, qd, kd, vd, pos, slots, qd)
    assert torch.equal(qd, outs[0])
    for a, b in zip(slab2, want):
        assert a is None or torch.equal(a, b)
    cache2.norm_rope_store(0, how, None, kd, vd, pos, None, None, kd, vd)
    assert torch.equal(kd, outs[1]) and torch.equal(vd, outs[2])


@pytest.mark.parametrize("D", [256, 512])
@pytest.mark.parametrize("norm", [0, 1, 2, 4, 7])
def test_each_norm_alone(D, norm):
    import full_attention_gb300 as fa
    T, hq, hkv = 37, 5, 1
    x, pos, qw, kw = inputs(T, hq, hkv, D, norm)
    how = fa.NormRope(D, freqs(D), qw, None, eps=0.5, norm_q=norm & 1, norm_k=norm & 2, norm_v=norm & 4)
    cache, _ = make(fa, D, hq, hkv)
    outs = [torch.empty((T, h, D), dtype=torch.bfloat16, device="cuda") for h in (hq, hkv, hkv)]
    q, k, v = x[:, :hq], x[:, hq: hq + hkv], x[:, hq + hkv:]
    cache.norm_rope_store(0, how, q, k, v, pos, None, *outs)
    near(outs[0], *formula(q, norm & 1, qw, 0, 0.5, freqs(D), pos))
    near(outs[1], *formula(k, norm & 2, None, 0, 0.5, freqs(D), pos))
    near(outs[2], *formula(v, norm & 4, None, 0, 0.5, [], pos))


@pytest.mark.parametrize("D,R", [(256, 256), (512, 512), (512, 32)])
def test_a_step_of_zero_and_position_zero_leave_pairs_as_they_are(D, R):
    import full_attention_gb300 as fa
    T, hq, hkv = 3000, 4, 1
    x, pos, _, _ = inputs(T, hq, hkv, D, 5)
    pos[5:100] = 0
    f = freqs(R)
    f[3] = f[R // 2 - 1] = 0.0
    how = fa.NormRope(D, f, norm_q=False, norm_k=False)
    cache, _ = make(fa, D, hq, hkv)
    q = torch.empty((T, hq, D), dtype=torch.bfloat16, device="cuda")
    cache.norm_rope_store(0, how, x[:, :hq], None, None, pos, None, q)
    for i in (3, R // 2 - 1):
        assert torch.equal(q[..., i], x[:, :hq, i]) and torch.equal(q[..., i + R // 2], x[:, :hq, i + R // 2])
    assert torch.equal(q[5:100], x[5:100, :hq]) and torch.equal(q[..., R:], x[:, :hq, R:])


@pytest.mark.parametrize("D", [256, 512])
@pytest.mark.parametrize("scale", [1e-30, 1e-12, 1e18, 3e35])
def test_magnitudes_far_from_one(D, scale):
    """Squares past fp32's range, and below it beside eps."""
    import full_attention_gb300 as fa
    T, hq, hkv = 50, 3, 1
    x, pos, qw, kw = inputs(T, hq, hkv, D, 8, scale)
    x[4] = 0.0
    how = fa.NormRope(D, freqs(D), qw, kw, eps=1e-24)
    cache, _ = make(fa, D, hq, hkv)
    q = torch.empty((T, hq, D), dtype=torch.bfloat16, device="cuda")
    cache.norm_rope_store(0, how, x[:, :hq], None, None, pos, None, q)
    near(q, *formula(x[:, :hq], True, qw, 0, 1e-24, freqs(D), pos))


def test_infinities_and_nan_stay_in_their_rows():
    import full_attention_gb300 as fa
    D, T, hq, hkv = 256, 9, 2, 1
    x, pos, qw, kw = inputs(T, hq, hkv, D, 3)
    x[2, 0, 5], x[3, 1, 130], x[4, 0, 7] = float("inf"), -float("inf"), float("nan")
    how = fa.NormRope(D, freqs(D), qw, kw)
    cache, _ = make(fa, D, hq, hkv)
    q = torch.empty((T, hq, D), dtype=torch.bfloat16, device="cuda")
    cache.norm_rope_store(0, how, x[:, :hq], None, None, pos, None, q)
    z, _ = formula(x[:, :hq], True, qw, 0, 1e-6, freqs(D), pos)
    assert torch.equal(torch.isnan(q).cpu(), torch.isnan(z))
    bad = torch.isnan(q).any(-1)
    assert bad.nonzero().tolist() == [[2, 0], [3, 1], [4, 0]]
    assert bool((q[2, 0][~torch.isnan(q[2, 0])] == 0).all())


@pytest.mark.parametrize("D,R", [(256, 64), (512, 64), (512, 320)])
def test_infinities_outside_the_turned_columns(D, R):
    """Without a norm, a column past R goes on as it is, beside turned ones."""
    import full_attention_gb300 as fa
    T, hq, hkv = 40, 2, 1
    x, pos, _, _ = inputs(T, hq, hkv, D, 4)
    x[3, 0, R], x[5, 1, D - 1], x[9, 1, R + 3] = float("inf"), -float("inf"), float("nan")
    how = fa.NormRope(D, freqs(R), norm_q=False, norm_k=False)
    cache, _ = make(fa, D, hq, hkv)
    q = torch.empty((T, hq, D), dtype=torch.bfloat16, device="cuda")
    cache.norm_rope_store(0, how, x[:, :hq], None, None, pos, None, q)
    assert torch.equal(torch.nan_to_num(q[..., R:], nan=7.0), torch.nan_to_num(x[:, :hq, R:], nan=7.0))
    assert bool(torch.isfinite(q[..., :R]).all())


def test_a_shared_layer_takes_its_queries_alone():
    import full_attention_gb300 as fa
    D, T, hq, hkv = 512, 20, 8, 2
    layers = [W.layer(W.FULL, D, hq, hkv), W.layer(W.FULL, D, hq, hkv, kv_source=W.KV_AUTO)]
    cache, slab = make(fa, D, hq, hkv, layers=layers)
    before = [t.clone() for t in slab if t is not None]
    x, pos, qw, kw = inputs(T, hq, hkv, D, 2)
    how = fa.NormRope(D, freqs(D), qw, kw)
    q = torch.empty((T, hq, D), dtype=torch.bfloat16, device="cuda")
    rows = torch.full((T, hkv, D), 3.0, dtype=torch.bfloat16, device="cuda")
    cache.norm_rope_store(1, how, x[:, :hq], x[:, hq: hq + hkv], x[:, hq + hkv:], pos, torch.arange(T, dtype=torch.int32, device="cuda"),
                          q, rows, rows)
    near(q, *formula(x[:, :hq], True, qw, 0, 1e-6, freqs(D), pos))
    assert bool((rows == 3).all()) and all(torch.equal(a, b) for a, b in zip(before, [t for t in slab if t is not None]))


@pytest.mark.parametrize("kv", FORMATS)
def test_slots_past_the_pool_are_reported(kv):
    import full_attention_gb300 as fa
    D, T, hq, hkv = 256, 4, 2, 2
    cache, slab = make(fa, D, hq, hkv, kv, 16, 3)
    x, pos, qw, kw = inputs(T, hq, hkv, D, 6)
    slots = torch.tensor([48, 5, 2 ** 31 - 1, -7], dtype=torch.int32, device="cuda")
    k, v = (torch.empty((T, hkv, D), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    q = torch.empty((T, hq, D), dtype=torch.bfloat16, device="cuda")
    cache.norm_rope_store(0, fa.NormRope(D, freqs(D)), x[:, :hq], x[:, hq: hq + hkv], x[:, hq + hkv:], pos, slots, q, k, v)
    assert cache.device_error() == fa.DEV_ERR_SLOT
    other, want = make(fa, D, hq, hkv, kv, 16, 3)
    other.store(0, k[1:2], v[1:2], slots[1:2])
    for a, b in zip(slab, want):
        assert a is None or torch.equal(a, b)


def test_captured_and_on_another_stream():
    import full_attention_gb300 as fa
    D, T, hq, hkv = 512, 300, 8, 1
    x, pos, qw, kw = inputs(T, hq, hkv, D, 12)
    how = fa.NormRope(D, freqs(D), qw, kw)
    cache, slab = make(fa, D, hq, hkv, W.KV_INT8, 16, 20)
    slots = torch.arange(T, dtype=torch.int32, device="cuda")
    q = torch.empty((T, hq, D), dtype=torch.bfloat16, device="cuda")
    args = (0, how, x[:, :hq], x[:, hq: hq + hkv], x[:, hq + hkv:], pos, slots, q)
    cache.norm_rope_store(*args)
    torch.cuda.synchronize()
    want = [q.clone()] + [t.clone() for t in slab]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cache.norm_rope_store(*args)
    x2 = x.clone()
    x.mul_(2.0)
    graph.replay()
    torch.cuda.synchronize()
    assert not torch.equal(slab[2], want[3])
    x.copy_(x2)
    graph.replay()
    s = torch.cuda.Stream()
    q.zero_()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        cache.norm_rope_store(*args)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip([q] + list(slab), want))
