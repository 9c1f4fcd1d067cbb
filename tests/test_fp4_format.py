"""The fp4 slab format without a GPU: the oracle's quantiser against exact
rationals, worked examples and planted mistakes; the library's sizes and
refusals."""
import ctypes
from fractions import Fraction as F

import numpy as np
import pytest
import torch

import oracle
from oracle import FULL, KV_AUTO, KV_FP4, SLIDING

E2M1 = [F(0), F(1, 2), F(1), F(3, 2), F(2), F(3), F(4), F(6)]
E4M3 = [F(m, 8) * F(1, 64) if e == 0 else (1 + F(m, 8)) * F(2) ** (e - 7) for e in range(16) for m in range(8)][:127]


def bits(x):
    return torch.as_tensor(x, dtype=torch.float64).to(torch.bfloat16).view(torch.int16).numpy().view(np.uint16)


def exact_row(x_bits):
    """The format's definition in rationals, for one row of finite bf16 values."""
    x = [F(float(v)) for v in oracle.bf16_to_f64(x_bits)]
    a, e = max(map(abs, x)), -116
    while a > 2688 * F(2) ** e:
        e += 1
    s = F(2) ** e

    def near(grid, v):   # ties to the even index
        return min(range(len(grid)), key=lambda i: (abs(grid[i] - v), i % 2))

    codes, scales = [], []
    for i in range(0, len(x), 16):
        sb = near(E4M3, max(map(abs, x[i:i + 16])) / (6 * s))
        scales.append(sb)
        for v in x[i:i + 16]:
            codes.append(near(E2M1, abs(v) / (s * E4M3[sb])) if sb else 0)
    return codes, scales, s


def rows(seed=0, D=256):
    r = np.random.default_rng(seed)
    out = [r.standard_normal(D), r.standard_normal(D) * 2.0 ** r.integers(-30, 8, D), np.zeros(D),
           np.full(D, 2688.0), np.full(D, -2704.0), r.choice([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0], D) * 7,
           r.standard_normal(D) * 2.0 ** -118, r.standard_normal(D) * 2.0 ** -130, r.standard_normal(D) * 2.0 ** 124,
           r.choice([-1.0, 1.0], D) * 2.0 ** r.integers(-133, 127, D)]
    blockwise = r.standard_normal(D) * np.repeat(2.0 ** r.integers(-14, 6, D // 16), 16)
    ties = np.repeat(r.integers(1, 16, D // 16) * 2.0, 16) * r.choice([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0], D)
    for i in range(0, D, 16):
        ties[i] = ties[i:i + 16].max() if i else 448 * 6.0
    return bits(np.stack(out + [blockwise, ties]))


@pytest.mark.parametrize("D", [256, 512])
def test_oracle_matches_exact_rationals(D):
    x = rows(3, D)
    got, scale = oracle.quantize_fp4(x)
    for i in range(len(x)):
        codes, scales, s = exact_row(x[i])
        b = got[i, : D // 2]
        c = np.stack([b & 15, b >> 4], -1).reshape(-1)
        assert F(float(scale[i])) == s
        assert (c & 7).tolist() == codes and got[i, D // 2:].tolist() == scales
        assert ((c >> 3) == (np.signbit(oracle.bf16_to_f64(x[i])) & (c != 0))).all()
        want = [(-1 if n else 1) * E2M1[k] * E4M3[scales[j // 16]] * s for j, (k, n) in enumerate(zip(codes, c >> 3))]
        assert [F(float(v)) for v in oracle.fp4_value(got[i:i + 1], scale[i:i + 1])[0]] == want


def test_values_fit_bf16_exactly():
    """Every value a row can hold has 6 significant bits at most and lies in bf16's normal range or is 0."""
    x = rows(5)
    v = oracle.fp4_value(*oracle.quantize_fp4(x))
    assert (torch.from_numpy(v).to(torch.bfloat16).double().numpy() == v).all()
    big = bits(np.full(256, 3.3e38))
    v = oracle.fp4_value(*oracle.quantize_fp4(big[None]))
    assert np.isfinite(torch.from_numpy(v).to(torch.bfloat16).double().numpy()).all()


def test_worked_example():
    """Largest magnitude 6: e = -8 (6 <= 2688 / 256 = 10.5 and 6 > 5.25), block scale 256 for its block."""
    x = np.zeros(256)
    x[:4] = [6.0, -3.0, 0.25, -0.75]      # 0.25 and 0.75 tie: to codes 0 and 2 (value 1)
    x[16:18] = [0.75, 0.125]               # its own block scale: 0.75 / 6 * 256 = 32
    rows_, s = oracle.quantize_fp4(bits(x)[None])
    assert s[0] == 2.0 ** -8
    assert rows_[0, :2].tolist() == [0x7 | (0x5 | 8) << 4, 0x0 | (0x2 | 8) << 4]
    assert oracle.e4m3_value(rows_[0, 128:130]).tolist() == [256.0, 32.0]
    assert rows_[0, 8] == (7 | 2 << 4)     # 0.75 -> 6, 0.125 / (32 / 256) = 1 -> code 2
    assert not rows_[0, 130:].any()


def test_special_values():
    x = bits(np.zeros((3, 256)))
    x[0, 5] = 0x7FC0                       # NaN
    x[0, 6] = bits([2.0])[0]
    x[1, 7] = 0xFF80                       # -inf
    v = oracle.fp4_value(*oracle.quantize_fp4(x))
    # 2 / (6 * 2^-10) = 341.3, whose nearest e4m3 value is 352: 6 * 352 * 2^-10 = 2.0625
    assert v[0, 5] == 0 and v[0, 6] == 2.0625 and v[1, 7] < -2.0 ** 126 and (v[2] == 0).all()
    assert (oracle.quantize_fp4(x)[1] == np.float32([2.0 ** -10, 2.0 ** 116, 2.0 ** -116])).all()


@pytest.mark.parametrize("mistake", ["ties away", "scale by 7", "block of 32", "e off by one"])
def test_planted_mistakes_are_seen(monkeypatch, mistake):
    good = oracle.quantize_fp4(rows(3))
    if mistake == "ties away":
        monkeypatch.setattr(oracle, "_nearest_even",
                            lambda g, a: np.searchsorted((g[1:] + g[:-1]) / 2, np.minimum(a, g[-1]), side="right"))
    elif mistake == "scale by 7":
        monkeypatch.setattr(oracle, "E2M1_MAGS", np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 7.0]))
    elif mistake == "block of 32":
        x = rows(3)
        b = oracle.quantize_fp4(np.sort(x, axis=-1))
        assert not np.array_equal(b[0], good[0])
        return
    else:
        keep = np.frexp
        monkeypatch.setattr(np, "frexp", lambda a: (keep(a)[0], keep(a)[1] + 1))
    bad = oracle.quantize_fp4(rows(3))
    assert not np.array_equal(bad[0], good[0]) or not np.array_equal(bad[1], good[1])


# ------------------------------------------------------------------ the library
@pytest.fixture(scope="module")
def fa():
    import __graft_entry__
    __graft_entry__.build()
    import full_attention_gb300 as fa
    return fa


def lay(kind, D, hq, hkv, W=0, src=oracle.KV_OWN):
    return dict(kind=kind, head_dim=D, num_q_heads=hq, num_kv_heads=hkv, window=W, kv_source=src, sm_scale=0.0625)


def test_sizes(fa):
    layers = [lay(SLIDING, 256, 8, 2, 64), lay(FULL, 512, 8, 1), lay(SLIDING, 256, 8, 2, 64, KV_AUTO)]
    c = fa.Cache(layers, 100, 32, fa.KV_FP4)
    assert c.slab_bytes(0) == (100 * 2 * 32 * 144, 100 * 2 * 32 * 4)
    assert c.slab_bytes(1) == (100 * 32 * 288, 100 * 32 * 4) and c.slab_bytes(2) == (0, 0)
    for kind in (FULL, SLIDING):
        assert c.bytes_per_token(kind) == oracle.kv_bytes_per_token(layers, kind, KV_FP4)
    assert c.bytes_per_token(FULL) == 2 * (256 + 32 + 4)
    with pytest.raises(fa.FAError) as e:
        fa.Cache(layers, 100, 32, 4)
    assert e.value.status == fa.ERR_UNSUPPORTED


def test_decode_workspace_grows_with_the_call(fa):
    """A workspace sized for the largest call serves every smaller one."""
    for D, hq, hkv in ((512, 8, 1), (256, 8, 2), (512, 13, 1), (256, 32, 8)):
        c = fa.Cache([lay(FULL, D, hq, hkv), lay(SLIDING, D, hq, hkv, 300)], 8, 16, fa.KV_FP4)
        for layer in (0, 1):
            lens = [1, 16, 100, 129, 200, 300, 333, 400, 600, 1000, 2000, 5000, 100_000]
            n = [[c.decode_workspace_bytes(layer, B, L) for L in lens] for B in (1, 2, 3, 7, 19, 50, 51, 75, 100, 150, 152, 153, 200, 456, 500)]
            for row in n:
                assert row == sorted(row), (D, hq, layer, row)
            for col in zip(*n):
                assert list(col) == sorted(col), (D, hq, layer, col)


def test_load_refusals(fa):
    """fa_kv_load checks its arguments on the host, before any launch."""
    lib = fa.lib()
    buf = np.zeros(4096, np.uint8)
    p = (buf.ctypes.data + 255) // 256 * 256
    for dt in (fa.KV_BF16, fa.KV_INT8, fa.KV_FP8, fa.KV_FP4):
        c = fa.Cache([lay(SLIDING, 256, 8, 1, 64), lay(SLIDING, 256, 8, 1, 64, KV_AUTO)], 8, 16, dt)
        assert lib.fa_kv_load(None, 0, p, 1, p, p, None) == fa.ERR_INVALID_ARG
        assert lib.fa_kv_load(c._h, 2, p, 1, p, p, None) == fa.ERR_INVALID_ARG
        assert lib.fa_kv_load(c._h, 0, p, -1, p, p, None) == fa.ERR_INVALID_ARG
        assert lib.fa_kv_load(c._h, 0, None, 0, None, None, None) == fa.OK
        for layer in (0, 1):   # a shared layer reads its source's slab, which is not bound either
            assert lib.fa_kv_load(c._h, layer, p, 1, p, p, None) == fa.ERR_NOT_BOUND
        for k in (torch.zeros(2, 1, 256), torch.zeros(2, 1, 256, dtype=torch.bfloat16)):   # type; not on a GPU
            with pytest.raises(fa.FAError) as e:
                c.load(0, torch.zeros(2, dtype=torch.int32), k, k)
            assert e.value.status == fa.ERR_INVALID_ARG
        with pytest.raises(fa.FAError) as e:
            c.load(5, torch.zeros(2, dtype=torch.int32))
        assert e.value.status == fa.ERR_INVALID_ARG


def test_bind_needs_scales_and_refuses_shared(fa):
    c = fa.Cache([lay(SLIDING, 256, 8, 1, 64), lay(SLIDING, 256, 8, 1, 64, KV_AUTO)], 8, 16, fa.KV_FP4)
    lib = fa.lib()
    buf = np.zeros(4096, np.uint8)
    p = (buf.ctypes.data + 255) // 256 * 256
    assert lib.fa_cache_bind_slab(c._h, 0, p, p, None, None) == fa.ERR_INVALID_ARG
    assert lib.fa_cache_bind_slab(c._h, 0, p + 8, p, p, p) == fa.ERR_INVALID_ARG
    assert lib.fa_cache_bind_slab(c._h, 1, p, p, p, p) == fa.ERR_INVALID_ARG
