"""Seeded differential-attention cases and their 64-bit results.

Slab rows that no query may see hold NaN (bf16 values; in the 8-bit formats the
scales, and e4m3's NaN code), and table entries of pages wholly outside a window -1.

Bounds.  With A_m = sum_j p_mj |v_j| of map m and lambda l, an output is off by at most
  2^-8 |out|                         its own rounding to bf16
  (2^-7 + 2^-12) (A_1 + |l| A_2)     the weights in bf16 (half a step each; the sum that
                                     divides them has the same rounded weights) and fp32 scores
  n 2^-24 max|v| (1 + |l|)           8-bit: weights that are f16 subnormals, n keys
and lse by 2^-13: fp32 scores of magnitude up to 30 (2^-20 relative), the hardware's 2^x and log2.
"""
from __future__ import annotations

import math

import numpy as np
import torch

import workloads as W

NAN = float("nan")


def kept(x, kv):
    """Codes, scales and 64-bit values of bf16 rows x [..., D] in a slab format (scales None in bf16)."""
    if kv == W.KV_BF16:
        return x, None, x.double()
    top = 127.0 if kv == W.KV_INT8 else 448.0
    a = x.float().abs().amax(-1)
    s = a / torch.full_like(a, top)   # (by a Python number, torch multiplies by its reciprocal)
    y = torch.where(s[..., None] > 0, x.float() / s[..., None], 0.0).clamp(-top, top)
    c = y.round().to(torch.int8) if kv == W.KV_INT8 else y.to(torch.float8_e4m3fn)
    return (c if kv == W.KV_INT8 else c.view(torch.uint8)), s, c.double() * s.double()[..., None]


class DiffCase:
    def __init__(self, D, hq, hkv, ps, lens, kv=W.KV_BF16, window=0, new=None, seed=0, shared=False, lam=None, scale=1.0,
                 early=False, offset=0.0):
        import full_attention_gb300 as fa
        self.fa, self.D, self.hq, self.hkv, self.ps, self.kv, self.window = fa, D, hq, hkv, ps, kv, window
        self.lens, self.new, self.B = list(lens), new, len(lens)
        g = torch.Generator().manual_seed(seed)
        sm = float(np.float32(1 / math.sqrt(D // 2)))
        lay = dict(kind=W.SLIDING if window else W.FULL, head_dim=D, num_q_heads=hq, num_kv_heads=hkv, window=window,
                   kv_source=W.KV_OWN, sm_scale=sm)
        self.layer = 1 if shared else 0
        self.sm = sm
        stored = [max(0, n) for n in lens]
        N = self.B if new is None else sum(new)
        self.q = (torch.randn(N, hq, D, generator=g) * scale).bfloat16().cuda()
        self.lam = (torch.randn(hq, generator=g) if lam is None else torch.as_tensor(lam).expand(hq).clone()).float().cuda()
        if new is not None:
            self.k_ext, self.v_ext = ((torch.randn(N, hkv, D, generator=g) + o).bfloat16().cuda() for o in (0.0, offset))
        # rows of every stored position that some query sees, at a random permutation of pages
        need = [-(-n // ps) for n in stored]
        first = [max(0, (n - window if new is None else n - window + 1)) // ps if window else 0 for n in stored]
        pool = sum(need) + 3
        ids = torch.randperm(pool, generator=g).tolist()
        self.bt = torch.full((self.B, max(1, max(need))), -1, dtype=torch.int32)
        self.cache = fa.Cache([lay, dict(lay, kv_source=W.KV_AUTO)] if shared else [lay], pool, ps, kv)
        if early:
            self.cache.set_flags(fa.FLAG_EARLY_METADATA)
        slabs = self.cache.allocate("cuda")[0]
        self.slabs = slabs
        for t in slabs:
            if t is not None:
                t.fill_(NAN if t.is_floating_point() else 0x7F)
        self.rows = []   # per sequence: (first seen position, k, v [n][hkv][D] in 64 bits)
        self.raw = []
        for b, n in enumerate(stored):
            for j in range(first[b], need[b]):
                self.bt[b, j] = ids.pop()
            lo = max(0, (n - window if new is None else n - window + 1)) if window else 0
            x = [(torch.randn(n - lo, hkv, D, generator=g) + o).bfloat16().cuda() for o in (0.0, offset)]
            self.raw.append((lo, x))
            pos = torch.arange(lo, n)
            page, off = self.bt[b][pos // ps].long().cuda(), (pos % ps).cuda()
            vals = []
            for i in range(2):
                c, s, v = kept(x[i], kv)
                slabs[i][page, :, off] = c
                if s is not None:
                    slabs[2 + i][page, :, off] = s
                vals.append(v)
            self.rows.append((lo, *vals))
        self.bt = self.bt.cuda()
        self.lens_dev = torch.tensor(self.lens, dtype=torch.int32, device="cuda")
        self.out = torch.full((N, hq, D), NAN, dtype=torch.bfloat16, device="cuda")
        self.lse = torch.full((N, hq, 2), NAN, device="cuda")
        if new is not None:
            self.indptr = torch.tensor(np.concatenate([[0], np.cumsum(new)]), dtype=torch.int32, device="cuda")

    def max_len(self):
        return max(1, max(self.lens))

    def decode(self, ws=None, **kw):
        if ws is None:
            ws = self.fa.workspace(self.cache.decode_diff_workspace_bytes(self.layer, self.B, self.max_len()))
        self.cache.decode_diff(self.layer, self.q, self.lam, self.bt, self.lens_dev, self.max_len(), self.out, self.lse, ws, **kw)
        return self.out, self.lse

    def extend(self):
        self.cache.extend_diff(self.layer, self.q, self.lam, self.k_ext, self.v_ext, self.indptr, self.lens_dev, self.bt,
                               max(self.new), max(self.lens), self.out, self.lse)
        return self.out, self.lse

    def reference(self):
        """out, lse and the bound on out, all 64-bit."""
        q, lam, W_ = self.q.double(), self.lam.double(), self.window
        out, lse, room = torch.zeros_like(q), torch.full(q.shape[:2] + (2,), -math.inf, dtype=torch.float64, device="cuda"), torch.zeros_like(q)
        g, at, half = self.hq // self.hkv, 0, self.D // 2
        for b, n in enumerate(self.lens):
            r = 1 if self.new is None else self.new[b]
            if (self.new is None and n <= 0) or r == 0:
                at += r
                continue
            lo, k, v = self.rows[b]
            if self.new is not None:
                k, v = torch.cat((k, self.k_ext[at: at + r].double())), torch.cat((v, self.v_ext[at: at + r].double()))
            kpos = lo + torch.arange(len(k), device="cuda")
            qpos = (n - 1 if self.new is None else n) + torch.arange(r, device="cuda")[:, None]
            seen = (kpos <= qpos) & ((qpos - kpos < W_) if W_ else True)
            for j in range(self.hq):
                h = j // g
                for m, sign in ((0, 1.0), (1, -lam[j])):
                    c = slice(m * half, (m + 1) * half)
                    s = torch.where(seen, (q[at: at + r, j, c] @ k[:, h, c].T) * self.sm, -math.inf)
                    p = torch.softmax(s, -1)
                    lse[at: at + r, j, m] = torch.logsumexp(s, -1)
                    out[at: at + r, j] += sign * (p @ v[:, h])
                    room[at: at + r, j] += abs(sign) * ((2.0 ** -7 + 2.0 ** -12) * (p @ v[:, h].abs())
                                                        + (len(k) * 2.0 ** -24 * v[:, h].abs().max() if self.kv != W.KV_BF16 else 0.0))
            at += r
        return out, lse, room + 2.0 ** -8 * out.abs()

    def check(self, out, lse=None):
        ref, ref_lse, room = self.reference()
        err = (out.double() - ref).abs()
        assert bool((err <= room).all()), f"out: {float((err / room.clamp(min=1e-30)).max()):.3f} of the bound"
        if lse is not None:
            same = torch.isinf(ref_lse)
            assert torch.equal(torch.isinf(lse), same) and bool(((lse.double() - ref_lse).abs()[~same] <= 2.0 ** -13).all()), \
                f"lse off by {float((lse.double() - ref_lse)[~same].abs().max()):.2e}"
        assert self.cache.device_error() == 0
