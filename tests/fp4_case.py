"""Seeded fp4 cache cases and their plain reference in float64.

Every slot that no query may see holds junk: random codes, NaN block scales and
NaN row scales.  The reference gathers the stored rows' values (from the oracle's
quantiser) and computes softmax attention in float64, along with the bounds an
output may be off by:

  out: a rounding to bf16 (2^-8 of the value), one rounding of every weight to
  f16 and one of its product with a power of two (2^-11 each), and the fp32
  score sums, at most D * 2^-24 * sum|q k| (512 * 2^-24 * 64 = 2^-9 for sums up to
  64, which also bounds the weights' relative error): together 2^-8 |out| +
  2^-8 * sum_j p_j |v_j|;
  lse: the score error, 2^-9, and a few fp32 roundings of its own size, 2^-20 |lse|.

Where a workspace for unpacked rows is bound, extend may run the bf16 kernel: its
weights p (1 + d) are rounded to bf16, |d| <= 2^-8, and divided by the sum of the
rounded ones, which moves the output by at most sum_j p_j |d_j| |v_j - out| <=
2^-8 (sum_j p_j |v_j| + |out|); with the output's own rounding and the score
error, 2^-7 |out| + (2^-8 + 2^-9) sum_j p_j |v_j|.
"""
import numpy as np
import torch

import oracle
import workloads as W
from paged_case import bits


def rows_like_a_model(T, H, D, seed):
    """Normal rows, some channels six times larger, token norms spread."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((T, H, D), generator=g)
    x = x * torch.where(torch.randn((H, D), generator=g) > 1.9, 6.0, 1.0)
    return (x * torch.exp(0.3 * torch.randn((T, 1, 1), generator=g))).to(torch.bfloat16)


def junk(slab, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    k, v, ks, vs = slab
    for t in (k, v):
        t.random_(0, 256, generator=g)
        D = t.shape[-1] * 16 // 9
        t[..., D // 2::2] = 0x7F       # NaN block scales
    ks.fill_(float("nan")), vs.fill_(float("nan"))


def attend(q, K, V, sm):
    """out, lse, bound on |out error| of one query row (float64 numpy)."""
    s = sm * (K @ q)
    m = np.max(s)
    p = np.exp(s - m)
    l = p.sum()
    p = p / l
    out = p @ V
    return out, m + np.log(l), 2.0 ** -8 * np.abs(out) + 2.0 ** -8 * (p @ np.abs(V)) + 1e-30


class DecodeCase4:
    """Sequences of stored rows, the last of each (the current token) kept apart."""

    def __init__(self, layers, lens, page_size=16, seed=0, edit=None, window_pool=False, pool_extra=0):
        import full_attention_gb300 as fa
        self.fa, self.layers, self.ps = fa, layers, page_size
        self.lens = np.asarray(lens, np.int32)
        self.B = len(lens)
        self.max_len = max(1, int(self.lens.max()))
        self.plans = {}
        pages = 1
        for i, d in enumerate(layers):
            win = d["window"] if d["kind"] == W.SLIDING else 0
            self.plans[i] = W.plan_pages(self.lens, page_size, seed + (0 if win == 0 else 1000), window=win,
                                         max_pages=-(-self.max_len // page_size))
            pages = max(pages, self.plans[i].num_pages)
        self.cache = fa.Cache(layers, pages + pool_extra, page_size, fa.KV_FP4)
        if window_pool:
            self.cache.set_window_pool(max(self.plans[i].num_pages for i, d in enumerate(layers) if d["kind"] == W.SLIDING))
        self.src = [self.cache.source(i) for i in range(len(layers))]
        for i, s in enumerate(self.src):
            self.plans[i] = self.plans[s]   # a shared layer's table is its source's
        self.slabs = self.cache.allocate("cuda")
        self.bt = {i: torch.from_numpy(p.block_table).cuda() for i, p in self.plans.items()}
        self.lens_dev = torch.from_numpy(self.lens).cuda()
        self.q, self.new, self.vals, self.slots = {}, {}, {}, {}
        for i, d in enumerate(layers):
            g = torch.Generator().manual_seed(seed * 77 + i)
            self.q[i] = torch.randn((self.B, d["num_q_heads"], d["head_dim"]), generator=g).to(torch.bfloat16).cuda()
            if self.src[i] != i:
                continue
            junk(self.slabs[i], seed + i)
            H, D = d["num_kv_heads"], d["head_dim"]
            pos = [np.arange(max(0, int(L) - d["window"]) if d["kind"] == W.SLIDING else 0, int(L)) for L in self.lens]
            T = sum(map(len, pos))
            kv = [rows_like_a_model(T, H, D, seed * 31 + 2 * i + s) for s in (0, 1)]
            if edit is not None:
                edit(i, *kv)
            slots = np.concatenate([W.slots_for_positions(self.plans[i].block_table[b], p, page_size)
                                    for b, p in enumerate(pos)]).astype(np.int32)
            last = np.array([np.cumsum([len(p) for p in pos])[b] - 1 for b in range(self.B) if self.lens[b] > 0], int)
            rest = np.setdiff1d(np.arange(T), last)
            if len(rest):
                self.cache.store(i, kv[0][rest].cuda(), kv[1][rest].cuda(), torch.from_numpy(slots[rest]).cuda())
            # the current rows, one per sequence (empty sequences: padding)
            new = [torch.zeros((self.B, H, D), dtype=torch.bfloat16) for _ in range(2)]
            sl = np.full(self.B, -1, np.int32)
            live = np.nonzero(self.lens > 0)[0]
            for n, x in zip(new, kv):
                n[live] = x[last]
            sl[live] = slots[last]
            self.new[i] = [n.cuda() for n in new]
            self.slots[i] = torch.from_numpy(sl).cuda()
            kept = [oracle.fp4_value(*oracle.quantize_fp4(bits(x))) if T else x for x in kv]
            self.vals[i] = [[x[a: a + len(p)] for x in kept]
                            for a, p in zip(np.concatenate([[0], np.cumsum([len(p) for p in pos])]), pos)]
        torch.cuda.synchronize()

    def store_current(self):
        for i, (k, v) in self.new.items():
            self.cache.store(i, k, v, self.slots[i])

    def outs(self, i):
        d = self.layers[i]
        return (torch.full((self.B, d["num_q_heads"], d["head_dim"]), float("nan"), dtype=torch.bfloat16, device="cuda"),
                torch.full((self.B, d["num_q_heads"]), float("nan"), device="cuda"))

    def workspace(self, i):
        return self.fa.workspace(self.cache.decode_workspace_bytes(i, self.B, self.max_len))

    def decode(self, i, ws=None, fused=False):
        out, lse = self.outs(i)
        ws = self.workspace(i) if ws is None else ws
        if fused:
            k, v = self.new.get(i, (None, None))
            self.cache.decode_store(i, self.q[i], k, v, self.slots.get(i), self.bt[i], self.lens_dev, self.max_len, out,
                                    lse, ws)
        else:
            self.cache.decode(i, self.q[i], self.bt[i], self.lens_dev, self.max_len, out, lse, ws)
        return out, lse

    def check(self, i, out, lse, seqs=None, q=None):
        d = self.layers[i]
        g = d["num_q_heads"] // d["num_kv_heads"]
        q = oracle.bf16_to_f64(bits(self.q[i] if q is None else q))
        out, lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
        for b in range(self.B) if seqs is None else seqs:
            if self.lens[b] <= 0:
                assert (out[b] == 0).all() and (lse[b] == -np.inf).all()
                continue
            K, V = self.vals[self.src[i]][b]
            win = d["window"] if d["kind"] == W.SLIDING else 0
            n = min(len(K), win) if win else len(K)
            for j in range(d["num_q_heads"]):
                o, s, tol = attend(q[b, j], K[len(K) - n:, j // g], V[len(K) - n:, j // g], d["sm_scale"])
                assert np.isfinite(out[b, j]).all(), (i, b, j)
                worst = np.max(np.abs(out[b, j] - o) / tol)
                assert worst <= 1, (i, b, j, int(self.lens[b]), worst)
                assert abs(lse[b, j] - s) <= 2.0 ** -9 + 2.0 ** -20 * abs(s), (i, b, j, lse[b, j], s)


class ExtendCase4:
    """Sequences of stored prefix rows and new tokens; with `stored` the new
    tokens' rows are in the slab too (multi-token decode)."""

    def __init__(self, layers, prefix, chunk, page_size=16, seed=0, stored=False, split=None, edit=None):
        import full_attention_gb300 as fa
        self.fa, self.layers, self.ps, self.stored = fa, layers, page_size, stored
        self.unpacked = split is not None and "unpack" in split
        self.prefix, self.chunk = np.asarray(prefix, np.int32), np.asarray(chunk, np.int32)
        self.B = len(prefix)
        total = self.prefix + self.chunk
        plan = W.plan_pages(np.maximum(total if stored else self.prefix, 1), page_size, seed)
        self.cache = fa.Cache(layers, plan.num_pages, page_size, fa.KV_FP4)
        self.src = [self.cache.source(i) for i in range(len(layers))]
        self.slabs = self.cache.allocate("cuda")
        if split == "all":
            self.cache.set_flags(fa.FLAG_EXTEND_SPLIT_ALL)
        if split is not None:   # "tail", "all": the split part only; "unpack": with room for the prefix as bf16 rows
            n = fa.extend_workspace_bytes()
            if "unpack" in split:
                if "all" in split:
                    self.cache.set_flags(fa.FLAG_EXTEND_SPLIT_ALL)
                most = int((self.prefix + self.chunk).max())
                n = max(self.cache.extend_workspace_bytes(i, self.B, int(self.chunk.max()), most) for i in range(len(layers)))
            self.ws = torch.full((n,), 255, dtype=torch.uint8, device="cuda")   # NaN rows where nothing is unpacked
            self.cache.bind_extend_workspace(self.ws)
        self.indptr = np.concatenate([[0], np.cumsum(self.chunk)]).astype(np.int32)
        self.N = int(self.indptr[-1])
        self.q, self.ext, self.vals = {}, {}, {}
        for i, d in enumerate(layers):
            g = torch.Generator().manual_seed(seed * 77 + i)
            self.q[i] = torch.randn((self.N, d["num_q_heads"], d["head_dim"]), generator=g).to(torch.bfloat16).cuda()
            if self.src[i] != i:
                continue
            junk(self.slabs[i], seed + i)
            H, D = d["num_kv_heads"], d["head_dim"]
            pre = [rows_like_a_model(int(self.prefix.sum()), H, D, seed * 31 + 4 * i + s) for s in (0, 1)]
            new = [rows_like_a_model(self.N, H, D, seed * 31 + 4 * i + 2 + s) for s in (0, 1)]
            if edit is not None:
                edit(i, *pre, *new)
            at = np.concatenate([[0], np.cumsum(self.prefix)])
            slots = [W.slots_for_positions(plan.block_table[b], np.arange(int(self.prefix[b])), page_size)
                     for b in range(self.B)]
            rows = [x for x in pre]
            if stored:
                slots += [W.slots_for_positions(plan.block_table[b], np.arange(int(self.prefix[b]), int(total[b])), page_size)
                          for b in range(self.B)]
                rows = [torch.cat([a, b]) for a, b in zip(pre, new)]
            sl = torch.from_numpy(np.concatenate(slots).astype(np.int32)).cuda()
            if sl.numel():
                self.cache.store(i, rows[0].cuda(), rows[1].cuda(), sl)
            self.ext[i] = [x.cuda() for x in new]
            kept = [oracle.fp4_value(*oracle.quantize_fp4(bits(x))) if len(x) else np.zeros((0, H, D)) for x in pre]
            fresh = [oracle.fp4_value(*oracle.quantize_fp4(bits(x))) if stored else oracle.bf16_to_f64(bits(x)) for x in new]
            self.vals[i] = [[np.concatenate([k[at[b]: at[b + 1]], f[self.indptr[b]: self.indptr[b + 1]]])
                             for k, f in zip(kept, fresh)] for b in range(self.B)]
        self.bt = torch.from_numpy(plan.block_table).cuda()
        self.indptr_dev = torch.from_numpy(self.indptr).cuda()
        self.prefix_dev = torch.from_numpy(self.prefix).cuda()
        self.lens_dev = torch.from_numpy(total.astype(np.int32)).cuda()
        torch.cuda.synchronize()

    def outs(self, i):
        d = self.layers[i]
        return (torch.full((self.N, d["num_q_heads"], d["head_dim"]), float("nan"), dtype=torch.bfloat16, device="cuda"),
                torch.full((self.N, d["num_q_heads"]), float("nan"), device="cuda"))

    def run(self, i):
        out, lse = self.outs(i)
        if self.stored:
            self.cache.decode_multi(i, self.q[i], self.indptr_dev, self.lens_dev, self.bt, int(self.chunk.max()),
                                    int((self.prefix + self.chunk).max()), out, lse)
        else:
            k, v = self.ext[self.src[i]]
            self.cache.extend(i, self.q[i], k, v, self.indptr_dev, self.prefix_dev, self.bt, int(self.chunk.max()),
                              int(self.prefix.max()), out, lse)
        return out, lse

    def check(self, i, out, lse, most=400):
        """Every new token (past `most` of a sequence, an even sample that holds the first and the last)."""
        d = self.layers[i]
        g = d["num_q_heads"] // d["num_kv_heads"]
        q = oracle.bf16_to_f64(bits(self.q[i]))
        out, lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
        assert np.isfinite(out).all() and np.isfinite(lse).all()
        win = d["window"] if d["kind"] == W.SLIDING else 0
        for b in range(self.B):
            n, P = int(self.chunk[b]), int(self.prefix[b])
            if n == 0:
                continue
            t = np.unique(np.linspace(0, n - 1, min(n, most)).astype(int))
            K, V = self.vals[self.src[i]][b]
            kpos = np.arange(P + n)
            seen = kpos[None] <= P + t[:, None]
            if win:
                seen &= P + t[:, None] - kpos[None] < win
            rows = self.indptr[b] + t
            for j in range(d["num_q_heads"]):
                k, v = K[:, j // g], V[:, j // g]
                s = np.where(seen, d["sm_scale"] * (q[rows, j] @ k.T), -np.inf)
                m = s.max(1, keepdims=True)
                p = np.exp(s - m)
                l = p.sum(1, keepdims=True)
                p /= l
                ref = p @ v
                a, w = (2.0 ** -7, 1.5 * 2.0 ** -8) if self.unpacked else (2.0 ** -8, 2.0 ** -8)
                tol = a * np.abs(ref) + w * (p @ np.abs(v)) + 1e-30
                worst = np.max(np.abs(out[rows, j] - ref) / tol)
                assert worst <= 1, (i, b, j, worst)
                r = (m + np.log(l))[:, 0]
                assert np.all(np.abs(lse[rows, j] - r) <= 2.0 ** -9 + 2.0 ** -20 * np.abs(r)), (i, b, j)
