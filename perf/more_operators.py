"""Measured cases of a paged serving step's three operators around and in its attention.

plan   One step's block tables and slot maps, from the numbers of new tokens.  Sequence
       b holds len[b] tokens, in pages first[b] .. ceil(len[b] / page) - 1 of its table
       row; new[b] >= 0 tokens join it, new[b] < 0 ends it.  The pages it keeps are all of
       them, or under a window W those from (len[b] - W + 1) / page on, which the first new
       token's query still sees.  Pages given up go behind the queue of free pages, pages
       needed come off its head, both in order of sequence and page.  Out come the offsets
       of the new tokens, their positions and their slots.
rows   Norms of queries and keys (and values) for each head, and the rotation by position,
       with the rows kept in the paged cache: y = x / sqrt(mean(x^2) + eps) * (offset + w),
       then for i < R / 2 the pair (y[i], y[i + R / 2]) turned by position * freq[i].
diff   Differential attention over that cache: queries and keys of D values are two of
       D / 2, and out = (softmax(q1 k1) - lambda softmax(q2 k2)) v, with a learned lambda
       a head; decode for single tokens, extend for a chunk over a prefix.
"""
import math
import random

import numpy as np
import torch

own = False

DEV = "cuda"
FORMATS = ("bf16", "int8", "fp8")


# ------------------------------------------------------------------ the cases
def _c(name, op, page, **more):
    return dict(name=name, op=op, page=page, **more)


def _rows(name, D, hq, hkv, page, T, kv="bf16", rot=None, offset=0.0, norm_v=True, chunk=False):
    return _c(name, "rows", page, D=D, hq=hq, hkv=hkv, T=T, kv=kv, rot=D if rot is None else rot, offset=offset, norm_v=norm_v, chunk=chunk)


def _plan(name, page, B, lo, hi, plo, phi, window=0, last=1, ends=0, joins=0, lens=0):
    return _c(name, "plan", page, B=B, lo=lo, hi=hi, plo=plo, phi=phi, window=window, last=last, ends=ends, joins=joins, lens=lens)


def _diff(name, D, hq, hkv, page, B, plo, phi, lo=0, hi=0, window=0, kv="bf16", lens=0):
    return _c(name, "extend" if hi else "decode", page, D=D, hq=hq, hkv=hkv, B=B, plo=plo, phi=phi, lo=lo, hi=hi, window=window, kv=kv, lens=lens)


def listed():
    return [
        # a decode step of 64 sequences, one token each: latency
        _plan("plan step", 16, 64, 1, 1, 512, 4096, lens=1),
        # 128 sequences in a pool of the window's pages, some of them ending and some starting with a prompt
        _plan("plan sliding", 16, 128, 1, 1, 1024, 8192, window=1024, ends=5, joins=3, lens=2),
        # whole prompts of 512 sequences at once, ragged
        _plan("plan prompts", 64, 512, 1, 8192, 0, 300, lens=3),
        # one token of one sequence: latency
        _rows("rows one", 256, 4, 1, 16, 1),
        # a decode step of 64 sequences, full layer, int8 slab
        _rows("rows step", 512, 8, 1, 16, 64, kv="int8"),
        # four 512-token chunks, eight KV heads, the chunk's rows for extend beside the slab
        _rows("rows chunk", 256, 16, 8, 16, 2048, offset=1.0, norm_v=False, chunk=True),
        # the prompts of a whole batch, an odd number of tokens, half of each head rotated, fp8 slab
        _rows("rows prompts", 512, 16, 2, 64, 30011, kv="fp8", rot=256),
        # a single short sequence, sliding layer: latency
        _diff("diff one", 256, 4, 1, 16, 1, 200, 200, window=64),
        # a batch of 64 chats, full layer
        _diff("diff batch", 512, 8, 1, 16, 64, 512, 4096, lens=1),
        # eight long contexts, full layer, int8 slab
        _diff("diff long", 512, 8, 1, 16, 8, 32768, 131072, kv="int8", lens=3),
        # the last 512-token chunk of four 4096-token prompts, sliding layer
        _diff("diff chunk", 256, 16, 8, 16, 4, 3584, 3584, 512, 512, window=1024, lens=2),
        # prompts of odd lengths packed together over odd prefixes, full layer, fp8 slab
        _diff("diff ragged", 512, 16, 2, 32, 5, 0, 4096, 1, 1500, kv="fp8", lens=5),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("plan", "rows", "decode", "extend"))
    page = rng.choice((16, 16, 32, 48, 64, 128, 256))
    lens = rng.randrange(1 << 20)
    if op == "plan":
        B = _log(rng, 1, 1024)
        hi = _log(rng, 1, min(65536, 2000000 // B + 1))
        window = rng.choice((0, _log(rng, 1, 4096)))
        return _plan("", page, B, rng.randint(0, hi), hi, 0, _log(rng, 1, 8192), window=window, last=_log(rng, 1, 512),
                     ends=rng.randint(0, 10), joins=rng.randint(0, 10), lens=lens)
    D = rng.choice((256, 512))
    hkv = rng.choice((1, 1, 2, 4, 8))
    kv = rng.choice(FORMATS)
    if op == "rows":
        return _rows("", D, hkv * rng.randint(1, 8), hkv, page, _log(rng, 1, 49152 // hkv), kv=kv, rot=16 * rng.randint(1, D // 16),
                     offset=rng.choice((0.0, 1.0)), norm_v=rng.random() < 0.5, chunk=rng.random() < 0.5)
    window = rng.choice((0, _log(rng, 1, 4096)))
    if op == "decode":
        hi = _log(rng, 1, 65536)
        B = _log(rng, 1, max(1, min(256, 300000 // (hi * hkv))))
        return _diff("", D, hkv * rng.randint(1, 16), hkv, page, B, rng.randint(0, hi), hi, window=window, kv=kv, lens=lens)
    hq = hkv * rng.choice((1, 2, 4, 8, 16))
    phi = _log(rng, 1, 8192)
    most = 3 * 10 ** 10 // (hq * D)   # pairs of a query and a key
    hi = _log(rng, 1, min(2048, most // (phi + 2048)))
    B = _log(rng, 1, max(1, min(16, most // (hi * (hi + phi)))))
    return _diff("", D, hq, hkv, page, B, rng.randint(0, phi), phi, rng.randint(1, hi), hi, window=window, kv=kv, lens=lens)


def _lens(case):
    """The context lengths, and of plan and extend the new tokens' numbers (plan: -1 where a sequence ends)."""
    r = random.Random(case["lens"])
    ctx = [r.randint(case["plo"], case["phi"]) for _ in range(case["B"])]
    if case["op"] == "decode":
        return ctx, None
    new = [r.randint(case["lo"], case["hi"]) for _ in range(case["B"])]
    if case["op"] == "plan":
        for b in r.sample(range(case["B"]), min(case["B"], case["ends"])):
            new[b] = -1
        for b in r.sample(range(case["B"]), min(case["B"], case["joins"])):
            ctx[b], new[b] = 0, r.randint(1, max(1, case["phi"]))
    return ctx, new


def _row_bytes(kv, D):
    return 2 * D if kv == "bf16" else D + 4


def work(case):
    if case["op"] == "plan":
        ctx, new = _lens(case)
        N, ps = sum(n for n in new if n > 0), case["page"]
        pages = sum(-(-(c + n) // ps) - -(-c // ps) for c, n in zip(ctx, new) if n > 0)
        # per new token a position and a slot, per page a table entry and its place in the queue, per sequence its state
        return {"bytes": 8 * N + 8 * pages + 4 * case["B"] * 7, "flops": 8 * N}
    D, hq, hkv = case["D"], case["hq"], case["hkv"]
    row = _row_bytes(case["kv"], D)
    if case["op"] == "rows":
        moved = hq * 4 * D + 2 * hkv * (2 * D + row) + (2 * hkv * 2 * D if case["chunk"] else 0)
        if case["kv"] != "bf16":   # the rows read back
            moved += 2 * hkv * (row + 2 * D)
        return {"bytes": case["T"] * (moved + 8), "flops": case["T"] * (hq + 2 * hkv) * D * 8}
    ctx, new = _lens(case)
    W = case["window"]
    if new is None:
        seen = [min(n, W) if W else n for n in ctx]
        return {"bytes": sum(seen) * hkv * 2 * row + case["B"] * hq * (4 * D + 8) + 4 * sum(-(-n // case["page"]) for n in seen),
                "flops": sum(seen) * hq * D * 6}
    pairs = sum(sum(min(p + i + 1, W) if W else p + i + 1 for i in range(n)) for p, n in zip(ctx, new))
    seen = [min(p, W - 1) if W else p for p in ctx]
    return {"bytes": sum(seen) * hkv * 2 * row + sum(new) * (hkv * 4 * D + hq * (4 * D + 8)), "flops": pairs * hq * D * 6}


# -------------------------------------------------------------------- inputs
def _normal(g, T, H, D):
    """Rows as a model's projections make them: normal values, some channels and tokens larger."""
    c = torch.randn(H, D, generator=g, device=DEV)
    x = torch.randn(T, H, D, generator=g, device=DEV) * torch.where(c > 1.9, 6.0, 1.0)
    return x * torch.exp(0.3 * torch.randn(T, 1, 1, generator=g, device=DEV))


def _pages(g, need, page):
    """A block table over a random permutation of a pool a quarter larger than what is needed."""
    n = [-(-v // page) for v in need]
    pool = max(1, math.ceil(1.25 * sum(n)))
    ids = torch.randperm(pool, generator=g, device=DEV).int()
    bt = torch.full((len(n), max(1, max(n))), -1, dtype=torch.int32, device=DEV)
    at = 0
    for b, k in enumerate(n):
        bt[b, :k] = ids[at: at + k]
        at += k
    return pool, bt


def _quantise(x, kv):
    """Codes and scales of rows x [..., D] of bf16 values: the scale max|x| / 127 or / 448, the code nearest to x / scale."""
    x = x.float()
    top = 127.0 if kv == "int8" else 448.0
    s = x.abs().amax(-1) / top
    y = torch.where(s[..., None] > 0, x / s[..., None], 0.0).clamp(-top, top)
    return (y.round().to(torch.int8) if kv == "int8" else y.to(torch.float8_e4m3fn).view(torch.uint8)), s


def _values(rows, s, kv, to=torch.float32):
    if kv == "bf16":
        return rows.to(to)
    return (rows if kv == "int8" else rows.view(torch.float8_e4m3fn)).to(to) * s.to(to)[..., None]


def _slabs(st, pool, make):
    """K and V slabs [pages][heads][page][D] and scales, from bf16 rows or zero."""
    hkv, ps, D, kv = st["hkv"], st["page"], st["D"], st["kv"]
    for n in "kv":
        x = make() if make else torch.zeros(pool * ps, hkv, D, dtype=torch.bfloat16, device=DEV)
        x = x.view(pool, ps, hkv, D).transpose(1, 2).contiguous()
        st[n], st[n + "s"] = (x, None) if kv == "bf16" else _quantise(x, kv)


def _cache(st, pool):
    """The handle that a serving program keeps."""
    import full_attention_gb300 as fa

    W = st.get("window", 0)
    layer = dict(kind=fa.SLIDING if W else fa.FULL, head_dim=st.get("D", 256), num_q_heads=st.get("hq", 1), num_kv_heads=st.get("hkv", 1),
                 window=W, kv_source=fa.KV_OWN, sm_scale=st.get("sm", 1.0))
    cache = fa.Cache([layer], pool, st["page"], {"bf16": fa.KV_BF16, "int8": fa.KV_INT8, "fp8": fa.KV_FP8}[st.get("kv", "bf16")])
    if "k" in st:
        cache.bind(0, st["k"], st["v"], st["ks"], st["vs"])
    return fa, cache


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    st = dict(case)
    return {"plan": _prepare_plan, "rows": _prepare_rows, "decode": _prepare_diff, "extend": _prepare_diff}[case["op"]](st, case, g)


def _prepare_plan(st, case, g):
    """The state that the steps before left: the sequences' pages off a shuffled queue, the rest of it free from a random place on."""
    ps, B, W = case["page"], case["B"], case["window"]
    ctx, new = (np.array(v, dtype=np.int64) for v in _lens(case))
    have = -(-ctx // ps)
    first = np.maximum(0, ctx - case["last"] - W + 1) // ps if W else np.zeros_like(ctx)   # what the last step's first query saw
    first = np.minimum(first, have)
    last = -(-(ctx + np.maximum(new, 0)) // ps)
    used, need = int((have - first).sum()), int((last - have).sum())
    pool = max(1, math.ceil(1.25 * (used + need)))
    ids = torch.randperm(pool, generator=g, device=DEV).int()
    cols = int(last.max()) + 2
    col = torch.arange(cols, device=DEV)
    f, h = (torch.from_numpy(v).to(DEV)[:, None] for v in (first, have))
    held = (col >= f) & (col < h)
    bt = torch.full((B, cols), -1, dtype=torch.int32, device=DEV)
    bt[held] = ids[:used]
    head = int(torch.randint(pool, (1,), generator=g, device=DEV))
    free = torch.roll(torch.cat((ids[used:], torch.full((used,), -1, dtype=torch.int32, device=DEV))), head)
    state = torch.zeros(4 + 2 * B, dtype=torch.int32)
    state[0], state[1] = head, pool - used
    state[4: 4 + B], state[4 + B:] = torch.from_numpy(ctx), torch.from_numpy(first)
    N = int(np.maximum(new, 0).sum())
    st["new"] = torch.from_numpy(new).int().to(DEV)
    st["bt"], st["free"], st["state"], st["state_out"] = bt, free, state.to(DEV), torch.zeros(4 + 2 * B, dtype=torch.int32, device=DEV)
    rows = max(1, -(-N // 64) * 64)   # the step's buffers are padded
    st["indptr"] = torch.zeros(B + 1, dtype=torch.int32, device=DEV)
    st["prefix"] = torch.zeros(B, dtype=torch.int32, device=DEV)
    st["pos"], st["slots"] = (torch.zeros(rows, dtype=torch.int32, device=DEV) for _ in range(2))
    if own:
        fa, cache = _cache(st, pool)
        st["cache"] = cache
        st["table"] = fa.PageTable(cache, fa.SLIDING if W else fa.FULL, st["bt"], st["free"], st["state"])
    return st


def _prepare_rows(st, case, g):
    D, hq, hkv, ps, T = case["D"], case["hq"], case["hkv"], case["page"], case["T"]
    pool, bt = _pages(g, [T], ps)
    at = torch.arange(T, device=DEV)
    st["slots"] = (bt[0].long()[at // ps] * ps + at % ps).int()
    # one projection's rows, [T][(hq + 2 hkv) D]
    st["qkv"] = _normal(g, T, hq + 2 * hkv, D).bfloat16().view(T, -1)
    start = int(torch.randint(131072 - min(T, 4096), (1,), generator=g, device=DEV))
    st["positions"] = (start + at % 4096).int()
    st["freq"] = 10000.0 ** (-torch.arange(case["rot"] // 2, dtype=torch.float64) / (case["rot"] // 2))
    base = 1.0 - case["offset"]
    st["qw"], st["kw"] = ((base + 0.1 * torch.randn(D, generator=g, device=DEV)).bfloat16() for _ in range(2))
    st["q_out"] = torch.empty(T, hq, D, dtype=torch.bfloat16, device=DEV)
    st["k_out"], st["v_out"] = (torch.empty(T, hkv, D, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    st["k_back"], st["v_back"] = (torch.empty(T, hkv, D, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    st["freq_dev"] = st["freq"].to(DEV)
    _slabs(st, pool, None)
    if own:
        fa, st["cache"] = _cache(st, pool)
        st["norm"] = fa.NormRope(D, st["freq"], q_weight=st["qw"], k_weight=st["kw"], eps=1e-6, weight_offset=case["offset"],
                                 norm_v=case["norm_v"], device=DEV)
    return st


def _prepare_diff(st, case, g):
    D, hq, hkv, ps, B = case["D"], case["hq"], case["hkv"], case["page"], case["B"]
    st["sm"] = float(np.float32(1 / math.sqrt(D // 2)))
    ctx, new = _lens(case)
    pool, st["bt"] = _pages(g, ctx, ps)
    if new is None:
        st["lens"] = torch.tensor(ctx, dtype=torch.int32, device=DEV)
        st["max_len"], N = max(1, max(ctx)), B
    else:
        st["prefix"] = torch.tensor(ctx, dtype=torch.int32, device=DEV)
        ptr = np.concatenate([[0], np.cumsum(new)])
        st["indptr"] = torch.from_numpy(ptr).int().to(DEV)
        st["max_new"], st["max_prefix"], N = max(new), max(ctx), int(ptr[-1])
        st["k_ext"], st["v_ext"] = (_normal(g, N, hkv, D).bfloat16() for _ in range(2))
    _slabs(st, pool, lambda: _normal(g, pool * ps, hkv, D).bfloat16())
    st["q"] = torch.randn(N, hq, D, generator=g, device=DEV).bfloat16()
    # lambda = exp(a . b) - exp(c . d) + start of four learned vectors, a head each
    a, b, c, d = (0.1 * torch.randn(hq, D // 2, generator=g, device=DEV) for _ in range(4))
    st["lam"] = torch.exp((a * b).sum(-1)) - torch.exp((c * d).sum(-1)) + 0.5
    st["out"] = torch.empty(N, hq, D, dtype=torch.bfloat16, device=DEV)
    st["lse"] = torch.empty(N, hq, 2, device=DEV)
    if own:
        fa, st["cache"] = _cache(st, pool)
        if new is None:
            st["ws"] = fa.workspace(st["cache"].decode_diff_workspace_bytes(0, B, st["max_len"]))
        else:
            st["ws"] = fa.workspace(st["cache"].extend_diff_workspace_bytes(0, B, st["max_new"], st["max_prefix"]))
            st["cache"].bind_extend_workspace(st["ws"])
    return st


# --------------------------------------------------------------- one pass
def run(st):
    return {"plan": _run_plan, "rows": _run_rows, "decode": _run_decode, "extend": _run_extend}[st["op"]](st)


def _run_plan(st):
    outs = tuple(st[n] for n in ("bt", "free", "state_out", "indptr", "prefix", "pos", "slots"))
    if own:
        st["table"].step(st["new"], st["indptr"], st["prefix"], st["pos"], st["slots"], state_out=st["state_out"])
        return outs
    ps, B, W = st["page"], st["B"], st["window"]
    bt, free, state, new = st["bt"], st["free"], st["state"].long(), st["new"].long()
    head, count, length, first = state[0], state[1], state[4: 4 + B], state[4 + B:]
    pool, cols = free.numel(), bt.shape[1]
    n, ended = new.clamp(min=0), new < 0
    have = (length + ps - 1) // ps
    after = torch.where(ended, 0, length + n)
    want = torch.where(ended, have, (after + ps - 1) // ps)
    keep = (length - W + 1).clamp(min=0) // ps if W else torch.zeros_like(length)
    keep = torch.where(ended, have, torch.maximum(keep, first))
    # pages given up, behind the queue
    col = torch.arange(cols, device=bt.device)
    gone = (col >= first[:, None]) & (col < keep[:, None])
    order = gone.flatten().long().cumsum(0) - 1
    at = torch.where(gone.flatten(), (head + count + order) % pool, pool)
    queue = torch.cat((free, free[:1])).index_put((at,), bt.flatten())[:pool]
    # pages needed, off its head
    need = want - have
    base = need.cumsum(0) - need
    fresh = (col >= have[:, None]) & (col < want[:, None])
    page = free[(head + base[:, None] + col - have[:, None]) % pool]
    bt.copy_(torch.where(fresh, page, bt))
    free.copy_(queue)
    out = st["state_out"]
    out[0] = (head + need.sum()) % pool
    out[1] = count - need.sum() + (keep - first).sum()
    out[4: 4 + B] = after
    out[4 + B:] = torch.where(ended, 0, keep)
    ptr = torch.cat((torch.zeros_like(n[:1]), n.cumsum(0)))
    st["indptr"].copy_(ptr)
    st["prefix"].copy_(torch.where(ended, 0, length))
    t = torch.arange(st["pos"].numel(), device=bt.device)
    b = (torch.searchsorted(ptr, t, right=True) - 1).clamp(max=B - 1)
    pos = length[b] + t - ptr[b]
    slot = bt[b, (pos // ps).clamp(max=cols - 1)].long() * ps + pos % ps
    st["pos"].copy_(torch.where(t < ptr[-1], pos, 0))
    st["slots"].copy_(torch.where(t < ptr[-1], slot, -1))
    return outs


def _normed(x, w, offset, dt):
    """x [T, H, D] over its root mean square, times the weights."""
    y = x / torch.sqrt(x.square().mean(-1, keepdim=True) + 1e-6)
    return y if w is None else y * (w.to(dt) + offset)


def _turned(y, angle, dt):
    """y [T, H, D] with pairs (i, i + R / 2) turned by angle [T, R / 2] (64 bits)."""
    half = angle.shape[1]
    c, s = torch.cos(angle)[:, None].to(dt), torch.sin(angle)[:, None].to(dt)
    a, b = y[..., :half], y[..., half: 2 * half]
    return torch.cat((a * c - b * s, b * c + a * s, y[..., 2 * half:]), -1)


def _run_rows(st):
    T, D, hq, hkv, ps, kv = (st[n] for n in ("T", "D", "hq", "hkv", "page", "kv"))
    x = st["qkv"].view(T, hq + 2 * hkv, D)
    q, k, v = x[:, :hq], x[:, hq: hq + hkv], x[:, hq + hkv:]
    if own:
        rows = (st["k_out"], st["v_out"]) if st["chunk"] else (None, None)
        st["cache"].norm_rope_store(0, st["norm"], q, k, v, st["positions"], st["slots"], st["q_out"], *rows)
        rows = rows if st["chunk"] else ()
        if kv == "bf16":
            return (st["q_out"], st["k"], st["v"]) + rows
        st["cache"].load(0, st["slots"], st["k_back"], st["v_back"])
        return (st["q_out"], st["k_back"], st["v_back"]) + rows
    f32 = torch.float32
    angle = st["positions"].double()[:, None] * st["freq_dev"]
    st["q_out"].copy_(_turned(_normed(q.float(), st["qw"], st["offset"], f32), angle, f32))
    k = _turned(_normed(k.float(), st["kw"], st["offset"], f32), angle, f32).bfloat16()
    v = _normed(v.float(), None, 0.0, f32).bfloat16() if st["norm_v"] else v
    rows = (k, v) if st["chunk"] else ()
    page, off = st["slots"].long() // ps, st["slots"].long() % ps
    if kv == "bf16":
        st["k"][page, :, off], st["v"][page, :, off] = k, v
        return (st["q_out"], st["k"], st["v"]) + rows
    st["k"][page, :, off], st["ks"][page, :, off] = _quantise(k, kv)
    st["v"][page, :, off], st["vs"][page, :, off] = _quantise(v, kv)
    return (st["q_out"],) + tuple(_values(st[n][page, :, off], st[n + "s"][page, :, off], kv).bfloat16() for n in "kv") + rows


def _gather(st, pos):
    """fp32 K and V [B, n, H, D] at positions pos [B, n] (clamped into the table)."""
    idx = (pos // st["page"]).clamp(0, st["bt"].shape[1] - 1)
    page = st["bt"].long().gather(1, idx).clamp(min=0)
    off = pos.clamp(min=0) % st["page"]
    s = [None if st[n + "s"] is None else st[n + "s"][page, :, off] for n in "kv"]
    return tuple(_values(st[n][page, :, off], x, st["kv"]) for n, x in zip("kv", s))


def _two_maps(q, k, v, lam, seen, sm):
    """q [B, H, r, D], k, v [B, n, H, D], lam broadcast to [B, H, r, 1], seen [B, 1, r, n]: out [B, H, r, D], lse [B, H, r, 2]."""
    half = q.shape[-1] // 2

    def one(m):
        s = torch.matmul(q[..., m * half: (m + 1) * half], k[..., m * half: (m + 1) * half].permute(0, 2, 3, 1)) * sm
        s = s.masked_fill_(~seen, float("-inf"))
        top = s.amax(-1, keepdim=True)
        top = torch.where(top == float("-inf"), 0.0, top)
        p = torch.exp(s.sub_(top))
        l = p.sum(-1, keepdim=True)
        return torch.matmul(p, v.transpose(1, 2)) / torch.where(l > 0, l, 1.0), (top + torch.log(l))[..., 0]

    (o1, l1), (o2, l2) = one(0), one(1)
    return o1 - lam * o2, torch.stack((l1, l2), -1)


def _run_decode(st):
    if own:
        st["cache"].decode_diff(0, st["q"], st["lam"], st["bt"], st["lens"], st["max_len"], st["out"], st["lse"], st["ws"])
        return st["out"], st["lse"]
    B, hq, D = st["q"].shape
    H, W = st["hkv"], st["window"]
    L = st["lens"].long()[:, None]
    lo = (L - W).clamp(min=0) if W else torch.zeros_like(L)
    n = min(st["max_len"], W) if W else st["max_len"]
    pos = lo + torch.arange(n, device=L.device)
    k, v = _gather(st, pos)
    out, lse = _two_maps(st["q"].float().view(B, H, hq // H, D), k, v, st["lam"].view(1, H, hq // H, 1), (pos < L)[:, None, None], st["sm"])
    return out.reshape(B, hq, D).bfloat16(), lse.reshape(B, hq, 2)


def _run_extend(st):
    if own:
        st["cache"].extend_diff(0, st["q"], st["lam"], st["k_ext"], st["v_ext"], st["indptr"], st["prefix"], st["bt"],
                                st["max_new"], st["max_prefix"], st["out"], st["lse"])
        return st["out"], st["lse"]
    N, hq, D = st["q"].shape
    H, W, B = st["hkv"], st["window"], st["B"]
    dev = st["q"].device
    ptr, P = st["indptr"].long(), st["prefix"].long()[:, None]
    i = torch.arange(st["max_new"], device=dev)
    row = (ptr[:-1, None] + i).clamp(max=N - 1)                     # [B, new]
    first = (P - W + 1).clamp(min=0) if W else torch.zeros_like(P)   # the first prefix key any query sees
    n = min(st["max_prefix"], W - 1) if W else st["max_prefix"]
    pos = first + torch.arange(n, device=dev)
    k, v = _gather(st, pos)
    k = torch.cat((k, st["k_ext"][row].float()), 1)
    v = torch.cat((v, st["v_ext"][row].float()), 1)
    kpos = torch.cat((torch.where(pos < P, pos, 1 << 40), P + i), 1)[:, None]   # [B, 1, keys]
    qpos = (P + i)[..., None]                                        # [B, new, 1]
    seen = kpos <= qpos
    if W:
        seen &= qpos - kpos < W
    g = hq // H
    q = st["q"].float()[row].view(B, -1, H, g, D).permute(0, 2, 3, 1, 4).reshape(B, H, -1, D)
    lam = st["lam"].view(H, g, 1).expand(H, g, q.shape[2] // g).reshape(1, H, -1, 1)
    out, lse = _two_maps(q, k, v, lam, seen.repeat(1, g, 1)[:, None], st["sm"])
    out = out.view(B, H, g, -1, D).permute(0, 3, 1, 2, 4).reshape(B, -1, hq, D)
    lse = lse.view(B, H, g, -1, 2).permute(0, 3, 1, 2, 4).reshape(B, -1, hq, 2)
    t = torch.arange(N, device=dev)
    b = torch.searchsorted(ptr, t, right=True) - 1
    return out[b, t - ptr[b]].bfloat16(), lse[b, t - ptr[b]]


# --------------------------------------------------- the definition in 64 bits
def exact(case, seed):
    if case["op"] == "plan":
        return None   # whole numbers
    st = prepare(case, seed)
    return _exact_rows(st) if case["op"] == "rows" else _exact_diff(st, case)


def _exact_rows(st):
    T, D, hq, hkv, ps, kv = (st[n] for n in ("T", "D", "hq", "hkv", "page", "kv"))
    x = st["qkv"].double().view(T, hq + 2 * hkv, D)
    angle = torch.outer(st["positions"].double(), st["freq_dev"])
    turn = torch.polar(torch.ones_like(angle), angle)[:, None]
    half = angle.shape[1]

    def rows(x, w, turned):
        y = x * torch.rsqrt((x * x).sum(-1, keepdim=True) / D + 1e-6)
        if w is not None:
            y = y * (st["offset"] + w.double())
        if turned:
            z = torch.complex(y[..., :half], y[..., half: 2 * half]) * turn
            y = torch.cat((z.real, z.imag, y[..., 2 * half:]), -1)
        return y

    q = rows(x[:, :hq], st["qw"], True)
    k = rows(x[:, hq: hq + hkv], st["kw"], True)
    v = rows(x[:, hq + hkv:], None, False) if st["norm_v"] else x[:, hq + hkv:]
    out = ()
    slots = st["slots"].long()
    for r in (k, v):
        if kv == "bf16":
            slab = torch.zeros(st["k"].shape, dtype=torch.float64, device=DEV)
            slab[slots // ps, :, slots % ps] = r
            out += (slab,)
        else:   # a format of codes keeps bf16 rows: its nearest code, an fp32 scale
            b = r.bfloat16().double()
            top = 127.0 if kv == "int8" else 448.0
            s = (b.abs().amax(-1, keepdim=True) / top).float().double()
            c = (b / s).clamp(-top, top)
            out += ((c.round() if kv == "int8" else c.float().to(torch.float8_e4m3fn).double()) * s,)
    return (q,) + out + ((k, v) if st["chunk"] else ())


def _exact_diff(st, case):
    ps, H, W, sm, D, kv = (st[n] for n in ("page", "hkv", "window", "sm", "D", "kv"))
    ctx, new = _lens(case)
    q, lam = st["q"].double(), st["lam"].double()
    out = torch.zeros_like(q)
    lse = torch.full(q.shape[:2] + (2,), float("-inf"), dtype=torch.float64, device=q.device)
    g, at = q.shape[1] // H, 0
    for b, n in enumerate(ctx):
        r = 1 if new is None else new[b]
        first = n - 1 if new is None else n          # the first query's position
        if new is None and n == 0:
            at += 1
            continue
        lo = max(0, first - W + 1) if W else 0
        pos = torch.arange(lo, n, device=q.device)
        page, off = st["bt"][b].long()[pos // ps], pos % ps
        kpos = torch.arange(lo, first + r, device=q.device)
        qpos = first + torch.arange(r, device=q.device)[:, None]
        seen = (kpos <= qpos) & ((qpos - kpos < W) if W else True)
        for h in range(H):
            k, v = (_values(st[m][page, h, off], None if kv == "bf16" else st[m + "s"][page, h, off], kv, torch.float64) for m in "kv")
            if new is not None:
                k, v = (torch.cat((x, st[m][at: at + r, h].double())) for x, m in ((k, "k_ext"), (v, "v_ext")))
            for j in range(h * g, (h + 1) * g):
                for m, sign in ((0, 1.0), (1, -lam[j])):
                    cut = slice(m * D // 2, (m + 1) * D // 2)
                    s = torch.where(seen, (q[at: at + r, j, cut] @ k[:, cut].T) * sm, float("-inf"))
                    lse[at: at + r, j, m] = torch.logsumexp(s, -1)
                    out[at: at + r, j] += sign * (torch.softmax(s, -1) @ v)
        at += r
    return out, lse
