"""Measured cases of the 4-bit paged KV cache: the format's write and read back, decode and extend attention over it.

The format (one row = one token's K or V of one KV head, D = 256 or 512 values):
with a the row's largest magnitude, its scale is s = 2^e, e the smallest integer
>= -116 with a <= 2688 * 2^e; each block of 16 values has an e4m3 scale, the one
nearest to (the block's largest magnitude) / (6 s), ties to even; each value is
the e2m1 number (0, 0.5, 1, 1.5, 2, 3, 4, 6 and their negatives) nearest to
value / (s * block scale), ties to the even code, at most 6.  A block whose scale
is 0 holds zeros.  A row of the slab [pages][KV heads][page size][D * 9 / 16] is D / 2
bytes of codes (element 2 i in the low half of byte i) and D / 16 bytes of block
scales; s stands beside it as fp32.
"""
import math
import random

import numpy as np
import torch

own = False

DEV = "cuda"


# ------------------------------------------------------------------ the cases
def _c(name, kind, D, hq, hkv, page, window=0, **more):
    return dict(name=name, kind=kind, D=D, hq=hq, hkv=hkv, page=page, window=window, **more)


def listed():
    return [
        # the rows one decode step stores in an owning layer, 64 sequences: latency
        _c("write step", "write", 512, 8, 1, 16, T=64),
        # a prompt chunk of four sequences of 512 tokens, eight KV heads
        _c("write chunk", "write", 256, 16, 8, 16, T=2048),
        # the prompts of a whole batch at once, an odd number of tokens
        _c("write prompts", "write", 512, 16, 2, 64, T=30011),
        # one prompt read back (handed to another cache, or inspected)
        _c("read prompt", "read", 512, 16, 2, 16, T=1001),
        # a long context read back
        _c("read long", "read", 512, 8, 1, 16, T=131072),
        # a single short sequence, sliding layer: latency
        _c("decode one", "decode", 256, 4, 1, 16, 64, B=1, lo=200, hi=200, lens=0),
        # a batch of 64 chats, full layer
        _c("decode batch full", "decode", 512, 8, 1, 16, B=64, lo=512, hi=4096, lens=1),
        # a batch of 128, sliding layer: every sequence ends in a window of 1024
        _c("decode batch sliding", "decode", 256, 8, 1, 16, 1024, B=128, lo=1024, hi=8192, lens=4),
        # eight long contexts, full layer
        _c("decode long", "decode", 512, 8, 1, 16, B=8, lo=32768, hi=131072, lens=3),
        # odd sizes: empty and short sequences among long ones, six query heads per KV head, pages of 48
        _c("decode ragged", "decode", 256, 12, 2, 48, B=33, lo=0, hi=2500, lens=7),
        # the last 512-token chunk of four 4096-token prompts, sliding layer
        _c("extend chunk sliding", "extend", 256, 16, 8, 16, 1024, B=4, plo=3584, phi=3584, lo=512, hi=512, lens=2),
        # prompts of odd lengths packed together, over odd prefixes, full layer
        _c("extend ragged full", "extend", 512, 16, 2, 32, B=5, plo=0, phi=4096, lo=1, hi=1500, lens=5),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    D = rng.choice((256, 512))
    hkv = rng.choice((1, 1, 2, 4, 8))
    page = rng.choice((16, 16, 32, 48, 64, 128, 256))
    window = rng.choice((0, _log(rng, 1, 2048))) if D == 512 else _log(rng, 1, 4096) if rng.random() < 0.7 else 0
    kind = rng.choice(("write", "read", "decode", "decode", "extend"))
    lens = rng.randrange(1 << 20)
    if kind in ("write", "read"):
        T = _log(rng, 1, 131072 // hkv)
        return _c("", kind, D, hkv, hkv, page, 0, T=T)
    if kind == "decode":
        hq = hkv * rng.randint(1, 16)
        hi = _log(rng, 1, 65536)
        B = _log(rng, 1, max(1, min(256, 400000 // (hi * hkv))))
        return _c("", kind, D, hq, hkv, page, window, B=B, lo=rng.randint(0, hi), hi=hi, lens=lens)
    hq = hkv * rng.choice((1, 2, 4, 8, 16))
    phi = _log(rng, 1, 8192)
    most = 4 * 10 ** 10 // (hq * D)   # pairs of a query and a key
    hi = _log(rng, 1, min(2048, most // (phi + 2048)))
    B = _log(rng, 1, max(1, min(16, most // (hi * (hi + phi)))))
    return _c("", kind, D, hq, hkv, page, window, B=B, plo=rng.randint(0, phi), phi=phi, lo=rng.randint(1, hi), hi=hi, lens=lens)


def _lens(case):
    """The context lengths, and for extend the new tokens' numbers, of a case."""
    r = random.Random(case["lens"])
    if case["kind"] == "decode":
        return [r.randint(case["lo"], case["hi"]) for _ in range(case["B"])], None
    return [r.randint(case["plo"], case["phi"]) for _ in range(case["B"])], [r.randint(case["lo"], case["hi"]) for _ in range(case["B"])]


def work(case):
    D, hq, hkv, W = case["D"], case["hq"], case["hkv"], case["window"]
    row = D // 2 + D // 16 + 4
    if case["kind"] in ("write", "read"):
        rows = 2 * case["T"] * hkv
        # write: rows in, the slab's rows out, those read back, rows out
        moved = rows * (2 * D + row) * (2 if case["kind"] == "write" else 1)
        return {"bytes": moved + 4 * case["T"], "flops": rows * D * (4 if case["kind"] == "write" else 2)}
    ctx, new = _lens(case)
    if new is None:
        seen = [min(n, W) if W else n for n in ctx]
        return {"bytes": sum(seen) * hkv * 2 * row + case["B"] * hq * (4 * D + 4) + 4 * sum(-(-n // case["page"]) for n in seen),
                "flops": sum(seen) * hq * D * 4}
    pairs = sum(sum(min(p + i + 1, W) if W else p + i + 1 for i in range(n)) for p, n in zip(ctx, new))
    seen = [min(p, W - 1) if W else p for p in ctx]
    return {"bytes": sum(seen) * hkv * 2 * row + sum(new) * (hkv * 4 * D + hq * (4 * D + 4)), "flops": pairs * hq * D * 4}


# ------------------------------------------------------- the format, plain form
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _quantise(x):
    """Slab rows [..., D * 9 / 16] and row scales [...] of values x [..., D].  In 64
    bits, as the borders between two codes are exact there."""
    x = x.double()
    a = x.abs().amax(-1)
    m, p = torch.frexp(a)
    e = torch.where(m <= 0.65625, p - 12, p - 11)   # 2688 = 0.65625 * 2^12
    e = torch.where(a > 0, e, -116).clamp(min=-116)
    s = ((e.long() + 1023) << 52).view(torch.float64)   # 2^e; pow and exp2 need not be exact
    y = (x / s[..., None]).unflatten(-1, (-1, 16))
    sb = (y.abs().amax(-1) / 6).float().to(torch.float8_e4m3fn)
    t = sb.double()[..., None]
    q = torch.where(t > 0, y.abs() / torch.where(t > 0, t, 1.0), 0.0)
    code = ((q > 0.25).byte() + (q >= 0.75).byte() + (q > 1.25).byte() + (q >= 1.75).byte() + (q > 2.5).byte()
            + (q >= 3.5).byte() + (q > 5.0).byte())
    code = (code | (torch.signbit(x).byte() << 3).view_as(code)).flatten(-2)
    return torch.cat((code[..., 0::2] | (code[..., 1::2] << 4), sb.view(torch.uint8)), -1), s.float()


def _values(rows, s):
    """fp32 values [..., D] of slab rows and their scales."""
    D = rows.shape[-1] * 16 // 9
    one = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=rows.device)
    two = torch.stack((one.repeat(16), one.repeat_interleave(16)), -1)   # a byte's two values
    v = two[rows[..., : D // 2].int()].flatten(-2).unflatten(-1, (-1, 16))
    sb = rows[..., D // 2:].contiguous().view(torch.float8_e4m3fn).float()
    return (v * (sb * s[..., None])[..., None]).flatten(-2)


# -------------------------------------------------------------------- inputs
def _rows(g, T, H, D):
    """Rows as a model's projections make them: normal values, some channels and tokens larger."""
    c = torch.randn(H, D, generator=g, device=DEV)
    x = torch.randn(T, H, D, generator=g, device=DEV) * torch.where(c > 1.9, 6.0, 1.0)
    return (x * torch.exp(0.3 * torch.randn(T, 1, 1, generator=g, device=DEV))).bfloat16()


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


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    D, hq, hkv, ps, kind = case["D"], case["hq"], case["hkv"], case["page"], case["kind"]
    st = dict(case)
    st["sm"] = float(np.float32(1 / math.sqrt(D)))
    if kind in ("write", "read"):
        T = case["T"]
        pool, bt = _pages(g, [T], ps)
        at = torch.arange(T, device=DEV)
        st["slots"] = (bt[0].long()[at // ps] * ps + at % ps).int()
        st["k_out"], st["v_out"] = (torch.empty(T, hkv, D, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    elif kind == "decode":
        ctx, _ = _lens(case)
        pool, st["bt"] = _pages(g, ctx, ps)
        st["lens"] = torch.tensor(ctx, dtype=torch.int32, device=DEV)
        st["max_len"] = max(1, max(ctx))
        N = case["B"]
    else:
        ctx, new = _lens(case)
        pool, st["bt"] = _pages(g, ctx, ps)
        st["prefix"] = torch.tensor(ctx, dtype=torch.int32, device=DEV)
        ptr = np.concatenate([[0], np.cumsum(new)])
        st["indptr"] = torch.from_numpy(ptr).int().to(DEV)
        st["max_new"], st["max_prefix"], N = max(new), max(ctx), int(ptr[-1])
        st["k_ext"], st["v_ext"] = _rows(g, N, hkv, D), _rows(g, N, hkv, D)
    for n in "kv":   # what earlier steps stored
        if kind == "write":
            st[n] = torch.zeros(pool, hkv, ps, D * 9 // 16, dtype=torch.uint8, device=DEV)
            st[n + "s"] = torch.zeros(pool, hkv, ps, device=DEV)
            st[n + "_new"] = _rows(g, case["T"], hkv, D)
        else:
            x = _rows(g, pool * ps, hkv, D).view(pool, ps, hkv, D).transpose(1, 2)
            st[n], st[n + "s"] = (t.contiguous() for t in _quantise(x))
    if kind in ("decode", "extend"):
        st["q"] = torch.randn(N, hq, D, generator=g, device=DEV).bfloat16()
        st["out"] = torch.empty(N, hq, D, dtype=torch.bfloat16, device=DEV)
        st["lse"] = torch.empty(N, hq, device=DEV)
    if own:   # the handle that a serving program keeps
        import full_attention_gb300 as fa

        layer = dict(kind=fa.SLIDING if case["window"] else fa.FULL, head_dim=D, num_q_heads=hq, num_kv_heads=hkv,
                     window=case["window"], kv_source=fa.KV_OWN, sm_scale=st["sm"])
        st["cache"] = fa.Cache([layer], pool, ps, fa.KV_FP4)
        st["cache"].bind(0, st["k"], st["v"], st["ks"], st["vs"])
        if kind == "decode":
            st["ws"] = fa.workspace(st["cache"].decode_workspace_bytes(0, case["B"], st["max_len"]))
        if kind == "extend":
            st["ws"] = fa.workspace(st["cache"].extend_workspace_bytes(0, case["B"], st["max_new"], st["max_prefix"]))
            st["cache"].bind_extend_workspace(st["ws"])
    return st


# --------------------------------------------------------------- one pass
def run(st):
    return {"write": _write, "read": _read, "decode": _decode, "extend": _extend}[st["kind"]](st)


def _write(st):
    if own:
        st["cache"].store(0, st["k_new"], st["v_new"], st["slots"])
    else:
        page, off = st["slots"].long() // st["page"], st["slots"].long() % st["page"]
        st["k"][page, :, off], st["ks"][page, :, off] = _quantise(st["k_new"])
        st["v"][page, :, off], st["vs"][page, :, off] = _quantise(st["v_new"])
    return _read(st)


def _read(st):
    if own:
        st["cache"].load(0, st["slots"], st["k_out"], st["v_out"])
        return st["k_out"], st["v_out"]
    page, off = st["slots"].long() // st["page"], st["slots"].long() % st["page"]
    return (_values(st["k"][page, :, off], st["ks"][page, :, off]).bfloat16(),
            _values(st["v"][page, :, off], st["vs"][page, :, off]).bfloat16())


def _gather(st, pos):
    """fp32 K and V [B, n, H, D] at positions pos [B, n] (clamped into the table)."""
    idx = (pos // st["page"]).clamp(0, st["bt"].shape[1] - 1)
    page = st["bt"].long().gather(1, idx).clamp(min=0)
    off = pos.clamp(min=0) % st["page"]
    return (_values(st["k"][page, :, off], st["ks"][page, :, off]), _values(st["v"][page, :, off], st["vs"][page, :, off]))


def _softmax(q, k, v, seen, sm):
    """q [B, H, r, D], k, v [B, n, H, D], seen [B, 1, r, n]: out [B, H, r, D], lse [B, H, r]."""
    s = torch.matmul(q, k.permute(0, 2, 3, 1)) * sm
    s = s.masked_fill_(~seen, float("-inf"))
    m = s.amax(-1, keepdim=True)
    m = torch.where(m == float("-inf"), 0.0, m)
    p = torch.exp(s.sub_(m))
    l = p.sum(-1, keepdim=True)
    out = torch.matmul(p, v.transpose(1, 2)) / torch.where(l > 0, l, 1.0)
    return out, (m + torch.log(l))[..., 0]


def _decode(st):
    if own:
        st["cache"].decode(0, st["q"], st["bt"], st["lens"], st["max_len"], st["out"], st["lse"], st["ws"])
        return st["out"], st["lse"]
    B, hq, D = st["q"].shape
    H, W = st["hkv"], st["window"]
    L = st["lens"].long()[:, None]
    lo = (L - W).clamp(min=0) if W else torch.zeros_like(L)
    n = min(st["max_len"], W) if W else st["max_len"]
    pos = lo + torch.arange(n, device=L.device)
    k, v = _gather(st, pos)
    out, lse = _softmax(st["q"].float().view(B, H, hq // H, D), k, v, (pos < L)[:, None, None], st["sm"])
    return out.reshape(B, hq, D).bfloat16(), lse.reshape(B, hq)


def _extend(st):
    if own:
        st["cache"].extend(0, st["q"], st["k_ext"], st["v_ext"], st["indptr"], st["prefix"], st["bt"], st["max_new"],
                           st["max_prefix"], st["out"], st["lse"])
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
    out, lse = _softmax(q, k, v, seen.repeat(1, g, 1)[:, None], st["sm"])
    out = out.view(B, H, g, -1, D).permute(0, 3, 1, 2, 4).reshape(B, -1, hq, D)
    lse = lse.view(B, H, g, -1).permute(0, 3, 1, 2).reshape(B, -1, hq)
    t = torch.arange(N, device=dev)
    b = torch.searchsorted(ptr, t, right=True) - 1
    return out[b, t - ptr[b]].bfloat16(), lse[b, t - ptr[b]]


# --------------------------------------------------- the definition in 64 bits
def _e4m3_all():
    return [(m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)) for e in range(16) for m in range(8)][:127]


def _nearest(x, grid):
    """The member of the ascending grid nearest to x >= 0, a tie to the even index."""
    at = torch.searchsorted(grid, x.contiguous()).clamp(1, len(grid) - 1)
    below, above = x - grid[at - 1], grid[at] - x
    up = (above < below) | ((above == below) & (at % 2 == 0))
    return grid[torch.where(up, at, at - 1)]


def _kept(x):
    """What the format keeps of rows x [..., D], in 64 bits."""
    x = x.double()
    a = x.abs().amax(-1).cpu().numpy()
    k = np.ceil(np.log2(np.where(a > 0, a, 1.0) / 2688)).astype(np.int64)
    k += a > np.ldexp(2688.0, k)           # log2's last bit
    k -= a <= np.ldexp(1344.0, k)
    k = np.where(a > 0, np.maximum(k, -116), -116)
    s = torch.from_numpy(np.ldexp(1.0, k)).to(x.device)[..., None, None]
    z = (x / s[..., 0]).unflatten(-1, (-1, 16))
    sb = _nearest(z.abs().amax(-1) / 6, torch.tensor(_e4m3_all(), dtype=torch.float64, device=x.device))[..., None]
    c = _nearest(torch.where(sb > 0, z.abs() / torch.where(sb > 0, sb, 1.0), 0.0).clamp(max=6.0),
                 torch.tensor(E2M1, dtype=torch.float64, device=x.device))
    return (torch.copysign(c, z) * sb * s).flatten(-2)


def _held(rows, s):
    """64-bit values of slab rows, from the bits of the two number formats."""
    D = rows.shape[-1] * 16 // 9
    b = rows[..., : D // 2]
    c = torch.stack((b & 15, b >> 4), -1).flatten(-2)
    e, m = ((c >> 1) & 3).double(), (c & 1).double()
    mag = torch.where(e == 0, m / 2, (1 + m / 2) * torch.exp2(e - 1))
    u = rows[..., D // 2:]
    e, m = ((u >> 3) & 15).double(), (u & 7).double()
    sb = torch.where(e == 0, m / 8 * 2.0 ** -6, (1 + m / 8) * torch.exp2(e - 7))
    val = torch.where(c >= 8, -mag, mag).unflatten(-1, (-1, 16)) * sb[..., None]
    return val.flatten(-2) * s.double()[..., None]


def exact(case, seed):
    st = prepare(case, seed)
    kind, ps, H, W, sm = case["kind"], case["page"], case["hkv"], case["window"], st["sm"]
    if kind == "write":
        return _kept(st["k_new"]), _kept(st["v_new"])
    if kind == "read":
        page, off = st["slots"].long() // ps, st["slots"].long() % ps
        return tuple(_held(st[n][page, :, off], st[n + "s"][page, :, off]) for n in "kv")
    ctx, new = _lens(case)
    q = st["q"].double()
    out = torch.zeros_like(q)
    lse = torch.full(q.shape[:2], float("-inf"), dtype=torch.float64, device=q.device)
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
            k, v = (_held(st[m][page, h, off], st[m + "s"][page, h, off]) for m in "kv")
            if new is not None:
                k, v = (torch.cat((x, st[m][at: at + r, h].double())) for x, m in ((k, "k_ext"), (v, "v_ext")))
            for j in range(h * g, (h + 1) * g):
                s = torch.where(seen, (q[at: at + r, j] @ k.T) * sm, float("-inf"))
                lse[at: at + r, j] = torch.logsumexp(s, -1)
                out[at: at + r, j] = torch.softmax(s, -1) @ v
        at += r
    return out, lse
