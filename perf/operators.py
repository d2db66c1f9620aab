"""The operators around the verification of drafted tokens, as they are measured: rotary positions, the paged
key/value cache (written, quantised, read back), the bookkeeping of a decoding step over a tree of drafts, and the
attention of the tree's nodes over the cache.

`run` with `own` false computes each in its plain form (elementary torch operations in 32 bits); with `own` true it makes
the calls of the package's binding.  `exact` computes the same in 64 bits from the definitions.
"""
import math

import numpy as np
import torch

own = False

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
TWO_PI_OVER_2_32 = 2.0 * math.pi / 4294967296.0


# ---------------------------------------------------------------- cases

def listed():
    return [
        # one request's chain of 3 drafts and its last token, rotated before the layer's attention: latency
        dict(name="rope_step_b1", op="rope", T=4, Hq=32, Hkv=8, D=128, rot=128, layout="half", dtype="bf16",
             scaling="none", factor=1.0, start=1900, inverse=False),
        # a long prompt, odd length, half of the head rotated, interleaved pairs, context stretched by parts
        dict(name="rope_prompt", op="rope", T=32771, Hq=32, Hkv=8, D=128, rot=64, layout="interleaved", dtype="bf16",
             scaling="by_parts", factor=8.0, start=0, inverse=False),
        # one request's tree of 32 nodes written as it is, key and query rotated on the way
        dict(name="cache_tree_b1", op="cache", T=32, Hq=32, Hkv=8, D=128, rot=128, layout="half", dtype="bf16",
             cache="bf16", page=64, start=5000),
        # 512 requests x (8 drafts + 1), keys rotated, quantised to 8 bits, read back
        dict(name="cache_fp8_b512", op="cache", T=4608, Hq=32, Hkv=8, D=128, rot=128, layout="half", dtype="bf16",
             cache="e4m3", page=64, start=0),
        # a prompt of odd length, many narrow heads, quantised, no rotation
        dict(name="cache_fp8_prompt", op="cache", T=20011, Hq=16, Hkv=16, D=64, rot=0, layout="half", dtype="f16",
             cache="e4m3", page=16, start=0),
        # after the verification: slots, positions and masks, the nodes' rows, the kept path's rows; 64 requests, chain of 4 + 1
        dict(name="step_chain_b64", op="step", B=64, N=5, Hkv=8, D=128, dtype="bf16", cache="bf16", page=64, lo=100,
             hi=4096, tree=False),
        # the same for 256 trees of up to 32 nodes in an 8-bit cache
        dict(name="step_tree_b256", op="step", B=256, N=32, Hkv=8, D=128, dtype="bf16", cache="e4m3", page=32, lo=1,
             hi=4000, tree=True),
        # one request, one token (plain decoding): latency
        dict(name="attn_token_b1", op="attn", B=1, N=1, Hq=32, Hkv=8, D=128, dtype="bf16", cache="bf16", page=16, lo=777,
             hi=777, tree=False),
        # 256 requests with 3 drafts each, ragged contexts
        dict(name="attn_chain_b256", op="attn", B=256, N=4, Hq=32, Hkv=8, D=128, dtype="bf16", cache="bf16", page=64,
             lo=64, hi=4096, tree=False),
        # trees of 32 nodes over an 8-bit cache
        dict(name="attn_tree_fp8_b32", op="attn", B=32, N=32, Hq=32, Hkv=8, D=128, dtype="bf16", cache="e4m3", page=64,
             lo=1000, hi=16384, tree=True),
        # two long contexts, 8 drafts, 8 query heads a key head
        dict(name="attn_long_b2", op="attn", B=2, N=9, Hq=64, Hkv=8, D=128, dtype="bf16", cache="bf16", page=128,
             lo=130001, hi=131063, tree=True),
        # narrow heads without sharing, odd sizes, half precision, some contexts of a token or none
        dict(name="attn_f16_odd", op="attn", B=7, N=5, Hq=12, Hkv=12, D=64, dtype="f16", cache="f16", page=16, lo=0,
             hi=5003, tree=True),
    ]


def _log(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


_CAPS = {}


def draw(rng):
    if not _CAPS:
        for c in listed():
            w = work(c)
            old = _CAPS.get(c["op"], (0, 0))
            _CAPS[c["op"]] = (max(old[0], w["bytes"]), max(old[1], w["flops"]))
    while True:
        op = rng.choice(["rope", "cache", "step", "attn", "attn"])
        D = rng.choice([64, 80, 96, 128, 128, 256])
        Hkv = rng.choice([1, 2, 4, 8, 8, 16])
        Hq = Hkv * rng.choice([1, 2, 4, 7, 8])
        dtype = rng.choice(["bf16", "bf16", "f16"])
        cache = rng.choice([dtype, "e4m3"])
        page = rng.choice([16, 32, 64, 128])
        rot = rng.choice([D, D // 2, D // 4 * 2])
        layout = rng.choice(["half", "interleaved"])
        if op == "rope":
            c = dict(op=op, T=_log(rng, 1, 32768), Hq=Hq, Hkv=Hkv, D=D, rot=rot, layout=layout,
                     dtype=rng.choice(["bf16", "f16", "f32"]), scaling=rng.choice(["none", "linear", "ntk", "by_parts"]),
                     factor=float(rng.choice([2, 4, 8, 32])), start=_log(rng, 1, 500000), inverse=rng.random() < 0.4)
            if c["scaling"] == "none":
                c["factor"] = 1.0
        elif op == "cache":
            c = dict(op=op, T=_log(rng, 1, 20000), Hq=Hq, Hkv=Hkv, D=D, rot=rng.choice([0, rot]), layout=layout,
                     dtype=dtype, cache=cache, page=page, start=_log(rng, 1, 100000))
        else:
            tree = rng.random() < 0.6
            N = rng.randint(1, 32) if tree else rng.randint(1, 9)
            hi = _log(rng, 16, 131000)
            c = dict(op=op, B=_log(rng, 1, 512), N=N, Hkv=Hkv, D=D, dtype=dtype, cache=cache, page=page,
                     lo=rng.randint(0, hi), hi=hi, tree=tree)
            if op == "attn":
                c["Hq"] = Hq
            padded = c["B"] * (c["hi"] + N)     # what the plain form gathers
            if padded > (1 << 21) or (op == "step" and padded * Hkv * D > (1 << 30)):
                continue
        w = work(c)
        if w["bytes"] <= _CAPS[op][0] and w["flops"] <= _CAPS[op][1]:
            return c


def _contexts(case):
    """Committed tokens of each request: spread evenly over [lo, hi], the first at hi."""
    B, lo, hi = case["B"], case["lo"], case["hi"]
    return [lo + int(round((hi - lo) * ((1.0 - b * 0.6180339887) % 1.0 or 1.0))) for b in range(B)]


def _nodes(case):
    """Nodes of each request: a tree has all of them or fewer, a chain its drafts and the last token."""
    N = case["N"]
    return [N - (b * 5) % (N // 2 + 1) if N > 1 else 1 for b in range(case["B"])]


def _last(m):
    """The last kept node of m: the kept path ends in the middle of each tree."""
    return (m + 1) // 2 - 1


def _item(case, which):
    return {"bf16": 2, "f16": 2, "f32": 4, "e4m3": 1}[case[which]]


def work(case):
    op, D = case["op"], case["D"]
    if op == "rope":
        n = case["T"] * (case["Hq"] + case["Hkv"])
        return {"bytes": 2 * n * D * _item(case, "dtype") + 4 * case["T"], "flops": 3 * n * case["rot"]}
    Hkv = case["Hkv"]
    row = Hkv * (D * _item(case, "cache") + (1 if case["cache"] == "e4m3" else 0))  # a token's keys (or values) in the cache
    src = Hkv * D * _item(case, "dtype")
    if op == "cache":
        T, qb = case["T"], case["Hq"] * D * _item(case, "dtype") if case["rot"] else 0
        # written: k and v in, cache rows out, q in and out; read back: cache rows in, k and v out
        return {"bytes": T * (2 * src + 2 * row + 2 * qb + 8 + 2 * row + 2 * src + 8),
                "flops": T * (3 * case["rot"] * (case["Hq"] + Hkv) + 4 * Hkv * D)}
    n, ctx = _nodes(case), _contexts(case)
    pages = sum(-(-(c + m) // case["page"]) for c, m in zip(ctx, n))
    if op == "step":
        t = sum(n)
        moved, par = 0, _parents(case)                  # nodes of the kept paths that are not in their place already
        for b, m in enumerate(n):
            path = [_last(m)]
            while path[-1] > 0:
                path.append(int(par[b, path[-1]]))
            moved += sum(u != d for d, u in enumerate(reversed(path)))
        return {"bytes": t * (2 * src + 2 * row) + 4 * moved * row + t * (2 * row + 2 * src)
                + case["B"] * case["N"] * (4 + 4 + 8 + 4) + 4 * pages, "flops": 4 * t * Hkv * D}
    Hq = case["Hq"]
    keys = sum(ctx) + sum(n)
    pairs = sum(c * m + m * (m + 1) // 2 for c, m in zip(ctx, n))
    return {"bytes": 2 * keys * row + 2 * case["B"] * case["N"] * Hq * D * _item(case, "dtype") + 4 * pages,
            "flops": 4 * pairs * Hq * D}


# ---------------------------------------------------------------- inputs

def _thetas(rot, scaling, factor, base=10000.0, original=4096.0, fast=32.0, slow=1.0):
    """The angle per position of each pair, and the factor on the rotated values."""
    if scaling == "ntk":
        base = base * factor ** (rot / max(1, rot - 2))
    out = []
    for i in range(rot // 2):
        t = base ** (-2.0 * i / rot)
        if scaling == "linear":
            t = t / factor
        elif scaling == "by_parts":
            g = min(1.0, max(0.0, (original * t / (2.0 * math.pi) - slow) / (fast - slow)))
            t = t * ((1.0 - g) / factor + g)
        out.append(t)
    return out, (0.1 * math.log(factor) + 1.0 if scaling == "by_parts" and factor > 1 else 1.0)


def _turns(thetas, dev):
    """Turns per position as 64-bit fractions: the product with a position wraps to the exact phase."""
    v = [int(t / (2.0 * math.pi) * 2.0 ** 64) & (2 ** 64 - 1) for t in thetas]
    return torch.tensor([x - 2 ** 64 if x >= 2 ** 63 else x for x in v], dtype=torch.int64, device=dev)


def _parents(case):
    """A trie whose node c hangs under one of the few nodes before it, or a chain."""
    N = case["N"]
    out = np.full((case["B"], N), -1, np.int32)
    for b in range(case["B"]):
        for c in range(1, N):
            out[b, c] = max(0, c - 1 - (b * 7 + c * 3) % 4) if case["tree"] else c - 1
    return out


def _new_cache(pages, Hkv, page, D, kind, g, dev, fill):
    if kind == "e4m3":
        k = torch.empty((2, pages, Hkv, page, D), dtype=torch.uint8, device=dev)
        s = torch.full((2, pages, Hkv, page), 127, dtype=torch.uint8, device=dev)
        if fill:  # values of 8 bits below the type's NaN pattern, scales of a few binades
            k.copy_(torch.randint(0, 104, k.shape, generator=g, dtype=torch.uint8, device=dev))
            k |= torch.randint(0, 2, k.shape, generator=g, dtype=torch.uint8, device=dev) << 7
            s.copy_(torch.randint(117, 121, s.shape, generator=g, dtype=torch.uint8, device=dev))
        return k[0], k[1], s[0], s[1]
    k = torch.empty((2, pages, Hkv, page, D), dtype=DT[kind], device=dev)
    if fill:
        k.normal_(generator=g)
    return k[0], k[1], None, None


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(int(seed))
    op, D = case["op"], case["D"]
    dt = DT[case["dtype"]]
    s = {"case": dict(case)}
    if own:
        from speculative_decoding_verification_51_gb300 import binding
        s["binding"] = binding
    if op in ("rope", "cache"):
        T = case["T"]
        s["positions"] = (case["start"] + torch.arange(T, device=dev)).to(torch.int32)
        s["q"] = torch.randn((T, case["Hq"], D), generator=g, device=dev).to(dt)
        s["k"] = torch.randn((T, case["Hkv"], D), generator=g, device=dev).to(dt)
        if case["rot"]:
            scaling, factor = case.get("scaling", "none"), case.get("factor", 1.0)
            if own:
                s["table"] = s["binding"].rope_table(case["rot"], layout=case["layout"], scaling=scaling,
                                                     factor=factor, original_len=4096, device=dev)
            else:
                th, s["mscale"] = _thetas(case["rot"], scaling, factor)
                s["turns"] = _turns(th, dev)
    if op == "cache":
        page = case["page"]
        pages = -(-T // page) + 2
        s["v"] = torch.randn((T, case["Hkv"], D), generator=g, device=dev).to(dt)
        slots = torch.randperm((pages - 1) * page, generator=g, device=dev)[:T].to(torch.int64)
        slots[torch.arange(T, device=dev) % 17 == 16] = -1     # rows of finished requests: not written
        s["slots"] = slots
        s["cache"] = _new_cache(pages, case["Hkv"], page, D, case["cache"], g, dev, False)
    if op in ("step", "attn"):
        B, N, Hkv, page = case["B"], case["N"], case["Hkv"], case["page"]
        ctx, n = _contexts(case), _nodes(case)
        need = [-(-(c + m) // page) for c, m in zip(ctx, n)]
        width, total = max(need), sum(need)
        perm = torch.randperm(total, generator=g, device=dev).to(torch.int32)
        cell = np.full((B, width), -1, np.int64)
        at = 0
        for b in range(B):
            cell[b, :need[b]] = np.arange(at, at + need[b])
            at += need[b]
        cell = torch.from_numpy(cell).to(dev)
        s["page_table"] = torch.where(cell >= 0, perm[cell.clamp(min=0)], torch.full_like(perm[cell.clamp(min=0)], -1))
        par = _parents(case)
        s["parents"] = torch.from_numpy(par).to(dev)
        s["nodes"] = torch.tensor(n, dtype=torch.int32, device=dev)
        s["ctx"] = torch.tensor(ctx, dtype=torch.int32, device=dev)
        s["cache"] = _new_cache(total + (1 if op == "step" else 0), Hkv, page, D, case["cache"], g, dev, op == "attn")
        if op == "step":
            s["k"] = torch.randn((B, N, Hkv, D), generator=g, device=dev).to(dt)
            s["v"] = torch.randn((B, N, Hkv, D), generator=g, device=dev).to(dt)
            s["last"] = torch.tensor([_last(m) for m in n], dtype=torch.int32, device=dev)
        else:
            s["q"] = (2.0 * torch.randn((B, N, case["Hq"], D), generator=g, device=dev)).to(dt)
    if own and "cache" in s:
        s["cache"] = s["binding"].KVCache(*s["cache"])
        if op == "attn":  # one plan serves every layer of a step
            s["plan"] = s["binding"].tree_plan(s["parents"], s["nodes"], s["ctx"], s["page_table"], s["cache"])
    return s


# ---------------------------------------------------------------- plain forms

def _rotate(x, positions, turns, mscale, layout, sign=1.0):
    """x [T, H, D]: the first 2 * len(turns) channels rotated, in 32 bits."""
    rot = 2 * turns.numel()
    phase = (positions.to(torch.int64)[:, None] * turns[None, :]) >> 32        # signed 32-bit fraction of a turn
    ang = phase.to(torch.float32) * TWO_PI_OVER_2_32
    c, s = (torch.cos(ang) * mscale)[:, None], (torch.sin(ang) * (mscale * sign))[:, None]
    x = x.float()
    if layout == "half":
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        return torch.cat((a * c - b * s, a * s + b * c, x[..., rot:]), -1)
    a, b = x[..., 0:rot:2], x[..., 1:rot:2]
    return torch.cat((torch.stack((a * c - b * s, a * s + b * c), -1).flatten(-2), x[..., rot:]), -1)


def _quantise(x):
    """(bytes, scale bytes): the power of two that brings a row's largest value to 448 or less, and e4m3 values."""
    amax = x.abs().amax(-1)
    m, e = torch.frexp(amax / 448.0)
    e = torch.where(m == 0.5, e - 1, e)                  # amax <= 448 * 2^e
    e = torch.where(amax > 0, e, torch.zeros_like(e)).clamp(-126, 127)
    y = torch.ldexp(x, -e[..., None])
    return y.to(torch.float8_e4m3fn).view(torch.uint8), (e + 127).to(torch.uint8)


def _values(k, s):
    """Cache contents as 32-bit values."""
    if s is None:
        return k.float()
    return torch.ldexp(k.view(torch.float8_e4m3fn).float(), (s.to(torch.int32) - 127)[..., None])


def _write(c, sc, at, page, x):
    """Rows x [T, Hkv, D] to the slots `at` of one cache tensor."""
    p, o = at // page, at % page
    if sc is None:
        c[p, :, o] = x.to(c.dtype)
    else:
        c[p, :, o], sc[p, :, o] = _quantise(x.float())


def _read(c, sc, at, page, dt):
    p, o = at // page, at % page
    return _values(c[p, :, o], None if sc is None else sc[p, :, o]).to(dt)


def _closure(parents):
    """[B, N, N]: whether u is v or above it (N <= 32: paths double five times)."""
    B, N = parents.shape
    eye = torch.eye(N, device=parents.device)
    one = (parents.clamp(min=0).long()[..., None] == torch.arange(N, device=parents.device)).float()
    one = torch.where((parents >= 0)[..., None], one, torch.zeros_like(one))
    a = (eye + one).clamp(max=1)
    a = (a @ a).clamp(max=1)
    a = (a @ a).clamp(max=1)
    a = (a @ a).clamp(max=1)
    a = (a @ a).clamp(max=1)
    return (a @ a).clamp(max=1) > 0


def _tables(s, page):
    """Positions, slots and ancestor masks of the nodes (a missing node: 0, -1 and no ancestor)."""
    B, N = s["parents"].shape
    dev = s["parents"].device
    i = torch.arange(N, device=dev)
    there = i[None] < s["nodes"][:, None]
    up = _closure(s["parents"]) & there[:, :, None]
    depth = up.sum(-1) - 1
    pos = torch.where(there, s["ctx"][:, None] + depth, torch.zeros_like(depth)).to(torch.int32)
    t = s["ctx"].long()[:, None] + i[None]
    pg = torch.gather(s["page_table"].long(), 1, (t // page).clamp(max=s["page_table"].shape[1] - 1))
    slots = torch.where(there, pg * page + t % page, torch.full_like(t, -1))
    m = (up.long() << i[None, None]).sum(-1)
    masks = torch.where(m >= 2 ** 31, m - 2 ** 32, m).to(torch.int32)
    return pos, slots, masks, up, depth


def _plain(s):
    case = s["case"]
    op = case["op"]
    if op == "rope":
        a = (s["positions"], s["turns"], s["mscale"], case["layout"], -1.0 if case["inverse"] else 1.0)
        return _rotate(s["q"], *a).to(s["q"].dtype), _rotate(s["k"], *a).to(s["k"].dtype)
    page, dt = case["page"], DT[case["dtype"]]
    ck, cv, sk, sv = s["cache"]
    if op == "cache":
        q, k = s["q"], s["k"]
        if case["rot"]:
            a = (s["positions"], s["turns"], s["mscale"], case["layout"])
            q, k = _rotate(q, *a).to(dt), _rotate(k, *a)
        spare = (ck.shape[0] - 1) * page                # a page that no slot names takes the rows not written
        at = torch.where(s["slots"] >= 0, s["slots"], torch.full_like(s["slots"], spare))
        _write(ck, sk, at, page, k)
        _write(cv, sv, at, page, s["v"])
        keep = (s["slots"] >= 0)[:, None, None]
        k, v = _read(ck, sk, at, page, dt), _read(cv, sv, at, page, dt)
        k, v = torch.where(keep, k, torch.zeros_like(k)), torch.where(keep, v, torch.zeros_like(v))
        return (q, k, v) if case["rot"] else (k, v)
    if op == "step":
        B, N = s["parents"].shape
        pos, slots, masks, up, depth = _tables(s, page)
        spare = (ck.shape[0] - 1) * page
        at = torch.where(slots >= 0, slots, torch.full_like(slots, spare)).flatten()
        _write(ck, sk, at, page, s["k"].flatten(0, 1))
        _write(cv, sv, at, page, s["v"].flatten(0, 1))
        # row i takes the kept path's node of depth i, the rows after the path keep their own
        i = torch.arange(N, device=slots.device).expand(B, N)
        path = torch.gather(up, 1, s["last"].long()[:, None, None].expand(B, 1, N))[:, 0]
        to = torch.where(path, depth, torch.full_like(depth, N))
        src = torch.cat((i, i[:, :1]), 1).scatter(1, to, i)[:, :N]
        frm = torch.gather(at.view(B, N), 1, src).flatten()
        p, o, pf, of = at // page, at % page, frm // page, frm % page
        ck[p, :, o] = ck[pf, :, of]
        cv[p, :, o] = cv[pf, :, of]
        if sk is not None:
            sk[p, :, o] = sk[pf, :, of]
            sv[p, :, o] = sv[pf, :, of]
        new = s["ctx"] + torch.gather(depth, 1, s["last"].long()[:, None])[:, 0].to(torch.int32) + 1
        keep = (slots >= 0)[..., None, None]
        k = _read(ck, sk, at, page, dt).view(B, N, *s["k"].shape[2:])
        v = _read(cv, sv, at, page, dt).view(B, N, *s["v"].shape[2:])
        return (pos, slots, masks, new, torch.where(keep, k, torch.zeros_like(k)),
                torch.where(keep, v, torch.zeros_like(v)))
    # attention: every request's pages side by side, as long as the longest
    B, N, Hq, D = s["q"].shape
    Hkv, G = case["Hkv"], Hq // case["Hkv"]
    tab = s["page_table"].clamp(min=0).long()
    L = tab.shape[1] * page
    K = _values(ck[tab], None if sk is None else sk[tab]).transpose(1, 2).reshape(B, Hkv, L, D)
    V = _values(cv[tab], None if sv is None else sv[tab]).transpose(1, 2).reshape(B, Hkv, L, D)
    q = s["q"].float().view(B, N, Hkv, G, D).permute(0, 2, 1, 3, 4).reshape(B, Hkv, N * G, D)
    score = (q @ K.transpose(-1, -2)).mul_(1.0 / math.sqrt(D)).view(B, Hkv, N, G, L)
    up = _tables(s, page)[3]
    t = torch.arange(L, device=q.device)
    u = t[None] - s["ctx"][:, None]                     # node index of each token of the cache
    seen = (u < 0)[:, None] | (torch.gather(up, 2, u.clamp(0, N - 1)[:, None].expand(B, N, L)) & ((u >= 0) & (u < N))[:, None])
    there = (torch.arange(N, device=q.device)[None] < s["nodes"][:, None])
    seen = seen & there[..., None]
    score.masked_fill_(~seen[:, None, :, None], -math.inf)
    top = score.amax(-1, keepdim=True)
    p = score.sub_(torch.where(torch.isfinite(top), top, torch.zeros_like(top))).exp_()
    tot = p.sum(-1, keepdim=True)
    V = torch.where((t[None] < (s["ctx"] + s["nodes"])[:, None])[:, None, :, None], V, torch.zeros_like(V))
    out = (p.view(B, Hkv, N * G, L) @ V).view(B, Hkv, N, G, D) / torch.where(tot > 0, tot, torch.ones_like(tot))
    return out.permute(0, 2, 1, 3, 4).reshape(B, N, Hq, D).to(s["q"].dtype)


def _own(s):
    b, case = s["binding"], s["case"]
    op = case["op"]
    if op == "rope":
        return b.rope(s["q"], s["k"], s["positions"], s["table"], inverse=case["inverse"])
    if op == "cache":
        q = None
        if case["rot"]:
            q = b.kv_write(s["cache"], s["k"], s["v"], s["slots"], positions=s["positions"], table=s["table"], q=s["q"])
        else:
            b.kv_write(s["cache"], s["k"], s["v"], s["slots"])
        k, v = b.kv_read(s["cache"], s["slots"], dtype=DT[case["dtype"]])
        return (q, k, v) if case["rot"] else (k, v)
    if op == "step":
        plan = b.tree_plan(s["parents"], s["nodes"], s["ctx"], s["page_table"], s["cache"])
        b.kv_write(s["cache"], s["k"], s["v"], plan.slots)
        new = b.kv_commit([s["cache"]], plan, s["last"])
        k, v = b.kv_read(s["cache"], plan.slots, dtype=DT[case["dtype"]])
        return plan.positions, plan.slots, plan.masks, new, k, v
    return b.tree_attention(s["q"], s["cache"], s["plan"])


def run(state):
    return _own(state) if own else _plain(state)


# ---------------------------------------------------------------- 64 bits

def _exact_rotate(x, pos, case, sign=1.0):
    th, ms = _thetas(case["rot"], case.get("scaling", "none"), case.get("factor", 1.0))
    x = x.double().clone()
    ang = pos.double()[:, None, None] * torch.tensor(th, dtype=torch.float64, device=x.device)
    z = torch.polar(torch.full_like(ang, ms), sign * ang)
    h = case["rot"] // 2
    if case["layout"] == "half":
        w = torch.complex(x[..., :h].contiguous(), x[..., h:2 * h].contiguous()) * z
        x[..., :h], x[..., h:2 * h] = w.real, w.imag
    else:
        w = torch.complex(x[..., 0:2 * h:2].contiguous(), x[..., 1:2 * h:2].contiguous()) * z
        x[..., 0:2 * h:2], x[..., 1:2 * h:2] = w.real, w.imag
    return x


def _exact_e4m3(x):
    """x (64 bits) as the 8-bit cache holds it: 4 significant bits, steps of 2^-9 at least, times a power of two a row."""
    top = x.abs().amax(-1, keepdim=True)
    e = torch.where(top > 0, torch.ceil(torch.log2(torch.where(top > 0, top, torch.ones_like(top)) / 448.0)), torch.zeros_like(top))
    e = torch.where(top > 448.0 * torch.exp2(e), e + 1, e)
    e = torch.where((top > 0) & (top <= 224.0 * torch.exp2(e)), e - 1, e).clamp(-126, 127)
    y = x * torch.exp2(-e)
    step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.round(y / step) * step * torch.exp2(e)


def _exact_held(x, case):
    if case["cache"] == "e4m3":
        return _exact_e4m3(x)
    return x


def _exact_attention(s, case):
    ck, cv, sk, sv = s["cache"]
    B, N, Hq, D = s["q"].shape
    G, page = Hq // case["Hkv"], case["page"]
    ctx, n, par = _contexts(case), _nodes(case), _parents(case)
    out = torch.zeros((B, N, Hq, D), dtype=torch.float64, device=s["q"].device)

    def rows(c, sc, pages, count):
        x = c[pages].transpose(1, 2).reshape(-1, case["Hkv"], D)[:count]
        if sc is None:
            return x.double()
        e = sc[pages].transpose(1, 2).reshape(-1, case["Hkv"])[:count].double() - 127.0
        b = x.long()
        ex, man = (b >> 3) & 15, (b & 7).double()
        val = torch.where(ex == 0, man * 2.0 ** -9, (1 + man / 8) * torch.exp2(ex.double() - 7))
        return torch.where(b >= 128, -val, val) * torch.exp2(e)[..., None]

    for b in range(B):
        count = ctx[b] + n[b]
        pages = s["page_table"][b, :-(-count // page)].long()
        K, V = rows(ck, sk, pages, count), rows(cv, sv, pages, count)
        seen = np.zeros((n[b], n[b]), bool)
        for v in range(n[b]):
            u = v
            while u >= 0:
                seen[v, u] = True
                u = int(par[b, u])
        seen = torch.from_numpy(seen).to(K.device)
        for h in range(case["Hkv"]):
            q = s["q"][b, :n[b], h * G:(h + 1) * G].double()              # [n, G, D]
            z = torch.einsum("ngd,ld->ngl", q, K[:, h]) / math.sqrt(D)
            z[:, :, ctx[b]:] = torch.where(seen[:, None, :], z[:, :, ctx[b]:], torch.full_like(z[:, :, ctx[b]:], -math.inf))
            out[b, :n[b], h * G:(h + 1) * G] = torch.einsum("ngl,ld->ngd", torch.softmax(z, -1), V[:, h])
    return out


def exact(case, seed):
    if case["op"] in ("step", "attn") and work(case)["flops"] > 4e11:
        return None
    s = prepare(case, seed)
    s["cache"] = (s["cache"].k, s["cache"].v, s["cache"].k_scale, s["cache"].v_scale) if own and "cache" in s else s.get("cache")
    op = case["op"]
    if op == "rope":
        sign = -1.0 if case["inverse"] else 1.0
        return _exact_rotate(s["q"], s["positions"], case, sign), _exact_rotate(s["k"], s["positions"], case, sign)
    if op == "cache":
        keep = (s["slots"] >= 0)[:, None, None]
        k = _exact_rotate(s["k"], s["positions"], case) if case["rot"] else s["k"].double()
        k = _exact_held(k, case) * keep
        v = _exact_held(s["v"].double(), case) * keep
        return (_exact_rotate(s["q"], s["positions"], case), k, v) if case["rot"] else (k, v)
    if op == "attn":
        return _exact_attention(s, case)
    # the step: node by node on the host
    B, N, page = case["B"], case["N"], case["page"]
    ctx, n, par = _contexts(case), _nodes(case), _parents(case)
    tab = s["page_table"].cpu().numpy()
    last = s["last"].cpu().numpy()
    kx, vx = _exact_held(s["k"].double(), case), _exact_held(s["v"].double(), case)
    pos, slots, masks = np.zeros((B, N), np.int32), np.full((B, N), -1, np.int64), np.zeros((B, N), np.int64)
    new = np.zeros(B, np.int32)
    rows = np.tile(np.arange(N), (B, 1))
    for b in range(B):
        depth = [0] * N
        for v in range(n[b]):
            depth[v] = 0 if v == 0 else depth[par[b, v]] + 1
            masks[b, v] = (1 << v) | (masks[b, par[b, v]] if v else 0)
            pos[b, v] = ctx[b] + depth[v]
            slots[b, v] = int(tab[b, (ctx[b] + v) // page]) * page + (ctx[b] + v) % page
        u = int(last[b])
        new[b] = ctx[b] + depth[u] + 1
        while u >= 0:
            rows[b, depth[u]] = u
            u = int(par[b, u])
    dev = kx.device
    at = torch.from_numpy(rows).to(dev)[..., None, None].expand_as(kx)
    there = torch.tensor([[v < n[b] for v in range(N)] for b in range(B)], device=dev)[..., None, None]
    masks = np.where(masks >= 2 ** 31, masks - 2 ** 32, masks).astype(np.int32)
    return (torch.from_numpy(pos), torch.from_numpy(slots), torch.from_numpy(masks), torch.from_numpy(new),
            torch.gather(kx, 1, at) * there, torch.gather(vx, 1, at) * there)
