"""Plain 64-bit forms of the operators around the verification, for the tests:
rotary positions, e4m3 rows, the step's plan, attention over a paged cache."""
from __future__ import annotations

import math

import numpy as np
import torch

# unit roundoff (2^-p for a significand of p bits) and half the least subnormal
U = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
TINY = {torch.float32: 2.0 ** -150, torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25}


def thetas(rot, base=10000.0, scaling="none", factor=1.0, original_len=0.0, fast=32.0, slow=1.0):
    if scaling == "ntk":
        base = base * factor ** (rot / max(1, rot - 2))
    th = np.array([base ** (-2.0 * i / rot) for i in range(rot // 2)])
    if scaling == "linear":
        th = th / factor
    scale = 1.0
    if scaling == "by_parts":
        g = np.clip((original_len * th / (2 * math.pi) - slow) / (fast - slow), 0.0, 1.0)
        th = th * ((1 - g) / factor + g)
        scale = 0.1 * math.log(factor) + 1.0
    return th, scale


def rotate(x, pos, th, layout, scale=1.0, inverse=False):
    """x [T, H, D] and pos [T] (any types), in float64."""
    x = x.detach().cpu().double()
    ang = pos.detach().cpu().double()[:, None, None] * torch.from_numpy(th)
    c, s = torch.cos(ang) * scale, torch.sin(ang) * scale * (-1 if inverse else 1)
    r = 2 * len(th)
    y = x.clone()
    if layout == "half":
        a, b = x[..., :r // 2], x[..., r // 2:r]
        y[..., :r // 2], y[..., r // 2:r] = a * c - b * s, a * s + b * c
    else:
        a, b = x[..., 0:r:2], x[..., 1:r:2]
        y[..., 0:r:2], y[..., 1:r:2] = a * c - b * s, a * s + b * c
    return y


def rotate_bound(x, th, layout, dtype, scale=1.0):
    """How far a float32 rotation, rounded once, may be from `rotate`: the
    phase as a float32 fraction of a turn and the sine within 2 ulp give
    (2^-24 pi + 2^-22) of |a| + |b|, three float32 roundings 3 * 2^-24 more;
    then the result's own rounding."""
    x = x.detach().cpu().double().abs()
    r = 2 * len(th)
    m = torch.zeros_like(x)
    if layout == "half":
        s = x[..., :r // 2] + x[..., r // 2:r]
        m[..., :r // 2], m[..., r // 2:r] = s, s
    else:
        s = x[..., 0:r:2] + x[..., 1:r:2]
        m[..., 0:r:2], m[..., 1:r:2] = s, s
    return scale * m * ((math.pi + 4 + 3) * 2.0 ** -24 + U[dtype]) + TINY[dtype]


def e4m3_values(x):
    """Rows of x (last dimension) as an e4m3 cache holds them, float64: (values,
    exponents).  Infinities and NaN become NaN and do not count for the max."""
    x = np.asarray(x, np.float64)
    fin = np.isfinite(x)
    amax = np.where(fin, np.abs(x), 0.0).max(-1, keepdims=True)
    m, e = np.frexp(np.where(amax > 0, amax, 1.0) / 448.0)   # amax / 448 = m 2^e, m in [0.5, 1)
    e = np.where(m == 0.5, e - 1, e)
    e = np.where(amax > 0, np.clip(e, -126, 127), -126).astype(np.int64)
    y = np.where(fin, x, 0.0) * np.exp2(-e.astype(np.float64))
    _, k = np.frexp(y)
    step = np.exp2(np.maximum(k - 1, -6) - 3.0)
    v = np.rint(y / step) * step * np.exp2(e.astype(np.float64))
    return np.where(fin, v, np.nan), e[..., 0]


def plan(parents, nodes, ctx, table, page, num_pages):
    """(positions, slots, masks, ok [B]) of spec_tree_plan."""
    B, N = parents.shape
    pos, slots = np.zeros((B, N), np.int32), np.full((B, N), -1, np.int64)
    masks, ok = np.zeros((B, N), np.uint32), np.ones(B, bool)
    for b in range(B):
        n, c = int(nodes[b]), int(ctx[b])
        if not 1 <= n <= N or c < 0 or c + n > table.shape[1] * page:
            ok[b] = False
            continue
        used = table[b, :-(-(c + n) // page)]
        if (used < 0).any() or (used >= num_pages).any():
            ok[b] = False
            continue
        if any(not 0 <= parents[b, v] < v for v in range(1, n)):
            ok[b] = False
            continue
        depth = [0] * n
        for v in range(n):
            m = np.uint32(1 << v)
            if v:
                depth[v] = depth[parents[b, v]] + 1
                m |= masks[b, parents[b, v]]
            masks[b, v] = m
            pos[b, v] = c + depth[v]
            slots[b, v] = int(table[b, (c + v) // page]) * page + (c + v) % page
    return pos, slots, masks, ok


def cache_rows(cache, pages, count):
    """The first `count` rows of a list of pages, float64 [count, heads, D]: (k, v)."""
    out = []
    for t, sc in ((cache.k, cache.k_scale), (cache.v, cache.v_scale)):
        x = t[pages]
        if sc is not None:
            x = x.view(torch.float8_e4m3fn).to(torch.float32).double()
            x = x * torch.exp2(sc[pages].double() - 127.0)[..., None]
        x = x.double().transpose(1, 2).reshape(-1, t.shape[1], t.shape[3])
        out.append(x[:count])
    return out


def attention(q, cache, table, ctx, nodes, masks, scale):
    """float64 (out, lse, bound) of spec_tree_attention, bound the error that
    the kernel's roundings allow (see tolerance below)."""
    B, N, Hq, D = q.shape
    G = Hq // cache.heads
    dev = q.device
    out = torch.zeros((B, N, Hq, D), dtype=torch.float64, device=dev)
    bound = torch.zeros_like(out)
    lse = torch.full((B, N, Hq), -math.inf, dtype=torch.float64, device=dev)
    e4 = cache.k_scale is not None
    for b in range(B):
        n, c = int(nodes[b]), int(ctx[b])
        if n <= 0:
            continue
        pages = table[b, :-(-(c + n) // cache.page_size)].long()
        K, V = cache_rows(cache, pages, c + n)
        seen = torch.ones((n, c + n), dtype=torch.bool, device=dev)
        for v in range(n):
            for u in range(n):
                seen[v, c + u] = bool(int(masks[b, v]) >> u & 1)
        for h in range(cache.heads):
            qq = q[b, :n, h * G:(h + 1) * G].double()
            none = ~seen.any(-1)
            s = torch.einsum("ngd,td->ngt", qq, K[:, h]) * scale
            # float32 sums of exact products, the scale and log2(e): 2^-22 of
            # the absolute sum covers 4 roundings; f16 queries and keys of an
            # e4m3 cache are exact down to 2^-24 of the row's largest
            mag = torch.einsum("ngd,td->ngt", qq.abs(), torch.nan_to_num(K[:, h], 0, 0, 0).abs()) * abs(scale)
            if e4:
                mag = mag + 4 * qq.abs().amax(-1, keepdim=True) * abs(scale) * torch.nan_to_num(K[:, h], 0, 0, 0).abs().sum(-1)
            s = torch.where(seen[:, None], s, torch.full_like(s, -math.inf))
            ds = torch.where(seen[:, None], mag, torch.zeros_like(mag)).amax(-1) * 2.0 ** -22
            top = s.amax(-1, keepdim=True)
            top = torch.where(torch.isfinite(top), top, torch.zeros_like(top))
            # a token that is not seen has no part in the sum, whatever it holds
            w = torch.where(seen[:, None], torch.exp(s - top), torch.zeros_like(s))
            tot = w.sum(-1)
            p = w / torch.where(tot > 0, tot, torch.ones_like(tot))[..., None]
            o = torch.zeros((n, G, D), dtype=torch.float64, device=dev)
            for v in range(n):
                if not none[v]:
                    o[v] = p[v][:, seen[v]] @ V[seen[v], h]
            out[b, :n, h * G:(h + 1) * G] = o
            lse[b, :n, h * G:(h + 1) * G] = torch.where(tot > 0, top[..., 0] + torch.log(tot), torch.full_like(tot, -math.inf))
            va = torch.nan_to_num(V[:, h], 0, 0, 0).abs()
            pv = torch.einsum("ngt,td->ngd", torch.nan_to_num(p), va)
            uw = U[q.dtype]  # weights are rounded to q's type, or to f16
            bd = pv * (uw + 2 * ds[..., None] + 2.0 ** -19)
            if e4:  # f16 weights below 2^-14 of the largest contribution
                big = (torch.nan_to_num(p) * va.amax(-1)).amax(-1)
                bd = bd + (c + n) * 2.0 ** -24 * 2 * big[..., None]
            elif q.dtype == torch.float16:
                bd = bd + (c + n) * 2.0 ** -24 * va.amax() * torch.nan_to_num(p).amax(-1)[..., None]
            bound[b, :n, h * G:(h + 1) * G] = bd
    bound = bound + U[q.dtype] * (out.nan_to_num(0, 0, 0).abs() + bound) + TINY[q.dtype]
    return out, lse, bound


def make_table(rng, ctx, nodes, page, spare=3):
    """A page table with the requests' pages in random order: (table, pages)."""
    need = [max(1, -(-(int(c) + max(int(n), 0)) // page)) for c, n in zip(ctx, nodes)]
    total = sum(need) + spare
    perm = rng.permutation(total)
    table = np.full((len(need), max(need)), -1, np.int32)
    at = 0
    for b, k in enumerate(need):
        table[b, :k] = perm[at:at + k]
        at += k
    return table, total


def random_tree(rng, B, N, width=4):
    par = np.full((B, N), -1, np.int32)
    for b in range(B):
        for c in range(1, N):
            par[b, c] = rng.integers(max(0, c - width), c)
    return par
