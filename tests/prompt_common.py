"""Plain 64-bit forms of the prompt's pass and of token log probabilities, for the tests."""
from __future__ import annotations

import math

import torch

from nodes_common import TINY, U


def norm(x, w, eps):
    """x [..., D]: each row over the root of its mean square, times w, in float64 on the CPU."""
    x = x.detach().cpu().double()
    y = x / torch.sqrt(x.square().mean(-1, keepdim=True) + eps)
    return y if w is None else y * w.detach().cpu().double()


def norm_bound(y, D):
    """How far a float32 norm is from `norm`, relative to the normalised value: the sum of D squares (D + 1 roundings,
    halved by the root), the mean and eps (2), the root (2 ulp: 2 * 2^-23), two products."""
    return y.abs() * ((D + 1) / 2 + 1 + 4 + 2) * 2.0 ** -24


def offsets(lens, first=0):
    out = [first]
    for n in lens:
        out.append(out[-1] + n)
    return out


def attention(q, k, v, off, koff, scale, window=0):
    """float64 (out, lse, bound, lse_bound) of spec_prompt_attention; rows of no prompt are NaN in all of them."""
    T, Hq, D = q.shape
    Hkv = k.shape[1]
    G = Hq // Hkv
    dev = q.device
    out = torch.full((T, Hq, D), math.nan, dtype=torch.float64, device=dev)
    bound = torch.full_like(out, math.nan)
    lse = torch.full((T, Hq), math.nan, dtype=torch.float64, device=dev)
    lse_bound = torch.full_like(lse, math.nan)
    for b in range(len(off) - 1):
        a, n, ka, m = off[b], off[b + 1] - off[b], koff[b], koff[b + 1] - koff[b]
        if n == 0:
            continue
        i, j = torch.arange(n, device=dev)[:, None] + (m - n), torch.arange(m, device=dev)[None]
        seen = j <= i
        if window:
            seen &= j > i - window
        for h in range(Hq):
            qq, K, V = q[a:a + n, h].double(), k[ka:ka + m, h // G].double(), v[ka:ka + m, h // G].double()
            s = qq @ K.T * scale
            # float32 sums of exact products, the scale and log2(e): 2^-22 of the absolute sum covers 4 roundings,
            # and D / 16 steps of the tensor cores' sums
            mag = (qq.nan_to_num(0, 0, 0).abs() @ K.nan_to_num(0, 0, 0).abs().T) * scale
            ds = (torch.where(seen, mag, torch.zeros_like(mag)).amax(-1) if m else torch.zeros(n, dtype=torch.float64, device=dev)) * (2.0 ** -22 + D / 16 * 2.0 ** -23)
            s = torch.where(seen, s, torch.full_like(s, -math.inf))
            none = ~seen.any(-1) if m else torch.ones(n, dtype=torch.bool, device=dev)
            top = s.amax(-1) if m else torch.full((n,), -math.inf, dtype=torch.float64, device=dev)
            top = torch.where(none, torch.zeros_like(top), top)
            w = torch.where(seen, torch.exp(s - top[:, None]), torch.zeros_like(s))
            tot = w.sum(-1)
            p = w / torch.where(none, torch.ones_like(tot), tot)[:, None]
            # a key that is not seen has no part in the sum, whatever it holds
            finite = V.isfinite()
            o = p @ torch.where(finite, V, torch.zeros_like(V))
            for key in (~finite).any(-1).nonzero()[:, 0].tolist():
                o = torch.where((seen[:, key] & ~none)[:, None], o + torch.where(finite[key], torch.zeros_like(V[key]), V[key]), o)
            out[a:a + n, h] = o
            lse[a:a + n, h] = torch.where(none, torch.full_like(tot, -math.inf), top + torch.log(tot))
            va = torch.where(finite, V, torch.zeros_like(V)).abs()
            # weights rounded to q's type and made by ex2.approx (2^-22), scores off by ds (in numerator and total);
            # the total: 64 + m / 128 roundings; the sums: m / 16 steps of 2^-23
            rel = U[q.dtype] + 2.0 ** -21 + 2 * ds + (64 + m / 128) * 2.0 ** -24 + m / 16 * 2.0 ** -23
            bd = (p.nan_to_num() @ va) * rel[:, None]
            if q.dtype == torch.float16:  # weights below 2^-33 of the largest
                bd = bd + m * 2.0 ** -33 * va.amax(0) if m else bd
            bound[a:a + n, h] = bd + U[q.dtype] * (o.nan_to_num(0, 0, 0).abs() + bd) + TINY[q.dtype]
            lse_bound[a:a + n, h] = ds + (70 + m / 128) * 2.0 ** -24 + 2.0 ** -21 * (1 + lse[a:a + n, h].nan_to_num(0, 0, 0).abs() + top.abs())
    return out, lse, bound, lse_bound


def logprobs(x, tokens, temperature=None, top=0):
    """float64 (log probability, entropy, ids, log probabilities) of rows x [E, V] on any device."""
    E, V = x.shape
    xd = x.double()
    T = torch.ones(E, dtype=torch.float64, device=x.device) if temperature is None else temperature.double()
    T = torch.where(T == 0, torch.ones_like(T), T)
    l = torch.log_softmax(xd / T[:, None], -1)
    p = l.exp()
    h = -torch.where(p > 0, p * l, torch.zeros_like(l)).sum(-1)
    lp = l.gather(1, tokens.long().clamp(0, V - 1)[:, None])[:, 0]
    order = torch.sort(xd, dim=-1, descending=True, stable=True).indices[:, :top]
    got = xd.gather(1, order)
    ids = torch.where(got > -math.inf, order, torch.full_like(order, -1))
    best = torch.where(got > -math.inf, l.gather(1, order), torch.full_like(got, -math.inf))
    if V < top:
        ids = torch.cat((ids, torch.full((E, top - V), -1, device=x.device)), 1)
        best = torch.cat((best, torch.full((E, top - V), -math.inf, dtype=torch.float64, device=x.device)), 1)
    return lp, h, ids, best


def logprob_bound(x, T=1.0):
    """How far the log probabilities of a row may be: (l - M) log2(e) / T by three roundings (of a size up to the row's
    span), weights by ex2.approx (2^-22) of exponents that are off by that, sums of V terms by lanes (V / 512 + 40 roundings)."""
    V = x.shape[-1]
    xd = x.double()
    fin = xd.isfinite()
    top = torch.where(fin, xd, torch.full_like(xd, -math.inf)).amax(-1)
    return lambda l: ((top - l).abs() / T + 1) * 4 * 2.0 ** -24 + 2.0 ** -21 + (V / 512 + 60) * 2.0 ** -24 + 2.0 ** -23 * math.log(V + 1) * 4
