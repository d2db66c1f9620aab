"""The operators of the prompt's pass and of the answer's probabilities, as they are measured: the norm of each head of
queries and keys with the rotation (alone, and on the way into the paged cache), causal attention over packed prompts,
both of them in a run behind the prompts' plan, and the log probabilities of given tokens with entropy and top alternatives.

`run` with `own` false computes each in its plain form (elementary torch operations in 32 bits); with `own` true it makes
the calls of the package's binding.  `exact` computes the same in 64 bits from the definitions.
"""
import math

import torch

own = False

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SIZE = {"bf16": 2, "f16": 2, "f32": 4, "e4m3": 1}
EPS = 1e-6
TWO_PI_OVER_2_32 = 2.0 * math.pi / 4294967296.0


# ---------------------------------------------------------------- cases

def listed():
    return [
        # a decoding step of one request, its last token and 3 drafts: latency
        dict(name="norm_step_b1", op="norm", T=4, Hq=32, Hkv=8, D=128, rot=128, layout="half", dtype="bf16", start=1900),
        # a long prompt of odd length, every head normalised and turned
        dict(name="norm_prompt", op="norm", T=32771, Hq=32, Hkv=8, D=128, rot=128, layout="half", dtype="bf16", start=0),
        # 512 requests x (8 drafts + 1): normalised, turned, written to an 8-bit cache and read back
        dict(name="norm_cache_fp8_b512", op="cache", T=4608, Hq=32, Hkv=8, D=128, rot=64, layout="interleaved",
             dtype="bf16", cache="e4m3", page=64, start=100),
        # one prompt of a few words: latency
        dict(name="prompt_b1", op="prompt", B=1, lo=45, hi=45, ctx=0, Hq=32, Hkv=8, D=128, dtype="bf16", window=0, pad=0),
        # 32 prompts of ragged lengths in a batch with room behind them
        dict(name="prompt_b32", op="prompt", B=32, lo=20, hi=2000, ctx=0, Hq=32, Hkv=8, D=128, dtype="bf16", window=0,
             pad=100),
        # one long prompt
        dict(name="prompt_long", op="prompt", B=1, lo=16001, hi=16001, ctx=0, Hq=32, Hkv=8, D=128, dtype="bf16", window=0,
             pad=0),
        # pieces of prompts behind up to 3000 tokens, a window, narrow heads without sharing, half precision
        dict(name="prompt_window_f16", op="prompt", B=7, lo=1, hi=1501, ctx=3000, Hq=12, Hkv=12, D=64, dtype="f16",
             window=1000, pad=0),
        # 16 prompts on their way into the cache: plan, norm and rotation and write, attention
        dict(name="prompt_run_b16", op="run", B=16, lo=10, hi=700, ctx=0, Hq=32, Hkv=8, D=128, dtype="bf16", window=0,
             pad=0, rot=128, layout="half", page=64),
        # the token that one request emitted, with the 20 best
        dict(name="logprob_b1", op="logprob", B=1, N=1, V=151936, dtype="bf16", top=20, entropy=True, temps=False,
             rows=False, masked=False),
        # 256 requests x (3 drafts + 1): the tokens that were kept, with the 5 best and the entropy
        dict(name="logprob_b256", op="logprob", B=256, N=4, V=151936, dtype="bf16", top=5, entropy=True, temps=False,
             rows=False, masked=False),
        # 64 trees of 32 nodes: the kept paths' rows, each request with its temperature
        dict(name="logprob_tree_b64", op="logprob", B=64, N=32, V=32000, dtype="f32", top=0, entropy=True, temps=True,
             rows=True, masked=False),
        # every token of a prompt, a vocabulary of odd size with a part of it masked
        dict(name="logprob_prompt_odd", op="logprob", B=1, N=2001, V=50001, dtype="f16", top=1, entropy=False, temps=False,
             rows=False, masked=True),
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
        op = rng.choice(["norm", "cache", "prompt", "prompt", "run", "logprob", "logprob"])
        D = rng.choice([64, 80, 96, 128, 128, 256])
        Hkv = rng.choice([1, 2, 4, 8, 8, 16])
        heads = dict(Hq=Hkv * rng.choice([1, 2, 4, 7, 8]), Hkv=Hkv, D=D)
        rot, layout = rng.choice([D, D // 2, D // 4 * 2]), rng.choice(["half", "interleaved"])
        dtype = rng.choice(["bf16", "bf16", "f16"])
        if op == "norm":
            c = dict(op=op, T=_log(rng, 1, 32768), rot=rot, layout=layout, dtype=rng.choice(["bf16", "f16", "f32"]),
                     start=_log(rng, 1, 100000), **heads)
        elif op == "cache":
            c = dict(op=op, T=_log(rng, 1, 20000), rot=rot, layout=layout, dtype=dtype, cache=rng.choice([dtype, "e4m3"]),
                     page=rng.choice([16, 32, 64, 128]), start=_log(rng, 1, 100000), **heads)
        elif op == "logprob":
            rows = rng.random() < 0.3
            c = dict(op=op, B=_log(rng, 1, 512), N=rng.randint(2, 32) if rows else rng.randint(1, 9),
                     V=_log(rng, 1000, 152000), dtype=rng.choice(["bf16", "f16", "f32"]), top=rng.choice([0, 1, 5, 20, 32]),
                     entropy=rng.random() < 0.6, temps=rng.random() < 0.5, rows=rows, masked=rng.random() < 0.3)
            if rng.random() < 0.5:
                c["V"] = max(1000, c["V"] // 64 * 64)
            if c["B"] * c["N"] * c["V"] > (1 << 29):       # what the plain form sorts
                continue
        else:
            hi = _log(rng, 1, 16000)
            c = dict(op=op, B=_log(rng, 1, 64), lo=rng.randint(0, hi), hi=hi, ctx=0, dtype=dtype, window=0,
                     pad=rng.choice([0, 0, 37]), **heads)
            if op == "run":
                c.update(rot=rot, layout=layout, page=rng.choice([16, 32, 64, 128]))
            elif rng.random() < 0.4:
                c["ctx"] = _log(rng, 1, 16000)
            if rng.random() < 0.3:
                c["window"] = _log(rng, 1, 4096)
            if c["B"] * c["Hq"] * c["hi"] * (c["hi"] + c["ctx"]) > (1 << 32):      # the plain form's scores
                continue
        w = work(c)
        if w["bytes"] <= _CAPS[op][0] and w["flops"] <= _CAPS[op][1]:
            return c


def _spread(lo, hi, B):
    """B lengths spread evenly over [lo, hi], the first at hi."""
    return [lo + int(round((hi - lo) * ((1.0 - b * 0.6180339887) % 1.0 or 1.0))) for b in range(B)]


def _lens(case):
    """(new tokens, all tokens) of each prompt."""
    new = _spread(case["lo"], case["hi"], case["B"])
    ahead = _spread(0, case["ctx"], case["B"]) if case["ctx"] else [0] * case["B"]
    return new, [n + a for n, a in zip(new, ahead)]


def _pairs(n, m, window):
    """Pairs (query, key) of n queries that end with the last of m keys, each seeing itself and those before it."""
    first = m - n
    if not window or window >= m:
        return n * first + n * (n + 1) // 2
    short = max(0, min(n, window - first))              # queries that see less than a window
    return short * first + short * (short + 1) // 2 + (n - short) * window


def _kept(case):
    """How many tokens each request of a step kept, the emitted one with them."""
    B, N = case["B"], case["N"]
    if B == 1:
        return [N]
    most = min(N, 8) if case["rows"] else N
    return [1 + (b * 7 + 3) % most for b in range(B)]


def work(case):
    op = case["op"]
    if op == "logprob":
        t = sum(_kept(case))
        out = 4 + (4 if case["entropy"] else 0) + 8 * case["top"]
        n = t if case["rows"] else case["B"] * case["N"]
        return {"bytes": t * case["V"] * SIZE[case["dtype"]] + n * (4 + out + (4 if case["rows"] else 0)), "flops": 5 * t * case["V"]}
    D, Hq, Hkv, es = case["D"], case["Hq"], case["Hkv"], SIZE[case["dtype"]]
    if op == "norm":
        n = case["T"] * (Hq + Hkv)
        return {"bytes": 2 * n * D * es + 4 * case["T"] + 2 * D * es, "flops": n * (4 * D + 3 * case["rot"])}
    if op == "cache":
        T, src = case["T"], Hkv * D * es
        row = Hkv * (D * SIZE[case["cache"]] + (1 if case["cache"] == "e4m3" else 0))
        # k, v and q in, the cache's rows and q out; read back: the rows in, k and v out
        return {"bytes": T * (2 * src + 2 * Hq * D * es + 2 * row + 12 + 2 * row + 2 * src + 8),
                "flops": T * (Hq + Hkv) * (4 * D + 3 * case["rot"])}
    new, all_ = _lens(case)
    pairs = sum(_pairs(n, m, case["window"]) for n, m in zip(new, all_))
    T, M = sum(new), sum(all_)
    w = {"bytes": 2 * T * Hq * D * es + 2 * M * Hkv * D * es + 8 * case["B"], "flops": 4 * pairs * Hq * D}
    if op == "prompt":
        w["bytes"] += T * Hq * 4                             # the log-sums
    else:
        w["bytes"] += 2 * T * Hkv * D * es + T * (4 + 8)     # the cache's rows, positions and slots out
        w["flops"] += T * (Hq + Hkv) * (4 * D + 3 * case["rot"])
    return w


# ---------------------------------------------------------------- inputs

def _turns(rot, dev):
    """Turns per position as 64-bit fractions: the product with a position wraps to the exact phase."""
    v = [int(10000.0 ** (-2.0 * i / rot) / (2.0 * math.pi) * 2.0 ** 64) for i in range(rot // 2)]
    return torch.tensor(v, dtype=torch.int64, device=dev)


def _cache(pages, Hkv, page, D, kind, dev):
    """An empty cache: (k, v, k_scale, v_scale)."""
    if kind == "e4m3":
        s = torch.full((2, pages, Hkv, page), 127, dtype=torch.uint8, device=dev)
        k = torch.zeros((2, pages, Hkv, page, D), dtype=torch.uint8, device=dev)
        return k[0], k[1], s[0], s[1]
    k = torch.zeros((2, pages, Hkv, page, D), dtype=DT[kind], device=dev)
    return k[0], k[1], None, None


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(int(seed))
    op, dt = case["op"], DT[case["dtype"]]
    s = {"case": dict(case)}
    b = None
    if own:
        from speculative_decoding_verification_51_gb300 import binding as b
        s["binding"] = b

    def randn(*shape, scale=1.0):
        return (scale * torch.randn(shape, generator=g, device=dev)).to(dt)

    if op == "logprob":
        B, N, V = case["B"], case["N"], case["V"]
        x = 3.0 * torch.randn((B, N, V), generator=g, device=dev)
        likely = torch.randint(0, V, (B, N, 4), generator=g, device=dev)           # what the target would say
        x.scatter_add_(-1, likely, torch.linspace(12.0, 6.0, 4, device=dev).expand(B, N, 4).contiguous())
        if case["masked"]:                                                           # tokens that a grammar forbids
            x.masked_fill_(torch.rand((1, 1, V), generator=g, device=dev) < 0.4, -math.inf)
        s["logits"] = x.to(dt)
        kept = torch.tensor(_kept(case), device=dev)
        pick = torch.randint(0, 4, (B, N, 1), generator=g, device=dev)
        tokens = likely.gather(-1, pick)[..., 0].to(torch.int32)
        j = torch.arange(N, device=dev)[None]
        tokens = torch.where(j < kept[:, None], tokens, torch.full_like(tokens, -1))
        if case["rows"]:                                       # node j of a kept path is row 3 j of the tree, or the last
            width = int(max(_kept(case)))
            tokens = tokens[:, :width].contiguous()
            node = (3 * j[:, :width]).clamp(max=N - 1).expand(B, width)
            s["rows"] = (node + N * torch.arange(B, device=dev)[:, None]).to(torch.int32).contiguous()
        s["tokens"] = tokens
        if case["temps"]:
            s["temps"] = 0.3 + 1.2 * torch.rand((B, 1), generator=g, device=dev).expand(tokens.shape).contiguous()
        return s
    D, Hq, Hkv = case["D"], case["Hq"], case["Hkv"]
    if op in ("norm", "cache"):
        T = M = case["T"]
        s["positions"] = (case["start"] + torch.arange(T, device=dev)).to(torch.int32)
    else:
        new, all_ = _lens(case)
        T, M = sum(new) + case["pad"], sum(all_) + (0 if case["ctx"] else case["pad"])
        s["offsets"] = torch.tensor([sum(new[:i]) for i in range(len(new) + 1)], dtype=torch.int32, device=dev)
        s["k_offsets"] = torch.tensor([sum(all_[:i]) for i in range(len(new) + 1)], dtype=torch.int32, device=dev)
        s["out"] = torch.zeros((T, Hq, D), dtype=dt, device=dev)
        s["lse"] = torch.zeros((T, Hq), dtype=torch.float32, device=dev)
    s["q"] = randn(T, Hq, D, scale=2.0)
    s["k"] = randn(M, Hkv, D)
    if op != "norm":
        s["v"] = randn(M, Hkv, D)
    if op != "prompt":
        s["wq"] = (1.0 + 0.2 * torch.randn(D, generator=g, device=dev)).to(dt)
        s["wk"] = (1.0 + 0.2 * torch.randn(D, generator=g, device=dev)).to(dt)
        if own:
            s["norm"] = b.HeadNorm(s["wq"], s["wk"], eps=EPS)
            s["table"] = b.rope_table(case["rot"], layout=case["layout"], device=dev)
        else:
            s["turns"] = _turns(case["rot"], dev)
    if op == "cache":
        page = case["page"]
        pages = -(-T // page) + 2
        slots = torch.randperm((pages - 1) * page, generator=g, device=dev)[:T].to(torch.int64)
        slots[torch.arange(T, device=dev) % 17 == 16] = -1     # rows of finished requests: not written
        s["slots"], s["cache"] = slots, _cache(pages, Hkv, page, D, case["cache"], dev)
    if op == "run":
        page = case["page"]
        need = [-(-n // page) for n in new]
        perm = torch.randperm(max(1, sum(need)), generator=g, device=dev).to(torch.int32).tolist()
        s["page_table"] = torch.tensor([perm[sum(need[:i]):sum(need[:i + 1])] + [-1] * (max(1, max(need)) - n) for i, n in enumerate(need)],
                                       dtype=torch.int32, device=dev)
        s["cache"] = _cache(len(perm) + 1, Hkv, page, D, case["dtype"], dev)
        s["k_turned"] = torch.zeros_like(s["k"])
    if own and "cache" in s:
        s["cache"] = b.KVCache(*s["cache"])
    if own and op == "prompt":     # one plan serves every layer
        s["plan"] = b.prompt_plan(s["offsets"], T, Hq, Hkv, k_offsets=s["k_offsets"] if case["ctx"] else None,
                                  num_keys=M if case["ctx"] else None)
    return s


# ---------------------------------------------------------------- plain forms

def _normed(x, w, positions, turns, layout):
    """x [T, H, D]: each head divided by its root mean square, times w, its first channels turned, in 32 bits."""
    x = x.float()
    x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w.float()
    rot = 2 * turns.numel()
    phase = (positions.to(torch.int64)[:, None] * turns[None, :]) >> 32        # signed 32-bit fraction of a turn
    ang = phase.to(torch.float32) * TWO_PI_OVER_2_32
    c, s = torch.cos(ang)[:, None], torch.sin(ang)[:, None]
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
    return torch.ldexp(x, -e[..., None]).to(torch.float8_e4m3fn).view(torch.uint8), (e + 127).to(torch.uint8)


def _write(c, sc, at, page, x):
    """Rows x [T, Hkv, D] to the slots `at` of one cache tensor."""
    p, o = at // page, at % page
    if sc is None:
        c[p, :, o] = x.to(c.dtype)
    else:
        c[p, :, o], sc[p, :, o] = _quantise(x.float())


def _read(c, sc, at, page, dt):
    p, o = at // page, at % page
    if sc is None:
        return c[p, :, o].to(dt)
    return torch.ldexp(c[p, :, o].view(torch.float8_e4m3fn).float(), (sc[p, :, o].to(torch.int32) - 127)[..., None]).to(dt)


def _owners(offsets, T):
    """The prompt of each packed token (the number of prompts: none), and its place in it."""
    t = torch.arange(T, device=offsets.device)
    b = torch.searchsorted(offsets[1:].contiguous(), t.to(torch.int32), right=True)
    return b, t - offsets[b.clamp(max=offsets.numel() - 2)].long()


def _attention(s, q, k):
    """Causal attention of packed prompts into s["out"] and s["lse"]: every prompt's rows side by side, as long as the longest."""
    case, off, koff = s["case"], s["offsets"].long(), s["k_offsets"].long()
    T, Hq, D = q.shape
    B, Hkv, dev = case["B"], case["Hkv"], q.device
    G = Hq // Hkv
    n, m = off[1:] - off[:-1], koff[1:] - koff[:-1]
    i, j = torch.arange(max(_lens(case)[0]), device=dev), torch.arange(max(1, max(_lens(case)[1])), device=dev)
    iq, jk = (off[:-1, None] + i).clamp(max=T - 1), (koff[:-1, None] + j).clamp(max=k.shape[0] - 1)
    Q = q[iq].float().view(B, -1, Hkv, G, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, G * i.numel(), D)
    K = k[jk].float().transpose(1, 2)
    there = (j < m[:, None])[:, None, :, None]
    V = torch.where(there, s["v"][jk].float().transpose(1, 2), torch.zeros((), device=dev))
    z = (Q @ K.transpose(-1, -2)).mul_(1.0 / math.sqrt(D)).view(B, Hkv, G, i.numel(), j.numel())
    last = i + (m - n)[:, None]                                   # the last key that a query sees
    seen = j <= last[..., None]
    if case["window"]:
        seen = seen & (j > last[..., None] - case["window"])
    z.masked_fill_(~seen[:, None, None], -math.inf)
    top = z.amax(-1, keepdim=True)
    top = torch.where(torch.isfinite(top), top, torch.zeros_like(top))
    tot = z.sub_(top).exp_().sum(-1, keepdim=True)
    o = (z.view(B, Hkv, G * i.numel(), j.numel()) @ V).view(B, Hkv, G, i.numel(), D) / torch.where(tot > 0, tot, torch.ones_like(tot))
    lse = (top + torch.log(tot))[..., 0]
    b, at = _owners(s["offsets"], T)
    mine = b < B
    b, at = b[mine], at[mine]
    s["out"][mine] = o.permute(0, 3, 1, 2, 4).reshape(B, i.numel(), Hq, D)[b, at].to(q.dtype)
    s["lse"][mine] = lse.permute(0, 3, 1, 2).reshape(B, i.numel(), Hq)[b, at]


def _logprob(s):
    """(log probabilities, entropy, best ids, their log probabilities) of the entries; zeros and -1 where there is no token."""
    case = s["case"]
    x = s["logits"]
    V = x.shape[-1]
    tokens = s["tokens"].flatten().long()
    x = x.reshape(-1, V)
    there = tokens >= 0
    if "rows" in s:
        x = x[s["rows"].flatten().long()]
    best = None
    if case["top"]:
        raw, ids = torch.sort(x, dim=-1, descending=True, stable=True)
        raw, ids = raw[:, :case["top"]], ids[:, :case["top"]]
        best = torch.where(there[:, None] & (raw > -math.inf), ids, torch.full_like(ids, -1)).to(torch.int32)
    x = x.float()
    x = x - x.amax(-1, keepdim=True)
    if "temps" in s:
        x = x / s["temps"].flatten()[:, None]
    z = x.exp().sum(-1, dtype=torch.float64).log().float()
    zero = torch.zeros_like(z)
    out = [torch.where(there, x.gather(1, tokens.clamp(min=0)[:, None])[:, 0] - z, zero)]
    if case["entropy"]:
        lp = x - z[:, None]
        h = -torch.where(lp > -math.inf, lp.exp() * lp, torch.zeros_like(lp)).sum(-1, dtype=torch.float64).float()
        out.append(torch.where(there, h, zero))
    if best is not None:
        lp = torch.where(best >= 0, x.gather(1, ids) - z[:, None], torch.full_like(x[:, :case["top"]], -math.inf))
        out += [best, torch.where(there[:, None], lp, torch.zeros_like(lp))]
    return out


def _plain(s):
    case = s["case"]
    op = case["op"]
    if op == "logprob":
        return _logprob(s)
    dt = DT[case["dtype"]]
    if op == "norm":
        a = (s["positions"], s["turns"], case["layout"])
        return _normed(s["q"], s["wq"], *a).to(dt), _normed(s["k"], s["wk"], *a).to(dt)
    if op == "cache":
        ck, cv, sk, sv = s["cache"]
        page = case["page"]
        a = (s["positions"], s["turns"], case["layout"])
        spare = (ck.shape[0] - 1) * page                # a page that no slot names takes the rows not written
        at = torch.where(s["slots"] >= 0, s["slots"], torch.full_like(s["slots"], spare))
        _write(ck, sk, at, page, _normed(s["k"], s["wk"], *a))
        _write(cv, sv, at, page, s["v"])
        keep = (s["slots"] >= 0)[:, None, None]
        k, v = _read(ck, sk, at, page, dt), _read(cv, sv, at, page, dt)
        return (_normed(s["q"], s["wq"], *a).to(dt), torch.where(keep, k, torch.zeros_like(k)),
                torch.where(keep, v, torch.zeros_like(v)))
    if op == "prompt":
        _attention(s, s["q"], s["k"])
        return s["out"], s["lse"]
    # the run: positions and slots of the packed tokens, their rows normalised, turned and written, attention
    T, page = s["q"].shape[0], case["page"]
    b, at = _owners(s["offsets"], T)
    mine = b < case["B"]
    pos = torch.where(mine, at, torch.zeros_like(at)).to(torch.int32)
    pages = s["page_table"][b.clamp(max=case["B"] - 1), (at // page).clamp(max=s["page_table"].shape[1] - 1)].long()
    slots = torch.where(mine, pages * page + at % page, torch.full_like(at, -1))
    ck, cv, _, _ = s["cache"]
    spare = (ck.shape[0] - 1) * page
    to = torch.where(mine, slots, torch.full_like(slots, spare))
    a = (pos, s["turns"], case["layout"])
    q, k = _normed(s["q"], s["wq"], *a).to(dt), _normed(s["k"], s["wk"], *a).to(dt)
    _write(ck, None, to, page, k)
    _write(cv, None, to, page, s["v"])
    _attention(s, q, k)
    return pos, slots, ck[:-1], cv[:-1], s["out"]


def _own(s):
    b, case = s["binding"], s["case"]
    op = case["op"]
    if op == "logprob":
        r = b.token_logprobs(s["logits"], s["tokens"], rows=s.get("rows"), temperature=s.get("temps"), top=case["top"],
                             entropy=case["entropy"])
        out = [r.logprobs.flatten()]
        if case["entropy"]:
            out.append(r.entropy.flatten())
        if case["top"]:
            out += [r.top_ids.flatten(0, -2), r.top_logprobs.flatten(0, -2)]
        return out
    if op == "norm":
        return b.rope(s["q"], s["k"], s["positions"], s["table"], norm=s["norm"])
    if op == "cache":
        q = b.kv_write(s["cache"], s["k"], s["v"], s["slots"], positions=s["positions"], table=s["table"], q=s["q"],
                       norm=s["norm"])
        k, v = b.kv_read(s["cache"], s["slots"], dtype=DT[case["dtype"]])
        return q, k, v
    if op == "prompt":
        b.prompt_attention(s["q"], s["k"], s["v"], s["plan"], window=case["window"], out=s["out"], lse=s["lse"])
        return s["out"], s["lse"]
    plan = b.prompt_plan(s["offsets"], s["q"].shape[0], case["Hq"], case["Hkv"], page_table=s["page_table"], cache=s["cache"])
    q = b.kv_write(s["cache"], s["k"], s["v"], plan.slots, positions=plan.positions, table=s["table"], q=s["q"],
                   out_k=s["k_turned"], norm=s["norm"])
    b.prompt_attention(q, s["k_turned"], s["v"], plan, window=case["window"], out=s["out"])
    return plan.positions, plan.slots, s["cache"].k[:-1], s["cache"].v[:-1], s["out"]


def run(state):
    return _own(state) if own else _plain(state)


# ---------------------------------------------------------------- 64 bits

def exact(case, seed):
    op = case["op"]
    if op in ("prompt", "run") and work(case)["flops"] > 3e12:
        return None
    s = prepare(case, seed)
    dev = s["q" if "q" in s else "logits"].device
    if op == "logprob":
        x, tokens = s["logits"].reshape(-1, case["V"]), s["tokens"].flatten().tolist()
        rows = s["rows"].flatten().tolist() if "rows" in s else list(range(len(tokens)))
        temps = s["temps"].flatten().tolist() if "temps" in s else [1.0] * len(tokens)
        lp, ent = torch.zeros(len(tokens), dtype=torch.float64, device=dev), torch.zeros(len(tokens), dtype=torch.float64, device=dev)
        ids = torch.full((len(tokens), max(1, case["top"])), -1, dtype=torch.int32, device=dev)
        best = torch.zeros(ids.shape, dtype=torch.float64, device=dev)
        for e, (t, r, T) in enumerate(zip(tokens, rows, temps)):
            if t < 0:
                continue
            l = torch.log_softmax(x[r].double() / T, -1)
            lp[e] = l[t]
            if case["entropy"]:
                ent[e] = -torch.special.xlogy(l.exp(), l.exp()).sum()
            if case["top"]:
                # by value, then by index: values are at most 32 bits, so a 64-bit key holds both
                order = torch.sort(-x[r].double(), dim=-1, stable=True).indices[:case["top"]]
                some = x[r][order] > -math.inf
                best[e, :order.numel()] = torch.where(some, l[order], torch.full_like(l[order], -math.inf))
                ids[e, :order.numel()] = torch.where(some, order, torch.full_like(order, -1)).to(torch.int32)
        return [lp] + ([ent] if case["entropy"] else []) + ([ids, best] if case["top"] else [])

    def normed(x, w, pos):
        x = x.double()
        x = x / torch.sqrt(x.square().sum(-1, keepdim=True) / x.shape[-1] + EPS) * w.double()
        h = case["rot"] // 2
        th = torch.tensor([10000.0 ** (-i / h) for i in range(h)], dtype=torch.float64, device=dev)
        ang = pos.double()[:, None, None] * th
        z = torch.polar(torch.ones_like(ang), ang)
        if case["layout"] == "half":
            w = torch.complex(x[..., :h].contiguous(), x[..., h:2 * h].contiguous()) * z
            x[..., :h], x[..., h:2 * h] = w.real, w.imag
        else:
            w = torch.complex(x[..., 0:2 * h:2].contiguous(), x[..., 1:2 * h:2].contiguous()) * z
            x[..., 0:2 * h:2], x[..., 1:2 * h:2] = w.real, w.imag
        return x

    def held(x):
        """x as the cache holds it: over 8 bits 4 significant ones, steps of 2^-9 at least, times a power of two a row."""
        if case["cache"] != "e4m3":
            return x
        top = x.abs().amax(-1, keepdim=True)
        safe = torch.where(top > 0, top, torch.ones_like(top))
        e = torch.ceil(torch.log2(safe / 448.0))
        e = torch.where(safe > 448.0 * torch.exp2(e), e + 1, e)
        e = torch.where(safe <= 224.0 * torch.exp2(e), e - 1, e)
        y = x * torch.exp2(-e)
        step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
        return torch.round(y / step) * step * torch.exp2(e)

    if op == "norm":
        return normed(s["q"], s["wq"], s["positions"]), normed(s["k"], s["wk"], s["positions"])
    if op == "cache":
        keep = (s["slots"] >= 0)[:, None, None]
        return (normed(s["q"], s["wq"], s["positions"]), held(normed(s["k"], s["wk"], s["positions"])) * keep,
                held(s["v"].double()) * keep)
    new, all_ = _lens(case)
    q, k, v, D = s["q"].double(), s["k"].double(), s["v"].double(), case["D"]
    T, G = q.shape[0], case["Hq"] // case["Hkv"]
    pos, slots = torch.zeros(T, dtype=torch.int32), torch.full((T,), -1, dtype=torch.int64)
    starts = [sum(new[:b]) for b in range(len(new))]
    if op == "run":
        page, table = case["page"], s["page_table"].tolist()
        for a, n, row in zip(starts, new, table):
            pos[a:a + n] = torch.arange(n, dtype=torch.int32)
            slots[a:a + n] = torch.tensor([row[i // page] * page + i % page for i in range(n)], dtype=torch.int64)
        pos, slots = pos.to(dev), slots.to(dev)
        q, k = normed(s["q"], s["wq"], pos), normed(s["k"], s["wk"], pos)
    out = torch.zeros((T, case["Hq"], D), dtype=torch.float64, device=dev)
    lse = torch.zeros((T, case["Hq"]), dtype=torch.float64, device=dev)
    for b, (n, m) in enumerate(zip(new, all_)):
        ka = sum(all_[:b])
        for h in range(case["Hq"]):
            K, V = k[ka:ka + m, h // G], v[ka:ka + m, h // G]
            for a in range(0, n, 4096):
                c = min(n, a + 4096)
                last = torch.arange(a, c, device=dev)[:, None] + (m - n)
                lo = max(0, a + m - n + 1 - case["window"]) if case["window"] else 0
                hi = max(0, c + m - n)
                j = torch.arange(lo, hi, device=dev)
                z = q[starts[b] + a:starts[b] + c, h] @ K[lo:hi].T / math.sqrt(D)
                hide = j > last
                if case["window"]:
                    hide |= j <= last - case["window"]
                z.masked_fill_(hide, -math.inf)
                lse[starts[b] + a:starts[b] + c, h] = torch.logsumexp(z, -1)
                out[starts[b] + a:starts[b] + c, h] = torch.softmax(z, -1) @ V[lo:hi]
    if op == "prompt":
        return out, lse
    held_k = torch.zeros((s["cache"].k if own else s["cache"][0])[:-1].shape, dtype=torch.float64, device=dev)
    held_v, mine = torch.zeros_like(held_k), slots >= 0
    held_k[slots[mine] // page, :, slots[mine] % page] = k[mine]
    held_v[slots[mine] // page, :, slots[mine] % page] = v[mine]
    return pos, slots, held_k, held_v, out
