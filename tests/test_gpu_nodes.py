"""The operators around the verification on the GPU against plain 64-bit forms:
rotary positions, the paged cache, the step's plan, the nodes' attention, the
kept path's rows."""
import math

import numpy as np
import pytest
import torch

import nodes_common as NC
from gpu_common import ensure_built
from speculative_decoding_verification_51_gb300 import binding

pytestmark = pytest.mark.gpu

BF, HF, FL = torch.bfloat16, torch.float16, torch.float32
E4 = torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def built():
    ensure_built()


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def randn(shape, dtype, g, scale=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)


# ---------------------------------------------------------------- rotary positions

ROPE = [
    # T, Hq, Hkv, D, rot, layout, dtype, scaling, factor, start
    (1, 1, 1, 64, 64, "half", BF, "none", 1.0, 0),
    (5, 32, 8, 128, 128, "half", BF, "none", 1.0, 1000000),
    (77, 14, 2, 128, 64, "interleaved", HF, "by_parts", 8.0, 9000),
    (33, 3, 3, 80, 40, "half", FL, "ntk", 4.0, 77777),
    (9, 7, 1, 256, 256, "half", FL, "linear", 2.0, 500000),
    (130, 4, 4, 96, 48, "interleaved", BF, "linear", 32.0, 12),
    (3, 2, 1, 10, 6, "half", HF, "none", 1.0, 3),
    (3, 2, 1, 10, 6, "interleaved", FL, "none", 1.0, 3),
    (2000, 16, 4, 64, 2, "interleaved", BF, "none", 1.0, 2147480000),
    (65, 40, 8, 128, 128, "half", HF, "by_parts", 32.0, 131000),
]


@pytest.mark.parametrize("inverse", [False, True])
@pytest.mark.parametrize("T,Hq,Hkv,D,rot,layout,dtype,scaling,factor,start", ROPE)
def test_rope(T, Hq, Hkv, D, rot, layout, dtype, scaling, factor, start, inverse):
    g = gen(T + D)
    q, k = randn((T, Hq, D), dtype, g), randn((T, Hkv, D), dtype, g)
    pos = (start + torch.randint(0, 700, (T,), generator=g, device="cuda")).to(torch.int32)
    table = binding.rope_table(rot, layout=layout, scaling=scaling, factor=factor, original_len=4096)
    th, scale = NC.thetas(rot, scaling=scaling, factor=factor, original_len=4096)
    oq, ok = binding.rope(q, k, pos, table, inverse=inverse)
    for x, y in ((q, oq), (k, ok)):
        ref = NC.rotate(x, pos, th, layout, scale, inverse)
        # 64 bits of angle: 2^-52 of it, below 1e-6 at any position here
        d = (y.cpu().double() - ref).abs()
        bound = NC.rotate_bound(x, th, layout, dtype, scale) + 2e-6 * x.cpu().double().abs().amax()
        assert bool((d <= bound).all()), float((d - bound).max())
        assert torch.equal(y[..., rot:], x[..., rot:])


def test_rope_strides_in_place_and_single():
    g = gen(3)
    T, Hq, Hkv, D = 11, 6, 2, 128
    table = binding.rope_table(128)
    th, _ = NC.thetas(128)
    pos = torch.randint(-50, 4000, (T,), generator=g, device="cuda").to(torch.int32)
    qkv = randn((T, Hq + 2 * Hkv, D), BF, g)          # one projection's output
    q, k = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv]
    rq, rk = NC.rotate(q, pos, th, "half"), NC.rotate(k, pos, th, "half")
    before = qkv.clone()
    binding.rope(q, k, pos, table, out_q=q, out_k=k)
    bq = NC.rotate_bound(before[:, :Hq], th, "half", BF) + 2e-6
    assert bool(((q.cpu().double() - rq).abs() <= bq).all())
    assert bool(((k.cpu().double() - rk).abs() <= NC.rotate_bound(before[:, Hq:Hq + Hkv], th, "half", BF) + 2e-6).all())
    assert torch.equal(qkv[:, Hq + Hkv:], before[:, Hq + Hkv:])
    # odd strides and offsets: an input that starts one element late
    for layout in ("half", "interleaved"):
        table = binding.rope_table(64, layout=layout)
        th, _ = NC.thetas(64)
        flat = randn((T * (3 * 65) + 1,), FL, g)
        x = flat[1:].view(T, 3, 65)[..., :64]
        y = binding.rope(x, None, pos, table)
        ref = NC.rotate(x, pos, th, layout)
        assert bool(((y.cpu().double() - ref).abs() <= NC.rotate_bound(x, th, layout, FL) + 2e-6).all())
    # heads before tokens
    x = randn((3, T, 64), BF, g).transpose(0, 1)
    y = binding.rope(x, None, pos, table)
    assert bool(((y.cpu().double() - NC.rotate(x, pos, th, "interleaved")).abs()
                 <= NC.rotate_bound(x, th, "interleaved", BF) + 1e-5).all())
    assert binding.rope(x[:0], None, pos[:0], table).shape == (0, 3, 64)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_rope_gradient(layout):
    """The inverse flag gives the gradient of the rotation: against the
    formula's own (autograd in 64 bits) and against differences."""
    g = gen(8)
    T, H, D, rot = 13, 3, 96, 64
    table = binding.rope_table(rot, layout=layout, scaling="by_parts", factor=4.0, original_len=100)
    th, scale = NC.thetas(rot, scaling="by_parts", factor=4.0, original_len=100)
    x, dy = randn((T, H, D), FL, g), randn((T, H, D), FL, g)
    pos = torch.randint(0, 5000, (T,), generator=g, device="cuda").to(torch.int32)
    dx = binding.rope(dy, None, pos, table, inverse=True).cpu().double()
    want = NC.rotate(dy, pos, th, layout, scale, inverse=True)
    assert bool(((dx - want).abs() <= NC.rotate_bound(dy, th, layout, FL, scale) + 1e-5).all())
    xd = x.cpu().double().requires_grad_(True)
    c = torch.from_numpy(th) * pos.cpu().double()[:, None, None]
    r = rot
    if layout == "half":
        a, b = xd[..., :r // 2], xd[..., r // 2:r]
    else:
        a, b = xd[..., 0:r:2], xd[..., 1:r:2]
    ya, yb = scale * (a * torch.cos(c) - b * torch.sin(c)), scale * (a * torch.sin(c) + b * torch.cos(c))
    gy = dy.cpu().double()
    ga, gb = (gy[..., :r // 2], gy[..., r // 2:r]) if layout == "half" else (gy[..., 0:r:2], gy[..., 1:r:2])
    ((ya * ga).sum() + (yb * gb).sum() + (xd[..., r:] * gy[..., r:]).sum()).backward()
    assert float((dx - xd.grad).abs().max()) < 2e-5
    # a difference along a random direction: f is linear, so any step is exact
    v = randn((T, H, D), FL, g)
    yp = binding.rope(x + v, None, pos, table).cpu().double()
    ym = binding.rope(x - v, None, pos, table).cpu().double()
    left = float((((yp - ym) / 2) * gy).sum())
    right = float((dx * v.cpu().double()).sum())
    # T*H*D terms of size 1 with errors below 1e-5 each, as a random sum
    assert abs(left - right) < 1e-5 * T * H * D


# ---------------------------------------------------------------- the cache

CACHES = [
    # src, cache, heads, D, page, rot, layout, T
    (BF, BF, 8, 128, 64, 128, "half", 45),
    (HF, HF, 3, 80, 16, 40, "interleaved", 100),
    (BF, E4, 8, 128, 64, 128, "half", 333),
    (HF, E4, 1, 64, 48, 32, "interleaved", 50),
    (FL, E4, 2, 256, 16, 256, "half", 19),
    (BF, E4, 5, 80, 16, 40, "half", 61),
    (HF, E4, 2, 16, 32, 0, "half", 7),
    (BF, E4, 16, 96, 128, 0, "half", 1),
    (BF, BF, 2, 8, 16, 0, "half", 3),
    (BF, BF, 4, 256, 32, 2, "half", 40),
]


@pytest.mark.parametrize("src,kind,H,D,page,rot,layout,T", CACHES)
def test_cache_write_read(src, kind, H, D, page, rot, layout, T):
    g = gen(T * D)
    pages = T // page + 3
    cache = binding.new_kv_cache(pages, page, H, D, dtype=kind)
    k, v, q = randn((T, H, D), src, g, 3.0), randn((T, H, D), src, g), randn((T, 2 * H, D), src, g)
    v[0] = 0
    v[T // 2] *= 1e-3
    slots = torch.randperm(pages * page, generator=g, device="cuda")[:T].clone()
    if T > 4:
        slots[3] = -1
    pos = torch.randint(0, 9000, (T,), generator=g, device="cuda").to(torch.int32)
    table = binding.rope_table(rot, layout=layout) if rot else None
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    if rot:
        oq = binding.kv_write(cache, k, v, slots, positions=pos, table=table, q=q, dev_status=st)
        assert torch.equal(oq, binding.rope(q, None, pos, table))
        turned = binding.rope(k.float(), None, pos, table)      # float32: tested above
    else:
        assert binding.kv_write(cache, k, v, slots, dev_status=st) is None
        turned = k.float()
    assert int(st) == 0
    rk, rv = binding.kv_read(cache, slots, dtype=FL)
    on = (slots >= 0).cpu().numpy()
    for got, want in ((rk, turned), (rv, v.float())):
        got, want = got.cpu().numpy(), want.cpu()
        assert (got[~on] == 0).all()
        if kind == E4:
            exp, _ = NC.e4m3_values(want.numpy())
        else:
            exp = want.to(kind).double().numpy()
        assert np.array_equal(got[on].astype(np.float64), exp[on])
    # 16-bit reads round once
    bk, _ = binding.kv_read(cache, slots, dtype=HF)
    assert torch.equal(bk, rk.half())
    # rows of other slots are as they were
    others = torch.ones(pages * page, dtype=torch.bool, device="cuda")
    others[slots[slots >= 0]] = False
    ok, ov = binding.kv_read(cache, torch.nonzero(others)[:, 0], dtype=FL)
    assert not ok.any() and not ov.any()


def test_cache_extreme_rows():
    """Rows of the 8-bit cache where a scale can go wrong: exact bounds between
    two exponents, subnormal values, infinities, NaN, rows with one value."""
    D = 32
    rows = np.zeros((12, 1, D), np.float32)
    rows[1, 0, :] = 448.0
    rows[2, 0, 0] = 449.0
    rows[3, 0, 5] = np.nextafter(np.float32(448.0 * 2.0 ** -7), np.float32(1e9))
    rows[4, 0, :] = 2.0 ** -140
    rows[5, 0, :4] = [np.inf, -np.inf, np.nan, 3.0]
    rows[6, 0, :] = np.nan
    rows[7, 0, :] = np.linspace(-1, 1, D)
    rows[8, 0, :2] = [3.0e38, -1.0]
    rows[9, 0, :] = 17.0 * 2.0 ** np.arange(-20, 12)          # ties and the lowest binade
    rows[10, 0, :] = np.float32(1.0) + np.arange(D, dtype=np.float32) / 16
    rows[11, 0, 31] = -2.0 ** -126
    x = torch.from_numpy(rows).cuda()
    cache = binding.new_kv_cache(1, 16, 1, D, dtype=E4)
    slots = torch.arange(12, device="cuda")
    binding.kv_write(cache, x, x, slots)
    want, e = NC.e4m3_values(rows)
    for got in binding.kv_read(cache, slots, dtype=FL):
        assert np.array_equal(got.cpu().numpy().astype(np.float64), want, equal_nan=True)
    assert np.array_equal(cache.k_scale[0, 0, :12].cpu().numpy().astype(np.int64) - 127, e[:, 0])


def test_cache_strides_and_bad_slots():
    g = gen(5)
    T, H, D, page = 21, 4, 64, 16
    base = torch.zeros((4, page, 2, H, D), dtype=BF, device="cuda")     # tokens before heads, k beside v
    cache = binding.KVCache(base[:, :, 0].transpose(1, 2), base[:, :, 1].transpose(1, 2))
    qkv = randn((T, 3 * H, D), BF, g)
    k, v = qkv[:, H:2 * H], qkv[:, 2 * H:]
    slots = torch.randperm(4 * page, generator=g, device="cuda")[:T].clone()
    slots[2], slots[9] = 4 * page, 2 ** 40
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    binding.kv_write(cache, k, v, slots, dev_status=st)
    assert int(st) == binding.BADBIT["page"]
    rk, rv = binding.kv_read(cache, slots)
    on = (slots < 4 * page)
    assert torch.equal(rk[on], k[on]) and torch.equal(rv[on], v[on])
    assert not rk[~on].any() and not rv[~on].any()
    used = slots[on]
    assert torch.equal(base[used // page, used % page, 0], k[on])
    binding.kv_write(cache, k[:0], v[:0], slots[:0])                     # nothing to do
    # a key tensor at an odd element offset
    kk = randn((T * H * D + 1,), BF, g)[1:].view(T, H, D)
    c2 = binding.new_kv_cache(4, page, H, D, dtype=E4)
    good = torch.arange(T, device="cuda")
    binding.kv_write(c2, kk, v, good)
    assert np.array_equal(binding.kv_read(c2, good, dtype=FL)[0].cpu().numpy().astype(np.float64),
                          NC.e4m3_values(kk.float().cpu().numpy())[0])


# ---------------------------------------------------------------- the plan

@pytest.mark.parametrize("B,N,page", [(1, 1, 16), (5, 32, 16), (700, 9, 48), (3, 31, 128), (257, 4, 64)])
def test_plan(B, N, page):
    rng = np.random.default_rng(B * N)
    ctx = rng.integers(0, 700, B).astype(np.int32)
    nodes = rng.integers(1, N + 1, B).astype(np.int32)
    par = NC.random_tree(rng, B, N, width=int(rng.integers(1, 8)))
    table, pages = NC.make_table(rng, ctx, nodes, page)
    bad = 0
    if B > 4:   # bad requests among the good
        nodes[0] = 0
        ctx[1] = table.shape[1] * page - nodes[1] + 1
        bad |= binding.BADBIT["num_draft"] | binding.BADBIT["page"]
        if nodes[2] > 1:
            par[2, nodes[2] - 1] = nodes[2] - 1
            bad |= binding.BADBIT["tree"]
        table[3, 0] = pages
        nodes[4] = N + 1
    cache = binding.new_kv_cache(pages, page, 1, 16)
    d = lambda x: torch.from_numpy(x).cuda()  # noqa: E731
    st = torch.full((1,), 4, dtype=torch.int32, device="cuda")
    p = binding.tree_plan(d(par), d(nodes), d(ctx), d(table), cache, dev_status=st)
    pos, slots, masks, ok = NC.plan(par, nodes, ctx, table, page, pages)
    assert np.array_equal(p.positions.cpu().numpy(), pos)
    assert np.array_equal(p.slots.cpu().numpy(), slots)
    assert np.array_equal(p.masks.cpu().numpy().view(np.uint32), masks)
    assert int(st) == bad
    buf = p.buffer.view(torch.int32).cpu().numpy()
    want = np.where(ok, ctx, 0)
    assert np.array_equal(buf[:B], want) and np.array_equal(buf[B:2 * B], np.where(ok, nodes, 0))
    lengths = np.where((nodes >= 1) & (nodes <= N) & (ctx + nodes.astype(np.int64) <= table.shape[1] * page),
                       ctx + nodes, 0)
    tiles = np.maximum(1, -(-lengths // 128))
    assert np.array_equal(buf[2 * B:3 * B + 1], np.concatenate(([0], np.cumsum(tiles))))
    assert not buf[3 * B + 1:3 * B + 1 + 1024].any()


# ---------------------------------------------------------------- attention

def attn_case(B, N, Hq, Hkv, D, page, qdt, kind, ctx, nodes, seed, *, width=4, vscale=1.0, poison=True):
    rng = np.random.default_rng(seed)
    g = gen(seed)
    ctx, nodes = np.asarray(ctx, np.int32), np.asarray(nodes, np.int32)
    table, pages = NC.make_table(rng, ctx, nodes, page)
    cache = binding.new_kv_cache(pages, page, Hkv, D, dtype=kind)
    par = NC.random_tree(rng, B, N, width)
    d = lambda x: torch.from_numpy(x).cuda()  # noqa: E731
    p = binding.tree_plan(d(par), d(nodes), d(ctx), d(table), cache)
    # every slot, then the requests' own are written over a cache of NaN
    if poison:
        if kind == E4:
            cache.k.fill_(0x7f)
            cache.v.fill_(0xff)
            cache.k_scale.fill_(255)
            cache.v_scale.fill_(255)
        else:
            cache.k.fill_(math.nan)
            cache.v.fill_(math.inf)
    slots = np.concatenate([int(1) * table[b, t // page].astype(np.int64) * page + t % page
                            for b in range(B) for t in [np.arange(max(0, int(ctx[b]) + int(nodes[b])))]])
    slots = d(slots)
    T = slots.numel()
    src = FL if kind == E4 else kind
    k = randn((T, Hkv, D), src, g)
    v = randn((T, Hkv, D), src, g) * torch.exp2(torch.randint(-6, 7, (T, 1, 1), generator=g, device="cuda").float()).to(src) * vscale
    binding.kv_write(cache, k, v.to(src), slots)
    q = randn((B, N, Hq, D), qdt, g, 1.5)
    return q, cache, p, d(table), ctx, nodes


def check_attention(q, cache, p, table, ctx, nodes, masks=None, scale=None):
    lse = torch.full(q.shape[:3], 7.0, dtype=FL, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = binding.tree_attention(q, cache, p, masks=masks, scale=scale, lse=lse, dev_status=st)
    assert int(st) == 0
    m = (p.masks if masks is None else masks).cpu().numpy().view(np.uint32)
    sc = 1 / math.sqrt(q.shape[3]) if scale is None else scale
    ref, rl, bound = NC.attention(q, cache, table, ctx, nodes, m, sc)
    o = out.double()
    fin = torch.isfinite(ref)
    assert torch.equal(torch.isnan(o), torch.isnan(ref)), "NaN in other places"
    assert torch.equal(o[~fin & ~torch.isnan(ref)], ref[~fin & ~torch.isnan(ref)])
    d = (o - ref).abs()
    assert bool((d[fin] <= bound[fin]).all()), (float((d / bound)[fin].max()), int((d > bound)[fin].sum()))
    lf = torch.isfinite(rl)
    assert torch.equal(lf, torch.isfinite(lse))
    assert torch.equal(lse[~lf].double().nan_to_num(7, 7, 9), rl[~lf].nan_to_num(7, 7, 9))
    if lf.any():
        # scores within 2^-22 of their absolute sums (at most 60 here), sums 2^-20
        assert float((lse.double() - rl)[lf].abs().max()) < 2.0 ** -13
    assert torch.equal(out, binding.tree_attention(q, cache, p, masks=masks, scale=scale))  # the same bits again
    return out


KINDS = [(BF, BF), (HF, HF), (BF, E4), (HF, E4)]
SHAPES = [
    # B, N, Hq, Hkv, D, page, ctx range
    (1, 1, 8, 2, 128, 16, (0, 1)),          # a context of none
    (1, 1, 32, 8, 128, 16, (777, 778)),
    (3, 1, 4, 4, 64, 64, (0, 40)),
    (4, 4, 8, 2, 128, 64, (1, 700)),
    (2, 9, 14, 2, 128, 48, (100, 1300)),
    (3, 32, 8, 2, 64, 128, (0, 500)),
    (2, 32, 32, 4, 128, 32, (130, 900)),
    (5, 17, 7, 7, 80, 16, (0, 300)),
    (2, 3, 6, 2, 96, 16, (5, 450)),
    (2, 5, 8, 1, 256, 16, (0, 333)),
    (1, 32, 16, 1, 256, 64, (200, 800)),
    (40, 2, 4, 2, 64, 16, (0, 260)),
    (2, 8, 4, 2, 16, 16, (3, 200)),
    (1, 7, 64, 8, 128, 128, (5000, 5001)),
]


@pytest.mark.parametrize("qdt,kind", KINDS)
@pytest.mark.parametrize("B,N,Hq,Hkv,D,page,rng", SHAPES)
def test_attention(B, N, Hq, Hkv, D, page, rng, qdt, kind):
    r = np.random.default_rng(B * 1000 + N * 10 + D)
    ctx = r.integers(rng[0], rng[1], B)
    nodes = r.integers(1, N + 1, B)
    nodes[0] = N
    check_attention(*attn_case(B, N, Hq, Hkv, D, page, qdt, kind, ctx, nodes, B + N + D))


@pytest.mark.parametrize("qdt,kind", KINDS)
@pytest.mark.parametrize("B,N,Hq,Hkv,D,page,ctx", [
    # every CTA has a dozen tiles and more, across several items
    (3, 12, 16, 4, 128, 64, (30000, 17, 21111)),
    (2, 9, 36, 6, 64, 128, (20000, 20001)),
    (3, 2, 12, 4, 128, 16, (30000, 300, 22222)),
    (2, 5, 20, 4, 96, 32, (15003, 29999)),
    (2, 3, 8, 2, 256, 32, (9000, 14001)),
    (300, 5, 28, 4, 64, 16, None),
])
def test_attention_long(B, N, Hq, Hkv, D, page, ctx, qdt, kind):
    r = np.random.default_rng(N)
    ctx = np.array(ctx) if ctx else r.integers(0, 700, B)
    nodes = np.maximum(1, N - np.arange(B) % 3)
    check_attention(*attn_case(B, N, Hq, Hkv, D, page, qdt, kind, ctx, nodes, 5 * N + D))


@pytest.mark.parametrize("qdt,kind", KINDS)
@pytest.mark.parametrize("N,Hq", [(6, 4), (12, 24)])
def test_attention_masks_and_bad_values(N, Hq, qdt, kind):
    """Arbitrary masks, rows that see nothing, bad requests, infinities and NaN in
    nodes that some rows do not see, and in nodes that nobody sees."""
    B, Hkv, D, page = 4, 2, 64, 16
    ctx, nodes = [0, 37, 0, 130], [N, N, 0, N - 1]
    q, cache, p, table, ctx, nodes = attn_case(B, N, Hq, Hkv, D, page, qdt, kind, ctx, nodes, 99)
    r = np.random.default_rng(1)
    masks = r.integers(0, 2 ** N, (B, N)).astype(np.uint32)
    masks[0, 0] = 0          # no context and no node: zeros
    masks[1, 1] = 0          # the context alone
    masks[:, 2] |= 0xFFFF0000 >> 0 & ~np.uint32((1 << N) - 1)   # bits past the nodes count for nothing
    masks[3, :] &= ~np.uint32(1 << 3)   # nobody sees node 3 of request 3
    m = torch.from_numpy(masks.view(np.int32)).cuda()

    def spoil(b, u, value, side, d=slice(None)):
        t = int(ctx[b]) + u
        pg, off = int(table[b, t // page]), t % page
        x = cache.k if side == "k" else cache.v
        x[pg, :, off, d] = 0x7f if kind == E4 else value

    spoil(3, 3, math.nan, "k")
    spoil(3, 3, math.nan, "v")
    spoil(1, 4, math.nan, "v", slice(3, 9))
    spoil(0, 5, math.nan, "v", 0)
    if kind != E4:
        spoil(0, 1, math.inf, "v", slice(0, 4))
        spoil(1, 0, -math.inf, "v", 63)
    spoil(1, 5, math.nan, "k")
    masked = masks & np.uint32((1 << N) - 1)
    mm = masked.copy()
    for b in range(B):
        mm[b] &= np.uint32((1 << max(0, int(nodes[b]))) - 1)
    lse = torch.zeros((B, N, Hq), device="cuda")
    out = binding.tree_attention(q, cache, p, masks=m, lse=lse)
    ref, rl, bound = NC.attention(q, cache, table, ctx, nodes, mm, 1 / 8)
    o = out.double()
    assert torch.equal(torch.isnan(o), torch.isnan(ref))
    fin = torch.isfinite(ref)
    inf = torch.isinf(ref)
    assert torch.equal(o[inf], ref[inf])
    assert bool(((o - ref).abs()[fin] <= bound[fin]).all())
    assert not out[0, 0].any() and bool((lse[0, 0] == -math.inf).all())
    assert not out[2].any() and bool((lse[2] == -math.inf).all())     # a bad request
    assert not out[3, N - 1].any()                                    # a node that is not there
    assert bool(torch.isfinite(out[3, :N - 1]).all())                 # what nobody sees harms nobody


def test_attention_strides_layout_stream_and_long_offsets():
    g = gen(4)
    B, N, Hq, Hkv, D, page = 2, 3, 8, 2, 128, 64
    # tokens before heads in the cache, queries inside a projection's output; the
    # pages in use lie past 2^32 bytes and 2^31 elements of the cache
    pages = 35000
    base_k = torch.empty((pages, page, Hkv, D), dtype=BF, device="cuda")   # 2.3 G elements
    big = torch.empty((2, pages, Hkv, page, D), dtype=BF, device="cuda")  # 2.3 G elements a side
    ctx, nodes = np.array([150, 511], np.int32), np.array([3, 2], np.int32)
    par = np.tile(np.array([-1, 0, 0], np.int32), (B, 1))
    d = lambda x: torch.from_numpy(x).cuda()  # noqa: E731
    for cache, last in ((binding.KVCache(base_k.transpose(1, 2), base_k.transpose(1, 2)), pages),
                        (binding.KVCache(big[0], big[1]), pages)):
        table = (last - 1 - np.arange(18, dtype=np.int32)).reshape(2, 9)
        p = binding.tree_plan(d(par), d(nodes), d(ctx), d(table), cache)
        for b in range(B):
            t = np.arange(int(ctx[b] + nodes[b]))
            slots = d(table[b, t // page].astype(np.int64) * page + t % page)
            x = randn((len(t), Hkv, D), BF, g)
            # the first cache has one tensor for both sides: keys equal values
            binding.kv_write(cache, x, x if cache.k.data_ptr() == cache.v.data_ptr() else randn((len(t), Hkv, D), BF, g), slots)
        qkv = randn((B, N, Hq + 4, D), BF, g)
        q = qkv[:, :, 2:2 + Hq]
        want = check_attention(q, cache, p, d(table), ctx, nodes)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        got = binding.tree_attention(q, cache, p, stream=side)
        side.synchronize()
        assert torch.equal(got, want)
    del base_k, big


def test_attention_large_scores_and_empty_batch():
    """Scores in the hundreds (one token has all the weight), equal scores, and
    rows whose values are tiny or huge powers of two."""
    for qdt, kind in KINDS:
        q, cache, p, table, ctx, nodes = attn_case(2, 4, 4, 2, 128, 16, qdt, kind, [300, 40], [4, 4], 7)
        check_attention(q * 40, cache, p, table, ctx, nodes)
        check_attention(torch.zeros_like(q), cache, p, table, ctx, nodes)
        check_attention(q, cache, p, table, ctx, nodes, scale=0.0)
        check_attention(q, cache, p, table, ctx, nodes, scale=-0.3)
    q, cache, p, table, ctx, nodes = attn_case(2, 4, 4, 2, 64, 16, BF, E4, [300, 40], [4, 4], 8, vscale=2.0 ** -40)
    check_attention(q, cache, p, table, ctx, nodes)
    z = torch.zeros((0, 4), dtype=torch.int32, device="cuda")
    z1 = torch.zeros((0,), dtype=torch.int32, device="cuda")
    p0 = binding.tree_plan(z, z1, z1, torch.zeros((0, 2), dtype=torch.int32, device="cuda"), cache)
    assert binding.tree_attention(q[:0], cache, p0).shape == (0, 4, 4, 64)
    assert binding.kv_commit([cache], p0, z1).shape == (0,)


def test_attention_zero_values_dominate():
    """An 8-bit row of zeros with nearly all the weight: its scale is the least
    there is, and the total must still count it."""
    B, N, H, D, page = 1, 1, 1, 64, 16
    cache = binding.new_kv_cache(8, page, H, D, dtype=E4)
    d = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    p = binding.tree_plan(d([[-1]]), d([1]), d([100]), d([[0, 1, 2, 3, 4, 5, 6, 7]]), cache)
    g = gen(1)
    k, v = randn((101, H, D), FL, g), randn((101, H, D), FL, g)
    q = randn((B, N, H, D), BF, g)
    k[17] = q[0, 0].float() * 1.0
    v[17] = 0
    binding.kv_write(cache, k, v, torch.arange(101, device="cuda"))
    check_attention(q, cache, p, d([[0, 1, 2, 3, 4, 5, 6, 7]]), np.array([100]), np.array([1]))


# ---------------------------------------------------------------- the kept path

@pytest.mark.parametrize("kind,H,D,page,N,B", [(BF, 2, 64, 16, 32, 6), (E4, 3, 80, 48, 20, 9), (HF, 1, 8, 16, 5, 3), (E4, 8, 128, 64, 32, 70)])
def test_commit(kind, H, D, page, N, B):
    rng = np.random.default_rng(N * D)
    g = gen(N)
    ctx = rng.integers(0, 100, B).astype(np.int32)
    nodes = rng.integers(1, N + 1, B).astype(np.int32)
    nodes[0] = N
    par = NC.random_tree(rng, B, N, 5)
    table, pages = NC.make_table(rng, ctx, nodes, page)
    d = lambda x: torch.from_numpy(x).cuda()  # noqa: E731
    caches = [binding.new_kv_cache(pages, page, H, D, dtype=kind) for _ in range(3)]
    p = binding.tree_plan(d(par), d(nodes), d(ctx), d(table), caches[0])
    last = np.array([rng.integers(0, n) for n in nodes], np.int32)
    last[0] = N - 1
    if B > 4:
        last[1], last[2] = -1, min(N, nodes[2])   # a bad request, a node that is not there
    everything = torch.arange(pages * page, device="cuda")
    olds = []
    for c in caches:
        x = randn((pages * page, H, D), FL if kind == E4 else kind, g)
        binding.kv_write(c, x, x * 2, everything)
        olds.append(binding.kv_read(c, everything, dtype=FL))
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    plan_ctx = p.context_len
    new = binding.kv_commit(caches, p, d(last), new_context_len=plan_ctx, dev_status=st)
    assert new.data_ptr() == plan_ctx.data_ptr()
    _, slots, masks, _ = NC.plan(par, nodes, ctx, table, page, pages)
    src = np.arange(pages * page)
    want = ctx.copy()
    for b in range(B):
        if last[b] < 0 or last[b] >= nodes[b]:
            continue
        path = [u for u in range(N) if masks[b, last[b]] >> u & 1]
        want[b] += len(path)
        for i, u in enumerate(path):
            src[slots[b, i]] = slots[b, u]
    assert np.array_equal(new.cpu().numpy(), want)
    assert int(st) == (binding.BADBIT["tree"] if B > 4 else 0)
    for c, (ok, ov) in zip(caches, olds):
        nk, nv = binding.kv_read(c, everything, dtype=FL)
        at = torch.from_numpy(src).cuda()
        assert torch.equal(nk, ok[at]) and torch.equal(nv, ov[at])


# ---------------------------------------------------------------- refusals

def test_refusals():
    t = lambda *s, dt=BF: torch.zeros(s, dtype=dt, device="cuda")  # noqa: E731
    i = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")  # noqa: E731
    table = binding.rope_table(64)
    cache = binding.new_kv_cache(4, 16, 2, 64)
    slots = torch.zeros(3, dtype=torch.int64, device="cuda")
    with pytest.raises(ValueError):
        binding.rope(t(3, 2, 64), None, i(4), table)                 # positions of other length
    with pytest.raises(ValueError):
        binding.rope(t(3, 2, 64), t(3, 2, 64, dt=HF), i(3), table)    # mixed types
    with pytest.raises(ValueError):
        binding.rope(t(3, 64, 2).transpose(1, 2), None, i(3), table)  # channels apart
    with pytest.raises(binding.SpecVerifyError):
        binding.rope(t(3, 2, 32), None, i(3), table)                  # more channels turn than there are
    with pytest.raises(ValueError):
        binding.rope_table(64, layout="other")
    with pytest.raises(binding.SpecVerifyError):
        binding.rope_table(63)
    with pytest.raises(binding.SpecVerifyError):
        binding.rope_table(64, scaling="by_parts", factor=2.0)        # needs the original length
    with pytest.raises(binding.SpecVerifyError):
        binding.kv_write(cache, t(3, 2, 64, dt=HF), t(3, 2, 64, dt=HF), slots)   # another 16-bit type
    with pytest.raises(ValueError):
        binding.kv_write(cache, t(3, 1, 64), t(3, 1, 64), slots)
    with pytest.raises(ValueError):
        binding.kv_write(cache, t(3, 2, 64), t(3, 2, 64), slots, q=t(3, 4, 64))
    with pytest.raises(ValueError):
        binding.KVCache(t(4, 2, 16, 64, dt=torch.uint8), t(4, 2, 16, 64, dt=torch.uint8))
    with pytest.raises(ValueError):
        binding.kv_read(cache, slots.int())
    odd = binding.KVCache(t(4, 2, 24, 64), t(4, 2, 24, 64))           # pages of 24 tokens
    with pytest.raises(binding.SpecVerifyError) as e:
        binding.kv_read(odd, slots)
    assert e.value.status == binding.SPEC_ERR_UNSUPPORTED
    p = binding.tree_plan(i(1, 2), torch.ones(1, dtype=torch.int32, device="cuda"), i(1), i(1, 1), cache)
    with pytest.raises(ValueError):
        binding.tree_attention(t(1, 3, 4, 64), cache, p)              # nodes of another plan
    with pytest.raises(ValueError):
        binding.tree_attention(t(1, 2, 3, 64), cache, p)              # 3 heads over 2
    with pytest.raises(binding.SpecVerifyError):
        binding.tree_attention(t(1, 2, 4, 64, dt=HF), cache, p)       # f16 queries, bf16 cache
    with pytest.raises(binding.SpecVerifyError):
        binding.tree_attention(t(1, 2, 4, 64), cache, p, workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
    with pytest.raises(binding.SpecVerifyError):
        binding.tree_attention(t(1, 2, 4, 65)[..., 1:], cache, p)     # strides not multiples of 8
    with pytest.raises(binding.SpecVerifyError):
        binding.tree_plan(i(1, 33), i(1), i(1), i(1, 1), cache)       # 33 nodes
    other = binding.new_kv_cache(5, 16, 2, 64)
    with pytest.raises(ValueError):
        binding.tree_attention(t(1, 2, 4, 64), other, p)
    with pytest.raises(ValueError):
        binding.kv_commit([], p, i(1))
