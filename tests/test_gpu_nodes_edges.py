"""The nodes' attention where it can go wrong, for few rows a key head
(k_attn_rows) and for many (the tile kernels): nodes that are not there, values
of very different sizes, queries that are not finite, scales of any sign, strides,
pages far into a cache, other streams, and a step in a CUDA graph."""
import math

import numpy as np
import pytest
import torch

import nodes_common as NC
from gpu_common import ensure_built
from speculative_decoding_verification_51_gb300 import binding
from test_gpu_nodes import BF, E4, FL, HF, KINDS, attn_case, check_attention, gen, randn

pytestmark = pytest.mark.gpu

# nodes and query heads over 2 key heads: at most 16 rows a key head, and more
FEW_AND_MANY = [(6, 4), (12, 24)]


@pytest.fixture(scope="module", autouse=True)
def built():
    ensure_built()


def dev(x):
    return torch.from_numpy(np.ascontiguousarray(x)).cuda()


def slots_of(table, ctx, page, b, tokens):
    """The cache slots of `tokens` of request b."""
    t = np.asarray(tokens)
    return dev(table[b].cpu().numpy()[t // page].astype(np.int64) * page + t % page)


def star_masks(B, N, nodes):
    """Node 0 and its children alone: a node sees node 0 and itself."""
    m = np.array([[(1 << v | 1) if v < nodes[b] else 0 for v in range(N)] for b in range(B)], np.uint32)
    return dev(m.view(np.int32))


# ---------------------------------------------------------------- nodes that are not there

@pytest.mark.parametrize("qdt,kind", KINDS)
@pytest.mark.parametrize("N,Hq", FEW_AND_MANY)
@pytest.mark.parametrize("ctx", [[40, 37, 300], [21000, 9, 30000]])   # whole items, and items joined from parts
def test_nodes_past_the_tree_are_zero_whatever_the_context_holds(ctx, N, Hq, qdt, kind):
    nodes = [N - 2, N - 3, 1]
    q, cache, p, table, ctx, nodes = attn_case(3, N, Hq, 2, 64, 16, qdt, kind, ctx, nodes, 5)
    for b, t, value in ((0, 11, math.nan), (2, 200, math.inf)):
        s = int(slots_of(table, ctx, 16, b, [t])[0])
        cache.k[s // 16, :, s % 16, 3] = 0x7f if kind == E4 else value
    lse = torch.zeros((3, N, Hq), device="cuda")
    out = binding.tree_attention(q, cache, p, lse=lse)
    for b in range(3):
        n = int(nodes[b])
        assert not out[b, n:].any() and bool((lse[b, n:] == -math.inf).all())
    m = p.masks.cpu().numpy().view(np.uint32)
    ref, _, bound = NC.attention(q, cache, table, ctx, nodes, m, 1 / 8)
    fin = torch.isfinite(ref)
    assert torch.equal(torch.isnan(out.double()), torch.isnan(ref))
    assert bool(((out.double() - ref).abs()[fin] <= bound[fin]).all())


# ---------------------------------------------------------------- values of very different sizes

@pytest.mark.parametrize("kind,power", [(BF, 40), (HF, 9), (E4, 7), (E4, 12), (E4, 17), (E4, 40), (E4, 90)])
@pytest.mark.parametrize("N,Hq", FEW_AND_MANY)
@pytest.mark.parametrize("ctx", [[0, 40], [101, 300], [2000, 21000]])
def test_unseen_nodes_of_large_values_have_no_effect(ctx, N, Hq, kind, power):
    """A sibling's values 2^power times the others': the nodes that do not see it
    lose nothing by it."""
    qdt = BF if kind == E4 else kind
    D, page = 128, 16
    q, cache, p, table, ctx, nodes = attn_case(2, N, Hq, 2, D, page, qdt, kind, ctx, [N, N - 1], 17)
    src = FL if kind == E4 else kind
    g = gen(power)
    for b in range(2):
        for u in (4, int(nodes[b]) - 1):
            s = slots_of(table, ctx, page, b, [int(ctx[b]) + u])
            big = randn((1, 2, D), FL, g) * 2.0 ** power
            binding.kv_write(cache, randn((1, 2, D), src, g), big.to(src), s)
    check_attention(q, cache, p, table, ctx, nodes, masks=star_masks(2, N, nodes))


@pytest.mark.parametrize("kind,power", [(BF, 30), (HF, 9), (E4, 6), (E4, 10), (E4, 16), (E4, 30), (E4, 80)])
@pytest.mark.parametrize("qdt", [BF, HF])
@pytest.mark.parametrize("N,Hq", FEW_AND_MANY)
def test_large_values_of_little_weight(N, Hq, qdt, kind, power):
    """Early tokens with values 2^power times the others' and scores some 90 octaves
    or more below: what they add is 2^(power - 90) at most, and the others keep their bits."""
    if kind != E4 and kind != qdt:
        pytest.skip("a 16-bit cache takes queries of its own type")
    D, page = 64, 16
    ctx, nodes = [700, 16000], [N, N - 1]
    q, cache, p, table, ctx, nodes = attn_case(2, N, Hq, 2, D, page, qdt, kind, ctx, nodes, 23)
    # all queries share a direction: + 8 in channel 0; the tokens have - 128 there
    # (score - 128 exp(-128) against scores of size 2 to 10)
    q[..., 0] = 8.0
    src = FL if kind == E4 else kind
    g = gen(power)
    for b in range(2):
        for t in (3, 130, 401):
            k = randn((1, 2, D), FL, g)
            k[..., 0] = -128.0
            v = randn((1, 2, D), FL, g) * 2.0 ** power
            binding.kv_write(cache, k.to(src), v.to(src), slots_of(table, ctx, page, b, [t]))
    check_attention(q, cache, p, table, ctx, nodes)


@pytest.mark.parametrize("N,Hq", FEW_AND_MANY)
@pytest.mark.parametrize("D", [48, 128])
def test_rows_of_zeros_among_values_of_every_size(D, N, Hq):
    """8 bits: rows of zeros, tiny ones and large ones side by side, in tiles of their
    own and mixed, the zeros with much of the weight."""
    ctx, nodes = [130, 1500], [N, N]
    q, cache, p, table, ctx, nodes = attn_case(2, N, Hq, 2, D, 16, BF, E4, ctx, nodes, 31)
    g = gen(3)
    for b in range(2):
        n = int(ctx[b]) + N
        k, v = randn((n, 2, D), FL, g), randn((n, 2, D), FL, g)
        v *= torch.exp2(torch.randint(-30, 31, (n, 1, 1), generator=g, device="cuda").float())
        v[::3] = 0
        if n > 600:
            v[:128] = 0                                   # whole tiles of zeros, first and later
            v[384:512] = 0
            v[256:384] *= 2.0 ** -60
        k[17] = q[b, 0, 0].float() * 2
        v[17] = 0
        binding.kv_write(cache, k, v, slots_of(table, ctx, 16, b, np.arange(n)))
    check_attention(q, cache, p, table, ctx, nodes)


@pytest.mark.parametrize("octave", [64, 72, 80, 88, 96, 104])
@pytest.mark.parametrize("N,Hq", FEW_AND_MANY)
def test_zeros_with_all_the_weight(N, Hq, octave):
    """8 bits: a row of zeros `octave` (in e) above all others' scores, 92 to 150 octaves
    of two: what is left of the others is 0 in every type, and the total is the zeros'."""
    D = 64
    q, cache, p, table, ctx, nodes = attn_case(1, N, Hq, 2, D, 16, BF, E4, [400], [N], 53)
    q[..., 0] = 8.0
    g = gen(2)
    n = 400 + N
    k, v = randn((n, 2, D), FL, g), randn((n, 2, D), FL, g)
    k[..., 0] = 0
    k[300], v[300] = 0, 0
    k[300, :, 0] = octave
    binding.kv_write(cache, k, v, slots_of(table, ctx, 16, 0, np.arange(n)))
    lse = torch.zeros((1, N, Hq), device="cuda")
    out = binding.tree_attention(q, cache, p, lse=lse)
    ref, rl, bound = NC.attention(q, cache, table, ctx, nodes, p.masks.cpu().numpy().view(np.uint32), 1 / 8)
    assert float((out.double() - ref).abs().max()) < 2.0 ** -80
    assert float((lse.double() - rl).abs().max()) < 2.0 ** -13      # scores within 2^-22 of sums below 250


@pytest.mark.parametrize("N,Hq", FEW_AND_MANY)
def test_all_values_zero(N, Hq):
    """8 bits, nothing but zeros over a long context: zeros, and the total still counts."""
    q, cache, p, table, ctx, nodes = attn_case(1, N, Hq, 2, 64, 64, BF, E4, [70000], [N], 37, vscale=0.0)
    assert not check_attention(q, cache, p, table, ctx, nodes).any()


@pytest.mark.parametrize("qdt,kind", [(HF, HF), (BF, E4), (HF, E4)])
@pytest.mark.parametrize("N,Hq", FEW_AND_MANY)
@pytest.mark.parametrize("dominant_at", [0, 59990])
def test_long_flat_tail(dominant_at, N, Hq, qdt, kind):
    """One token with nearly all the weight, 60000 with 2^-25.97 of it each: 9.1e-4 in all.
    f16 weights relative to the largest would be zero, all of them."""
    D, n = 64, 60000
    q, cache, p, table, ctx, nodes = attn_case(1, N, Hq, 2, D, 64, qdt, kind, [n], [N], 41)
    q = torch.zeros_like(q)
    q[..., 0] = 1.0
    src = FL if kind == E4 else kind
    k, v = torch.zeros((n + N, 2, D), device="cuda"), torch.zeros((n + N, 2, D), device="cuda")
    k[dominant_at, :, 0] = 18.0                            # 18 log2(e) = 25.97 octaves
    v[:, :, 1] = 1.0
    v[dominant_at, :, 0], v[dominant_at, :, 1] = 1.0, 0.0
    binding.kv_write(cache, k.to(src), v.to(src), slots_of(table, ctx, 64, 0, np.arange(n + N)))
    out = binding.tree_attention(q, cache, p, scale=1.0).double()
    m = p.masks.cpu().numpy().view(np.uint32)
    ref, _, _ = NC.attention(q, cache, table, ctx, nodes, m, 1.0)
    # a weight of 2^(8 - 25.97) of f16's steps of 2^-24 is off by 2^-7.03 of itself at
    # most, the output's rounding by 2^-9: 0.0096
    assert float(((out - ref).abs() / ref)[..., :2].max()) < 0.01
    assert not out[..., 2:].any()


# ---------------------------------------------------------------- queries

@pytest.mark.parametrize("qdt,kind", KINDS)
@pytest.mark.parametrize("N,Hq", FEW_AND_MANY)
def test_a_bad_query_that_sees_nothing_gives_zeros(N, Hq, qdt, kind):
    q, cache, p, table, ctx, nodes = attn_case(3, N, Hq, 2, 64, 16, qdt, kind, [0, 50, 0], [N, N, N - 1], 43)
    masks = p.masks.clone()
    masks[0, 1] = masks[0, 3] = masks[2, 2] = 0
    q[0, 1, 1, 5], q[0, 3, 0, 60], q[2, 2, :, 0] = math.nan, math.inf, -math.inf
    lse = torch.zeros((3, N, Hq), device="cuda")
    out = binding.tree_attention(q, cache, p, masks=masks, lse=lse)
    for b, v in ((0, 1), (0, 3), (2, 2)):
        assert not out[b, v].any() and bool((lse[b, v] == -math.inf).all())
    good = torch.ones((3, N), dtype=torch.bool, device="cuda")
    good[0, 1] = good[0, 3] = good[2, 2] = False
    ref, _, bound = NC.attention(q.nan_to_num(0, 0, 0), cache, table, ctx, nodes, masks.cpu().numpy().view(np.uint32), 1 / 8)
    assert bool(((out.double() - ref).abs() <= bound)[good].all())
    # a node past the tree, with such a query
    q[2, N - 1] = math.nan
    assert not binding.tree_attention(q, cache, p, masks=masks)[2, N - 1].any()


@pytest.mark.parametrize("qdt", [BF, HF])
@pytest.mark.parametrize("N,Hq", FEW_AND_MANY)
def test_outlier_channel_of_the_queries(N, Hq, qdt):
    """8 bits: one channel of the queries 300 times the others, on which the keys have
    nothing, so that the scores are the others'.  A query's channel is held to 2^-21.8
    of the row's largest (bf16 queries, many rows) or 2^-24, so a score to that times
    the sum of |k|."""
    D = 64
    q, cache, p, table, ctx, nodes = attn_case(2, N, Hq, 2, D, 16, qdt, E4, [333, 9000], [N, N], 47)
    g = gen(9)
    for b in range(2):
        n = int(ctx[b]) + N
        k = randn((n, 2, D), FL, g)
        k[..., 7] = 0
        binding.kv_write(cache, k, randn((n, 2, D), FL, g), slots_of(table, ctx, 16, b, np.arange(n)))
    q[..., 7] = 300 * (1 + q[..., 7].abs())
    held = 2.0 ** -21.8 if qdt == BF and N * Hq // 2 > 16 else 2.0 ** -24
    lse = torch.zeros((2, N, Hq), device="cuda")
    out = binding.tree_attention(q, cache, p, lse=lse).double()
    ref, rl, bound = NC.attention(q, cache, table, ctx, nodes, p.masks.cpu().numpy().view(np.uint32), 1 / 8)
    assert bool(((out - ref).abs() <= bound).all())
    for b in range(2):
        K, _ = NC.cache_rows(cache, table[b, :-(-(int(ctx[b]) + N) // 16)].long(), int(ctx[b]) + N)
        big = K.abs().sum(-1).amax(0)                                     # the largest sum of |k|, by key head
        off = q[b].double().abs().amax(-1) * big.repeat_interleave(Hq // 2) / 8 * (held + 2.0 ** -24)
        # scores' own sums (the seen channels' are below 200) to 2^-22, the total's to 2^-20
        assert bool(((lse[b].double() - rl[b]).abs() <= off + 200 * 2.0 ** -22 + 2.0 ** -20).all())


# ---------------------------------------------------------------- many rows: what few rows are tested for elsewhere

@pytest.mark.parametrize("qdt,kind", KINDS)
def test_many_rows_large_scores_and_scales_of_any_sign(qdt, kind):
    N, Hq = 12, 24
    case = attn_case(2, N, Hq, 2, 128, 16, qdt, kind, [300, 40], [N, N - 1], 7)
    q, rest = case[0], case[1:]
    check_attention(q * 40, *rest)
    check_attention(torch.zeros_like(q), *rest)
    check_attention(q, *rest, scale=0.0)
    check_attention(q, *rest, scale=-0.3)
    check_attention(q * 40, *rest, scale=-0.1)
    check_attention(q, *rest, scale=1e-6)
    check_attention(*attn_case(2, N, Hq, 2, 64, 16, qdt, kind, [300, 4000], [N, N], 8,
                               vscale=2.0 ** -40 if kind == E4 else 2.0 ** -6))


@pytest.mark.parametrize("qdt", [BF, HF])
def test_many_rows_zero_values_dominate(qdt):
    q, cache, p, table, ctx, nodes = attn_case(1, 12, 24, 2, 64, 16, qdt, E4, [400], [12], 51)
    g = gen(1)
    n = 412
    k, v = randn((n, 2, 64), FL, g), randn((n, 2, 64), FL, g)
    k[17], v[17] = q[0, 0, 0].float(), 0
    k[300], v[300] = q[0, 3, 20].float(), 0
    binding.kv_write(cache, k, v, slots_of(table, ctx, 16, 0, np.arange(n)))
    check_attention(q, cache, p, table, ctx, nodes)


@pytest.mark.parametrize("kind,pages", [(BF, 140000), (E4, 270000)])
@pytest.mark.parametrize("N,Hq", [(3, 8), (12, 24)])
def test_strides_stream_and_pages_past_32_bits(N, Hq, kind, pages):
    """Tokens before heads in the cache, queries inside a projection's output, the pages
    in use past 2^31 elements and 2^32 bytes of it, and a stream of its own."""
    g = gen(4)
    B, Hkv, D, page = 2, 2, 128, 64
    dt = torch.uint8 if kind == E4 else kind
    assert pages * page * Hkv * D > 2 ** 31 and pages * page * Hkv * D * dt.itemsize > 2 ** 32
    base = torch.empty((pages, page, Hkv, D), dtype=dt, device="cuda")
    both = base.transpose(1, 2)                                   # one tensor: keys equal values
    scales = [torch.full((pages, Hkv, page), 127, dtype=torch.uint8, device="cuda")] * 2 if kind == E4 else []
    cache = binding.KVCache(both, both, *scales)
    ctx, nodes = np.array([150, 511], np.int32), np.array([N, N - 1], np.int32)
    par = np.zeros((B, N), np.int32)
    par[:, 0] = -1
    table = (pages - 1 - np.arange(18, dtype=np.int32)).reshape(2, 9)
    p = binding.tree_plan(dev(par), dev(nodes), dev(ctx), dev(table), cache)
    for b in range(B):
        t = np.arange(int(ctx[b] + nodes[b]))
        x = randn((len(t), Hkv, D), BF, g)
        binding.kv_write(cache, x, x, slots_of(dev(table), ctx, page, b, t))
    q = randn((B, N, Hq + 4, D), BF, g)[:, :, 2:2 + Hq]
    want = check_attention(q, cache, p, dev(table), ctx, nodes)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = binding.tree_attention(q, cache, p, stream=side)
    side.synchronize()
    assert torch.equal(got, want)


# ---------------------------------------------------------------- a step in a CUDA graph

@pytest.mark.parametrize("qdt,kind", KINDS)
@pytest.mark.parametrize("N,Hq", FEW_AND_MANY)
def test_step_in_a_graph(N, Hq, qdt, kind):
    """Plan, write, attention and commit of two layers captured once and replayed over
    changing lengths: the same bits as the calls themselves."""
    B, Hkv, D, page = 3, 2, 64, 16
    g = gen(6)
    rng = np.random.default_rng(6)
    top = np.array([900, 8000, 60])
    table, pages = NC.make_table(rng, top, [N] * B, page)
    table = dev(table.clip(0))
    caches = [binding.new_kv_cache(pages, page, Hkv, D, dtype=kind) for _ in range(4)]
    src = qdt if kind == E4 else kind
    every = torch.arange(pages * page, device="cuda")
    for a, b in zip(caches[:2], caches[2:]):
        x, y = randn((pages * page, Hkv, D), src, g), randn((pages * page, Hkv, D), src, g)
        binding.kv_write(a, x, y, every)
        binding.kv_write(b, x, y, every)
    rot = binding.rope_table(D)
    ctx = torch.zeros(B, dtype=torch.int32, device="cuda")
    par = dev(NC.random_tree(rng, B, N))
    nodes = torch.zeros(B, dtype=torch.int32, device="cuda")
    last = torch.zeros(B, dtype=torch.int32, device="cuda")
    q, k, v = randn((B, N, Hq, D), src, g), randn((B, N, Hkv, D), src, g), randn((B, N, Hkv, D), src, g)

    def step(caches):
        p = binding.tree_plan(par, nodes, ctx, table, caches[0])
        outs = []
        for c in caches:
            t = binding.kv_write(c, k, v, p.slots.view(-1), positions=p.positions.view(-1), table=rot, q=q)
            outs.append(binding.tree_attention(t.view(B, N, Hq, D), c, p))
        return outs + [binding.kv_commit(caches, p, last)]

    def lengths(i):
        ctx.copy_(dev((top * [0.1, 1.0, 0.5][i]).astype(np.int32)))
        nodes.copy_(dev(np.array([[N, 1, N - 1], [N, N, N], [1, N, 2]][i], np.int32)))
        last.copy_(nodes - 1)

    lengths(0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(caches[:2])
    torch.cuda.current_stream().wait_stream(side)
    step(caches[2:])                                            # both sets of caches alike again
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step(caches[:2])
    for i in (1, 0, 2, 1):
        lengths(i)
        graph.replay()
        got = [o.clone() for o in outs]
        want = step(caches[2:])
        for a, b in zip(got, want):
            assert torch.equal(a, b)
    for a, b in zip(caches[:2], caches[2:]):
        assert torch.equal(a.k, b.k) and torch.equal(a.v, b.v)
