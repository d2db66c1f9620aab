"""Causal attention over packed prompts against its 64-bit form: types, heads, lengths, strides, windows, rows that see
nothing, what a row does not see, and the plan."""
import math

import numpy as np
import pytest
import torch

import prompt_common as P
from gpu_common import ensure_built
from speculative_decoding_verification_51_gb300 import binding

pytestmark = pytest.mark.gpu
BF, HF = torch.bfloat16, torch.float16


@pytest.fixture(scope="module", autouse=True)
def built():
    ensure_built()


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def randn(shape, dt, g, scale=1.0):
    return (scale * torch.randn(shape, generator=g, device="cuda")).to(dt)


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def case(lens, Hq, Hkv, D, dt, seed, ahead=None, front=0, pad=0):
    """(q, k, v, off, koff): `ahead` more keys than queries; `front` and `pad` rows of no prompt."""
    g = gen(seed)
    off = P.offsets(lens, front)
    koff = off if ahead is None else P.offsets([max(0, n + a) for n, a in zip(lens, ahead)])
    T, M = off[-1] + pad, off[-1] + pad if ahead is None else koff[-1]
    return randn((T, Hq, D), dt, g, 1.5), randn((M, Hkv, D), dt, g), randn((M, Hkv, D), dt, g), off, koff


def make_plan(q, k, off, koff, **kw):
    if koff is off:
        return binding.prompt_plan(i32(off), q.shape[0], q.shape[1], k.shape[1], **kw)
    return binding.prompt_plan(i32(off), q.shape[0], q.shape[1], k.shape[1], k_offsets=i32(koff), num_keys=k.shape[0], **kw)


def check(q, k, v, off, koff, window=0, scale=None, plan=None):
    plan = plan or make_plan(q, k, off, koff)
    out = torch.full(q.shape, 7.0, dtype=q.dtype, device="cuda")
    lse = torch.full(q.shape[:2], 7.0, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    binding.prompt_attention(q, k, v, plan, window=window, scale=scale, out=out, lse=lse, dev_status=status)
    want, wl, bound, bl = P.attention(q, k, v, off, koff, scale or 1 / math.sqrt(q.shape[2]), window)
    assert int(status) == 0
    mine = torch.zeros(q.shape[0], dtype=torch.bool, device="cuda")
    mine[off[0]:off[-1]] = True
    assert bool((out[~mine] == 7).all()) and bool((lse[~mine] == 7).all())
    got, want, bound = out[mine].double(), want[mine], bound[mine]
    fine = want.isfinite()
    assert torch.equal(fine, got.isfinite())
    assert torch.equal(want.isnan(), got.isnan())
    far = ((got - want).abs() - bound)[fine]
    assert far.numel() == 0 or float(far.max()) <= 0, float(far.max())
    inf = want.isinf()
    assert torch.equal(got[inf], want[inf])
    gl, wl, bl = lse[mine].double(), wl[mine], bl[mine]
    fine = wl.isfinite()
    assert torch.equal(gl[~fine].nan_to_num(5, 6, 7), wl[~fine].nan_to_num(5, 6, 7))
    assert fine.sum() == 0 or float(((gl - wl).abs() - bl)[fine].max()) <= 0
    return out


@pytest.mark.parametrize("dt", [BF, HF])
@pytest.mark.parametrize("D", [8, 64, 72, 128, 136, 256])
def test_head_sizes(D, dt):
    check(*case([1, 200, 129, 64], 4, 2, D, dt, D))


@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (3, 3), (8, 1), (14, 2), (12, 4), (128, 1), (100, 1), (65, 1)])
def test_groups_of_heads(Hq, Hkv):
    check(*case([150, 3, 1, 40], Hq, Hkv, 64, BF, Hq))
    check(*case([33, 257], Hq, Hkv, 128, HF, Hq))


@pytest.mark.parametrize("lens", [[1], [2], [127], [128], [129], [255], [256], [257], [384, 0, 1, 0], [0, 0, 5], [1] * 40,
                                  [700, 31, 512, 513]])
@pytest.mark.parametrize("D", [64, 128, 192])
def test_lengths(lens, D):
    check(*case(lens, 2, 1, D, BF, len(lens)))


def test_no_tokens():
    q, k, v, off, koff = case([0, 0], 2, 1, 64, BF, 0, pad=3)
    check(q, k, v, off, koff)
    e = q[:0]
    plan = binding.prompt_plan(i32([0, 0]), 0, 2, 1)
    assert binding.prompt_attention(e, k[:0], v[:0], plan).shape == (0, 2, 64)
    plan = binding.prompt_plan(i32([0]), 3, 2, 1)
    out = torch.full_like(q, 3.0)
    binding.prompt_attention(q, k, v, plan, out=out)
    assert bool((out == 3).all())


@pytest.mark.parametrize("D", [64, 256])
def test_no_keys(D):
    """Queries without any key: zeros, and no key tensor is touched."""
    q = randn((40, 4, D), BF, gen(1))
    k = torch.empty((0, 2, D), dtype=BF, device="cuda")
    out = check(q, k, k, [0, 33, 40], [0, 0, 0])
    assert bool((out == 0).all())


@pytest.mark.parametrize("D", [64, 128, 256])
def test_keys_ahead_and_queries_that_see_nothing(D):
    """With fewer keys than queries the first queries see nothing: zeros."""
    q, k, v, off, koff = case([5, 130, 1, 200, 7], 4, 2, D, BF, 5, ahead=[300, 1000, 129, -150, -7], pad=4)
    out = check(q, k, v, off, koff)
    assert bool((out[off[3]:off[3] + 150] == 0).all()) and bool((out[off[4]:off[5]] == 0).all())


@pytest.mark.parametrize("window", [1, 2, 63, 128, 129, 300, 5000, 2 ** 31 - 1])
@pytest.mark.parametrize("Hq,D", [(4, 128), (1, 64), (2, 256)])
def test_windows(window, Hq, D):
    check(*case([700, 90, 1, 260], Hq, 1, D, BF, window % 97), window=window)
    check(*case([50, 300], Hq, 1, D, HF, window % 89, ahead=[900, 77]), window=window)


@pytest.mark.parametrize("dt", [BF, HF])
@pytest.mark.parametrize("D,Hq,Hkv,window", [(64, 4, 2, 0), (128, 4, 2, 0), (128, 3, 3, 100), (256, 2, 1, 0), (128, 128, 1, 0)])
def test_many_items_a_cta(D, Hq, Hkv, window, dt):
    """Items of one step to many behind one another, row tiles without tokens or keys among them."""
    rng = np.random.default_rng(D + Hq)
    lens = rng.choice([0, 1, 2, 30, 64, 65, 127, 128, 129, 200, 300, 513], 300 if Hq < 100 else 24).tolist()
    ahead = rng.choice([0, 0, 0, 5, 128, -1, -64, -130, 400], len(lens)).tolist()
    check(*case(lens, Hq, Hkv, D, dt, 21, ahead=ahead), window=window)


def test_marks_belong_to_their_item():
    """Values that are not finite in some items of a CTA's and not in others."""
    lens = [200] * 250
    q, k, v, off, koff = case(lens, 4, 2, 64, BF, 13)
    for b in range(0, 250, 7):
        v[off[b] + 30 * (b % 6), b % 2, b % 64] = (math.nan, math.inf, -math.inf)[b % 3]
    check(q, k, v, off, koff)


def test_front_rows_and_rows_behind():
    check(*case([100, 50], 4, 2, 64, BF, 1, front=13, pad=29))


@pytest.mark.parametrize("D", [64, 128, 256])
def test_large_scores_and_scale(D):
    """References that have to be raised again and again, and weights that vanish."""
    g = gen(3)
    q, k, v, off, koff = case([600], 2, 1, D, BF, 3)
    k = (k.float() * torch.linspace(0.1, 6, 600, device="cuda")[:, None, None]).to(BF)
    check(q, k, v, off, koff)
    check(q, k, v, off, koff, scale=2.0)
    check(q.half(), k.half(), v.half(), off, koff, scale=0.7)
    assert g is not None


def test_strides():
    g = gen(7)
    lens = [90, 1, 200]
    off = P.offsets(lens)
    T = off[-1]
    qkv = randn((T, 8 + 2 + 2, 128), BF, g)
    check(qkv[:, :8], qkv[:, 8:10], qkv[:, 10:], off, off)
    q = randn((8, T, 128), BF, g).transpose(0, 1)
    k, v = (randn((T, 3, 2, 136), BF, g)[:, 1, :, :128] for _ in range(2))
    check(q, k, v, off, off)
    check(q, k[:, :1].expand(T, 2, 128), v[:, :1].expand(T, 2, 128), off, off)     # one head for both


@pytest.mark.parametrize("dt", [BF, HF])
@pytest.mark.parametrize("D,Hq", [(64, 3), (128, 4), (256, 2)])
@pytest.mark.parametrize("window", [0, 60])
def test_what_is_not_seen_has_no_effect(D, Hq, dt, window):
    """Infinities and NaN: of keys and values behind a query, of the next prompt, of rows of no prompt."""
    q, k, v, off, koff = case([150, 133, 300], Hq, 1, D, dt, 9, pad=40)
    for x in (k, v):
        x[off[-1]:] = math.nan
    v[off[0] + 140, 0, 3] = math.nan
    v[off[0] + 145, 0, 5] = math.inf
    v[off[1] + 5, 0, 1] = -math.inf
    v[off[1] + 5, 0, D - 1] = math.nan
    v[off[2] + 200, 0, 0] = math.inf
    k[off[1] + 131, 0, 2] = math.nan                       # seen by that prompt's last two queries
    q[off[2] + 7] = math.nan                               # a query's own
    plan = make_plan(q, k, off, koff)
    out, lse = torch.empty_like(q), torch.empty(q.shape[:2], device="cuda")
    binding.prompt_attention(q, k, v, plan, window=window, out=out, lse=lse)
    clean = [x.nan_to_num(0, 0, 0) for x in (q, k, v)]
    want, _, bound, _ = P.attention(*clean, off, koff, 1 / math.sqrt(D), window)
    touched = torch.zeros(q.shape, dtype=torch.bool, device="cuda")

    def seen_from(b, key):
        last = off[b + 1] if not window else min(off[b + 1], off[b] + key + window)
        return slice(off[b] + key, last)
    touched[seen_from(0, 140), :, 3] = True
    touched[seen_from(0, 145), :, 5] = True
    touched[seen_from(1, 5), :, 1] = True
    touched[seen_from(1, 5), :, D - 1] = True
    touched[seen_from(2, 200), :, 0] = True
    touched[seen_from(1, 131)] = True
    touched[off[2] + 7] = True
    touched[off[-1]:] = True
    got = out.double()
    assert bool(got[~touched].isfinite().all())
    assert float(((got - want).abs() - bound)[~touched].max()) <= 0
    assert bool(got[seen_from(0, 140), :, 3].isnan().all())
    assert bool((got[seen_from(0, 145), :, 5] == math.inf).all())
    first = seen_from(1, 5)
    assert bool((got[first.start:min(first.stop, off[1] + 131), :, 1] == -math.inf).all())
    assert bool(lse[off[1]:off[1] + 131].isfinite().all()) and bool(lse[off[1] + 131:off[2]].isnan().all())


def test_same_bits_every_time_and_under_a_graph():
    q, k, v, off, koff = case([300, 77, 1000], 8, 2, 128, BF, 11)
    plan = make_plan(q, k, off, koff)
    want = binding.prompt_attention(q, k, v, plan)
    for _ in range(3):
        assert torch.equal(binding.prompt_attention(q, k, v, plan), want)
    o = i32(off)
    out = torch.zeros_like(q)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        p2 = binding.prompt_plan(o, q.shape[0], 8, 2)
        binding.prompt_attention(q, k, v, p2, out=out)
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        p2 = binding.prompt_plan(o, q.shape[0], 8, 2)
        binding.prompt_attention(q, k, v, p2, out=out)
    out.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    # other lengths in the captured call: rows behind the last prompt stay
    off2 = [0, 10, 400, 500]
    o.copy_(i32(off2))
    out.fill_(9)
    graph.replay()
    w2 = P.attention(q, k, v, off2, off2, 1 / math.sqrt(128))
    assert float(((out.double() - w2[0]).abs() - w2[2])[:500].max()) <= 0
    assert bool((out[500:] == 9).all())


def test_streams():
    q, k, v, off, koff = case([300, 77, 400], 8, 2, 64, BF, 12)
    plan = make_plan(q, k, off, koff)
    want = binding.prompt_attention(q, k, v, plan)
    streams = [torch.cuda.Stream() for _ in range(3)]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got = [binding.prompt_attention(q, k, v, plan, stream=streams[i % 3]) for i in range(12)]
    torch.cuda.synchronize()
    assert all(torch.equal(x, want) for x in got)


# ---------------------------------------------------------------- the plan

def plan_words(plan):
    w = plan.buffer.cpu().numpy().view(np.int32)
    items = w[64:64 + 8 * w[0]].reshape(-1, 8)
    return w[:4].tolist(), items


@pytest.mark.parametrize("Hq,Hkv", [(4, 1), (7, 1), (2, 2), (128, 1)])
@pytest.mark.parametrize("seed", range(3))
def test_plan(Hq, Hkv, seed):
    rng = np.random.default_rng(seed)
    B = int(rng.integers(1, 3000 if seed == 2 else 40))
    lens = rng.integers(0, 400, B).tolist()
    ahead = rng.integers(-50, 300, B).tolist() if seed else None
    off = P.offsets(lens, 3)
    koff = off if ahead is None else P.offsets([max(0, n + a) for n, a in zip(lens, ahead)])
    page = 16
    keys = [b - a for a, b in zip(koff, koff[1:])]
    width = max(1, max(-(-m // page) for m in keys))
    table = rng.permutation(B * width).astype(np.int32).reshape(B, width)
    cache = binding.new_kv_cache(B * width, page, Hkv, 8)
    T = off[-1] + 5
    kw = dict() if ahead is None else dict(k_offsets=i32(koff), num_keys=koff[-1])
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    p = binding.prompt_plan(i32(off), T, Hq, Hkv, page_table=torch.from_numpy(table).cuda(), cache=cache, dev_status=status, **kw)
    assert int(status) == 0
    pos, slots = np.zeros(T, np.int64), np.full(T, -1, np.int64)
    want = set()
    each = 2 * (128 // (Hq // Hkv))
    for b in range(B):
        n, m = lens[b], keys[b]
        for i in range(n):
            pos[off[b] + i] = at = m - n + i
            if at >= 0:
                slots[off[b] + i] = table[b, at // page] * page + at % page
        for i in range(0, n, each):
            want.add((off[b] + i, min(each, n - i), koff[b], m - n + i, m))
    assert np.array_equal(p.positions.cpu().numpy(), pos) and np.array_equal(p.slots.cpu().numpy(), slots)
    head, items = plan_words(p)
    assert head == [len(want), T, T if ahead is None else koff[-1], each // 2]
    assert {tuple(x[:5]) for x in items.tolist()} == want
    seen = np.maximum(items[:, 3] + items[:, 1], 0)
    assert np.all(np.diff(seen) <= 0) if seen.max(initial=0) < 2048 else True


@pytest.mark.parametrize("off,koff", [([0, 5, 3, 8], None), ([-1, 5], None), ([0, 9], None), ([0, 5], [0, 100]), ([0, 5], [4, 3]),
                                      ([0, 2 ** 31 - 1], None), ([0, 5], [-(2 ** 31), 5])])
def test_bad_offsets(off, koff):
    """A batch whose offsets fall or leave their tensors has no tokens, and says so."""
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    kw = {} if koff is None else dict(k_offsets=i32(koff), num_keys=8)
    p = binding.prompt_plan(i32(off), 8, 2, 1, dev_status=status, **kw)
    assert int(status) == binding.BADBIT["offsets"]
    assert bool((p.positions == 0).all()) and plan_words(p)[0][0] == 0
    g = gen(0)
    q, k, v = randn((8, 2, 64), BF, g), randn((8, 1, 64), BF, g), randn((8, 1, 64), BF, g)
    out = torch.full_like(q, 2.0)
    binding.prompt_attention(q, k, v, p, out=out)
    assert bool((out == 2).all())


def test_pages_outside():
    cache = binding.new_kv_cache(4, 16, 1, 8)
    table = i32([[0, 9, 3], [-1, 2, 1]])
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    p = binding.prompt_plan(i32([0, 60, 80]), 80, 1, 1, page_table=table, cache=cache, dev_status=status)
    assert int(status) == binding.BADBIT["page"]
    s = p.slots.cpu().tolist()
    assert s[:16] == list(range(16)) and s[16:32] == [-1] * 16 and s[32:48] == list(range(48, 64)) and s[48:60] == [-1] * 12
    assert s[60:76] == [-1] * 16 and s[76:80] == [32, 33, 34, 35]


def test_a_plan_of_other_sizes_is_not_used():
    """The kernel checks the plan's own sizes (the wrapper's fields can be set)."""
    q, k, v, off, koff = case([40, 20], 4, 2, 64, BF, 1)
    plan = binding.prompt_plan(i32([0, 300, 1000]), 1000, 4, 2)
    plan.num_tokens = plan.num_keys = 60
    out = torch.full_like(q, 5.0)
    binding.prompt_attention(q, k, v, plan, out=out)
    assert bool((out == 5).all())
