"""Log probabilities of given tokens, entropy and alternatives against their 64-bit form."""
import math

import pytest
import torch

import prompt_common as P
from gpu_common import ensure_built
from speculative_decoding_verification_51_gb300 import binding

pytestmark = pytest.mark.gpu
BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def built():
    ensure_built()


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def make(E, V, dt, seed, scale=3.0):
    return (scale * torch.randn((E, V), generator=gen(seed), device="cuda")).to(dt)


def most(x):
    return float(x.max()) if x.numel() else 0.0


def check(x, tokens, temperature=None, top=0, rows=None, logits=None, status_bits=0):
    """x [E, V]: what each entry reads."""
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    r = binding.token_logprobs(x if logits is None else logits, tokens, rows=rows, temperature=temperature, top=top, entropy=True,
                               dev_status=status)
    assert int(status) == status_bits
    there = (tokens >= 0).flatten()
    T = None if temperature is None else temperature.flatten()
    lp, h, ids, best = P.logprobs(x, tokens.flatten(), T, top)
    Td = 1.0 if T is None else torch.where(T == 0, torch.ones_like(T), T).double()
    b = P.logprob_bound(x, Td)
    at = x.double().gather(1, tokens.flatten().long().clamp(min=0)[:, None])[:, 0]
    got = r.logprobs.flatten().double()
    fin = lp.isfinite() & there
    assert most(((got - lp).abs() - b(torch.where(fin, at, torch.zeros_like(at))))[fin]) <= 0
    assert bool((got[~there] == 0).all()) and torch.equal(got[there & ~fin], lp[there & ~fin])
    # the entropy: its terms p (a - log Z) are off by the same, relative to at most 1 + H
    hb = b(x.double().where(x.isfinite(), torch.zeros_like(x).double()).amax(-1)) * 4 * (2 + h)
    assert most(((r.entropy.flatten().double() - h).abs() - hb)[there]) <= 0
    assert bool((r.entropy.flatten()[~there] == 0).all())
    if top:
        gi, gl = r.top_ids.view(-1, top), r.top_logprobs.view(-1, top).double()
        assert torch.equal(gi[there].long(), ids[there]) and bool((gi[~there] == -1).all())
        val = x.double().gather(1, ids.clamp(min=0))
        some = (ids >= 0) & there[:, None]
        for i in range(top):
            assert most(((gl[:, i] - best[:, i]).abs() - b(val[:, i]))[some[:, i]]) <= 0
        assert bool((gl[there] == -math.inf)[(ids < 0)[there]].all()) and bool((gl[~there] == 0).all())
    else:
        assert r.top_ids is None and r.top_logprobs is None
    # without entropy: the same bits
    r2 = binding.token_logprobs(x if logits is None else logits, tokens, rows=rows, temperature=temperature, top=top)
    assert torch.equal(r2.logprobs, r.logprobs) and r2.entropy is None
    if top:
        assert torch.equal(r2.top_ids, r.top_ids) and torch.equal(r2.top_logprobs, r.top_logprobs)
    return r


def some_tokens(E, V, seed):
    return torch.randint(0, V, (E,), generator=gen(seed), device="cuda").to(torch.int32)


@pytest.mark.parametrize("dt", [BF, HF, F32])
@pytest.mark.parametrize("V", [1, 2, 7, 8, 33, 511, 512, 513, 1000, 4097, 32000, 50001, 151936])
def test_vocabularies(V, dt):
    for E in (1, 5):
        check(make(E, V, dt, V + E), some_tokens(E, V, V), top=min(32, V + 3) if V < 600 else 20)


@pytest.mark.parametrize("E", [1, 2, 40, 151, 303, 304, 700])
@pytest.mark.parametrize("top", [0, 1, 32])
def test_rows_by_one_cta_and_by_several(E, top):
    V = 20011
    t = some_tokens(E, V, E)
    t[::3] = -1
    check(make(E, V, BF, E), t, top=top)


@pytest.mark.parametrize("dt", [BF, F32])
def test_temperatures(dt):
    E, V = 12, 5003
    T = torch.tensor([0.0, 1.0, 0.3, 1.7, 1e-3, 1e-20, 100.0, 1e-45, 1e30, 0.5, 2.0, 0.9], device="cuda")
    x = make(E, V, dt, 4)
    r = check(x[:7], some_tokens(7, V, 5), temperature=T[:7], top=5)
    plain = binding.token_logprobs(x[:2], some_tokens(7, V, 5)[:2], top=5)
    assert torch.equal(r.logprobs[:2], plain.logprobs)
    big = binding.token_logprobs(x, some_tokens(E, V, 5), temperature=T, entropy=True)
    assert not bool(big.logprobs.isnan().any()) and not bool(big.entropy.isnan().any())
    best = x.float().argmax(1).to(torch.int32)
    r = binding.token_logprobs(x, best, temperature=T, entropy=True)
    one = (x.float() == x.float().amax(1, keepdim=True)).sum(1)
    for i in (5, 7):                                                    # all of the mass on the largest
        assert abs(float(r.logprobs[i]) + math.log(int(one[i]))) < 1e-5 and abs(float(r.entropy[i]) - math.log(int(one[i]))) < 1e-5
    assert abs(float(r.entropy[8]) - math.log(V)) < 1e-4                # flat


def test_ties_take_the_lowest_index():
    V = 3000
    x = torch.zeros((6, V), dtype=BF, device="cuda")
    x[1] = -math.inf
    x[1, [2999, 17, 1500]] = 2.0
    x[2, ::2] = -0.0                                                    # equal to 0
    x[3] = torch.arange(V, device="cuda") // 100
    x[4] = 5.0
    x[4, 40:] = 5.0
    x[5, 1024:] = 1.0
    check(x, some_tokens(6, V, 1).clamp(min=0) * 0 + 17, top=32)
    big = torch.full((400, 30011), 1.5, dtype=F32, device="cuda")       # by one CTA: more equal ones than there is room for
    big[:, 29000] = 2.0
    r = binding.token_logprobs(big, torch.zeros(400, dtype=torch.int32, device="cuda"), top=20)
    assert torch.equal(r.top_ids, torch.tensor([29000] + list(range(19)), dtype=torch.int32, device="cuda").expand(400, 20))


def test_masked_tokens_and_rows():
    V = 2048
    x = make(5, V, F32, 2)
    x[0, 100:] = -math.inf
    x[1, :-3] = -math.inf
    x[2] = -math.inf
    x[2, 7] = 3.0
    x[3] = torch.finfo(F32).min                                         # a mask of the lowest value: a flat row
    x[4, 5] = torch.finfo(F32).min
    t = torch.tensor([500, V - 1, 7, 3, 5], dtype=torch.int32, device="cuda")
    r = check(x, t, top=8)
    assert float(r.logprobs[0]) == -math.inf and float(r.logprobs[2]) == 0 and float(r.entropy[2]) == 0
    assert abs(float(r.logprobs[3]) + math.log(V)) < 1e-5
    x[2] = -math.inf
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    r = binding.token_logprobs(x, t, top=3, entropy=True, dev_status=status)
    assert int(status) == binding.BADBIT["empty_row"]
    assert float(r.logprobs[2]) == -math.inf and float(r.entropy[2]) == 0 and r.top_ids[2].tolist() == [-1] * 3
    assert bool(r.logprobs[4] < -1e30)


def test_values_that_are_not_finite():
    x = make(4, 5000, BF, 3)
    x[1, 7], x[2, 4999], x[3, 0] = math.nan, math.inf, math.nan
    r = binding.token_logprobs(x, torch.tensor([1, 2, 3, 4], dtype=torch.int32, device="cuda"), top=4, entropy=True)
    assert r.logprobs.isnan().tolist() == [False, True, True, True] == r.entropy.isnan().tolist()
    assert int(r.top_ids[2, 0]) == 4999 and bool(((r.top_ids >= -1) & (r.top_ids < 5000)).all())


def test_bad_entries():
    x = make(6, 1000, BF, 4)
    t = torch.tensor([5, 1000, 2 ** 31 - 1, 7, 8, -5], dtype=torch.int32, device="cuda")
    T = torch.tensor([1.0, 1.0, 1.0, -1.0, math.nan, 1.0], device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    r = binding.token_logprobs(x, t, temperature=T, top=2, entropy=True, dev_status=status)
    assert int(status) == binding.BADBIT["token"] | binding.BADBIT["temperature"]
    assert float(r.logprobs[0]) < 0 and bool((r.logprobs[1:] == 0).all()) and bool((r.top_ids[1:] == -1).all())
    rows = torch.tensor([5, 6, -1, 0, 1, 2], dtype=torch.int32, device="cuda")
    status.zero_()
    r = binding.token_logprobs(x, t.clamp(0, 999), rows=rows, dev_status=status)
    assert int(status) == binding.BADBIT["token"] and (r.logprobs == 0).tolist() == [False, True, True, False, False, False]


@pytest.mark.parametrize("dt", [BF, HF, F32])
def test_rows_and_strides(dt):
    V = 1003
    wide = make(40, V + 24, dt, 6)
    for first in (0, 1, 5):                                             # rows that begin anywhere
        x = wide[:, first:first + V]
        rows = torch.tensor([[3, 3, 39], [0, 17, 21]], dtype=torch.int32, device="cuda")
        t = torch.tensor([[5, V - 1, 0], [-1, 7, 500]], dtype=torch.int32, device="cuda")
        check(x[rows.flatten().long()], t, top=6, rows=rows, logits=x)
        check(x.contiguous(), some_tokens(40, V, 1), top=3, logits=x)
    x = make(24, V, dt, 7)
    shaped = x.view(4, 6, V)
    t = some_tokens(24, V, 2)
    want = binding.token_logprobs(x, t, top=4, entropy=True)
    got = binding.token_logprobs(shaped, t.view(4, 6), top=4, entropy=True)
    assert got.logprobs.shape == (4, 6) and got.top_ids.shape == (4, 6, 4)
    assert torch.equal(got.logprobs.flatten(), want.logprobs) and torch.equal(got.top_ids.view(24, 4), want.top_ids)
    cut = shaped[:, :5]
    with pytest.raises(ValueError, match="run of rows"):
        binding.token_logprobs(cut, t.view(4, 6)[:, :5].contiguous())


def test_no_entries():
    x = make(3, 100, BF, 1)
    e = torch.zeros(0, dtype=torch.int32, device="cuda")
    r = binding.token_logprobs(x, e, rows=e, top=3, entropy=True)
    assert r.logprobs.shape == (0,) and r.top_ids.shape == (0, 3)
    assert binding.token_logprobs(x[:0], e).logprobs.shape == (0,)


def test_large_vocabulary():
    """Groups of several units."""
    V = (1 << 21) + 77
    x = make(2, V, BF, 8)
    check(x, some_tokens(2, V, 3), top=32)
    check(x.expand(2, V)[:1].repeat(310, 1), some_tokens(310, V, 4), top=2)


def test_same_bits_and_a_graph():
    x = make(20, 151936, BF, 9)
    t = some_tokens(20, 151936, 5)
    want = binding.token_logprobs(x, t, top=20, entropy=True)
    room = torch.full((int(binding.lib().spec_token_logprobs_workspace_size(20, 151936)),), 0xff, dtype=torch.uint8, device="cuda")
    for _ in range(3):
        r = binding.token_logprobs(x, t, top=20, entropy=True, workspace=room)
        assert all(torch.equal(getattr(r, n), getattr(want, n)) for n in ("logprobs", "entropy", "top_ids", "top_logprobs"))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        binding.token_logprobs(x, t, top=20)
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r = binding.token_logprobs(x, t, top=20, entropy=True)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(r.logprobs, want.logprobs) and torch.equal(r.top_ids, want.top_ids)
    x.copy_(make(20, 151936, BF, 10))
    w2 = binding.token_logprobs(x, t, top=20)
    graph.replay()
    assert torch.equal(r.logprobs, w2.logprobs) and torch.equal(r.top_ids, w2.top_ids)


def test_of_a_verification():
    """spec_verify's ids go in as they are: the emitted tokens of each request under their rows."""
    from speculative_decoding_verification_51_gb300 import workloads as W
    w = W.make_workload(2, device="cuda:0")
    ids, acc = binding.spec_verify(w.target_logits, w.draft_probs, w.draft_ids, w.num_draft, w.temperature, w.seed)
    B, K1, V = w.target_logits.shape
    T = w.temperature[:, None].expand(B, K1).contiguous()
    r = binding.token_logprobs(w.target_logits, ids, temperature=T, top=3)
    lp, _, top, _ = P.logprobs(w.target_logits.view(-1, V), ids.flatten(), T.flatten(), 3)
    there = ids.flatten() >= 0
    assert float((r.logprobs.flatten().double() - lp).abs()[there].max()) < 1e-4
    assert torch.equal(r.top_ids.view(-1, 3)[there].long(), top[there])
