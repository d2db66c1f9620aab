"""The prompt's operators on tensors of more than 2^31 elements (4 GB of 16 bits): what is read and written lies past 32
bits of an offset.  Each against the same call on a copy of the last rows, or the 64-bit form."""
import math

import pytest
import torch

import prompt_common as P
from gpu_common import ensure_built
from speculative_decoding_verification_51_gb300 import binding

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def built():
    ensure_built()


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


@pytest.mark.parametrize("D", [128, 256])
def test_prompts_behind_many_rows(D):
    H, T, lens = 16, 2 ** 32 // (16 * D) // 2 + 1000, [130, 1, 300]
    off = P.offsets(lens, T - sum(lens))
    near = P.offsets(lens)
    q, k, v = (torch.zeros((T, H, D), dtype=BF, device="cuda") for _ in range(3))
    for t, seed in ((q, 1), (k, 2), (v, 3)):
        t[off[0]:] = torch.randn((sum(lens), H, D), generator=gen(seed), device="cuda").to(BF)
    v[off[2] + 40, 3, 5] = math.inf  # (read again from where it lies)
    out = torch.full((T, H, D), 7.0, dtype=BF, device="cuda")
    lse = torch.full((T, H), 7.0, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    plan = binding.prompt_plan(i32(off), T, H, H, dev_status=status)
    assert q.numel() > 2 ** 31
    binding.prompt_attention(q, k, v, plan, out=out, lse=lse, dev_status=status)
    assert int(status) == 0
    a, b, c = (t[off[0]:].clone() for t in (q, k, v))
    lse_near = torch.zeros(a.shape[:2], device="cuda")
    want = binding.prompt_attention(a, b, c, binding.prompt_plan(i32(near), sum(lens), H, H), lse=lse_near)
    assert torch.equal(out[off[0]:], want) and torch.equal(lse[off[0]:], lse_near)
    assert bool(want[near[2] + 40:, 3, 5].isinf().all()) and int(want.isinf().sum()) == 300 - 40
    assert bool((out[:off[0]] == 7).all()) and bool((lse[:off[0]] == 7).all())
    assert torch.equal(plan.positions[off[2]:].cpu(), torch.arange(300, dtype=torch.int32))


def test_norms_of_many_rows():
    D, H = 128, 16
    T = 2 ** 31 // (H * D) + 100
    table = binding.rope_table(64)
    norm = binding.HeadNorm(1.0 + 0.3 * torch.randn(D, generator=gen(1), device="cuda"))
    x = torch.zeros((T, H, D), dtype=BF, device="cuda")
    x[-300:] = torch.randn((300, H, D), generator=gen(2), device="cuda").to(BF)
    x[:300] = x[-300:]
    pos = torch.arange(T, dtype=torch.int32, device="cuda")
    pos[:300] = pos[-300:]
    y = binding.rope(x, None, pos, table, norm=norm)
    assert torch.equal(y[:300], y[-300:]) and bool((y[300:-300] == 0).all())
    want = binding.rope(x[-300:].clone(), None, pos[-300:].clone(), table, norm=norm)
    # (another share of the heads a CTA, the same arithmetic)
    assert torch.equal(want, y[-300:])
    binding.rope(x, None, pos, table, out_q=x, norm=norm)
    assert torch.equal(x[-300:], want) and torch.equal(x[:300], want)


def test_logits_of_many_rows():
    V = 151936
    R = 2 ** 31 // V + 300
    x = torch.zeros((R, V), dtype=BF, device="cuda")
    rows = i32([R - 1, 0, R - 200, R - 1, R // 2])
    at = rows.long().unique()
    x[at] = (3 * torch.randn((len(at), V), generator=gen(1), device="cuda")).to(BF)
    tokens = i32([5, 7, V - 1, 100, 12345])
    r = binding.token_logprobs(x, tokens, rows=rows, top=3, entropy=True)
    few = x[rows.long()].clone()
    want = binding.token_logprobs(few, tokens, top=3, entropy=True)
    for name in ("logprobs", "entropy", "top_ids", "top_logprobs"):
        assert torch.equal(getattr(r, name), getattr(want, name)), name
    lp = torch.log_softmax(few.double(), -1)
    got = r.logprobs.double()
    ref = lp.gather(1, tokens.long()[:, None])[:, 0]
    b = P.logprob_bound(few, 1.0)(few.double().gather(1, tokens.long()[:, None])[:, 0])
    assert bool(((got - ref).abs() <= b).all())
    assert torch.equal(few.gather(1, r.top_ids.long()), few.topk(3).values)
