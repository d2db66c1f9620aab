"""Prompts that come in pieces: the keys ahead of a piece's queries are read back from the paged cache.  And the plan's order for
prompts of many keys."""
import math

import numpy as np
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


def context_slots(page_table, lens, page):
    """The cache slots of the first lens[b] tokens of each prompt, one behind the other."""
    at = [torch.arange(n, device="cuda") for n in lens]
    return torch.cat([page_table[b, i // page].long() * page + i % page for b, i in enumerate(at)])


@pytest.mark.parametrize("kind", [BF, torch.float8_e4m3fn])
@pytest.mark.parametrize("D,Hq,Hkv,window", [(64, 4, 2, 0), (128, 8, 2, 0), (128, 4, 4, 70), (256, 2, 1, 0)])
def test_pieces_through_the_cache(kind, D, Hq, Hkv, window):
    page, lens = 16, [300, 1, 77]
    pieces = [[128, 1, 0], [130, 0, 70], [0, 0, 1], [42, 0, 6]]
    g = torch.Generator(device="cuda").manual_seed(D)
    q, k, v = ([torch.randn((n, h, D), generator=g, device="cuda").to(BF) for n in lens] for h in (Hq, Hkv, Hkv))
    width = -(-max(lens) // page)
    page_table = torch.randperm(3 * width, generator=g, device="cuda").to(torch.int32).view(3, width)
    cache = binding.new_kv_cache(3 * width, page, Hkv, D, dtype=kind)
    table, norm = binding.rope_table(D), binding.HeadNorm(eps=1e-6)
    done, outs, turned = [0, 0, 0], [[] for _ in lens], [[] for _ in lens]
    for new in pieces:
        have = [a + n for a, n in zip(done, new)]
        off, koff = P.offsets(new), P.offsets(have)
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        plan = binding.prompt_plan(i32(off), off[-1], Hq, Hkv, k_offsets=i32(koff), num_keys=koff[-1], page_table=page_table,
                                   cache=cache, dev_status=status)
        assert torch.equal(plan.positions.cpu(), torch.cat([torch.arange(a, a + n, dtype=torch.int32) for a, n in zip(done, new)]))

        def part(x):
            return torch.cat([x[b][a:a + n] for b, (a, n) in enumerate(zip(done, new))])
        qt = binding.kv_write(cache, part(k), part(v), plan.slots, positions=plan.positions, table=table, q=part(q), norm=norm)
        kc, vc = binding.kv_read(cache, context_slots(page_table, have, page), dtype=BF)
        out = binding.prompt_attention(qt, kc, vc, plan, window=window, dev_status=status)
        want, _, bound, _ = P.attention(qt, kc, vc, off, koff, 1 / math.sqrt(D), window)
        assert int(status) == 0 and float(((out.double() - want).abs() - bound).max()) <= 0
        for b in range(3):
            outs[b].append(out[off[b]:off[b + 1]])
            turned[b].append(qt[off[b]:off[b + 1]])
        done = have
    assert done == lens
    # the same in one pass over what the cache holds in the end
    off = P.offsets(lens)
    kc, vc = binding.kv_read(cache, context_slots(page_table, lens, page), dtype=BF)
    qt = torch.cat([torch.cat(x) for x in turned])
    want, _, bound, _ = P.attention(qt, kc, vc, off, off, 1 / math.sqrt(D), window)
    got = torch.cat([torch.cat(x) for x in outs])
    assert float(((got.double() - want).abs() - bound).max()) <= 0


@pytest.mark.parametrize("Hq,Hkv", [(4, 1), (1, 1), (128, 1)])
@pytest.mark.parametrize("lens,ahead", [([5000, 30, 4096, 1, 700], [0] * 5), ([300, 2500, 0, 17], [9000, 40, 50000, 60000]),
                                        ([2047, 2048, 2049], [0] * 3), ([100, 3], [2 ** 29, -3])])
def test_the_longest_pieces_come_first(Hq, Hkv, lens, ahead):
    """In steps of the longest prompt's keys over 2048 (the plan alone: no key tensor is needed)."""
    off, koff = P.offsets(lens), P.offsets([n + a for n, a in zip(lens, ahead)])
    p = binding.prompt_plan(i32(off), off[-1], Hq, Hkv, k_offsets=i32(koff), num_keys=koff[-1])
    w = p.buffer.cpu().numpy().view(np.int32)
    items = w[64:64 + 8 * w[0]].reshape(-1, 8).astype(np.int64)
    each = 2 * (128 // (Hq // Hkv))
    assert int(w[0]) == sum(-(-n // each) for n in lens) and int(items[:, 1].sum()) == off[-1]
    unit = max(n + a for n, a in zip(lens, ahead)) // 2048 + 1
    rank = np.minimum(np.maximum(items[:, 3] + items[:, 1], 0) // unit, 2047)
    assert np.all(np.diff(rank) <= 0)
    if max(lens) > 2048:
        assert unit > 1 and rank[0] > rank[-1]
