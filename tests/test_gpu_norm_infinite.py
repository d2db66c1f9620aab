"""Heads with values that are not finite: each channel by its own value and the head's norm, alike for every alignment,
layout and type, where the pair's other channel turns it and where nothing does."""
import math

import pytest
import torch

import nodes_common as C
from gpu_common import ensure_built
from speculative_decoding_verification_51_gb300 import binding

pytestmark = pytest.mark.gpu
BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32
ROTS = [(None, "half"), (64, "half"), (64, "interleaved"), (32, "half"), (32, "interleaved"), (8, "interleaved")]


@pytest.fixture(scope="module", autouse=True)
def built():
    ensure_built()


def formula(x, w, pos, rot, layout, eps=1e-6):
    """In 64 bits, as it is written: infinities divided by an infinite norm are NaN, everything else 0."""
    x = x.double().cpu()
    y = x / torch.sqrt(x.square().mean(-1, keepdim=True) + eps)
    if w is not None:
        y = y * w.double().cpu()
    return y if rot is None else C.rotate(y, pos, C.thetas(rot)[0], layout, 1.0)


def heads(D, dt):
    """A head for every channel and value that is not finite, and one with two of them."""
    x = (1.0 + torch.arange(D, device="cuda") % 7).to(dt).repeat(3 * D + 1, 1)
    for i, v in enumerate((math.inf, -math.inf, math.nan)):
        x[i * D + torch.arange(D), torch.arange(D)] = v
    x[-1, 0], x[-1, D - 1] = math.inf, -math.inf
    return x[:, None]


@pytest.mark.parametrize("dt", [BF, HF, F32])
@pytest.mark.parametrize("rot,layout", ROTS)
def test_infinities_stay_in_their_channel_or_pair(rot, layout, dt):
    D = 64
    x = heads(D, dt)
    T = x.shape[0]
    pos = (torch.arange(T, dtype=torch.int32, device="cuda") * 3 + 1) if rot else None
    table = binding.rope_table(rot, layout=layout) if rot else None
    w = (0.5 + torch.arange(D, device="cuda") % 5).to(dt)
    odd = torch.empty((T, 1, D + 3), dtype=dt, device="cuda")[:, :, 1:D + 1].copy_(x)       # one value at a time
    for weight in (None, w):
        want = formula(x, weight, pos, rot, layout)
        norm = binding.HeadNorm(weight)
        for given in (x, odd):
            got = binding.rope(given, None, pos, table, norm=norm).double().cpu()
            assert torch.equal(got.isnan(), want.isnan())
            assert bool((got[~got.isnan()] == 0).all()) and bool((want[~want.isnan()] == 0).all())


@pytest.mark.parametrize("rot,layout", [(None, "half"), (16, "half"), (16, "interleaved")])
@pytest.mark.parametrize("kind", [BF, torch.float8_e4m3fn])
def test_on_the_way_into_the_cache(kind, rot, layout):
    D = 64
    x = heads(D, BF)
    T = x.shape[0]
    pos = (torch.arange(T, dtype=torch.int32, device="cuda") * 3 + 1) if rot else None
    table = binding.rope_table(rot, layout=layout) if rot else None
    cache = binding.new_kv_cache(-(-T // 16), 16, 1, D, dtype=kind)
    slots = torch.arange(T, device="cuda")
    out_k = torch.empty_like(x)
    binding.kv_write(cache, x, torch.ones_like(x), slots, positions=pos, table=table, out_k=out_k, norm=binding.HeadNorm())
    want = formula(x, None, pos, rot, layout)
    for got in (out_k.double().cpu(), binding.kv_read(cache, slots, dtype=F32)[0].double().cpu()):
        assert torch.equal(got.isnan(), want.isnan()) and bool((got[~got.isnan()] == 0).all())
