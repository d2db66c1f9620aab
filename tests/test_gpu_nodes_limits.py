"""The operators around the verification at the ends of their ranges: page tables
near 2^31 tokens, as many heads as the calls take."""
import numpy as np
import pytest
import torch

import nodes_common as NC
from gpu_common import ensure_built
from speculative_decoding_verification_51_gb300 import binding
from test_gpu_nodes import BF, gen, randn

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    ensure_built()


def ints(x):
    return torch.from_numpy(np.asarray(x, np.int32)).cuda()


@pytest.mark.parametrize("page,pages", [(65504, 32784), (65536, 32767), (16, 134217719)])
def test_plan_of_the_longest_tables(page, pages):
    """Contexts that end in the last page of the longest table there may be: what a page
    outside the cache is found for, wherever it stands."""
    N, longest = 2, page * pages
    assert longest < 2 ** 31 - 128 and longest + page >= 2 ** 31 - 128
    cache = binding.new_kv_cache(1, page, 1, 8)
    table = torch.zeros((3, pages), dtype=torch.int32, device="cuda")
    table[1, 100] = 1
    table[2, pages - 1] = -1
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    p = binding.tree_plan(ints([[-1, 0]] * 3), ints([N] * 3), ints([longest - N] * 3), table, cache, dev_status=st)
    assert int(st) == binding.BADBIT["page"]
    assert p.slots.tolist() == [[page - 2, page - 1], [-1, -1], [-1, -1]]
    assert p.positions.tolist() == [[longest - 2, longest - 1], [0, 0], [0, 0]]
    assert p.masks.tolist() == [[1, 3], [0, 0], [0, 0]]


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("T,Hkv", [(1, 1000), (1, 65536), (3, 65536)])
def test_rotation_of_the_most_heads(T, Hkv, layout):
    """65536 query heads, 1000 key heads (a block takes one head then) or as many again, and
    one more than the calls take."""
    D, most = 8, 65536
    g, table = gen(T), binding.rope_table(D, layout=layout)
    th, _ = NC.thetas(D)
    pos = ints(np.arange(T) + 7)
    q, k = randn((T, most, D), BF, g), randn((T, Hkv, D), BF, g)
    for x, y in zip((q, k), binding.rope(q, k, pos, table)):
        d = (y.cpu().double() - NC.rotate(x, pos, th, layout)).abs()
        assert bool((d <= NC.rotate_bound(x, th, layout, BF) + 2e-6 * x.cpu().double().abs().amax()).all())
    with pytest.raises(binding.SpecVerifyError) as e:
        binding.rope(randn((T, most + 1, D), BF, g), None, pos, table)
    assert e.value.status == binding.SPEC_ERR_INVALID_ARG
