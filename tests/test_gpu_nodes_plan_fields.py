"""A plan whose fields were set to something else is refused by the calls that would
read it: other lengths, types and devices."""
import dataclasses

import pytest
import torch

from gpu_common import ensure_built
from speculative_decoding_verification_51_gb300 import binding

pytestmark = pytest.mark.gpu

I32, I64 = torch.int32, torch.int64
FIELDS = [
    ("slots", lambda x: x.to(I32)), ("slots", lambda x: x[:1]), ("slots", lambda x: x.cpu()), ("slots", lambda x: x.t()),
    ("masks", lambda x: x.to(I64)), ("masks", lambda x: x[:, :2].contiguous()), ("masks", lambda x: x.cpu()),
    ("context_len", lambda x: x.to(I64)), ("context_len", lambda x: x[:1]), ("context_len", lambda x: x.cpu()),
    ("page_table", lambda x: x.to(I64)), ("page_table", lambda x: x[:1]), ("page_table", lambda x: x.cpu()),
    ("page_table", lambda x: x.view(-1)), ("buffer", lambda x: x[:16]), ("buffer", lambda x: x.cpu()),
]


@pytest.mark.parametrize("field,change", FIELDS)
def test_changed_fields_are_refused(field, change):
    ensure_built()
    i = lambda x: torch.tensor(x, dtype=I32, device="cuda")  # noqa: E731
    cache = binding.new_kv_cache(4, 16, 2, 64)
    p = binding.tree_plan(i([[-1, 0, 0], [-1, 0, 1]]), i([3, 3]), i([5, 20]), i([[0, 1], [2, 3]]), cache)
    q = torch.randn(2, 3, 4, 64, device="cuda").to(torch.bfloat16)
    good = binding.tree_attention(q, cache, p)
    bad = dataclasses.replace(p, **{field: change(getattr(p, field))})
    if field in ("masks", "page_table", "buffer"):
        with pytest.raises(ValueError):
            binding.tree_attention(q, cache, bad)
    if field in ("masks", "slots", "context_len"):
        with pytest.raises(ValueError):
            binding.kv_commit([cache], bad, i([1, 2]))
    assert torch.equal(binding.tree_attention(q, cache, p), good)
    assert binding.kv_commit([cache], p, i([1, 2])).tolist() == [7, 23]
