"""Speculative decoding with token trees, end to end on one GPU, over a toy target.

The target has one attention layer with random weights; the drafter is its output
projection applied to the last token's embedding.  Prompts go ahead, all in one pass:

  prompt_plan          positions and cache slots of their tokens, packed
  kv_write             normalises and rotates queries and keys, writes the cache
  prompt_attention     each token over those before it
  lmhead_logits, token_logprobs   how probable the prompts' tokens are

Every step:

  tree_plan            positions, cache slots and ancestor masks of the nodes
  kv_write             rotates queries and keys, writes the nodes' rows
  tree_attention       the nodes over the context and their ancestors
  lmhead_logits        the nodes' logits
  spec_verify_tree     which nodes are kept, and the token after them
  token_logprobs       the kept tokens' log probabilities
  kv_commit            the kept path's rows become part of the context

    python examples/tree_decode.py --requests 8 --nodes 16 --steps 20 --cache e4m3
"""
from __future__ import annotations

import argparse
import math
import os
import sys
from dataclasses import dataclass, field

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from speculative_decoding_verification_51_gb300 import binding  # noqa: E402

CACHE_TYPES = {"bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}


@dataclass
class Target:
    """One attention layer between an embedding and an output projection."""
    embed: torch.Tensor     # [V, H] bf16
    wq: torch.Tensor        # [H, q_heads * D]
    wk: torch.Tensor        # [H, kv_heads * D]
    wv: torch.Tensor
    wo: torch.Tensor        # [q_heads * D, H]
    lm_head: torch.Tensor   # [V, H]
    q_heads: int
    kv_heads: int
    head_dim: int
    norm: binding.HeadNorm | None = None   # of each head of queries and keys


def make_target(V=512, H=256, q_heads=8, kv_heads=2, head_dim=64, seed=0, device="cuda", head_norm=False) -> Target:
    g = torch.Generator(device="cpu").manual_seed(seed)

    def w(*shape, scale):
        return (torch.randn(shape, generator=g) * scale).to(device, torch.bfloat16)

    embed = w(V, H, scale=1.0)
    # the projection is near the embedding, so that the drafter (which does not
    # attend) is often right
    lm = (embed.float().roll(1, 0) * 0.3 + w(V, H, scale=0.2).float()).to(torch.bfloat16)
    return Target(embed, w(H, q_heads * head_dim, scale=H ** -0.5),
                  w(H, kv_heads * head_dim, scale=H ** -0.5),
                  w(H, kv_heads * head_dim, scale=H ** -0.5),
                  w(q_heads * head_dim, H, scale=(q_heads * head_dim) ** -0.5), lm.contiguous(),
                  q_heads, kv_heads, head_dim,
                  binding.HeadNorm(*(1.0 + w(head_dim, scale=0.2) for _ in range(2))) if head_norm else None)


@dataclass
class Batch:
    """The requests: their cache pages, lengths and tokens so far."""
    cache: binding.KVCache
    page_table: torch.Tensor             # [B, max_pages] int32
    context_len: torch.Tensor            # [B] int32
    last: torch.Tensor                   # [B] int32: the token emitted last (its row is not cached)
    tokens: list = field(default_factory=list)
    logprobs: list = field(default_factory=list)   # of every token after a request's first


def start(target: Target, first, max_tokens: int, page_size=16, cache="bf16") -> Batch:
    """Requests that begin with one token each."""
    B = len(first)
    dev = target.embed.device
    pages = -(-max_tokens // page_size)
    kv = binding.new_kv_cache(B * pages, page_size, target.kv_heads, target.head_dim,
                              dtype=CACHE_TYPES[cache], device=dev)
    # pages handed out in an order of their own, as an allocator would
    table = torch.randperm(B * pages, generator=torch.Generator().manual_seed(1)).to(torch.int32)
    return Batch(kv, table.view(B, pages).to(dev),
                 torch.zeros(B, dtype=torch.int32, device=dev),
                 torch.tensor(first, dtype=torch.int32, device=dev), [[int(t)] for t in first], [[] for _ in first])


def prefill(target: Target, batch: Batch, prompts: list, table: binding.RopeTable) -> None:
    """Requests that begin with whole prompts (of at least one token): all tokens but the last, which
    the first step takes, go into the cache in one pass."""
    dev, D = target.embed.device, target.head_dim
    lens = [len(p) - 1 for p in prompts]
    offsets = torch.tensor([0] + lens, dtype=torch.int32).cumsum(0, dtype=torch.int32).to(dev)
    flat = [t for p in prompts for t in p[:-1]]
    T = len(flat)
    batch.tokens = [list(p) for p in prompts]
    batch.last = torch.tensor([p[-1] for p in prompts], dtype=torch.int32, device=dev)
    if T == 0:
        return
    plan = binding.prompt_plan(offsets, T, target.q_heads, target.kv_heads, page_table=batch.page_table, cache=batch.cache)
    x = target.embed[torch.tensor(flat, device=dev)]                      # [T, H]
    q = (x @ target.wq).view(T, target.q_heads, D)
    k = (x @ target.wk).view(T, target.kv_heads, D)
    v = (x @ target.wv).view(T, target.kv_heads, D)
    q = binding.kv_write(batch.cache, k, v, plan.slots, positions=plan.positions, table=table, q=q, out_k=k,
                         norm=target.norm)
    out = binding.prompt_attention(q, k, v, plan)
    batch.context_len.copy_(offsets[1:] - offsets[:-1])
    hidden = (x + out.view(T, -1) @ target.wo).contiguous()
    logits = binding.lmhead_logits(hidden, target.lm_head)
    after = torch.tensor([t for p in prompts for t in p[1:]], dtype=torch.int32, device=dev)
    lp = binding.token_logprobs(logits, after).logprobs.cpu().tolist()
    at = 0
    for b, n in enumerate(lens):
        batch.logprobs[b] += lp[at:at + n]
        at += n


def draft(target: Target, last: torch.Tensor, parents: torch.Tensor, temperature: torch.Tensor,
          g: torch.Generator):
    """Tokens [B, N] of the trees (node 0 is the last token) and the
    distributions [B, N, V] that they were drawn from."""
    B, N = parents.shape
    V = target.lm_head.shape[0]
    tokens = torch.empty((B, N), dtype=torch.int32, device=last.device)
    probs = torch.zeros((B, N, V), dtype=torch.float32, device=last.device)
    tokens[:, 0] = last
    rows = torch.arange(B, device=last.device)
    soft = torch.where(temperature > 0, temperature, torch.ones_like(temperature))
    for c in range(1, N):
        up = tokens[rows, parents[:, c].long()].long()
        logits = target.embed[up].float() @ target.lm_head.float().T
        q = torch.softmax(logits / soft[:, None], -1)
        drawn = torch.multinomial(q, 1, generator=g)[:, 0]
        # greedy requests: the siblings in order of their probability
        older = (parents[:, 1:c] == parents[:, c:c + 1]).sum(1) if c > 1 else torch.zeros_like(last)
        best = torch.topk(q, min(N, V), -1).indices[rows, older.long()]
        tokens[:, c] = torch.where(temperature > 0, drawn, best).to(torch.int32)
        probs[:, c] = q
    return tokens, probs


def step(target: Target, batch: Batch, parents: torch.Tensor, num_nodes: torch.Tensor,
         temperature: torch.Tensor, table: binding.RopeTable, seed: int, g: torch.Generator):
    """One decoding step of all requests; returns the accepted counts [B]."""
    B, N = parents.shape
    tokens, probs = draft(target, batch.last, parents, temperature, g)
    plan = binding.tree_plan(parents, num_nodes, batch.context_len, batch.page_table, batch.cache)
    x = target.embed[tokens.long()]                                       # [B, N, H]
    D = target.head_dim
    q = (x @ target.wq).view(B, N, target.q_heads, D)
    k = (x @ target.wk).view(B, N, target.kv_heads, D)
    v = (x @ target.wv).view(B, N, target.kv_heads, D)
    q = binding.kv_write(batch.cache, k, v, plan.slots, positions=plan.positions, table=table, q=q, norm=target.norm)
    out = binding.tree_attention(q, batch.cache, plan)
    hidden = (x + out.view(B, N, -1) @ target.wo).contiguous()
    logits = binding.lmhead_logits(hidden.view(B * N, -1), target.lm_head).view(B, N, -1)
    ids, accepted, last_node = binding.spec_verify_tree(logits, probs, tokens, parents, num_nodes,
                                                        temperature, seed)
    binding.kv_commit([batch.cache], plan, last_node, new_context_len=batch.context_len)
    rows = torch.arange(B, device=ids.device)
    batch.last = ids[rows, accepted.long()].contiguous()
    # token i comes from the logits of the kept path's node of depth i (the root is of depth 0)
    depth = plan.positions - plan.positions[:, :1]
    kept_mask = plan.masks[rows, last_node.long().clamp(min=0)]
    on_path = (kept_mask[:, None] >> torch.arange(N, device=ids.device)) & 1
    node = torch.zeros((B, N), dtype=torch.int64, device=ids.device)
    node.scatter_(1, torch.where(on_path > 0, depth, N - 1).long(), torch.arange(N, device=ids.device).expand(B, N))
    node[rows, accepted.long()] = last_node.long()
    lp = binding.token_logprobs(logits, ids, rows=(rows[:, None] * N + node).to(torch.int32)).logprobs.cpu().tolist()
    host = ids.cpu().tolist()
    for b, a in enumerate(accepted.cpu().tolist()):
        batch.tokens[b] += host[b][:a + 1]
        batch.logprobs[b] += lp[b][:a + 1]
    return accepted


def tree_parents(B: int, N: int, width: int, device) -> torch.Tensor:
    """Nodes 1 .. width hang under the root, the others each under the node
    `width` before them."""
    p = [-1] + [max(0, c - width) for c in range(1, N)]
    return torch.tensor(p, dtype=torch.int32, device=device).expand(B, N).contiguous()


def reference_logits(target: Target, tokens: list, table_base=10000.0) -> torch.Tensor:
    """float32 logits after every token of one sequence, computed whole (no
    cache, no kernels of the library)."""
    dev = target.embed.device
    t = torch.tensor(tokens, device=dev)
    x = target.embed[t].float()
    D, n = target.head_dim, len(tokens)
    th = table_base ** (-2.0 * torch.arange(D // 2, dtype=torch.float64, device=dev) / D)
    ang = torch.arange(n, device=dev, dtype=torch.float64)[:, None, None] * th
    c, s = torch.cos(ang).float(), torch.sin(ang).float()

    def turn(y):
        a, b = y[..., :D // 2], y[..., D // 2:]
        return torch.cat((a * c - b * s, a * s + b * c), -1)

    def normed(y, w):
        return y if target.norm is None else y * torch.rsqrt(y.square().mean(-1, keepdim=True) + target.norm.eps) * w.float()

    wq, wk = (None, None) if target.norm is None else (target.norm.q_weight, target.norm.k_weight)
    q = turn(normed((x @ target.wq.float()).view(n, target.q_heads, D), wq))
    k = turn(normed((x @ target.wk.float()).view(n, target.kv_heads, D), wk))
    v = (x @ target.wv.float()).view(n, target.kv_heads, D)
    G = target.q_heads // target.kv_heads
    k, v = k.repeat_interleave(G, 1), v.repeat_interleave(G, 1)
    z = torch.einsum("nhd,mhd->hnm", q, k) / math.sqrt(D)
    z = z.masked_fill(torch.ones((n, n), dtype=torch.bool, device=dev).triu(1), -math.inf)
    o = torch.einsum("hnm,mhd->nhd", torch.softmax(z, -1), v).reshape(n, -1)
    return (x + o @ target.wo.float()) @ target.lm_head.float().T


def decode(requests=8, nodes=16, width=3, steps=20, temperature=0.0, cache="bf16", seed=0,
           target: Target | None = None, prompts: list | None = None, logprobs: list | None = None):
    """Decode and return (target, tokens of every request, accepted drafts a step).  prompts: what
    the requests begin with; logprobs: gets each request's list, one for each token after its first."""
    target = target or make_target()
    dev = target.embed.device
    room = steps * nodes + nodes
    if prompts is not None:
        requests, room = len(prompts), room + max(len(p) for p in prompts)
    batch = start(target, [(37 * b + 11) % target.embed.shape[0] for b in range(requests)], room, cache=cache)
    table = binding.rope_table(target.head_dim, device=dev)
    parents = tree_parents(requests, nodes, width, dev)
    num = torch.full((requests,), nodes, dtype=torch.int32, device=dev)
    temp = torch.full((requests,), float(temperature), device=dev)
    g = torch.Generator(device=dev).manual_seed(seed)
    if prompts is not None:
        prefill(target, batch, prompts, table)
    kept = 0.0
    for i in range(steps):
        kept += float(step(target, batch, parents, num, temp, table, seed * 1000 + i, g).float().mean())
    if logprobs is not None:
        logprobs += batch.logprobs
    return target, batch.tokens, kept / steps


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--requests", type=int, default=8)
    ap.add_argument("--nodes", type=int, default=16, help="nodes of a tree, the root included (<= 32)")
    ap.add_argument("--width", type=int, default=3)
    ap.add_argument("--steps", type=int, default=20)
    ap.add_argument("--temperature", type=float, default=0.0)
    ap.add_argument("--cache", choices=sorted(CACHE_TYPES), default="bf16")
    ap.add_argument("--prompt", type=int, default=0, help="tokens of each request's prompt (random ones)")
    ap.add_argument("--head-norm", action="store_true", help="a target that normalises the heads of queries and keys")
    a = ap.parse_args()
    target = make_target(head_norm=a.head_norm)
    prompts, lp = None, []
    if a.prompt:
        g = torch.Generator().manual_seed(5)
        prompts = torch.randint(0, target.embed.shape[0], (a.requests, a.prompt), generator=g).tolist()
    _, tokens, kept = decode(a.requests, a.nodes, a.width, a.steps, a.temperature, a.cache, target=target,
                             prompts=prompts, logprobs=lp)
    print(f"{a.steps} steps, {kept:.2f} drafts kept a step and request")
    for b, t in enumerate(tokens[:4]):
        print(f"request {b}: {len(t)} tokens, log probability {sum(lp[b]):.2f}: {t[:16]} ...")


if __name__ == "__main__":
    main()
