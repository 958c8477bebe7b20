"""One sparse-attention layer serving a batch of requests: prompts go into the
caches, then every decode step plans its pages, norms, turns and stores the new
keys and values, selects positions with the indexer and attends to them.  The
decode step is captured once as a CUDA graph and replayed.

    python examples/sparse_decode.py [--requests 16] [--prompt 4000] [--steps 32]

Weights and inputs are random; there is no model behind them.  The first step is
compared with attention over the whole context: positions that the indexer does
not select are what may differ, so with prompts shorter than the selection the
two agree to rounding.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from sparse_attention_indexer_quant_gb300 import binding as idx  # noqa: E402

HIDDEN, HQ, HKV, D = 1024, 32, 8, 128      # the layer
IDX_HEADS, IDX_DIM, TOPK = 32, 128, 2048   # its indexer
PAGE = idx.PAGE_SIZE
EPS = 1e-6


class Layer:
    """Projections, norms and the two paged caches (main and indexer), which
    share their pages: one block table and one slot map serve both."""

    def __init__(self, requests: int, max_len: int, seed: int = 0):
        g = torch.Generator(device="cuda").manual_seed(seed)

        def weight(n):
            return (torch.randn(HIDDEN, n, device="cuda", generator=g) / HIDDEN ** 0.5).bfloat16()

        self.qkv = weight((HQ + 2 * HKV) * D)
        self.index_q, self.index_k = weight(IDX_HEADS * IDX_DIM), weight(IDX_DIM)
        self.index_w = weight(IDX_HEADS)
        self.q_norm, self.k_norm = (1 + 0.1 * torch.randn(D, device="cuda", generator=g)
                                    for _ in range(2))
        # the layer turns its whole heads, the indexer half of its own
        self.cos, self.sin = idx.rope_table(max_len, D, scaling="yarn", factor=4.0, orig_len=8192)
        self.index_cos, self.index_sin = idx.rope_table(max_len, IDX_DIM // 2)
        pages = -(-max_len // PAGE)
        self.num_blocks = requests * pages + 1
        self.k_cache, self.v_cache = idx.new_kv_cache(self.num_blocks, HKV, D)
        self.index_cache = idx.new_cache(self.num_blocks)
        self.block_table = torch.zeros(requests, pages, dtype=torch.int32, device="cuda")
        self.free_pages = torch.randperm(self.num_blocks, device="cuda", generator=g).int()
        self.pool_head = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.cached = torch.zeros(requests, dtype=torch.int32, device="cuda")
        self.errors = idx.new_errors()

    def store(self, x, new_lens, num_tokens):
        """Plans the step's pages and stores its tokens; returns (plan, queries)."""
        plan = idx.plan_step(self.cached, new_lens, self.block_table, self.free_pages,
                             self.pool_head, num_tokens, self.num_blocks, errors=self.errors)
        qkv = (x @ self.qkv).view(num_tokens, HQ + 2 * HKV, D)
        q = idx.qk_norm_rope_insert(qkv[:, :HQ], qkv[:, HQ:HQ + HKV], qkv[:, HQ + HKV:],
                                    self.q_norm, self.k_norm, EPS, plan.positions, self.cos,
                                    self.sin, D, plan.slot_mapping, self.k_cache, self.v_cache,
                                    errors=self.errors)
        idx.quant_insert(x @ self.index_k, plan.slot_mapping, self.index_cache, self.errors)
        self.cached.copy_(plan.context_lens)
        self.pool_head.copy_(plan.pool_head)
        return plan, q

    def decode(self, x, new_lens):
        """One token per request; returns (plan, queries, selected positions, output)."""
        B = x.shape[0]
        plan, q = self.store(x, new_lens, B)
        iq = (x @ self.index_q).view(B, IDX_HEADS, IDX_DIM)
        vals, scales = idx.rope_quant_q(iq, plan.positions, self.index_cos, self.index_sin,
                                        IDX_DIM // 2, errors=self.errors)
        top = idx.paged_logits_topk(vals, scales, (x @ self.index_w).float(), self.index_cache,
                                    self.block_table, plan.context_lens, 1, IDX_HEADS, TOPK,
                                    errors=self.errors)
        out = idx.paged_attention(q, self.k_cache, self.v_cache, self.block_table,
                                  plan.context_lens, 1, topk=top, errors=self.errors)
        return plan, q, top, out


@torch.no_grad()
def run(requests: int = 16, prompt: int = 4000, steps: int = 32, seed: int = 0) -> dict:
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    layer = Layer(requests, prompt + steps + 4, seed)
    # prompts of different lengths, the last one of the full length
    lens = torch.randint(1, prompt + 1, (requests,), device="cuda", generator=g).int()
    lens[-1] = prompt
    tokens = int(lens.sum())
    layer.store(torch.randn(tokens, HIDDEN, device="cuda", generator=g).bfloat16(), lens, tokens)

    x = torch.randn(requests, HIDDEN, device="cuda", generator=g).bfloat16()
    one = torch.ones(requests, dtype=torch.int32, device="cuda")
    plan, q, top, out = layer.decode(x, one)
    whole = idx.paged_attention(q, layer.k_cache, layer.v_cache, layer.block_table,
                                plan.context_lens, 1)
    covered = plan.context_lens <= TOPK  # the selection is the whole context there
    diff = (out.float() - whole.float()).abs().amax(dim=(1, 2))

    layer.decode(x, one)  # warm up outside the graph
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer.decode(x, one)
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    start.record()
    for _ in range(steps):
        graph.replay()
    end.record()
    torch.cuda.synchronize()
    return {"us_per_step": start.elapsed_time(end) / max(steps, 1) * 1e3,
            "covered": int(covered.sum()),
            "diff_covered": float(diff[covered].max()) if covered.any() else 0.0,
            "diff_selected": float(diff[~covered].max()) if (~covered).any() else 0.0,
            "cached": layer.cached.cpu(), "prompt_lens": lens.cpu(),
            "errors": layer.errors.cpu().tolist()}


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--requests", type=int, default=16)
    ap.add_argument("--prompt", type=int, default=4000)
    ap.add_argument("--steps", type=int, default=32)
    a = ap.parse_args()
    r = run(a.requests, a.prompt, a.steps)
    print(f"{r['us_per_step']:.1f} us a step; {r['covered']} of {a.requests} requests are selected "
          f"whole, off by {r['diff_covered']:.2g} from whole-context attention (others by "
          f"{r['diff_selected']:.2g}); errors {r['errors']}")
