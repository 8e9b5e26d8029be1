"""One attention layer of a speculative decoding step on quantised weights.

Prompts of several requests are put into a paged cache in one step (causal
chunks); then each request verifies a drafted tree in one step; then, for
comparison, the tokens on one branch of each tree are decoded one at a time.
Every branch token's attention output has to agree with what the tree step gave
it.  Shapes are the Qwen3-0.6B projections (16 query heads, 8 key heads of 128),
weights and hidden states are random (no rotary embedding or norms: they act on
the projections' rows before the append and change nothing here).

    python examples/tree_decode.py [--cache s8]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

HIDDEN, HEADS, KV_HEADS, HEAD_DIM, PAGE = 1024, 16, 8, 128, 16


class Layer:
    """q/k/v/o projections (q4 tiles), the cache's pages and the step's plan."""

    def __init__(self, qmm, requests, max_len, cache_type, dev):
        self.qmm, self.dev = qmm, dev
        g = torch.Generator(device=dev).manual_seed(1)
        self.shape = {"q": (HEADS * HEAD_DIM, HIDDEN), "k": (KV_HEADS * HEAD_DIM, HIDDEN),
                      "v": (KV_HEADS * HEAD_DIM, HIDDEN), "o": (HIDDEN, HEADS * HEAD_DIM)}
        self.w = {n: qmm.pack_q4(torch.randn(s, generator=g, device=dev) * 0.05) for n, s in self.shape.items()}
        self.blocks = -(-max_len // PAGE)
        pages = requests * self.blocks
        dtype = torch.int8 if cache_type == "s8" else torch.bfloat16
        self.k, self.v = (torch.zeros((pages, PAGE, KV_HEADS, HEAD_DIM), dtype=dtype, device=dev) for _ in range(2))
        self.scales = {}
        if cache_type == "s8":
            self.scales = {n: torch.zeros((pages, KV_HEADS, PAGE), device=dev) for n in ("k_scale", "v_scale")}
        self.table = torch.zeros((requests, self.blocks), dtype=torch.int32, device=dev)
        self.ctx = torch.zeros(requests, dtype=torch.int32, device=dev)
        self.free = torch.arange(pages, dtype=torch.int32, device=dev)
        self.status = torch.zeros(1, dtype=torch.int32, device=dev)

    def step(self, hidden, new, parents=None, keep=True):
        """hidden bf16 [T][HIDDEN], new tokens per request.  Returns the attention
        output bf16 [T][HEADS][HEAD_DIM] and the projected rows [T][HIDDEN]."""
        q, T, dev = self.qmm, hidden.shape[0], self.dev
        new_lens = torch.tensor(new, dtype=torch.int32, device=dev)
        slots = torch.empty(T, dtype=torch.int64, device=dev)
        positions = torch.empty(T, dtype=torch.int32, device=dev)
        mask = None
        if parents is not None:
            mask = torch.empty((T, -(-max(new) // 32)), dtype=torch.int32, device=dev)
        cu, taken = q.kv_plan(self.ctx, new_lens, self.free, self.table, PAGE, slots, positions, parents=parents,
                              mask=mask, dev_status=self.status)
        rows = {n: q.q4_gemm(self.w[n], *self.shape[n], hidden, dev_status=self.status).view(T, -1, HEAD_DIM)
                for n in ("q", "k", "v")}
        q.kv_append(rows["k"], rows["v"], slots, self.k, self.v, dev_status=self.status, **self.scales)
        att = q.tree_attention(rows["q"], self.k, self.v, self.table, self.ctx, cu, max(new), mask=mask,
                               dev_status=self.status, **self.scales)
        out = q.q4_gemm(self.w["o"], *self.shape["o"], att.view(T, -1), dev_status=self.status)
        if keep:                                  # the step's tokens stay: pages and lengths advance
            self.free = self.free[int(taken):]
            self.ctx = self.ctx + new_lens
        return att, out


def main(cache_type="bf16"):
    import quantized_matmul_qmm_gb300.qmm as qmm
    dev = torch.device("cuda")
    prompts, nodes = [37, 200, 64], 13
    layer = Layer(qmm, len(prompts), 256, cache_type, dev)
    g = torch.Generator(device=dev).manual_seed(2)
    hidden = lambda n: torch.randn((n, HIDDEN), generator=g, device=dev).to(torch.bfloat16)
    layer.step(hidden(sum(prompts)), prompts)

    # each request drafts a binary tree; node i hangs below (i - 1) // 2
    tree = [-1] + [(i - 1) // 2 for i in range(1, nodes)]
    drafted = hidden(nodes * len(prompts))
    parents = torch.tensor(tree * len(prompts), dtype=torch.int32, device=dev)
    att, out = layer.step(drafted, [nodes] * len(prompts), parents, keep=False)

    branch = [0, 2, 5, 12]
    worst = 0.0
    for node in branch:
        rows = torch.tensor([r * nodes + node for r in range(len(prompts))], device=dev)
        one, _ = layer.step(drafted[rows], [1] * len(prompts))
        worst = max(worst, float((one.float() - att[rows].float()).abs().max() / att[rows].float().abs().max()))
    assert int(layer.status) == 0, qmm.status_string(int(layer.status))
    print(f"{cache_type} cache: tree step of {len(prompts)} x {nodes} nodes, output rows {tuple(out.shape)}; "
          f"branch decoded token by token differs by at most {worst:.2g} of the largest value")
    # both round their outputs to bf16 once and sum in different orders: two bf16 steps at most
    assert worst <= 2 ** -7, worst
    return worst


if __name__ == "__main__":
    from quantized_matmul_qmm_gb300 import build
    build.build()
    p = argparse.ArgumentParser()
    p.add_argument("--cache", choices=["bf16", "s8"], default="bf16")
    main(p.parse_args().cache)
