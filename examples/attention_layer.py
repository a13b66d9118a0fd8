"""Attention of a layer over a paged NVFP4 cache, from the framework's operators.

    python examples/attention_layer.py [--sequences 16] [--prompt 1000] [--tokens 8] [--heads 32] [--kv-heads 8] [--size 128]

The q, k and v of new tokens lie in one packed projection [T][heads + 2 * kv_heads][size]:

    nvfp4_rope             the heads of q and k, in place
    nvfp4_cache_write      k and v into the slots of their tokens
    nvfp4_cache_attention  q over the pages of its sequence

Prompts come first, all tokens at once; then tokens one by one, replayed from a graph whose
positions, slots and lengths are device tensors that change between the replays.
"""
import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import block_scaled_fp4_gemv_amd as g  # noqa: E402


class AttentionLayer:
    """The cache of one layer with room for `length` tokens of each of `sequences`, whose pages
    are dealt out of one shuffled pool."""

    def __init__(self, sequences, length, heads, kv_heads, size, k_scale, v_scale, page_size=64, base=500000.0, device="cuda"):
        self.B, self.H, self.heads, self.D, self.page_size = sequences, heads, kv_heads, size, page_size
        self.width = g.cdiv(length, page_size)
        pages = sequences * self.width
        empty = lambda n: torch.zeros(pages, kv_heads, page_size, size // n, dtype=torch.uint8, device=device)  # noqa: E731
        scale = lambda x: torch.tensor([x], dtype=torch.float32, device=device)  # noqa: E731
        self.cache = g.Nvfp4Cache(empty(2), empty(16), empty(2), empty(16), pages, page_size, kv_heads, size,
                                  k_scale=scale(k_scale), v_scale=scale(v_scale))
        self.table = torch.randperm(pages, device=device).reshape(sequences, self.width).to(torch.int32)
        self.frequencies = torch.tensor(g.nvfp4_rope_frequencies(size, base), dtype=torch.float64, device=device)
        # one zero-filled workspace serves every call in turn
        self.workspace = torch.zeros(g.NVFP4_WORKSPACE_MAX_BYTES, dtype=torch.uint8, device=device)

    def slots(self, sequence, positions):
        """Slots of tokens at `positions` of their sequences (int64 [T] each)."""
        return self.table[sequence, positions // self.page_size].long() * self.page_size + positions % self.page_size

    def __call__(self, qkv, positions, slots, offsets, lengths, max_q, out=None):
        """qkv [T][heads + 2 * kv_heads][size] (turned in place) -> out [T][heads][size]."""
        T, H, heads, D = qkv.shape[0], self.H, self.heads, self.D
        row = qkv.stride(0)
        if out is None:
            out = torch.empty(T, H, D, dtype=qkv.dtype, device=qkv.device)
        q, k, v = qkv[:, :H], qkv[:, H:H + heads], qkv[:, H + heads:]
        g.nvfp4_rope(qkv, qkv, positions, self.frequencies, T, H + heads, D, D, token_stride=row, head_stride=D)
        g.nvfp4_cache_write(self.cache, k, v, slots, T, k_strides=(row, D), v_strides=(row, D))
        g.nvfp4_cache_attention(self.cache, q, out, offsets, lengths, self.table, T, H, self.B, max_q,
                                self.width * self.page_size, token_stride=row, head_stride=D, workspace=self.workspace)
        return out


def run(sequences, prompt, tokens, heads, kv_heads, size, dtype=torch.bfloat16):
    """Prompts of `prompt` tokens, then `tokens` single ones from a graph. Returns the outputs of the
    single tokens from the graph, those of the same tokens eagerly in a second cache, and us per replay."""
    B, columns = sequences, heads + 2 * kv_heads
    rand = lambda *s: torch.randn(*s, device="cuda").to(dtype)  # noqa: E731
    first, single = rand(B * prompt, columns, size), rand(tokens, B, columns, size)
    of = lambda *a: torch.arange(*a, device="cuda")  # noqa: E731
    results, us = [], 0.0
    for graphed in (True, False):
        # values of one normal distribution: a block's largest is about 2 of 6 * 448 steps at most
        layer = AttentionLayer(B, prompt + tokens, heads, kv_heads, size, 0.004, 0.004)
        whole = torch.full((B,), prompt, dtype=torch.int32, device="cuda")
        sequence, positions = of(B).repeat_interleave(prompt), of(prompt).repeat(B)
        layer(first.clone(), positions, layer.slots(sequence, positions), of(0, B * prompt + 1, prompt).to(torch.int32), whole, prompt)
        qkv, out = single[0].clone(), torch.empty(B, heads, size, dtype=dtype, device="cuda")
        offsets, positions, lengths = of(B + 1).to(torch.int32), torch.zeros(B, dtype=torch.int64, device="cuda"), torch.zeros_like(whole)
        slots = torch.full((B,), -1, dtype=torch.int64, device="cuda")     # of no token: nothing is written yet
        step = lambda: layer(qkv, positions, slots, offsets, lengths, 1, out)  # noqa: E731
        if graphed:
            side = torch.cuda.Stream()
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(side):
                step()
            torch.cuda.current_stream().wait_stream(side)
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                step()
            step = graph.replay
        outs = []
        for n in range(tokens):
            qkv.copy_(single[n])
            positions.fill_(prompt + n)
            slots.copy_(layer.slots(of(B), positions))
            lengths.fill_(prompt + n + 1)
            step()
            outs.append(out.clone())
        results.append(torch.stack(outs))
        if graphed:
            torch.cuda.synchronize()
            start = time.perf_counter()
            for _ in range(50):                                             # the last token again: its slots again
                step()
            torch.cuda.synchronize()
            us = (time.perf_counter() - start) / 50 * 1e6
    return results[0], results[1], us


def main(argv=None):
    p = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    for name, default in (("sequences", 16), ("prompt", 1000), ("tokens", 8), ("heads", 32), ("kv-heads", 8), ("size", 128)):
        p.add_argument("--" + name, type=int, default=default)
    a = p.parse_args(argv)
    torch.manual_seed(0)
    replayed, eager, us = run(a.sequences, a.prompt, a.tokens, a.heads, a.kv_heads, a.size)
    print(f"{a.sequences} sequences of {a.prompt} tokens, {a.heads} and {a.kv_heads} heads of {a.size}: {us:.0f} us a token replayed, "
          f"{'the same as' if torch.equal(replayed, eager) else 'other than'} eagerly")


if __name__ == "__main__":
    main()
