"""A layer of routed NVFP4 experts, from the framework's operators.

    python examples/expert_layer.py [--tokens 64] [--hidden 2048] [--inner 1024] [--experts 32] [--top 4]

For every token: a router picks k of E experts; an expert is two products,
inner = W1 x (a gate and an up half, joined as silu(gate) * up) and y = W2 inner;
the token's k results are summed with the router's weights. Weights are quantised
once, activations on the way, each by its own global scale:

    nvfp4_moe_route     router scores -> ids, weights, the experts' lists
    nvfp4_global_scale, nvfp4_quantize   x -> NVFP4
    nvfp4_gemm_experts  W1: a token's row serves its k slots
    nvfp4_global_scale, nvfp4_quantize   the joined halves -> NVFP4
    nvfp4_gemm_experts  W2: a row per slot
    nvfp4_moe_combine   k slots -> the token

Nothing waits for the device, so the layer can be captured into a graph, as main()
does. It prints the error against the same layer in float32 on the dequantised
weights and the time per call, eager and replayed.
"""
import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import block_scaled_fp4_gemv_amd as g  # noqa: E402


def scale_bytes(rows, K, L=1):
    """Bytes of the 128x4 blocked scales of L batches."""
    return L * g.cdiv(rows, 128) * g.cdiv(K, 64) * 512


class Quantized:
    """NVFP4 rows [L][rows][K] on the device: codes, blocked scales, global scale."""

    def __init__(self, rows, K, L=1, device="cuda"):
        self.rows, self.K, self.L = rows, K, L
        self.codes = torch.empty(L * rows * K // 2, dtype=torch.uint8, device=device)
        self.scales = torch.empty(scale_bytes(rows, K, L), dtype=torch.uint8, device=device)
        self.scale = torch.empty(1, dtype=torch.float32, device=device)

    def take(self, x, workspace):
        g.nvfp4_global_scale(x, self.scale, self.rows, self.K, self.L, workspace)
        g.nvfp4_quantize(x, self.codes, self.scales, self.rows, self.K, self.L, "blocked", global_scale=self.scale)
        return self

    def values(self):
        out = torch.empty(self.L, self.rows, self.K, dtype=torch.float32, device=self.codes.device)
        g.nvfp4_dequantize(self.codes, self.scales, out, self.rows, self.K, self.L, "blocked", global_scale=self.scale)
        return out


class ExpertLayer:
    """w1 [E][2 * inner][hidden] (gate rows, then up rows), w2 [E][hidden][inner], for up to `tokens` tokens a call."""

    def __init__(self, w1, w2, top, tokens, score="softmax", **routing):
        E, F2, H = w1.shape
        S = tokens * top
        self.E, self.H, self.F, self.k, self.tokens = E, H, F2 // 2, top, tokens
        self.routing = dict(score=score, **routing)
        device = w1.device
        empty = lambda *s, dtype: torch.empty(*s, dtype=dtype, device=device)  # noqa: E731
        # one zero-filled workspace serves every call in turn: each leaves its counters
        # zero. Fewer tokens may need more of it, so it has the size that serves any
        self.workspace = torch.zeros(g.NVFP4_WORKSPACE_MAX_BYTES, dtype=torch.uint8, device=device)
        self.w1 = Quantized(F2, H, E, device).take(w1, self.workspace)
        self.w2 = Quantized(H, self.F, E, device).take(w2, self.workspace)
        # the products take a scale per expert; here all share the tensor's
        self.scale1, self.scale2 = self.w1.scale.repeat(E), self.w2.scale.repeat(E)
        self.weights, self.ids = empty(S, dtype=torch.float32), empty(S, dtype=torch.int32)
        self.offsets, self.order = empty(E + 1, dtype=torch.int32), empty(S, dtype=torch.int32)
        self.inner = torch.zeros(S, F2, dtype=w1.dtype, device=device)
        self.y = torch.zeros(S, H, dtype=w1.dtype, device=device)

    def __call__(self, x, logits, bias=None, out=None):
        T, S = x.shape[0], x.shape[0] * self.k
        assert T <= self.tokens and x.is_contiguous() and logits.is_contiguous()
        if out is None:
            out = torch.empty_like(x)
        ids, weights, order, ws = self.ids[:S], self.weights[:S], self.order[:S], self.workspace
        g.nvfp4_moe_route(logits, ids, weights, self.offsets, order, T, self.E, self.k, bias=bias, workspace=ws,
                          **self.routing)
        rows = Quantized(T, self.H, device=x.device).take(x, ws)
        # a slot without an expert (all logits masked) is in no list and not
        # written; zeroed, it stays out of the next global scale
        inner = self.inner[:S].zero_()
        g.nvfp4_gemm_experts(self.w1.codes, rows.codes, self.w1.scales, rows.scales, inner, 2 * self.F, self.H, self.E,
                             T, self.k, "blocked", self.offsets, order, scale_a=self.scale1, scale_b=rows.scale,
                             workspace=ws)
        joined = torch.nn.functional.silu(inner[:, :self.F]) * inner[:, self.F:]
        rows = Quantized(S, self.F, device=x.device).take(joined, ws)
        g.nvfp4_gemm_experts(self.w2.codes, rows.codes, self.w2.scales, rows.scales, self.y, self.H, self.F, self.E,
                             S, 1, "blocked", self.offsets, order, scale_a=self.scale2, scale_b=rows.scale,
                             workspace=ws)
        g.nvfp4_moe_combine(self.y, ids, weights, out, T, self.k, self.H)
        return out

    def plain(self, x, logits):
        """The same layer in float32 on the dequantised weights, activations as they are (softmax, no groups)."""
        w1, w2 = self.w1.values(), self.w2.values()
        weights, ids = torch.softmax(logits.float(), dim=1).topk(self.k, dim=1)
        weights = weights / weights.sum(dim=1, keepdim=True)
        out = torch.zeros(x.shape, dtype=torch.float32, device=x.device)
        for e in range(self.E):
            t, j = (ids == e).nonzero(as_tuple=True)
            h = x[t].float() @ w1[e].t().contiguous()
            y = (torch.nn.functional.silu(h[:, :self.F]) * h[:, self.F:]) @ w2[e].t().contiguous()
            out.index_add_(0, t, y * weights[t, j, None])
        return out


def us_per_call(f, n=50):
    for _ in range(5):
        f()
    torch.cuda.synchronize()
    start = time.perf_counter()
    for _ in range(n):
        f()
    torch.cuda.synchronize()
    return (time.perf_counter() - start) / n * 1e6


def main(argv=None):
    p = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    for name, default in (("tokens", 64), ("hidden", 2048), ("inner", 1024), ("experts", 32), ("top", 4)):
        p.add_argument("--" + name, type=int, default=default)
    a = p.parse_args(argv)
    torch.manual_seed(0)
    rand = lambda *s: torch.randn(*s, device="cuda")  # noqa: E731
    layer = ExpertLayer((rand(a.experts, 2 * a.inner, a.hidden) * a.hidden ** -0.5).bfloat16(),
                        (rand(a.experts, a.hidden, a.inner) * a.inner ** -0.5).bfloat16(), a.top, a.tokens)
    x, logits = rand(a.tokens, a.hidden).bfloat16(), rand(a.tokens, a.experts)
    out = layer(x, logits)
    want = layer.plain(x, logits)
    error = float((out.float() - want).norm() / want.norm())
    print(f"{a.tokens} tokens, {a.experts} experts of {a.hidden} x {a.inner}, {a.top} each: "
          f"relative error of the quantised activations {error:.3f}")
    eager = us_per_call(lambda: layer(x, logits, out=out))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer(x, logits, out=out)
    print(f"{eager:.1f} us eager, {us_per_call(graph.replay):.1f} us replayed")
    return error


if __name__ == "__main__":
    main()
