"""GPU: the example layer of routed experts (examples/expert_layer.py): near the
float32 layer on the same weights, the same bits eager and replayed, and for fewer
tokens than it has room for."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

_spec = importlib.util.spec_from_file_location(
    "expert_layer", os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "expert_layer.py"))
example = importlib.util.module_from_spec(_spec)
_spec.loader.exec_module(example)


def build(tokens, hidden, inner, experts, top, seed, **kw):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rand = lambda *s: torch.randn(*s, device="cuda", generator=gen)  # noqa: E731
    layer = example.ExpertLayer((rand(experts, 2 * inner, hidden) * hidden ** -0.5).bfloat16(),
                                (rand(experts, hidden, inner) * inner ** -0.5).bfloat16(), top, tokens, **kw)
    return layer, rand


@pytest.mark.parametrize("tokens,hidden,inner,experts,top", [(1, 512, 256, 8, 2), (5, 288, 160, 4, 1), (150, 1024, 512, 16, 4)])
def test_near_the_float32_layer(tokens, hidden, inner, experts, top):
    """A value of a block of 16 normal ones moves by a step of 1/12 to 1/3 of the block's
    largest, uniformly, so by under a tenth of the values' rms; x and the joined
    halves are rounded so, and the first error passes through silu(g) * u, which
    doubles it at most: 0.1 + 2 * 0.1 bounds the whole, whose parts add as squares."""
    layer, rand = build(tokens, hidden, inner, experts, top, tokens)
    x, logits = rand(tokens, hidden).bfloat16(), rand(tokens, experts)
    out, want = layer(x, logits).float(), layer.plain(x, logits)
    assert (out - want).norm() <= 0.3 * want.norm()


def test_fewer_tokens_and_masked_ones():
    layer, rand = build(40, 512, 256, 8, 2, 3, score="sigmoid", n_group=4, topk_group=2, group_top=2)
    x, logits, bias = rand(40, 512).bfloat16(), rand(40, 8), rand(8) * 0.1
    logits[4] = float("-inf")
    layer(x, logits, bias)
    # one token at a time: other tiles, other global scales; a masked token gives zeros
    for t in (0, 4, 39):
        out = layer(x[t:t + 1], logits[t:t + 1], bias)
        assert torch.equal(out, layer(x[t:t + 1], logits[t:t + 1], bias))
        assert bool((out == 0).all()) == (t == 4)


def test_replays_equal_eager_calls():
    layer, rand = build(16, 512, 256, 8, 2, 4)
    x, logits = rand(16, 512).bfloat16(), rand(16, 8)
    out = layer(x, logits)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer(x, logits, out=out)
    for _ in range(3):
        x.copy_(rand(16, 512))
        logits.copy_(rand(16, 8))
        want = layer(x, logits).clone()
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
