"""GPU: the example of attention over a cache (examples/attention_layer.py) runs, and its
tokens have the same bits from a graph and eagerly, in caches whose pages lie otherwise."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

_spec = importlib.util.spec_from_file_location(
    "attention_layer", os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "attention_layer.py"))
example = importlib.util.module_from_spec(_spec)
_spec.loader.exec_module(example)


@pytest.mark.parametrize("sequences,prompt,heads,kv_heads,size", [(1, 5, 4, 4, 64), (3, 130, 8, 2, 128), (2, 700, 7, 1, 96)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
def test_replayed_as_eager(sequences, prompt, heads, kv_heads, size, dtype):
    torch.manual_seed(prompt)
    replayed, eager, _ = example.run(sequences, prompt, 4, heads, kv_heads, size, dtype)
    assert torch.equal(replayed, eager) and bool(torch.isfinite(replayed).all()) and bool((replayed != 0).any())


def test_main_runs(capsys):
    example.main(["--sequences", "2", "--prompt", "100", "--tokens", "3", "--heads", "8", "--kv-heads", "2", "--size", "64"])
    assert "the same as eagerly" in capsys.readouterr().out
