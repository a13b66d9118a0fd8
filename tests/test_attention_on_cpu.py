"""CPU run of the source of attention over the paged cache (nvfp4_attention.hip),
launches included, compiled for the host (tests/cpu_wave): buffers end, and once more
start, at a page that is not mapped; copies to LDS land at once, and once more as late as
the kernels' waits let them; LDS starts as NaN; results are the 64-bit form's within
its tolerance, for tables, offsets and lengths that lead nowhere too."""
import numpy as np
import pytest

import attention_reference as ref
import cpu_wave_util as cpu_wave
from cache_cases import poisoned

torch = pytest.importorskip("torch")

DTYPES = [torch.float16, torch.bfloat16, torch.float32]     # by nvfp4_dtype_t


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    return cpu_wave.build(tmp_path_factory.mktemp("attention"), "attention")


def run(program, folder, c, table, lengths, offsets, H, T, dt, max_q, max_length=None, window=0, causal=True, q=None, twice=()):
    rng = np.random.default_rng([H, T, dt])
    D, B = c.D, len(lengths)
    if q is None:
        q = torch.from_numpy(rng.standard_normal((T, H, D)) * 2).to(DTYPES[dt])
    max_length = max_length or table.shape[1] * c.page_size
    scale = np.float32(D ** -0.5)
    head = np.array([dt, T, H, B, max_q, max_length, table.shape[1], c.pages, c.page_size, c.heads, D, window, causal], np.int32)
    got, names = cpu_wave.run(program, folder, [head, np.array([scale, c.gk, c.gv], np.float32), c.kc, c.ks, c.vc, c.vs,
                                                q.view(torch.uint8).numpy(), np.array(offsets, np.int32), np.array(lengths, np.int32),
                                                table.astype(np.int32)])
    n = T * H * D * q.element_size()
    out = torch.from_numpy(got[:n].copy()).view(DTYPES[dt]).reshape(T, H, D)
    lse = torch.from_numpy(got[n:].copy()).view(torch.float32).reshape(T, H)
    want = ref.attention(c, q.double().numpy(), offsets, lengths, table, max_q, max_length, np.float64(scale), causal, window)
    for t in twice:
        want["written"][t] = False
    ref.check_attention(out, lse, want, DTYPES[dt])
    kept = ~want["written"]
    kept[list(twice)] = False
    assert (got[:n].reshape(T, -1)[kept] == 0xA5).all()
    return names


@pytest.mark.parametrize("dt", [0, 1, 2])
@pytest.mark.parametrize("D,H,heads,page_size", [(64, 2, 1, 16), (96, 4, 2, 32), (128, 3, 3, 16), (192, 5, 1, 64), (256, 2, 1, 16)])
def test_single_tokens(program, tmp_path, D, H, heads, page_size, dt):
    rng = np.random.default_rng(D)
    lengths = [0, 1, 16, 65, 150]
    c, table = poisoned(rng, lengths, page_size, heads, D, spare=1)
    run(program, tmp_path, c, table, lengths, list(range(6)), H, 6, dt, 1, window=40 if H % 2 else 0)


@pytest.mark.parametrize("dt", [1, 2])
def test_long_ones_are_split(program, tmp_path, dt):
    rng = np.random.default_rng(2)
    lengths = [700, 300]
    c, table = poisoned(rng, lengths, 32, 1, 64, spare=0)
    run(program, tmp_path, c, table, lengths, [0, 1, 3], 2, 3, dt, 2)


@pytest.mark.parametrize("dt", [0, 2])
@pytest.mark.parametrize("D,H,n", [(64, 2, 1), (128, 3, 2), (256, 4, 1), (96, 20, 1), (64, 10, 4), (192, 16, 3)])
def test_a_long_bound_on_short_lengths(program, tmp_path, D, H, n, dt):
    """A table for 5000 positions: eight waves a workgroup, more splits than there are tiles, rows
    joined by the last workgroup and by a kernel of its own."""
    rng = np.random.default_rng(7)
    lengths = [500, 40]
    c, table = poisoned(rng, lengths, 16, 1, D, spare=0, width=313)
    names = run(program, tmp_path, c, table, lengths, [0, n, 2 * n], H, 2 * n, dt, n)
    assert ("join" in names) == (min(H * n, 32) > 8) and "rows" in names


@pytest.mark.parametrize("dt", [0, 2])
@pytest.mark.parametrize("window", [0, 20])
@pytest.mark.parametrize("causal", [True, False])
def test_drafts(program, tmp_path, window, causal, dt):
    rng = np.random.default_rng(3)
    lengths, counts = [70, 3, 20, 9], [3, 5, 0, 1]
    c, table = poisoned(rng, lengths, 16, 2, 64, spare=0, width=6)
    run(program, tmp_path, c, table, lengths, np.cumsum([1] + counts), 8, 12, dt, 5, window=window, causal=causal)


@pytest.mark.parametrize("dt", [1, 2])
@pytest.mark.parametrize("D", [64, 96, 128, 192, 256])
def test_prompts(program, tmp_path, D, dt):
    rng = np.random.default_rng(4)
    lengths, counts = [140, 45, 30, 90], [70, 45, 1, 9]
    c, table = poisoned(rng, lengths, 16, 1, D, spare=0, width=10)
    run(program, tmp_path, c, table, lengths, np.cumsum([0] + counts), 3, 127, dt, 70)


def test_what_leads_nowhere(program, tmp_path):
    rng = np.random.default_rng(5)
    c, table = poisoned(rng, [100, 64, 64, 64], 16, 2, 64, spare=0)
    table[0, 2], table[0, 5], table[1, :] = -1, c.pages, 2 ** 31 - 1
    table[2, 1], table[3, 0] = -2 ** 31, c.pages + 5
    for offsets, lengths, max_q, twice in (([0, 1, 2, 3, 4], [100, 64, 64, 64], 1, ()), ([-4, 3, 3, 60, 99], [10 ** 9, -5, 64, 2 ** 31 - 1], 40, ()),
                                           ([2, 44, 1, 9, -7], [64, 64, 1, 0], 42, range(2, 9)), ([0, 1, 44, 44, 44], [100, 100, 3, 64], 2, ())):
        for window in (0, 30):
            run(program, tmp_path, c, table, lengths, offsets, 2, 44, 0, max_q, max_length=100, window=window, twice=twice)


@pytest.mark.parametrize("n", [1, 40])
def test_nan_scales_reach_only_who_sees_them(program, tmp_path, n):
    rng = np.random.default_rng(6)
    c, table = poisoned(rng, [100, 100], 16, 1, 64, spare=0)
    late = 99 - n // 2
    c.vs[table[0, late // 16], 0, late % 16, 1] = 0x7F
    c.ks[table[1, late // 16], 0, late % 16, 3] = 0xFF
    run(program, tmp_path, c, table, [100, 100], [0, n, 2 * n], 2, 2 * n, 0, n)


@pytest.mark.parametrize("n", [0, 1, 20, 63])
@pytest.mark.parametrize("D,dt", [(64, 0), (192, 2)])
def test_a_lone_sequence_below_its_bound(program, tmp_path, D, dt, n):
    """Room for 63 queries of 2 shared heads, for fewer of them: the many rows' kernel alone."""
    rng = np.random.default_rng(8)
    c, table = poisoned(rng, [300], 16, 1, D, spare=0)
    names = run(program, tmp_path, c, table, [300], [0, n], 2, 63, dt, 63, window=100 if n == 20 else 0)
    assert "tile" in names and "rows" not in names
