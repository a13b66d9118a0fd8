"""CPU run of the source of router and combine (nvfp4_moe.hip): their launches and
kernels compiled for the host (tests/cpu_wave), on buffers that end where their
mapping ends, and once more on ones that start where it starts. A read or write
outside ends the run with a segmentation fault; what it writes is the definition's.

The rows of T tokens are packed four to a wave where k < 16, E <= 256 and T > 16,
so the token counts stand around multiples of 4, of a workgroup's 16 tokens, and
of 64, up to which one workgroup does it all.
"""
import numpy as np
import pytest

import block_scaled_fp4_gemv_amd as g
import cpu_wave_util as cpu_wave
import fp4_reference as ref

torch = pytest.importorskip("torch")

DTYPES = {g.NVFP4_F16: torch.float16, g.NVFP4_BF16: torch.bfloat16, g.NVFP4_F32: torch.float32}


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    return cpu_wave.build(tmp_path_factory.mktemp("route"), "route")


def run(program, folder, logits, dtype, k, score, bias, n_group, topk_group, group_top, renormalize, scaling):
    """The router's outputs for logits [T][E], a tensor of the type `dtype`."""
    T, E = logits.shape
    head = np.array([0, dtype, T, E, k, score, n_group, topk_group, group_top, renormalize, bias is not None], np.int32)
    out, _ = cpu_wave.run(program, folder, [head, np.float32(scaling), logits.contiguous().view(torch.uint8).numpy()] +
                          ([] if bias is None else [bias]))
    words, S = out.view(np.int32), T * k
    ids, weights = words[:S].reshape(T, k), words[S:2 * S].view(np.float32).reshape(T, k)
    return ids, weights, words[2 * S:2 * S + E + 1], words[2 * S + E + 1:]


# (E, k, n_group, topk_group, group_top): every width of the kernels, groups of 1,
# 2, 4 .. lanes and others, the most picks
ROUTERS = [(64, 8, 1, 1, 1), (64, 6, 4, 2, 2), (128, 4, 8, 3, 1), (256, 8, 8, 4, 2), (256, 15, 1, 1, 1), (60, 4, 4, 2, 2),
           (160, 6, 8, 3, 1), (8, 2, 1, 1, 1), (100, 16, 1, 1, 1), (384, 8, 4, 2, 2), (1024, 64, 1, 1, 1)]
TOKENS = [1, 16, 17, 18, 19, 20, 63, 66, 131]


@pytest.mark.parametrize("E,k,n_group,topk_group,group_top", ROUTERS)
@pytest.mark.parametrize("T", TOKENS)
def test_router_stays_inside_its_buffers(program, tmp_path, T, E, k, n_group, topk_group, group_top):
    rng = np.random.default_rng([T, E, k])
    dtype = int(rng.integers(3))
    score, renormalize, biased = (int(v) for v in rng.integers(2, size=3))
    logits = torch.from_numpy(rng.standard_normal((T, E)) * 2).to(DTYPES[dtype])
    logits[T // 2, : E // 3] = float("-inf")
    bias = (rng.standard_normal(E) * 0.1).astype(np.float32) if biased else None
    ids, weights, offsets, order = run(program, tmp_path, logits, dtype, k, score, bias, n_group, topk_group, group_top,
                                       renormalize, 1.5)
    want, want_w = ref.route(logits.double().numpy(), bias, k, "sigmoid" if score else "softmax", n_group, topk_group,
                             group_top, bool(renormalize), 1.5)
    want_o, want_l = ref.lists(want, E)
    assert np.array_equal(ids, want) and np.array_equal(offsets, want_o) and np.array_equal(order[:want_l.size], want_l)
    # one rounding to float32 of a float64 value that is off by far less
    assert np.all(np.abs(weights - want_w) <= 2.0 ** -24 * (1 + 2.0 ** -10) * np.abs(want_w) + 2.0 ** -150)


@pytest.mark.parametrize("dtype", sorted(DTYPES))
@pytest.mark.parametrize("T", [17, 18, 19, 66, 67])
def test_last_wave_reads_no_token_past_the_end(program, tmp_path, T, dtype):
    """Lanes of the last wave without a token: the first token's picks are the last
    experts, so an address formed with a token past the end lies past the logits."""
    E, k = 256, 8
    logits = torch.arange(E, dtype=torch.float32).repeat(T, 1).div(64).to(DTYPES[dtype])
    for score in (0, 1):
        ids, _, _, _ = run(program, tmp_path, logits, dtype, k, score, None, 1, 1, 1, 1, 1.0)
        assert np.array_equal(ids, ref.route(logits.double().numpy(), None, k, "sigmoid" if score else "softmax")[0])


@pytest.mark.parametrize("dtype", sorted(DTYPES))
@pytest.mark.parametrize("T,k,M", [(1, 1, 1), (3, 2, 7), (5, 4, 130), (2, 9, 33), (7, 64, 8), (1, 8, 1001)])
def test_combine_stays_inside_its_buffers(program, tmp_path, T, k, M, dtype):
    rng = np.random.default_rng([T, k, M])
    y = torch.from_numpy(rng.standard_normal((T * k, M))).to(DTYPES[dtype])
    w = rng.uniform(-1, 1, (T, k)).astype(np.float32)
    ids = rng.integers(-1, 4, (T, k)).astype(np.int32)
    y[torch.from_numpy(ids.reshape(-1) < 0)] = float("nan")          # never read
    out, _ = cpu_wave.run(program, tmp_path, [np.array([1, dtype, T, k, M], np.int32), y.view(torch.uint8).numpy(), ids, w])
    terms = np.where(ids < 0, 0.0, w.astype(np.float64))[:, :, None] * np.nan_to_num(y.double().numpy()).reshape(T, k, M)
    got = torch.from_numpy(out).view(DTYPES[dtype]).double().numpy().reshape(T, M)
    want, size = terms.sum(1), np.abs(terms).sum(1)
    tol = k * 2.0 ** -24 * size + ref.HALF_STEP[DTYPES[dtype]] * (1 + 2.0 ** -10) * np.abs(want) + ref.LEAST[DTYPES[dtype]]
    assert (np.abs(got - want) <= tol).all()


@pytest.mark.parametrize("score", [0, 1], ids=["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,k", [(19, 64, 1), (19, 64, 2), (18, 128, 8), (17, 256, 8), (66, 256, 15), (5, 256, 6), (3, 512, 4), (2, 1024, 8)])
def test_equals_at_the_last_pick_hide_no_larger_one(program, tmp_path, T, E, k, score):
    """Expert of the last pick and the next share a logit: what stands behind them, as close
    in float32, may be larger."""
    rng = np.random.default_rng([T, E, k, score])
    for biased in (False, True):
        logits = ref.equals_at_the_last_pick(rng, T, E, k, score)
        bias = np.full(E, 0.03125, np.float32) if biased else None
        ids, _, offsets, order = run(program, tmp_path, logits, g.NVFP4_F32, k, score, bias, 1, 1, 1, 1, 1.0)
        want, _ = ref.route(logits.double().numpy(), bias, k, "sigmoid" if score else "softmax")
        assert np.array_equal(ids, want), np.argwhere(ids != want)[:4]
