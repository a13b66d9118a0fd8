"""CPU run of the products' source (nvfp4_gemm.hip): every kernel that is built,
dense and routed, its launches included, compiled for the host (tests/cpu_wave).
Buffers end, and once more start, at a page that is not mapped, so an access
outside ends the run; copies to LDS land at once, and once more as late as the
kernels' waits let them, so a missing wait gives other results; LDS starts as NaN
codes; results are the 64-bit product's within float32 accumulation's bound.

The kernel is forced, so that each meets the edges: fewer rows than a fragment
and one more than a tile, K of one block pair, of less than a stage, of a stage
and a bit, K % 64 = 32, batches, slices.
"""
import ast
import os
import subprocess

import numpy as np
import pytest

import cpu_wave_util as cpu_wave
import fp4_reference as ref
import synth

torch = pytest.importorskip("torch")

DTYPES = [torch.float16, torch.bfloat16, torch.float32]     # by nvfp4_dtype_t
# kind -> rows of A, of B per tile; with (from, to) slices of K, and which uses
KINDS = {0: (256, 256), 1: (256, 128), 2: (128, 128), 3: (64, 64), 4: (128, 32), 5: (64, 32), 6: (32, 32), 7: (32, 32)}
SLICED = (3, 4, 5, 6, 7)
DENSE, ROUTED = (0, 2, 3, 4, 5, 6, 7), (1, 2, 3, 4, 5, 6)


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    return cpu_wave.build(tmp_path_factory.mktemp("products"), "products")


def operand(rng, L, rows, K):
    return synth.pack_nibbles(synth.e2m1_codes(rng, (L, rows, K), "uniform")), synth.scale_codes(rng, (L, rows, K // 16), "uniform")


def dense(program, folder, kind, splits, dt, M, N, K, L, layout):
    rng = np.random.default_rng([M, N, K, L])
    (a, sfa), (b, sfb) = operand(rng, L, M, K), operand(rng, L, N, K)
    lay = synth.to_blocked if layout else (lambda s: s)         # blocked padding: NaN codes
    ga, gb = np.float32([0.02]), np.float32([-0.3])
    head = np.array([0, kind, splits, dt, M, N, K, L, 1, layout], np.int32)
    got, names = cpu_wave.run(program, folder, [head, np.float32(1.5), np.ones(2, np.int32), a, b, lay(sfa), lay(sfb), ga, gb])
    assert len(names.splitlines()) == 2, names
    va, vb = ref.values(a, sfa), ref.values(b, sfb)
    f = 1.5 * np.float64(ga[0]) * np.float64(gb[0])
    want = np.stack([vb[i] @ va[i].T for i in range(L)]) * f
    size = np.stack([np.abs(vb[i]) @ np.abs(va[i]).T for i in range(L)]) * abs(f)
    ref.check_product(torch.from_numpy(got).view(DTYPES[dt]).reshape(L, N, M), want, size, K, DTYPES[dt])


# M, N against the tile (x: a multiple of it, + what is added), K, L
EDGES = [(0, 1, 0, 1, 32, 1), (0, 33, 0, 15, 64, 2), (1, 0, 1, 0, 128, 1), (1, 1, 1, 1, 160, 1), (0, 7, 0, 31, 416, 2), (1, -1, 1, -1, 352, 1),
         (0, 31, 0, 17, 736, 1), (1, 33, 0, 16, 1024, 1)]


@pytest.mark.parametrize("layout", [0, 1], ids=["plain", "blocked"])
@pytest.mark.parametrize("edge", range(len(EDGES)))
@pytest.mark.parametrize("kind", DENSE)
def test_dense(program, tmp_path, kind, edge, layout):
    xm, am, xn, an, K, L = EDGES[edge]
    bm, bn = KINDS[kind]
    dense(program, tmp_path, kind, 1, (edge + kind) % 3, xm * bm + am, xn * bn + an, K, L, layout)


@pytest.mark.parametrize("layout", [0, 1], ids=["plain", "blocked"])
@pytest.mark.parametrize("M,N,K,L,splits", [(33, 5, 288, 2, 3), (70, 40, 1056, 1, 4), (129, 33, 2048, 1, 16), (1, 1, 4128, 1, 7)])
@pytest.mark.parametrize("kind", SLICED)
def test_dense_in_slices(program, tmp_path, kind, M, N, K, L, splits, layout):
    dense(program, tmp_path, kind, splits, 2, M, N, K, L, layout)


def routed(program, folder, kind, splits, dt, M, K, E, rows, per, layout, lists, want_ids):
    """lists: offsets, order; want_ids [S]: the expert that each slot's result is, -1 for none."""
    S = rows * per
    rng = np.random.default_rng([M, K, S])
    (a, sfa), (b, sfb) = operand(rng, E, M, K), operand(rng, 1, rows, K)
    lay = synth.to_blocked if layout else (lambda s: s)
    ga, gb = rng.uniform(0.01, 0.1, E).astype(np.float32), np.float32([0.5])
    head = np.array([1, kind, splits, dt, M, S, K, E, per, layout], np.int32)
    got, _ = cpu_wave.run(program, folder, [head, np.float32(1.0), np.ones(2, np.int32), a, b, lay(sfa), lay(sfb),
                                            lists[0].astype(np.int32), lists[1].astype(np.int32), ga, gb])
    got = got.reshape(S, -1)
    vb = ref.values(b, sfb)[0]
    for e in range(E):
        slots = np.nonzero(want_ids == e)[0]
        if slots.size:
            va = ref.values(a[e], sfa[e])
            f = np.float64(ga[e]) * 0.5
            want, size = vb[slots // per] @ va.T * f, np.abs(vb[slots // per]) @ np.abs(va).T * f
            ref.check_product(torch.from_numpy(got[slots].copy()).view(DTYPES[dt]), want, size, K, DTYPES[dt], f"expert {e}")
    assert (got[want_ids < 0] == 0xA5).all(), "a slot of no list was written"


def some_lists(rng, E, S, drop):
    ids = rng.integers(0, E, S)
    ids[rng.random(S) < drop] = -1
    if E > 2:
        ids[ids == 1] = 0                                   # an empty list, and a long one
    offsets, order = ref.lists(ids.reshape(S, 1), E)
    return (offsets, np.concatenate([order, np.full(S - order.size, 1 << 30)])), ids


@pytest.mark.parametrize("layout", [0, 1], ids=["plain", "blocked"])
@pytest.mark.parametrize("E,rows,per,M,K,splits", [(1, 1, 1, 1, 32, 1), (5, 9, 4, 33, 96, 1), (3, 150, 2, 130, 160, 1), (70, 33, 3, 40, 352, 1),
                                                   (2, 40, 1, 257, 128, 1), (4, 3, 8, 65, 1056, 4), (2, 1, 5, 31, 2080, 9)])
@pytest.mark.parametrize("kind", ROUTED)
def test_routed(program, tmp_path, kind, E, rows, per, M, K, splits, layout):
    rng = np.random.default_rng([E, rows, per])
    lists, ids = some_lists(rng, E, rows * per, 0.1 if rows > 1 else 0.0)
    routed(program, tmp_path, kind, splits if kind in SLICED else 1, (kind + per) % 3, M, K, E, rows, per, layout, lists, ids)


@pytest.mark.parametrize("kind", ROUTED)
def test_lists_out_of_range(program, tmp_path, kind):
    """Offsets that fall, pass the slots' end or are negative; entries that are no slots."""
    rows, per, E, M, K = 9, 2, 4, 70, 224
    S = rows * per
    offsets = np.array([-5, 1, 5, 1 << 30, 4])
    order = np.array([-1, 3, 18, 17, 1 << 30] + [99] * (S - 5))
    ids = np.full(S, -1)
    ids[[3, 17]] = 1
    for splits in (1, 2) if kind in SLICED else (1,):
        routed(program, tmp_path, kind, splits, 2, M, K, E, rows, per, 0, (offsets, order), ids)
    none = (np.zeros(E + 1), np.full(S, -7))
    routed(program, tmp_path, kind, 1, 0, M, K, E, rows, per, 1, none, np.full(S, -1))


def shapes_in(name, *lists):
    """The named lists of shapes of a GPU test file, joined."""
    tree = ast.parse(open(os.path.join(cpu_wave.HERE, name)).read())
    found = {node.targets[0].id: node.value for node in tree.body
             if isinstance(node, ast.Assign) and isinstance(node.targets[0], ast.Name)}
    return [shape for name in lists for shape in ast.literal_eval(found[name])]


def test_gpu_tests_meet_every_kernel(program):
    """The shapes of the GPU tests of products, by the plans: each kernel that is built for a
    use is there with whole scale words and with halves, and in slices where it has any."""
    shapes = [(0, M, N, K, L) for M, N, K, L, *_ in shapes_in("test_gpu_fp4_gemm.py", "SHAPES", "TILES")]
    shapes += [(1, M, T * k, K, E) for T, E, k, M, K in shapes_in("test_gpu_fp4_moe.py", "EXPERTS", "TILES", "SLICED_TILES")]
    lines = "".join("%d %d %d %d %d\n" % s for s in shapes)
    done = subprocess.run([program], input=lines, capture_output=True, text=True, check=True).stdout.splitlines()
    built = [tuple(map(int, line.split()[1:])) for line in done if line.startswith("built")]
    plans = [tuple(map(int, line.split())) for line in done if not line.startswith("built")]
    assert sorted(k for k, _, _ in built) == sorted(KINDS) and len(plans) == len(shapes)
    met = {(experts, kind, K % 64 != 0, splits > 1) for (experts, _, _, K, _), (kind, splits) in zip(shapes, plans)}
    missing = []
    for kind, uses, most in built:
        for experts in (0, 1):
            if uses & (2 if experts else 1):
                here = [m[2:] for m in met if m[:2] == (experts, kind)]
                missing += [(experts, kind, odd) for odd in (False, True) if odd not in [o for o, _ in here]]
                missing += [(experts, kind, "slices")] if most > 1 and not any(s for _, s in here) else []
    assert not missing, missing
