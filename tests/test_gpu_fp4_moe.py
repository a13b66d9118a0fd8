"""GPU: router, experts' products and combine against the 64-bit definition.
Ids and lists have to be equal; weights within float32 steps; products within the
tolerance of float32 accumulation."""
import numpy as np
import pytest

import fp4_reference as ref
import synth

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import block_scaled_fp4_gemv_amd as g  # noqa: E402
from test_gpu_fp4_gemm import DTYPES, dev, operand  # noqa: E402


def run_route(logits, k, bias=None, **kw):
    T, E = logits.shape
    ids = torch.full((T, k), -7, dtype=torch.int32, device="cuda")
    weights = torch.full((T, k), 9.0, device="cuda")
    offsets = torch.full((E + 2,), -7, dtype=torch.int32, device="cuda")
    order = torch.full((T * k + 1,), -7, dtype=torch.int32, device="cuda")
    ws = torch.zeros(g.nvfp4_moe_route_workspace_bytes(T, E, k), dtype=torch.uint8, device="cuda")
    g.nvfp4_moe_route(logits.cuda(), ids, weights, offsets, order, T, E, k,
                      bias=None if bias is None else bias.cuda(), workspace=ws, **kw)
    torch.cuda.synchronize()
    assert offsets[-1] == -7 and order[-1] == -7, "write past the end"
    assert not ws.any(), "counters are not cleared"
    return ids.cpu().numpy(), weights.cpu().numpy(), offsets[:-1].cpu().numpy(), order[:-1].cpu().numpy()


def check_route(logits, k, bias=None, **kw):
    ids, weights, offsets, order = run_route(logits, k, bias, **kw)
    E = logits.shape[1]
    wi, ww = ref.route(logits.double().numpy(), None if bias is None else bias.double().numpy(), k, **kw)
    assert np.array_equal(ids, wi), np.argwhere(ids != wi)[:4]
    # one rounding to float32, and the 64-bit sums' own
    assert (np.abs(weights - ww) <= 2.0 ** -24 * (1 + 2.0 ** -20) * np.abs(ww) + 2.0 ** -150).all()
    wo, wl = ref.lists(wi, E)
    assert np.array_equal(offsets, wo)
    assert np.array_equal(order[:wo[-1]], wl) and (order[wo[-1]:] == -7).all()


ROUTES = [(1, 1, 1, {}), (1, 256, 8, dict(score="sigmoid", n_group=8, topk_group=4, group_top=2, scaling=2.5)),
          (5, 8, 2, {}), (63, 60, 4, dict(renormalize=False)), (130, 64, 6, dict(score="sigmoid", renormalize=False)),
          (300, 160, 6, dict(n_group=8, topk_group=3)), (77, 384, 8, dict(score="sigmoid")),
          (33, 1024, 64, dict(score="sigmoid", n_group=64, topk_group=5, group_top=1)), (400, 3, 3, {}),
          (1000, 128, 1, dict(n_group=4, topk_group=1, group_top=2))]


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("with_bias", [False, True])
@pytest.mark.parametrize("T,E,k,kw", ROUTES)
def test_route(T, E, k, kw, with_bias, dtype):
    gen = torch.Generator().manual_seed(T + E)
    logits = (torch.randn(T, E, generator=gen) * 2).to(dtype)
    bias = torch.randn(E, generator=gen) * 0.05 if with_bias else None
    check_route(logits, k, bias, score=kw.get("score", "softmax"), **{n: v for n, v in kw.items() if n != "score"})


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_ties_and_masks(score):
    """Few distinct logits (ties everywhere), masked, NaN and infinite ones, rows with nothing left."""
    rng = np.random.default_rng(2)
    x = rng.choice([-1.0, 0.0, 0.5, 2.0], (200, 96))
    x[rng.random(x.shape) < 0.4] = -np.inf
    x[rng.random(x.shape) < 0.05] = np.nan
    x[10:20] = -np.inf
    x[20:30] = np.nan
    x[30:40, 5:] = -np.inf
    x[40:44, 7] = np.inf
    x[44:48] = np.inf
    x[50] = np.finfo(np.float32).min
    x[51, 3:] = np.finfo(np.float32).min
    x[52], x[53] = 200.0, -200.0
    logits = torch.from_numpy(x).float()
    for kw in (dict(), dict(n_group=8, topk_group=2, group_top=2), dict(renormalize=False, n_group=4, topk_group=3)):
        check_route(logits, 8, None, score=score, **kw)
    bias = torch.zeros(96)
    bias[4], bias[9], bias[11] = float("nan"), float("-inf"), 3.0
    check_route(logits[:30], 8, bias, score=score)


# experts per lane and lanes per token; groups of 16 and 64 experts (and others), up to the largest k
FORMS = [(66, 64, 15, dict(n_group=4, topk_group=2, group_top=2)), (70, 128, 9, dict(n_group=8, topk_group=7)),
         (90, 256, 15, dict(n_group=16, topk_group=5, group_top=2)), (65, 256, 16, dict()), (90, 250, 4, dict()),
         (67, 256, 33, dict(n_group=4, topk_group=3, group_top=2)), (80, 512, 12, dict(n_group=8, topk_group=2)),
         (70, 1024, 20, dict(n_group=16, topk_group=9, group_top=2)), (70, 1024, 63, dict()), (70, 512, 64, dict()),
         (3, 16, 15, dict()), (9, 256, 8, dict(n_group=2, topk_group=1, group_top=2)), (129, 17, 16, dict()),
         (7, 256, 8, dict(n_group=8, topk_group=4, group_top=2)), (16, 128, 6, dict(n_group=8, topk_group=3)),
         (5, 160, 4, dict(n_group=5, topk_group=2, group_top=2)), (66, 256, 40, dict(n_group=16, topk_group=6, group_top=2)),
         (70, 512, 20, dict(n_group=16, topk_group=4, group_top=2)), (66, 1024, 30, dict(n_group=64, topk_group=9))]


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,k,kw", FORMS)
def test_route_forms(T, E, k, kw, score):
    gen = torch.Generator().manual_seed(T * E + k)
    logits = torch.randn(T, E, generator=gen) * 1.5
    logits[::5] = torch.where(torch.rand(logits[::5].shape, generator=gen) < 0.7, float("-inf"), logits[::5])
    check_route(logits, k, None, score=score, **kw)
    check_route(logits, k, torch.randn(E, generator=gen) * 0.2, score=score, **kw)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,kw", [(64, dict()), (256, dict(n_group=8, topk_group=4, group_top=2)), (512, dict()),
                                  (1024, dict(n_group=16, topk_group=4, group_top=2))])
def test_route_close_picks(E, kw, score):
    """Logits a few float32 steps apart, biases that bring unlike scores together or drown them: float32 cannot
    tell these picks."""
    rng = np.random.default_rng(E)
    T = 150
    x = rng.choice(np.array([0.5, 1.25, -0.75], np.float32), (T, E))
    x = x * (1 + rng.integers(-3, 4, (T, E)) * 2.0 ** -23)
    x[100:] = rng.standard_normal((50, E))
    logits = torch.from_numpy(x).float()
    near = torch.from_numpy(-1 / (1 + np.exp(-x[120]))).float()             # row 120: every sum near zero
    for bias in (None, near, torch.from_numpy(rng.standard_normal(E) * 1e5).float(), torch.full((E,), 3e4)):
        check_route(logits, 8, bias, score=score, **kw)


@pytest.mark.parametrize("T,E,k", [(16384, 256, 8), (9000, 1024, 2), (70000, 8, 2), (40000, 60, 4)])
def test_lists_of_many_slots(T, E, k):
    gen = torch.Generator().manual_seed(T)
    logits = torch.randn(T, E, generator=gen) + torch.randn(E, generator=gen) * 2
    logits[::7] = float("-inf")
    ids, _, offsets, order = run_route(logits, k, score="softmax")
    top = torch.sort(logits.double(), dim=1, descending=True, stable=True).indices[:, :k].numpy().astype(np.int32)
    top[::7] = -1
    assert np.array_equal(ids, top)
    wo, wl = ref.lists(ids, E)
    assert np.array_equal(offsets, wo) and np.array_equal(order[:wo[-1]], wl)


def routed(rng, T, E, k, drop=0.0):
    """Distinct experts per token, some popular and some without a token."""
    liked = rng.standard_normal(E) * 1.5
    liked[rng.random(E) < 0.2] = -50.0
    ids = np.argsort(-(rng.gumbel(size=(T, E)) + liked), axis=1)[:, :k].astype(np.int32)
    ids[rng.random(ids.shape) < drop] = -1
    return ids


def run_experts(a, sfa, b, sfb, ids, per, dtype, layout, alpha=1.0, ga=None, gb=None, offsets=None, order=None):
    E, M, K = a.shape[0], a.shape[1], a.shape[2] * 2
    rows, S = b.shape[1], b.shape[1] * per
    if offsets is None:
        offsets, order = ref.lists(ids, E)
        order = np.concatenate([order, np.full(S - order.size, 1 << 30, np.int32)])
    c = torch.full((S + 1, M), -3.0, dtype=dtype, device="cuda")
    ws = torch.zeros(g.nvfp4_gemm_experts_workspace_bytes(M, K, E, S), dtype=torch.uint8, device="cuda")
    lay = lambda s: dev(synth.to_blocked(s) if layout == "blocked" else s)  # noqa: E731
    g.nvfp4_gemm_experts(dev(a), dev(b), lay(sfa), lay(sfb), c, M, K, E, rows, per, layout, dev(offsets), dev(order), alpha,
                         scale_a=None if ga is None else dev(ga), scale_b=None if gb is None else dev(gb),
                         workspace=ws if ws.numel() else None)
    torch.cuda.synchronize()
    assert (c[S] == -3).all(), "write past the end of c"
    assert not ws[:65536].any(), "tickets are not cleared"
    return c[:S]


def check_experts(got, a, sfa, b, sfb, ids, per, dtype, f=None):
    E, K = a.shape[0], a.shape[2] * 2
    flat = ids.reshape(-1)
    vb = dev(ref.values(b, sfb)[0])
    for e in range(E):
        slots = np.nonzero(flat == e)[0]
        if not slots.size:
            continue
        va = dev(ref.values(a[e], sfa[e]))
        rb = vb[dev(slots // per)]
        scale = 1.0 if f is None else f[e]
        want = (rb @ va.t().contiguous()).cpu().numpy() * scale
        size = (rb.abs() @ va.abs().t().contiguous()).cpu().numpy() * abs(scale)
        ref.check_product(got[dev(slots)], want, size, K, dtype, f"expert {e}")
    out = torch.from_numpy((flat < 0) | (flat >= E)).cuda()
    assert (got[out] == -3).all(), "a slot of no list was written"


# every tile shape (mean list up to 32, 64, longer), lists shorter and longer than
# a tile, empty lists, one token, ragged K, K % 64 = 32, M around the tiles' edges
EXPERTS = [(1, 8, 1, 7, 96), (1, 64, 8, 300, 2048), (3, 16, 4, 129, 1056), (40, 64, 4, 100, 544), (200, 8, 2, 257, 160),
           (150, 4, 1, 130, 4128), (300, 8, 4, 128, 224), (700, 3, 2, 260, 288), (5, 1000, 4, 33, 64), (64, 1, 1, 64, 32)]


@pytest.mark.parametrize("per_token", [True, False])
@pytest.mark.parametrize("T,E,k,M,K", EXPERTS)
def test_experts(T, E, k, M, K, per_token):
    rng = np.random.default_rng([T, E, M])
    per = k if per_token else 1
    (a, sfa), (b, sfb) = operand(rng, E, M, K), operand(rng, 1, T if per_token else T * k, K)
    ids = routed(rng, T, E, k, drop=0.1 if T > 1 else 0.0)
    for dtype in DTYPES:
        got = {lay: run_experts(a, sfa, b, sfb, ids, per, dtype, lay) for lay in ("plain", "blocked")}
        check_experts(got["blocked"], a, sfa, b, sfb, ids, per, dtype)
        assert torch.equal(got["plain"], got["blocked"])


# longer lists and rows: every tile, slices of K
TILES = [(1606, 64, 4, 897, 1408), (1606, 64, 4, 897, 1440), (4000, 4, 4, 130, 96), (1220, 1, 1, 2346, 256),
         (4000, 4, 4, 33, 96), (619, 16, 8, 133, 256), (1103, 1, 1, 618, 22976), (20, 64, 4, 513, 96),
         (980, 1, 1, 851, 256), (144, 64, 2, 39, 8992), (64, 64, 1, 260, 96), (64, 64, 1, 300, 320), (9, 64, 8, 33, 3008)]


@pytest.mark.parametrize("T,E,k,M,K", TILES)
def test_experts_every_tile(T, E, k, M, K):
    rng = np.random.default_rng([T, E, M])
    (a, sfa), (b, sfb) = operand(rng, E, M, K), operand(rng, 1, T, K)
    ids = routed(rng, T, E, k, drop=0.02)
    for dtype in DTYPES:
        got = {lay: run_experts(a, sfa, b, sfb, ids, k, dtype, lay) for lay in ("plain", "blocked")}
        check_experts(got["blocked"], a, sfa, b, sfb, ids, k, dtype)
        assert torch.equal(got["plain"], got["blocked"])


def test_experts_scales():
    rng = np.random.default_rng(8)
    T, E, k, M, K = 50, 6, 2, 140, 1024
    (a, sfa), (b, sfb) = operand(rng, E, M, K, "edge"), operand(rng, 1, T, K, "edge")
    ids = routed(rng, T, E, k)
    ga, gb = rng.uniform(1e-4, 2e-3, E).astype(np.float32), np.array([0.01], np.float32)
    for dtype in DTYPES:
        got = run_experts(a, sfa, b, sfb, ids, k, dtype, "blocked", -0.5, ga, gb)
        check_experts(got, a, sfa, b, sfb, ids, k, dtype, -0.5 * ga.astype(np.float64) * np.float64(gb[0]))


def test_experts_empty_and_bad_lists():
    """No slot in any list; entries and offsets out of range are passed over."""
    rng = np.random.default_rng(9)
    T, E, k, M, K = 9, 4, 2, 70, 256
    (a, sfa), (b, sfb) = operand(rng, E, M, K), operand(rng, 1, T, K)
    none = np.full((T, k), -1, np.int32)
    assert (run_experts(a, sfa, b, sfb, none, k, torch.float32, "plain") == -3).all()
    # in range: list 1 holds slots 3 and 17; the rest is -1, past the slots, or an offset past the end
    offsets = np.array([0, 1, 5, 1 << 30, 4], np.int32)
    order = np.array([-1, 3, 18, 17, 1 << 30] + [99] * (T * k - 5), np.int32)
    ids = np.full((T, k), -1, np.int32)
    ids.reshape(-1)[[3, 17]] = 1
    got = run_experts(a, sfa, b, sfb, ids, k, torch.float32, "plain", offsets=offsets, order=order)
    check_experts(got, a, sfa, b, sfb, ids, k, torch.float32)


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("T,k,M", [(1, 1, 1), (1, 8, 7168), (3, 2, 7), (65, 4, 1001), (500, 8, 130), (9, 64, 33), (2000, 3, 257)])
def test_combine(T, k, M, dtype):
    rng = np.random.default_rng([T, k, M])
    y = torch.from_numpy(rng.standard_normal((T * k, M))).to(dtype)
    w = torch.from_numpy(rng.uniform(-1, 1, (T, k))).float()
    ids = rng.integers(0, 9, (T, k)).astype(np.int32)
    ids[rng.random(ids.shape) < 0.2] = -1
    ids[T // 2] = -1
    y[torch.from_numpy(ids.reshape(-1) < 0)] = float("nan")          # never read
    out = torch.full((T * M + 64,), 5.0, dtype=dtype, device="cuda")
    g.nvfp4_moe_combine(y.cuda(), dev(ids), w.cuda(), out[:T * M], T, k, M)
    torch.cuda.synchronize()
    assert (out[T * M:] == 5).all()
    use = np.where(ids < 0, 0.0, w.double().numpy())[:, :, None]
    terms = use * np.nan_to_num(y.double().numpy()).reshape(T, k, M)
    want, size = terms.sum(1), np.abs(terms).sum(1)
    got = out[:T * M].double().cpu().numpy().reshape(T, M)
    tol = k * 2.0 ** -24 * size + ref.HALF_STEP[dtype] * (1 + 2.0 ** -10) * np.abs(want) + ref.LEAST[dtype]
    assert (np.abs(got - want) <= tol).all()


def test_far_logits():
    """Logits past 2^32 bytes, and as many tokens: every token's expert and every list."""
    T, E = (1 << 21) + 5, 1024
    want = (torch.arange(T, device="cuda") * 7 % E).int()
    logits = torch.zeros(T, E, device="cuda")
    logits.scatter_(1, want[:, None].long(), 1.0)
    z = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")  # noqa: E731
    ids, offsets, order, weights = z(T), z(E + 1), z(T), torch.zeros(T, device="cuda")
    ws = torch.zeros(g.nvfp4_moe_route_workspace_bytes(T, E, 1), dtype=torch.uint8, device="cuda")
    g.nvfp4_moe_route(logits, ids, weights, offsets, order, T, E, 1, workspace=ws)
    assert torch.equal(ids, want) and (weights == 1).all()
    assert torch.equal(order, torch.argsort(want, stable=True).int())
    assert torch.equal(offsets[1:], torch.bincount(want, minlength=E).cumsum(0).int()) and offsets[0] == 0


def test_far_experts():
    """Weights and results past 2^32 bytes: the last expert's rows and the last slot are their own."""
    E, M, K, T = 3, 1 << 18, 16384, 2
    codes = torch.zeros(E, M, K // 2, dtype=torch.uint8, device="cuda")
    sfa = torch.zeros(E * M * (K // 16), dtype=torch.uint8, device="cuda")
    rng = np.random.default_rng(2)
    (a, sa), (b, sfb) = operand(rng, 1, 64, K), operand(rng, 1, T, K)
    codes[E - 1, M - 64:] = dev(a[0])
    sfa[-64 * (K // 16):] = dev(sa.reshape(-1))
    per = 2100                                                              # 4200 slots of 2^18 float32: 4.4 GB
    S = T * per
    offsets = dev(np.array([0, 1, 1, 3], np.int32))
    order = dev(np.array([5, 17, S - 1] + [S] * (S - 3), np.int32))
    c = torch.full((S, M), 7.0, device="cuda")
    ws = torch.zeros(g.nvfp4_gemm_experts_workspace_bytes(M, K, E, S), dtype=torch.uint8, device="cuda")
    g.nvfp4_gemm_experts(codes, dev(b), sfa, dev(sfb), c, M, K, E, T, per, "plain", offsets, order,
                         workspace=ws if ws.numel() else None)
    va, vb = dev(ref.values(a[0], sa[0])), dev(ref.values(b[0], sfb[0]))
    want, size = (vb @ va.t().contiguous()).cpu().numpy(), (vb.abs() @ va.abs().t().contiguous()).cpu().numpy()
    ref.check_product(c[[17, S - 1], M - 64:], want, size, K, torch.float32, "last expert")
    assert not c[[17, S - 1], :M - 64].any() and not c[5].any()
    assert (c[6:17] == 7).all() and (c[S - 2] == 7).all()


def test_far_slots():
    """Rows to combine past 2^32 elements: the last token gets its own."""
    T, k, M = 70000, 8, 8192
    y = torch.zeros(T * k, M, dtype=torch.float16, device="cuda")
    y[-k:] = torch.randn(k, M, device="cuda")
    ids = torch.zeros(T, k, dtype=torch.int32, device="cuda")
    weights = torch.rand(T, k, device="cuda")
    out = torch.full((T, M), 7.0, dtype=torch.float16, device="cuda")
    g.nvfp4_moe_combine(y, ids, weights, out, T, k, M)
    terms = y[-k:].double() * weights[-1, :, None].double()
    tol = terms.abs().sum(0) * (k + 1) * 2.0 ** -24 + terms.sum(0).abs() * 2.0 ** -11 + 2.0 ** -25
    assert ((out[-1].double() - terms.sum(0)).abs() <= tol).all() and not out[:-1].any()


def test_router_after_a_split_product_in_one_workspace():
    """The partial sums that a product leaves in the workspace do not reach the lists."""
    T, E, k, M, K = 300, 1024, 4, 128, 16384
    assert g.nvfp4_gemm_plan(M, 16, K, 1)["k_splits"] > 1
    rng = np.random.default_rng(5)
    (a, sfa), (b, sfb) = operand(rng, 1, M, K), operand(rng, 1, 16, K)
    ws = torch.zeros(max(g.nvfp4_gemm_workspace_bytes(M, 16, K, 1), g.nvfp4_moe_route_workspace_bytes(T, E, k)),
                     dtype=torch.uint8, device="cuda")
    c = torch.empty(16 * M, device="cuda")
    logits = torch.randn(T, E, device="cuda")
    z = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")  # noqa: E731
    ids, offsets, order, weights = z(T, k), z(E + 1), z(T * k), torch.zeros(T, k, device="cuda")
    for _ in range(2):
        g.nvfp4_gemm(dev(a), dev(b), dev(sfa), dev(sfb), c, M, 16, K, 1, "plain", workspace=ws)
        assert ws[65536:].any() and not ws[:65536].any()
        g.nvfp4_moe_route(logits, ids, weights, offsets, order, T, E, k, workspace=ws)
        wo, wl = ref.lists(ids.cpu().numpy(), E)
        assert np.array_equal(offsets.cpu().numpy(), wo) and np.array_equal(order.cpu().numpy(), wl)


def test_layer_in_a_graph():
    """Route, quantise, both products and the combine captured together; replays
    with other inputs agree with the eager chain bit for bit."""
    T, E, k, H, F = 37, 16, 4, 512, 256
    rng = np.random.default_rng(12)
    (a1, s1), (a2, s2) = operand(rng, E, F, H), operand(rng, E, H, F)
    w1, w2, f1, f2 = dev(a1), dev(a2), dev(synth.to_blocked(s1)), dev(synth.to_blocked(s2))
    x, logits = torch.randn(T, H, device="cuda"), torch.randn(T, E, device="cuda")
    z = lambda *s, dtype=torch.float32: torch.zeros(*s, dtype=dtype, device="cuda")  # noqa: E731
    u8, i32, S = torch.uint8, torch.int32, T * k
    ids, weights, offsets, order = z(T, k, dtype=i32), z(T, k), z(E + 1, dtype=i32), z(S, dtype=i32)
    ws = z(max(g.nvfp4_moe_route_workspace_bytes(T, E, k), g.nvfp4_gemm_experts_workspace_bytes(F, H, E, S),
               g.nvfp4_gemm_experts_workspace_bytes(H, F, E, S), 256), dtype=u8)
    g1, g2 = z(1), z(1)
    q1, p1 = z(T * H // 2, dtype=u8), z(ref.cdiv(T, 128) * ref.cdiv(H, 64) * 512, dtype=u8)
    q2, p2 = z(S * F // 2, dtype=u8), z(ref.cdiv(S, 128) * ref.cdiv(F, 64) * 512, dtype=u8)
    h, y, out = z(S, F, dtype=torch.bfloat16), z(S, H, dtype=torch.bfloat16), z(T, H, dtype=torch.bfloat16)

    def layer():
        g.nvfp4_moe_route(logits, ids, weights, offsets, order, T, E, k, workspace=ws)
        g.nvfp4_global_scale(x, g1, T, H, 1, ws)
        g.nvfp4_quantize(x, q1, p1, T, H, 1, "blocked", global_scale=g1)
        g.nvfp4_gemm_experts(w1, q1, f1, p1, h, F, H, E, T, k, "blocked", offsets, order, scale_b=g1, workspace=ws)
        g.nvfp4_global_scale(h, g2, S, F, 1, ws)
        g.nvfp4_quantize(h, q2, p2, S, F, 1, "blocked", global_scale=g2)
        g.nvfp4_gemm_experts(w2, q2, f2, p2, y, H, F, E, S, 1, "blocked", offsets, order, scale_b=g2, workspace=ws)
        g.nvfp4_moe_combine(y, ids, weights, out, T, k, H)

    layer()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer()
    for _ in range(3):
        x.copy_(torch.randn_like(x))
        logits.copy_(torch.randn_like(logits))
        layer()
        torch.cuda.synchronize()
        want = out.clone()
        assert want.abs().max() > 0
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)


def test_experts_scales_far_from_one():
    """Each expert's scale times the rows' leaves float32's range where the scaled sums do not."""
    rng = np.random.default_rng(18)
    T, E, k, M, K = 50, 6, 2, 140, 1024
    (a, sfa), (b, sfb) = operand(rng, E, M, K, "edge"), operand(rng, 1, T, K, "edge")
    ids = routed(rng, T, E, k)
    for alpha, ga, gb in ((1.0, 2.0 ** -75, 2.0 ** -75), (1.0, 2.0 ** -70, 2.0 ** -70), (2.0 ** 60, 2.0 ** 100, 2.0 ** -120)):
        ga = (ga * rng.uniform(0.5, 2, E)).astype(np.float32)
        f = alpha * ga.astype(np.float64) * gb
        for dtype in DTYPES:
            got = run_experts(a, sfa, b, sfb, ids, k, dtype, "blocked", alpha, ga, np.array([gb], np.float32))
            for e in range(E):
                slots = np.nonzero(ids.reshape(-1) == e)[0]
                va, vb = ref.values(a[e], sfa[e]), ref.values(b[0], sfb[0])[slots // k]
                want, size = vb @ va.T * f[e], np.abs(vb) @ np.abs(va).T * f[e]
                off = np.abs(got[dev(slots)].double().cpu().numpy() - want) - ref.product_tolerance(K, size, want, dtype)
                fine = np.abs(want) < torch.finfo(dtype).max * 0.99
                assert not fine.any() or off[fine].max() <= 0, f"{dtype} expert {e}: worst by {off[fine].max():.3g}"


# a tile in slices that the lists above do not reach: 128 x 32
SLICED_TILES = [(52, 37, 4, 240, 32160)]


@pytest.mark.parametrize("T,E,k,M,K", SLICED_TILES)
def test_experts_more_tiles_in_slices(T, E, k, M, K):
    test_experts_every_tile(T, E, k, M, K)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,k", [(19, 64, 1), (200, 64, 2), (18, 128, 8), (301, 256, 8), (66, 256, 15), (5, 256, 6), (90, 512, 4), (70, 1024, 8)])
def test_equals_at_the_last_pick_hide_no_larger_one(T, E, k, score):
    """The expert of the last pick and the next share a logit: what stands behind them, as
    close in float32, may be larger."""
    rng = np.random.default_rng([T, E, k])
    logits = ref.equals_at_the_last_pick(rng, T, E, k, score == "sigmoid")
    for bias in (None, np.full(E, 0.03125, np.float32)):
        z = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")  # noqa: E731
        ids, offsets, order, weights = z(T, k), z(E + 1), z(T * k), torch.zeros(T, k, device="cuda")
        ws = torch.zeros(max(256, g.nvfp4_moe_route_workspace_bytes(T, E, k)), dtype=torch.uint8, device="cuda")
        g.nvfp4_moe_route(logits.cuda(), ids, weights, offsets, order, T, E, k, score=score,
                          bias=None if bias is None else dev(bias), workspace=ws)
        want, _ = ref.route(logits.double().numpy(), bias, k, score)
        assert np.array_equal(ids.cpu().numpy(), want), np.argwhere(ids.cpu().numpy() != want)[:4]


@pytest.mark.parametrize("k,score,biased", [(1, "sigmoid", True), (2, "softmax", False), (8, "sigmoid", False), (8, "softmax", True)])
def test_ids_of_many_near_ties(k, score, biased):
    """Logits on a coarse grid, some a few 2^-20 off it: 20000 tokens against 64 bits."""
    T, E = 20000, 64
    gen = torch.Generator(device="cuda").manual_seed(k)
    x = (torch.randn(T, E, device="cuda", generator=gen) * (12 if k < 8 else 2) * 16).round() / 16
    x += torch.randint(-2, 3, (T, E), device="cuda", generator=gen) * 2.0 ** -20
    bias = (torch.randn(E, device="cuda", generator=gen) * 2).round() / 64 if biased else None
    z = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")  # noqa: E731
    ids, offsets, order, weights = z(T, k), z(E + 1), z(T * k), torch.zeros(T, k, device="cuda")
    ws = torch.zeros(g.nvfp4_moe_route_workspace_bytes(T, E, k), dtype=torch.uint8, device="cuda")
    g.nvfp4_moe_route(x, ids, weights, offsets, order, T, E, k, score=score, bias=bias, workspace=ws)
    v = x.double()
    if score == "softmax":
        pick = torch.exp(v - v.amax(1, keepdim=True))
        pick = pick / pick.sum(1, keepdim=True)
    else:
        pick = 1 / (1 + torch.exp(-v))
    if biased:
        pick = pick + bias.double()
    # both sides' float64 scores are a few 2^-53 off: an id that differs is of such a pick
    want = pick.sort(dim=1, descending=True, stable=True).indices[:, :k]
    off = (pick.gather(1, ids.long()) - pick.gather(1, want)).abs()
    assert off.max() <= 2.0 ** -50, (int((off > 2.0 ** -50).sum()), off.max())
