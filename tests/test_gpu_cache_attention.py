"""GPU: attention over a paged NVFP4 cache against a 64-bit form: head sizes and
layouts, lengths from none to long ones, ragged batches of single tokens, drafts and
prompts, masks that leave a row empty, pages that are not there, values that are not
finite in seen and in hidden places, rows of no sequence, far pages, captured graphs."""
import numpy as np
import pytest

import attention_reference as ref
from cache_cases import poisoned
from test_gpu_cache import on_device

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import block_scaled_fp4_gemv_amd as g  # noqa: E402

DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module")
def workspace():
    return torch.zeros(g.NVFP4_WORKSPACE_MAX_BYTES, dtype=torch.uint8, device="cuda")


def run(c, table, lengths, counts, H, dtype, workspace, seed=0, max_q=None, max_length=None, scale=None, causal=True, window=0,
        lead=0, tail=3, q=None, size=2.0, what=""):
    """One call on ragged rows (`lead` rows of no sequence before them, `tail` behind), checked; returns out."""
    rng = np.random.default_rng([seed, H, len(lengths)])
    offsets = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32) + lead
    T, D = int(offsets[-1]) + tail, c.D
    if q is None:
        q = torch.from_numpy(rng.standard_normal((T, H, D)) * size).to(dtype)
    max_q = max_q or max(1, max(counts))
    max_length = max_length or table.shape[1] * c.page_size
    scale = D ** -0.5 if scale is None else scale
    handle, _ = on_device(c)
    out = torch.full((T, H, D), 7.0, dtype=dtype, device="cuda")
    lse = torch.full((T, H), 7.0, device="cuda")
    g.nvfp4_cache_attention(handle, q.cuda(), out, torch.from_numpy(offsets).cuda(), torch.tensor(lengths, dtype=torch.int32).cuda(),
                            torch.from_numpy(table).cuda(), T, H, len(lengths), max_q, max_length, scale=scale, causal=causal,
                            window=window, lse=lse, workspace=workspace)
    # k's values are the definition's, the logits' factor is float32's product
    want = ref.attention(c, q.double().numpy(), offsets, lengths, table, max_q, max_length, np.float64(np.float32(scale)), causal, window)
    ref.check_attention(out, lse, want, dtype, what)
    assert (out[torch.from_numpy(~want["written"]).cuda()] == 7).all() and (lse[torch.from_numpy(~want["written"]).cuda()] == 7).all()
    if workspace is not None:
        assert not workspace[:65536].any(), "the workspace's counters are not zero"
    return out


@pytest.mark.parametrize("dtype", sorted(DTYPES))
@pytest.mark.parametrize("D,H,heads,page_size", [(64, 1, 1, 16), (64, 8, 1, 64), (96, 6, 2, 32), (128, 8, 2, 16), (128, 40, 1, 16),
                                                 (128, 7, 7, 128), (192, 16, 2, 32), (256, 4, 1, 64), (256, 24, 2, 16)])
def test_single_tokens_of_ragged_lengths(D, H, heads, page_size, dtype, workspace):
    rng = np.random.default_rng([D, H])
    lengths = [0, 1, 2, 15, 16, 17, 31, 33, 63, 64, 65, 127, 200, 517]
    c, table = poisoned(rng, lengths, page_size, heads, D)
    run(c, table, lengths, [1] * len(lengths), H, DTYPES[dtype], workspace)


@pytest.mark.parametrize("dtype", sorted(DTYPES))
@pytest.mark.parametrize("D,H,heads", [(64, 8, 2), (96, 4, 4), (128, 8, 1), (128, 32, 4), (192, 6, 2), (256, 8, 4)])
@pytest.mark.parametrize("window", [0, 1, 40])
def test_drafts_and_prompts_in_one_batch(D, H, heads, window, dtype, workspace):
    """Sequences without a row, single tokens, drafts, prompts; more rows than positions, whose first ones see nothing."""
    rng = np.random.default_rng([D, H, window])
    counts = [1, 0, 5, 70, 3, 130, 1, 17, 9]
    lengths = [77, 40, 5, 70, 290, 200, 1, 0, 4]
    c, table = poisoned(rng, lengths, 16, heads, D, width=20)
    run(c, table, lengths, counts, H, DTYPES[dtype], workspace, window=window, lead=2)


@pytest.mark.parametrize("dtype", sorted(DTYPES))
@pytest.mark.parametrize("window", [0, 30])
def test_without_the_causal_mask(dtype, window, workspace):
    rng = np.random.default_rng(window)
    lengths, counts = [100, 33, 0, 64], [7, 40, 3, 1]
    c, table = poisoned(rng, lengths, 32, 2, 128)
    run(c, table, lengths, counts, 4, DTYPES[dtype], workspace, causal=False, window=window)


@pytest.mark.parametrize("dtype", sorted(DTYPES))
@pytest.mark.parametrize("D,H,heads,B,n", [(128, 8, 2, 1, 1), (64, 4, 1, 3, 2), (192, 2, 1, 2, 40), (256, 8, 1, 1, 20), (96, 3, 3, 2, 1),
                                           (256, 2, 1, 1, 1), (192, 3, 1, 1, 2), (128, 16, 1, 1, 2), (64, 8, 1, 2, 6), (96, 16, 1, 1, 3),
                                           (64, 40, 1, 1, 7), (96, 4, 1, 1, 50), (128, 4, 1, 1, 130), (256, 20, 1, 1, 1)])
def test_long_lengths_are_split_and_joined(D, H, heads, B, n, dtype, workspace):
    rng = np.random.default_rng([D, B, n])
    lengths = [int(v) for v in rng.integers(5000, 9000, B)]
    c, table = poisoned(rng, lengths, 64, heads, D)
    out = run(c, table, lengths, [n] * B, H, DTYPES[dtype], workspace)
    assert torch.equal(out, run(c, table, lengths, [n] * B, H, DTYPES[dtype], workspace)), "equal calls differ"
    # bounds far above the lengths plan another grid
    wide = np.concatenate([table, np.full((B, 500), -1, np.int32)], 1)
    run(c, wide, lengths, [n] * B, H, DTYPES[dtype], workspace)


@pytest.mark.parametrize("dtype", sorted(DTYPES))
@pytest.mark.parametrize("D,H,heads,n,window", [(128, 8, 2, 1, 2500), (64, 16, 1, 3, 1000), (192, 4, 1, 40, 1500), (256, 4, 2, 60, 3000),
                                                (128, 4, 4, 200, 700), (96, 8, 1, 9, 4000)])
def test_windows_of_long_lengths(D, H, heads, n, window, dtype, workspace):
    rng = np.random.default_rng([D, n, window])
    lengths = [6007, 300, 4096]
    c, table = poisoned(rng, lengths, 32, heads, D)
    run(c, table, lengths, [n] * 3, H, DTYPES[dtype], workspace, window=window)


def test_two_streams_at_once_with_workspaces_of_their_own():
    rng = np.random.default_rng(21)
    lengths, D, H, heads = [4000, 5000], 128, 8, 2
    c, table = poisoned(rng, lengths, 64, heads, D)
    handle, _ = on_device(c)
    streams = [torch.cuda.Stream() for _ in range(2)]
    calls = []
    for n in (1, 30):
        q = torch.from_numpy(rng.standard_normal((2 * n, H, D)) * 2).bfloat16().cuda()
        off, ln, tb = (torch.arange(3, dtype=torch.int32) * n).cuda(), torch.tensor(lengths, dtype=torch.int32).cuda(), torch.from_numpy(table).cuda()
        ws = torch.zeros(g.NVFP4_WORKSPACE_MAX_BYTES, dtype=torch.uint8, device="cuda")
        calls.append((q, off, ln, tb, n, ws, [torch.zeros_like(q) for _ in range(20)]))
    torch.cuda.synchronize()
    for k in range(20):
        for stream, (q, off, ln, tb, n, ws, outs) in zip(streams, calls):
            g.nvfp4_cache_attention(handle, q, outs[k], off, ln, tb, 2 * n, H, 2, n, 5056, workspace=ws, stream=stream)
    torch.cuda.synchronize()
    for q, off, ln, tb, n, ws, outs in calls:
        want = ref.attention(c, q.double().cpu().numpy(), off.tolist(), lengths, table, n, 5056, np.float64(np.float32(D ** -0.5)))
        ref.check_attention(outs[0], None, want, torch.bfloat16)
        assert all(torch.equal(o, outs[0]) for o in outs)


def test_tables_with_pages_that_are_not_there(workspace):
    rng = np.random.default_rng(3)
    lengths, counts = [150, 40, 300, 16], [1, 6, 80, 1]
    c, table = poisoned(rng, lengths, 16, 2, 64)
    table[0, 3], table[0, 9], table[1, :] = -1, c.pages, 2 ** 31 - 1
    table[2, 4:9], table[2, 0] = -2 ** 31, -7
    table[3, 0] = -1
    for dtype in DTYPES.values():
        run(c, table, lengths, counts, 4, dtype, workspace)
        run(c, table, lengths, counts, 4, dtype, workspace, window=20)


def test_offsets_and_lengths_are_clamped(workspace):
    rng = np.random.default_rng(4)
    c, table = poisoned(rng, [64, 64, 64], 16, 1, 64)
    handle, _ = on_device(c)
    T, H = 12, 2
    q = torch.from_numpy(rng.standard_normal((T, H, 64))).half()
    for offsets, lengths, max_q, max_length in (([-5, 3, 7, 100], [64, 64, 64], 4, 64), ([0, 5, 4, 9], [1000, -3, 20], 5, 50),
                                                ([0, 1, 2, 3], [2 ** 31 - 1, -2 ** 31, 64], 1, 64), ([0, 6, 9, 12], [64, 10, 2], 2, 64)):
        off, ln = torch.tensor(offsets, dtype=torch.int32), torch.tensor(lengths, dtype=torch.int32)
        out, lse = torch.full((T, H, 64), 7.0, dtype=torch.float16, device="cuda"), torch.full((T, H), 7.0, device="cuda")
        g.nvfp4_cache_attention(handle, q.cuda(), out, off.cuda(), ln.cuda(), torch.from_numpy(table).cuda(), T, H, 3, max_q, max_length,
                                lse=lse, workspace=workspace)
        want = ref.attention(c, q.double().numpy(), offsets, lengths, table, max_q, max_length, 0.125)
        # offsets that fall give a row to two sequences: either's result may stay there
        rows = np.zeros(T, int)
        for b in range(3):
            first = min(max(offsets[b], 0), T)
            rows[first:min(first + max_q, max(offsets[b + 1], first), T)] += 1
        twice = rows > 1
        want["written"] &= ~twice
        ref.check_attention(out, lse, want, torch.float16, str(offsets))
        assert (out[torch.from_numpy(~want["written"] & ~twice).cuda()] == 7).all()


@pytest.mark.parametrize("dtype", sorted(DTYPES))
@pytest.mark.parametrize("n", [1, 6, 90])
def test_values_that_are_not_finite(n, dtype, workspace):
    """NaN scales of a key make NaN of the queries that see it, of a value the block of
    those; a query's own NaN or infinity the query. Queries before them are untouched."""
    rng = np.random.default_rng(n)
    length = 200
    c, table = poisoned(rng, [length] * 6, 16, 2, 128)
    place = lambda b, t: (table[b, t // 16], slice(None), t % 16)  # noqa: E731
    late = length - 1 - n // 2
    c.ks[place(0, late)][0, 3] = 0x7F
    c.vs[place(1, late)][1, 5] = 0xFF
    c.vs[place(2, 7)][0, 0] = 0x7F
    c.vs[place(5, late - 1)][0, 7], c.vs[place(5, late)][0, 2] = 0x7F, 0x7F
    H = 4
    q = torch.from_numpy(rng.standard_normal((6 * n + 3, H, 128)) * 2).to(DTYPES[dtype])
    q[3 * n, 1, 17], q[3 * n, 2, 0], q[4 * n, 0, 127] = float("nan"), float("inf"), float("-inf")
    for window in (0, 50):
        out = run(c, table, [length] * 6, [n] * 6, H, DTYPES[dtype], workspace, q=q, window=window)
        assert torch.isnan(out).any() and not torch.isnan(out).all()


@pytest.mark.parametrize("dtype", sorted(DTYPES))
def test_large_and_small_queries(dtype, workspace):
    """Rows of very different sizes; logits in the hundreds, where one position takes all; none at all."""
    rng = np.random.default_rng(11)
    lengths = [90, 400, 33]
    c, table = poisoned(rng, lengths, 16, 1, 64)
    for n in (1, 40):
        T = 3 * n + 3
        size = 2.0 ** rng.integers(-12, 9, (T, 1, 1))
        q = torch.from_numpy(rng.standard_normal((T, 4, 64)) * size).to(DTYPES[dtype])
        q[0] = 0
        run(c, table, lengths, [n] * 3, 4, DTYPES[dtype], workspace, q=q)
    if dtype != "f16":
        q = torch.from_numpy(rng.standard_normal((6, 4, 64)) * 1e-30).to(DTYPES[dtype])
        run(c, table, lengths, [1] * 3, 4, DTYPES[dtype], workspace, q=q, scale=1e29)
        q = torch.from_numpy(rng.standard_normal((6, 4, 64)) * 1e30).to(DTYPES[dtype])
        run(c, table, lengths, [1] * 3, 4, DTYPES[dtype], workspace, q=q, scale=-1e-31)


def test_strided_queries_no_lse_and_no_global_scales(workspace):
    rng = np.random.default_rng(12)
    lengths, counts, H, D = [50, 61], [3, 40], 6, 64
    c, table = poisoned(rng, lengths, 32, 2, D)
    c.gk = c.gv = 1.0
    handle, views = on_device(c)
    bare = g.Nvfp4Cache(*views, c.pages, 32, 2, D)
    T = sum(counts)
    packed = torch.from_numpy(rng.standard_normal((T, H + 4, D)) * 0.02).half().cuda()
    q = packed[:, 2:2 + H]
    off, ln, tb = torch.tensor([0, 3, 43], dtype=torch.int32).cuda(), torch.tensor(lengths, dtype=torch.int32).cuda(), torch.from_numpy(table).cuda()
    out = torch.empty(T, H, D, dtype=torch.float16, device="cuda")
    g.nvfp4_cache_attention(bare, q, out, off, ln, tb, T, H, 2, 40, 64, token_stride=q.stride(0), head_stride=q.stride(1),
                            workspace=workspace)
    want = ref.attention(c, q.double().cpu().numpy(), [0, 3, 43], lengths, table, 40, 64, D ** -0.5)
    ref.check_attention(out, None, want, torch.float16)
    again = torch.empty_like(out)
    g.nvfp4_cache_attention(handle, q.contiguous(), again, off, ln, tb, T, H, 2, 40, 64, workspace=workspace)
    assert torch.equal(out, again)


def test_a_cache_past_4_gib(workspace):
    """Pages 3 GiB apart, codes and scales in one allocation."""
    rng = np.random.default_rng(13)
    D, heads, stride = 128, 1, 3 << 30
    c, table = poisoned(rng, [48], 16, heads, D, spare=0)
    room = torch.zeros(2 * stride + (1 << 14), dtype=torch.uint8, device="cuda")
    views = []
    for i, name in enumerate(("kc", "ks", "vc", "vs")):
        a = torch.from_numpy(getattr(c, name))
        view = room[i * 2048:].as_strided(a.shape, (stride, a.stride(1), a.stride(2), 1))
        view.copy_(a)
        views.append(view)
    gk, gv = (torch.tensor([v], dtype=torch.float32, device="cuda") for v in (c.gk, c.gv))
    handle = g.Nvfp4Cache(*views, 3, 16, heads, D, k_scale=gk, v_scale=gv, code_page_stride=stride, scale_page_stride=stride)
    for n in (1, 40):
        q = torch.from_numpy(rng.standard_normal((n, 4, D)) * 2).bfloat16()
        out, lse = torch.empty(n, 4, D, dtype=torch.bfloat16, device="cuda"), torch.empty(n, 4, device="cuda")
        g.nvfp4_cache_attention(handle, q.cuda(), out, torch.tensor([0, n], dtype=torch.int32).cuda(),
                                torch.tensor([48], dtype=torch.int32).cuda(), torch.from_numpy(table).cuda(), n, 4, 1, n, 48, lse=lse,
                                workspace=workspace)
        want = ref.attention(c, q.double().numpy(), [0, n], [48], table, n, 48, D ** -0.5)
        ref.check_attention(out, lse, want, torch.bfloat16)


@pytest.mark.parametrize("n,lengths", [(1, [700, 3000, 64]), (37, [700, 3000, 64])])
def test_captured_calls_follow_their_inputs(n, lengths):
    """Replays, with eager calls between, equal eager calls on the same values; lengths, offsets and tables change."""
    rng = np.random.default_rng(14)
    D, H, heads, B = 128, 8, 2, 3
    c, table = poisoned(rng, lengths, 64, heads, D)
    handle, _ = on_device(c)
    T = B * n
    q = torch.randn(T, H, D, device="cuda").bfloat16()
    off, ln = torch.arange(B + 1, device="cuda", dtype=torch.int32) * n, torch.tensor(lengths, dtype=torch.int32, device="cuda")
    tb = torch.from_numpy(table).cuda()
    out, eager = torch.zeros(T, H, D, dtype=torch.bfloat16, device="cuda"), torch.zeros(T, H, D, dtype=torch.bfloat16, device="cuda")
    ws = torch.zeros(max(256, g.nvfp4_cache_attention_workspace_bytes(handle, torch.bfloat16, T, H, B, n, 3008)), dtype=torch.uint8, device="cuda")

    def call(to):
        g.nvfp4_cache_attention(handle, q, to, off, ln, tb, T, H, B, n, 3008, workspace=ws)

    call(out)
    torch.cuda.synchronize()
    graph, second = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(out)
    with torch.cuda.graph(second):
        call(eager)
    for k in range(4):
        q.copy_(torch.randn(T, H, D, device="cuda"))
        ln.copy_(torch.tensor([max(n, v // (k + 1)) for v in lengths], dtype=torch.int32))
        tb.copy_(torch.from_numpy(np.roll(table, k, 0)))
        out.fill_(7), eager.fill_(9)
        graph.replay()
        if k % 2:
            second.replay()
        else:
            call(eager)
        torch.cuda.synchronize()
        assert torch.equal(out.view(torch.int16), eager.view(torch.int16))        # NaN where a rolled table meets other pages
    assert not ws[:65536].any()


def test_workspace_rules():
    rng = np.random.default_rng(15)
    c, table = poisoned(rng, [4096], 64, 1, 128)
    handle, _ = on_device(c)
    q, out = torch.randn(1, 4, 128, device="cuda").half(), torch.empty(1, 4, 128, dtype=torch.float16, device="cuda")
    args = (handle, q, out, torch.tensor([0, 1], dtype=torch.int32).cuda(), torch.tensor([4096], dtype=torch.int32).cuda(),
            torch.from_numpy(table).cuda(), 1, 4, 1, 1, 4096)
    need = g.nvfp4_cache_attention_workspace_bytes(handle, torch.float16, 1, 4, 1, 1, 4096)
    assert 0 < need <= g.NVFP4_WORKSPACE_MAX_BYTES and need % 256 == 0
    ws = torch.zeros(need + 256, dtype=torch.uint8, device="cuda")
    g.nvfp4_cache_attention(*args, workspace=ws[:need])
    for bad in (dict(workspace=None), dict(workspace=ws[:need - 1]), dict(workspace=ws[16:16 + need])):
        with pytest.raises(g.Nvfp4Error) as e:
            g.nvfp4_cache_attention(*args, **bad)
        assert e.value.status == g.NVFP4_ERR_WORKSPACE
    with pytest.raises(ValueError, match="workspace holds"):
        g.nvfp4_cache_attention(*args, workspace=ws, workspace_bytes=need + 4096)


def test_binding_refuses_what_does_not_fit(workspace):
    rng = np.random.default_rng(16)
    c, table = poisoned(rng, [64, 64], 16, 2, 64)
    handle, _ = on_device(c)
    q, out = torch.zeros(4, 4, 64, device="cuda"), torch.zeros(4, 4, 64, device="cuda")
    off, ln, tb = torch.tensor([0, 2, 4], dtype=torch.int32).cuda(), torch.tensor([64, 64], dtype=torch.int32).cuda(), torch.from_numpy(table).cuda()
    good = dict(q=q, out=out, offsets=off, lengths=ln, table=tb, T=4, H=4, B=2, max_q=2, max_length=64, workspace=workspace)
    g.nvfp4_cache_attention(handle, **good)
    for bad, what in ((dict(q=q[:3]), "q holds"), (dict(out=out.half()), "out is"), (dict(offsets=off[:2]), "offsets holds"),
                      (dict(lengths=ln.long()), "int64, not int32"), (dict(table=tb.float()), "not int32"), (dict(lse=out[0, 0, :15]), "lse holds"),
                      (dict(q=q[:, :2], H=2), "not contiguous"), (dict(table=tb[:, ::2]), "contiguous"), (dict(q=q.cpu()), "device")):
        with pytest.raises(ValueError, match=what):
            g.nvfp4_cache_attention(handle, **{**good, **bad})
    with pytest.raises(g.Nvfp4Error) as e:
        g.nvfp4_cache_attention(handle, **{**good, "max_length": 65})
    assert e.value.status == g.NVFP4_ERR_INVALID_SHAPE


def test_rows_of_a_layer_step_by_step_and_at_once(workspace):
    """Rope, write and attention as a layer uses them: a prompt at once, then tokens one by
    one, then drafts; each step equals the 64-bit attention over what the cache then holds."""
    gen = torch.Generator(device="cuda").manual_seed(17)
    B, H, heads, D, page_size, prompt = 3, 8, 2, 128, 16, [40, 1, 90]
    pages, width = 40, 12
    views = [torch.zeros(pages, heads, page_size, D // n, dtype=torch.uint8, device="cuda") for n in (2, 16, 2, 16)]
    gk, gv = torch.tensor([0.004], device="cuda"), torch.tensor([0.003], device="cuda")
    cache = g.Nvfp4Cache(*views, pages, page_size, heads, D, k_scale=gk, v_scale=gv)
    table = torch.randperm(pages, generator=gen, device="cuda")[:B * width].reshape(B, width).to(torch.int32)
    f = torch.tensor(g.nvfp4_rope_frequencies(D, 500000.0, "bands", 8.0, 8192.0, 1.0, 4.0), dtype=torch.float64, device="cuda")
    lengths = [0] * B
    for counts in (prompt, [1, 1, 1], [1, 0, 1], [4, 4, 4]):
        T = sum(counts)
        qkv = torch.randn(T, H + 2 * heads, D, device="cuda", generator=gen).bfloat16()
        before = qkv.clone()
        positions = torch.cat([torch.arange(n, n + m) for n, m in zip(lengths, counts)]).cuda()
        seq = torch.cat([torch.full((m,), b) for b, m in enumerate(counts)]).cuda()
        lengths = [n + m for n, m in zip(lengths, counts)]
        g.nvfp4_rope(qkv, qkv, positions, f, T, H + heads, D, D, token_stride=qkv.stride(0), head_stride=D)
        assert torch.equal(qkv[:, H + heads:], before[:, H + heads:]) and not torch.equal(qkv[:, :H], before[:, :H])
        slots = table[seq, positions // page_size].long() * page_size + positions % page_size
        k, v = qkv[:, H:H + heads], qkv[:, H + heads:]
        g.nvfp4_cache_write(cache, k, v, slots, T, k_strides=(k.stride(0), D), v_strides=(v.stride(0), D))
        out = torch.empty(T, H, D, dtype=torch.bfloat16, device="cuda")
        off = torch.tensor([0] + list(np.cumsum(counts)), dtype=torch.int32).cuda()
        q = qkv[:, :H]
        g.nvfp4_cache_attention(cache, q, out, off, torch.tensor(lengths, dtype=torch.int32).cuda(), table, T, H, B, max(counts),
                                width * page_size, token_stride=q.stride(0), head_stride=D, workspace=workspace)
        c = ref.Cache.__new__(ref.Cache)
        c.pages, c.page_size, c.heads, c.D, c.gk, c.gv = pages, page_size, heads, D, float(gk.double()), float(gv.double())
        c.kc, c.ks, c.vc, c.vs = (x.cpu().numpy() for x in views)
        want = ref.attention(c, q.double().cpu().numpy(), off.tolist(), lengths, table.cpu().numpy(), max(counts), width * page_size,
                             np.float64(np.float32(D ** -0.5)))
        ref.check_attention(out, None, want, torch.bfloat16, str(counts))


@pytest.mark.parametrize("n", [0, 1, 7, 64, 130])
@pytest.mark.parametrize("D,G,dtype", [(64, 1, torch.float16), (128, 4, torch.bfloat16), (192, 4, torch.float32), (256, 8, torch.bfloat16)])
def test_a_lone_sequence_below_its_bound(workspace, D, G, dtype, n):
    """Room for 130 queries, for fewer of them; the rows behind stay as they were."""
    rng = np.random.default_rng(D + n)
    c, table = poisoned(rng, [2111], 32, 2, D)
    run(c, table, [2111], [n], 2 * G, dtype, workspace, max_q=130, tail=130 - n)
