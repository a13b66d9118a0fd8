"""FP4 linear layers and routed experts: the cases that are measured.

Operators (names of block_scaled_fp4_gemv_amd, symbols of include/nvfp4_gemv.h):

  quantize  nvfp4_global_scale, nvfp4_quantize, nvfp4_dequantize: activations to NVFP4 with a scale of
            their own, and the values that the codes stand for
  gemm      nvfp4_gemm: NVFP4 weights times N quantised rows
  route     nvfp4_moe_route: scores to the top-k experts of each token, and the experts' lists
  experts   nvfp4_gemm_experts: each slot's row times its expert's NVFP4 weights
  combine   nvfp4_moe_combine: the weighted sum of each token's slots

``run`` is either the framework's call or its plain form in elementary torch
operations; ``exact`` is the definition in 64 bits, on its own code.
"""
import math

import torch

own = False

E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
DTYPES = {"float16": torch.float16, "bfloat16": torch.bfloat16, "float32": torch.float32}


def _cdiv(a, b):
    return -(-a // b)


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # activations of one decoding batch: three short launches, latency counts
        dict(name="quantize decode", op="quantize", rows=16, K=7168, L=1, pad=0, dtype="bfloat16", layout="blocked"),
        # a long prompt's activations in one call
        dict(name="quantize prompt", op="quantize", rows=8192, K=7168, L=1, pad=0, dtype="bfloat16", layout="blocked"),
        # the output projection of a decoding batch of 16 sequences
        dict(name="gemm decode", op="gemm", M=7168, N=16, K=2048, L=1, out="float16", layout="blocked"),
        # a ragged batch of a few hundred tokens, scales as an exporter writes them
        dict(name="gemm ragged plain", op="gemm", M=4096, N=333, K=7168, L=1, out="bfloat16", layout="plain"),
        # a prompt of 4096 tokens through the repository's largest matrix
        dict(name="gemm prompt", op="gemm", M=7168, N=4096, K=16384, L=1, out="bfloat16", layout="blocked"),
        # one token of a decoding step: sigmoid scores, a bias for balance, 4 of 8 groups
        dict(name="route one token", op="route", T=1, E=256, k=8, score="sigmoid", bias=True, n_group=8, topk_group=4,
             group_top=2, renormalize=True, scaling=2.5, dtype="float32"),
        # a batch of prompts, the same router
        dict(name="route prompt", op="route", T=16384, E=256, k=8, score="sigmoid", bias=True, n_group=8, topk_group=4,
             group_top=2, renormalize=True, scaling=2.5, dtype="float32"),
        # one token's first product: 8 experts' weights read, nothing shared
        dict(name="experts one token", op="experts", T=1, k=8, M=2048, K=7168, E=64, each=True, out="bfloat16",
             layout="blocked"),
        # a decoding batch: every expert has a few rows
        dict(name="experts decode batch", op="experts", T=64, k=4, M=4096, K=2048, E=64, each=False, out="float16",
             layout="blocked"),
        # a prompt's second product: ragged lists of hundreds of rows
        dict(name="experts prompt", op="experts", T=4096, k=4, M=7168, K=4096, E=32, each=False, out="bfloat16",
             layout="blocked"),
        # the combine of a decoding batch, and of a prompt
        dict(name="combine decode", op="combine", T=64, k=4, M=7168, dtype="float16"),
        dict(name="combine prompt", op="combine", T=8192, k=8, M=7168, dtype="bfloat16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("quantize", "gemm", "gemm", "route", "experts", "experts", "combine"))
    layout = rng.choice(("plain", "blocked"))
    out = rng.choice(tuple(DTYPES))
    if op == "quantize":
        rows, K = _log(rng, 1, 8192), 32 * _log(rng, 1, 512)
        rows = max(1, min(rows, 8192 * 7168 // 2 // K))
        L = rng.choice((1, 1, 3))
        return dict(op=op, rows=max(1, rows // L), K=K, L=L, pad=rng.choice((0, 0, 8, 33)), dtype=out, layout=layout)
    if op == "gemm":
        M, N, K = _log(rng, 1, 8192), _log(rng, 1, 4096), 32 * _log(rng, 1, 512)
        L = rng.choice((1, 1, 1, 2))
        return dict(op=op, M=M, N=max(1, min(N, int(4.5e11 / (L * M * K)))), K=K, L=L, out=out, layout=layout)
    if op == "route":
        E = rng.choice((8, 16, 60, 64, 128, 160, 256, 384))
        groups = rng.choice((1, 4)) if E % 4 == 0 else 1
        k = rng.choice((1, 2, 4, 6, 8))
        top = groups if groups == 1 or E // groups * 2 < k else 2
        return dict(op=op, T=_log(rng, 1, 10000), E=E, k=min(k, E // groups * top), score=rng.choice(("softmax", "sigmoid")),
                    bias=rng.random() < 0.5, n_group=groups, topk_group=top,
                    group_top=rng.choice((1, 2)) if E // groups > 1 else 1, renormalize=rng.random() < 0.7,
                    scaling=rng.choice((1.0, 2.5)), dtype=out)
    if op == "experts":
        k, E = rng.choice((1, 2, 4, 8)), rng.choice((8, 16, 32, 64))
        T, M, K = _log(rng, 1, 4096), _log(rng, 16, 4096), 32 * _log(rng, 2, 224)
        T = max(1, min(T, 16384 // k))
        return dict(op=op, T=T, k=k, M=M, K=K, E=E, each=rng.random() < 0.5, out=out, layout=layout)
    k, M = rng.choice((1, 2, 4, 8)), _log(rng, 32, 7168)
    T = max(1, min(_log(rng, 1, 8192), int(9e8 / ((k + 1) * M * DTYPES[out].itemsize))))
    return dict(op=op, T=T, k=k, M=M, dtype=out)


def work(case):
    c = case
    if c["op"] == "quantize":
        n, size = c["L"] * c["rows"] * c["K"], DTYPES[c["dtype"]].itemsize
        # read; codes and scales written; read again and the values written
        return {"bytes": n * (size + 2 * 9 / 16 + size), "flops": 0}
    if c["op"] == "gemm":
        M, N, K = c["M"], c["N"], c["K"]
        return {"bytes": c["L"] * ((M + N) * K * 9 / 16 + M * N * DTYPES[c["out"]].itemsize),
                "flops": 2 * c["L"] * M * N * K}
    if c["op"] == "route":
        return {"bytes": c["T"] * c["E"] * DTYPES[c["dtype"]].itemsize + 12 * c["T"] * c["k"] + 8 * c["E"], "flops": 0}
    if c["op"] == "experts":
        S, rows = c["T"] * c["k"], c["T"] * (1 if c["each"] else c["k"])
        hit = c["E"] * (1 - (1 - min(1.0, c["k"] / c["E"])) ** c["T"])
        return {"bytes": (hit * c["M"] + rows) * c["K"] * 9 / 16 + S * c["M"] * DTYPES[c["out"]].itemsize + 4 * S,
                "flops": 2 * S * c["M"] * c["K"]}
    n = c["T"] * c["M"] * DTYPES[c["dtype"]].itemsize
    return {"bytes": n * (c["k"] + 1) + 8 * c["T"] * c["k"], "flops": 2 * c["T"] * c["k"] * c["M"]}


# ------------------------------------------------------------------ inputs

def _scale_bytes(rows, K, L, layout):
    return L * (_cdiv(rows, 128) * _cdiv(K, 64) * 512 if layout == "blocked" else rows * (K // 16))


def _weights(gen, rows, K, L, layout):
    """Codes and scales as a quantiser leaves them: all codes, scales 2^u with u in [-3, 3]."""
    codes = torch.randint(0, 256, (L, rows, K // 2), dtype=torch.uint8, device="cuda", generator=gen)
    u = torch.rand(_scale_bytes(rows, K, L, layout), device="cuda", generator=gen) * 6 - 3
    return codes, torch.exp2(u).to(torch.float8_e4m3fn).view(torch.uint8)


def _activations(gen, *shape):
    """Rows of a normal distribution whose channels differ in size, some a lot."""
    size = torch.exp(torch.randn(shape[-1], device="cuda", generator=gen))
    return torch.randn(shape, device="cuda", generator=gen) * size


def _ids(gen, T, k, E):
    """Distinct experts for each token, some far more popular than others."""
    liked = torch.randn(E, device="cuda", generator=gen)
    gumbel = -torch.log(-torch.log(torch.rand(T, E, device="cuda", generator=gen).clamp(1e-9, 1 - 1e-7)))
    return torch.topk(gumbel + liked, k, dim=1).indices.to(torch.int32)


def prepare(case, seed):
    c = case
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    s = dict(case)
    if c["op"] == "quantize":
        rows, K, L, dt = c["rows"], c["K"], c["L"], DTYPES[c["dtype"]]
        s["x"] = _activations(gen, L, rows, K + c["pad"]).to(dt)[:, :, :K]
        s["g"] = torch.zeros(1, device="cuda")
        s["workspace"] = torch.zeros(256, dtype=torch.uint8, device="cuda")
        s["codes"] = torch.zeros(L, rows, K // 2, dtype=torch.uint8, device="cuda")
        s["scales"] = torch.zeros(_scale_bytes(rows, K, L, c["layout"]), dtype=torch.uint8, device="cuda")
        s["y"] = torch.zeros(L, rows, K, dtype=dt, device="cuda")
    elif c["op"] == "gemm":
        M, N, K, L = c["M"], c["N"], c["K"], c["L"]
        s["a"], s["sfa"] = _weights(gen, M, K, L, c["layout"])
        s["b"], s["sfb"] = _weights(gen, N, K, L, c["layout"])
        s["ga"], s["gb"] = (torch.rand(1, device="cuda", generator=gen) * 1e-2 + 1e-3 for _ in range(2))
        s["c"] = torch.zeros(L, N, M, dtype=DTYPES[c["out"]], device="cuda")
        s["workspace"] = torch.zeros(_gemm_workspace(M, N, K, L), dtype=torch.uint8, device="cuda")
    elif c["op"] == "route":
        T, E, k = c["T"], c["E"], c["k"]
        liked = torch.randn(E, device="cuda", generator=gen) * 0.5
        s["logits"] = (torch.randn(T, E, device="cuda", generator=gen) * 1.5 + liked).to(DTYPES[c["dtype"]])
        s["bias"] = torch.randn(E, device="cuda", generator=gen) * 0.02 if c["bias"] else None
        s["ids"] = torch.zeros(T, k, dtype=torch.int32, device="cuda")
        s["weights"] = torch.zeros(T, k, device="cuda")
        s["offsets"] = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
        s["order"] = torch.zeros(T * k, dtype=torch.int32, device="cuda")
        s["workspace"] = torch.zeros(_route_workspace(T, E, k), dtype=torch.uint8, device="cuda")
    elif c["op"] == "experts":
        T, k, M, K, E = c["T"], c["k"], c["M"], c["K"], c["E"]
        rows = T if c["each"] else T * k
        s["a"], s["sfa"] = _weights(gen, M, K, E, c["layout"])
        s["b"], s["sfb"] = _weights(gen, rows, K, 1, c["layout"])
        s["ga"] = torch.rand(E, device="cuda", generator=gen) * 1e-2 + 1e-3
        s["gb"] = torch.rand(1, device="cuda", generator=gen) * 1e-2 + 1e-3
        ids = _ids(gen, T, k, E).reshape(-1)
        counts = torch.bincount(ids.long(), minlength=E)
        s["offsets"] = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32)
        s["order"] = torch.argsort(ids, stable=True).to(torch.int32)
        s["ids"], s["most"] = ids, int(counts.max())
        s["c"] = torch.zeros(T * k, M, dtype=DTYPES[c["out"]], device="cuda")
        s["workspace"] = torch.zeros(_experts_workspace(M, K, E, T * k), dtype=torch.uint8, device="cuda")
    else:
        T, k, M, dt = c["T"], c["k"], c["M"], DTYPES[c["dtype"]]
        s["y"] = torch.randn(T * k, M, device="cuda", generator=gen).to(dt)
        w = torch.rand(T, k, device="cuda", generator=gen) + 0.05
        s["weights"] = w / w.sum(1, keepdim=True)
        ids = torch.randint(0, 64, (T, k), dtype=torch.int32, device="cuda", generator=gen)
        drop = torch.rand(T, k, device="cuda", generator=gen) < 0.02
        s["ids"] = torch.where(drop, torch.full_like(ids, -1), ids)
        s["out"] = torch.zeros(T, M, dtype=dt, device="cuda")
    return s


# Bytes of scratch that hold any plan of these shapes: counters, then float32
# partial sums of at most 64 MiB (products), or one counter per expert and
# block of slots (lists).
def _gemm_workspace(M, N, K, L):
    return 65536 + min(64 << 20, 4 * 16 * L * _cdiv(M, 256) * 256 * _cdiv(N, 256) * 256)


def _experts_workspace(M, K, E, S):
    return 65536 + min(64 << 20, 4 * 16 * S * _cdiv(M, 256) * 256)


def _route_workspace(T, E, k):
    return 4096 + 4 * (E + 64) * (_cdiv(T * k, 256) + 1)


# ------------------------------------------------------------------ one pass

def run(state):
    s = state
    if own:
        return _own(s)
    return {"quantize": _plain_quantize, "gemm": _plain_gemm, "route": _plain_route, "experts": _plain_experts,
            "combine": _plain_combine}[s["op"]](s)


def _own(s):
    import block_scaled_fp4_gemv_amd as g
    if s["op"] == "quantize":
        rows, K, L, x = s["rows"], s["K"], s["L"], s["x"]
        g.nvfp4_global_scale(x, s["g"], rows, K, L, s["workspace"], row_stride=x.stride(1), batch_stride=x.stride(0))
        g.nvfp4_quantize(x, s["codes"], s["scales"], rows, K, L, s["layout"], global_scale=s["g"],
                         row_stride=x.stride(1), batch_stride=x.stride(0))
        g.nvfp4_dequantize(s["codes"], s["scales"], s["y"], rows, K, L, s["layout"], global_scale=s["g"])
        return {"g": s["g"], "scales": s["scales"].view(torch.float8_e4m3fn), "values": s["y"]}
    if s["op"] == "gemm":
        g.nvfp4_gemm(s["a"], s["b"], s["sfa"], s["sfb"], s["c"], s["M"], s["N"], s["K"], s["L"], s["layout"],
                     scale_a=s["ga"], scale_b=s["gb"], workspace=s["workspace"])
        return s["c"]
    if s["op"] == "route":
        g.nvfp4_moe_route(s["logits"], s["ids"], s["weights"], s["offsets"], s["order"], s["T"], s["E"], s["k"],
                          score=s["score"], bias=s["bias"], n_group=s["n_group"], topk_group=s["topk_group"],
                          group_top=s["group_top"], renormalize=s["renormalize"], scaling=s["scaling"],
                          workspace=s["workspace"])
        return {"ids": s["ids"], "weights": s["weights"], "offsets": s["offsets"], "order": s["order"]}
    if s["op"] == "experts":
        rows, per = (s["T"], s["k"]) if s["each"] else (s["T"] * s["k"], 1)
        g.nvfp4_gemm_experts(s["a"], s["b"], s["sfa"], s["sfb"], s["c"], s["M"], s["K"], s["E"], rows, per, s["layout"],
                             s["offsets"], s["order"], scale_a=s["ga"], scale_b=s["gb"], workspace=s["workspace"])
        return s["c"]
    g.nvfp4_moe_combine(s["y"], s["ids"], s["weights"], s["out"], s["T"], s["k"], s["M"])
    return s["out"]


# ------------------------------------------------------------------ plain forms

def _blocked(m):
    """[L][rows][cols] -> the 128x4 blocked bytes, padding 0."""
    L, rows, cols = m.shape
    nrb, ncb = _cdiv(rows, 128), _cdiv(cols, 4)
    m = torch.nn.functional.pad(m, (0, 4 * ncb - cols, 0, 128 * nrb - rows))
    return m.reshape(L, nrb, 4, 32, ncb, 4).permute(0, 1, 4, 3, 2, 5).reshape(-1)


def _scale_matrix(scales, rows, K, L, layout):
    """The scale bytes as float32 [L][rows][K/16]."""
    v = scales.view(torch.float8_e4m3fn).float()
    if layout == "blocked":
        nrb, ncb = _cdiv(rows, 128), _cdiv(K, 64)
        v = v.reshape(L, nrb, ncb, 32, 4, 4).permute(0, 1, 4, 3, 2, 5).reshape(L, nrb * 128, ncb * 4)
    return v.reshape(L, -1, v.shape[-1] if layout == "blocked" else K // 16)[:, :rows, :K // 16]


def _code_values(codes):
    """[..., K/2] packed codes -> float32 [..., K]."""
    one = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=codes.device)
    both = torch.stack((one.repeat(16), one.repeat_interleave(16)), 1)      # low nibble first
    return both[codes.long()].reshape(*codes.shape[:-1], -1)


def _values(codes, scales, rows, K, L, layout):
    """e2m1 * e4m3, float32 [L][rows][K] (exact)."""
    v = _code_values(codes).reshape(L, rows, K // 16, 16)
    return (v * _scale_matrix(scales, rows, K, L, layout).unsqueeze(-1)).reshape(L, rows, K)


def _plain_quantize(s):
    rows, K, L, x = s["rows"], s["K"], s["L"], s["x"]
    amax = x.abs().amax().float()
    g = torch.where(amax > 0, amax / 2688, torch.ones_like(amax))
    v = x.double().reshape(L, rows, K // 16, 16)
    # scale: E4M3 steps of 2^(e-3), e >= -6, ties to even
    want = v.abs().amax(-1, keepdim=True) / (6 * g.double())
    step = torch.exp2(torch.floor(torch.log2(want.clamp(min=2.0 ** -6))) - 3)
    scale = (torch.round(want / step) * step).clamp(max=448)
    # codes: E2M1 steps of 2^(e-1), 0 <= e <= 2
    unit = scale * g.double()
    q = torch.where(unit > 0, v / unit, torch.zeros_like(v)).clamp(-6, 6)
    step = torch.exp2(torch.floor(torch.log2(q.abs().clamp(min=1.0))) - 1)
    q = torch.round(q / step) * step
    values = (q * unit).reshape(L, rows, K).to(x.dtype)
    m = scale.reshape(L, rows, K // 16).float()
    m = _blocked(m) if s["layout"] == "blocked" else m.reshape(-1)
    return {"g": g.reshape(1), "scales": m.to(torch.float8_e4m3fn), "values": values}


def _plain_gemm(s):
    M, N, K, L = s["M"], s["N"], s["K"], s["L"]
    a = _values(s["a"], s["sfa"], M, K, L, s["layout"])
    b = _values(s["b"], s["sfb"], N, K, L, s["layout"])
    acc = torch.bmm(b, a.transpose(1, 2).contiguous()) if L > 1 else torch.mm(b[0], a[0].t())
    return (acc.reshape(L, N, M) * (s["ga"] * s["gb"])).to(s["c"].dtype)


def _lists(ids, E):
    """Offsets of the experts' lists, and the slots sorted by expert."""
    flat = ids.reshape(-1)
    counts = torch.zeros(E, dtype=torch.int64, device=flat.device).index_add_(0, flat.long(), torch.ones_like(flat, dtype=torch.int64))
    offsets = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32)
    return offsets, torch.sort(flat, stable=True).indices.to(torch.int32)


def _plain_route(s):
    T, E, k, G = s["T"], s["E"], s["k"], s["n_group"]
    x = s["logits"].double()                                   # picks stand next to each other: 64 bits
    if s["score"] == "softmax":
        e = torch.exp(x - x.amax(1, keepdim=True))
        score = e / e.sum(1, keepdim=True)
    else:
        score = 1 / (1 + torch.exp(-x))
    pick = score + s["bias"].double() if s["bias"] is not None else score
    if G > 1:
        group = pick.reshape(T, G, -1).sort(dim=2, descending=True, stable=True).values[:, :, :s["group_top"]].sum(2)
        best = group.sort(dim=1, descending=True, stable=True).indices[:, :s["topk_group"]]
        keep = torch.zeros(T, G, dtype=torch.bool, device=x.device).scatter_(1, best, True)
        pick = pick.masked_fill(~keep.repeat_interleave(E // G, dim=1), -math.inf)
    ids = pick.sort(dim=1, descending=True, stable=True).indices[:, :k]
    w = score.gather(1, ids)
    if s["renormalize"]:
        w = w / w.sum(1, keepdim=True)
    ids = ids.to(torch.int32)
    offsets, order = _lists(ids, E)
    return {"ids": ids, "weights": (w * s["scaling"]).float(), "offsets": offsets, "order": order}


def _plain_experts(s):
    T, k, M, K, E, S = s["T"], s["k"], s["M"], s["K"], s["E"], s["T"] * s["k"]
    rows = T if s["each"] else S
    b = _values(s["b"], s["sfb"], rows, K, 1, s["layout"])[0]
    slot_row = torch.arange(S, device=b.device) // (k if s["each"] else 1)
    e = s["ids"].long()
    if S * 4 <= E:                                             # few slots: their experts' weights alone
        v = _code_values(s["a"][e])
        m = _scale_matrix(s["sfa"], M, K, E, s["layout"])[e]
        a = (v.reshape(S, M, K // 16, 16) * m.unsqueeze(-1)).reshape(S, M, K)
        acc = torch.bmm(a, b[slot_row].unsqueeze(2).contiguous()).squeeze(2)
    else:                                                      # each expert's rows, padded to the longest list
        a = _values(s["a"], s["sfa"], M, K, E, s["layout"])
        order = s["order"].long()
        place = torch.arange(S, device=b.device) - s["offsets"].long()[e[order]]
        packed = torch.zeros(E, s["most"], K, device=b.device)
        packed[e[order], place] = b[slot_row[order]]
        acc = torch.zeros(S, M, device=b.device)
        acc[order] = torch.bmm(packed, a.transpose(1, 2).contiguous())[e[order], place]
    return (acc * (s["ga"][e] * s["gb"]).unsqueeze(1)).to(s["c"].dtype)


def _plain_combine(s):
    T, k, M = s["T"], s["k"], s["M"]
    w = torch.where(s["ids"] >= 0, s["weights"], torch.zeros_like(s["weights"]))
    return (s["y"].float().reshape(T, k, M) * w.unsqueeze(2)).sum(1).to(s["y"].dtype)


# ------------------------------------------------------------------ the definition in 64 bits

def _nearest(v, table):
    """Each value's nearest entry of a sorted table whose entry i is code i: ties to the even code."""
    mids = (table[1:] + table[:-1]) / 2
    below, above = torch.bucketize(v, mids, right=False), torch.bucketize(v, mids, right=True)
    return table[torch.where(below == above, below, below + below % 2)]


def _operand(codes, scales, row, K, rows, layout, batch):
    """Rows `row` of batch `batch` in float64: codes [L][rows][K/2], scale positions by the formula."""
    kb = torch.arange(K // 16, device=codes.device).unsqueeze(0)
    r = row.unsqueeze(1)
    if layout == "blocked":
        at = ((r // 128) * _cdiv(K, 64) + kb // 4) * 512 + (r % 32) * 16 + ((r % 128) // 32) * 4 + kb % 4
    else:
        at = r * (K // 16) + kb
    at = at + batch * (_scale_bytes(rows, K, 1, layout))
    bits = scales[at].int()
    exponent, mantissa = (bits >> 3) & 15, (bits & 7).double()
    size = torch.where(exponent > 0, (8 + mantissa) * torch.exp2(exponent.double() - 10), mantissa * 2.0 ** -9)
    scale = torch.where(bits >= 128, -size, size)
    c = codes[batch][row].int()
    nibble = torch.stack((c & 15, c >> 4), 2).reshape(row.numel(), K)
    mag, up = (nibble & 1).double(), (nibble >> 1) & 3
    val = torch.where(up > 0, (1 + mag / 2) * torch.exp2(up.double() - 1), mag / 2)
    return torch.where(nibble >= 8, -val, val) * scale.repeat_interleave(16, dim=1)


def exact(case, seed):
    s = prepare(case, seed)
    c = case
    if c["op"] == "quantize":
        rows, K, L = c["rows"], c["K"], c["L"]
        x = s["x"].double()
        top = x.abs().max()
        g = (top / 2688).float().double() if float(top) > 0 else torch.ones_like(top)
        bits = torch.arange(127, device=x.device)
        e4m3 = torch.where(bits < 8, bits * 2.0 ** -9, (8 + bits % 8).double() * torch.exp2((bits // 8).double() - 10))
        e2m1 = torch.tensor(E2M1, dtype=torch.float64, device=x.device)
        blocks = x.reshape(L * rows * (K // 16), 16)
        scale = _nearest(blocks.abs().max(dim=1).values / (6 * g), e4m3)
        unit = (scale * g).unsqueeze(1)
        mag = _nearest(torch.where(unit > 0, blocks.abs() / unit, torch.zeros_like(blocks)), e2m1)
        values = torch.copysign(mag * unit, blocks).reshape(L, rows, K)
        if c["layout"] == "blocked":
            out = torch.zeros(s["scales"].numel(), dtype=torch.float64, device=x.device)
            l = torch.arange(L, device=x.device).reshape(L, 1, 1)
            r = torch.arange(rows, device=x.device).reshape(1, rows, 1)
            kb = torch.arange(K // 16, device=x.device).reshape(1, 1, K // 16)
            at = ((r // 128) * _cdiv(K, 64) + kb // 4) * 512 + (r % 32) * 16 + ((r % 128) // 32) * 4 + kb % 4
            out[(at + l * _scale_bytes(rows, K, 1, "blocked")).reshape(-1)] = scale
            scale = out
        # the global scale is a float32 by definition; in 64 bits it is the quotient
        return {"g": (top / 2688).reshape(1) if float(top) > 0 else g.reshape(1), "scales": scale, "values": values}
    if c["op"] == "gemm":
        M, N, K, L = c["M"], c["N"], c["K"], c["L"]
        m, n = torch.arange(M, device="cuda"), torch.arange(N, device="cuda")
        each = [_operand(s["b"], s["sfb"], n, K, N, c["layout"], l) @ _operand(s["a"], s["sfa"], m, K, M, c["layout"], l).t()
                for l in range(L)]
        return torch.stack(each) * s["ga"].double() * s["gb"].double()
    if c["op"] == "route":
        T, E, k, G = c["T"], c["E"], c["k"], c["n_group"]
        x = s["logits"].double()
        score = torch.softmax(x, 1) if c["score"] == "softmax" else torch.sigmoid(x)
        left = score.clone() if s["bias"] is None else score + s["bias"].double()
        if G > 1:
            best = left.reshape(T, G, E // G).topk(c["group_top"], dim=2).values.sum(2)
            groups = torch.zeros(T, G, dtype=torch.bool, device=x.device)
            for _ in range(c["topk_group"]):
                first = (best == best.max(1, keepdim=True).values).int().argmax(1, keepdim=True)
                groups.scatter_(1, first, True)
                best = best.scatter(1, first, -math.inf)
            left = torch.where(groups.unsqueeze(2).expand(T, G, E // G).reshape(T, E), left, torch.full_like(left, -math.inf))
        chosen = []
        for _ in range(k):
            first = (left == left.max(1, keepdim=True).values).int().argmax(1, keepdim=True)
            chosen.append(score.gather(1, first))
            left = left.scatter(1, first, -math.inf)
        w = torch.cat(chosen, 1)
        w = w / w.sum(1, keepdim=True) if c["renormalize"] else w
        return {"ids": None, "weights": w * c["scaling"], "offsets": None, "order": None}
    if c["op"] == "experts":
        T, k, M, K, E, S = c["T"], c["k"], c["M"], c["K"], c["E"], c["T"] * c["k"]
        rows = T if c["each"] else S
        out = torch.zeros(S, M, dtype=torch.float64, device="cuda")
        m, ids = torch.arange(M, device="cuda"), s["ids"]
        for e in range(E):
            slot = torch.nonzero(ids == e).reshape(-1)
            if slot.numel():
                a = _operand(s["a"], s["sfa"], m, K, M, c["layout"], e)
                b = _operand(s["b"], s["sfb"], slot // (k if c["each"] else 1), K, rows, c["layout"], 0)
                out[slot] = (b @ a.t()) * (s["ga"][e].double() * s["gb"].double())
        return out
    y = s["y"].double().reshape(c["T"], c["k"], c["M"])
    w = torch.where(s["ids"] < 0, 0.0, s["weights"].double()).reshape(c["T"], c["k"], 1)
    out = torch.zeros(c["T"], c["M"], dtype=torch.float64, device=y.device)
    for j in range(c["k"]):
        out += w[:, j] * y[:, j]
    return out
