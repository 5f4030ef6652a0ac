"""Cases of the 8-bit block-scaled products and of the routing to experts.

Five operators, in the order in which a layer of experts uses them:

* ``route``    router logits to the k chosen experts of each token, their weights, and the plan of rows by expert.
* ``pack``     real rows to e4m3 codes with one fp32 scale for each block of 1 x 128 (activations, with an optional
               gather of rows) or 128 x 128 (weights): s = max(max |x| / 448, 2^-126), code = e4m3(x * (1 / s)).
* ``gemm``     C[m, n] = sum over blocks b of K of sA[b, m] * sW[b, n / 128] * sum_{k in b} a[m, k] w[n, k].
* ``experts``  that product for rows grouped by expert, each group with its own weights.
* ``combine``  out[t] = sum_j weight[t, j] * Y[row of (t, j)].

Scales are block-major: the scale of row block i and K block b is ``scales[b, i]``.  Code rows are padded with
zeros to a multiple of 16 bytes.
"""
import math

import torch

own = False

BLOCK = 128
E4M3_MAX = 448.0
SCALE_MIN = 2.0 ** -126
DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


# --------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------

def listed():
    return [
        # one token through a softmax router (a decode step), fp32 logits
        {"name": "route_token", "op": "route", "T": 1, "E": 64, "k": 4, "score": "softmax", "bias": False,
         "groups": 1, "kept": 1, "dtype": "fp32"},
        # a prompt through a sigmoid router with a balance bias and groups of experts
        {"name": "route_prompt", "op": "route", "T": 8192, "E": 256, "k": 8, "score": "sigmoid", "bias": True,
         "groups": 8, "kept": 4, "dtype": "fp32"},
        # a prompt's rows gathered for its experts: 4096 tokens, 4 experts each
        {"name": "pack_gather", "op": "pack", "rows": 16384, "K": 4096, "source": 4096, "dtype": "bf16", "block_rows": 1},
        # one-off quantisation of fp32 weights, a K that fills no block
        {"name": "pack_weights", "op": "pack", "rows": 11008, "K": 4090, "source": 11008, "dtype": "fp32",
         "block_rows": 128},
        # the decode projection for a single token: the weights are streamed once
        {"name": "gemm_token", "op": "gemm", "M": 1, "N": 11008, "K": 4096, "out": "bf16"},
        # the down projection of a decode batch, fp32 out
        {"name": "gemm_batch", "op": "gemm", "M": 48, "N": 4096, "K": 11008, "out": "fp32"},
        # a ragged product: no size is a multiple of a block
        {"name": "gemm_ragged", "op": "gemm", "M": 333, "N": 1000, "K": 1000, "out": "fp32"},
        # the square compute-bound product
        {"name": "gemm_square", "op": "gemm", "M": 8192, "N": 8192, "K": 8192, "out": "bf16"},
        # experts' products for a decode batch: a few rows for most of the experts
        {"name": "experts_decode", "op": "experts", "T": 32, "k": 4, "E": 64, "N": 2048, "K": 4096, "out": "bf16"},
        # experts' products for a prompt: groups of uneven sizes
        {"name": "experts_prompt", "op": "experts", "T": 4096, "k": 4, "E": 32, "N": 2048, "K": 4096, "out": "bf16"},
        # a decode batch's expert rows back to its tokens
        {"name": "combine_decode", "op": "combine", "T": 32, "k": 8, "N": 4096, "dtype": "bf16"},
        # a prompt's expert rows back to its tokens
        {"name": "combine_prompt", "op": "combine", "T": 4096, "k": 4, "N": 4096, "dtype": "bf16"},
    ]


def _log(rng, lo, hi):
    """A whole number spread over the logarithm of [lo, hi]."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("route", "pack", "gemm", "gemm", "experts", "experts", "combine"))
    if op == "route":
        groups = rng.choice((1, 1, 2, 4, 8))
        per = rng.randint(max(2, 8 // groups), 256 // groups)
        kept = rng.randint(1, groups)
        return {"op": op, "T": _log(rng, 1, 8192), "E": groups * per, "k": rng.randint(1, min(8, kept * per)),
                "score": rng.choice(("softmax", "sigmoid")), "bias": rng.random() < 0.5, "groups": groups, "kept": kept,
                "dtype": rng.choice(("fp32", "bf16"))}
    if op == "pack":
        block_rows = rng.choice((1, 1, 128))
        rows, K = _log(rng, 1, 16384), _log(rng, 16, 11008)
        source = rows if block_rows == 128 else max(1, rows // rng.choice((1, 2, 4, 8)))
        return {"op": op, "rows": rows, "K": K, "source": source, "dtype": rng.choice(("fp32", "bf16")),
                "block_rows": block_rows}
    if op == "gemm":
        return {"op": op, "M": _log(rng, 1, 4096), "N": _log(rng, 64, 11008), "K": _log(rng, 64, 11008),
                "out": rng.choice(("fp32", "bf16"))}
    if op == "experts":
        E = rng.choice((4, 8, 16, 24, 32, 64))
        return {"op": op, "T": _log(rng, 1, 4096), "k": rng.randint(1, 4), "E": E, "N": _log(rng, 128, 2048),
                "K": _log(rng, 128, 4096), "out": rng.choice(("fp32", "bf16"))}
    return {"op": op, "T": _log(rng, 1, 8192), "k": rng.randint(1, 8), "N": _log(rng, 64, 4096),
            "dtype": rng.choice(("fp32", "bf16"))}


def _ld(K):
    return (K + 15) // 16 * 16


def _blocks(n):
    return (n + BLOCK - 1) // BLOCK


def work(case):
    op = case["op"]
    if op == "route":
        T, E, k = case["T"], case["E"], case["k"]
        size = 4 if case["dtype"] == "fp32" else 2
        plan = 4 * (E + 1) + 2 * 4 * T * k
        return {"bytes": T * E * size + (4 * E if case["bias"] else 0) + 8 * T * k + plan, "flops": 8 * T * E}
    if op == "pack":
        rows, K = case["rows"], case["K"]
        size = 4 if case["dtype"] == "fp32" else 2
        gather = 0 if case["source"] == rows else 4 * rows
        scales = 4 * _blocks(K) * (rows if case["block_rows"] == 1 else _blocks(rows))
        return {"bytes": case["source"] * K * size + gather + rows * _ld(K) + scales, "flops": 2 * rows * K}
    if op == "gemm":
        M, N, K = case["M"], case["N"], case["K"]
        out = 4 if case["out"] == "fp32" else 2
        return {"bytes": (M + N) * _ld(K) + 4 * _blocks(K) * (M + _blocks(N)) + M * N * out, "flops": 2 * M * N * K}
    if op == "experts":
        R, E, N, K = case["T"] * case["k"], case["E"], case["N"], case["K"]
        out = 4 if case["out"] == "fp32" else 2
        hit = min(E, R) if R < 4 * E else E
        return {"bytes": (R + hit * N) * _ld(K) + 4 * _blocks(K) * (R + hit * _blocks(N)) + R * N * out + 4 * (E + 1),
                "flops": 2 * R * N * K}
    T, k, N = case["T"], case["k"], case["N"]
    size = 4 if case["dtype"] == "fp32" else 2
    return {"bytes": T * k * N * size + 8 * T * k + T * N * size, "flops": 2 * T * k * N}


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------

def _device():
    return torch.device("cuda" if torch.cuda.is_available() else "cpu")


def _normal(g, shape, std=1.0):
    return torch.randn(shape, generator=g, device=g.device, dtype=torch.float32).mul_(std)


def _quantised(x, block_rows):
    """Codes (float8_e4m3fn, rows padded to 16 bytes) and block-major scales of fp32 x [rows, K]."""
    rows, K = x.shape
    nb, nr = _blocks(K), (rows + block_rows - 1) // block_rows
    full = torch.zeros(nr * block_rows, nb * BLOCK, device=x.device, dtype=torch.float32)
    full[:rows, :K] = x
    t = full.view(nr, block_rows, nb, BLOCK)
    s = (t.abs().amax(dim=(1, 3)) / E4M3_MAX).clamp_min_(SCALE_MIN)
    t = t * torch.reciprocal(s)[:, None, :, None]
    t = t.clamp_(-E4M3_MAX, E4M3_MAX).view(nr * block_rows, nb * BLOCK)
    return t[:rows, :_ld(K)].to(torch.float8_e4m3fn).contiguous(), s.t().contiguous()


def _activations(g, shape):
    """N(0, 1) with a scale of its own for each row and a few large channels, as hidden states have."""
    x = _normal(g, shape)
    x *= torch.exp(0.5 * _normal(g, (shape[0], 1)))
    x[:, :: 97] *= 8.0
    return x


def prepare(case, seed):
    dev = _device()
    g = torch.Generator(device=dev).manual_seed(int(seed))
    op = case["op"]
    s = {"case": case}
    if op == "route":
        T, E, k = case["T"], case["E"], case["k"]
        # a router's logits: some experts are liked by all tokens more than others
        s["logits"] = (_normal(g, (T, E), 1.5) + _normal(g, (1, E), 0.5)).to(DTYPES[case["dtype"]])
        s["bias"] = _normal(g, (E,), 0.05) if case["bias"] else None
        s["idx"] = torch.empty(T, k, dtype=torch.int32, device=dev)
        s["weights"] = torch.empty(T, k, dtype=torch.float32, device=dev)
        s["offsets"] = torch.empty(E + 1, dtype=torch.int32, device=dev)
        s["row_token"] = torch.empty(T * k, dtype=torch.int32, device=dev)
        s["slot_row"] = torch.empty(T, k, dtype=torch.int32, device=dev)
    elif op == "pack":
        rows, K = case["rows"], case["K"]
        x = _activations(g, (case["source"], K)) if case["block_rows"] == 1 else _normal(g, (rows, K), 0.02)
        s["x"] = x.to(DTYPES[case["dtype"]])
        s["row_index"] = None
        if case["source"] != rows:                        # the source row of each packed row
            s["row_index"] = torch.randint(0, case["source"], (rows,), generator=g, device=dev, dtype=torch.int32)
        nr = (rows + case["block_rows"] - 1) // case["block_rows"]
        s["codes"] = torch.empty(rows, _ld(K), dtype=torch.float8_e4m3fn, device=dev)
        s["scales"] = torch.empty(_blocks(K), nr, dtype=torch.float32, device=dev)
    elif op == "gemm":
        M, N, K = case["M"], case["N"], case["K"]
        s["A"], s["a_scales"] = _quantised(_activations(g, (M, K)), 1)
        s["W"], s["w_scales"] = _quantised(_normal(g, (N, K), 0.02), BLOCK)
        s["out"] = torch.empty(M, N, dtype=DTYPES[case["out"]], device=dev)
    elif op == "experts":
        R, E, N, K = case["T"] * case["k"], case["E"], case["N"], case["K"]
        # uneven choice of experts: a popularity for each
        p = torch.softmax(0.5 * _normal(g, (E,)), dim=0)
        expert = torch.multinomial(p, R, replacement=True, generator=g)
        count = (expert[:, None] == torch.arange(E, device=dev)[None, :]).sum(0)
        s["offsets"] = torch.cat([count.new_zeros(1), count.cumsum(0)]).to(torch.int32)
        s["A"], s["a_scales"] = _quantised(_activations(g, (R, K)), 1)
        s["W"] = torch.empty(E, N, _ld(K), dtype=torch.float8_e4m3fn, device=dev)
        s["w_scales"] = torch.empty(E, _blocks(K), _blocks(N), dtype=torch.float32, device=dev)
        for e in range(E):
            s["W"][e], s["w_scales"][e] = _quantised(_normal(g, (N, K), 0.02), BLOCK)
        s["out"] = torch.empty(R, N, dtype=DTYPES[case["out"]], device=dev)
    else:
        T, k, N = case["T"], case["k"], case["N"]
        s["Y"] = _normal(g, (T * k, N)).to(DTYPES[case["dtype"]])
        s["slot_row"] = torch.randperm(T * k, generator=g, device=dev).to(torch.int32).view(T, k)
        s["weights"] = torch.softmax(_normal(g, (T, k)), dim=1)
        s["out"] = torch.empty(T, N, dtype=DTYPES[case["dtype"]], device=dev)
    return s


# --------------------------------------------------------------------------
# plain forms
# --------------------------------------------------------------------------

def _plain_route(s):
    """Scores and choices in 64 bits (neighbouring scores can be nearer than 32 bits tell apart), ties to the lowest index."""
    c = s["case"]
    T, E, k, G = c["T"], c["E"], c["k"], c["groups"]
    l = s["logits"].double()
    if c["score"] == "sigmoid":
        score = 1.0 / (1.0 + torch.exp(-l))
    else:
        e = torch.exp(l - l.amax(dim=1, keepdim=True))
        score = e / e.sum(dim=1, keepdim=True)
    choice = score if s["bias"] is None else score + s["bias"].double()
    if G > 1:
        top2 = torch.sort(choice.view(T, G, E // G), dim=2, descending=True).values[:, :, :2].sum(dim=2)
        order = torch.sort(top2, dim=1, descending=True, stable=True).indices
        keep = torch.zeros(T, G, dtype=torch.bool, device=l.device).scatter_(1, order[:, :c["kept"]], True)
        choice = torch.where(keep.repeat_interleave(E // G, dim=1), choice, torch.full_like(choice, -math.inf))
    idx = torch.sort(choice, dim=1, descending=True, stable=True).indices[:, :k]
    w = torch.gather(score, 1, idx)
    w = w / w.sum(dim=1, keepdim=True)
    flat = idx.reshape(-1)
    order = torch.sort(flat, stable=True).indices
    count = torch.zeros(E, dtype=torch.int64, device=l.device).index_add_(0, flat, torch.ones_like(flat))
    offsets = torch.cat([count.new_zeros(1), count.cumsum(0)])
    slot_row = torch.empty_like(flat)
    slot_row[order] = torch.arange(T * k, device=l.device)
    i32 = torch.int32
    return {"idx": idx.to(i32), "weights": w.float(), "offsets": offsets.to(i32),
            "row_token": (order // k).to(i32), "slot_row": slot_row.view(T, k).to(i32)}


def _plain_pack(s):
    c = s["case"]
    x = s["x"].float()
    if s["row_index"] is not None:
        x = x[s["row_index"].long()]
    codes, scales = _quantised(x, c["block_rows"])
    return {"codes": codes, "scales": scales}


def _values(codes, scales, K, block_rows):
    """fp32 values of codes [..., rows, ld] with block-major scales [..., blocks of K, row blocks]."""
    rows = codes.shape[-2]
    v = codes[..., :K].float()
    f = scales.transpose(-1, -2)
    if block_rows > 1:
        f = f.repeat_interleave(block_rows, dim=-2)[..., :rows, :]
    return v * f.repeat_interleave(BLOCK, dim=-1)[..., :K]


def _plain_gemm(s):
    K = s["case"]["K"]
    a = _values(s["A"], s["a_scales"], K, 1)
    w = _values(s["W"], s["w_scales"], K, BLOCK)
    return (a @ w.t()).to(s["out"].dtype)


def _plain_experts(s):
    c = s["case"]
    R, E, K = c["T"] * c["k"], c["E"], c["K"]
    a = _values(s["A"], s["a_scales"], K, 1)
    w = _values(s["W"], s["w_scales"], K, BLOCK)
    offsets = s["offsets"].long()
    row = torch.arange(R, device=a.device)
    expert = (row[:, None] >= offsets[None, 1:]).sum(dim=1)
    place = row - offsets[expert]
    most = int((offsets[1:] - offsets[:-1]).max())
    padded = torch.zeros(E, most, K, device=a.device)
    padded[expert, place] = a
    y = padded @ w.transpose(1, 2)
    return y[expert, place].to(s["out"].dtype)


def _plain_combine(s):
    y = s["Y"][s["slot_row"].long()].float()
    return (s["weights"][:, :, None] * y).sum(dim=1).to(s["out"].dtype)


# --------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------

def run(s):
    c = s["case"]
    op = c["op"]
    if own:
        import xnor_popcount_gemm_bnn_b200 as bnn
        if op == "route":
            bnn.bnn_route(s["logits"], s["idx"], s["weights"],
                          score=bnn.BNN_ROUTE_SIGMOID if c["score"] == "sigmoid" else bnn.BNN_ROUTE_SOFTMAX,
                          bias=s["bias"], n_groups=c["groups"], kept_groups=c["kept"], renormalize=True,
                          offsets=s["offsets"], row_token=s["row_token"], slot_row=s["slot_row"])
            return {n: s[n] for n in ("idx", "weights", "offsets", "row_token", "slot_row")}
        if op == "pack":
            bnn.bnn_fp8_pack(s["x"], s["codes"], s["scales"], block_rows=c["block_rows"], row_index=s["row_index"])
            return {"codes": s["codes"], "scales": s["scales"]}
        if op == "gemm":
            bnn.bnn_fp8_gemm(s["A"], s["a_scales"], s["W"], s["w_scales"], c["K"], s["out"])
        elif op == "experts":
            bnn.bnn_fp8_gemm_grouped(s["A"], s["a_scales"], s["offsets"], s["W"], s["w_scales"], c["K"], s["out"])
        else:
            bnn.bnn_route_combine(s["Y"], s["slot_row"], s["weights"], s["out"])
        return s["out"]
    return {"route": _plain_route, "pack": _plain_pack, "gemm": _plain_gemm, "experts": _plain_experts,
            "combine": _plain_combine}[op](s)


# --------------------------------------------------------------------------
# the definitions in 64 bits
# --------------------------------------------------------------------------

def _wide(codes, scales, K, block_rows):
    """float64 values, every element with the scale of its own block."""
    rows = codes.shape[0]
    i = torch.arange(rows, device=codes.device) // block_rows
    b = torch.arange(K, device=codes.device) // BLOCK
    return codes[:, :K].to(torch.float64) * scales.double()[b[None, :], i[:, None]]


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "route":
        # the chosen experts' weights, found anew: the k largest of the experts of the kept groups
        T, E, G = case["T"], case["E"], case["groups"]
        l = s["logits"].to(torch.float64)
        score = torch.sigmoid(l) if case["score"] == "sigmoid" else torch.softmax(l, dim=1)
        choice = score.clone() if s["bias"] is None else score + s["bias"].to(torch.float64)
        if G > 1:
            by_group = choice.view(T, G, E // G)
            kept = by_group.topk(2, dim=2).values.sum(dim=2).topk(case["kept"], dim=1).indices
            out = torch.ones(T, G, dtype=torch.bool, device=l.device)
            out[torch.arange(T, device=l.device)[:, None], kept] = False
            by_group[out] = -math.inf
        w = torch.gather(score, 1, choice.topk(case["k"], dim=1).indices)
        return {"idx": None, "weights": w / w.sum(dim=1, keepdim=True), "offsets": None, "row_token": None,
                "slot_row": None}
    if op == "pack":
        x = s["x"].double()
        if s["row_index"] is not None:
            x = torch.index_select(x, 0, s["row_index"].long())
        rows, K = x.shape
        br = case["block_rows"]
        scales = torch.empty(s["scales"].shape, dtype=torch.float64, device=x.device)
        codes = torch.zeros(s["codes"].shape, dtype=torch.float64, device=x.device)
        nr = scales.shape[1]
        for b in range(scales.shape[0]):
            part = x[:, b * BLOCK:(b + 1) * BLOCK]
            top = torch.zeros(nr * br, dtype=torch.float64, device=x.device)
            top[:rows] = part.abs().max(dim=1).values
            scales[b] = (top.view(nr, br).max(dim=1).values / E4M3_MAX).clamp_min(SCALE_MIN)
            # to the nearest e4m3 value: steps of 2^(exponent - 3), not below 2^-9, ties to even
            q = part / scales[b].repeat_interleave(br)[:rows, None]
            step = torch.exp2(torch.floor(torch.log2(q.abs().clamp_min(2.0 ** -6))) - 3.0)
            codes[:, b * BLOCK:b * BLOCK + part.shape[1]] = torch.round(q / step) * step
        return {"codes": codes, "scales": scales}
    if op == "gemm":
        K = case["K"]
        return torch.mm(_wide(s["A"], s["a_scales"], K, 1), _wide(s["W"], s["w_scales"], K, BLOCK).t())
    if op == "experts":
        K, off = case["K"], s["offsets"].tolist()
        y = torch.zeros(s["out"].shape, dtype=torch.float64, device=s["out"].device)
        a = _wide(s["A"], s["a_scales"], K, 1)
        for e in range(case["E"]):
            if off[e + 1] > off[e]:
                y[off[e]:off[e + 1]] = torch.mm(a[off[e]:off[e + 1]], _wide(s["W"][e], s["w_scales"][e], K, BLOCK).t())
        return y
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device=s["out"].device)
    for j in range(case["k"]):
        out += s["weights"][:, j:j + 1].double() * s["Y"].double()[s["slot_row"][:, j].long()]
    return out
