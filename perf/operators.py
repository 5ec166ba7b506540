"""Routing from logits, MXFP4 quantisation, MXFP4 expert products and the weighted combine: the
cases that are measured, their plain forms in elementary torch operations, and their values in
64 bits.

A case's "op" names the operator:
  route     logits -> top-k experts, weights and the token -> expert permutation
  quantize  rows -> MXFP4 (E2M1 codes, one E8M0 scale per 32 inputs) -> the values they stand for
  product   MXFP4 rows, grouped by expert, times the experts' MXFP4 matrices
  combine   the weighted sum of each token's expert rows

MXFP4: element 2i of a row is the low nibble of code byte i; a code is a sign bit and the index of
one of 0, 0.5, 1, 1.5, 2, 3, 4, 6; the scale byte s of a block of 32 stands for 2^(s - 127).
"""
import math

import torch

own = False

MAGNITUDES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
DTYPES = {"float32": torch.float32, "bfloat16": torch.bfloat16, "float16": torch.float16}
SIZES = {"float32": 4, "bfloat16": 2, "float16": 2}
SCORES = ("softmax", "sigmoid", "sqrt_softplus")
FLOAT_MAX = torch.finfo(torch.float32).max


# ----------------------------------------------------------------------------- the cases

def listed():
    return [
        # one generated token of a 256-expert layer: eight groups, four kept, bias for balance
        dict(name="route_t1_groups", op="route", tokens=1, experts=256, top_k=8, score="sigmoid", dtype="float32",
             bias=True, groups=8, topk_groups=4, group_score="top2", renormalise=True, scale=2.5, masked=False),
        # a prompt chunk: softmax scores from a bf16 router product, no bias, no groups
        dict(name="route_t2048_softmax", op="route", tokens=2048, experts=256, top_k=8, score="softmax",
             dtype="bfloat16", bias=False, groups=1, topk_groups=1, group_score="max", renormalise=True, scale=1.0,
             masked=False),
        # the longest call a handle takes, the framework's own score with a bias on the choice alone
        dict(name="route_t65536_bias", op="route", tokens=65536, experts=256, top_k=8, score="sqrt_softplus",
             dtype="float32", bias=True, groups=1, topk_groups=1, group_score="max", renormalise=True, scale=1.0,
             masked=False),
        # activations of 16 concurrent sessions, before the gate and up products
        dict(name="quantize_t16", op="quantize", tokens=16, width=4096, dtype="bfloat16", top_k=0, experts=0),
        # a prompt chunk's activations, written once per chosen expert in the experts' order
        dict(name="quantize_t2048_pairs", op="quantize", tokens=2048, width=4096, dtype="bfloat16", top_k=8,
             experts=256),
        # single-token decode: gate and up of the eight chosen experts, bound by their weights' bytes
        dict(name="gated_t1", op="product", experts=256, rows=8, out=2048, width=4096, gated=True, dtype="bfloat16",
             load="one_each"),
        # 16 sessions: the down product of about a hundred experts with one or two rows each
        dict(name="down_t16", op="product", experts=256, rows=128, out=4096, width=2048, gated=False,
             dtype="bfloat16", load="even"),
        # a 2048-token prompt chunk with uneven loads, its h left in MXFP4 for the down product
        dict(name="gated_t2048", op="product", experts=256, rows=16384, out=2048, width=4096, gated=True,
             dtype="mxfp4", load="uneven"),
        # an 8192-token chunk of the wide layer
        dict(name="down_t8192_wide", op="product", experts=256, rows=65536, out=7168, width=2048, gated=False,
             dtype="bfloat16", load="even"),
        # one matrix for every token (a shared expert), where the products themselves count
        dict(name="dense_t8191", op="product", experts=1, rows=8191, out=4096, width=4096, gated=False,
             dtype="float32", load="even"),
        # one generated token: eight rows and the shared expert's
        dict(name="combine_t1", op="combine", tokens=1, width=4096, top_k=8, dtype="bfloat16", out="float32", add=True),
        # the 8192-token chunk of the wide layer
        dict(name="combine_t8192_wide", op="combine", tokens=8192, width=7168, top_k=8, dtype="bfloat16",
             out="float32", add=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("route", "quantize", "product", "product", "combine"))
    if op == "route":
        groups = rng.choice((1, 1, 4, 8))
        experts = groups * rng.randint(max(2, -(-16 // groups)), 256 // groups)
        return dict(op=op, tokens=_log_int(rng, 1, 65536), experts=experts, top_k=rng.randint(1, 8),
                    score=rng.choice(SCORES), dtype=rng.choice(tuple(DTYPES)), bias=rng.random() < 0.5, groups=groups,
                    topk_groups=rng.randint(-(-groups // 2), groups), group_score=rng.choice(("max", "top2")),
                    renormalise=rng.random() < 0.7, scale=rng.choice((1.0, 2.5)), masked=rng.random() < 0.3)
    if op == "quantize":
        pairs = rng.random() < 0.5
        return dict(op=op, tokens=_log_int(rng, 1, 2048), width=32 * rng.randint(1, 224),
                    dtype=rng.choice(tuple(DTYPES)), top_k=rng.randint(1, 8) if pairs else 0,
                    experts=rng.randint(8, 256) if pairs else 0)
    if op == "product":
        experts = _log_int(rng, 1, 64)
        gated = rng.random() < 0.5
        out = 32 * rng.randint(8, 128) if gated else rng.randint(200, 4096)
        return dict(op=op, experts=experts, rows=_log_int(rng, 1, 8192), out=out, width=32 * rng.randint(8, 128),
                    gated=gated, dtype=rng.choice(tuple(DTYPES) + (("mxfp4",) if gated else ())),
                    load=rng.choice(("even", "uneven")))
    return dict(op=op, tokens=_log_int(rng, 1, 8192), width=rng.randint(256, 7168), top_k=rng.randint(1, 8),
                dtype=rng.choice(tuple(DTYPES)), out=rng.choice(tuple(DTYPES)), add=rng.random() < 0.5)


def work(case):
    c = case
    if c["op"] == "route":
        T, E, k = c["tokens"], c["experts"], c["top_k"]
        return {"bytes": T * E * SIZES[c["dtype"]] + (4 * E if c["bias"] else 0) + 20 * T * k + 4 * (E + 1),
                "flops": 20 * T * E}
    if c["op"] == "quantize":
        n = c["tokens"] * c["width"]
        m = n * max(1, c["top_k"])
        return {"bytes": n * SIZES[c["dtype"]] + 2 * (m * 17 // 32) + 2 * m, "flops": 4 * n + m}
    if c["op"] == "product":
        mats = 2 if c["gated"] else 1
        R, N, K = c["rows"], c["out"], c["width"]
        # the experts that a spread of R rows reaches, on average
        reached = min(R, c["experts"]) if c["load"] == "one_each" else c["experts"] * -math.expm1(-R / c["experts"])
        held = R * N * (17 / 32) * 2 + R * N * 2 if c["dtype"] == "mxfp4" else R * N * SIZES[c["dtype"]]
        return {"bytes": int((reached * mats * N * K + R * K) * 17 / 32 + held), "flops": 2 * mats * R * N * K}
    T, H, k = c["tokens"], c["width"], c["top_k"]
    return {"bytes": T * k * H * SIZES[c["dtype"]] + T * H * SIZES[c["out"]] + (4 * T * H if c["add"] else 0) + 8 * T * k,
            "flops": 2 * T * k * H}


# ----------------------------------------------------------------------------- inputs

def _encode(x):
    """MXFP4 codes and scales of float32 rows [..., K] (inputs of the product cases)."""
    b = x.reshape(*x.shape[:-1], -1, 32)
    e = (torch.frexp(b.abs().amax(-1))[1] - 3).clamp(-127, 125)
    a = torch.ldexp(b.abs(), -e[..., None])
    code = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0)
            + 8 * (b < 0)).reshape(*x.shape[:-1], -1)
    return (code[..., 0::2] | (code[..., 1::2] << 4)).to(torch.uint8), (e + 127).to(torch.uint8)


def _weights(E, N, K, gen):
    """Codes [E, N, K/2] and scales [E, N, K/32] of N(0, 0.02) matrices."""
    codes = torch.empty(E, N, K // 2, dtype=torch.uint8, device="cuda")
    scales = torch.empty(E, N, K // 32, dtype=torch.uint8, device="cuda")
    step = max(1, (1 << 28) // (N * K))
    for e in range(0, E, step):
        n = min(step, E - e)
        codes[e:e + n], scales[e:e + n] = _encode(torch.randn(n, N, K, generator=gen, device="cuda") * 0.02)
    return codes, scales


def _chosen(T, E, k, gen, spread):
    """k different experts for each of T tokens, some experts likelier than others."""
    lean = torch.randn(E, generator=gen, device="cuda") * spread
    noise = -torch.log(-torch.log(torch.rand(T, E, generator=gen, device="cuda").clamp(1e-7, 1 - 1e-7)))
    return (lean + noise).topk(k, dim=1).indices


def _places(chosen, E):
    """offsets [E + 1] and inv_pos [T, k] of the (token, slot) pairs ordered by expert, then token."""
    e = chosen.reshape(-1)
    order = torch.argsort(e, stable=True)
    inv = torch.empty_like(order)
    inv[order] = torch.arange(len(order), device=order.device)
    offsets = torch.zeros(E + 1, dtype=torch.int64, device=order.device)
    offsets[1:] = torch.cumsum(torch.bincount(e, minlength=E), 0)
    return offsets, inv.reshape(chosen.shape)


def _loads(case, gen):
    E, R = case["experts"], case["rows"]
    if case["load"] == "one_each":
        e = torch.randperm(E, generator=gen, device="cuda")[:R]
    else:
        e = _chosen(R, E, 1, gen, 0.5 if case["load"] == "uneven" else 0.0).reshape(-1)
    counts = torch.bincount(e, minlength=E)
    offsets = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    offsets[1:] = torch.cumsum(counts, 0).int()
    return offsets, int(counts.max())


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    s = dict(case)
    if case["op"] == "route":
        T, E, k = case["tokens"], case["experts"], case["top_k"]
        logits = torch.randn(T, E, generator=gen, device="cuda") * 1.5
        if case["masked"]:   # experts that are switched off for a token; k stay at least
            off = torch.rand(T, E, generator=gen, device="cuda") < 0.1
            off.view(T, case["groups"], -1)[:, :, :min(k, E // case["groups"])] = False
            logits = logits.masked_fill(off, -math.inf)
        s["logits"] = logits.to(DTYPES[case["dtype"]])
        s["lean"] = torch.randn(E, generator=gen, device="cuda") * 0.05 if case["bias"] else None
        if own:
            import bit_quantized_routed_sqrt_b200 as ds4
            s["router"] = ds4.Router(E, k, score=case["score"], n_groups=case["groups"],
                                     topk_groups=case["topk_groups"], group_score=case["group_score"],
                                     renormalise=case["renormalise"], scale=case["scale"])
            s["buffers"] = s["router"].buffers(T, device="cuda")
    elif case["op"] == "quantize":
        T, K, k = case["tokens"], case["width"], case["top_k"]
        s["x"] = torch.randn(T, K, generator=gen, device="cuda").to(DTYPES[case["dtype"]])
        s["rows"] = T * max(1, k)
        s["inv_pos"] = None
        if k:
            s["inv_pos"] = _places(_chosen(T, case["experts"], k, gen, 0.5), case["experts"])[1].int().contiguous()
        s["codes"] = torch.empty(s["rows"], K // 2, dtype=torch.uint8, device="cuda")
        s["scales"] = torch.empty(s["rows"], K // 32, dtype=torch.uint8, device="cuda")
        s["values"] = torch.empty(s["rows"], K, dtype=torch.bfloat16, device="cuda")
    elif case["op"] == "product":
        E, R, N, K = (case[n] for n in ("experts", "rows", "out", "width"))
        s["offsets"], s["most"] = _loads(case, gen)
        s["codes"], s["scales"] = _encode(torch.randn(R, K, generator=gen, device="cuda"))
        s["weights"] = [_weights(E, N, K, gen) for _ in range(2 if case["gated"] else 1)]
        if own:
            import bit_quantized_routed_sqrt_b200 as ds4
            s["matrix"] = ds4.Mxfp4Experts(E, N, K, gated=case["gated"])
            s["matrix"].load(*(t for pair in s["weights"] for t in pair))
            if case["dtype"] == "mxfp4":
                s["h"] = torch.empty(R, N // 2, dtype=torch.uint8, device="cuda")
                s["h_scales"] = torch.empty(R, N // 32, dtype=torch.uint8, device="cuda")
            s["result"] = torch.empty(R, N, dtype=DTYPES.get(case["dtype"], torch.bfloat16), device="cuda")
    else:
        T, H, k = case["tokens"], case["width"], case["top_k"]
        s["o"] = torch.randn(T * k, H, generator=gen, device="cuda").to(DTYPES[case["dtype"]])
        s["inv_pos"] = torch.randperm(T * k, generator=gen, device="cuda").int().reshape(T, k)
        w = torch.rand(T, k, generator=gen, device="cuda") + 0.1
        s["weight"] = w / w.sum(1, keepdim=True)
        s["shared"] = torch.randn(T, H, generator=gen, device="cuda") if case["add"] else None
        s["y"] = torch.empty(T, H, dtype=DTYPES[case["out"]], device="cuda")
    return s


# ----------------------------------------------------------------------------- the plain forms

def _route_plain(s):
    T, E, k, G = s["tokens"], s["experts"], s["top_k"], s["groups"]
    logit = s["logits"].double().clamp(max=FLOAT_MAX)   # borders between experts: 64 bits
    live = logit > -math.inf
    if s["score"] == "softmax":
        e = torch.exp(logit - logit.amax(1, keepdim=True))
        score = e / e.sum(1, keepdim=True)
    elif s["score"] == "sigmoid":
        score = 1.0 / (1.0 + torch.exp(-logit))
    else:
        score = torch.sqrt(logit.clamp(min=0.0) + torch.log1p(torch.exp(-logit.abs())))
    choice = logit if s["lean"] is None else score + s["lean"].double()
    choice = torch.where(live, choice, -math.inf)
    if G > 1:
        if s["group_score"] == "max":
            of_group = choice.view(T, G, -1).amax(2)
        else:
            c = score if s["lean"] is None else score + s["lean"].double()
            two = torch.where(live, c, -math.inf).view(T, G, -1).topk(2, dim=2).values
            of_group = two[..., 0] + torch.where(two[..., 1] > -math.inf, two[..., 1], 0.0)
        kept = torch.sort(of_group, dim=1, descending=True, stable=True).indices[:, :s["topk_groups"]]
        keep = torch.zeros(T, G, dtype=torch.bool, device=logit.device).scatter_(1, kept, True)
        choice = torch.where(keep.repeat_interleave(E // G, 1), choice, -math.inf)
    idx = torch.sort(choice, dim=1, descending=True, stable=True).indices[:, :k]
    w = score.gather(1, idx)
    if s["renormalise"]:
        w = w / w.sum(1, keepdim=True)
    offsets, inv = _places(idx, E)
    order = torch.empty(T * k, dtype=torch.int64, device=idx.device)
    order[inv.reshape(-1)] = torch.arange(T * k, device=idx.device)
    return {"idx": idx.int(), "weight": (w * s["scale"]).float(), "offsets": offsets.int(),
            "sorted_token": (order // k).int(), "sorted_slot": (order % k).int(), "inv_pos": inv.int().reshape(-1)}


def _values(codes, scales):
    """float32 values of MXFP4 rows."""
    one = torch.tensor(MAGNITUDES + tuple(-m for m in MAGNITUDES), device=codes.device)
    pair = torch.stack((one.repeat(16), one.repeat_interleave(16)), 1)   # of each code byte: low, high nibble
    v = pair[codes.int()].reshape(*scales.shape, 32)
    return (v * torch.exp2(scales.float() - 127.0)[..., None]).reshape(*codes.shape[:-1], -1)


def _quantize_plain(s):
    x = s["x"].float()
    b = x.reshape(x.shape[0], -1, 32)
    e = (torch.frexp(b.abs().amax(-1, keepdim=True))[1] - 3).clamp(-127, 125)
    a = torch.ldexp(b.abs(), -e)
    ladder = torch.tensor(MAGNITUDES, device=x.device)
    near = ladder[(a > 0.25).int() + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0)]
    v = torch.ldexp(torch.where(b < 0, -near, near), e).reshape(x.shape).bfloat16()
    if s["inv_pos"] is None:
        return v
    out = torch.empty(s["rows"], x.shape[1], dtype=v.dtype, device=v.device)
    out[s["inv_pos"].reshape(-1)] = v.repeat_interleave(s["top_k"], 0)
    return out


def _product_plain(s):
    a = _values(s["codes"], s["scales"])
    R, K = a.shape
    offsets = s["offsets"].long()
    expert = torch.bucketize(torch.arange(R, device=a.device), offsets[1:], right=True)
    if R <= 16:   # few rows: each with its own expert's matrix
        products = [torch.bmm(_values(c[expert], e[expert]), a[:, :, None])[..., 0] for c, e in s["weights"]]
    else:         # every expert's rows, filled up to the longest group
        place = torch.arange(R, device=a.device) - offsets[expert]
        filled = torch.zeros(s["experts"], s["most"], K, device=a.device)
        filled[expert, place] = a
        products = [torch.bmm(filled, _values(c, e).transpose(1, 2))[expert, place] for c, e in s["weights"]]
    if not s["gated"]:
        return products[0].to(DTYPES[s["dtype"]])
    g, u = products
    h = g / (1.0 + torch.exp(-g)) * u
    if s["dtype"] == "mxfp4":
        return _quantize_plain({"x": h, "inv_pos": None})
    return h.to(DTYPES[s["dtype"]])


def _combine_plain(s):
    rows = s["o"].float()[s["inv_pos"].reshape(-1).long()].reshape(*s["weight"].shape, -1)
    y = (rows * s["weight"][..., None]).sum(1)
    if s["shared"] is not None:
        y = y + s["shared"]
    return y.to(s["y"].dtype)


# ----------------------------------------------------------------------------- one pass

def run(state):
    s = state
    if not own:
        return {"route": _route_plain, "quantize": _quantize_plain, "product": _product_plain,
                "combine": _combine_plain}[s["op"]](s)
    import bit_quantized_routed_sqrt_b200 as ds4
    if s["op"] == "route":
        b = s["buffers"]
        s["router"].route(s["logits"], s["lean"], b)
        return {"idx": b.topk_idx, "weight": b.topk_w, "offsets": b.expert_offsets, "sorted_token": b.sorted_token,
                "sorted_slot": b.sorted_slot, "inv_pos": b.inv_pos}
    if s["op"] == "quantize":
        ds4.mxfp4_quantize(s["x"], s["inv_pos"], s["codes"], s["scales"])
        return ds4.mxfp4_dequantize(s["codes"], s["scales"], s["values"])
    if s["op"] == "product":
        if s["dtype"] == "mxfp4":
            s["matrix"].product(s["codes"], s["scales"], s["offsets"], s["h"], s["h_scales"])
            return ds4.mxfp4_dequantize(s["h"], s["h_scales"], s["result"])
        return s["matrix"].product(s["codes"], s["scales"], s["offsets"], s["result"])
    return ds4.combine(s["o"], s["inv_pos"], s["weight"], s["y"], s["shared"])


# ----------------------------------------------------------------------------- in 64 bits

def _decode64(codes, scales):
    c = torch.stack((codes & 15, codes >> 4), -1).reshape(*codes.shape[:-1], -1).long()
    m, e = c & 1, (c >> 1) & 3   # E2M1: one mantissa bit, two exponent bits of bias 1
    size = torch.where(e == 0, 0.5 * m, torch.ldexp(1.0 + 0.5 * m.double(), e - 1))
    value = torch.where(c >= 8, -size, size).double()
    return value * torch.ldexp(torch.ones_like(scales, dtype=torch.float64),
                               scales.long() - 127).repeat_interleave(32, -1)


def _e2m1_64(x):
    """The MXFP4 value next to each input, in float64: the nearest multiple of the step at its size."""
    b = x.double().reshape(*x.shape[:-1], -1, 32)
    top = b.abs().amax(-1, keepdim=True)
    shared = torch.where(top > 0, torch.frexp(top)[1] - 3, -127).clamp(-127, 125)
    a = torch.ldexp(b, -shared)
    step = torch.where(a.abs() < 2.0, 0.5, torch.where(a.abs() < 4.0, 1.0, 2.0))
    q = (torch.round(a / step) * step).clamp(-6.0, 6.0)   # round() takes ties to the even multiple
    return torch.ldexp(q, shared).reshape(x.shape)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "route":
        x = s["logits"].double().clamp(max=FLOAT_MAX)
        lg = torch.where(x > -math.inf, x, -1e30)
        if case["score"] == "softmax":
            score = torch.softmax(lg, 1)
        elif case["score"] == "sigmoid":
            score = torch.sigmoid(lg)
        else:
            score = torch.sqrt(torch.logaddexp(lg, torch.zeros_like(lg)))
        rank = lg.clone() if s["lean"] is None else score + s["lean"].double()
        rank[x == -math.inf] = -1e30
        G, E, k = case["groups"], case["experts"], case["top_k"]
        if G > 1:
            if case["group_score"] == "max":
                best = rank.reshape(-1, G, E // G).max(2).values
            else:
                both = score if s["lean"] is None else score + s["lean"].double()
                both = both.masked_fill(x == -math.inf, -1e30).reshape(-1, G, E // G).sort(2, descending=True).values
                best = both[..., 0] + both[..., 1].masked_fill(both[..., 1] < -1e29, 0.0)
            # a group is kept where fewer than topk_groups are above it (an equal one of a lower index counts)
            i = torch.arange(G, device=best.device)
            above = (best[:, None, :] > best[:, :, None]) | ((best[:, None, :] == best[:, :, None]) & (i[None, :] < i[:, None]))
            drop = above.sum(2) >= case["topk_groups"]
            rank = rank.masked_fill(drop.repeat_interleave(E // G, 1), -1e31)
        idx = torch.empty(x.shape[0], k, dtype=torch.long, device=x.device)
        for j in range(k):
            m = rank.max(1, keepdim=True).values
            idx[:, j] = (rank == m).int().argmax(1)
            rank.scatter_(1, idx[:, j:j + 1], -1e32)
        w = score.gather(1, idx)
        if case["renormalise"]:
            w = w / w.sum(1, keepdim=True)
        return {"idx": None, "weight": w * case["scale"], "offsets": None, "sorted_token": None, "sorted_slot": None,
                "inv_pos": None}
    if case["op"] == "quantize":
        v = _e2m1_64(s["x"])
        if s["inv_pos"] is None:
            return v
        token = torch.empty(s["rows"], dtype=torch.long, device=v.device)
        flat = s["inv_pos"].reshape(-1).long()
        token[flat] = torch.arange(s["rows"], device=v.device) // case["top_k"]
        return v[token]
    if case["op"] == "product":
        a = _decode64(s["codes"], s["scales"])
        ends = s["offsets"].tolist()
        parts = [torch.empty(case["rows"], case["out"], dtype=torch.float64, device=a.device) for _ in s["weights"]]
        for e in range(case["experts"]):
            if ends[e + 1] > ends[e]:
                for p, (c, sc) in zip(parts, s["weights"]):
                    p[ends[e]:ends[e + 1]] = a[ends[e]:ends[e + 1]] @ _decode64(c[e], sc[e]).T
        if not case["gated"]:
            return parts[0]
        h = parts[0] * torch.sigmoid(parts[0]) * parts[1]
        return _e2m1_64(h) if case["dtype"] == "mxfp4" else h
    y = s["shared"].double() if case["add"] else torch.zeros(case["tokens"], case["width"], dtype=torch.float64, device="cuda")
    for j in range(case["top_k"]):
        y = y + s["weight"][:, j, None].double() * s["o"].double()[s["inv_pos"][:, j].long()]
    return y
