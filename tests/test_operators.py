"""The operators beside the layer on the GPU, through the public binding, against plain float64 forms:
routing from logits, MXFP4 quantisation and products, the combine, and a run of them together."""
import numpy as np
import pytest

import operator_refs as ref

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


@pytest.fixture(scope="module")
def ds4():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build_library()
    import bit_quantized_routed_sqrt_b200 as m
    return m


def gen(seed):
    return torch.Generator().manual_seed(seed)


# ------------------------------------------------------------------ routing from logits
# Weights: expf, log1pf, the square root and the quotients cost at most two steps each, a sum of up to 32
# scores by halves five roundings, the scale one: 16 half steps of float32 in all.
W_RTOL = 16 * ref.U24


def check_route(ds4, logits, k, bias=None, out=None, **kw):
    E = logits.shape[1]
    r = ds4.Router(E, k, **kw)
    got = r.route(logits.cuda() if not logits.is_cuda else logits, None if bias is None else bias.cuda(), out)
    torch.cuda.synchronize()
    idx, w = ref.route(logits.cpu(), k, kw.get("score", "softmax"), bias, kw.get("n_groups", 1), kw.get("topk_groups", 1),
                       kw.get("group_score", "max"), kw.get("renormalise", True), kw.get("scale", 1.0))
    g = got.topk_idx.cpu().numpy()
    assert np.array_equal(g, idx), np.argwhere(g != idx)[:4]
    np.testing.assert_allclose(got.topk_w.cpu().numpy(), w, rtol=W_RTOL, atol=1e-37)
    off, st, ss, inv = ref.permute(idx, E)
    n = off[-1]
    assert np.array_equal(got.expert_offsets.cpu().numpy(), off)
    assert np.array_equal(got.sorted_token.cpu().numpy()[:n], st)
    assert np.array_equal(got.sorted_slot.cpu().numpy()[:n], ss)
    assert np.array_equal(got.inv_pos.cpu().numpy(), inv)
    return got


@pytest.mark.parametrize("T", [1, 2, 63, 64, 65, 300])
@pytest.mark.parametrize("score", ["softmax", "sigmoid", "sqrt_softplus"])
@pytest.mark.parametrize("biased", [False, True])
def test_route_lengths(ds4, T, score, biased):
    g = gen(T)
    logits = torch.randn(T, 96, generator=g) * 2
    bias = torch.randn(96, generator=g) * 0.1 if biased else None
    check_route(ds4, logits, 6, bias, score=score, renormalise=T % 2 == 0, scale=1.5)


@pytest.mark.parametrize("E,k", [(1, 1), (2, 2), (5, 3), (31, 4), (32, 32), (33, 8), (64, 1), (100, 7), (128, 16), (160, 6),
                                 (256, 8), (257, 8), (384, 8), (512, 32)])
@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
def test_route_expert_counts_and_types(ds4, E, k, kind):
    g = gen(E)
    logits = (torch.randn(70, E, generator=g) * 2).to(TYPES[kind])
    check_route(ds4, logits, k, score="softmax", renormalise=False)
    check_route(ds4, logits, k, torch.randn(E, generator=g) * 0.2, score="sigmoid")


@pytest.mark.parametrize("E,G,tg,k", [(256, 8, 4, 8), (160, 8, 3, 6), (64, 32, 5, 10), (12, 4, 2, 6), (512, 2, 1, 8),
                                      (6, 6, 3, 3), (96, 3, 3, 5), (256, 1, 1, 8), (512, 32, 32, 32)])
@pytest.mark.parametrize("group_score", ["max", "top2"])
@pytest.mark.parametrize("biased", [False, True])
def test_route_groups(ds4, E, G, tg, k, group_score, biased):
    g = gen(E + G)
    logits = torch.randn(67, E, generator=g)
    bias = torch.randn(E, generator=g) * 0.3 if biased else None
    for score in ("softmax", "sigmoid", "sqrt_softplus"):
        check_route(ds4, logits, k, bias, score=score, n_groups=G, topk_groups=tg, group_score=group_score)


@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("G", [1, 4])
def test_route_ties_go_to_the_lower_index(ds4, biased, G):
    logits = torch.randint(-2, 3, (130, 64), generator=gen(3)).float() * 0.5
    bias = torch.zeros(64) if biased else None
    for score in ("softmax", "sigmoid", "sqrt_softplus"):
        check_route(ds4, logits, 8, bias, score=score, n_groups=G, topk_groups=max(1, G // 2), group_score="top2")
    check_route(ds4, torch.zeros(3, 64), 8, bias, n_groups=G, topk_groups=max(1, G // 2))


@pytest.mark.parametrize("score", ["softmax", "sigmoid", "sqrt_softplus"])
def test_route_near_ties_are_ordered_in_64_bits(ds4, score):
    """Biases that cancel the scores' differences down to a few float32 steps of the sum: the order is that of
    float64 values (an order by float32 sums differs from it in most rows)."""
    g = gen(11)
    E = 64
    base = torch.randn(E, generator=g)
    s = ref.score64(score, base.double().numpy())
    bias = torch.from_numpy((1.0 - s).astype(np.float32))
    logits = base.repeat(40, 1)
    check_route(ds4, logits, 8, bias, score=score)
    check_route(ds4, logits, 8, bias, score=score, n_groups=8, topk_groups=3, group_score="top2")


@pytest.mark.parametrize("score", ["softmax", "sigmoid", "sqrt_softplus"])
@pytest.mark.parametrize("biased", [False, True])
def test_route_masked_and_extreme_logits(ds4, score, biased):
    g = gen(5)
    E, k = 40, 6
    logits = torch.randn(24, E, generator=g)
    inf, big = float("inf"), torch.finfo(torch.float32).max
    logits[0] = -inf                                   # nothing left
    logits[1] = float("nan")
    logits[2, :-1] = -inf                              # one expert
    logits[3, 4:] = -inf                               # fewer than k
    logits[4, ::2] = float("nan")
    logits[5, 7] = inf                                 # counts as the largest finite value
    logits[6, 3] = logits[6, 9] = inf
    logits[7] = -big                                   # the type's lowest value is a logit like others
    logits[8, :20] = -big
    logits[9, 1:] = -big
    logits[10] = -200.0 - torch.arange(E)              # scores that underflow in fp32
    logits[11] = -2000.0 + torch.arange(E) * 0.5       # and in fp64
    logits[12] = 200.0 + torch.arange(E)
    logits[13, 2] = big
    logits[14] = -1e-30 * torch.arange(E)
    bias = None
    if biased:
        bias = torch.randn(E, generator=g)
        bias[3], bias[5], bias[8] = -inf, float("nan"), inf
    check_route(ds4, logits, k, bias, score=score)
    check_route(ds4, logits, k, bias, score=score, n_groups=5, topk_groups=2, group_score="top2", renormalise=False)
    check_route(ds4, logits, k, bias, score=score, n_groups=5, topk_groups=2, group_score="max")


def test_route_strided_rows_and_untouched_places(ds4):
    wide = torch.randn(50, 80, generator=gen(8)).cuda()
    logits = wide[:, 3:43]
    assert not logits.is_contiguous()
    masked = logits.cpu().clone()
    masked[::3, 2:] = float("-inf")
    wide[:, 3:43] = masked.cuda()
    r = ds4.Router(40, 4)
    out = r.buffers(50)
    out.sorted_token.fill_(-7)
    out.sorted_slot.fill_(-7)
    check_route(ds4, wide[:, 3:43], 4, out=out)
    n = int(out.expert_offsets[-1])
    assert n < 200 and (out.sorted_token[n:] == -7).all() and (out.sorted_slot[n:] == -7).all()


@pytest.mark.parametrize("T", [4700, 6000, 16462, 40000])
def test_route_many_tokens(ds4, T):
    """Few and many blocks, counts added up by every block or scanned, blocks of 32 to 128 tokens: the last ragged."""
    logits = torch.randn(T, 24, generator=gen(9))
    check_route(ds4, logits, 3, torch.randn(24, generator=gen(1)) * 0.1, score="sigmoid")


def test_route_optional_outputs_and_no_tokens(ds4):
    r = ds4.Router(16, 2)
    logits = torch.randn(100, 16, generator=gen(2)).cuda()
    full = r.route(logits)
    idx, w = torch.full((100, 2), -5, dtype=torch.int32, device="cuda"), torch.zeros(100, 2, device="cuda")
    ds4.ds4moe_route_logits(r.cfg, logits, ds4.F32, 16, 100, None, idx, w)   # no permutation: no workspace
    inv = torch.full((200,), -5, dtype=torch.int32, device="cuda")
    ws = torch.empty(ds4.ds4moe_route_logits_workspace(r.cfg, 100), dtype=torch.uint8, device="cuda")
    ds4.ds4moe_route_logits(r.cfg, logits, ds4.F32, 16, 100, None, idx, w, None, None, None, inv, ws, ws.numel())
    torch.cuda.synchronize()
    assert torch.equal(idx, full.topk_idx) and torch.equal(w, full.topk_w) and torch.equal(inv, full.inv_pos)
    none = r.route(logits[:0])
    assert int(none.expert_offsets.abs().sum()) == 0


def test_route_agrees_with_the_layers_own_rule(ds4):
    """sqrt-softplus without a bias on given logits: the layer's choice and weights for the same logits."""
    import synth
    from gpu_common import layer_weights, make_layer, to_dev, tokens
    name = "decode_t16_h4096_e256_k8"
    w, lw, x = synth.workload(name), layer_weights(name), tokens(name)
    layer = make_layer(ds4, w)
    layer.load(lw)
    idx, wt, off, st, ss, inv = layer.route(to_dev(x))
    xs = torch.from_numpy(x.view(np.int16)).view(torch.bfloat16).double()
    wr = torch.from_numpy(np.ascontiguousarray(lw.router).view(np.int16)).view(torch.bfloat16).double()
    got = ds4.Router(w.n_experts, w.top_k, score="sqrt_softplus").route((xs @ wr.T.reshape(w.hidden, -1)).float().cuda())
    assert torch.equal(got.topk_idx, idx) and torch.equal(got.inv_pos, inv.reshape(-1)) and torch.equal(got.expert_offsets, off)
    torch.testing.assert_close(got.topk_w, wt, rtol=4e-6, atol=0)
    layer.close()


# ------------------------------------------------------------------ MXFP4 rows
def awkward(rows, K, seed, kind):
    """Rows with every border of the format: ties, powers of two, zeros, subnormals, large values."""
    g = gen(seed)
    x = torch.randn(rows, K, generator=g) * torch.exp2(torch.randint(-12, 12, (rows, 1), generator=g).float())
    flat = x.view(-1, 32)
    n = flat.shape[0]
    ties = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 4.0, 7.0, 7.9, -0.25, -2.5, -5.0, 0.0, -0.0])
    flat[0, :16] = ties
    flat[0, 16:] = 0
    if n > 1:
        flat[1] = 0
    if n > 2:
        flat[2, :16] = ties * 2.0 ** -10
        flat[2, 16:] = torch.nextafter(ties, torch.full((16,), 10.0)) * 2.0 ** -10
    if kind != "f16":
        if n > 3:
            flat[3] = torch.randn(32, generator=g) * 2.0 ** -124      # scales at the low end
        if n > 4:
            flat[4] = torch.randn(32, generator=g) * 2.0 ** -130      # subnormal in fp32
        if n > 5:
            flat[5] = torch.randn(32, generator=g) * 2.0 ** 124       # near the largest values
        if n > 6:
            flat[6] = 0
            flat[6, 31] = 2.0 ** -149 if kind == "f32" else 2.0 ** -133
    else:
        if n > 3:
            flat[3] = torch.randn(32, generator=g) * 2.0 ** -20       # subnormal in fp16
        if n > 4:
            flat[4] = 65504.0
    return x.to(TYPES[kind])


@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("rows,K", [(1, 32), (3, 32), (1, 4096), (7, 288), (130, 96), (33, 7168)])
def test_quantize_is_exact(ds4, kind, rows, K):
    x = awkward(rows, K, rows + K, kind)
    codes, scales = ds4.mxfp4_quantize(x.cuda())
    c, s = ref.quantize(x.double().numpy())
    assert np.array_equal(scales.cpu().numpy(), s)
    assert np.array_equal(codes.cpu().numpy(), c)


def test_quantize_keeps_no_block_with_a_nan_or_an_infinity(ds4):
    for kind in TYPES:
        x = torch.randn(4, 96, generator=gen(1)).to(TYPES[kind])
        x[0, 40], x[1, 95], x[2, 0] = float("nan"), float("inf"), float("-inf")
        codes, scales = ds4.mxfp4_quantize(x.cuda())
        c, s = ref.quantize(x.double().numpy())
        assert np.array_equal(scales.cpu().numpy(), s) and np.array_equal(codes.cpu().numpy(), c)
        assert (s == 255).sum() == 3
        back = ds4.mxfp4_dequantize(codes, scales).double().cpu().numpy()
        assert np.isnan(back).sum() == 96 and np.isnan(back[0, 32:64]).all()


@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
def test_quantize_strided_and_unaligned_rows(ds4, kind):
    wide = awkward(9, 256, 4, kind).cuda()
    for lo, hi in ((1, 65), (3, 227), (0, 224), (8, 40)):
        codes, scales = ds4.mxfp4_quantize(wide[:, lo:hi])
        c, s = ref.quantize(wide[:, lo:hi].double().cpu().numpy())
        assert np.array_equal(codes.cpu().numpy(), c) and np.array_equal(scales.cpu().numpy(), s)


@pytest.mark.parametrize("T,k,K", [(1, 1, 32), (1, 8, 4096), (21, 3, 160), (300, 8, 64)])
def test_quantize_into_expert_order(ds4, T, k, K):
    g = gen(T)
    x = torch.randn(T, K, generator=g).bfloat16()
    inv = torch.randperm(T * k, generator=g).int().reshape(T, k)
    hole = inv.clone()
    if T > 1:
        hole[::4, 0] = -1
        hole[1, -1] = T * k          # outside: skipped
    codes = torch.full((T * k, K // 2), 0xAB, dtype=torch.uint8, device="cuda")
    scales = torch.full((T * k, K // 32), 0xCD, dtype=torch.uint8, device="cuda")
    ds4.mxfp4_quantize(x.cuda(), hole.cuda(), codes, scales)
    c, s = ref.quantize(x.double().numpy())
    want_c, want_s = np.full((T * k, K // 2), 0xAB, np.uint8), np.full((T * k, K // 32), 0xCD, np.uint8)
    for t in range(T):
        for j in range(k):
            if 0 <= hole[t, j] < T * k:
                want_c[hole[t, j]], want_s[hole[t, j]] = c[t], s[t]
    assert np.array_equal(codes.cpu().numpy(), want_c) and np.array_equal(scales.cpu().numpy(), want_s)


@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("rows,K", [(1, 32), (5, 96), (40, 2048)])
def test_dequantize_is_exact(ds4, kind, rows, K):
    g = gen(rows)
    codes = torch.randint(0, 256, (rows, K // 2), generator=g).to(torch.uint8)
    low, high = (0, 256) if kind != "f16" else (90, 145)
    scales = torch.randint(low, high, (rows, K // 32), generator=g).to(torch.uint8)
    scales[0, 0] = 0 if kind != "f16" else 100
    scales[-1, -1] = 254 if kind != "f16" else 130
    wide = torch.zeros(rows, K + 5, dtype=TYPES[kind], device="cuda")
    for out in (None if kind == "bf16" else torch.empty(rows, K, dtype=TYPES[kind], device="cuda"), wide[:, 5:]):
        got = ds4.mxfp4_dequantize(codes.cuda(), scales.cuda(), out)
        want = torch.from_numpy(ref.dequantize(codes.numpy(), scales.numpy())).float().to(TYPES[kind])
        assert torch.equal(got.cpu().nan_to_num(7.0), want.nan_to_num(7.0))
    assert (wide[:, :5] == 0).all()


# ------------------------------------------------------------------ products
def mx_random(shape, g, spread=2, centre=121):
    """Codes and scales of random MXFP4 values (uint8 tensors on the CPU)."""
    *lead, K = shape
    codes = torch.randint(0, 256, (*lead, K // 2), generator=g).to(torch.uint8)
    scales = torch.randint(centre - spread, centre + spread + 1, (*lead, K // 32), generator=g).to(torch.uint8)
    return codes, scales


def values(codes, scales):
    v = ref.dequantize(codes.reshape(-1, codes.shape[-1]).numpy(), scales.reshape(-1, scales.shape[-1]).numpy())
    return v.reshape(*codes.shape[:-1], -1)


def offsets_of(counts):
    return torch.tensor([0] + list(np.cumsum(counts)), dtype=torch.int32)


def make(ds4, E, N, K, gated, seed, **kw):
    g = gen(seed)
    mats = [mx_random((E, N, K), g, **kw) for _ in range(2 if gated else 1)]
    ex = ds4.Mxfp4Experts(E, N, K, gated=gated)
    ex.load(*(t.cuda() for m in mats for t in m))
    return ex, [values(*m) for m in mats]


def check_product(ds4, ex, mats, counts, kind, seed, behind=0, ld_extra=0, **kw):
    R = int(sum(counts)) + behind
    N, K = ex.n_out, ex.n_in
    codes, scales = mx_random((R, K), gen(seed), **kw)
    off = offsets_of(counts)
    a = values(codes, scales)
    want, bound = ref.product(a, mats, off.numpy())
    n = R - behind
    args = (codes.cuda(), scales.cuda(), off.cuda() if len(counts) > 1 or behind else None)
    if kind == "mxfp4":
        out = torch.full((R, N // 2), 0xAB, dtype=torch.uint8, device="cuda")
        out_s = torch.full((R, N // 32), 0xCD, dtype=torch.uint8, device="cuda")
        ex.product(*args, out, out_s)
        ex.sync_status()
        c, s = out.cpu().numpy(), out_s.cpu().numpy()
        assert (c[n:] == 0xAB).all() and (s[n:] == 0xCD).all()
        c, s, want, bound = c[:n], s[:n], want[:n], bound[:n]
        mag = np.abs(want).reshape(n, N // 32, 32)
        b = bound.reshape(n, N // 32, 32)
        lo, hi = ref.mx_scale(np.maximum(mag - b, 0).max(2)), ref.mx_scale((mag + b).max(2))
        assert ((s >= lo) & (s <= hi)).all()
        f = np.ldexp(1.0, s.astype(np.int64) - 127).repeat(32, 1)
        got = ref.dequantize(c, s) / f

        def to_ladder(v):
            return np.where(v < 0, -ref.LADDER[ref.mx_round(v)], ref.LADDER[ref.mx_round(v)])
        assert (got >= to_ladder((want - bound) / f)).all() and (got <= to_ladder((want + bound) / f)).all()
        return
    t = TYPES[kind]
    buf = torch.full((R, N + ld_extra), 123.0, dtype=t, device="cuda")
    out = buf[:, :N]
    ex.product(*args, out)
    ex.sync_status()
    got = out.double().cpu().numpy()
    assert (got[n:] == 123.0).all() and (ld_extra == 0 or (buf[:, N:] == 123.0).all())
    tol = bound[:n] + (np.abs(want[:n]) + bound[:n]) * ref.HALF_STEP[t]
    if kind == "f16":   # below 2^-14 the values of fp16 lie 2^-24 apart: a rounding there is off by up to 2^-25
        tol = tol + 2.0 ** -25
    bad = ~(np.abs(got[:n] - want[:n]) <= tol)
    assert not bad.any(), (np.argwhere(bad)[:5], bad.mean())


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("K", [32, 64, 96, 224, 256, 288, 512, 1024, 2080])
def test_product_inner_lengths(ds4, gated, K):
    ex, mats = make(ds4, 3, 160, K, gated, K)
    check_product(ds4, ex, mats, [3, 0, 5], "f32", K + 1)


@pytest.mark.parametrize("N", [1, 2, 31, 32, 33, 64, 65, 127, 128, 129, 200, 256, 300])
@pytest.mark.parametrize("gated", [False, True])
def test_product_output_widths(ds4, N, gated):
    ex, mats = make(ds4, 2, N, 320, gated, N)
    for kind in ("f32", "bf16", "f16"):
        check_product(ds4, ex, mats, [4, 9], kind, N + 1, ld_extra=N % 5)


@pytest.mark.parametrize("rows", [1, 2, 7, 8, 9, 15, 16, 17, 31, 32, 33, 63, 64, 65, 100, 127, 128, 129, 190, 191, 192, 193,
                                  255, 256, 257, 513])
def test_product_group_sizes(ds4, rows):
    ex, mats = make(ds4, 1, 192, 512, False, 7)
    check_product(ds4, ex, mats, [rows], "bf16", rows)
    ex, mats = make(ds4, 1, 96, 512, True, 8)
    check_product(ds4, ex, mats, [rows], "mxfp4", rows)
    check_product(ds4, ex, mats, [rows], "f16", rows, behind=3)


COUNTS = {"empty": [0, 0, 0, 0, 0, 0, 0], "ends": [0, 5, 0, 0, 0, 9, 0], "ones": [1, 1, 1, 1, 1, 1, 1],
          "heavy": [1, 300, 0, 2, 17, 0, 64], "last": [0, 0, 0, 0, 0, 0, 40], "first": [33, 0, 0, 0, 0, 0, 0]}


@pytest.mark.parametrize("counts", sorted(COUNTS))
@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("behind", [0, 1, 70])
def test_product_loads(ds4, counts, kind, behind):
    if not sum(COUNTS[counts]) + behind:
        behind = 2
    ex, mats = make(ds4, 7, 144, 544, False, 3)
    check_product(ds4, ex, mats, COUNTS[counts], kind, 5, behind)


@pytest.mark.parametrize("counts", sorted(COUNTS))
@pytest.mark.parametrize("kind", ["f32", "bf16", "mxfp4"])
def test_gated_product_loads(ds4, counts, kind):
    ex, mats = make(ds4, 7, 96, 544, True, 4)
    check_product(ds4, ex, mats, COUNTS[counts], kind, 6, behind=4)


def test_product_many_experts(ds4):
    rng = np.random.default_rng(0)
    ex, mats = make(ds4, 512, 40, 64, False, 12)
    counts = rng.integers(0, 4, 512) * (rng.random(512) < 0.4)
    check_product(ds4, ex, mats, counts, "f32", 13)
    check_product(ds4, ex, mats, rng.integers(0, 30, 512), "bf16", 14, behind=5)


def test_product_decode_shapes(ds4):
    """One and sixteen tokens of a layer of the framework's decode width, all of it read."""
    ex, mats = make(ds4, 8, 512, 4096, True, 15, centre=118)
    check_product(ds4, ex, mats, [1] * 8, "mxfp4", 16)
    check_product(ds4, ex, mats, [1, 0, 3, 16, 0, 2, 4, 1], "bf16", 17)
    ex, mats = make(ds4, 8, 1000, 2048, False, 18, centre=118)
    check_product(ds4, ex, mats, [1] * 8, "f32", 19)


def test_product_wide_scales(ds4):
    """Scale bytes over most of their range, products inside fp32's normal range."""
    ex, mats = make(ds4, 2, 130, 256, False, 20, spread=25, centre=127)
    check_product(ds4, ex, mats, [5, 40], "f32", 21, spread=25, centre=127)


def test_product_nan_scales_stay_in_their_rows(ds4):
    ex, mats = make(ds4, 1, 130, 512, False, 22)
    codes, scales = mx_random((20, 512), gen(23))
    scales[7, 3] = 255
    codes[7, 48:64] = 0x77
    out = ex.product(codes.cuda(), scales.cuda(), None, torch.empty(20, 130, device="cuda")).cpu()
    assert out[7].isnan().all()
    assert not out[torch.arange(20) != 7].isnan().any()


def test_product_ignores_what_lies_behind_the_rows(ds4):
    """A view of a longer buffer whose later rows hold NaN scales: no effect on the rows in use."""
    ex, mats = make(ds4, 2, 64, 256, False, 24)
    codes, scales = mx_random((300, 256), gen(25))
    scales[13:] = 255
    codes[13:] = 0x77
    off = offsets_of([5, 8])
    out = torch.full((300, 64), 9.0, device="cuda")
    ex.product(codes.cuda(), scales.cuda(), off.cuda(), out)
    want, bound = ref.product(values(codes[:13], scales[:13]), mats, off.numpy())
    got = out.cpu().double().numpy()
    assert (np.abs(got[:13] - want) <= bound + np.abs(want) * ref.U24).all() and (got[13:] == 9.0).all()


def test_product_offsets_out_of_range_are_clipped(ds4):
    ex, mats = make(ds4, 3, 64, 256, False, 26)
    codes, scales = mx_random((10, 256), gen(27))
    out = torch.full((10, 64), 9.0, device="cuda")
    ex.product(codes.cuda(), scales.cuda(), torch.tensor([-4, 3, 3, 1000], dtype=torch.int32).cuda(), out)
    want, bound = ref.product(values(codes, scales), mats, [0, 3, 3, 10])
    assert (np.abs(out.cpu().double().numpy() - want) <= bound + np.abs(want) * ref.U24).all()


def test_product_refuses_offsets_that_decrease(ds4):
    ex, mats = make(ds4, 3, 64, 256, False, 26)
    codes, scales = (t.cuda() for t in mx_random((10, 256), gen(27)))
    out = torch.full((10, 64), 9.0, device="cuda")
    ex.product(codes, scales, torch.tensor([0, 8, 2, 10], dtype=torch.int32).cuda(), out)
    with pytest.raises(ds4.Ds4MoeError, match="EDEVICE"):
        ex.sync_status()
    assert (out == 9.0).all()
    ex.product(codes, scales, torch.tensor([0, 2, 8, 10], dtype=torch.int32).cuda(), out)
    ex.sync_status()
    assert (out != 9.0).all()


def test_product_repeats_bit_for_bit(ds4):
    ex, mats = make(ds4, 4, 256, 4096, True, 28, centre=118)
    codes, scales = (t.cuda() for t in mx_random((9, 4096), gen(29)))
    off = offsets_of([1, 0, 6, 2]).cuda()
    first = ex.product(codes, scales, off, torch.empty(9, 256, device="cuda")).clone()
    for _ in range(20):
        assert torch.equal(ex.product(codes, scales, off, torch.empty(9, 256, device="cuda")), first)


# ------------------------------------------------------------------ combine
@pytest.mark.parametrize("o_kind", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("y_kind", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("T,k,H", [(1, 1, 1), (1, 8, 4096), (5, 3, 257), (130, 6, 96), (3, 32, 1030)])
def test_combine(ds4, o_kind, y_kind, T, k, H):
    g = gen(T * k + H)
    o = torch.randn(T * k, H, generator=g).to(TYPES[o_kind])
    inv = torch.randperm(T * k, generator=g).int().reshape(T, k)
    w = torch.rand(T, k, generator=g)
    if k > 1:
        inv[0, 1] = -1
        inv[T // 2, 0] = T * k
        o[int(torch.nonzero(torch.ones(T * k))[0])] = o[0]
    for add_kind in (None, "f32", "bf16", "f16"):
        add = None if add_kind is None else torch.randn(T, H, generator=g).to(TYPES[add_kind])
        y = torch.empty(T, H, dtype=TYPES[y_kind], device="cuda")
        ds4.combine(o.cuda(), inv.cuda(), w.cuda(), y, None if add is None else add.cuda())
        rows = np.concatenate((o.double().numpy(), np.zeros((1, H))))
        pick = np.where((inv.numpy() < 0) | (inv.numpy() >= T * k), T * k, inv.numpy())
        terms = rows[pick] * w.double().numpy()[:, :, None]
        want, size = terms.sum(1), np.abs(terms).sum(1)
        if add is not None:
            want, size = want + add.double().numpy(), size + np.abs(add.double().numpy())
        # k + 1 fp32 operations on partial sums no larger than the sum of magnitudes, then one rounding
        tol = (k + 1) * ref.U24 * size
        tol = tol + (np.abs(want) + tol) * ref.HALF_STEP[TYPES[y_kind]] + 2.0 ** -24 * (y_kind == "f16")
        assert (np.abs(y.double().cpu().numpy() - want) <= tol).all()


def test_combine_skips_rows_that_hold_nan(ds4):
    o = torch.full((4, 64), float("nan"))
    o[2] = 1.0
    y = ds4.combine(o.cuda(), torch.tensor([[2, -1], [-1, -1]], dtype=torch.int32).cuda(), torch.ones(2, 2).cuda())
    assert (y[0] == 1).all() and (y[1] == 0).all()


def test_combine_in_place(ds4):
    g = gen(4)
    o, inv, w = torch.randn(12, 100, generator=g).cuda(), torch.randperm(12, generator=g).int().reshape(6, 2).cuda(), torch.rand(6, 2, generator=g).cuda()
    add = torch.randn(6, 100, generator=g).cuda()
    want = ds4.combine(o, inv, w, add=add)
    ds4.combine(o, inv, w, add, add)
    assert torch.equal(add, want)


# ------------------------------------------------------------------ unaligned and far places
@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("E", [128, 256, 512])
def test_route_rows_that_are_not_aligned_pieces(ds4, kind, E):
    wide = torch.randn(20, E + 5, generator=gen(E)).to(TYPES[kind]).cuda()
    check_route(ds4, wide[:, 2:2 + E], 8, score="sigmoid")
    check_route(ds4, wide[:, 2:2 + E], 8, torch.randn(E, generator=gen(1)) * 0.1, score="softmax", n_groups=8, topk_groups=3)


@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("H", [1, 7, 33, 96, 1021, 2050])
@pytest.mark.parametrize("first", [0, 1, 3])
def test_combine_rows_at_any_element(ds4, kind, H, first):
    g = gen(H)
    T, k = 9, 5
    o = torch.randn(T * k + 4, H, generator=g).to(TYPES[kind]).cuda()[first:first + T * k]
    inv = torch.randperm(T * k, generator=g).int().reshape(T, k)
    w = torch.rand(T, k, generator=g)
    add = torch.randn(T + 1, H, generator=g).cuda()[1:]
    y = torch.full((T + 2, H), 77.0, device="cuda")
    ds4.combine(o, inv.cuda(), w.cuda(), y[1:T + 1], add)
    terms = o.double().cpu().numpy()[inv.numpy()] * w.double().numpy()[:, :, None]
    want, size = terms.sum(1) + add.double().cpu().numpy(), np.abs(terms).sum(1) + np.abs(add.double().cpu().numpy())
    tol = (k + 1) * ref.U24 * size + np.abs(want) * ref.U24
    assert (np.abs(y[1:T + 1].double().cpu().numpy() - want) <= tol).all()
    assert (y[0] == 77).all() and (y[T + 1] == 77).all()


@pytest.mark.parametrize("K", [64, 512, 1024])
@pytest.mark.parametrize("shift", [1, 2, 4, 7])
def test_product_scales_at_any_byte(ds4, K, shift):
    ex, mats = make(ds4, 2, 96, K, False, 40)
    codes, scales = mx_random((30, K), gen(41))
    held = torch.zeros(scales.numel() + 16, dtype=torch.uint8, device="cuda")
    held[shift:shift + scales.numel()] = scales.reshape(-1).cuda()
    off = offsets_of([11, 19])
    out = ex.product(codes.cuda(), held[shift:shift + scales.numel()].view(30, K // 32), off.cuda(), torch.empty(30, 96, device="cuda"))
    want, bound = ref.product(values(codes, scales), mats, off.numpy())
    assert (np.abs(out.double().cpu().numpy() - want) <= bound + np.abs(want) * ref.U24).all()


def test_rows_far_apart(ds4):
    """Row strides of 2^30 + 32 elements: offsets beyond 32 bits, of elements and of bytes."""
    far = (1 << 30) + 32
    g = gen(50)
    held = torch.zeros(4 * far + 4096, dtype=torch.bfloat16, device="cuda")
    view = held.as_strided((5, 256), (far, 1))
    x = torch.randn(5, 256, generator=g).bfloat16()
    view.copy_(x.cuda())
    codes, scales = ds4.mxfp4_quantize(view)
    c, s = ref.quantize(x.double().numpy())
    assert np.array_equal(codes.cpu().numpy(), c) and np.array_equal(scales.cpu().numpy(), s)
    check_route(ds4, view, 8, score="sigmoid")
    held.zero_()
    ds4.mxfp4_dequantize(codes, scales, view)
    assert torch.equal(view.cpu().double(), torch.from_numpy(ref.dequantize(c, s)))
    ex, mats = make(ds4, 1, 256, 256, False, 51)
    ex.product(codes, scales, None, view)
    want, bound = ref.product(ref.dequantize(c, s), mats, [0, 5])
    assert (np.abs(view.double().cpu().numpy() - want) <= bound + (np.abs(want) + bound) * 2.0 ** -8).all()
    del view, held
    # rows of o beyond 2^31 elements
    H, rows = 1 << 20, 2200
    o = torch.zeros(rows, H, dtype=torch.bfloat16, device="cuda")
    o[rows - 1], o[rows - 2, 5] = 3.0, 1.0
    inv = torch.tensor([[rows - 1, 0], [rows - 2, rows]], dtype=torch.int32).cuda()
    y = ds4.combine(o, inv, torch.tensor([[0.5, 1.0], [2.0, 1.0]]).cuda())
    assert (y[0] == 1.5).all() and y[1, 5] == 2.0 and y[1].sum() == 2.0


# ------------------------------------------------------------------ together
class Chain:
    """An MoE FFN of MXFP4 experts as a program runs it, every buffer its own."""

    def __init__(self, ds4, T, H, I, E, k, seed):
        g = gen(seed)
        self.ds4, self.T, self.E, self.k = ds4, T, E, k
        self.up = [mx_random((E, I, H), g, centre=119) for _ in range(2)]
        self.dn = mx_random((E, H, I), g, centre=119)
        self.gate_up, self.down = ds4.Mxfp4Experts(E, I, H, gated=True), ds4.Mxfp4Experts(E, H, I)
        self.gate_up.load(*(t.cuda() for m in self.up for t in m))
        self.down.load(*(t.cuda() for t in self.dn))
        self.bias = torch.randn(E, generator=g) * 0.1
        self.router = ds4.Router(E, k, score="sigmoid", n_groups=2, topk_groups=2, group_score="top2", scale=2.5)
        P, u8 = T * k, dict(dtype=torch.uint8, device="cuda")
        self.r = self.router.buffers(T)
        self.xq, self.xs = torch.zeros(P, H // 2, **u8), torch.zeros(P, H // 32, **u8)
        self.hq, self.hs = torch.zeros(P, I // 2, **u8), torch.zeros(P, I // 32, **u8)
        self.o = torch.empty(P, H, device="cuda")
        self.y = torch.empty(T, H, device="cuda")
        self.dbias = self.bias.cuda()

    def __call__(self, x, logits, shared):
        self.router.route(logits, self.dbias, self.r)
        self.ds4.mxfp4_quantize(x, self.r.inv_pos.view(self.T, self.k), self.xq, self.xs)
        self.gate_up.product(self.xq, self.xs, self.r.expert_offsets, self.hq, self.hs)
        self.down.product(self.hq, self.hs, self.r.expert_offsets, self.o)
        return self.ds4.combine(self.o, self.r.inv_pos, self.r.topk_w, self.y, shared)

    def check(self, x, logits, shared, y):
        """y against the run in float64; h is taken from the GPU's own MXFP4 rows, which the product tests hold to
        the formula, so that a value at a border of two codes does not count twice."""
        idx, w = ref.route(logits.cpu(), self.k, "sigmoid", self.bias, 2, 2, "top2", True, 2.5)
        off, st, ss, inv = ref.permute(idx, self.E)
        n = off[-1]
        assert np.array_equal(self.r.topk_idx.cpu().numpy(), idx)
        c, s = ref.quantize(x.double().cpu().numpy())
        assert np.array_equal(self.xq.cpu().numpy()[:n], c[st]) and np.array_equal(self.xs.cpu().numpy()[:n], s[st])
        h, hb = ref.product(ref.dequantize(c, s)[st], [values(*m) for m in self.up], off)
        hv = ref.dequantize(self.hq.cpu().numpy()[:n], self.hs.cpu().numpy()[:n])
        # a block whose largest value is m * 2^e, 4 <= m < 8, has steps of at most 2 * 2^e, and 8 is cut to 6: every
        # value is within a quarter of the largest (0.26 leaves room for a scale chosen one lower by the bound)
        per_block = [np.abs(v).reshape(n, h.shape[1] // 32, 32).max(2) for v in (hv - h, h, hb)]
        assert (per_block[0] <= 0.26 * per_block[1] + per_block[2]).all()
        o, ob = ref.product(hv, [values(*self.dn)], off)
        want, tol = shared.double().cpu().numpy(), np.zeros((self.T, o.shape[1]))
        for t in range(self.T):
            for j in range(self.k):
                p = inv[t * self.k + j]
                if p >= 0:
                    want[t] += w[t, j] * o[p]
                    tol[t] += w[t, j] * (ob[p] + (self.k + 20) * ref.U24 * np.abs(o[p]))
        tol += (self.k + 2) * ref.U24 * (np.abs(shared.double().cpu().numpy()) + np.abs(want))
        assert (np.abs(y.double().cpu().numpy() - want) <= tol).all()

    def inputs(self, seed, masked=False):
        g = gen(seed)
        H = self.down.n_out
        logits = torch.randn(self.T, self.E, generator=g)
        if masked:
            logits[self.T // 2] = float("-inf")
            logits[0, 1:] = float("-inf")
        return torch.randn(self.T, H, generator=g).bfloat16().cuda(), logits.cuda(), torch.randn(self.T, H, generator=g).cuda()


@pytest.mark.parametrize("T,H,I,E,k", [(1, 256, 128, 8, 2), (3, 512, 288, 8, 4), (40, 320, 96, 16, 4), (200, 256, 160, 6, 3),
                                       (1, 1024, 512, 4, 1)])
@pytest.mark.parametrize("masked", [False, True])
def test_run_together(ds4, T, H, I, E, k, masked):
    c = Chain(ds4, T, H, I, E, k, T)
    args = c.inputs(T + 1, masked)
    y = c(*args)
    c.gate_up.sync_status()
    c.down.sync_status()
    c.check(*args, y)


def test_run_together_captured_and_replayed(ds4):
    """Two graphs of two chains, replayed in turn and at the same time on two streams, with new inputs each time."""
    chains = [Chain(ds4, 70, 256, 128, 8, 3, s) for s in (1, 2)]
    held = [c.inputs(9) for c in chains]
    graphs = []
    for c, args in zip(chains, held):
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            c(*args)
        torch.cuda.current_stream().wait_stream(s)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            c(*args)
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in chains]
    for turn in range(4):
        fresh = [c.inputs(20 + 2 * turn + i, masked=turn == 2) for i, c in enumerate(chains)]
        for args, new in zip(held, fresh):
            for a, b in zip(args, new):
                a.copy_(b)
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for c, args in zip(chains, held):
            c.check(*args, c.y)


@pytest.mark.parametrize("captured", [False, True])
def test_runs_behind_one_another(ds4, captured):
    """Kernels are launched ahead of the end of those before them: many runs through the same buffers, nothing
    waited for between them, give what they give one at a time."""
    c = Chain(ds4, 50, 512, 256, 8, 3, 71)
    several = [c.inputs(80 + i, masked=i == 2) for i in range(6)]
    want = []
    for args in several:
        want.append(c(*args).clone())
        torch.cuda.synchronize()
    got = [torch.zeros_like(w) for _ in range(8) for w in want]

    def all_of_them():
        for i, g in enumerate(got):
            g.copy_(c(*several[i % 6]))
    if captured:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            all_of_them()
        graph.replay()
    else:
        all_of_them()
    torch.cuda.synchronize()
    assert all(torch.equal(g, want[i % 6]) for i, g in enumerate(got))


def test_calls_use_the_current_stream(ds4):
    c = Chain(ds4, 33, 256, 128, 8, 3, 5)
    args = c.inputs(6)
    want = c(*args).clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        late = [torch.zeros_like(a) for a in args]
        torch.cuda._sleep(20_000_000)
        for a, b in zip(late, args):
            a.copy_(b, non_blocking=True)
        c.y.zero_()
        got = c(*late)
    s.synchronize()
    assert torch.equal(got, want)


def test_two_products_of_one_handle_at_once(ds4):
    """A handle has no workspace: its calls may overlap on two streams."""
    ex, mats = make(ds4, 4, 512, 1024, True, 60)
    a = [tuple(t.cuda() for t in mx_random((40, 1024), gen(61 + i))) + (offsets_of(c).cuda(),)
         for i, c in enumerate(([40, 0, 0, 0], [1, 13, 20, 6]))]
    want = [ex.product(*x, torch.empty(40, 512, device="cuda")).clone() for x in a]
    streams = [torch.cuda.Stream() for _ in a]
    torch.cuda.synchronize()
    for _ in range(5):
        got = []
        for x, s in zip(a, streams):
            with torch.cuda.stream(s):
                got.append(ex.product(*x, torch.zeros(40, 512, device="cuda")))
        torch.cuda.synchronize()
        assert all(torch.equal(g, w) for g, w in zip(got, want))
    ex.sync_status()


def test_routing_buffers_are_fixed(ds4):
    b = ds4.Router(8, 2).buffers(3)
    with pytest.raises(AttributeError):
        b.topk_w = torch.empty(3, 2, device="cuda")


def test_reload_replaces_the_weights(ds4):
    ex, mats = make(ds4, 2, 64, 256, False, 30)
    check_product(ds4, ex, mats, [3, 4], "f32", 31)
    codes, scales = mx_random((2, 64, 256), gen(32))
    ex.load(codes.cuda(), scales.cuda())
    check_product(ds4, ex, [values(codes, scales)], [3, 4], "f32", 31)


def test_injected_launch_failure(ds4, monkeypatch):
    ex, mats = make(ds4, 1, 32, 32, False, 33)
    codes, scales = (t.cuda() for t in mx_random((2, 32), gen(1)))
    monkeypatch.setenv("DS4MOE_FAULT", "launch")
    with pytest.raises(ds4.Ds4MoeError, match="injected"):
        ex.product(codes, scales)
    with pytest.raises(ds4.Ds4MoeError):
        ds4.mxfp4_quantize(torch.zeros(1, 32, device="cuda"))
    monkeypatch.delenv("DS4MOE_FAULT")
    ex.product(codes, scales)
    ex.sync_status()


def test_product_without_weights_is_refused(ds4):
    ex = ds4.Mxfp4Experts(1, 32, 32)
    with pytest.raises(ds4.Ds4MoeError, match="no weights"):
        ex.product(torch.zeros(1, 16, dtype=torch.uint8, device="cuda"), torch.zeros(1, 1, dtype=torch.uint8, device="cuda"))


def test_binding_refuses_wrong_tensors(ds4):
    cu = dict(device="cuda")
    r = ds4.Router(8, 2)
    for bad in (torch.zeros(2, 8), torch.zeros(2, 9, **cu), torch.zeros(2, 8, dtype=torch.float64, **cu),
                torch.zeros(8, **cu), torch.zeros(8, 2, **cu).t()):
        with pytest.raises(ValueError):
            r.route(bad)
    with pytest.raises(ValueError):
        r.route(torch.zeros(2, 8, **cu), torch.zeros(8, dtype=torch.float64, **cu))
    with pytest.raises(ValueError):
        r.route(torch.zeros(2, 8, **cu), None, r.buffers(3))
    with pytest.raises(ValueError):
        ds4.mxfp4_quantize(torch.zeros(2, 40, **cu))
    with pytest.raises(ValueError):
        ds4.mxfp4_quantize(torch.zeros(2, 64, **cu), torch.zeros(3, 1, dtype=torch.int32, **cu))
    with pytest.raises(ValueError):
        ds4.mxfp4_quantize(torch.zeros(2, 64, **cu), None, torch.zeros(2, 16, dtype=torch.uint8, **cu))
    ex, _ = make(ds4, 2, 32, 64, False, 1)
    codes, scales = torch.zeros(3, 32, dtype=torch.uint8, **cu), torch.zeros(3, 2, dtype=torch.uint8, **cu)
    off = torch.zeros(3, dtype=torch.int32, **cu)
    with pytest.raises(ValueError):
        ex.product(codes[:, :16].contiguous(), scales, off)
    with pytest.raises(ValueError):
        ex.product(codes, scales[:2], off)
    with pytest.raises(ValueError):
        ex.product(codes, scales, off.long())
    with pytest.raises(ds4.Ds4MoeError, match="offsets are required"):
        ex.product(codes, scales)
    with pytest.raises(ValueError):
        ex.product(codes, scales, off, torch.zeros(3, 33, **cu))
    with pytest.raises(ValueError):
        ds4.combine(torch.zeros(4, 8, **cu), torch.zeros(2, 2, dtype=torch.int32, **cu), torch.zeros(2, 3, **cu))
