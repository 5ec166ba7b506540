"""The operators beside the layer at their edges: values, sizes and calls that the other tests leave out."""
import os
import subprocess
import sys
import threading

import numpy as np
import pytest

import operator_refs as ref

torch = pytest.importorskip("torch")
from test_operators import TYPES, check_route, ds4, gen, make, mx_random  # noqa: E402, F401  (ds4: the fixture)

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


# ------------------------------------------------------------------ signed zeros
@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("E", [3, 64, 128, 200, 256, 512])
def test_zeros_of_both_signs_are_a_tie(ds4, kind, E):
    """-0 and +0 are equal logits: the lower index goes first, in the order and at the k-th place."""
    g = gen(E)
    some = torch.tensor([-1.0, -0.0, 0.0, -0.0, 0.0, 1.0])
    logits = some[torch.randint(0, 6, (90, E), generator=g)]
    logits[0], logits[1] = -0.0, 0.0
    logits[2, 0::2], logits[2, 1::2] = -0.0, 0.0
    logits[3, 0::2], logits[3, 1::2] = 0.0, -0.0
    logits[4], logits[4, E - 1], logits[4, E - 2] = -1.0, 0.0, -0.0       # the last places, in turn
    logits[5], logits[5, E - 1], logits[5, 0], logits[5, 1] = -0.0, 5.0, -0.0, 0.0
    logits = logits.to(TYPES[kind])
    assert bool(torch.signbit(logits[0, 0])) and not bool(torch.signbit(logits[1, 0]))
    for bias in (None, torch.zeros(E), -torch.zeros(E)):
        for score in ("softmax", "sigmoid", "sqrt_softplus"):
            check_route(ds4, logits, 1, bias, score=score)
            check_route(ds4, logits, min(E, 8), bias, score=score, renormalise=False)
            if E % 4 == 0:
                for group_score in ("max", "top2"):
                    check_route(ds4, logits, 8, bias, score=score, n_groups=4, topk_groups=2, group_score=group_score)


@pytest.mark.gpu
def test_zeros_by_underflow_are_a_tie(ds4):
    """Products that underflow to -0 and +0 in fp16, with a +0 of a higher index."""
    logits = torch.tensor([[-1e-9, 1e-9, -1.0], [1e-9, -1e-9, -1.0], [-1.0, -1e-9, 1e-9]]).half()
    check_route(ds4, logits, 1)
    check_route(ds4, logits, 2)


# ------------------------------------------------------------------ shared memory of the routing
@pytest.mark.gpu
@pytest.mark.parametrize("E,G,T", [(336, 4, 22), (340, 4, 22), (339, 3, 23), (341, 11, 22), (455, 5, 76001)])
def test_route_at_the_limit_of_plain_shared_memory(ds4, E, G, T):
    """Dynamic sizes within the kernel's own static bytes of 48 KB, each in a process of its own (an earlier call
    could have raised the kernel's limit)."""
    program = """
import torch, numpy as np
import bit_quantized_routed_sqrt_b200 as ds4
import operator_refs as ref
E, G, T = %d, %d, %d
logits = torch.randn(T, E, generator=torch.Generator().manual_seed(E))
r = ds4.Router(E, 4, n_groups=G, topk_groups=2).route(logits.cuda())
torch.cuda.synchronize()
rows = list(range(min(T, 40))) + ([T - 1] if T > 40 else [])
idx, w = ref.route(logits[rows], 4, "softmax", None, G, 2)
got = r.topk_idx.cpu().numpy()
assert np.array_equal(got[rows], idx)
off, st, ss, inv = ref.permute(got, E)
assert np.array_equal(r.expert_offsets.cpu().numpy(), off) and np.array_equal(r.inv_pos.cpu().numpy(), inv)
assert np.array_equal(r.sorted_token.cpu().numpy(), st) and np.array_equal(r.sorted_slot.cpu().numpy(), ss)
""" % (E, G, T)
    env = dict(os.environ, PYTHONPATH=os.pathsep.join([ROOT, os.path.join(ROOT, "tests")]))
    done = subprocess.run([sys.executable, "-c", program], env=env, cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert done.returncode == 0, done.stderr[-2000:]


@pytest.mark.gpu
def test_route_from_several_threads(ds4):
    """Calls of host threads at once that need different amounts of shared memory of the same kernel."""
    state, want = [], []
    for E, T in [(508, 64), (300, 24), (508, 64), (300, 24)]:
        r = ds4.Router(E, 4, n_groups=4, topk_groups=2)
        logits = torch.randn(T, E, generator=gen(E)).cuda()
        out, stream = r.buffers(T), torch.cuda.Stream()
        args = [ds4.C.byref(r.cfg), logits.data_ptr(), ds4.F32, E, T, None, *out.addresses, stream.cuda_stream]
        state.append((args, out, r, logits, stream))
        want.append(r.route(logits).topk_idx.clone())
    torch.cuda.synchronize()
    wrong = [0] * len(state)
    start = threading.Barrier(len(state))

    def work(i):   # the library's call alone, so that the threads meet inside it
        args, call = state[i][0], ds4.lib.ds4moe_route_logits
        start.wait(30)
        for _ in range(30000):
            wrong[i] += call(*args) != 0

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(state))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert wrong == [0] * len(state)
    for s, w in zip(state, want):
        assert torch.equal(s[1].topk_idx, w)


# ------------------------------------------------------------------ gates far below zero
@pytest.mark.gpu
@pytest.mark.parametrize("low,high", [(-130, -84), (-86, -60), (-172, -130)])
def test_gates_far_below_zero(ds4, low, high):
    """silu(g) * u where e^-g is beyond 2^126 or infinite in fp32 and u is large: a normal value, not zero.
    Rows of ones make the sums exact.  What is left, in half steps: the exponential 2, a quotient 4, a product 1.
    Far below zero that is g e (2 + 1) over one (4), u e (2 + 1) and their product (1): 11; above, 1 + e (2 + 1),
    the quotient (4) and the product (1): 8."""
    rng = np.random.default_rng(-low)
    N = 64
    wg = np.zeros((N, 32))
    for n in range(N):   # codes whose sum is a multiple of 0.5 in the range
        left = rng.integers(2 * -high, 2 * -low + 1) / 2.0
        for i in range(32):
            v = ref.LADDER[ref.LADDER <= min(left, 6.0)][-1]
            wg[n, i], left = -v, left - v
        assert left == 0.0
    wu = ref.LADDER[rng.integers(1, 8, (N, 32))] * 2.0 ** 110
    wu[::3] *= -1
    gc, gs = quantised(wg)
    uc, us = quantised(wu)
    ones_c = torch.full((3, 16), 0x22, dtype=torch.uint8)
    ones_s = torch.full((3, 1), 127, dtype=torch.uint8)
    g, u = ref.dequantize(gc, gs).sum(1), ref.dequantize(uc, us).sum(1)
    assert g.max() <= high and g.min() >= low
    want = np.tile(ref.silu(g) * u, (3, 1))
    ex = ds4.Mxfp4Experts(1, N, 32, gated=True)
    ex.load(*(torch.from_numpy(t).reshape(1, N, -1).cuda() for t in (gc, gs, uc, us)))
    a = (ones_c.cuda(), ones_s.cuda(), None)
    out = torch.empty(3, N, device="cuda")
    ex.product(*a, out)
    got = out.double().cpu().numpy()
    normal = np.abs(want) >= 2.0 ** -126
    assert normal.any()
    assert (np.abs(got - want) <= 11 * ref.U24 * 1.001 * np.abs(want) + 2.0 ** -126 * ~normal).all()
    codes, scales = torch.zeros(3, N // 2, dtype=torch.uint8, device="cuda"), torch.zeros(3, N // 32, dtype=torch.uint8, device="cuda")
    ex.product(*a, codes, scales)
    c, s = ds4.mxfp4_quantize(out)
    assert torch.equal(c, codes) and torch.equal(s, scales)


def quantised(w):
    c, s = ref.quantize(w)
    return np.ascontiguousarray(c), np.ascontiguousarray(s)


# ------------------------------------------------------------------ sizes next to 2^31
@pytest.mark.gpu
def test_product_refuses_more_rows_than_it_can_index(ds4):
    """Row indexes past a tile's end stay below 2^31; the call is refused before any buffer is looked at."""
    ex = ds4.Mxfp4Experts(1, 1, 32)
    one = torch.full((1, 16), 0x22, dtype=torch.uint8, device="cuda")
    scale = torch.full((1, 1), 127, dtype=torch.uint8, device="cuda")
    ex.load(one, scale)
    out = torch.zeros(1, 1, dtype=torch.bfloat16, device="cuda")
    for rows in (-1, 2 ** 31 - 255, 2 ** 31 - 1):
        with pytest.raises(ds4.Ds4MoeError, match="rows"):
            ds4.ds4moe_mxfp4_product(ex.h, one, scale, rows, None, out, ds4.BF16, 1)
    ex.product(one, scale, None, out)
    ex.sync_status()
    assert out.item() == 32.0


@pytest.mark.gpu
@pytest.mark.parametrize("H", [2 ** 31 - 1, 2 ** 31 - 7])
def test_combine_of_the_widest_rows(ds4, H):
    """Rows whose last piece of 16 bytes ends at or behind element 2^31."""
    o = torch.ones(1, H, dtype=torch.bfloat16, device="cuda")
    o[0, -9:] = torch.arange(9.0).bfloat16().cuda()
    o[0, 5] = -2.0
    y = torch.zeros(1, H, dtype=torch.bfloat16, device="cuda")
    ds4.combine(o, torch.zeros(1, 1, dtype=torch.int32, device="cuda"), torch.full((1, 1), 2.0, device="cuda"), y)
    o *= 2
    assert torch.equal(y, o)


class Claims:
    """A tensor that claims a shape and to be on the GPU; no refused call may look at its memory."""
    is_cuda = True

    def __init__(self, *shape, dtype=None):
        self.shape, self.dtype, self.device = shape, dtype or torch.bfloat16, torch.device("cuda", 0)

    def stride(self):
        return (self.shape[1], 1)

    def dim(self):
        return len(self.shape)

    def numel(self):
        return self.shape[0] * self.shape[1]

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return 1 << 20


def test_sizes_beyond_32_bits_are_refused(ds4_cpu, monkeypatch):
    """A size past 2^31 - 1 would reach the library as another one."""
    ds4 = ds4_cpu
    monkeypatch.setattr(ds4, "_run", lambda *a: pytest.fail("the library was called"))
    big, u8, i32, f32 = 2 ** 32, torch.uint8, torch.int32, torch.float32
    one = Claims(1, 1, dtype=f32)
    for call in (lambda: ds4.Router(1, 1).route(Claims(big + 3, 1)),
                 lambda: ds4.mxfp4_quantize(Claims(1, big + 32)),
                 lambda: ds4.mxfp4_quantize(Claims(big + 1, 32)),
                 lambda: ds4.mxfp4_quantize(Claims(1, 32), Claims(1, big + 1, dtype=i32)),
                 lambda: ds4.mxfp4_quantize(Claims(1, 32), None, Claims(big + 1, 16, dtype=u8), Claims(big + 1, 1, dtype=u8)),
                 lambda: ds4.mxfp4_dequantize(Claims(big + 1, 16, dtype=u8), Claims(big + 1, 1, dtype=u8), Claims(big + 1, 32)),
                 lambda: ds4.mxfp4_dequantize(Claims(1, 2 ** 31 - 16, dtype=u8), Claims(1, 2 ** 27 - 1, dtype=u8), Claims(1, 2 ** 32 - 32)),
                 lambda: ds4.combine(Claims(1, big + 8), Claims(1, 1, dtype=i32), one, Claims(1, big + 8)),
                 lambda: ds4.combine(Claims(1, 8), Claims(big + 1, 1, dtype=i32), Claims(big + 1, 1, dtype=f32), Claims(big + 1, 8)),
                 lambda: experts(ds4).product(Claims(big + 1, 16, dtype=u8), Claims(big + 1, 1, dtype=u8), None, Claims(big + 1, 1)),
                 lambda: ds4.combine(Claims(1, 8), Claims(1, big + 1, dtype=i32), Claims(1, big + 1, dtype=f32), Claims(1, 8))):
        with pytest.raises(ValueError, match="2\\^31"):
            call()


def experts(ds4):
    """A handle's object without the handle."""
    e = object.__new__(ds4.Mxfp4Experts)
    e.h, e.device, e.n_experts, e.n_out, e.n_in, e.gated = None, 0, 1, 1, 32, False
    return e


@pytest.fixture(scope="module")
def ds4_cpu():
    import __graft_entry__
    __graft_entry__.build_library()
    import bit_quantized_routed_sqrt_b200 as m
    m._bind_torch()
    return m


# ------------------------------------------------------------------ the binding
@pytest.mark.gpu
def test_product_makes_mxfp4_codes_for_given_scales(ds4):
    ex, _ = make(ds4, 3, 64, 96, True, 40)
    codes, scales = (t.cuda() for t in mx_random((9, 96), gen(41)))
    off = torch.tensor([0, 4, 4, 9], dtype=torch.int32, device="cuda")
    want, want_s = torch.zeros(9, 32, dtype=torch.uint8, device="cuda"), torch.zeros(9, 2, dtype=torch.uint8, device="cuda")
    ex.product(codes, scales, off, want, want_s)
    got_s = torch.zeros_like(want_s)
    got = ex.product(codes, scales, off, out_scales=got_s)
    ex.sync_status()
    assert torch.equal(got, want) and torch.equal(got_s, want_s)
    with pytest.raises(ValueError, match="out_scales"):
        ex.product(codes, scales, off, out_scales=got_s[:8])
