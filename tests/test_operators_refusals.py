"""What the operators beside the layer refuse, and their plain forms' own pins (CPU only: every refusal comes
before anything touches CUDA)."""
import ctypes as C

import numpy as np
import pytest

import operator_refs as ref

EINVAL = 1
P = 1 << 20          # an aligned address that no refused call may look at


@pytest.fixture(scope="module")
def ds4():
    import __graft_entry__
    __graft_entry__.build_library()
    import bit_quantized_routed_sqrt_b200 as m
    return m


def router(ds4, **kw):
    f = dict(n_experts=8, top_k=2, score=0, n_groups=1, topk_groups=1, group_score=0, renormalise=1, scale=1.0)
    f.update(kw)
    return ds4.ds4moe_router(*f.values())


@pytest.mark.parametrize("bad", [
    dict(n_experts=0), dict(n_experts=513), dict(top_k=0), dict(top_k=33, n_experts=64), dict(top_k=9), dict(score=-1),
    dict(score=3), dict(n_groups=0), dict(n_groups=3), dict(n_groups=64, n_experts=64), dict(topk_groups=0),
    dict(topk_groups=2), dict(n_groups=4, topk_groups=1, top_k=3), dict(group_score=2), dict(renormalise=2),
    dict(scale=float("nan")), dict(scale=float("inf"))])
def test_bad_routers(ds4, bad):
    r = router(ds4, **bad)
    assert ds4.lib.ds4moe_route_logits_workspace(C.byref(r), 1000) == 0
    assert ds4.lib.ds4moe_route_logits(C.byref(r), P, 0, 600, 4, None, P, P, P, P, P, P, P, 1 << 30, None) == EINVAL


@pytest.mark.parametrize("change", [
    dict(router=None), dict(logits=None), dict(type=3), dict(type=-1), dict(ld=7), dict(T=-1), dict(idx=None), dict(w=None),
    dict(logits=P + 2), dict(T=1 << 30), dict(T=65, ws=None), dict(T=65, ws_bytes=100), dict(T=65, ws=P + 2)])
def test_bad_route_calls(ds4, change):
    a = dict(router=router(ds4), logits=P, type=0, ld=8, T=4, idx=P, w=P, ws=P, ws_bytes=1 << 30)
    a.update(change)
    r = C.byref(a["router"]) if a["router"] is not None else None
    assert ds4.lib.ds4moe_route_logits(r, a["logits"], a["type"], a["ld"], a["T"], None, a["idx"], a["w"], P, P, P, P,
                                       a["ws"], a["ws_bytes"], None) == EINVAL


def test_route_workspace_sizes(ds4):
    r = router(ds4, n_experts=256, top_k=8)
    sizes = [ds4.lib.ds4moe_route_logits_workspace(C.byref(r), T) for T in (-1, 0, 1, 64, 65, 2048, 65536)]
    assert sizes[:4] == [0, 0, 0, 0] and 0 < sizes[4] <= sizes[5] <= sizes[6]


@pytest.mark.parametrize("change", [
    dict(x=None), dict(x=P + 2), dict(type=3), dict(ld=63), dict(rows=-1), dict(K=0), dict(K=48), dict(K=-32),
    dict(out_rows=3), dict(out_rows=-1), dict(codes=None), dict(codes=P + 8), dict(scales=None), dict(inv=P, k=0),
    dict(inv=P, k=33)])
def test_bad_quantize_calls(ds4, change):
    a = dict(x=P, type=0, ld=64, rows=4, K=64, inv=None, k=1, out_rows=4, codes=P, scales=P)
    a.update(change)
    assert ds4.lib.ds4moe_mxfp4_quantize(*a.values(), None) == EINVAL


@pytest.mark.parametrize("change", [
    dict(codes=None), dict(codes=P + 4), dict(scales=None), dict(rows=-1), dict(K=16), dict(K=0), dict(out=None),
    dict(out=P + 1), dict(type=3), dict(ld=63)])
def test_bad_dequantize_calls(ds4, change):
    a = dict(codes=P, scales=P, rows=4, K=64, out=P, type=1, ld=64)
    a.update(change)
    assert ds4.lib.ds4moe_mxfp4_dequantize(*a.values(), None) == EINVAL


@pytest.mark.parametrize("change", [
    dict(o=None), dict(o=P + 1), dict(o_type=3), dict(o_rows=-1), dict(T=-1), dict(k=0), dict(k=33), dict(H=0), dict(inv=None),
    dict(w=None), dict(add_type=9), dict(add=P + 2), dict(y=None), dict(y=P + 2), dict(y_type=3)])
def test_bad_combine_calls(ds4, change):
    a = dict(o=P, o_type=1, o_rows=8, T=4, k=2, H=64, inv=P, w=P, add=P, add_type=0, y=P, y_type=0)
    a.update(change)
    assert ds4.lib.ds4moe_combine(*a.values(), None) == EINVAL


@pytest.mark.parametrize("bad", [
    dict(n_experts=0), dict(n_experts=513), dict(n_out=0), dict(n_out=65537), dict(n_in=0), dict(n_in=48), dict(n_in=65568),
    dict(gated=2), dict(gated=-1)])
def test_bad_expert_configs(ds4, bad):
    f = dict(n_experts=2, n_out=64, n_in=64, gated=0)
    f.update(bad)
    h = C.c_void_p()
    assert ds4.lib.ds4moe_mxfp4_create(C.byref(ds4.ds4moe_mxfp4_config(*f.values())), 0, C.byref(h)) == EINVAL and not h.value


def test_null_expert_handles(ds4, monkeypatch):
    assert ds4.lib.ds4moe_mxfp4_create(None, 0, None) == EINVAL
    assert ds4.lib.ds4moe_mxfp4_load(None, P, P, None, None, None) == EINVAL
    assert ds4.lib.ds4moe_mxfp4_product(None, P, P, 1, None, P, 0, 64, None, None) == EINVAL
    assert ds4.lib.ds4moe_mxfp4_sync_status(None) == EINVAL
    ds4.lib.ds4moe_mxfp4_destroy(None)
    monkeypatch.setenv("DS4MOE_FAULT", "alloc")
    h = C.c_void_p()
    assert ds4.lib.ds4moe_mxfp4_create(C.byref(ds4.ds4moe_mxfp4_config(1, 32, 32, 0)), 0, C.byref(h)) == 2 and not h.value


def test_binding_refuses_host_tensors(ds4):
    torch = pytest.importorskip("torch")
    with pytest.raises(ValueError, match="CUDA device"):
        ds4.Router(8, 2).route(torch.zeros(2, 8))
    with pytest.raises(ValueError, match="CUDA device"):
        ds4.mxfp4_quantize(torch.zeros(2, 64))
    with pytest.raises(ValueError, match="CUDA device"):
        ds4.mxfp4_dequantize(torch.zeros(2, 32, dtype=torch.uint8), torch.zeros(2, 2, dtype=torch.uint8))
    with pytest.raises(ValueError, match="CUDA device"):
        ds4.combine(torch.zeros(4, 8), torch.zeros(2, 2, dtype=torch.int32), torch.zeros(2, 2))
    with pytest.raises(ValueError):
        ds4.Router(8, 2, score="tanh")
    with pytest.raises(ValueError):
        ds4.Router(8, 2, group_score="mean")


# ------------------------------------------------------------------ the plain forms themselves
def test_ladder_rounding_by_hand():
    a = [0.0, 0.2, 0.25, 0.26, 0.5, 0.74, 0.75, 1.25, 1.26, 1.75, 2.5, 2.51, 3.5, 3.49, 5.0, 5.01, 6.0, 7.9]
    want = [0, 0, 0, 1, 1, 1, 2, 2, 3, 4, 4, 5, 6, 5, 6, 7, 7, 7]
    assert ref.mx_round(np.array(a)).tolist() == want


def test_quantize_by_hand():
    x = np.zeros((1, 32))
    x[0, :6] = [6.0, -3.0, 0.5, 1.0, -0.25, 5.0]
    c, s = ref.quantize(x)
    assert s[0, 0] == 127 and c[0, :3].tolist() == [0x7 | 0xD << 4, 0x1 | 0x2 << 4, 0x8 | 0x6 << 4]
    c, s = ref.quantize(x * 2.0 ** -9)
    assert s[0, 0] == 118 and ref.dequantize(c, s)[0, 1] == -3.0 * 2.0 ** -9
    assert ref.mx_scale(np.array([0.0, 1.0, 4.0, 3.99, 2.0 ** -130, np.inf, np.nan])).tolist() == [0, 125, 127, 126, 0, 255, 255]


def test_route_by_hand():
    torch = pytest.importorskip("torch")
    idx, w = ref.route(torch.tensor([[0.0, np.log(3.0), 0.0, -np.inf]]), 2, "softmax")
    assert idx.tolist() == [[1, 0]] and np.allclose(w, [[0.75, 0.25]])
    idx, w = ref.route(torch.tensor([[0.0, 1.0, 5.0, 5.0]]), 2, "sigmoid", torch.tensor([9.0, 0.0, 0.0, 0.0]), renormalise=False)
    assert idx.tolist() == [[0, 2]] and np.allclose(w[0, 0], 0.5)
    # the second group's sum of two is larger than the first's, whose best value is the largest
    idx, w = ref.route(torch.tensor([[3.0, -9.0, 2.0, 2.0]]), 1, "sigmoid", None, 2, 1, "top2")
    assert idx.tolist() == [[2]] and w.tolist() == [[1.0]]
    off, st, ss, inv = ref.permute(np.array([[2, 0], [-1, -1], [0, 2]]), 3)
    assert off.tolist() == [0, 2, 2, 4] and st.tolist() == [0, 2, 0, 2] and ss.tolist() == [1, 0, 0, 1]
    assert inv.tolist() == [2, 0, -1, -1, 1, 3]
