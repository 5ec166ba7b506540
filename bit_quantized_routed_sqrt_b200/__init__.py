"""Thin ctypes binding of ``libds4moe.so``: the routed Q2_K mixture-of-experts layer.

Every function mirrors one ``extern "C"`` entry point of ``include/ds4moe.h`` under
the same name and only marshals arguments (torch tensors become device pointers,
torch's current stream becomes the ``cuda_stream`` argument).  All arithmetic runs
in the library's CUDA kernels; there is no fallback: importing this package fails
if the library has not been built, and every call raises on a non-OK status.
"""
from __future__ import annotations

import ctypes as C
import os
from typing import Optional

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libds4moe.so")
HEADER = os.path.join(os.path.dirname(_HERE), "include", "ds4moe.h")

FLAG_FORCE_DECODE = 0x1
FLAG_FORCE_PREFILL = 0x2
FLAG_PROFILE = 0x4
FLAG_TRACE = 0x8
FLAG_TEST_TIMEOUT = 0x10
ROUTE_STATIC_MAX_TOKENS = 256
F32, BF16, F16, MXFP4 = 0, 1, 2, 3
SCORES = {"softmax": 0, "sigmoid": 1, "sqrt_softplus": 2}
GROUP_SCORES = {"max": 0, "top2": 1}
INT_MAX = 2 ** 31 - 1

STATUS = {0: "DS4MOE_OK", 1: "DS4MOE_EINVAL", 2: "DS4MOE_ENOMEM", 3: "DS4MOE_ECUDA",
          4: "DS4MOE_ESTATE", 5: "DS4MOE_ETIMEOUT", 6: "DS4MOE_EDEVICE"}

if not os.path.exists(LIB_PATH):
    raise ImportError("libds4moe.so is not built (run __graft_entry__.build()); "
                      "this package has no CPU fallback")


class ds4moe_config(C.Structure):
    _fields_ = [("hidden", C.c_int32), ("n_experts", C.c_int32), ("top_k", C.c_int32),
                ("inter", C.c_int32), ("shared_inter", C.c_int32), ("max_tokens", C.c_int32),
                ("flags", C.c_uint32)]


class ds4moe_router(C.Structure):
    _fields_ = [("n_experts", C.c_int32), ("top_k", C.c_int32), ("score", C.c_int32), ("n_groups", C.c_int32),
                ("topk_groups", C.c_int32), ("group_score", C.c_int32), ("renormalise", C.c_int32), ("scale", C.c_float)]


class ds4moe_mxfp4_config(C.Structure):
    _fields_ = [("n_experts", C.c_int32), ("n_out", C.c_int32), ("n_in", C.c_int32), ("gated", C.c_int32)]


class ds4moe_stats(C.Structure):
    _fields_ = [("router_fallback_tokens", C.c_int64), ("last_path", C.c_int32),
                ("last_tokens", C.c_int32), ("n_stages", C.c_int32), ("stage_ms", C.c_float * 8)]


lib = C.CDLL(LIB_PATH)
_vp, _i32 = C.c_void_p, C.c_int32
lib.ds4moe_create.argtypes = [C.POINTER(ds4moe_config), C.c_int, C.POINTER(_vp)]
lib.ds4moe_destroy.argtypes = [_vp]
lib.ds4moe_destroy.restype = None
lib.ds4moe_load_q2k_experts.argtypes = [_vp] * 10
lib.ds4moe_route.argtypes = [_vp, _vp, _i32, _vp, _vp, _vp, _vp, _vp, _vp, _vp]
lib.ds4moe_route_static.argtypes = [_vp, _vp, _i32, _vp, _vp, _vp, _vp, _vp, _vp, _vp]
lib.ds4moe_forward.argtypes = [_vp, _vp, _i32, _vp, _vp]
lib.ds4moe_forward_host.argtypes = [_vp, _vp, _i32, _vp, _vp]
lib.ds4moe_rms_renorm.argtypes = [_vp, _i32, _i32, _vp, _vp]
lib.ds4moe_score_eval.argtypes = [_vp, _i32, _vp, _i32, _vp]
lib.ds4moe_export_q2k.argtypes = [_vp, _i32, _i32, _vp]
lib.ds4moe_sync_status.argtypes = [_vp]
lib.ds4moe_get_stats.argtypes = [_vp, C.POINTER(ds4moe_stats)]
lib.ds4moe_get_trace.argtypes = [_vp, _vp, _i32, C.POINTER(_i32), _vp]
lib.ds4moe_status_string.argtypes = [C.c_int]
lib.ds4moe_status_string.restype = C.c_char_p
lib.ds4moe_last_error.argtypes = [_vp]
lib.ds4moe_last_error.restype = C.c_char_p
_i64, _sz = C.c_int64, C.c_size_t
lib.ds4moe_route_logits_workspace.argtypes = [C.POINTER(ds4moe_router), _i32]
lib.ds4moe_route_logits_workspace.restype = _sz
lib.ds4moe_route_logits.argtypes = [C.POINTER(ds4moe_router), _vp, _i32, _i64, _i32] + [_vp] * 8 + [_sz, _vp]
lib.ds4moe_mxfp4_quantize.argtypes = [_vp, _i32, _i64, _i32, _i32, _vp, _i32, _i32, _vp, _vp, _vp]
lib.ds4moe_mxfp4_dequantize.argtypes = [_vp, _vp, _i32, _i32, _vp, _i32, _i64, _vp]
lib.ds4moe_combine.argtypes = [_vp, _i32, _i64, _i32, _i32, _i32, _vp, _vp, _vp, _i32, _vp, _i32, _vp]
lib.ds4moe_mxfp4_create.argtypes = [C.POINTER(ds4moe_mxfp4_config), C.c_int, C.POINTER(_vp)]
lib.ds4moe_mxfp4_destroy.argtypes = [_vp]
lib.ds4moe_mxfp4_destroy.restype = None
lib.ds4moe_mxfp4_load.argtypes = [_vp] * 6
lib.ds4moe_mxfp4_product.argtypes = [_vp, _vp, _vp, _i32, _vp, _vp, _i32, _i64, _vp, _vp]
lib.ds4moe_mxfp4_sync_status.argtypes = [_vp]
lib.ds4moe_mxfp4_last_error.argtypes = [_vp]
lib.ds4moe_mxfp4_last_error.restype = C.c_char_p
for _n in ("ds4moe_route_logits", "ds4moe_mxfp4_quantize", "ds4moe_mxfp4_dequantize", "ds4moe_combine", "ds4moe_mxfp4_create",
           "ds4moe_mxfp4_load", "ds4moe_mxfp4_product", "ds4moe_mxfp4_sync_status"):
    getattr(lib, _n).restype = C.c_int
for _n in ("ds4moe_create", "ds4moe_load_q2k_experts", "ds4moe_route", "ds4moe_route_static", "ds4moe_forward", "ds4moe_forward_host",
           "ds4moe_rms_renorm", "ds4moe_score_eval", "ds4moe_export_q2k", "ds4moe_sync_status", "ds4moe_get_stats",
           "ds4moe_get_trace"):
    getattr(lib, _n).restype = C.c_int


class Ds4MoeError(RuntimeError):
    pass


def _check(rc: int, handle=None, what: str = ""):
    if rc != 0:
        detail = lib.ds4moe_last_error(handle).decode() if handle else ""
        raise Ds4MoeError("%s failed: %s (%s) %s" % (what, STATUS.get(rc, rc),
                                                   lib.ds4moe_status_string(rc).decode(), detail))


def _ptr(t) -> Optional[int]:
    """Device/host address of a torch tensor or numpy array (None stays None)."""
    if t is None:
        return None
    if hasattr(t, "data_ptr"):
        return t.data_ptr()
    return t.ctypes.data


def _stream(stream) -> Optional[int]:
    if stream is not None:
        return int(stream)
    import torch
    return torch.cuda.current_stream().cuda_stream


def ds4moe_status_string(status: int) -> str:
    return lib.ds4moe_status_string(status).decode()


def ds4moe_rms_renorm(y, T: int, H: int, x_out, stream=None):
    _check(lib.ds4moe_rms_renorm(_ptr(y), T, H, _ptr(x_out), _stream(stream)), None, "ds4moe_rms_renorm")


def ds4moe_score_eval(logits, n: int, scores, variant: int = 0, stream=None):
    _check(lib.ds4moe_score_eval(_ptr(logits), n, _ptr(scores), variant, _stream(stream)), None, "ds4moe_score_eval")


# -- operators beside the layer ------------------------------------------------------
# The ds4moe_* functions take what the C calls take (tensors or addresses); the classes and the
# functions below them read types, sizes and the device from torch tensors and refuse, with a
# ValueError, tensors of another type, shape, layout or device than the call needs.

def ds4moe_route_logits_workspace(router: ds4moe_router, T: int) -> int:
    return lib.ds4moe_route_logits_workspace(C.byref(router), T)


def ds4moe_route_logits(router: ds4moe_router, logits, logits_type, ld, T, bias, topk_idx, topk_w, offsets=None,
                        sorted_token=None, sorted_slot=None, inv_pos=None, workspace=None, workspace_bytes=0, stream=None):
    _check(lib.ds4moe_route_logits(C.byref(router), _ptr(logits), logits_type, ld, T, _ptr(bias), _ptr(topk_idx),
                                   _ptr(topk_w), _ptr(offsets), _ptr(sorted_token), _ptr(sorted_slot), _ptr(inv_pos),
                                   _ptr(workspace), workspace_bytes, _stream(stream)), None, "ds4moe_route_logits")


def ds4moe_mxfp4_quantize(x, x_type, ld, rows, K, inv_pos, top_k, out_rows, codes, scales, stream=None):
    _check(lib.ds4moe_mxfp4_quantize(_ptr(x), x_type, ld, rows, K, _ptr(inv_pos), top_k, out_rows, _ptr(codes),
                                     _ptr(scales), _stream(stream)), None, "ds4moe_mxfp4_quantize")


def ds4moe_mxfp4_dequantize(codes, scales, rows, K, out, out_type, ld, stream=None):
    _check(lib.ds4moe_mxfp4_dequantize(_ptr(codes), _ptr(scales), rows, K, _ptr(out), out_type, ld, _stream(stream)),
           None, "ds4moe_mxfp4_dequantize")


def ds4moe_combine(o, o_type, o_rows, T, top_k, H, inv_pos, topk_w, add, add_type, y, y_type, stream=None):
    _check(lib.ds4moe_combine(_ptr(o), o_type, o_rows, T, top_k, H, _ptr(inv_pos), _ptr(topk_w), _ptr(add), add_type,
                              _ptr(y), y_type, _stream(stream)), None, "ds4moe_combine")


def _check_mxfp4(rc: int, handle, what: str):
    if rc != 0:
        detail = lib.ds4moe_mxfp4_last_error(handle).decode() if handle else ""
        raise Ds4MoeError("%s failed: %s (%s) %s" % (what, STATUS.get(rc, rc),
                                                   lib.ds4moe_status_string(rc).decode(), detail))


def ds4moe_mxfp4_create(cfg: ds4moe_mxfp4_config, device: int) -> int:
    h = _vp()
    _check_mxfp4(lib.ds4moe_mxfp4_create(C.byref(cfg), device, C.byref(h)), None, "ds4moe_mxfp4_create")
    return h


def ds4moe_mxfp4_destroy(handle):
    lib.ds4moe_mxfp4_destroy(handle)


def ds4moe_mxfp4_load(handle, codes, scales, up_codes=None, up_scales=None, stream=None):
    _check_mxfp4(lib.ds4moe_mxfp4_load(handle, _ptr(codes), _ptr(scales), _ptr(up_codes), _ptr(up_scales),
                                       _stream(stream)), handle, "ds4moe_mxfp4_load")


def ds4moe_mxfp4_product(handle, a_codes, a_scales, rows, offsets, out, out_type, ld, out_scales=None, stream=None):
    _check_mxfp4(lib.ds4moe_mxfp4_product(handle, _ptr(a_codes), _ptr(a_scales), rows, _ptr(offsets), _ptr(out), out_type,
                                          ld, _ptr(out_scales), _stream(stream)), handle, "ds4moe_mxfp4_product")


def ds4moe_mxfp4_sync_status(handle):
    _check_mxfp4(lib.ds4moe_mxfp4_sync_status(handle), handle, "ds4moe_mxfp4_sync_status")


def ds4moe_mxfp4_last_error(handle) -> str:
    return lib.ds4moe_mxfp4_last_error(handle).decode()


_torch = None
_types, _dtypes = {}, {}
_raw_stream = _current_device = None


def _bind_torch():
    """What the functions below take from torch, looked up once."""
    global _torch, _raw_stream, _current_device
    import torch
    _types.update({torch.float32: F32, torch.bfloat16: BF16, torch.float16: F16})
    _dtypes.update(int32=torch.int32, uint8=torch.uint8, float32=torch.float32)
    # the address of a device's current stream without a Stream object (3 us a call less)
    _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
        lambda index: torch.cuda.current_stream(index).cuda_stream)
    _current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
    _torch = torch


def _type_of(t, what: str) -> int:
    code = _types.get(t.dtype)
    if code is None:
        raise ValueError("%s must be float32, bfloat16 or float16, not %s" % (what, t.dtype))
    return code


def _rows_of(t, what: str):
    """(rows, width, elements between rows) of a matrix whose rows are contiguous."""
    shape = t.shape
    if len(shape) != 2:
        raise ValueError("%s must have two dimensions" % what)
    rows, width = shape
    ld, step = t.stride()
    if rows <= 1:
        ld = width
    if (width > 1 and step != 1) or ld < width:
        raise ValueError("%s must have contiguous rows, one behind the other" % what)
    return rows, width, ld


def _fits(sizes: int):
    """Refuses sizes that the C calls' 32-bit arguments cannot hold; sizes: all of them, or-ed."""
    if sizes > INT_MAX:
        raise ValueError("sizes must be at most 2^31 - 1")


def _flat(t, dtype: str, n: int, what: str, device):
    """The address of a contiguous tensor of n elements of the type on the device (None stays None)."""
    if t is None:
        return None
    if t.dtype is not _dtypes[dtype] or t.numel() != n or not t.is_contiguous() or t.device != device:
        raise ValueError("%s must be a contiguous %s tensor of %d elements on %s" % (what, dtype, n, device))
    return t.data_ptr()


def _device_of(t, what: str):
    """The tensor's CUDA device."""
    if _torch is None:
        _bind_torch()
    if not t.is_cuda:
        raise ValueError("%s must be on a CUDA device" % what)
    return t.device


def _run(device, call, *args):
    """call(*args, stream) on the device and its current stream; the current device is the same afterwards."""
    index = device.index
    if _current_device() == index:
        return call(*args, _raw_stream(index))
    with _torch.cuda.device(index):
        return call(*args, _raw_stream(index))


class Routing:
    """Outputs and workspace of Router.route for T tokens (Router.buffers); its tensors stay the same."""

    def __setattr__(self, name, value):
        if hasattr(self, "addresses"):
            raise AttributeError("the buffers of a Routing are fixed")
        object.__setattr__(self, name, value)

    def __init__(self, router: "Router", T: int, device):
        import torch
        k, E = router.cfg.top_k, router.cfg.n_experts
        self.size = (T, k, E)
        self.topk_idx = torch.empty((T, k), dtype=torch.int32, device=device)
        self.topk_w = torch.empty((T, k), dtype=torch.float32, device=device)
        self.expert_offsets = torch.empty(E + 1, dtype=torch.int32, device=device)
        self.sorted_token = torch.empty(T * k, dtype=torch.int32, device=device)
        self.sorted_slot = torch.empty(T * k, dtype=torch.int32, device=device)
        self.inv_pos = torch.empty(T * k, dtype=torch.int32, device=device)
        n = ds4moe_route_logits_workspace(router.cfg, T)
        self.workspace = torch.empty(n, dtype=torch.uint8, device=device) if n else None

        self.addresses = (self.topk_idx.data_ptr(), self.topk_w.data_ptr(), self.expert_offsets.data_ptr(),
                          self.sorted_token.data_ptr(), self.sorted_slot.data_ptr(), self.inv_pos.data_ptr(),
                          self.workspace.data_ptr() if n else None, n)


class Router:
    """How experts are chosen and weighted (``ds4moe_router``), applied to router logits."""

    def __init__(self, n_experts: int, top_k: int, score: str = "softmax", n_groups: int = 1, topk_groups: int = 1,
                 group_score: str = "max", renormalise: bool = True, scale: float = 1.0):
        if score not in SCORES or group_score not in GROUP_SCORES:
            raise ValueError("score must be one of %s, group_score of %s" % (sorted(SCORES), sorted(GROUP_SCORES)))
        self.cfg = ds4moe_router(n_experts, top_k, SCORES[score], n_groups, topk_groups, GROUP_SCORES[group_score],
                                 int(bool(renormalise)), scale)

    def buffers(self, T: int, device="cuda") -> Routing:
        return Routing(self, T, device)

    def route(self, logits, bias=None, out: Optional[Routing] = None) -> Routing:
        """Routes the rows of logits [T, E] (rows may be strided); out: buffers of T tokens to write to."""
        device = _device_of(logits, "logits")
        T, E, ld = _rows_of(logits, "logits")
        code = _type_of(logits, "logits")
        _fits(T)
        if E != self.cfg.n_experts:
            raise ValueError("logits have %d columns for %d experts" % (E, self.cfg.n_experts))
        bias_at = _flat(bias, "float32", E, "bias", device)   # bias itself stays alive to the call
        if out is None:
            out = Routing(self, T, device)
        elif out.size != (T, self.cfg.top_k, E) or out.topk_idx.device != device:
            raise ValueError("out holds buffers of another size or device")
        _check(_run(device, lib.ds4moe_route_logits, C.byref(self.cfg), logits.data_ptr(), code, ld, T, bias_at,
                    *out.addresses), None, "ds4moe_route_logits")
        return out


def mxfp4_quantize(x, inv_pos=None, codes=None, scales=None):
    """(codes, scales) of the rows of x; with inv_pos [rows, k] (int32) row r goes to rows inv_pos[r, j]
    of codes / scales (rows * k of them where they are not given)."""
    device = _device_of(x, "x")
    rows, K, ld = _rows_of(x, "x")
    code = _type_of(x, "x")
    if K == 0 or K % 32:
        raise ValueError("the rows of x must have a multiple of 32 elements")
    k, places = 1, None
    if inv_pos is not None:
        if inv_pos.dim() != 2 or inv_pos.shape[0] != rows:
            raise ValueError("inv_pos must have a row for each row of x")
        k = inv_pos.shape[1]
        places = _flat(inv_pos, "int32", rows * k, "inv_pos", device)
    if codes is None:
        _fits(rows * k | K)
        codes = _torch.empty((rows * k, K // 2), dtype=_torch.uint8, device=device)
    out_rows = codes.shape[0]
    _fits(rows | K | k | out_rows)
    if scales is None:
        scales = _torch.empty((out_rows, K // 32), dtype=_torch.uint8, device=device)
    _check(_run(device, lib.ds4moe_mxfp4_quantize, x.data_ptr(), code, ld, rows, K, places, k, out_rows,
                _flat(codes, "uint8", out_rows * (K // 2), "codes", device),
                _flat(scales, "uint8", out_rows * (K // 32), "scales", device)), None, "ds4moe_mxfp4_quantize")
    return codes, scales


def mxfp4_dequantize(codes, scales, out=None):
    """The values of MXFP4 rows, in out (float32, bfloat16 or float16 [rows, K]; bfloat16 where it is not given:
    it and float32 hold every value exactly, but those of 2^128 and above, at scale bytes 253 and 254, are
    infinite)."""
    device = _device_of(codes, "codes")
    rows, half, _ = _rows_of(codes, "codes")
    K = 2 * half
    _fits(rows | K)
    if out is None:
        out = _torch.empty((rows, K), dtype=_torch.bfloat16, device=device)
    r, w, ld = _rows_of(out, "out")
    if r != rows or w != K or out.device != device:
        raise ValueError("out must be [%d, %d] on %s" % (rows, K, device))
    _check(_run(device, lib.ds4moe_mxfp4_dequantize, _flat(codes, "uint8", rows * half, "codes", device),
                _flat(scales, "uint8", rows * (K // 32), "scales", device), rows, K, out.data_ptr(), _type_of(out, "out"),
                ld), None, "ds4moe_mxfp4_dequantize")
    return out


def combine(o, inv_pos, topk_w, y=None, add=None):
    """y[t] = add[t] + sum_j topk_w[t, j] * o[inv_pos[t, j]] (a row outside o adds nothing); y is float32 where it
    is not given."""
    device = _device_of(o, "o")
    o_rows, H, ld = _rows_of(o, "o")
    if ld != H:
        raise ValueError("o must be contiguous")
    if topk_w.dim() != 2:
        raise ValueError("topk_w must be [T, k]")
    T, k = topk_w.shape
    _fits(T | k | H)
    if y is None:
        y = _torch.empty((T, H), dtype=_torch.float32, device=device)
    for t, what in ((y, "y"), (add, "add")):
        if t is not None and (t.shape != (T, H) or not t.is_contiguous() or t.device != device):
            raise ValueError("%s must be a contiguous [%d, %d] tensor on %s" % (what, T, H, device))
    _check(_run(device, lib.ds4moe_combine, o.data_ptr(), _type_of(o, "o"), o_rows, T, k, H,
                _flat(inv_pos, "int32", T * k, "inv_pos", device), _flat(topk_w, "float32", T * k, "topk_w", device),
                None if add is None else add.data_ptr(), F32 if add is None else _type_of(add, "add"), y.data_ptr(),
                _type_of(y, "y")), None, "ds4moe_combine")
    return y


class Mxfp4Experts:
    """One projection of E experts in MXFP4 (the ``ds4moe_mxfp4`` handle): W [E, n_out, n_in], or a gate and an up
    matrix whose product is silu(gate x) * (up x)."""

    def __init__(self, n_experts: int, n_out: int, n_in: int, gated: bool = False, device: Optional[int] = None):
        if device is None:
            import torch
            device = torch.cuda.current_device()
        self.h = None
        self.n_experts, self.n_out, self.n_in, self.gated = n_experts, n_out, n_in, bool(gated)
        self.h = ds4moe_mxfp4_create(ds4moe_mxfp4_config(n_experts, n_out, n_in, int(self.gated)), device)
        self.device = device

    def close(self):
        if getattr(self, "h", None):
            ds4moe_mxfp4_destroy(self.h)
            self.h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def _device_of(self, t, what):
        device = _device_of(t, what)
        if device.index != self.device:
            raise ValueError("%s is on %s, the experts on device %d" % (what, device, self.device))
        return device

    def load(self, codes, scales, up_codes=None, up_scales=None):
        """codes uint8 [E, n_out, n_in / 2] and scales uint8 [E, n_out, n_in / 32] on the device; a gated projection
        takes the gate's and the up matrix's."""
        if (up_codes is None) != (up_scales is None) or (up_codes is not None) != self.gated:
            raise ValueError("a gated projection takes two matrices, another takes one")
        device = self._device_of(codes, "codes")
        n = self.n_experts * self.n_out
        _check_mxfp4(_run(device, lib.ds4moe_mxfp4_load, self.h,
                          _flat(codes, "uint8", n * (self.n_in // 2), "codes", device),
                          _flat(scales, "uint8", n * (self.n_in // 32), "scales", device),
                          _flat(up_codes, "uint8", n * (self.n_in // 2), "up_codes", device),
                          _flat(up_scales, "uint8", n * (self.n_in // 32), "up_scales", device)), self.h, "ds4moe_mxfp4_load")

    def product(self, a_codes, a_scales, offsets=None, out=None, out_scales=None):
        """Rows of a [rows, n_in] in MXFP4, grouped by offsets int32 [E + 1] (None for one expert), times their
        experts' matrices.  out: [rows, n_out] of float32, bfloat16 (where it is not given) or float16, rows may be
        strided; or, with out_scales uint8 [rows, n_out / 32], the codes of MXFP4, uint8 [rows, n_out / 2] (made
        where they are not given).  Returns out."""
        device = self._device_of(a_codes, "a_codes")
        rows, half, _ = _rows_of(a_codes, "a_codes")
        _fits(rows)
        if half * 2 != self.n_in:
            raise ValueError("a_codes has rows of %d inputs, the experts take %d" % (half * 2, self.n_in))
        if out is None:
            out = _torch.empty((rows, self.n_out if out_scales is None else self.n_out // 2),
                               dtype=_torch.bfloat16 if out_scales is None else _torch.uint8, device=device)
        if out_scales is not None:
            to, ld, code = _flat(out, "uint8", rows * (self.n_out // 2), "out", device), self.n_out, MXFP4
        else:
            r, n, ld = _rows_of(out, "out")
            if r != rows or n != self.n_out or out.device != device:
                raise ValueError("out must be [%d, %d] on %s" % (rows, self.n_out, device))
            to, code = out.data_ptr(), _type_of(out, "out")
        _check_mxfp4(_run(device, lib.ds4moe_mxfp4_product, self.h, _flat(a_codes, "uint8", rows * half, "a_codes", device),
                          _flat(a_scales, "uint8", rows * (self.n_in // 32), "a_scales", device), rows,
                          _flat(offsets, "int32", self.n_experts + 1, "offsets", device), to, code, ld,
                          _flat(out_scales, "uint8", rows * (self.n_out // 32), "out_scales", device)), self.h,
                     "ds4moe_mxfp4_product")
        return out

    def sync_status(self):
        ds4moe_mxfp4_sync_status(self.h)


class Ds4Moe:
    """One layer on one device (the ``ds4moe`` handle)."""

    def __init__(self, hidden: int, n_experts: int, top_k: int, inter: int, shared_inter: int,
                 max_tokens: int, flags: int = 0, device: int = 0):
        self.cfg = ds4moe_config(hidden, n_experts, top_k, inter, shared_inter, max_tokens, flags)
        self.hidden, self.n_experts, self.top_k = hidden, n_experts, top_k
        self.inter, self.shared_inter, self.max_tokens = inter, shared_inter, max_tokens
        self.device = device
        h = _vp()
        _check(lib.ds4moe_create(C.byref(self.cfg), device, C.byref(h)), None, "ds4moe_create")
        self.h = h

    def close(self):
        if getattr(self, "h", None):
            lib.ds4moe_destroy(self.h)
            self.h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    # -- calls with the C names -------------------------------------------------
    def ds4moe_load_q2k_experts(self, gate, up, down, router, bias=None, shared_gate=None, shared_up=None,
                                shared_down=None, stream=None):
        """Host arrays (numpy) in the layouts of include/ds4moe.h."""
        import numpy as np
        keep = [np.ascontiguousarray(a) if a is not None else None
                for a in (gate, up, down, router, bias, shared_gate, shared_up, shared_down)]
        _check(lib.ds4moe_load_q2k_experts(self.h, *[_ptr(a) for a in keep], _stream(stream)), self.h,
               "ds4moe_load_q2k_experts")

    def load(self, lw, stream=None):
        """Load a ``synth.LayerWeights``-like object (fields gate, up, down, router, bias, shared_*)."""
        self.ds4moe_load_q2k_experts(lw.gate, lw.up, lw.down, lw.router, lw.bias, lw.shared_gate, lw.shared_up,
                                     lw.shared_down, stream)

    def ds4moe_route(self, x, T, topk_idx, topk_w, offsets=None, sorted_token=None, sorted_slot=None,
                     inv_pos=None, stream=None):
        _check(lib.ds4moe_route(self.h, _ptr(x), T, _ptr(topk_idx), _ptr(topk_w), _ptr(offsets),
                                _ptr(sorted_token), _ptr(sorted_slot), _ptr(inv_pos), _stream(stream)),
               self.h, "ds4moe_route")

    def ds4moe_route_static(self, x, T, topk_idx, topk_w, offsets, sorted_token, sorted_slot, inv_pos,
                            stream=None):
        _check(lib.ds4moe_route_static(self.h, _ptr(x), T, _ptr(topk_idx), _ptr(topk_w), _ptr(offsets),
                                       _ptr(sorted_token), _ptr(sorted_slot), _ptr(inv_pos), _stream(stream)),
               self.h, "ds4moe_route_static")

    def ds4moe_forward(self, x, T, y, stream=None):
        _check(lib.ds4moe_forward(self.h, _ptr(x), T, _ptr(y), _stream(stream)), self.h, "ds4moe_forward")

    def ds4moe_forward_host(self, x_host, T, y_host, stream=None):
        _check(lib.ds4moe_forward_host(self.h, _ptr(x_host), T, _ptr(y_host), _stream(stream)), self.h,
               "ds4moe_forward_host")

    def ds4moe_export_q2k(self, which: int, expert: int, out):
        _check(lib.ds4moe_export_q2k(self.h, which, expert, _ptr(out)), self.h, "ds4moe_export_q2k")

    def ds4moe_sync_status(self):
        _check(lib.ds4moe_sync_status(self.h), self.h, "ds4moe_sync_status")

    def ds4moe_get_stats(self) -> ds4moe_stats:
        s = ds4moe_stats()
        _check(lib.ds4moe_get_stats(self.h, C.byref(s)), self.h, "ds4moe_get_stats")
        return s

    def ds4moe_get_trace(self, max_records: int = 1 << 20):
        """Returns (records int64 [n, 4], unit_bounds int32 [7]) of the last batched-GEMV launch
        (record layout in include/ds4moe.h)."""
        import numpy as np
        out = np.zeros((max_records, 4), dtype=np.int64)
        n = C.c_int32()
        bounds = np.zeros(7, dtype=np.int32)
        _check(lib.ds4moe_get_trace(self.h, out.ctypes.data, max_records, C.byref(n), bounds.ctypes.data), self.h,
               "ds4moe_get_trace")
        return out[:n.value], bounds

    # -- torch conveniences (marshalling only) -----------------------------------
    def route(self, x):
        import torch
        T = x.shape[0]
        k = self.top_k
        dev = x.device
        idx = torch.empty((T, k), dtype=torch.int32, device=dev)
        w = torch.empty((T, k), dtype=torch.float32, device=dev)
        off = torch.empty(self.n_experts + 1, dtype=torch.int32, device=dev)
        st = torch.empty(T * k, dtype=torch.int32, device=dev)
        ss = torch.empty(T * k, dtype=torch.int32, device=dev)
        inv = torch.empty(T * k, dtype=torch.int32, device=dev)
        self.ds4moe_route(x, T, idx, w, off, st, ss, inv)
        return idx, w, off, st, ss, inv

    def forward(self, x, y=None):
        import torch
        T = x.shape[0]
        if y is None:
            y = torch.empty((T, self.hidden), dtype=torch.float32, device=x.device)
        self.ds4moe_forward(x, T, y)
        return y


def exported_symbols():
    """Names of the ``ds4moe_*`` functions declared in include/ds4moe.h."""
    import re
    src = open(HEADER).read()
    return sorted(set(re.findall(r"\b(ds4moe_[a-z_0-9]+)\s*\(", src)))
