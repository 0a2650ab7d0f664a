"""GB300 (sm_103a) routed-expert MoE layer: Python binding of libmnw_moe.so.

Argument marshalling only: every step runs in the library's CUDA kernels.
The function names are those of the C ABI in include/mnw_moe.h.  Tensors are
torch CUDA tensors; the current torch stream is used unless ``stream`` is given.
If the library is missing it is built with nvcc on first import; if that
fails, importing this package fails (there is no fallback path).
"""
from __future__ import annotations

import ctypes
import functools
import importlib.machinery
import importlib.util
import os
import warnings

import torch

from . import build as _build

_HERE = os.path.dirname(os.path.abspath(__file__))

MNW_OK = 0
FMT_BF16, FMT_INT8_G128, FMT_INT4_G128, FMT_NVFP4_G16 = 0, 1, 2, 3
ACT_BF16, ACT_INT8_G128, ACT_NVFP4_G16, ACT_F16_ROWS = 0, 1, 2, 3
KIND_GATE_UP, KIND_DOWN, KIND_GATE, KIND_UP = 0, 1, 2, 3
DEVERR_BAD_EXPERT_ID, DEVERR_TIMEOUT, DEVERR_BAD_LENGTH, DEVERR_BAD_PAGE, DEVERR_BAD_ADAPTER = 0x1, 0x2, 0x4, 0x8, 0x10
KV_BF16, KV_INT8, KV_INT4 = 0, 1, 2
ROPE_HALF, ROPE_INTERLEAVED = 0, 1
ROPE_SCALE_NONE, ROPE_SCALE_LINEAR, ROPE_SCALE_NTK, ROPE_SCALE_BY_PARTS = 0, 1, 2, 3
PATH_AUTO, PATH_TCGEN05, PATH_WARP_MMA, PATH_ROWS = 0, 1, 2, 3

# Symbols of include/mnw_moe.h, with their ctypes signatures.
_P, _I, _SZ, _U32P = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t, ctypes.c_void_p
_LL = ctypes.c_longlong
SIGNATURES = {
    "mnw_status_string": (ctypes.c_char_p, [_I]),
    "mnw_moe_layer_init": (_I, [_P, _P, _SZ, ctypes.POINTER(_P)]),
    "mnw_moe_layer_destroy": (None, [_P]),
    "mnw_moe_layer_info": (_I, [_P, _P, _P, _P, _P]),
    "mnw_moe_permute": (_I, [_P, _I, _I, _I, _P, _P, _P, _P, _I, _P, _U32P, _P]),
    "mnw_moe_quantize_act": (_I, [_I, _P, _I, _I, _P, _I, _P, _P, _P, _P]),
    "mnw_moe_permute_host": (_I, [_P, _I, _I, _I, _P, _P, _P, _U32P]),
    "mnw_moe_route_scratch_size": (_SZ, [_I, _I]),
    "mnw_moe_route": (_I, [_P, _P, _I, _I, _I, _I, _P, _P, _P, _P, _P, _P, _SZ, _U32P, _P]),
    "mnw_moe_workspace_size_routed": (_SZ, [_P, _I, _I, _I]),
    "mnw_moe_forward_routed": (_I, [_P, _I, _P, _P, _I, _I, _P, _P, _P, _P, _SZ, _P]),
    "mnw_moe_grouped_gemm_bf16": (_I, [_P, _I, _P, _P, _I, _P, _U32P, _P]),
    "mnw_moe_grouped_gemm_w8a16": (_I, [_P, _I, _P, _P, _I, _P, _U32P, _P]),
    "mnw_moe_grouped_gemm_w4a16": (_I, [_P, _I, _P, _P, _I, _P, _U32P, _P]),
    "mnw_moe_grouped_gemm_w8a16_f16rows": (_I, [_P, _I, _P, _P, _P, _I, _P, _U32P, _P]),
    "mnw_moe_grouped_gemm_w4a16_f16rows": (_I, [_P, _I, _P, _P, _P, _I, _P, _U32P, _P]),
    "mnw_moe_grouped_gemm_w8a8": (_I, [_P, _I, _P, _P, _P, _I, _P, _P, _U32P, _P]),
    "mnw_moe_grouped_gemm_w4a8": (_I, [_P, _I, _P, _P, _P, _I, _P, _P, _U32P, _P]),
    "mnw_moe_grouped_gemm_nvfp4": (_I, [_P, _I, _P, _P, _P, _P, _I, _P, _U32P, _P]),
    "mnw_moe_combine": (_I, [_P, _P, _P, _I, _I, _I, _P, _P]),
    "mnw_moe_workspace_size": (_SZ, [_P, _I, _I, _I]),
    "mnw_moe_forward": (_I, [_P, _I, _P, _P, _P, _I, _I, _P, _P, _SZ, _P]),
    "mnw_moe_workspace_error_word": (_P, [_P]),
    "mnw_moe_workspace_size_host": (_SZ, [_P, _I, _I, _I]),
    "mnw_moe_forward_host": (_I, [_P, _I, _P, _P, _P, _I, _I, _P, _P, _SZ, _P]),
    "mnw_moe_read_error": (_I, [_P, _P, _P]),
    "mnw_moe_set_gemm_path": (_I, [_I]),
    "mnw_moe_set_fused_activation": (_I, [_I]),
    "mnw_moe_set_host_routing": (_I, [_I]),
    "mnw_moe_silu_mul": (_I, [_P, _P, _SZ, _P, _P]),
    "mnw_moe_launch_count": (ctypes.c_uint64, []),
    "mnw_moe_forward_static": (_I, [_P, _I, _P, _P, _P, _I, _I, _P, _U32P, _P]),
    "mnw_moe_selftest_wait_timeout": (_I, [ctypes.c_uint32, _U32P, _U32P, _P]),
    "mnw_moe_selftest_polled_wait_timeout": (_I, [ctypes.c_uint32, _U32P, _U32P, _P]),
    "mnw_moe_selftest_counter_timeout": (_I, [ctypes.c_uint32, _U32P, ctypes.c_uint32, _U32P, _P]),
    "mnw_rmsnorm": (_I, [_P, _LL, _P, _P, _I, _I, ctypes.c_float, _P, _P, _P, _P, _P]),
    "mnw_kv_append": (_I, [_P, _LL, _P, _LL, _P, _LL, _I, _I, _I, _I, _I, _P, _I, _I, ctypes.c_float, _P, _P, _P, _P,
                           _I, _I, _I, _LL, _P, _I, _P, _P, _P, _U32P, _P]),
    "mnw_attn_paged_workspace_size": (_SZ, [_I, _I, _I, _I, _I]),
    "mnw_attn_paged": (_I, [_P, _LL, _I, _I, _I, _I, _I, _P, _P, _P, _P, _I, _I, _I, _LL, _P, _I, _P, _P, _I,
                            ctypes.c_float, _P, _P, _P, _SZ, _U32P, _P]),
    "mnw_kv_values": (_I, [_P, _P, _I, _I, _I, _I, _I, _LL, _P, _P]),
    "mnw_lora_workspace_size": (_SZ, [_I, _I, _I, _I]),
    "mnw_lora_add": (_I, [_P, _LL, _P, _P, _P, _P, _I, _I, _P, _I, _I, _I, _P, _LL, _P, _LL, _P, _SZ, _U32P, _P]),
    "mnw_rope_frequencies": (_I, [_I, ctypes.c_double, _I, ctypes.c_double, ctypes.c_double, ctypes.c_double,
                                  ctypes.c_double, _P, _P]),
    "mnw_attn_workspace_size": (_SZ, [_I, _I, _I, _I]),
    "mnw_attn_prefill": (_I, [_P, _P, _P, _I, _I, _I, _I, _I, _I, ctypes.c_float, _P, _P, _SZ, _U32P, _P]),
}

_lib = None


def lib_path() -> str:
    return _build.LIB


def load() -> ctypes.CDLL:
    """Load (building first if needed) libmnw_moe.so."""
    global _lib
    if _lib is None:
        path = _build.build()
        lib = ctypes.CDLL(path)
        for name, (res, args) in SIGNATURES.items():
            fn = getattr(lib, name)
            fn.restype = res
            fn.argtypes = args
        _lib = lib
    return _lib


_calls = None
_CALLS = ("kv_append", "attn_paged", "kv_values", "lora_add")


class _NoCalls:
    """In the binding's place where there is none: leaves every call to the Python form."""

    def __getattr__(self, name):
        if name not in _CALLS:
            raise AttributeError(name)
        return lambda *args: NotImplemented


def _load_calls():
    """The native form of the paged cache's and the adapters' calls (csrc/mnw_calls.cpp), bound to the library.  Where it
    could not be compiled or loaded, says so once and leaves the calls to the Python form."""
    global _calls
    lib = load()
    path = _build.calls_path()
    try:
        if not os.path.exists(path):
            with open(_build.calls_failed()) as f:
                raise ImportError(f.read())
        spec = importlib.util.spec_from_loader("mnw_calls", importlib.machinery.ExtensionFileLoader("mnw_calls", path))
        mod = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(mod)
    except (ImportError, OSError) as e:
        warnings.warn(f"the calls on the paged cache and the adapters go through Python (7 to 14 us more of the host's time each): {e}",
                      RuntimeWarning, stacklevel=3)
        _calls = _NoCalls()
        return _calls
    mod.bind(*(ctypes.cast(getattr(lib, f), ctypes.c_void_p).value for f in (
        "mnw_kv_append", "mnw_attn_paged", "mnw_attn_paged_workspace_size", "mnw_kv_values", "mnw_lora_add", "mnw_lora_workspace_size")))
    _calls = mod
    return mod


class MnwError(RuntimeError):
    pass


def _check(rc: int, what: str):
    if rc != MNW_OK:
        msg = load().mnw_status_string(rc).decode()
        raise MnwError(f"{what}: {msg} (status {rc})")


def _ptr(t):
    if t is None:
        return None
    if not t.is_cuda:
        raise MnwError("expected a CUDA tensor")
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


class Layer:
    """An expert blob (device uint8 tensor) described to the library.  The
    blob tensor is kept alive by this object."""

    def __init__(self, blob: torch.Tensor, header: bytes):
        self.blob = blob
        self.header = bytes(header)
        h = ctypes.create_string_buffer(self.header, len(self.header))
        out = ctypes.c_void_p()
        _check(load().mnw_moe_layer_init(h, _ptr(blob), blob.numel(), ctypes.byref(out)), "mnw_moe_layer_init")
        self.handle = out
        fmt, E, H, I = (ctypes.c_int() for _ in range(4))
        _check(load().mnw_moe_layer_info(self.handle, ctypes.byref(fmt), ctypes.byref(E), ctypes.byref(H),
                                         ctypes.byref(I)), "mnw_moe_layer_info")
        self.wfmt, self.E, self.H, self.I = fmt.value, E.value, H.value, I.value

    def __del__(self):
        if getattr(self, "handle", None) and _lib is not None:
            _lib.mnw_moe_layer_destroy(self.handle)
            self.handle = None


def mnw_moe_permute(ids, E, x=None, stream=None, err=None):
    """Returns (expert_offsets [E+1], sorted_assign [P], assign_pos [P], x_perm or None)."""
    T, k = ids.shape
    P = T * k
    dev = ids.device
    offsets = torch.empty(E + 1, dtype=torch.int32, device=dev)
    sorted_assign = torch.empty(P, dtype=torch.int32, device=dev)
    assign_pos = torch.empty(P, dtype=torch.int32, device=dev)
    x_perm = None
    H = 0
    if x is not None:
        H = x.shape[1]
        x_perm = torch.empty((P, H), dtype=x.dtype, device=dev)
    _check(load().mnw_moe_permute(_ptr(ids), T, k, E, _ptr(offsets), _ptr(sorted_assign), _ptr(assign_pos),
                                  _ptr(x), H, _ptr(x_perm), _ptr(err), _stream(stream)), "mnw_moe_permute")
    return offsets, sorted_assign, assign_pos, x_perm


def mnw_moe_route(x, w_router, k, scratch=None, stream=None, err=None):
    """GPU routing fused with the permutation (see include/mnw_moe.h).
    x: bf16 [T, H]; w_router: bf16 [E, H].  Returns (ids int32 [T,k], w f32
    [T,k], expert_offsets, sorted_assign, assign_pos, logits f32 [T,E]).
    scratch: a uint8 device tensor reused across calls (zero-filled when new)."""
    T, H = x.shape
    E = w_router.shape[0]
    dev = x.device
    need = load().mnw_moe_route_scratch_size(T, E)
    if scratch is None:
        scratch = torch.zeros(need + 256, dtype=torch.uint8, device=dev)
    base = (-scratch.data_ptr()) % 256
    view = scratch[base:base + need]
    ids = torch.empty((T, k), dtype=torch.int32, device=dev)
    w = torch.empty((T, k), dtype=torch.float32, device=dev)
    off = torch.empty(E + 1, dtype=torch.int32, device=dev)
    sa = torch.empty(T * k, dtype=torch.int32, device=dev)
    pos = torch.empty(T * k, dtype=torch.int32, device=dev)
    _check(load().mnw_moe_route(_ptr(x), _ptr(w_router), T, H, E, k, _ptr(ids), _ptr(w), _ptr(off), _ptr(sa),
                                _ptr(pos), _ptr(view), need, _ptr(err), _stream(stream)), "mnw_moe_route")
    cb = (((1 + (T + 15) // 16) * 4 + 255) // 256) * 256  # the counters come first
    logits = view[cb:cb + T * E * 4].view(torch.float32).view(T, E)
    return ids, w, off, sa, pos, logits


def mnw_moe_workspace_size_routed(layer, act, T, k) -> int:
    return load().mnw_moe_workspace_size_routed(layer.handle, act, T, k)


def mnw_moe_forward_routed(layer, act, x, w_router, k, ws=None, out=None, stream=None):
    """The layer with GPU routing; returns (out bf16 [T,H], ids int32 [T,k], w f32 [T,k])."""
    T = x.shape[0]
    if ws is None:
        n = mnw_moe_workspace_size_routed(layer, act, T, k)
        ws = torch.empty(n + 256, dtype=torch.uint8, device=x.device)
    base = (-ws.data_ptr()) % 256
    ids = torch.empty((T, k), dtype=torch.int32, device=x.device)
    w = torch.empty((T, k), dtype=torch.float32, device=x.device)
    if out is None:
        out = torch.empty((T, layer.H), dtype=torch.bfloat16, device=x.device)
    _check(load().mnw_moe_forward_routed(layer.handle, act, _ptr(x), _ptr(w_router), T, k, _ptr(ids), _ptr(w),
                                         _ptr(out), ctypes.c_void_p(ws.data_ptr() + base), ws.numel() - base,
                                         _stream(stream)), "mnw_moe_forward_routed")
    return out, ids, w


def mnw_moe_permute_host(ids, E):
    """Host-side permutation (numpy int32 [T, k] in): (offsets, sorted_assign,
    assign_pos, dropped) as numpy arrays, the same as mnw_moe_permute's."""
    import numpy as np
    ids = np.ascontiguousarray(ids, dtype=np.int32)
    T, k = ids.shape
    P = T * k
    off = np.zeros(E + 1, np.int32)
    sa = np.zeros(P, np.int32)
    pos = np.zeros(P, np.int32)
    dropped = ctypes.c_uint32()
    p = lambda a: a.ctypes.data_as(ctypes.c_void_p)
    _check(load().mnw_moe_permute_host(p(ids), T, k, E, p(off), p(sa), p(pos), ctypes.byref(dropped)),
           "mnw_moe_permute_host")
    return off, sa, pos, int(dropped.value)


def mnw_moe_quantize_act(act, x, row_index=None, index_div=1, rows=None, stream=None):
    """INT8_G128 -> (codes int8 [R,K], scales f32 [R,K/128]);
    NVFP4_G16 -> (codes u8 [R,K/2], sf u8 [R,K/16], outer f32 [R]);
    F16_ROWS -> (codes fp16 [R,K], factor f32 [R])."""
    R = rows if rows is not None else (row_index.numel() if row_index is not None else x.shape[0])
    K = x.shape[1]
    dev = x.device
    if act == ACT_F16_ROWS:
        codes = torch.empty((R, K), dtype=torch.float16, device=dev)
        outer = torch.empty((R,), dtype=torch.float32, device=dev)
        _check(load().mnw_moe_quantize_act(act, _ptr(x), R, K, _ptr(row_index), index_div, _ptr(codes), None,
                                           _ptr(outer), _stream(stream)), "mnw_moe_quantize_act")
        return codes, outer
    if act == ACT_INT8_G128:
        codes = torch.empty((R, K), dtype=torch.int8, device=dev)
        scales = torch.empty((R, K // 128), dtype=torch.float32, device=dev)
        outer = None
    else:
        codes = torch.empty((R, K // 2), dtype=torch.uint8, device=dev)
        scales = torch.empty((R, K // 16), dtype=torch.uint8, device=dev)
        outer = torch.empty((R,), dtype=torch.float32, device=dev)
    _check(load().mnw_moe_quantize_act(act, _ptr(x), R, K, _ptr(row_index), index_div, _ptr(codes), _ptr(scales),
                                       _ptr(outer), _stream(stream)), "mnw_moe_quantize_act")
    return (codes, scales) if act == ACT_INT8_G128 else (codes, scales, outer)


def mnw_moe_set_fused_activation(fused: bool) -> None:
    _check(load().mnw_moe_set_fused_activation(1 if fused else 0), "mnw_moe_set_fused_activation")


def mnw_moe_set_host_routing(on: bool) -> None:
    _check(load().mnw_moe_set_host_routing(1 if on else 0), "mnw_moe_set_host_routing")


def mnw_moe_silu_mul(g, u, stream=None):
    """bf16(SiLU(g) * u) of two bf16 tensors of the same shape."""
    h = torch.empty_like(g)
    _check(load().mnw_moe_silu_mul(_ptr(g), _ptr(u), g.numel(), _ptr(h), _stream(stream)), "mnw_moe_silu_mul")
    return h


def mnw_attn_prefill(q, k, v, blk: int, scale: float, out=None, ws=None, err=None, stream=None):
    """Block attention of bf16 q [B, T, Hq, d] over k, v [B, T, Hkv, d]; key j
    is allowed for token t when j // blk <= t // blk.  Returns out [B, T, Hq, d]."""
    B, T, Hq, d = q.shape
    Hkv = k.shape[2]
    L = load()
    if out is None:
        out = torch.empty_like(q)
    if ws is None:
        ws = torch.empty((max(1, L.mnw_attn_workspace_size(B, T, Hkv, d)),), dtype=torch.uint8, device=q.device)
    _check(L.mnw_attn_prefill(_ptr(q), _ptr(k), _ptr(v), B, T, Hq, Hkv, d, int(blk), float(scale), _ptr(out),
                              _ptr(ws), ws.numel(), _ptr(err), _stream(stream)), "mnw_attn_prefill")
    return out


# ---- the decode step around the layer: norm, paged cache, attention ----
# The calls on the cache and the adapters' go through _calls where nothing is amiss; the Python below it takes the others:
# a stream of the caller's, and arguments that it refuses by name, among them tensors of another device than the current one.


def _need(t, dtype, what, dim=None):
    """Address of a CUDA tensor of the given type (and, with `dim`, that many dimensions, the last one contiguous)."""
    if not t.is_cuda or t.dtype is not dtype:
        raise MnwError(f"{what}: expected a CUDA tensor of {dtype}")
    if dim is not None and (t.dim() != dim or (t.stride(-1) != 1 and t.shape[-1] > 1)):
        raise MnwError(f"{what}: expected {dim} dimensions, the last one contiguous")
    return t.data_ptr()


def _whole(t, dtype, shape, what):
    """Address of a contiguous CUDA tensor of the given type and shape."""
    if not t.is_cuda or t.dtype is not dtype or t.shape != shape or not t.is_contiguous():
        raise MnwError(f"{what}: expected a contiguous CUDA tensor of {dtype} and shape {tuple(shape)}")
    return t.data_ptr()


def _word(err):
    """Address of the device error word, the first four bytes of any CUDA tensor that has them (None where it has none)."""
    if err is None:
        return None
    if not err.is_cuda or 0 < err.numel() * err.element_size() < 4 or err.data_ptr() % 4:
        raise MnwError("err: expected a CUDA tensor that begins with a 32-bit word")
    return err.data_ptr()


def _new(shape, dtype, device, stream):
    """A device tensor for results written on `stream`: allocated under it, so its memory is reused in its order."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


# the current stream's handle without a stream object (2 us less on a decode call of 10)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _stream_of(t, stream):
    """The handle to launch on: the given stream's, or the current one's.  The library launches on the current device."""
    device = t.get_device()
    if _current_device() != device or (stream is not None and getattr(stream, "device_index", device) != device):
        raise MnwError(f"the tensors are on device {device}, which has to be the current device and the stream's")
    if stream is not None:
        return stream.cuda_stream
    return _raw_stream(device) if _raw_stream else torch.cuda.current_stream(t.device).cuda_stream


def _one_device(t, **others):
    """Every tensor of a call has to be on tensor t's device: an address of another one is none here."""
    device = t.get_device()
    for what, o in others.items():
        if o is not None and o.get_device() != device:
            raise MnwError(f"{what}: on device {o.get_device()}, where the call's other tensors are on {device}")


# A call's scratch memory, straight from torch's caching allocator: allocated on the call's stream and given back behind
# the launches, so the next user on that stream comes after them (a tensor for it costs 4 us of the host's time more).
_raw_alloc = getattr(torch._C, "_cuda_cudaCachingAllocator_raw_alloc", None)
_raw_delete = getattr(torch._C, "_cuda_cudaCachingAllocator_raw_delete", None)


def _scratch(n, t, stream, handle):
    """(address, what has to be given to _give_back) of n bytes for a call on the current device and the given stream."""
    if _raw_alloc and _raw_delete:
        p = _raw_alloc(n, handle)
        return p, p
    ws = _new((n,), torch.uint8, t.device, stream)
    return ws.data_ptr(), ws


def _give_back(held):
    if held.__class__ is int:
        _raw_delete(held)


def mnw_rmsnorm(x, weight, eps=1e-6, residual=None, residual_out=None, y=None, codes=None, scales=None, int8=False,
                stream=None, want_y=True):
    """Root-mean-square norm of bf16 x [T, H] with the residual's addition
    (see include/mnw_moe.h).  Returns (y bf16 [T, H], residual_out bf16 [T, H]
    or None, codes int8 [T, H] or None, scales f32 [T, H/128] or None); with
    int8 the last two are the INT8 groups of y, as mnw_moe_quantize_act gives
    them for the rows of y (the W8A8 / W4A8 GEMMs take them gathered by
    sorted_assign // k; the forward calls take y), and want_y=False leaves y
    itself out (None).  residual_out may be `residual` (in place)."""
    bf16 = torch.bfloat16
    xp = _need(x, bf16, "x", 2)
    shape = T, H = x.shape
    dev = x.device
    wp = _whole(weight, bf16, (H,), "weight")
    rp = ro = cp = sp = None
    if residual is not None:
        rp = _whole(residual, bf16, shape, "residual")
        if residual_out is None:
            residual_out = _new(shape, bf16, dev, stream)
            ro = residual_out.data_ptr()
        else:
            ro = _whole(residual_out, bf16, shape, "residual_out")
    elif residual_out is not None:
        raise MnwError("residual_out needs a residual")
    if y is not None:
        yp = _whole(y, bf16, shape, "y")
    elif want_y:
        y = _new(shape, bf16, dev, stream)
        yp = y.data_ptr()
    else:
        yp = None
    if int8 or codes is not None or scales is not None:
        if codes is None:
            codes = _new(shape, torch.int8, dev, stream)
        if scales is None:
            scales = _new((T, H // 128), torch.float32, dev, stream)
        cp = _whole(codes, torch.int8, shape, "codes")
        sp = _whole(scales, torch.float32, (T, H // 128), "scales")
    stride = x.stride(0) if T > 1 else max(H, x.stride(0) // 8 * 8)
    rc = load().mnw_rmsnorm(xp, stride, rp, wp, T, H, eps, ro, yp, cp, sp, _stream_of(x, stream))
    if rc:
        _check(rc, "mnw_rmsnorm")
    return y, residual_out, codes, scales


def _token_rows(t, what, d=None):
    """(address, tokens, heads, d, elements between tokens) of bf16 [T, heads, d], a token's heads contiguous."""
    shape, st = t.shape, t.stride()
    if not t.is_cuda or t.dtype is not torch.bfloat16 or len(shape) != 3 or (st[2] != 1 and shape[2] > 1):
        raise MnwError(f"{what}: expected a CUDA tensor of torch.bfloat16 with 3 dimensions, the last one contiguous")
    T, h, dd = shape
    if (d is not None and dd != d) or (h > 1 and st[1] != dd):
        raise MnwError(f"{what}: expected [T, heads, {d or 'd'}] with a token's heads contiguous")
    return t.data_ptr(), T, h, dd, st[0] if T > 1 else max(h * dd, st[0] // 8 * 8)


def _cache_args(k_cache, v_cache, k_scale, v_scale):
    """The cache's part of the C arguments: k, v, k_scale, v_scale, fmt, n_pages, page_size, page_stride; Hkv and d."""
    dtype, shape, st = k_cache.dtype, k_cache.shape, k_cache.stride()
    if not (k_cache.is_cuda and v_cache.is_cuda) or v_cache.dtype is not dtype or len(shape) != 4:
        raise MnwError("k_cache and v_cache: expected CUDA tensors of one type and 4 dimensions")
    if v_cache.shape != shape or v_cache.stride() != st:
        raise MnwError("k_cache and v_cache differ in shape or strides")
    n, h, page, d = shape
    if (page > 1 and st[2] != d) or (h > 1 and st[1] != page * d) or (d > 1 and st[3] != 1):
        raise MnwError("a page of the cache [Hkv, page_size, d] has to be contiguous")
    page_stride = st[0] if n > 1 else h * page * d
    ks = vs = None
    if dtype is torch.bfloat16:
        fmt = KV_BF16
        if k_scale is not None or v_scale is not None:
            raise MnwError("a bf16 cache has no scales")
    elif dtype is not torch.int8 and dtype is not torch.uint8:
        raise MnwError("the cache is bf16, int8, or uint8 (two 4-bit codes a byte)")
    elif k_scale is None or v_scale is None:
        raise MnwError("a quantised cache needs k_scale and v_scale")
    elif dtype is torch.int8:
        fmt = KV_INT8
        ks = _whole(k_scale, torch.float32, (n, h, page), "k_scale")
        vs = _whole(v_scale, torch.float32, (n, h, page), "v_scale")
    else:
        fmt = KV_INT4
        ks = _whole(k_scale, torch.uint8, (n, h, page, 8), "k_scale")
        vs = _whole(v_scale, torch.uint8, (n, h, page, 8), "v_scale")
        d, page_stride = 2 * d, 2 * page_stride
    return k_cache.data_ptr(), v_cache.data_ptr(), ks, vs, fmt, n, page, page_stride, h, d


def _batch_args(block_table, cache_lens, q_start):
    shape = block_table.shape
    if not block_table.is_cuda or block_table.dtype is not torch.int32 or len(shape) != 2 or not block_table.is_contiguous():
        raise MnwError("block_table: expected a contiguous CUDA tensor of torch.int32 with 2 dimensions")
    B, most = shape
    lp = _whole(cache_lens, torch.int32, (B,), "cache_lens")
    sp = None if q_start is None else _whole(q_start, torch.int32, (B + 1,), "q_start")
    return B, most, block_table.data_ptr(), lp, sp


def mnw_kv_append(q, k, v, k_cache, v_cache, block_table, cache_lens, inv_freq=None, layout=ROPE_HALF, mscale=1.0,
                  k_scale=None, v_scale=None, q_start=None, q_out=None, err=None, stream=None):
    """Writes new tokens' keys and values into a paged cache, keys rotated by
    position; returns the rotated queries [T, Hq, d] (None where q is None).
    q [T, Hq, d], k and v [T, Hkv, d] bf16, slices of one projection's output
    at will; caches [n_pages, Hkv, page_size, d] bf16, or int8 with scales f32
    [n_pages, Hkv, page_size], or uint8 [n_pages, Hkv, page_size, d / 2] (two
    4-bit codes a byte) with records uint8 [n_pages, Hkv, page_size, 8] as
    scales; block_table int32 [B, max_pages]; cache_lens
    int32 [B], the new tokens included; q_start int32 [B + 1] or None (T / B
    tokens each).  inv_freq f32 [rot / 2] (None: no rotation); see
    mnw_rope_frequencies and include/mnw_moe.h."""
    if stream is None:
        r = (_calls or _load_calls()).kv_append(q, k, v, k_cache, v_cache, block_table, cache_lens, inv_freq, layout, mscale,
                                                k_scale, v_scale, q_start, q_out, err)
        if r.__class__ is int:
            _check(r, "mnw_kv_append")
        if r is not NotImplemented:
            return r
    kc, vc, ks, vs, fmt, n_pages, page, page_stride, Hkv, d = _cache_args(k_cache, v_cache, k_scale, v_scale)
    B, most, tp, lp, sp = _batch_args(block_table, cache_lens, q_start)
    kp, T, hk, _, kst = _token_rows(k, "k", d)
    vp, Tv, hv, _, vst = _token_rows(v, "v", d)
    if hk != Hkv or hv != Hkv or Tv != T:
        raise MnwError("k and v have to be [T, Hkv, d] with the cache's Hkv")
    qp = qo = None
    Hq = qst = 0
    if q is not None:
        qp, Tq, Hq, _, qst = _token_rows(q, "q", d)
        if Tq != T:
            raise MnwError("q has another number of tokens than k")
        if q_out is None:
            q_out = _new((T, Hq, d), torch.bfloat16, q.device, stream)
        qo = _whole(q_out, torch.bfloat16, (T, Hq, d), "q_out")
    elif q_out is not None:
        raise MnwError("q_out needs q")
    fp, rot = None, 0
    if inv_freq is not None:
        rot = 2 * inv_freq.numel()
        fp = _whole(inv_freq, torch.float32, (rot // 2,), "inv_freq")
    ep = _word(err)
    _one_device(k, v=v, q=q, k_cache=k_cache, v_cache=v_cache, k_scale=k_scale, v_scale=v_scale, block_table=block_table,
                cache_lens=cache_lens, q_start=q_start, inv_freq=inv_freq, q_out=q_out, err=err)
    rc = load().mnw_kv_append(qp, qst, kp, kst, vp, vst, B, T, Hq, Hkv, d, fp, rot, layout, mscale, kc, vc, ks, vs, fmt,
                              n_pages, page, page_stride, tp, most, lp, sp, qo, ep, _stream_of(k, stream))
    if rc:
        _check(rc, "mnw_kv_append")
    return q_out


def mnw_attn_paged_workspace_size(B, T, Hq, Hkv, d) -> int:
    return int(load().mnw_attn_paged_workspace_size(B, T, Hq, Hkv, d))


@functools.lru_cache(maxsize=256)
def _paged_workspace(B, T, Hq, Hkv, d, device):
    return max(256, mnw_attn_paged_workspace_size(B, T, Hq, Hkv, d))


def mnw_attn_paged(q, k_cache, v_cache, block_table, cache_lens, blk, scale, k_scale=None, v_scale=None, q_start=None,
                   out=None, lse=None, want_lse=False, ws=None, err=None, stream=None):
    """Attention of new tokens q [T, Hq, d] over a paged cache (arguments as
    mnw_kv_append; append first).  A token at position p sees positions below
    (p // blk + 1) * blk.  Returns out [T, Hq, d] bf16, with want_lse or lse
    (out, lse f32 [T, Hq]).  ws: a uint8 device tensor of at least
    mnw_attn_paged_workspace_size bytes, 256-byte aligned."""
    if stream is None:
        r = (_calls or _load_calls()).attn_paged(q, k_cache, v_cache, block_table, cache_lens, blk, scale, k_scale, v_scale,
                                                 q_start, out, lse, want_lse, ws, err)
        if r.__class__ is int:
            _check(r, "mnw_attn_paged")
        if r is not NotImplemented:
            return r
    kc, vc, ks, vs, fmt, n_pages, page, page_stride, Hkv, d = _cache_args(k_cache, v_cache, k_scale, v_scale)
    B, most, tp, lp, sp = _batch_args(block_table, cache_lens, q_start)
    qp, T, Hq, _, qst = _token_rows(q, "q", d)
    dev = q.device
    if out is None:
        out = _new((T, Hq, d), torch.bfloat16, dev, stream)
        op = out.data_ptr()
    else:
        op = _whole(out, torch.bfloat16, (T, Hq, d), "out")
    if lse is None and want_lse:
        lse = _new((T, Hq), torch.float32, dev, stream)
    ep = _word(err)
    lsp = None if lse is None else _whole(lse, torch.float32, (T, Hq), "lse")
    _one_device(q, k_cache=k_cache, v_cache=v_cache, k_scale=k_scale, v_scale=v_scale, block_table=block_table,
                cache_lens=cache_lens, q_start=q_start, out=out, lse=lse, ws=ws, err=err)
    st, held = _stream_of(q, stream), None
    if ws is None:
        wn = _paged_workspace(B, T, Hq, Hkv, d, q.get_device())
        wp, held = _scratch(wn, q, stream, st)
    else:
        wp, wn = _whole(ws, torch.uint8, ws.shape, "ws"), ws.numel()
    try:
        rc = load().mnw_attn_paged(qp, qst, B, T, Hq, Hkv, d, kc, vc, ks, vs, fmt, n_pages, page, page_stride, tp, most, lp, sp,
                                   blk, scale, op, lsp, wp, wn, ep, st)
    finally:
        _give_back(held)
    if rc:
        _check(rc, "mnw_attn_paged")
    return out if lse is None else (out, lse)


def mnw_kv_values(cache, scale, out=None, stream=None):
    """The bf16 values [n_pages, Hkv, page_size, d] of all pages of a quantised
    cache: int8 [n_pages, Hkv, page_size, d] with scales f32, or uint8
    [n_pages, Hkv, page_size, d / 2] with records uint8 [n_pages, Hkv,
    page_size, 8] (arguments as mnw_kv_append's)."""
    if stream is None:
        r = (_calls or _load_calls()).kv_values(cache, scale, out)
        if r.__class__ is int:
            _check(r, "mnw_kv_values")
        if r is not NotImplemented:
            return r
    dtype, shape, st = cache.dtype, cache.shape, cache.stride()
    if not cache.is_cuda or (dtype is not torch.int8 and dtype is not torch.uint8) or len(shape) != 4:
        raise MnwError("cache: expected a CUDA tensor of int8, or uint8 (two 4-bit codes a byte), and 4 dimensions")
    n_pages, Hkv, page, d = shape
    if (page > 1 and st[2] != d) or (Hkv > 1 and st[1] != page * d) or (d > 1 and st[3] != 1):
        raise MnwError("a page of the cache [Hkv, page_size, d] has to be contiguous")
    page_stride = st[0] if n_pages > 1 else Hkv * page * d
    if dtype is torch.int8:
        fmt, sp = KV_INT8, _whole(scale, torch.float32, (n_pages, Hkv, page), "scale")
    else:
        fmt, sp = KV_INT4, _whole(scale, torch.uint8, (n_pages, Hkv, page, 8), "scale")
        d, page_stride = 2 * d, 2 * page_stride
    shape = (n_pages, Hkv, page, d)
    if out is None:
        out = _new(shape, torch.bfloat16, cache.device, stream)
    op = _whole(out, torch.bfloat16, shape, "out")
    _one_device(cache, scale=scale, out=out)
    rc = load().mnw_kv_values(cache.data_ptr(), sp, fmt, n_pages, page, Hkv, d, page_stride, op, _stream_of(cache, stream))
    if rc:
        _check(rc, "mnw_kv_values")
    return out


def mnw_lora_workspace_size(T, H, R, n_adapters) -> int:
    return int(load().mnw_lora_workspace_size(T, H, R, n_adapters))


@functools.lru_cache(maxsize=256)
def _lora_workspace(T, H, R, n, device):
    return mnw_lora_workspace_size(T, H, R, n)


def _rows(t, what):
    """(address, rows, columns, elements between rows) of a bf16 matrix whose rows are contiguous."""
    p = _need(t, torch.bfloat16, what, 2)
    T, n = t.shape
    return p, T, n, t.stride(0) if T > 1 else max(n, t.stride(0) // 8 * 8)


def mnw_lora_add(y, x, a, b, adapter, scale=None, ranks=None, out=None, ws=None, err=None, stream=None):
    """Low-rank adapters beside a shared projection: bf16(y[t] + scale[i] *
    b[i] (a[i] x[t])), i = adapter[t], or y[t] where that is -1.  y bf16 [T, N]
    (the projection's output), x bf16 [T, H], rows at any stride that is a
    multiple of 8; a bf16 [n, R, H]; b bf16 [n, N, R]; adapter int32 [T]; scale
    f32 [n] or None (1); ranks int32 [n] or None (R): the rows of a and columns
    of b that count.  out may be y (in place).  ws: a uint8 device tensor of at
    least mnw_lora_workspace_size bytes, 256-byte aligned."""
    if stream is None:
        r = (_calls or _load_calls()).lora_add(y, x, a, b, adapter, scale, ranks, out, ws, err)
        if r.__class__ is int:
            _check(r, "mnw_lora_add")
        if r is not NotImplemented:
            return r
    yp, T, N, y_stride = _rows(y, "y")
    xp, Tx, H, x_stride = _rows(x, "x")
    if Tx != T:
        raise MnwError("x and y have different numbers of tokens")
    if a.dim() != 3 or b.dim() != 3:
        raise MnwError("a and b have to be [n, R, H] and [n, N, R]")
    n, R = a.shape[:2]
    ap, bp = _whole(a, torch.bfloat16, (n, R, H), "a"), _whole(b, torch.bfloat16, (n, N, R), "b")
    ip = _whole(adapter, torch.int32, (T,), "adapter")
    sp = None if scale is None else _whole(scale, torch.float32, (n,), "scale")
    kp = None if ranks is None else _whole(ranks, torch.int32, (n,), "ranks")
    if out is None:
        out = _new((T, N), torch.bfloat16, y.device, stream)
    op, To, No, out_stride = _rows(out, "out")
    if (To, No) != (T, N):
        raise MnwError("out has another shape than y")
    ep = _word(err)
    _one_device(y, x=x, a=a, b=b, adapter=adapter, scale=scale, ranks=ranks, out=out, ws=ws, err=err)
    st, held, wp = _stream_of(y, stream), None, None
    if ws is None:
        wn = _lora_workspace(T, H, R, n, y.get_device())
        if wn:
            wp, held = _scratch(wn, y, stream, st)
    else:
        wp, wn = _whole(ws, torch.uint8, ws.shape, "ws"), ws.numel()
    try:
        rc = load().mnw_lora_add(xp, x_stride, ap, bp, sp, kp, n, R, ip, T, H, N, yp, y_stride, op, out_stride, wp, wn, ep, st)
    finally:
        _give_back(held)
    if rc:
        _check(rc, "mnw_lora_add")
    return out


def mnw_rope_frequencies(rot, base=10000.0, scale=ROPE_SCALE_NONE, factor=1.0, original_len=4096, beta_fast=32.0,
                         beta_slow=1.0, device=None):
    """(inv_freq f32 [rot / 2], mscale) for mnw_kv_append, scaled for contexts
    `factor` times original_len (see include/mnw_moe.h)."""
    f = torch.empty(max(rot, 0) // 2, dtype=torch.float32)
    m = ctypes.c_float()
    _check(load().mnw_rope_frequencies(rot, base, scale, factor, original_len, beta_fast, beta_slow,
                                       ctypes.c_void_p(f.data_ptr()), ctypes.byref(m)), "mnw_rope_frequencies")
    return (f if device is None else f.to(device)), m.value


def _gemm_out(layer, kind, P, dev):
    N = layer.H if kind == KIND_DOWN else layer.I
    return torch.empty((P, N), dtype=torch.bfloat16, device=dev)


def _gemm_a16(name, layer, kind, a, expert_offsets, err=None, stream=None):
    P = a.shape[0]
    out = _gemm_out(layer, kind, P, a.device)
    fn = getattr(load(), name)
    _check(fn(layer.handle, kind, _ptr(a), _ptr(expert_offsets), P, _ptr(out), _ptr(err), _stream(stream)), name)
    return out


def mnw_moe_grouped_gemm_bf16(layer, kind, a, expert_offsets, err=None, stream=None):
    return _gemm_a16("mnw_moe_grouped_gemm_bf16", layer, kind, a, expert_offsets, err, stream)


def mnw_moe_grouped_gemm_w8a16(layer, kind, a, expert_offsets, err=None, stream=None):
    return _gemm_a16("mnw_moe_grouped_gemm_w8a16", layer, kind, a, expert_offsets, err, stream)


def mnw_moe_grouped_gemm_w4a16(layer, kind, a, expert_offsets, err=None, stream=None):
    return _gemm_a16("mnw_moe_grouped_gemm_w4a16", layer, kind, a, expert_offsets, err, stream)


def _gemm_f16rows(name, layer, kind, a, row_outer, expert_offsets, err=None, stream=None):
    P = a.shape[0]
    out = _gemm_out(layer, kind, P, a.device)
    fn = getattr(load(), name)
    _check(fn(layer.handle, kind, _ptr(a), _ptr(row_outer), _ptr(expert_offsets), P, _ptr(out), _ptr(err),
              _stream(stream)), name)
    return out


def mnw_moe_grouped_gemm_w8a16_f16rows(layer, kind, a, row_outer, expert_offsets, err=None, stream=None):
    return _gemm_f16rows("mnw_moe_grouped_gemm_w8a16_f16rows", layer, kind, a, row_outer, expert_offsets, err,
                         stream)


def mnw_moe_grouped_gemm_w4a16_f16rows(layer, kind, a, row_outer, expert_offsets, err=None, stream=None):
    return _gemm_f16rows("mnw_moe_grouped_gemm_w4a16_f16rows", layer, kind, a, row_outer, expert_offsets, err,
                         stream)


def _gemm_a8(name, layer, kind, a_codes, a_scales, expert_offsets, want_dots=False, err=None, stream=None):
    P, K = a_codes.shape
    out = _gemm_out(layer, kind, P, a_codes.device)
    dots = None
    if want_dots:
        C = (2 * layer.I) if kind == KIND_GATE_UP else (layer.H if kind == KIND_DOWN else layer.I)
        dots = torch.zeros((P, C, K // 128), dtype=torch.int32, device=a_codes.device)
    fn = getattr(load(), name)
    _check(fn(layer.handle, kind, _ptr(a_codes), _ptr(a_scales), _ptr(expert_offsets), P, _ptr(out), _ptr(dots),
              _ptr(err), _stream(stream)), name)
    return (out, dots) if want_dots else out


def mnw_moe_grouped_gemm_w8a8(layer, kind, a_codes, a_scales, expert_offsets, want_dots=False, err=None, stream=None):
    return _gemm_a8("mnw_moe_grouped_gemm_w8a8", layer, kind, a_codes, a_scales, expert_offsets, want_dots, err,
                    stream)


def mnw_moe_grouped_gemm_w4a8(layer, kind, a_codes, a_scales, expert_offsets, want_dots=False, err=None, stream=None):
    return _gemm_a8("mnw_moe_grouped_gemm_w4a8", layer, kind, a_codes, a_scales, expert_offsets, want_dots, err,
                    stream)


def mnw_moe_grouped_gemm_nvfp4(layer, kind, a_codes, a_sf, a_outer, expert_offsets, err=None, stream=None):
    P = a_codes.shape[0]
    out = _gemm_out(layer, kind, P, a_codes.device)
    _check(load().mnw_moe_grouped_gemm_nvfp4(layer.handle, kind, _ptr(a_codes), _ptr(a_sf), _ptr(a_outer),
                                             _ptr(expert_offsets), P, _ptr(out), _ptr(err), _stream(stream)),
           "mnw_moe_grouped_gemm_nvfp4")
    return out


def mnw_moe_combine(y, assign_pos, w, stream=None, out=None):
    T, k = w.shape
    H = y.shape[1]
    if out is None:
        out = torch.empty((T, H), dtype=torch.bfloat16, device=y.device)
    _check(load().mnw_moe_combine(_ptr(y), _ptr(assign_pos), _ptr(w), T, k, H, _ptr(out), _stream(stream)),
           "mnw_moe_combine")
    return out


def mnw_moe_workspace_size(layer, act, T, k) -> int:
    return int(load().mnw_moe_workspace_size(layer.handle, act, T, k))


def mnw_moe_workspace_size_host(layer, act, T, k) -> int:
    return int(load().mnw_moe_workspace_size_host(layer.handle, act, T, k))


def workspace(layer, act, T, k, host=False, device=None) -> torch.Tensor:
    n = mnw_moe_workspace_size_host(layer, act, T, k) if host else mnw_moe_workspace_size(layer, act, T, k)
    return torch.empty(max(n, 256), dtype=torch.uint8, device=device or layer.blob.device)


def mnw_moe_forward(layer, act, x, ids, w, ws=None, out=None, stream=None):
    T, k = ids.shape
    if ws is None:
        ws = workspace(layer, act, T, k, device=x.device)
    if out is None:
        out = torch.empty((T, layer.H), dtype=torch.bfloat16, device=x.device)
    _check(load().mnw_moe_forward(layer.handle, act, _ptr(x), _ptr(ids), _ptr(w), T, k, _ptr(out), _ptr(ws),
                                  ws.numel(), _stream(stream)), "mnw_moe_forward")
    return out


def mnw_moe_forward_host(layer, act, x_host, ids_host, w_host, ws, out_host, stream=None):
    """Host tensors in and out (pinned memory gives overlap); synchronises."""
    T, k = ids_host.shape
    _check(load().mnw_moe_forward_host(layer.handle, act, ctypes.c_void_p(x_host.data_ptr()),
                                       ctypes.c_void_p(ids_host.data_ptr()), ctypes.c_void_p(w_host.data_ptr()),
                                       T, k, ctypes.c_void_p(out_host.data_ptr()), _ptr(ws), ws.numel(),
                                       _stream(stream)), "mnw_moe_forward_host")
    return out_host


def workspace_error_word(ws):
    """The forward's device error word as an int32 view of ws[0:4]."""
    return ws[:4].view(torch.int32)


def mnw_moe_read_error(err, stream=None) -> int:
    out = ctypes.c_uint32()
    _check(load().mnw_moe_read_error(_ptr(err), ctypes.byref(out), _stream(stream)), "mnw_moe_read_error")
    return out.value


def mnw_moe_launch_count() -> int:
    """Kernels this library has enqueued since it was loaded (host-side count)."""
    return int(load().mnw_moe_launch_count())


def mnw_moe_set_gemm_path(path: int) -> None:
    """Process-wide grouped-GEMM kernel choice (PATH_AUTO, PATH_TCGEN05, PATH_WARP_MMA)."""
    _check(load().mnw_moe_set_gemm_path(path), "mnw_moe_set_gemm_path")


STATIC_WS_BYTES = 32 * 1024 * 1024


def mnw_moe_forward_static(layer, act, x, ids, w, out=None, err=None, stream=None):
    """The whole layer with the library's built-in scratch array: no workspace
    and no device allocation by the library (see include/mnw_moe.h)."""
    T, k = ids.shape
    if out is None:
        out = torch.empty((T, layer.H), dtype=torch.bfloat16, device=x.device)
    _check(load().mnw_moe_forward_static(layer.handle, act, _ptr(x), _ptr(ids), _ptr(w), T, k, _ptr(out), _ptr(err),
                                         _stream(stream)), "mnw_moe_forward_static")
    return out


def mnw_moe_selftest_wait_timeout(limit_us, err, left_early, stream=None):
    """Launch the bounded-wait self-test (see include/mnw_moe.h); err and
    left_early are zeroed int32 device tensors of one element."""
    _check(load().mnw_moe_selftest_wait_timeout(limit_us, _ptr(err), _ptr(left_early), _stream(stream)),
           "mnw_moe_selftest_wait_timeout")


def mnw_moe_selftest_polled_wait_timeout(limit_us, err, left_early, stream=None):
    """As mnw_moe_selftest_wait_timeout, for the wait of the paged attention's
    block kernel."""
    _check(load().mnw_moe_selftest_polled_wait_timeout(limit_us, _ptr(err), _ptr(left_early), _stream(stream)),
           "mnw_moe_selftest_polled_wait_timeout")


def mnw_moe_selftest_counter_timeout(limit_us, counter, need, err, stream=None):
    """Launch the token-tile counter wait self-test (see include/mnw_moe.h);
    counter and err are int32 device tensors of one element."""
    _check(load().mnw_moe_selftest_counter_timeout(limit_us, _ptr(counter), need, _ptr(err), _stream(stream)),
           "mnw_moe_selftest_counter_timeout")
