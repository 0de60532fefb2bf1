"""Python binding of the fe_moe C ABI (include/fe_moe.h): argument marshalling only.

Every function named ``fe_moe_*`` here calls the C entry point of the same
name in ``libfe_moe.so``; all computation runs in the library's CUDA kernels.
The library must have been built (``python -m fp4_expert_gemv_b200.build``);
importing this package without it raises ImportError: there is no fallback.

``MoELayer`` is a convenience wrapper that takes torch tensors (device memory
and streams only) and checks status codes.
"""
from __future__ import annotations

import ctypes
import functools
import os

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libfe_moe.so")

FE_OK = 0
FE_ERR_INVALID_ARG = -1
FE_ERR_UNSUPPORTED = -2
FE_ERR_NOT_LOADED = -3
FE_ERR_CAPACITY = -4
FE_ERR_OOM = -5
FE_ERR_CUDA = -6
FE_ERR_DEVICE_STATUS = -7
FE_DEVICE_BAD_EXPERT = 0x1
FE_DEVICE_NAN_LOGIT = 0x2
FE_DEVICE_EXCHANGE_TIMEOUT = 0x4
FE_DEVICE_LOAD_TIMEOUT = 0x8
FE_DEVICE_TC_TIMEOUT = 0x10

PATH_AUTO, PATH_GEMV, PATH_TCGEN05, PATH_FUSED_DECODE, PATH_NVFP4 = 0, 1, 2, 3, 4
DTYPE_BF16, DTYPE_F32 = 0, 1
GATE_NONE, GATE_CHANNEL, GATE_TOKEN, GATE_FULL, GATE_SIGMOID = 0, 1, 2, 3, 16
ACT_NONE, ACT_RELU, ACT_GELU, ACT_SILU, ACT_SWIGLU = 0, 1, 2, 3, 4

if not os.path.exists(LIB_PATH):
    raise ImportError(f"{LIB_PATH} is not built; run `python fp4_expert_gemv_b200/build.py`")

lib = ctypes.CDLL(LIB_PATH)

_P = ctypes.c_void_p
_i32 = ctypes.c_int
_i64 = ctypes.c_int64
_st = ctypes.c_int
_f32 = ctypes.c_float
_sz = ctypes.c_size_t


class BlockWeights(ctypes.Structure):
    """fe_moe_block_t of include/fe_moe.h (device addresses)."""
    _fields_ = [("w_pre", _P), ("w_router", _P), ("shared_gate_up", _P), ("shared_down", _P), ("shared_I", _i32),
                ("w_post", _P), ("gate", _P), ("gate_kind", _i32), ("scale", _f32), ("w_next_pre", _P), ("eps", _f32)]


_SIGS = {
    "fe_moe_create": (_st, [_i32, _i32, _i32, _i32, ctypes.POINTER(_P)]),
    "fe_moe_reserve": (_st, [_P, _i32, _i32]),
    "fe_moe_load_packed": (_st, [_P, _P, _P, _P, _P, _i32, _P]),
    "fe_moe_forward": (_st, [_P, _P, _P, _i32, _i32, _P, _P]),
    "fe_moe_forward_host": (_st, [_P, _P, _P, _i32, _i32, _P, _P]),
    "fe_moe_get_routing": (_st, [_P, _P, _P, _P, _P, _P]),
    "fe_moe_get_status": (_st, [_P, ctypes.POINTER(ctypes.c_uint32)]),
    "fe_moe_set_path": (_st, [_P, _i32]),
    "fe_moe_last_forward_info": (_st, [_P, ctypes.POINTER(_i32), ctypes.POINTER(_i32)]),
    "fe_moe_set_trace": (_st, [_P, _P]),
    "fe_moe_status_string": (ctypes.c_char_p, [_st]),
    "fe_moe_destroy": (None, [_P]),
    "fe_moe_pack_host": (_st, [_P, _i64, _i64, _i64, _P, _P]),
    "fe_moe_pack_device": (_st, [_P, _i64, _i64, _i64, _P, _P, _P]),
    "fe_moe_device_bytes": (ctypes.c_size_t, [_P]),
    "fe_moe_last_error": (ctypes.c_char_p, []),
    "fe_moe_forward_noalloc": (_st, [_i32, _i32, _i32, _P, _P, _P, _P, _P, _P, _i32, _i32, _P, _P]),
    "fe_moe_get_grouping": (_st, [_P, _P, _P, _P]),
    "fe_moe_noalloc_get_status": (_st, [ctypes.POINTER(ctypes.c_uint32)]),
    "fe_moe_noalloc_get_routing": (_st, [_i32, _i32, _i32, _P, _P, _P, _P, _P, _P, _P]),
    "fe_moe_stack_create": (_st, [ctypes.POINTER(_P), _i32, ctypes.POINTER(_P)]),
    "fe_moe_stack_forward": (_st, [_P, _P, _P, _i32, _i32, _P, _P]),
    "fe_moe_stack_forward_host": (_st, [_P, _P, _P, _i32, _i32, _P, _i32, _P]),
    "fe_moe_stack_destroy": (None, [_P]),
    "fe_moe_stack_set_prefetch": (_st, [_P, _i32]),
    "fe_moe_stack_last_launches": (_i32, [_P]),
    "fe_moe_set_exchange_test": (_st, [_P, _i32, ctypes.c_uint64]),
    "fe_moe_router": (_st, [_P, _P, _P, _i32, _i32, _P, _P, _P, _P]),
    "fe_moe_load_int2": (_st, [_P, _P, _P, _P, _P, _P, _i32, _P]),
    "fe_moe_pack_int2_host": (_st, [_P, _i64, _i64, _i64, _P, _P]),
    "fe_moe_pack_int2_device": (_st, [_P, _i64, _i64, _i64, _P, _P, _P]),
    "fe_moe_forward_router": (_st, [_P, _P, _P, _i32, _i32, _P, _P, _P]),
    "fe_moe_load_nvfp4": (_st, [_P, _P, _P, _P, _P, _i32, _P]),
    "fe_moe_nvfp4_quantize_device": (_st, [_P, _i64, _i64, _P, _P, _P, _P]),
    "fe_moe_block_norm": (_st, [_P, _i32, _P, _P, _P, _i32, _f32, _P, _f32, _i64, _i32, _P, _P, _P]),
    "fe_moe_block_norm_workspace": (_sz, [_i64, _i32]),
    "fe_moe_block_norm_backward": (_st, [_P, _P, _P, _i32, _P, _P, _P, _i32, _f32, _P, _f32, _i64, _i32, _P, _P, _P, _P,
                                         _P, _P, _sz, _P]),
    "fe_moe_balance_workspace": (_sz, [_i64, _i32]),
    "fe_moe_balance_loss": (_st, [_P, _P, _P, _i64, _i32, _i32, _f32, _f32, _P, _P, _P, _P, _sz, _P]),
    "fe_moe_balance_loss_backward": (_st, [_P, _P, _P, _P, _P, _i64, _i32, _i32, _f32, _f32, _P, _i32, _P]),
    "fe_moe_linear": (_st, [_P, _i64, _P, _P, _P, _i64, _i64, _i32, _i32, _i32, _P, _i64, _P, _P]),
    "fe_moe_linear_workspace": (_sz, [_i64, _i32, _i32, _i32]),
    "fe_moe_linear_backward_workspace": (_sz, [_i64, _i32, _i32, _i32, _i32, _i32, _i32, _i32]),
    "fe_moe_linear_backward": (_st, [_P, _i64, _P, _i64, _P, _P, _i64, _i32, _i32, _i32, _P, _i64, _P, _P, _P, _sz, _P]),
    "fe_moe_get_op_status": (_st, [ctypes.POINTER(ctypes.c_uint32)]),
    "fe_moe_forward_block_workspace": (_sz, [_P, _i32, _i32]),
    "fe_moe_forward_block": (_st, [_P, ctypes.POINTER(BlockWeights), _P, _i32, _P, _i32, _i32, _P, _P, _P, _P, _sz, _P]),
}

for _name, (_res, _args) in _SIGS.items():
    _f = getattr(lib, _name)
    _f.restype = _res
    _f.argtypes = _args
    globals()[_name] = _f


class FeMoeError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        msg = fe_moe_status_string(status)
        detail = ""
        if status in (FE_ERR_CUDA, FE_ERR_OOM):
            detail = " [" + (fe_moe_last_error() or b"").decode(errors="replace") + "]"
        super().__init__(f"{what}: {msg.decode() if msg else status} ({status}){detail}")


def check(status: int, what: str = "fe_moe") -> None:
    if status != FE_OK:
        raise FeMoeError(status, what)


def _dptr(t) -> int:
    """Device address of a torch tensor (or an int address)."""
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _stream_ptr(stream) -> int:
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


class MoELayer:
    """One fe_moe handle: create + reserve, load packed weights, forward."""

    def __init__(self, E: int, H: int, I: int, max_T: int, max_top_k: int, group: int = 32):
        h = _P()
        check(fe_moe_create(E, H, I, group, ctypes.byref(h)), "fe_moe_create")
        self.h = h
        import torch
        self.device = torch.cuda.current_device()   # the one it was made on
        self.E, self.H, self.I = E, H, I
        self.max_T, self.max_top_k = max_T, max_top_k
        try:
            check(fe_moe_reserve(self.h, max_T, max_top_k), "fe_moe_reserve")
        except Exception:
            fe_moe_destroy(self.h)
            self.h = None
            raise

    def load_packed(self, gu_codes, gu_scales, dn_codes, dn_scales, stream=None):
        """Device torch tensors (uint8 codes, int16/uint16/bfloat16 scales) or host numpy arrays."""
        import numpy as np
        if isinstance(gu_codes, np.ndarray):
            arrs = [np.ascontiguousarray(a) for a in (gu_codes, gu_scales, dn_codes, dn_scales)]
            check(fe_moe_load_packed(self.h, *[a.ctypes.data for a in arrs], 0, _stream_ptr(stream)),
                  "fe_moe_load_packed")
            import torch
            torch.cuda.current_stream().synchronize() if stream is None else stream.synchronize()
        else:
            for t in (gu_codes, gu_scales, dn_codes, dn_scales):
                assert t.is_cuda and t.is_contiguous()
            check(fe_moe_load_packed(self.h, _dptr(gu_codes), _dptr(gu_scales), _dptr(dn_codes), _dptr(dn_scales),
                                     1, _stream_ptr(stream)), "fe_moe_load_packed")

    def forward(self, x_bf16, logits, top_k: int, y_bf16=None, stream=None):
        import torch
        T = x_bf16.shape[0]
        if y_bf16 is None:
            y_bf16 = torch.empty((T, self.H), dtype=torch.bfloat16, device=x_bf16.device)
        check(fe_moe_forward(self.h, _dptr(x_bf16), _dptr(logits), T, top_k, _dptr(y_bf16), _stream_ptr(stream)),
              "fe_moe_forward")
        return y_bf16

    def load_int2(self, formats, gu_codes, gu_scales, dn_codes, dn_scales, stream=None):
        """INT2 weights for the experts e with formats[e] = 1 (host numpy arrays or device
        torch tensors, full size [E, ...]); synchronous."""
        import numpy as np
        fmt = np.ascontiguousarray(np.asarray(formats, dtype=np.uint8))
        assert fmt.shape == (self.E,)
        if isinstance(gu_codes, np.ndarray):
            arrs = [np.ascontiguousarray(a) for a in (gu_codes, gu_scales, dn_codes, dn_scales)]
            check(fe_moe_load_int2(self.h, fmt.ctypes.data, *[a.ctypes.data for a in arrs], 0, _stream_ptr(stream)),
                  "fe_moe_load_int2")
        else:
            check(fe_moe_load_int2(self.h, fmt.ctypes.data, _dptr(gu_codes), _dptr(gu_scales), _dptr(dn_codes),
                                   _dptr(dn_scales), 1, _stream_ptr(stream)), "fe_moe_load_int2")

    def load_nvfp4(self, gu_codes, gu_scales, dn_codes, dn_scales, stream=None):
        """The block-scaled FP4 re-encoding of the packed weights (the arrays of load_packed:
        host numpy arrays or device torch tensors); then set_path(PATH_NVFP4) runs the variant."""
        import numpy as np
        if isinstance(gu_codes, np.ndarray):
            arrs = [np.ascontiguousarray(a) for a in (gu_codes, gu_scales, dn_codes, dn_scales)]
            check(fe_moe_load_nvfp4(self.h, *[a.ctypes.data for a in arrs], 0, _stream_ptr(stream)),
                  "fe_moe_load_nvfp4")
            import torch
            torch.cuda.current_stream().synchronize() if stream is None else stream.synchronize()
        else:
            for t in (gu_codes, gu_scales, dn_codes, dn_scales):
                assert t.is_cuda and t.is_contiguous()
            check(fe_moe_load_nvfp4(self.h, _dptr(gu_codes), _dptr(gu_scales), _dptr(dn_codes), _dptr(dn_scales),
                                    1, _stream_ptr(stream)), "fe_moe_load_nvfp4")

    def router(self, x_bf16, w_router_bf16, top_k: int, logits=None, idx=None, w=None, stream=None):
        """The router GEMM fused with the top-k: (logits [T, E] f32, idx [T, k] i32, w [T, k] f32)."""
        import torch
        T = x_bf16.shape[0]
        dev = x_bf16.device
        if logits is None:
            logits = torch.empty((T, self.E), dtype=torch.float32, device=dev)
        if idx is None:
            idx = torch.empty((T, top_k), dtype=torch.int32, device=dev)
        if w is None:
            w = torch.empty((T, top_k), dtype=torch.float32, device=dev)
        check(fe_moe_router(self.h, _dptr(x_bf16), _dptr(w_router_bf16), T, top_k, _dptr(logits), _dptr(idx),
                            _dptr(w), _stream_ptr(stream)), "fe_moe_router")
        return logits, idx, w

    def forward_router(self, x_bf16, w_router_bf16, top_k: int, y_bf16=None, logits=None, stream=None):
        """The layer from x alone (router GEMM, top-k, layer): (y [T, H] bf16, logits [T, E] f32)."""
        import torch
        T = x_bf16.shape[0]
        if y_bf16 is None:
            y_bf16 = torch.empty((T, self.H), dtype=torch.bfloat16, device=x_bf16.device)
        if logits is None:
            logits = torch.empty((T, self.E), dtype=torch.float32, device=x_bf16.device)
        check(fe_moe_forward_router(self.h, _dptr(x_bf16), _dptr(w_router_bf16), T, top_k, _dptr(y_bf16),
                                    _dptr(logits), _stream_ptr(stream)), "fe_moe_forward_router")
        return y_bf16, logits

    def forward_block(self, r, top_k: int, w_router, w_pre=None, u_in=None, shared=None, w_post=None, gate=None,
                      gate_kind=GATE_NONE, scale=1.0, w_next_pre=None, eps=1e-6, r_out=None, u_out=None, logits=None,
                      stream=None):
        """One block on the residual stream r [T, H] (bf16 or float32): norm (or u_in, the previous call's
        u_out), router, routed experts, shared expert (shared = (gate_up [2 I_s, H], down [H, I_s]) or None),
        norm, gate, residual, and the next block's norm.  Returns (r_out, u_out or None, logits)."""
        if stream is not None:
            with _on_stream(stream, r.device):
                return self.forward_block(r, top_k, w_router, w_pre, u_in, shared, w_post, gate, gate_kind, scale,
                                          w_next_pre, eps, r_out, u_out, logits)
        import torch
        bf, dev = torch.bfloat16, r.device
        T, H = r.shape
        dt = _dtype_of(r, "r")
        if dev.type == "cuda" and dev.index != self.device:
            raise ValueError(f"the tensors are on {dev}, the layer on cuda:{self.device}")
        _arg(r, "r", r.dtype, (T, self.H), dev)
        _arg(w_router, "w_router", bf, (self.E, H), dev)
        for name, t in (("w_pre", w_pre), ("w_post", w_post), ("w_next_pre", w_next_pre)):
            _arg(t, name, bf, (H,), dev, optional=True)
        _arg(u_in, "u_in", bf, (T, H), dev, optional=True)
        _arg_gate(gate, gate_kind, T, H, dev)
        Is = 0
        if shared is not None:
            Is = shared[1].shape[1]
            _arg(shared[0], "shared gate_up", bf, (2 * Is, H), dev)
            _arg(shared[1], "shared down", bf, (H, Is), dev)
        r_out = _out(r_out, "r_out", r.dtype, (T, H), dev, r)
        if w_next_pre is not None:
            u_out = _out(u_out, "u_out", bf, (T, H), dev, r)
        elif u_out is not None:
            raise ValueError("u_out needs w_next_pre")
        logits = _out(logits, "logits", torch.float32, (T, self.E), dev, r)
        nb = fe_moe_forward_block_workspace(self.h, T, Is)
        b = BlockWeights(_dptr(w_pre), _dptr(w_router), _dptr(shared[0]) if shared else None,
                         _dptr(shared[1]) if shared else None, Is, _dptr(w_post), _dptr(gate), gate_kind, scale,
                         _dptr(w_next_pre), eps)
        ws = r.new_empty(max(nb, 16), dtype=torch.uint8)
        _run("fe_moe_forward_block", fe_moe_forward_block, dev, self.h, ctypes.byref(b), _dptr(r), dt, _dptr(u_in), T, top_k,
             _dptr(r_out), _dptr(u_out), _dptr(logits), _dptr(ws), ws.numel())
        _written(r_out, u_out)
        _written(logits, None)
        return r_out, u_out, logits

    def forward_host(self, x_bf16_host, logits_host, top_k: int, y_bf16_host, stream=None):
        """Host (ideally pinned) numpy/torch CPU buffers in and out; synchronous."""
        def hp(a):
            return a.ctypes.data if hasattr(a, "ctypes") else a.data_ptr()
        T = x_bf16_host.shape[0]
        check(fe_moe_forward_host(self.h, hp(x_bf16_host), hp(logits_host), T, top_k, hp(y_bf16_host),
                                  _stream_ptr(stream)), "fe_moe_forward_host")
        return y_bf16_host

    def routing(self, T: int, top_k: int, stream=None):
        import torch
        dev = torch.device("cuda", torch.cuda.current_device())
        idx = torch.empty((T, top_k), dtype=torch.int32, device=dev)
        w = torch.empty((T, top_k), dtype=torch.float32, device=dev)
        offsets = torch.empty(self.E + 1, dtype=torch.int32, device=dev)
        sp = torch.empty(T * top_k, dtype=torch.int32, device=dev)
        check(fe_moe_get_routing(self.h, _dptr(idx), _dptr(w), _dptr(offsets), _dptr(sp), _stream_ptr(stream)),
              "fe_moe_get_routing")
        return idx, w, offsets, sp

    def grouping(self, T: int, top_k: int, stream=None):
        """(counts int32 [E], pair_row int32 [T*top_k]) of the last forward, as device tensors."""
        import torch
        dev = torch.device("cuda", torch.cuda.current_device())
        counts = torch.empty(self.E, dtype=torch.int32, device=dev)
        pair_row = torch.empty(T * top_k, dtype=torch.int32, device=dev)
        check(fe_moe_get_grouping(self.h, _dptr(counts), _dptr(pair_row), _stream_ptr(stream)), "fe_moe_get_grouping")
        return counts, pair_row

    def status(self):
        bits = ctypes.c_uint32(0)
        st = fe_moe_get_status(self.h, ctypes.byref(bits))
        return st, bits.value

    def set_path(self, path: int):
        check(fe_moe_set_path(self.h, path), "fe_moe_set_path")

    def last_forward_info(self):
        path, kernels = _i32(0), _i32(0)
        check(fe_moe_last_forward_info(self.h, ctypes.byref(path), ctypes.byref(kernels)), "fe_moe_last_forward_info")
        return path.value, kernels.value

    def device_bytes(self) -> int:
        return fe_moe_device_bytes(self.h)

    def close(self):
        if getattr(self, "h", None):
            fe_moe_destroy(self.h)
            self.h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class Stack:
    """fe_moe_stack over MoELayer objects (kept alive here): n layers back to back on one stream."""

    def __init__(self, layers):
        self.layers = list(layers)
        arr = (_P * len(self.layers))(*[m.h for m in self.layers])
        h = _P()
        check(fe_moe_stack_create(arr, len(self.layers), ctypes.byref(h)), "fe_moe_stack_create")
        self.h = h
        self.n = len(self.layers)
        self.E, self.H = self.layers[0].E, self.layers[0].H

    def forward(self, x_bf16, logits, top_k: int, y_bf16, stream=None):
        """x device bf16 [n, T, H] (layer l reads x[l]), logits device float32 [n, T, E], y device bf16
        [n, T, H] (layer l writes y[l]); pass y = a view of x shifted by one layer to chain them."""
        T = logits.shape[1]
        check(fe_moe_stack_forward(self.h, _dptr(x_bf16), _dptr(logits), T, top_k, _dptr(y_bf16),
                                   _stream_ptr(stream)), "fe_moe_stack_forward")
        return y_bf16

    def forward_host(self, x_bf16_host, logits_host, top_k: int, y_bf16_host, chained=False, stream=None):
        """Host buffers (numpy or CPU torch, ideally pinned), bf16 as int16/uint16 bits; logits [n, T, E].
        chained=False: x, y [n, T, H]; chained=True: x [T, H] into layer 0, y [T, H] out of the last."""
        def hp(a):
            return a.ctypes.data if hasattr(a, "ctypes") else a.data_ptr()
        T = logits_host.shape[1]
        check(fe_moe_stack_forward_host(self.h, hp(x_bf16_host), hp(logits_host), T, top_k, hp(y_bf16_host),
                                        1 if chained else 0, _stream_ptr(stream)), "fe_moe_stack_forward_host")
        return y_bf16_host

    def set_prefetch(self, on: bool):
        """Cross-layer streaming (one persistent launch at T=1) on or off."""
        check(fe_moe_stack_set_prefetch(self.h, 1 if on else 0), "fe_moe_stack_set_prefetch")

    def last_launches(self) -> int:
        return fe_moe_stack_last_launches(self.h)

    def close(self):
        if getattr(self, "h", None):
            fe_moe_stack_destroy(self.h)
            self.h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def noalloc_status():
    """(status, bits) of the last fe_moe_forward_noalloc call on the current device."""
    bits = ctypes.c_uint32(0)
    st = fe_moe_noalloc_get_status(ctypes.byref(bits))
    return st, bits.value


def pack_host(W):
    """numpy float32 [E, K, N] -> (codes uint8 [E, K/2, N], scales uint16 [E, K/32, N]) via fe_moe_pack_host."""
    import numpy as np
    W = np.ascontiguousarray(W, dtype=np.float32)
    E, K, N = W.shape
    codes = np.empty((E, K // 2, N), dtype=np.uint8)
    scales = np.empty((E, K // 32, N), dtype=np.uint16)
    check(fe_moe_pack_host(W.ctypes.data, E, K, N, codes.ctypes.data, scales.ctypes.data), "fe_moe_pack_host")
    return codes, scales


def pack_int2_host(W):
    """numpy float32 [E, K, N] -> (INT2 codes uint8 [E, K/4, N], scales uint16 [E, K/32, N])."""
    import numpy as np
    W = np.ascontiguousarray(W, dtype=np.float32)
    E, K, N = W.shape
    codes = np.empty((E, K // 4, N), dtype=np.uint8)
    scales = np.empty((E, K // 32, N), dtype=np.uint16)
    check(fe_moe_pack_int2_host(W.ctypes.data, E, K, N, codes.ctypes.data, scales.ctypes.data),
          "fe_moe_pack_int2_host")
    return codes, scales


def pack_int2_device(W, codes=None, scales=None, stream=None):
    """torch float32 CUDA [E, K, N] -> (INT2 codes uint8 [E, K/4, N], scales int16 bf16-bits)."""
    import torch
    E, K, N = W.shape
    if codes is None:
        codes = torch.empty((E, K // 4, N), dtype=torch.uint8, device=W.device)
    if scales is None:
        scales = torch.empty((E, K // 32, N), dtype=torch.int16, device=W.device)
    check(fe_moe_pack_int2_device(_dptr(W), E, K, N, _dptr(codes), _dptr(scales), _stream_ptr(stream)),
          "fe_moe_pack_int2_device")
    return codes, scales


def nvfp4_quantize_device(V, stream=None):
    """torch float32 CUDA [R, K] -> NVFP4 (codes uint8 [R, K/2], E4M3 scale factors uint8 [R, K/16],
    row scales float32 [R])."""
    import torch
    R, K = V.shape
    assert V.is_cuda and V.is_contiguous() and V.dtype == torch.float32
    codes = torch.empty((R, K // 2), dtype=torch.uint8, device=V.device)
    sf = torch.empty((R, K // 16), dtype=torch.uint8, device=V.device)
    g = torch.empty((R,), dtype=torch.float32, device=V.device)
    check(fe_moe_nvfp4_quantize_device(_dptr(V), R, K, _dptr(codes), _dptr(sf), _dptr(g), _stream_ptr(stream)),
          "fe_moe_nvfp4_quantize_device")
    return codes, sf, g


def pack_device(W, codes=None, scales=None, stream=None):
    """torch float32 CUDA [E, K, N] -> (codes uint8, scales int16 bf16-bits) via fe_moe_pack_device."""
    import torch
    E, K, N = W.shape
    if codes is None:
        codes = torch.empty((E, K // 2, N), dtype=torch.uint8, device=W.device)
    if scales is None:
        scales = torch.empty((E, K // 32, N), dtype=torch.int16, device=W.device)
    check(fe_moe_pack_device(_dptr(W), E, K, N, _dptr(codes), _dptr(scales), _stream_ptr(stream)),
          "fe_moe_pack_device")
    return codes, scales


# ---- the operators around the experts ---------------------------------------------------
# Torch CUDA tensors in and out; outputs that are not given are allocated.  `stream` (a torch
# stream or an address) makes the call, its allocations included, on that stream; otherwise it
# runs on the current stream of the tensors' device.
#
# The calls record no autograd graph: the gradients are the *_backward calls', made by hand or from a
# torch.autograd.Function.  As torch's functions with an out= argument do, they refuse tensors that
# require grad while grad mode is on, and a tensor that is given to be written counts as changed in
# place, so that a backward pass that saved its old contents raises instead of using the new ones.


# The sizes' answers alone: a model asks for the same few at every step.
_norm_workspace, _balance_workspace, _linear_backward_workspace = (
    functools.lru_cache(1024)(lambda *sizes, query=query: query(*sizes))
    for query in (fe_moe_block_norm_workspace, fe_moe_balance_workspace, fe_moe_linear_backward_workspace))


@functools.cache
def _current():
    """torch's current device, and a device's current stream as an address (without the Stream object where torch
    offers that)."""
    import torch
    raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    return torch.cuda.current_device, raw or (lambda index: torch.cuda.current_stream(index).cuda_stream)


def _run(what, fn, dev, *args):
    """fn(*args, the current stream of dev) with dev current; raises on a status."""
    if dev.type != "cuda":
        raise ValueError(f"{what}: CUDA tensors are needed, got {dev}")
    device, stream = _current()
    index = dev.index
    if index == device():
        status = fn(*args, stream(index))
    else:
        import torch
        with torch.cuda.device(dev):
            status = fn(*args, stream(index))
    if status != FE_OK:
        raise FeMoeError(status, what)


def _refuse_grad(t, name):
    import torch
    if torch.is_grad_enabled():
        raise ValueError(f"{name} requires grad, but this call records no graph: call it under torch.no_grad() or from a "
                         f"torch.autograd.Function")


@functools.cache
def _types():
    """torch.bfloat16, float32 and int32."""
    import torch
    return torch.bfloat16, torch.float32, torch.int32


@functools.cache
def _bump():
    """Counts a tuple of tensors as changed in place (without the checks on its argument where torch offers that)."""
    import torch
    return getattr(torch._C, "_increment_version", None) or torch.autograd.graph.increment_version


def _written(a, b):
    """Counts a call's outputs, or the one there is, as changed in place; an output of the call's own does not mind."""
    _bump()((a,) if b is None else (b,) if a is None else (a, b))


def _on_stream(stream, dev):
    """The stream made current, so that what the call allocates belongs to it."""
    import torch
    if isinstance(stream, int):
        stream = torch.cuda.ExternalStream(stream, device=dev)
    if stream.device != dev:
        raise ValueError(f"the stream is on {stream.device}, the tensors on {dev}")
    return torch.cuda.stream(stream)


def _arg(t, name, dtype, shape, dev, optional=False):
    """The address of a contiguous CUDA tensor of this type and shape on dev (None for None, where allowed)."""
    if t is None:
        if optional:
            return None
        raise ValueError(f"{name} is needed")
    if t.dtype is not dtype or t.shape != shape or t.device != dev or not t.is_contiguous():
        raise ValueError(f"{name}: a contiguous {dtype} CUDA tensor of shape {tuple(shape)} on {dev} is needed, "
                         f"got {t.dtype} {tuple(t.shape)} strides {tuple(t.stride())} on {t.device}")
    if t.requires_grad:
        _refuse_grad(t, name)
    return t.data_ptr()


def _first(t, name, dtype):
    """_arg for the tensor that the others' shape and device are taken from."""
    if t.dtype is not dtype or t.requires_grad or not t.is_contiguous():
        return _arg(t, name, dtype, t.shape, t.device)
    return t.data_ptr()


def _arg_rows(t, name, dtype, shape, dev):
    """The address and row stride of a CUDA matrix whose rows are contiguous."""
    if t.requires_grad:
        _refuse_grad(t, name)
    if t.dtype is dtype and t.shape == shape and t.device == dev and t.is_contiguous():
        return t.data_ptr(), shape[1] if shape[0] > 1 else (shape[1] + 7) // 8 * 8
    if (t.dtype is not dtype or t.shape != shape or t.device != dev
            or (shape[1] > 1 and shape[0] > 0 and t.stride(1) != 1)):
        raise ValueError(f"{name}: a {dtype} CUDA matrix of shape {tuple(shape)} on {dev} with contiguous rows is needed, "
                         f"got {t.dtype} {tuple(t.shape)} strides {tuple(t.stride())} on {t.device}")
    if shape[0] <= 1:
        return t.data_ptr(), (shape[1] + 7) // 8 * 8
    ld = t.stride(0)
    if ld < shape[1]:
        raise ValueError(f"{name}: rows overlap (strides {tuple(t.stride())})")
    return t.data_ptr(), ld


def _arg_gate(gate, kind, T, H, dev):
    if gate is None and kind == GATE_NONE:
        return None
    k = kind & ~GATE_SIGMOID
    if k not in (GATE_NONE, GATE_CHANNEL, GATE_TOKEN, GATE_FULL) or (gate is None) != (k == GATE_NONE):
        raise ValueError("gate and gate_kind do not go together")
    if gate is None:
        return None
    return _arg(gate, "gate", _types()[0], (H,) if k == GATE_CHANNEL else (T,) if k == GATE_TOKEN else (T, H), dev)


def _new(like, dtype, *shape):
    """An uninitialised tensor on like's device (by the cheapest of torch's ways: a third of a small call's host time
    goes into its outputs)."""
    return like.new_empty(*shape) if like.dtype is dtype else like.new_empty(*shape, dtype=dtype)


def _out(t, name, dtype, shape, dev, like):
    if t is None:
        return like.new_empty(*shape) if like.dtype is dtype else like.new_empty(*shape, dtype=dtype)
    _arg(t, name, dtype, shape, dev)
    return t


def _dtype_of(t, name):
    bf, f32, _ = _types()
    if t.dtype is bf:
        return DTYPE_BF16
    if t.dtype is f32:
        return DTYPE_F32
    raise ValueError(f"{name}: bfloat16 or float32 is needed, got {t.dtype}")


def block_norm(r, y=None, w_post=None, w_pre=None, gate=None, gate_kind=GATE_NONE, scale=1.0, eps=1e-6, r_out=None,
               u=None, stream=None):
    """r' = r + scale * a(gate) * w_post * y / rms(y) and u = w_pre * r' / rms(r') in one pass
    (fe_moe_block_norm).  r [T, H] bf16 or float32, the rest bf16.  Returns (r', u): None for what
    was not asked for (r' without y, u without w_pre)."""
    if stream is not None:
        with _on_stream(stream, r.device):
            return block_norm(r, y, w_post, w_pre, gate, gate_kind, scale, eps, r_out, u)
    bf, _, _ = _types()
    dev, shape = r.device, r.shape
    T, H = shape
    dt = _dtype_of(r, "r")
    rp = _first(r, "r", r.dtype)
    yp = _arg(y, "y", bf, shape, dev, True)
    postp = _arg(w_post, "w_post", bf, (H,), dev, True)
    prep = _arg(w_pre, "w_pre", bf, (H,), dev, True)
    gp = _arg_gate(gate, gate_kind, T, H, dev)
    if y is not None:
        r_out = _out(r_out, "r_out", r.dtype, shape, dev, r)
    if w_pre is not None:
        u = _out(u, "u", bf, shape, dev, r)
    _run("fe_moe_block_norm", fe_moe_block_norm, dev, rp, dt, yp, postp, gp, gate_kind, scale, prep, eps, T, H,
         _dptr(r_out), _dptr(u))
    _written(r_out, u)
    return r_out, u


def block_norm_backward(dr_out, du, r, y=None, w_post=None, w_pre=None, gate=None, gate_kind=GATE_NONE, scale=1.0,
                        eps=1e-6, weight_grads=True, stream=None):
    """The gradients of block_norm: (dr, dy, dgate, dw_post, dw_pre), None for an operand that is None.
    dr_out (like r) or du (bf16) may be None for no gradient.  dgate is float32 for a channel or
    token gate, bf16 for a full one; dw_post and dw_pre are float32.  weight_grads=False leaves
    out dw_post, dw_pre and a channel dgate."""
    if stream is not None:
        with _on_stream(stream, r.device):
            return block_norm_backward(dr_out, du, r, y, w_post, w_pre, gate, gate_kind, scale, eps, weight_grads)
    import torch
    bf, f32, _ = _types()
    dev, shape = r.device, r.shape
    T, H = shape
    dt = _dtype_of(r, "r")
    rp = _first(r, "r", r.dtype)
    drop = _arg(dr_out, "dr_out", r.dtype, shape, dev, True)
    dup = _arg(du, "du", bf, shape, dev, True)
    yp = _arg(y, "y", bf, shape, dev, True)
    postp = _arg(w_post, "w_post", bf, (H,), dev, True)
    prep = _arg(w_pre, "w_pre", bf, (H,), dev, True)
    gp = _arg_gate(gate, gate_kind, T, H, dev)
    kind = gate_kind & ~GATE_SIGMOID
    dr = torch.empty_like(r)
    dy = torch.empty_like(y) if y is not None else None
    dw_post = _new(r, f32, H) if weight_grads and w_post is not None else None
    dw_pre = _new(r, f32, H) if weight_grads and w_pre is not None else None
    dgate = None
    if kind == GATE_FULL:
        dgate = torch.empty_like(gate)
    elif kind == GATE_TOKEN:
        dgate = _new(r, f32, T)
    elif kind == GATE_CHANNEL and weight_grads:
        dgate = _new(r, f32, H)
    ws, nb = None, 0
    if dw_post is not None or dw_pre is not None or (kind == GATE_CHANNEL and weight_grads):
        nb = _norm_workspace(T, H)
        ws = _new(r, f32, (nb + 3) // 4)
    _run("fe_moe_block_norm_backward", fe_moe_block_norm_backward, dev, drop, dup, rp, dt, yp, postp, gp, gate_kind,
         scale, prep, eps, T, H, _dptr(dr), _dptr(dy), _dptr(dgate), _dptr(dw_post), _dptr(dw_pre), _dptr(ws), nb)
    return dr, dy, dgate, dw_post, dw_pre


def balance_loss(logits, idx, mask=None, balance_coef=1.0, z_coef=0.0, loss=None, counts=None, n_tokens=None,
                 stream=None):
    """The router's balance loss: logits float32 [T, E], idx int32 [T, k], mask uint8 [T] (0 = padding).
    Returns (float32 [3]: loss, balance, z; int32 [E] counts; int32 [1] kept tokens)."""
    if stream is not None:
        with _on_stream(stream, logits.device):
            return balance_loss(logits, idx, mask, balance_coef, z_coef, loss, counts, n_tokens)
    import torch
    i32, f32, dev = torch.int32, torch.float32, logits.device
    T, E = logits.shape
    k = idx.shape[1]
    lp = _first(logits, "logits", f32)
    ip = _arg(idx, "idx", i32, (T, k), dev)
    mp = _arg(mask, "mask", torch.uint8, (T,), dev, True)
    given = loss is not None or counts is not None or n_tokens is not None
    loss = _out(loss, "loss", f32, (3,), dev, logits)
    counts = _out(counts, "counts", i32, (E,), dev, idx)
    n_tokens = _out(n_tokens, "n_tokens", i32, (1,), dev, idx)
    nb = _balance_workspace(T, E)
    ws = logits.new_empty((nb + 3) // 4) if nb else None
    _run("fe_moe_balance_loss", fe_moe_balance_loss, dev, lp, ip, mp, T, E, k, balance_coef, z_coef, loss.data_ptr(),
         counts.data_ptr(), n_tokens.data_ptr(), _dptr(ws), nb)
    if given:
        _bump()((loss, counts, n_tokens))
    return loss, counts, n_tokens


def balance_loss_backward(logits, counts, n_tokens, top_k: int, mask=None, dloss=None, balance_coef=1.0, z_coef=0.0,
                          dlogits=None, dtype=None, stream=None):
    """dloss/dlogits [T, E] of balance_loss (float32, or bf16 with dtype=torch.bfloat16), times dloss
    (float32 [1] on the device, None = 1); counts and n_tokens as balance_loss returned them."""
    if stream is not None:
        with _on_stream(stream, logits.device):
            return balance_loss_backward(logits, counts, n_tokens, top_k, mask, dloss, balance_coef, z_coef, dlogits, dtype)
    import torch
    f32, i32, dev = torch.float32, torch.int32, logits.device
    T, E = logits.shape
    lp = _first(logits, "logits", f32)
    cp = _arg(counts, "counts", i32, (E,), dev)
    np_ = _arg(n_tokens, "n_tokens", i32, (1,), dev)
    mp = _arg(mask, "mask", torch.uint8, (T,), dev, True)
    dp = _arg(dloss, "dloss", f32, (1,), dev, True)
    dlogits = _out(dlogits, "dlogits", dtype or (f32 if dlogits is None else dlogits.dtype), (T, E), dev, logits)
    dt = _dtype_of(dlogits, "dlogits")
    _run("fe_moe_balance_loss_backward", fe_moe_balance_loss_backward, dev, lp, cp, np_, mp, dp, T, E, top_k,
         balance_coef, z_coef, dlogits.data_ptr(), dt)
    _written(dlogits, None)
    return dlogits


def linear(x, w, bias=None, act=ACT_NONE, residual=None, y=None, z=None, stream=None):
    """y = act(x w^T + bias) + residual on bf16 matrices: x [M, K], w [N, K], bias [N]; residual and y
    [M, N] ([M, N / 2] for ACT_SWIGLU).  The rows of x, residual and y may be strided; y may be the
    residual.  z [M, N], if given, receives the pre-activation for linear_backward."""
    if stream is not None:
        with _on_stream(stream, x.device):
            return linear(x, w, bias, act, residual, y, z)
    bf, _, _ = _types()
    dev = x.device
    M, K = x.shape
    N = w.shape[0]
    out = (M, N // 2 if act == ACT_SWIGLU else N)
    if x.dtype is bf and not x.requires_grad and x.is_contiguous():
        xp, ldx = x.data_ptr(), K
    else:
        xp, ldx = _arg_rows(x, "x", bf, (M, K), dev)
    wp = _arg(w, "w", bf, (N, K), dev)
    bp = _arg(bias, "bias", bf, (N,), dev, True)
    zp = _arg(z, "z", bf, (M, N), dev, True)
    resp, ldr = (None, 0) if residual is None else _arg_rows(residual, "residual", bf, out, dev)
    given = y is not None or z is not None
    if y is None:
        y = x.new_empty(*out)
        yp, ldy = y.data_ptr(), out[1]
    else:
        yp, ldy = _arg_rows(y, "y", bf, out, dev)
    _run("fe_moe_linear", fe_moe_linear, dev, xp, ldx, wp, bp, resp, ldr, M, N, K, act, yp, ldy, zp)
    if given:
        _written(y, z)
    return y


def linear_backward(dy, x, w, z=None, act=ACT_NONE, need_dx=True, need_dw=True, need_db=True, stream=None):
    """The gradients of linear: (dx bf16 [M, K], dw bf16 [N, K], db float32 [N]), None for what is not
    needed; z is the pre-activation that linear wrote.  The residual's gradient is dy."""
    if stream is not None:
        with _on_stream(stream, x.device):
            return linear_backward(dy, x, w, z, act, need_dx, need_dw, need_db)
    import torch
    bf, dev = torch.bfloat16, x.device
    M, K = x.shape
    N = w.shape[0]
    xp, ldx = _arg_rows(x, "x", bf, (M, K), dev)
    wp = _arg(w, "w", bf, (N, K), dev)
    zp = _arg(z, "z", bf, (M, N), dev, act == ACT_NONE)
    dyp, lddy = _arg_rows(dy, "dy", bf, (M, N // 2 if act == ACT_SWIGLU else N), dev)
    dx = (torch.empty_like(x) if x.is_contiguous() else x.new_empty(M, K)) if need_dx else None
    dw = torch.empty_like(w) if need_dw else None
    db = _new(x, torch.float32, N) if need_db else None
    nb = _linear_backward_workspace(M, N, K, act, lddy % 8 == 0 and dyp % 16 == 0, need_dx, need_dw, need_db)
    ws = x.new_empty((nb + 1) // 2) if nb else None
    _run("fe_moe_linear_backward", fe_moe_linear_backward, dev, dyp, lddy, xp, ldx, wp, zp, M, N, K, act, _dptr(dx),
         K, _dptr(dw), _dptr(db), _dptr(ws), nb)
    return dx, dw, db


def op_status():
    """(status, bits) of the operators around the experts on the current device since the last query."""
    bits = ctypes.c_uint32(0)
    st = fe_moe_get_op_status(ctypes.byref(bits))
    return st, bits.value
