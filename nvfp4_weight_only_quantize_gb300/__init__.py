"""Python binding of libqerl, the sm_103a NVFP4 weight-only LoRA linear library.

Argument marshalling only: each function passes torch tensors' device pointers,
sizes and the current CUDA stream to the C entry point of the same name in
``include/qerl.h`` and raises ``QerlError`` on a non-OK status.  Every step of
the computation runs in the library's CUDA kernels; there is no fallback.  If
``_lib/libqerl.so`` is missing the import of the library fails loudly (run
``build()``).
"""
from __future__ import annotations

import contextlib
import ctypes as C
import os
import threading

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "_lib", "libqerl.so")

QERL_OK = 0
STATUS_NAMES = {0: "QERL_OK", 1: "QERL_ERR_INVALID_ARG", 2: "QERL_ERR_SHAPE", 3: "QERL_ERR_ALIGN",
                4: "QERL_ERR_NONFINITE", 5: "QERL_ERR_CUDA", 6: "QERL_ERR_TIMEOUT",
                7: "QERL_ERR_UNSUPPORTED_DEVICE", 8: "QERL_ERR_WORKSPACE", 9: "QERL_ERR_TOO_LARGE",
                10: "QERL_ERR_HOST_MEMORY"}
NOALLOC_SCRATCH_BYTES = 8 << 20  # QERL_NOALLOC_SCRATCH_BYTES
SCALE_ROUND_UP, SCALE_ROUND_NEAREST_EVEN = 0, 1
OP_QUANTIZE, OP_LINEAR_FWD, OP_LINEAR_BWD, OP_AQN_RMSNORM, OP_MXFP4_FWD, OP_LINEAR_FWD_F32AB = 0, 1, 2, 3, 4, 5
OP_POLICY_LOSS = 6
DTYPE_F32, DTYPE_BF16 = 0, 1
ALGO_AUTO, ALGO_SIMT, ALGO_TCGEN05, ALGO_GEMV = 0, 1, 2, 3
AQN_NOISE_ADD, AQN_NOISE_MUL = 0, 1
KERNEL_ATTN_ROWS16, KERNEL_ATTN_ROWS128, KERNEL_LOSS_ROW, KERNEL_LOSS_RING = 0, 1, 2, 3
KERNEL_KV4_ROWS8, KERNEL_KV4_ROWS128 = 4, 5

# Every C symbol include/qerl.h declares (checked by the CPU test suite).
EXPORTED = ["qerl_nvfp4_quantize", "qerl_nvfp4_dequantize", "qerl_nvfp4_lora_linear_fwd",
            "qerl_nvfp4_lora_linear_fwd_noalloc", "qerl_nvfp4_pack_codes", "qerl_nvfp4_unpack_codes",
            "qerl_nvfp4_lora_linear_fwd_packed", "qerl_nvfp4_lora_linear_bwd_packed",
            "qerl_nvfp4_lora_linear_bwd", "qerl_aqn_rmsnorm", "qerl_aqn_rmsnorm_mode", "qerl_aqn_noise",
            "qerl_aqn_sigma",
            "qerl_workspace_bytes", "qerl_get_error", "qerl_status_string", "qerl_set_linear_algo",
            "qerl_set_launch_chaining", "qerl_lora_linear_fwd_grouped_ws_bytes",
            "qerl_nvfp4_lora_linear_fwd_grouped",
            "qerl_launch_count", "qerl_kernel_launch_count", "qerl_decoder_chain_ws_bytes", "qerl_decoder_chain_plan",
            "qerl_decoder_chain_run", "qerl_decoder_chain_destroy", "qerl_mxfp4_quantize",
            "qerl_mxfp4_lora_linear_fwd", "qerl_nvfp4_lora_linear_fwd_f32ab", "qerl_residual_add", "qerl_swiglu",
            "qerl_prefix_attention_ws_bytes", "qerl_prefix_attention", "qerl_token_logp", "qerl_policy_loss",
            "qerl_adamw_ws_bytes", "qerl_adamw_plan", "qerl_adamw_step", "qerl_adamw_read_state", "qerl_adamw_destroy",
            "qerl_kv4_append", "qerl_kv4_read", "qerl_kv4_attention_ws_bytes", "qerl_kv4_attention", "qerl_sample"]


class QerlError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {STATUS_NAMES.get(status, status)} ({status_string(status)})")


class _QuantOpts(C.Structure):
    _fields_ = [("scale_round", C.c_int)]


_lib = None
_lock = threading.Lock()


def build(force: bool = False) -> str:
    this = build
    from .build import build as _build
    globals()["build"] = this  # importing the submodule has put the module under this name
    return _build(force=force)


def lib() -> C.CDLL:
    """The loaded libqerl.so (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise ImportError(f"libqerl.so not built ({LIB_PATH}); call "
                                  "nvfp4_weight_only_quantize_gb300.build()")
            L = C.CDLL(LIB_PATH)
            vp, i64, i32, f32, u64, u32, sz = (C.c_void_p, C.c_int64, C.c_int, C.c_float, C.c_uint64,
                                               C.c_uint32, C.c_size_t)
            sig = {
                "qerl_nvfp4_quantize": ([vp, i64, i64, i64, vp, vp, vp, vp, vp, sz, vp], i32),
                "qerl_nvfp4_dequantize": ([vp, vp, vp, i64, i64, vp, i32, vp], i32),
                "qerl_nvfp4_lora_linear_fwd": ([vp, i64, i64, i64, vp, vp, vp, vp, vp, i32, f32, vp, vp, vp,
                                                sz, vp], i32),
                "qerl_nvfp4_lora_linear_fwd_noalloc": ([vp, i64, i64, i64, vp, vp, vp, vp, vp, i32, f32, vp, vp,
                                                        vp], i32),
                "qerl_nvfp4_lora_linear_bwd": ([vp, vp, i64, i64, i64, vp, vp, vp, vp, vp, i32, f32, vp, vp,
                                                vp, vp, i32, vp, sz, vp], i32),
                "qerl_nvfp4_pack_codes": ([vp, i64, i64, vp, vp], i32),
                "qerl_nvfp4_unpack_codes": ([vp, i64, i64, vp, vp], i32),
                "qerl_aqn_rmsnorm": ([vp, i64, i64, vp, f32, f32, u64, u64, u32, vp, vp, sz, vp], i32),
                "qerl_aqn_rmsnorm_mode": ([vp, i64, i64, vp, f32, f32, u64, u64, u32, i32, vp, vp, sz, vp], i32),
                "qerl_aqn_noise": ([i64, u64, u64, u32, vp, vp, vp], i32),
                "qerl_aqn_sigma": ([i64, i64, f32, f32, i32], f32),
                "qerl_workspace_bytes": ([i32, i64, i64, i64, i32], sz),
                "qerl_get_error": ([vp], i32),
                "qerl_status_string": ([i32], C.c_char_p),
                "qerl_set_linear_algo": ([i32], i32),
                "qerl_set_launch_chaining": ([i32], i32),
                "qerl_launch_count": ([], u64),
                "qerl_kernel_launch_count": ([i32], u64),
            }
            sig["qerl_lora_linear_fwd_grouped_ws_bytes"] = ([i64, i64, i32, vp, i32], sz)
            sig["qerl_nvfp4_lora_linear_fwd_grouped"] = ([vp, i64, i64, i32, f32, vp, i32, i32, vp, sz, vp], i32)
            sig["qerl_mxfp4_quantize"] = ([vp, i64, i64, i64, vp, vp, vp], i32)
            sig["qerl_mxfp4_lora_linear_fwd"] = ([vp, i64, i64, i64, vp, vp, vp, vp, i32, f32, vp, vp, vp, sz, vp], i32)
            sig["qerl_nvfp4_lora_linear_fwd_f32ab"] = ([vp, i64, i64, i64, vp, vp, vp, vp, vp, i32, f32, vp, vp, vp,
                                                        sz, vp], i32)
            sig["qerl_decoder_chain_ws_bytes"] = ([vp, i32], sz)
            sig["qerl_decoder_chain_plan"] = ([vp, i32, vp, vp, vp, vp, sz, vp], i32)
            sig["qerl_decoder_chain_run"] = ([vp, f32, u64, u64, u32, vp], i32)
            sig["qerl_decoder_chain_destroy"] = ([vp], None)
            sig["qerl_residual_add"] = ([vp, vp, i64, vp, vp], i32)
            sig["qerl_swiglu"] = ([vp, vp, i64, vp, vp], i32)
            sig["qerl_prefix_attention_ws_bytes"] = ([vp], sz)
            sig["qerl_prefix_attention"] = ([vp, vp, vp, vp, vp, vp, vp, vp, f32, vp, vp, vp, sz, vp], i32)
            sig["qerl_token_logp"] = ([vp, i32, i64, i64, i64, vp, i32, vp, f32, vp, vp, vp], i32)
            sig["qerl_policy_loss"] = ([vp, i32, i64, i64, i64, vp, i32, vp, vp, vp, vp, vp, vp, vp, vp, vp, i64, vp,
                                        sz, vp], i32)
            sig["qerl_adamw_ws_bytes"] = ([vp, i64], sz)
            sig["qerl_adamw_plan"] = ([vp, i64, vp, vp, sz, vp], i32)
            sig["qerl_adamw_step"] = ([vp, vp, vp, vp], i32)
            sig["qerl_adamw_read_state"] = ([vp, vp, vp, i32, vp], i32)
            sig["qerl_adamw_destroy"] = ([vp], None)
            sig["qerl_kv4_append"] = ([vp, i64, vp, vp, vp, vp, vp, vp, vp], i32)
            sig["qerl_kv4_read"] = ([vp, i64, vp, vp, vp, vp, vp, vp], i32)
            sig["qerl_kv4_attention_ws_bytes"] = ([vp, vp, vp], sz)
            sig["qerl_kv4_attention"] = ([vp, vp, vp, vp, vp, vp, f32, vp, vp, vp, sz, vp], i32)
            sig["qerl_sample"] = ([vp, i32, i64, i64, i64, vp, vp, vp, vp, vp, vp], i32)
            sig["qerl_nvfp4_lora_linear_fwd_packed"] = sig["qerl_nvfp4_lora_linear_fwd"]
            sig["qerl_nvfp4_lora_linear_bwd_packed"] = sig["qerl_nvfp4_lora_linear_bwd"]
            for name, (args, res) in sig.items():
                fn = getattr(L, name)
                fn.argtypes = args
                fn.restype = res
            _lib = L
    return _lib


def status_string(status: int) -> str:
    return lib().qerl_status_string(status).decode()


def _check(status: int, where: str):
    if status != QERL_OK:
        raise QerlError(status, where)


def _p(t):
    return None if t is None else t.data_ptr()


# The current stream's handle without the Stream object around it, whose making takes longer than a small kernel.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream=None):
    if stream is not None:
        return stream.cuda_stream
    if _raw_stream is None or not torch.cuda.is_initialized():
        return torch.cuda.current_stream().cuda_stream
    return _raw_stream(torch._C._cuda_getDevice())


def workspace_bytes(op: int, M: int, N: int, K: int, r: int) -> int:
    return lib().qerl_workspace_bytes(op, M, N, K, r)


def workspace(op: int, M: int, N: int, K: int, r: int, device="cuda") -> torch.Tensor:
    """A caller-owned scratch buffer of the size the library asks for."""
    return torch.empty(max(workspace_bytes(op, M, N, K, r), 1), dtype=torch.uint8, device=device)


def _here(*tensors):
    """All of them on the current device, whose stream the call is launched on."""
    device = torch._C._cuda_getDevice()
    for t in tensors:
        assert t is None or t.get_device() == device


def _new(make, stream, *args, **kw):
    """make(*args, **kw), a tensor of a call's own.  With `stream` it comes from that stream's memory, so that nothing still
    queued elsewhere for its last owner meets the call; the caller goes on with it on the current stream."""
    if stream is None:
        return make(*args, **kw)
    current = torch.cuda.current_stream()
    with torch.cuda.stream(stream):
        t = make(*args, **kw)
    t.record_stream(current)
    return t


def _hold(stream, handle, seen, tensors):
    """Called for a launch stream that is not among `seen`, those that an object was launched on (at first the one that it was
    made on): its own tensors then stay allocated, after it is dropped, until that stream has finished with them."""
    for t in tensors:
        t.record_stream(torch.cuda.current_stream() if stream is None else stream)
    seen.add(handle)


def set_linear_algo(algo: int):
    _check(lib().qerl_set_linear_algo(algo), "qerl_set_linear_algo")


def set_launch_chaining(on: bool):
    """Programmatic dependent launches between consecutive calls (default on)."""
    _check(lib().qerl_set_launch_chaining(int(bool(on))), "qerl_set_launch_chaining")


def launch_count() -> int:
    return lib().qerl_launch_count()


def kernel_launch_count(kernel: int) -> int:
    """Launches of one of KERNEL_*, between which a call chooses by its sizes."""
    return lib().qerl_kernel_launch_count(kernel)


def get_error(stream=None) -> int:
    return lib().qerl_get_error(_stream(stream))


# ---------------------------------------------------------------- quantizer
def qerl_nvfp4_quantize(W: torch.Tensor, scale_round: int = SCALE_ROUND_UP, out=None, ws=None, stream=None):
    """W bf16 [N, K] (row stride W.stride(0)) -> (codes u8 [N,K/2], scales u8 [N,K/16], s_t f32 [1])."""
    assert W.dtype == torch.bfloat16 and W.dim() == 2 and W.stride(1) == 1
    N, K = W.shape
    if out is None:
        out = (_new(torch.empty, stream, N, K // 2, dtype=torch.uint8, device=W.device),
               _new(torch.empty, stream, N, K // 16, dtype=torch.uint8, device=W.device),
               _new(torch.empty, stream, 1, dtype=torch.float32, device=W.device))
    codes, scales, ts = out
    ws = _new(workspace, stream, OP_QUANTIZE, 0, N, K, 0, W.device) if ws is None else ws
    opts = _QuantOpts(scale_round)
    _check(lib().qerl_nvfp4_quantize(_p(W), N, K, W.stride(0), _p(codes), _p(scales), _p(ts), C.byref(opts),
                                     _p(ws), ws.numel(), _stream(stream)), "qerl_nvfp4_quantize")
    return codes, scales, ts


def qerl_nvfp4_dequantize(codes, scales, tensor_scale, N: int, K: int, apply_tensor_scale: bool = True,
                          out=None, stream=None):
    out = _new(torch.empty, stream, N, K, dtype=torch.bfloat16, device=codes.device) if out is None else out
    _check(lib().qerl_nvfp4_dequantize(_p(codes), _p(scales), _p(tensor_scale), N, K, _p(out),
                                       int(apply_tensor_scale), _stream(stream)), "qerl_nvfp4_dequantize")
    return out


# ---------------------------------------------------------------- linear
def _fwd(name, x, codes, scales, tensor_scale, A, B, lora_scale, y, t_out, ws, stream):
    M, K = x.shape
    N, r = B.shape
    y = _new(torch.empty, stream, M, N, dtype=torch.bfloat16, device=x.device) if y is None else y
    ws = _new(workspace, stream, OP_LINEAR_FWD, M, N, K, r, x.device) if ws is None else ws
    _check(getattr(lib(), name)(_p(x), M, K, N, _p(codes), _p(scales), _p(tensor_scale), _p(A), _p(B), r,
                                float(lora_scale), _p(y), _p(t_out), _p(ws), ws.numel(), _stream(stream)), name)
    return y


def qerl_nvfp4_lora_linear_fwd(x, codes, scales, tensor_scale, A, B, lora_scale: float, y=None, t_out=None,
                               ws=None, stream=None):
    """y = x w_hat^T + s (x A^T) B^T.  x bf16 [M,K], A bf16 [r,K], B bf16 [N,r] -> y bf16 [M,N]."""
    return _fwd("qerl_nvfp4_lora_linear_fwd", x, codes, scales, tensor_scale, A, B, lora_scale, y, t_out, ws, stream)


def qerl_nvfp4_lora_linear_fwd_packed(x, packed_codes, scales, tensor_scale, A, B, lora_scale: float, y=None,
                                      t_out=None, ws=None, stream=None):
    """The forward with the codes in the packed layout (qerl_nvfp4_pack_codes)."""
    return _fwd("qerl_nvfp4_lora_linear_fwd_packed", x, packed_codes, scales, tensor_scale, A, B, lora_scale, y,
                t_out, ws, stream)


class _Group(C.Structure):
    _fields_ = [("N", C.c_int64), ("codes", C.c_void_p), ("scales", C.c_void_p), ("tensor_scale", C.c_void_p),
                ("A", C.c_void_p), ("B", C.c_void_p), ("y", C.c_void_p), ("t_out", C.c_void_p)]


def grouped_ws_bytes(M: int, K: int, r: int, Ns) -> int:
    arr = (C.c_int64 * len(Ns))(*Ns)
    return lib().qerl_lora_linear_fwd_grouped_ws_bytes(M, K, r, C.cast(arr, C.c_void_p), len(Ns))


def qerl_nvfp4_lora_linear_fwd_grouped(x, groups, lora_scale: float, packed: bool = False, ys=None, t_outs=None,
                                       ws=None, stream=None):
    """Linears sharing x: groups = [(codes, scales, tensor_scale, A, B), ...].  Returns [y_g]."""
    M, K = x.shape
    r = groups[0][3].shape[0]
    Ns = [g[4].shape[0] for g in groups]
    ys = [_new(torch.empty, stream, M, N, dtype=torch.bfloat16, device=x.device) for N in Ns] if ys is None else ys
    t_outs = [None] * len(groups) if t_outs is None else t_outs
    arr = (_Group * len(groups))()
    for i, (codes, scales, ts, A, B) in enumerate(groups):
        arr[i] = _Group(Ns[i], _p(codes), _p(scales), _p(ts), _p(A), _p(B), _p(ys[i]), _p(t_outs[i]))
    if ws is None:
        ws = _new(torch.empty, stream, max(grouped_ws_bytes(M, K, r, Ns), 1), dtype=torch.uint8, device=x.device)
    _check(lib().qerl_nvfp4_lora_linear_fwd_grouped(_p(x), M, K, r, float(lora_scale), C.cast(arr, C.c_void_p),
                                                    len(groups), int(bool(packed)), _p(ws), ws.numel(),
                                                    _stream(stream)), "qerl_nvfp4_lora_linear_fwd_grouped")
    return ys


def qerl_nvfp4_pack_codes(codes, out=None, stream=None):
    """Standard NVFP4 codes [N, K/2] -> the packed layout (same shape; out may be codes itself)."""
    N, half = codes.shape
    out = _new(torch.empty_like, stream, codes) if out is None else out
    _check(lib().qerl_nvfp4_pack_codes(_p(codes), N, 2 * half, _p(out), _stream(stream)), "qerl_nvfp4_pack_codes")
    return out


def qerl_nvfp4_unpack_codes(packed, out=None, stream=None):
    """Inverse of qerl_nvfp4_pack_codes."""
    N, half = packed.shape
    out = _new(torch.empty_like, stream, packed) if out is None else out
    _check(lib().qerl_nvfp4_unpack_codes(_p(packed), N, 2 * half, _p(out), _stream(stream)),
           "qerl_nvfp4_unpack_codes")
    return out


def qerl_nvfp4_lora_linear_fwd_noalloc(x, codes, scales, tensor_scale, A, B, lora_scale: float, y=None,
                                       t_out=None, stream=None):
    """The forward with the library's fixed device scratch instead of a workspace
    (for callers that cannot allocate device memory; see include/qerl.h)."""
    M, K = x.shape
    N, r = B.shape
    y = _new(torch.empty, stream, M, N, dtype=torch.bfloat16, device=x.device) if y is None else y
    _check(lib().qerl_nvfp4_lora_linear_fwd_noalloc(_p(x), M, K, N, _p(codes), _p(scales), _p(tensor_scale), _p(A),
                                                    _p(B), r, float(lora_scale), _p(y), _p(t_out), _stream(stream)),
           "qerl_nvfp4_lora_linear_fwd_noalloc")
    return y


def qerl_nvfp4_lora_linear_bwd(dy, x, codes, scales, tensor_scale, A, B, lora_scale: float, t_saved=None,
                               dx=None, dA=None, dB=None, accumulate: bool = False, want=("dx", "dA", "dB"),
                               ws=None, stream=None):
    """Returns (dx bf16 [M,K], dA f32 [r,K], dB f32 [N,r]); outputs not in ``want`` are None."""
    return _bwd("qerl_nvfp4_lora_linear_bwd", dy, x, codes, scales, tensor_scale, A, B, lora_scale, t_saved, dx, dA,
                dB, accumulate, want, ws, stream)


def qerl_nvfp4_lora_linear_bwd_packed(dy, x, packed_codes, scales, tensor_scale, A, B, lora_scale: float,
                                      t_saved=None, dx=None, dA=None, dB=None, accumulate: bool = False,
                                      want=("dx", "dA", "dB"), ws=None, stream=None):
    """The backward with the codes in the packed layout."""
    return _bwd("qerl_nvfp4_lora_linear_bwd_packed", dy, x, packed_codes, scales, tensor_scale, A, B, lora_scale,
                t_saved, dx, dA, dB, accumulate, want, ws, stream)


def _bwd(name, dy, x, codes, scales, tensor_scale, A, B, lora_scale, t_saved, dx, dA, dB, accumulate, want, ws,
         stream):
    M, N = dy.shape
    K = x.shape[1]
    r = A.shape[0]
    dev = x.device
    if dx is None and "dx" in want:
        dx = _new(torch.empty, stream, M, K, dtype=torch.bfloat16, device=dev)
    if dA is None and "dA" in want:
        dA = _new(torch.zeros, stream, r, K, dtype=torch.float32, device=dev)
    if dB is None and "dB" in want:
        dB = _new(torch.zeros, stream, N, r, dtype=torch.float32, device=dev)
    ws = _new(workspace, stream, OP_LINEAR_BWD, M, N, K, r, dev) if ws is None else ws
    _check(getattr(lib(), name)(_p(dy), _p(x), M, K, N, _p(codes), _p(scales), _p(tensor_scale), _p(A), _p(B), r,
                                float(lora_scale), _p(t_saved), _p(dx), _p(dA), _p(dB), int(accumulate), _p(ws),
                                ws.numel(), _stream(stream)), name)
    return dx, dA, dB


# ---------------------------------------------------------------- format variants
def qerl_mxfp4_quantize(W: torch.Tensor, out=None, stream=None):
    """W bf16 [N, K] -> (codes u8 [N, K/2], E8M0 scales u8 [N, K/32])."""
    assert W.dtype == torch.bfloat16 and W.dim() == 2 and W.stride(1) == 1
    N, K = W.shape
    if out is None:
        out = (_new(torch.empty, stream, N, K // 2, dtype=torch.uint8, device=W.device),
               _new(torch.empty, stream, N, K // 32, dtype=torch.uint8, device=W.device))
    codes, scales = out
    _check(lib().qerl_mxfp4_quantize(_p(W), N, K, W.stride(0), _p(codes), _p(scales), _stream(stream)),
           "qerl_mxfp4_quantize")
    return codes, scales


def qerl_mxfp4_lora_linear_fwd(x, codes, scales, A, B, lora_scale: float, y=None, t_out=None, ws=None, stream=None):
    M, K = x.shape
    N, r = B.shape
    y = _new(torch.empty, stream, M, N, dtype=torch.bfloat16, device=x.device) if y is None else y
    ws = _new(workspace, stream, OP_MXFP4_FWD, M, N, K, r, x.device) if ws is None else ws
    _check(lib().qerl_mxfp4_lora_linear_fwd(_p(x), M, K, N, _p(codes), _p(scales), _p(A), _p(B), r, float(lora_scale),
                                            _p(y), _p(t_out), _p(ws), ws.numel(), _stream(stream)),
           "qerl_mxfp4_lora_linear_fwd")
    return y


def qerl_nvfp4_lora_linear_fwd_f32ab(x, codes, scales, tensor_scale, A, B, lora_scale: float, y=None, t_out=None,
                                     ws=None, stream=None):
    """The forward with FP32 LoRA adapters A [r, K] and B [N, r] (float32)."""
    assert A.dtype == torch.float32 and B.dtype == torch.float32
    M, K = x.shape
    N, r = B.shape
    y = _new(torch.empty, stream, M, N, dtype=torch.bfloat16, device=x.device) if y is None else y
    ws = _new(workspace, stream, OP_LINEAR_FWD_F32AB, M, N, K, r, x.device) if ws is None else ws
    _check(lib().qerl_nvfp4_lora_linear_fwd_f32ab(_p(x), M, K, N, _p(codes), _p(scales), _p(tensor_scale), _p(A),
                                                  _p(B), r, float(lora_scale), _p(y), _p(t_out), _p(ws), ws.numel(),
                                                  _stream(stream)),
           "qerl_nvfp4_lora_linear_fwd_f32ab")
    return y


# ---------------------------------------------------------------- decoder-layer glue
def qerl_residual_add(h, y, out=None, stream=None):
    """out = bf16(h + y) elementwise (bf16 tensors of one shape); out may be h."""
    assert h.shape == y.shape and h.dtype == y.dtype == torch.bfloat16
    out = _new(torch.empty_like, stream, h) if out is None else out
    _check(lib().qerl_residual_add(_p(h), _p(y), h.numel(), _p(out), _stream(stream)), "qerl_residual_add")
    return out


def qerl_swiglu(g, u, out=None, stream=None):
    """out = bf16(silu(g) * u) elementwise (bf16 tensors of one shape)."""
    assert g.shape == u.shape and g.dtype == u.dtype == torch.bfloat16
    out = _new(torch.empty_like, stream, g) if out is None else out
    _check(lib().qerl_swiglu(_p(g), _p(u), g.numel(), _p(out), _stream(stream)), "qerl_swiglu")
    return out


# ---------------------------------------------------------------- AQN
def qerl_aqn_rmsnorm(x, gamma, eps: float, sigma: float, seed: int, step: int, layer_id: int, y=None, ws=None,
                     stream=None, noise_mode: int = None):
    """noise_mode None: qerl_aqn_rmsnorm (additive); AQN_NOISE_ADD / AQN_NOISE_MUL:
    qerl_aqn_rmsnorm_mode."""
    M, H = x.shape
    y = _new(torch.empty_like, stream, x) if y is None else y
    ws = _new(workspace, stream, OP_AQN_RMSNORM, M, 0, H, 0, x.device) if ws is None else ws
    if noise_mode is None:
        _check(lib().qerl_aqn_rmsnorm(_p(x), M, H, _p(gamma), float(eps), float(sigma), seed, step, layer_id, _p(y),
                                      _p(ws), ws.numel(), _stream(stream)), "qerl_aqn_rmsnorm")
    else:
        _check(lib().qerl_aqn_rmsnorm_mode(_p(x), M, H, _p(gamma), float(eps), float(sigma), seed, step, layer_id,
                                           int(noise_mode), _p(y), _p(ws), ws.numel(), _stream(stream)),
               "qerl_aqn_rmsnorm_mode")
    return y


def qerl_aqn_noise(H: int, seed: int, step: int, layer_id: int, want_raw: bool = False, device="cuda",
                   stream=None):
    z = _new(torch.empty, stream, H, dtype=torch.float32, device=device)
    raw = _new(torch.empty, stream, H, dtype=torch.int64, device=device) if want_raw else None
    _check(lib().qerl_aqn_noise(H, seed, step, layer_id, _p(z), _p(raw), _stream(stream)), "qerl_aqn_noise")
    return (z, raw) if want_raw else z


def qerl_aqn_sigma(step: int, total_steps: int, sigma_start: float, sigma_end: float, num_stages: int) -> float:
    return lib().qerl_aqn_sigma(step, total_steps, sigma_start, sigma_end, num_stages)


# ---------------------------------------------------------------- decoder chain
class _LinW(C.Structure):
    _fields_ = [("codes", C.c_void_p), ("scales", C.c_void_p), ("tensor_scale", C.c_void_p), ("A", C.c_void_p),
                ("B", C.c_void_p)]


CHAIN_LINEARS = ("q", "k", "v", "o", "gate", "up", "down")


class _Layer(C.Structure):
    _fields_ = [(n, _LinW) for n in CHAIN_LINEARS] + [
        ("gamma_attn", C.c_void_p), ("gamma_mlp", C.c_void_p), ("attn", C.c_void_p), ("q_out", C.c_void_p),
        ("k_out", C.c_void_p), ("v_out", C.c_void_p)]


class _Dims(C.Structure):
    _fields_ = [("M", C.c_int64), ("hidden", C.c_int64), ("q_dim", C.c_int64), ("kv_dim", C.c_int64),
                ("intermediate", C.c_int64), ("r", C.c_int), ("lora_scale", C.c_float), ("eps", C.c_float)]


def decoder_chain_ws_bytes(M, hidden, q_dim, kv_dim, intermediate, r, lora_scale, eps, n_layers) -> int:
    d = _Dims(M, hidden, q_dim, kv_dim, intermediate, r, lora_scale, eps)
    return lib().qerl_decoder_chain_ws_bytes(C.byref(d), n_layers)


class DecoderChain:
    """A planned chain of decoder layers (qerl_decoder_chain_plan / _run).

    layers: one dict per layer with the seven linears under "q", "k", "v", "o",
    "gate", "up", "down" as (packed codes, scales, tensor_scale, A, B), and
    "gamma_attn", "gamma_mlp", "attn" (bf16 [M, hidden]) and optional "q_out",
    "k_out", "v_out".  The tensors are kept referenced while the plan lives."""

    def __init__(self, layers, M, hidden, q_dim, kv_dim, intermediate, r, lora_scale, eps, x_in, x_out, ws=None):
        self._keep = [[{k: Ly[k] for k in Ly} for Ly in layers], x_in, x_out]
        d = _Dims(M, hidden, q_dim, kv_dim, intermediate, r, lora_scale, eps)
        n = lib().qerl_decoder_chain_ws_bytes(C.byref(d), len(layers))
        if n == 0:
            raise QerlError(2, "qerl_decoder_chain_ws_bytes")
        self.ws = torch.empty(n, dtype=torch.uint8, device=x_in.device) if ws is None else ws
        self._launched_on = {_stream()}
        arr = (_Layer * len(layers))()
        for i, Ly in enumerate(layers):
            for nm in CHAIN_LINEARS:
                codes, scales, ts, A, B = Ly[nm]
                setattr(arr[i], nm, _LinW(_p(codes), _p(scales), _p(ts), _p(A), _p(B)))
            arr[i].gamma_attn = _p(Ly["gamma_attn"])
            arr[i].gamma_mlp = _p(Ly["gamma_mlp"])
            arr[i].attn = _p(Ly["attn"])
            arr[i].q_out = _p(Ly.get("q_out"))
            arr[i].k_out = _p(Ly.get("k_out"))
            arr[i].v_out = _p(Ly.get("v_out"))
        h = C.c_void_p()
        _check(lib().qerl_decoder_chain_plan(C.cast(arr, C.c_void_p), len(layers), C.byref(d), _p(x_in), _p(x_out),
                                             _p(self.ws), self.ws.numel(), C.byref(h)), "qerl_decoder_chain_plan")
        self._h = h

    def run(self, sigma: float, seed: int, step: int, first_layer: int = 0, stream=None):
        handle = _stream(stream)
        if handle not in self._launched_on:
            _hold(stream, handle, self._launched_on, (self.ws,))
        _check(lib().qerl_decoder_chain_run(self._h, float(sigma), seed, step, first_layer, handle),
               "qerl_decoder_chain_run")

    def close(self):
        if self._h:
            lib().qerl_decoder_chain_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


# ---------------------------------------------------------------- attention over shared prefixes
class _AttnDims(C.Structure):
    _fields_ = [(n, C.c_int64) for n in ("B", "Lq", "Hq", "Hkv", "D", "n_prefix", "P", "S")] + [
        (n, C.c_int64 * 3) for n in ("q_stride", "out_stride", "k_prefix_stride", "v_prefix_stride", "k_suffix_stride",
                                     "v_suffix_stride")]


class PrefixAttention:
    """Attention of a rollout batch over shared prefixes and per-sequence suffixes
    (qerl_prefix_attention), for caches that stay in place from step to step.

    k_prefix, v_prefix: bf16 [n_prefix, P, Hkv, D]; k_suffix, v_suffix: bf16
    [B, S, Hkv, D] (any strides that are multiples of 8, last dimension
    contiguous); sequence b reads prefix b // (B // n_prefix).  q_heads: query
    heads; q_len: new tokens per sequence and call; scale: 1 / sqrt(D) if None.
    The tensors are kept referenced; the workspace is this object's (calls that
    may overlap need an object each).  A stream other than the one that was
    current when the object was made has to wait for that one before its first
    run, as for any tensor made there."""

    def __init__(self, k_prefix, v_prefix, k_suffix, v_suffix, q_heads: int, q_len: int = 1, scale: float = None, ws=None):
        n, P, Hkv, D = k_prefix.shape
        B, S = k_suffix.shape[:2]
        for t in (k_prefix, v_prefix, k_suffix, v_suffix):
            assert t.dtype == torch.bfloat16 and t.dim() == 4 and (t.stride(3) == 1 or t.numel() == 0)
        assert v_prefix.shape == k_prefix.shape and v_suffix.shape == k_suffix.shape and k_suffix.shape[2:] == (Hkv, D)
        self._keep = (k_prefix, v_prefix, k_suffix, v_suffix)
        st = lambda t: (C.c_int64 * 3)(*t.stride()[:3])  # noqa: E731
        self._d = _AttnDims(B, q_len, q_heads, Hkv, D, n, P, S)
        self._d.k_prefix_stride, self._d.v_prefix_stride = st(k_prefix), st(v_prefix)
        self._d.k_suffix_stride, self._d.v_suffix_stride = st(k_suffix), st(v_suffix)
        nbytes = lib().qerl_prefix_attention_ws_bytes(C.byref(self._d))
        if nbytes == 0:
            raise QerlError(2, "qerl_prefix_attention_ws_bytes")
        self.ws = torch.empty(nbytes, dtype=torch.uint8, device=k_suffix.device) if ws is None else ws
        self._ws = (self.ws.data_ptr(), self.ws.numel())
        self._launched_on = {_stream()}
        self._q_shape = torch.Size((B, q_len, q_heads, D))
        self._scale = D ** -0.5 if scale is None else float(scale)
        self._p = [_p(t) for t in self._keep]
        self._strides = None  # of the last q and out
        self._ref = C.byref(self._d)

    def run(self, q, suffix_lens, prefix_lens=None, out=None, lse=None, stream=None):
        """q bf16 [B, Lq, Hq, D], suffix_lens int32 [B] (new tokens included),
        prefix_lens int32 [n_prefix] or None (P) -> out bf16 like q; lse f32 [B, Lq, Hq] is filled if given."""
        d = self._d
        if out is None:
            out = _new(torch.empty, stream, self._q_shape, dtype=torch.bfloat16, device=q.device)
        assert q.shape == self._q_shape and out.shape == self._q_shape and q.dtype == out.dtype == torch.bfloat16
        assert suffix_lens.dtype == torch.int32 and suffix_lens.is_contiguous() and suffix_lens.numel() == d.B
        if prefix_lens is not None:
            assert prefix_lens.dtype == torch.int32 and prefix_lens.is_contiguous() and prefix_lens.numel() == d.n_prefix
        if lse is not None:
            assert lse.dtype == torch.float32 and lse.is_contiguous() and lse.shape == self._q_shape[:3]
        strides = (q.stride(), out.stride())
        if strides != self._strides:
            assert strides[0][3] == strides[1][3] == 1
            d.q_stride[:], d.out_stride[:] = strides[0][:3], strides[1][:3]
            self._strides = strides
        handle = _stream(stream)
        if handle not in self._launched_on:
            _hold(stream, handle, self._launched_on, (self.ws,))
        kp, vp, ks, vs = self._p
        _check(lib().qerl_prefix_attention(self._ref, q.data_ptr(), kp, vp, _p(prefix_lens), ks, vs, suffix_lens.data_ptr(),
                                           self._scale, out.data_ptr(), _p(lse), self._ws[0], self._ws[1], handle),
               "qerl_prefix_attention")
        return out


def qerl_prefix_attention(q, k_prefix, v_prefix, k_suffix, v_suffix, suffix_lens, prefix_lens=None, scale: float = None,
                          out=None, lse=None, ws=None, stream=None):
    """One call of PrefixAttention: out bf16 [B, Lq, Hq, D]."""
    with contextlib.nullcontext() if stream is None else torch.cuda.stream(stream):  # the workspace is that stream's
        plan = PrefixAttention(k_prefix, v_prefix, k_suffix, v_suffix, q.shape[2], q.shape[1], scale, ws)
    return plan.run(q, suffix_lens, prefix_lens, out, lse, stream)


# ---------------------------------------------------------------- keys and values in 4 bits
class _Kv4Cache(C.Structure):
    _fields_ = [("data", C.c_void_p)] + [(n, C.c_int64) for n in ("n", "T", "Hkv", "D")] + [
        ("stride", C.c_int64 * 3), ("k_scale", C.c_float), ("v_scale", C.c_float)]


class _Kv4AttnDims(C.Structure):
    _fields_ = [(n, C.c_int64) for n in ("B", "Lq", "Hq")] + [("q_stride", C.c_int64 * 3), ("out_stride", C.c_int64 * 3)]


class Kv4Cache:
    """Keys and values of n sequences in NVFP4, up to T tokens each (qerl_kv4_cache): append and read.

    k_scale, v_scale: the fixed factors of the keys' and the values' scales (values from about 1e-3 to 2688 times the
    factor are held well).  data: uint8 [n, Hkv, ceil(T / 32), 36 D], zeros if None; its strides may be any multiples of 16
    with the last dimension contiguous.  A stream other than the one that was current when the object was made has to
    wait for that one before its first call, as for any tensor made there."""

    def __init__(self, n: int, T: int, Hkv: int, D: int, k_scale: float = 1.0, v_scale: float = 1.0, device="cuda", data=None):
        shape = (n, Hkv, -(-T // 32), 36 * D)
        self._own = data is None
        self.data = torch.zeros(shape, dtype=torch.uint8, device=device) if data is None else data
        assert self.data.shape == shape and self.data.dtype == torch.uint8 and self.data.stride(3) == 1
        self.n, self.T, self.Hkv, self.D = n, T, Hkv, D
        self._rows, self._lens = (n, Hkv, D), torch.Size((n,))
        self._last = (None, None, None)  # the last tokens' strides, and as the library takes them: one tuple, for threads' sake
        self._c = _Kv4Cache(self.data.data_ptr(), n, T, Hkv, D, (C.c_int64 * 3)(*self.data.stride()[:3]), k_scale, v_scale)
        self._ref = C.byref(self._c)
        self._launched_on = {_stream()} if self.data.is_cuda else set()

    def _tokens(self, k, v, lens):
        shape = k.shape
        assert k.dtype == v.dtype == torch.bfloat16 and shape == v.shape and (shape[0], shape[2], shape[3]) == self._rows
        assert lens.dtype == torch.int32 and lens.shape == self._lens and lens.is_contiguous()
        strides, last = (k.stride(), v.stride()), self._last
        if strides != last[0]:
            assert (strides[0][3] == strides[1][3] == 1) or k.numel() == 0
            last = (strides, *((C.c_int64 * 3)(*t[:3]) for t in strides))
            if k.numel():
                self._last = last
        return k.data_ptr() or 16, last[1], v.data_ptr() or 16, last[2]  # an empty tensor has no address

    def _launch(self, stream):
        handle = _stream(stream)
        if self._own and handle not in self._launched_on:
            _hold(stream, handle, self._launched_on, (self.data,))
        return handle

    def append(self, k, v, lens, counts=None, stream=None):
        """k, v bf16 [n, L, Hkv, D]: the last tokens of sequences that are lens (int32 [n]) long with them; counts
        (int32 [n]): how many of the L each sequence has, all if None."""
        args = self._tokens(k, v, lens)
        assert counts is None or (counts.dtype == torch.int32 and counts.is_contiguous() and counts.numel() == self.n)
        _here(self.data, k, v, lens, counts)
        _check(lib().qerl_kv4_append(self._ref, k.shape[1], *args, lens.data_ptr(), _p(counts), self._launch(stream)), "qerl_kv4_append")

    def read(self, lens, L: int, k=None, v=None, stream=None):
        """The values held of the last L tokens of sequences that are lens long: (k, v) bf16 [n, L, Hkv, D]."""
        k = _new(torch.empty, stream, self.n, L, self.Hkv, self.D, dtype=torch.bfloat16, device=self.data.device) if k is None else k
        v = _new(torch.empty, stream, self.n, L, self.Hkv, self.D, dtype=torch.bfloat16, device=self.data.device) if v is None else v
        kp, ks, vp, vs = self._tokens(k, v, lens)
        assert k.shape[1] == L
        _here(self.data, k, v, lens)
        _check(lib().qerl_kv4_read(self._ref, L, lens.data_ptr(), kp, ks, vp, vs, self._launch(stream)), "qerl_kv4_read")
        return k, v


class Kv4Attention:
    """PrefixAttention over 4-bit caches (qerl_kv4_attention).

    suffix: Kv4Cache of the B sequences' own tokens; prefix: Kv4Cache of n_prefix shared ones (sequence b reads prefix
    b // (B // n_prefix)), or None; suffix None: batch sequences that have only their prefix.  The caches are kept
    referenced; the workspace is this object's (calls that may overlap need an object each)."""

    def __init__(self, suffix, q_heads: int, q_len: int = 1, prefix=None, scale: float = None, batch: int = None, ws=None):
        one = suffix if suffix is not None else prefix
        B = suffix.n if suffix is not None else batch
        self._caches = (prefix, suffix)
        device = one.data.device  # of q and the rest too, which run() checks
        assert prefix is None or prefix.data.device == device
        assert ws is None or ws.device == device
        self._pref, self._suf = (None if c is None else c._ref for c in self._caches)
        nbytes = lib().qerl_kv4_attention_ws_bytes(C.byref(_Kv4AttnDims(B, q_len, q_heads)), self._pref, self._suf)
        if nbytes == 0:
            raise QerlError(2, "qerl_kv4_attention_ws_bytes")
        self.ws = torch.empty(nbytes, dtype=torch.uint8, device=device) if ws is None else ws
        self._ws = (self.ws.data_ptr(), self.ws.numel())
        self._launched_on = {_stream()}
        self._q_shape = torch.Size((B, q_len, q_heads, one.D))
        self._scale = one.D ** -0.5 if scale is None else float(scale)
        self._last = (None, None)  # strides of the last q and out, and the call's sizes with them; exchanged whole

    def run(self, q, suffix_lens=None, prefix_lens=None, out=None, lse=None, stream=None):
        """q bf16 [B, Lq, Hq, D], suffix_lens int32 [B] (new tokens included), prefix_lens int32 [n_prefix] or None
        (full) -> out bf16 like q; lse f32 [B, Lq, Hq] is filled if given."""
        prefix, suffix = self._caches
        if out is None:
            out = _new(torch.empty, stream, self._q_shape, dtype=torch.bfloat16, device=q.device)
        assert q.shape == self._q_shape and out.shape == self._q_shape and q.dtype == out.dtype == torch.bfloat16
        assert (suffix is None) == (suffix_lens is None) and (prefix is not None or prefix_lens is None)
        assert suffix is None or (suffix_lens.dtype == torch.int32 and suffix_lens.shape == suffix._lens and suffix_lens.is_contiguous())
        if prefix_lens is not None:
            assert prefix_lens.dtype == torch.int32 and prefix_lens.shape == prefix._lens and prefix_lens.is_contiguous()
        if lse is not None:
            assert lse.dtype == torch.float32 and lse.is_contiguous() and lse.shape == self._q_shape[:3]
        strides, last = (q.stride(), out.stride()), self._last
        if strides != last[0]:
            assert strides[0][3] == strides[1][3] == 1
            dims = _Kv4AttnDims(*self._q_shape[:3], *((C.c_int64 * 3)(*t[:3]) for t in strides))
            last = self._last = (strides, C.byref(dims))
        handle = _stream(stream)
        if handle not in self._launched_on:
            _hold(stream, handle, self._launched_on, (self.ws,))
        for c in self._caches:
            if c is not None and handle not in c._launched_on:
                c._launch(stream)
        _here(self.ws, q, out, suffix_lens, prefix_lens, lse)
        _check(lib().qerl_kv4_attention(last[1], q.data_ptr(), self._pref, _p(prefix_lens), self._suf, _p(suffix_lens), self._scale,
                                        out.data_ptr(), _p(lse), self._ws[0], self._ws[1], handle), "qerl_kv4_attention")
        return out


# ---------------------------------------------------------------- policy loss
class _PolicyOpts(C.Structure):
    _fields_ = [(n, C.c_float) for n in ("clip_low", "clip_high", "beta", "temperature", "grad_scale")]


_DTYPES = {torch.float32: DTYPE_F32, torch.bfloat16: DTYPE_BF16}
_ID_BITS = {torch.int32: 32, torch.int64: 64}


def _logits_args(logits, ids, vectors):
    """(pointer, dtype, T, V, ld, ids pointer, ids bits) of a logits matrix, after the checks of its companions."""
    T, V = shape = logits.shape
    ld, one = logits.stride()
    vec, f32, bits = shape[:1], torch.float32, _ID_BITS[ids.dtype]
    assert logits.dtype in _DTYPES and (one == 1 or V == 1) and ids.shape == vec and ids.is_contiguous()
    for t in vectors:
        assert t is None or (t.dtype is f32 and t.shape == vec and t.is_contiguous())
    return logits.data_ptr(), _DTYPES[logits.dtype], T, V, ld if T > 1 else V, ids.data_ptr(), bits


def qerl_token_logp(logits, ids, weights=None, temperature: float = 1.0, logp=None, entropy=None, stream=None):
    """logits bf16/f32 [T, V], ids int32/int64 [T] -> (logp, entropy) f32 [T]; rows of weight 0 are not read."""
    T = logits.shape[0]
    logp = _new(torch.empty, stream, T, dtype=torch.float32, device=logits.device) if logp is None else logp
    entropy = _new(torch.empty, stream, T, dtype=torch.float32, device=logits.device) if entropy is None else entropy
    args = _logits_args(logits, ids, (weights, logp, entropy))
    _check(lib().qerl_token_logp(*args, _p(weights), float(temperature), _p(logp), _p(entropy), _stream(stream)),
           "qerl_token_logp")
    return logp, entropy


def qerl_policy_loss(logits, ids, old_logp, advantages, weights=None, ref_logp=None, clip_low: float = 0.2,
                     clip_high: float = 0.2, beta: float = 0.0, temperature: float = 1.0, grad_scale: float = 1.0,
                     want_grad: bool = True, dlogits=None, logp=None, entropy=None, sums=None, ws=None, stream=None):
    """Clipped policy loss with a KL term and the gradient of the logits:
    (sums f32 [4] = loss, policy term, KL term, clipped weight; logp f32 [T]; entropy f32 [T]; dlogits like logits,
    or None without want_grad).  dlogits may be logits."""
    T, V = logits.shape
    dev = logits.device
    logp = _new(torch.empty, stream, T, dtype=torch.float32, device=dev) if logp is None else logp
    entropy = _new(torch.empty, stream, T, dtype=torch.float32, device=dev) if entropy is None else entropy
    sums = _new(torch.empty, stream, 4, dtype=torch.float32, device=dev) if sums is None else sums
    if dlogits is None and want_grad:
        dlogits = _new(torch.empty, stream, T, V, dtype=logits.dtype, device=dev)
    ws = _new(workspace, stream, OP_POLICY_LOSS, T, V, 0, 0, dev) if ws is None else ws
    args = _logits_args(logits, ids, (old_logp, ref_logp, advantages, weights, logp, entropy))
    assert sums.dtype == torch.float32 and sums.numel() == 4 and sums.is_contiguous()
    ldd = V
    if dlogits is not None:
        assert dlogits.shape == (T, V) and dlogits.dtype == logits.dtype and (dlogits.stride(1) == 1 or V == 1)
        ldd = dlogits.stride(0) if T > 1 else V
    opts = _PolicyOpts(clip_low, clip_high, beta, temperature, grad_scale)
    _check(lib().qerl_policy_loss(*args, _p(old_logp), _p(ref_logp), _p(advantages), _p(weights), C.byref(opts), _p(sums),
                                  _p(logp), _p(entropy), _p(dlogits), ldd, _p(ws), ws.numel(), _stream(stream)),
           "qerl_policy_loss")
    return sums, logp, entropy, dlogits


class _SampleOpts(C.Structure):
    _fields_ = [(n, C.c_float) for n in ("temperature", "top_p", "min_p")] + [("top_k", C.c_int32)] + [
        (n, C.c_void_p) for n in ("temperatures", "top_ps", "min_ps", "top_ks")]


def qerl_sample(logits, u, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0, ids=None, logp=None, logq=None, stream=None):
    """The next tokens from logits bf16/f32 [T, V] and uniform numbers u f32 [T]: (ids int64 [T], logp f32 [T] in the whole
    distribution, logq f32 [T] in the cut one).  temperature, top_p, min_p: numbers or f32 [T]; top_k: a number or int32 [T]."""
    T, V = shape = logits.shape
    ld, one = logits.stride()
    vec, f32, dev = shape[:1], torch.float32, logits.device
    ids = _new(torch.empty, stream, T, dtype=torch.int64, device=dev) if ids is None else ids
    logp = _new(torch.empty, stream, T, dtype=f32, device=dev) if logp is None else logp
    logq = _new(torch.empty, stream, T, dtype=f32, device=dev) if logq is None else logq
    assert logits.dtype in _DTYPES and (one == 1 or V == 1) and ids.dtype is torch.int64 and ids.shape == vec and ids.is_contiguous()
    for t in (u, logp, logq):
        assert t.dtype is f32 and t.shape == vec and t.is_contiguous()
    o = _SampleOpts(1.0, 1.0, 0.0, 0)
    for name, v, dt in (("temperature", temperature, f32), ("top_p", top_p, f32), ("min_p", min_p, f32), ("top_k", top_k, torch.int32)):
        if isinstance(v, torch.Tensor):
            assert v.dtype is dt and v.shape == vec and v.is_contiguous()
            setattr(o, name + "s", v.data_ptr())
        else:
            setattr(o, name, v if dt is f32 else max(-1, min(v, 0x7FFFFFFF)))  # 32 bits: more would be cut off without a word
    _here(logits, u, ids, logp, logq, *(v for v in (temperature, top_k, top_p, min_p) if isinstance(v, torch.Tensor)))
    _check(lib().qerl_sample(logits.data_ptr(), _DTYPES[logits.dtype], T, V, ld if T > 1 else V, u.data_ptr(), C.byref(o), ids.data_ptr(),
                             logp.data_ptr(), logq.data_ptr(), _stream(stream)), "qerl_sample")
    return ids, logp, logq


# ---------------------------------------------------------------- AdamW
class _AdamTensor(C.Structure):
    _fields_ = [("n", C.c_int64)] + [(n, C.c_void_p) for n in ("param", "master", "grad", "m", "v", "m_scale", "v_scale")] + [
        ("lr_scale", C.c_double), ("weight_decay", C.c_double)]


class _AdamFormat(C.Structure):
    _fields_ = [("param_dtype", C.c_int), ("grad_dtype", C.c_int), ("state_bits", C.c_int)]


class _AdamHyper(C.Structure):
    _fields_ = [(n, C.c_double) for n in ("lr", "beta1", "beta2", "eps", "max_grad_norm")] + [
        ("step", C.c_int64), ("seed", C.c_uint64)]


class AdamW:
    """AdamW over many tensors at once (qerl_adamw_plan / _step).

    params: contiguous f32 tensors, or bf16 ones with f32 `masters`; grads: f32 or
    bf16 of the same shapes.  State: state_bits 32 or 8 allocates zeros (in m, v,
    m_scale, v_scale: lists of tensors); given lists are used as they are, and
    their type (float32 or uint8) sets the bits.  lr_scale and weight_decay: one
    number, or one per tensor.  The tensors are kept referenced."""

    BLOCK = 256

    def __init__(self, params, grads, masters=None, state_bits: int = 32, m=None, v=None, m_scale=None, v_scale=None,
                 betas=(0.9, 0.999), eps: float = 1e-8, weight_decay=0.01, lr_scale=1.0, ws=None):
        self._h = None
        n = len(params)
        assert n > 0 and len(grads) == n and (masters is None or len(masters) == n)
        if m is not None:
            state_bits = 8 if m[0].dtype == torch.uint8 else 32
        sdt = torch.uint8 if state_bits == 8 else torch.float32
        new = lambda: [torch.zeros(p.numel(), dtype=sdt, device=p.device) for p in params]  # noqa: E731
        news = lambda: [torch.zeros(-(-p.numel() // self.BLOCK), dtype=torch.float32, device=p.device) for p in params]  # noqa: E731
        self.params, self.grads, self.masters = list(params), list(grads), None if masters is None else list(masters)
        self.m = new() if m is None else list(m)
        self.v = new() if v is None else list(v)
        self.m_scale = self.v_scale = [None] * n
        if state_bits == 8:
            self.m_scale = news() if m_scale is None else list(m_scale)
            self.v_scale = news() if v_scale is None else list(v_scale)
        per = lambda x: [float(x)] * n if isinstance(x, (int, float)) else [float(k) for k in x]  # noqa: E731
        lrs, wds = per(lr_scale), per(weight_decay)
        assert len(lrs) == n and len(wds) == n
        table = (_AdamTensor * n)()
        ptr = lambda t: None if t is None else t.data_ptr()  # noqa: E731
        for i in range(n):
            p, g, w, c = params[i], grads[i], None if masters is None else masters[i], params[i].numel()
            assert p.dtype == params[0].dtype and g.dtype == grads[0].dtype and p.dtype in _DTYPES and g.dtype in _DTYPES
            assert (w is None) == (p.dtype == torch.float32) and (w is None or w.dtype == torch.float32)
            blocks = -(-c // self.BLOCK)
            for t, size, dt in ((p, c, p.dtype), (g, c, g.dtype), (w, c, torch.float32), (self.m[i], c, sdt), (self.v[i], c, sdt),
                                (self.m_scale[i], blocks, torch.float32), (self.v_scale[i], blocks, torch.float32)):
                assert t is None or (t.numel() == size and t.dtype == dt and t.is_contiguous())
            table[i] = _AdamTensor(c, ptr(p), ptr(w), ptr(g), ptr(self.m[i]), ptr(self.v[i]), ptr(self.m_scale[i]),
                                   ptr(self.v_scale[i]), lrs[i], wds[i])
        nbytes = lib().qerl_adamw_ws_bytes(C.cast(table, C.c_void_p), n)
        if nbytes == 0:
            raise QerlError(1, "qerl_adamw_ws_bytes")
        self.ws = torch.empty(nbytes, dtype=torch.uint8, device=params[0].device) if ws is None else ws
        fmt = _AdamFormat(_DTYPES[params[0].dtype], _DTYPES[grads[0].dtype], state_bits)
        h = C.c_void_p()
        _check(lib().qerl_adamw_plan(C.cast(table, C.c_void_p), n, C.byref(fmt), _p(self.ws), self.ws.numel(), C.byref(h)),
               "qerl_adamw_plan")
        self._h = h
        self._launched_on = {_stream()}
        made = [(m, self.m), (v, self.v)] + ([(m_scale, self.m_scale), (v_scale, self.v_scale)] if state_bits == 8 else [])
        self._own = [self.ws] + [t for given, tensors in made if given is None for t in tensors]
        self._flat = sum(-(-p.numel() // self.BLOCK) for p in params[:-1]) * self.BLOCK + params[-1].numel()
        self._hyper = _AdamHyper(0.0, betas[0], betas[1], eps, 0.0, 1, 0)

    def step(self, lr: float, step: int, seed: int = 0, max_grad_norm: float = 0.0, grad_norm=None, stream=None):
        """Step number `step` (1, 2, ...) with the gradients in place; max_grad_norm > 0 clips by the norm of all of
        them, which goes to grad_norm (f32 [1]) if given."""
        hy = self._hyper
        hy.lr, hy.step, hy.seed, hy.max_grad_norm = lr, step, seed, max_grad_norm
        handle = _stream(stream)
        if handle not in self._launched_on:
            _hold(stream, handle, self._launched_on, self._own)
        _check(lib().qerl_adamw_step(self._h, C.byref(hy), _p(grad_norm), handle), "qerl_adamw_step")

    def read_state(self, m_out, v_out, stream=None):
        """The values of the 8-bit states, f32 or bf16: the tensors in order, each from a multiple of 256 elements on."""
        size = self._flat
        assert m_out.dtype == v_out.dtype and m_out.dtype in _DTYPES and m_out.is_contiguous() and v_out.is_contiguous()
        assert m_out.numel() >= size and v_out.numel() >= size
        handle = _stream(stream)
        if handle not in self._launched_on:
            _hold(stream, handle, self._launched_on, self._own)
        _check(lib().qerl_adamw_read_state(self._h, _p(m_out), _p(v_out), _DTYPES[m_out.dtype], handle),
               "qerl_adamw_read_state")

    def close(self):
        if self._h:
            lib().qerl_adamw_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass
