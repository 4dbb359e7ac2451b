"""Python binding of the VQ MoE expert matmul library (MI355X / gfx950).

Thin ctypes layer over the C ABI in ``include/vq.h``: it marshals torch
device tensors into ``vq_tensor`` descriptors and raw pointers, passes the
current HIP stream, allocates outputs and workspaces with torch, and raises
``VQError`` on a non-zero status.  Every step of the computation runs in the
HIP kernels of ``libvqmm.so``; there is no CPU or PyTorch fallback, and
loading fails loudly when the library is missing or no GPU is present.

Names follow the C ABI: ``vq_dequantize``, ``vq_row_gather``, ``vq_expert_gemv``,
``vq_expert_gemm``, ``vq_moe_ffn`` and their workspace-size queries.
"""
from __future__ import annotations

import ctypes
import functools
import os
import struct
from dataclasses import dataclass
from typing import Optional

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libvqmm.so")

VQ_OK, VQ_ERR_INVALID_ARGUMENT, VQ_ERR_UNSUPPORTED, VQ_ERR_WORKSPACE, VQ_ERR_HIP = range(5)
VQ_F32, VQ_BF16, VQ_F16 = 0, 1, 2
VQ_SCORE_SOFTMAX, VQ_SCORE_SIGMOID = 0, 1
VQ_GATE_NONE, VQ_GATE_TOKEN, VQ_GATE_CHANNEL = 0, 1, 2


class VQError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"{_status_name(status)}: {message}")
        self.status = status


class _CTensor(ctypes.Structure):
    _fields_ = [
        ("rows", ctypes.c_int32), ("cols", ctypes.c_int32), ("d", ctypes.c_int32),
        ("bits", ctypes.c_int32), ("K", ctypes.c_int32), ("n_experts", ctypes.c_int32),
        ("n_stored", ctypes.c_int64),
        ("codebook", ctypes.c_void_p), ("codes", ctypes.c_void_p),
        ("scales", ctypes.c_void_p), ("row_map", ctypes.c_void_p),
    ]


class _CLayer(ctypes.Structure):
    _fields_ = [
        ("gate", ctypes.POINTER(_CTensor)), ("up", ctypes.POINTER(_CTensor)),
        ("down", ctypes.POINTER(_CTensor)),
        ("topk_ids", ctypes.c_void_p), ("topk_weights", ctypes.c_void_p),
    ]


class _CQ4(ctypes.Structure):
    _fields_ = [
        ("rows", ctypes.c_int32), ("cols", ctypes.c_int32), ("group", ctypes.c_int32),
        ("scale_dtype", ctypes.c_int), ("codes", ctypes.c_void_p),
        ("scales", ctypes.c_void_p), ("biases", ctypes.c_void_p),
    ]


class _CRoute(ctypes.Structure):
    _fields_ = [
        ("n_experts", ctypes.c_int32), ("top_k", ctypes.c_int32), ("score", ctypes.c_int32),
        ("renormalize", ctypes.c_int32), ("scale", ctypes.c_float),
    ]


class _CNorm(ctypes.Structure):
    _fields_ = [
        ("n_tokens", ctypes.c_int32), ("hidden", ctypes.c_int32),
        ("h_dtype", ctypes.c_int), ("y_dtype", ctypes.c_int), ("x_dtype", ctypes.c_int),
        ("weight_dtype", ctypes.c_int),
        ("h_stride", ctypes.c_int64), ("y_stride", ctypes.c_int64),
        ("h_out_stride", ctypes.c_int64), ("x_stride", ctypes.c_int64),
        ("h", ctypes.c_void_p), ("y", ctypes.c_void_p), ("post_weight", ctypes.c_void_p),
        ("pre_weight", ctypes.c_void_p), ("gate", ctypes.c_void_p),
        ("gate_kind", ctypes.c_int32), ("eps", ctypes.c_float),
        ("weight_offset", ctypes.c_float), ("skip_scale", ctypes.c_float),
        ("block_scale", ctypes.c_float), ("h_out", ctypes.c_void_p), ("x", ctypes.c_void_p),
    ]


class _CBlock(ctypes.Structure):
    _fields_ = [
        ("gate", ctypes.POINTER(_CTensor)), ("up", ctypes.POINTER(_CTensor)),
        ("down", ctypes.POINTER(_CTensor)),
        ("shared_gate", ctypes.POINTER(_CQ4)), ("shared_up", ctypes.POINTER(_CQ4)),
        ("shared_down", ctypes.POINTER(_CQ4)),
        ("router", ctypes.c_void_p), ("route_bias", ctypes.c_void_p), ("route", _CRoute),
        ("x_dtype", ctypes.c_int), ("weight_dtype", ctypes.c_int),
        ("pre_weight", ctypes.c_void_p), ("post_weight", ctypes.c_void_p),
        ("channel_gate", ctypes.c_void_p), ("eps", ctypes.c_float),
        ("weight_offset", ctypes.c_float), ("skip_scale", ctypes.c_float),
        ("block_scale", ctypes.c_float),
    ]


_lib = None


def build() -> str:
    """Compile libvqmm.so for gfx950 with hipcc (in-tree)."""
    from . import _build
    return _build.build()


def load_library():
    """Load libvqmm.so (building it first only if it does not exist)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        build()
    lib = ctypes.CDLL(LIB_PATH)
    P, I32, I64, SZ = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
    T = ctypes.POINTER(_CTensor)
    sigs = {
        "vq_abi_version": (I32, []),
        "vq_status_string": (ctypes.c_char_p, [ctypes.c_int]),
        "vq_last_error": (ctypes.c_char_p, []),
        "vq_validate": (ctypes.c_int, [T]),
        "vq_dequantize": (ctypes.c_int, [T, I32, P, P]),
        "vq_row_gather": (ctypes.c_int, [T, I64, P, P, P]),
        "vq_fit_workspace_size": (SZ, [I32, I32, I64]),
        "vq_fit": (ctypes.c_int, [I64, I32, I32, I32, I32, P, I64, P, P, I32, P, P, P, P, SZ, P]),
        "vq_expert_gemv": (ctypes.c_int, [T, I32, I32, P, ctypes.c_int, P, P]),
        "vq_expert_gemm_workspace_size": (SZ, [T, I32]),
        "vq_expert_gemm": (ctypes.c_int, [T, I32, P, ctypes.c_int, P, P, P, SZ, P]),
        "vq_moe_ffn_workspace_size": (SZ, [T, T, T, I32, I32]),
        "vq_moe_ffn_engine": (ctypes.c_int, [T, T, T, I32, I32, P]),
        "vq_probe_read": (ctypes.c_int, [P, SZ, I32, P, P]),
        "vq_probe_mfma": (ctypes.c_int, [I32, I32, P, P]),
        "vq_moe_ffn": (ctypes.c_int, [T, T, T, I32, I32, P, ctypes.c_int, P, P, P, P, SZ, P]),
        "vq_moe_ffn_noalloc": (ctypes.c_int, [T, T, T, I32, I32, P, ctypes.c_int, P, P, P, P]),
        "vq_moe_gate_up": (ctypes.c_int, [T, T, I32, I32, P, ctypes.c_int, P, P, P]),
        "vq_moe_down": (ctypes.c_int, [T, I32, I32, P, P, P, P]),
        "vq_moe_combine": (ctypes.c_int, [I32, I32, I32, P, P, P, P]),
        "vq_set_kernel_events": (ctypes.c_int, [P, P]),
        "vq_q4_gemv": (ctypes.c_int, [P, I32, P, ctypes.c_int, P, I32, P]),
        "vq_q4_gate_up": (ctypes.c_int, [P, P, I32, P, ctypes.c_int, P, P]),
        "vq_router_logits": (ctypes.c_int, [I32, I32, P, I32, P, ctypes.c_int, P, P]),
        "vq_moe_route_workspace_size": (SZ, [P, I32]),
        "vq_moe_route": (ctypes.c_int, [P, I32, P, ctypes.c_int, P, P, P, P, P, P, P, SZ, P]),
        "vq_moe_route_grad": (ctypes.c_int, [P, I32, P, ctypes.c_int, P, P, P, P, P, P, P]),
        "vq_block_norm": (ctypes.c_int, [P, P]),
        "vq_moe_block_workspace_size": (SZ, [P, I32]),
        "vq_moe_block": (ctypes.c_int, [P, I32, P, P, P, P, P, P, SZ, P]),
        "vq_block_norm_grad_workspace_size": (SZ, [P]),
        "vq_block_norm_grad": (ctypes.c_int, [P, P, P, P, P, P, P, P, P, SZ, P]),
        "vq_moe_stack_workspace_size": (SZ, [ctypes.POINTER(_CLayer), I32, I32, I32]),
        "vq_moe_stack": (ctypes.c_int, [ctypes.POINTER(_CLayer), I32, I32, I32, P, P, SZ, P]),
    }
    for name, (res, args) in sigs.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    _lib = lib
    return lib


def _status_name(status: int) -> str:
    names = {0: "VQ_OK", 1: "VQ_ERR_INVALID_ARGUMENT", 2: "VQ_ERR_UNSUPPORTED",
             3: "VQ_ERR_WORKSPACE", 4: "VQ_ERR_HIP"}
    return names.get(status, f"status {status}")


def _check(status: int):
    if status != VQ_OK:
        msg = load_library().vq_last_error().decode()
        raise VQError(status, msg)


def _require_gpu():
    if not torch.cuda.is_available():
        raise RuntimeError("vq_dequant_matmul_amd needs a ROCm GPU (gfx950); none is visible")


def _stream():
    return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


@dataclass
class VQTensor:
    """One VQ linear tensor stacked over experts, resident on the GPU.

    codebook: int16 [K, d] (fp16 bit patterns); codes: int32 [n_stored, wpr]
    (uint32 words); scales: int16 [n_stored, cols // 64] (fp16 bit patterns);
    row_map: int32 [n_experts * rows] (stored row or -1) or None (dense).
    """

    rows: int
    cols: int
    d: int
    bits: int
    K: int
    n_experts: int
    codebook: torch.Tensor
    codes: torch.Tensor
    scales: torch.Tensor
    row_map: Optional[torch.Tensor] = None

    @property
    def n_stored(self) -> int:
        return int(self.scales.shape[0])

    @classmethod
    def from_arrays(cls, *, rows, cols, d, bits, K, n_experts, codebook, codes, scales,
                    row_map=None, device="cuda"):
        """Upload numpy arrays (uint16 codebook/scales, uint32 codes, int32
        row map) to the device."""
        import numpy as np

        def up(a, dt):
            return torch.from_numpy(np.ascontiguousarray(a).view(dt)).to(device)
        return cls(rows, cols, d, bits, K, n_experts,
                   up(codebook, np.int16), up(codes, np.int32), up(scales, np.int16),
                   None if row_map is None else up(row_map, np.int32))

    @classmethod
    def from_host(cls, h, device="cuda"):
        """From any host object with the same attribute names (numpy arrays)."""
        return cls.from_arrays(rows=h.rows, cols=h.cols, d=h.d, bits=h.bits, K=h.K,
                               n_experts=h.n_experts, codebook=h.codebook, codes=h.codes,
                               scales=h.scales, row_map=h.row_map, device=device)

    def clone(self) -> "VQTensor":
        """A copy at new device addresses (same contents)."""
        return VQTensor(self.rows, self.cols, self.d, self.bits, self.K, self.n_experts,
                        self.codebook.clone(), self.codes.clone(), self.scales.clone(),
                        None if self.row_map is None else self.row_map.clone())

    def c(self) -> _CTensor:
        for t in (self.codebook, self.codes, self.scales, self.row_map):
            if t is not None and (not t.is_cuda or not t.is_contiguous()):
                raise ValueError("VQTensor arrays must be contiguous device tensors")
        return _CTensor(self.rows, self.cols, self.d, self.bits, self.K, self.n_experts,
                        self.n_stored, self.codebook.data_ptr(), self.codes.data_ptr(),
                        self.scales.data_ptr(),
                        None if self.row_map is None else self.row_map.data_ptr())

    def stored_bytes(self) -> int:
        n = self.codes.numel() * 4 + self.scales.numel() * 2
        if self.row_map is not None:
            n += self.row_map.numel() * 4
        return n


def _x_dtype(x: torch.Tensor) -> int:
    if x.dtype == torch.float32:
        return VQ_F32
    if x.dtype == torch.bfloat16:
        return VQ_BF16
    raise TypeError("activations must be float32 or bfloat16")


def vq_validate(W: VQTensor) -> None:
    c = W.c()
    _check(load_library().vq_validate(ctypes.byref(c)))


def vq_dequantize(W: VQTensor, expert: int, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    _require_gpu()
    lib = load_library()
    if out is None:
        out = torch.empty((W.rows, W.cols), dtype=torch.float32, device=W.codes.device)
    c = W.c()
    _check(lib.vq_dequantize(ctypes.byref(c), expert, _ptr(out), _stream()))
    return out


def vq_row_gather(W: VQTensor, ids: torch.Tensor,
                  out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Rows ids[i] = e*rows + r of the stacked tensor, decoded to fp32
    [n, cols]; dead rows +0.0, out-of-range ids NaN rows."""
    _require_gpu()
    lib = load_library()
    if ids.dtype != torch.int64 or not ids.is_cuda:
        raise TypeError("ids must be an int64 device tensor")
    ids = ids.contiguous().view(-1)
    n = ids.numel()
    if out is None:
        out = torch.empty((n, W.cols), dtype=torch.float32, device=ids.device)
    c = W.c()
    _check(lib.vq_row_gather(ctypes.byref(c), n, _ptr(ids), _ptr(out), _stream()))
    return out


def vq_fit(w: torch.Tensor, d: int, bits: int, K: int, sample: torch.Tensor,
           init: torch.Tensor, iters: int, workspace: Optional[torch.Tensor] = None):
    """Fit the format to bf16 weights w [n_rows, cols]: returns (codebook
    int16 [K, d] fp16 bits, scales int16 [n_rows, cols/64] fp16 bits, codes
    int32 [n_rows, wpr]), a dense tensor's arrays (see vq.h, vq_fit)."""
    _require_gpu()
    lib = load_library()
    if w.dtype != torch.bfloat16 or w.dim() != 2 or not w.is_contiguous():
        raise TypeError("w must be a contiguous 2-D bfloat16 device tensor")
    for name, t in (("sample", sample), ("init", init)):
        if t.dtype != torch.int64 or not t.is_cuda or not t.is_contiguous():
            raise TypeError(f"{name} must be a contiguous int64 device tensor")
    n_rows, cols = w.shape
    wpr = ((cols // d + 31) // 32) * bits
    dev = w.device
    codebook = torch.empty((K, d), dtype=torch.int16, device=dev)
    scales = torch.empty((n_rows, cols // 64), dtype=torch.int16, device=dev)
    codes = torch.empty((n_rows, wpr), dtype=torch.int32, device=dev)
    if workspace is None:
        ws = lib.vq_fit_workspace_size(d, K, sample.numel())
        workspace = torch.empty(max(int(ws), 256), dtype=torch.uint8, device=dev)
    _check(lib.vq_fit(n_rows, cols, d, bits, K, _ptr(w), sample.numel(), _ptr(sample),
                      _ptr(init), iters, _ptr(codebook), _ptr(scales), _ptr(codes),
                      _ptr(workspace), workspace.numel(), _stream()))
    return codebook, scales, codes


def vq_expert_gemv(W: VQTensor, expert: int, x: torch.Tensor,
                   out: Optional[torch.Tensor] = None) -> torch.Tensor:
    _require_gpu()
    lib = load_library()
    x = x.contiguous()
    n = x.shape[0]
    if out is None:
        out = torch.empty((n, W.rows), dtype=torch.float32, device=x.device)
    c = W.c()
    _check(lib.vq_expert_gemv(ctypes.byref(c), expert, n, _ptr(x), _x_dtype(x), _ptr(out),
                              _stream()))
    return out


def vq_expert_gemm_workspace_size(W: VQTensor, n_x_rows: int) -> int:
    c = W.c()
    return int(load_library().vq_expert_gemm_workspace_size(ctypes.byref(c), n_x_rows))


def vq_expert_gemm(W: VQTensor, x: torch.Tensor, expert_offsets: torch.Tensor,
                   out: Optional[torch.Tensor] = None,
                   workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    _require_gpu()
    lib = load_library()
    x = x.contiguous()
    n = x.shape[0]
    if out is None:
        out = torch.empty((n, W.rows), dtype=torch.float32, device=x.device)
    ws_bytes = vq_expert_gemm_workspace_size(W, n)
    if workspace is None and ws_bytes:
        workspace = torch.empty(ws_bytes, dtype=torch.uint8, device=x.device)
    c = W.c()
    _check(lib.vq_expert_gemm(ctypes.byref(c), n, _ptr(x), _x_dtype(x),
                              _ptr(expert_offsets.contiguous()), _ptr(out), _ptr(workspace),
                              0 if workspace is None else workspace.numel(), _stream()))
    return out


def vq_moe_ffn_workspace_size(gate: VQTensor, up: VQTensor, down: VQTensor, n_tokens: int,
                              top_k: int) -> int:
    g, u, d = gate.c(), up.c(), down.c()
    return int(load_library().vq_moe_ffn_workspace_size(ctypes.byref(g), ctypes.byref(u),
                                                        ctypes.byref(d), n_tokens, top_k))


VQ_ENGINE_DECODE = 0
VQ_ENGINE_MFMA = 1


def vq_moe_ffn_engine(gate: VQTensor, up: VQTensor, down: VQTensor, n_tokens: int,
                      top_k: int) -> int:
    """VQ_ENGINE_DECODE or VQ_ENGINE_MFMA: the engine vq_moe_ffn runs for
    this batch (host only)."""
    g, u, d = gate.c(), up.c(), down.c()
    eng = ctypes.c_int32(-1)
    _check(load_library().vq_moe_ffn_engine(ctypes.byref(g), ctypes.byref(u), ctypes.byref(d),
                                            n_tokens, top_k, ctypes.byref(eng)))
    return int(eng.value)


def vq_probe_read(buf: torch.Tensor, n_workgroups: int, out: torch.Tensor) -> None:
    """Streaming-read ceiling probe over buf (device, any dtype); out: device
    uint32/int32 of n_workgroups*256 entries."""
    _check(load_library().vq_probe_read(_ptr(buf), buf.numel() * buf.element_size(),
                                        n_workgroups, _ptr(out), _stream()))


def vq_probe_mfma(n_workgroups: int, iters: int, out: torch.Tensor) -> None:
    """MFMA-only ceiling probe: iters x 4 v_mfma_f32_32x32x16_f16 per wave;
    out: device fp32 of n_workgroups*256 entries."""
    _check(load_library().vq_probe_mfma(n_workgroups, iters, _ptr(out), _stream()))


def vq_moe_ffn(gate: VQTensor, up: VQTensor, down: VQTensor, x: torch.Tensor,
               topk_ids: torch.Tensor, topk_weights: torch.Tensor,
               out: Optional[torch.Tensor] = None,
               workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    _require_gpu()
    lib = load_library()
    x = x.contiguous()
    n, k = topk_ids.shape
    if out is None:
        out = torch.empty((n, gate.cols), dtype=torch.float32, device=x.device)
    if workspace is None:
        ws = vq_moe_ffn_workspace_size(gate, up, down, n, k)
        workspace = torch.empty(max(ws, 1), dtype=torch.uint8, device=x.device)
    g, u, d = gate.c(), up.c(), down.c()
    _check(lib.vq_moe_ffn(ctypes.byref(g), ctypes.byref(u), ctypes.byref(d), n, k, _ptr(x),
                          _x_dtype(x), _ptr(topk_ids.contiguous()),
                          _ptr(topk_weights.contiguous()), _ptr(out), _ptr(workspace),
                          workspace.numel(), _stream()))
    return out


def vq_moe_ffn_noalloc(gate: VQTensor, up: VQTensor, down: VQTensor, x: torch.Tensor,
                       topk_ids: torch.Tensor, topk_weights: torch.Tensor,
                       out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """vq_moe_ffn with its workspace in the library's static device array
    (no workspace argument; raises VQError for batches that need more)."""
    _require_gpu()
    lib = load_library()
    x = x.contiguous()
    n, k = topk_ids.shape
    if out is None:
        out = torch.empty((n, gate.cols), dtype=torch.float32, device=x.device)
    g, u, dn = gate.c(), up.c(), down.c()
    _check(lib.vq_moe_ffn_noalloc(ctypes.byref(g), ctypes.byref(u), ctypes.byref(dn), n, k,
                                  _ptr(x), _x_dtype(x), _ptr(topk_ids.contiguous()),
                                  _ptr(topk_weights.contiguous()), _ptr(out), _stream()))
    return out


class _StackArgs:
    """The C layer array and the descriptors it points at, kept alive together."""

    def __init__(self, layers):
        self.tensors = []
        self.arr = (_CLayer * max(len(layers), 1))()
        for i, (g, u, d, ids, w) in enumerate(layers):
            if ids.dtype != torch.int32 or w.dtype != torch.float32:
                raise TypeError("topk_ids must be int32 and topk_weights float32")
            if not (ids.is_contiguous() and w.is_contiguous()):
                raise ValueError("topk_ids and topk_weights must be contiguous")
            cs = (g.c(), u.c(), d.c())
            self.tensors.append(cs)
            self.arr[i] = _CLayer(ctypes.pointer(cs[0]), ctypes.pointer(cs[1]),
                                  ctypes.pointer(cs[2]), ids.data_ptr(), w.data_ptr())


def vq_moe_stack_workspace_size(layers, n_tokens: int, top_k: int) -> int:
    a = _StackArgs(layers)
    return int(load_library().vq_moe_stack_workspace_size(a.arr, len(layers), n_tokens, top_k))


def vq_moe_stack(layers, hidden: torch.Tensor,
                 workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """hidden <- hidden + FFN_l(hidden) for each layer (gate, up, down,
    topk_ids, topk_weights) in order; fp32 [n_tokens, hidden], in place."""
    _require_gpu()
    lib = load_library()
    if hidden.dtype != torch.float32 or not hidden.is_contiguous():
        raise TypeError("hidden must be a contiguous float32 device tensor")
    n = hidden.shape[0]
    k = layers[0][3].shape[1] if layers else 1
    a = _StackArgs(layers)
    if workspace is None:
        ws = lib.vq_moe_stack_workspace_size(a.arr, len(layers), n, k)
        workspace = torch.empty(max(int(ws), 1), dtype=torch.uint8, device=hidden.device)
    _check(lib.vq_moe_stack(a.arr, len(layers), n, k, _ptr(hidden), _ptr(workspace),
                            workspace.numel(), _stream()))
    return hidden


def vq_moe_gate_up(gate: VQTensor, up: VQTensor, x: torch.Tensor, topk_ids: torch.Tensor,
                   out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """h[t*top_k + s] = silu(W_gate_e x_t) * (W_up_e x_t), e = topk_ids[t, s]."""
    _require_gpu()
    lib = load_library()
    x = x.contiguous()
    n, k = topk_ids.shape
    if out is None:
        out = torch.empty((n * k, gate.rows), dtype=torch.float32, device=x.device)
    g, u = gate.c(), up.c()
    _check(lib.vq_moe_gate_up(ctypes.byref(g), ctypes.byref(u), n, k, _ptr(x), _x_dtype(x),
                              _ptr(topk_ids.contiguous()), _ptr(out), _stream()))
    return out


def vq_moe_down(down: VQTensor, h: torch.Tensor, topk_ids: torch.Tensor,
                out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """z[q] = W_down_e h[q] for every (token, slot) pair q."""
    _require_gpu()
    lib = load_library()
    n, k = topk_ids.shape
    if out is None:
        out = torch.empty((n * k, down.rows), dtype=torch.float32, device=h.device)
    dc = down.c()
    _check(lib.vq_moe_down(ctypes.byref(dc), n, k, _ptr(h.contiguous()),
                           _ptr(topk_ids.contiguous()), _ptr(out), _stream()))
    return out


def vq_moe_combine(z: torch.Tensor, topk_weights: torch.Tensor,
                   out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """y[t] = sum over slots s of topk_weights[t, s] * z[t*top_k + s]."""
    _require_gpu()
    lib = load_library()
    n, k = topk_weights.shape
    hidden = z.shape[1]
    if out is None:
        out = torch.empty((n, hidden), dtype=torch.float32, device=z.device)
    _check(lib.vq_moe_combine(n, k, hidden, _ptr(z.contiguous()),
                              _ptr(topk_weights.contiguous()), _ptr(out), _stream()))
    return out


# ---- the operators around the routed experts --------------------------------------------
#
# One token's call runs a few microseconds on the GPU, so these bindings keep
# the host's part short: descriptors are built once, pointers go to ctypes as
# plain integers.  They record no autograd history and refuse tensors that would
# need one (the gradients that there are have calls of their own).

_DTYPE = {torch.float32: VQ_F32, torch.bfloat16: VQ_BF16}
_F32 = torch.float32


def _dtype(name, t: torch.Tensor) -> int:
    code = _DTYPE.get(t.dtype)
    if code is None:
        raise TypeError(f"{name} must be float32 or bfloat16")
    return code


def _on_device(t: torch.Tensor, fn, *args):
    """fn(*args, stream) with t's device current, on that device's current stream."""
    if not t.is_cuda:
        _require_gpu()
        raise TypeError("arguments must be device tensors")
    i = t.device.index
    if i == torch._C._cuda_getDevice():
        st = fn(*args, torch._C._cuda_getCurrentRawStream(i))
    else:
        with torch.cuda.device(i):
            st = fn(*args, torch._C._cuda_getCurrentRawStream(i))
    if st != VQ_OK:
        _check(st)


def _same_device(device, **tensors):
    for name, t in tensors.items():
        if t is not None and t.device != device:
            raise ValueError(f"{name} is on {t.device}, the other arguments on {device}")


def _refuse_history(name, gradient=None):
    """For tensors that require grad: what these calls return has no history, and
    a backward pass would leave them out without a word."""
    if torch.is_grad_enabled():
        raise ValueError(f"{name} records no autograd history: call it under torch.no_grad()" +
                         (f" and take the gradient from {gradient}" if gradient else ""))


def _addr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _check_array(name, t, shape, dtype, device):
    if t is None:
        return
    if t.dtype != dtype or t.shape != shape or not t.is_contiguous() or t.device != device:
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {tuple(shape)} "
                         f"on {device}")


def _out(out, shape, dtype, device):
    """The output tensor: a new one, or the caller's after a check of it."""
    if out is None:
        return torch.empty(shape, dtype=dtype, device=device)
    _check_array("out", out, shape, dtype, device)
    return out


def _workspace(workspace, size, device):
    if workspace is None:
        return torch.empty(max(size, 1), dtype=torch.uint8, device=device)
    _same_device(device, workspace=workspace)
    return workspace


@dataclass(frozen=True)
class VQQ4Tensor:
    """A dense matrix [rows, cols] in 4 bits with a scale (and bias) per
    `group` weights of a row (see vq.h, vq_q4_tensor).

    codes: int32 [rows, cols // 8]; scales: float16 or bfloat16
    [rows, cols // group]; biases: the same, or None for codes centred at 8.
    The descriptor is built once: the tensors may change in place and must not
    be given other storage.
    """

    rows: int
    cols: int
    group: int
    codes: torch.Tensor
    scales: torch.Tensor
    biases: Optional[torch.Tensor] = None

    def __post_init__(self):
        if self.group not in (32, 64, 128) or self.cols % self.group != 0:
            raise ValueError("group must be 32, 64 or 128 and cols a multiple of it")
        if self.codes.dtype != torch.int32 or tuple(self.codes.shape) != (self.rows,
                                                                           self.cols // 8):
            raise ValueError(f"codes must be int32 [{self.rows}, {self.cols // 8}]")
        if self.scales.dtype not in (torch.float16, torch.bfloat16):
            raise TypeError("scales must be float16 or bfloat16")
        for name, t in (("scales", self.scales), ("biases", self.biases)):
            if t is None:
                continue
            if t.dtype != self.scales.dtype or tuple(t.shape) != (self.rows,
                                                                  self.cols // self.group):
                raise ValueError(f"{name} must be {self.scales.dtype} "
                                 f"[{self.rows}, {self.cols // self.group}]")
        for t in (self.codes, self.scales, self.biases):
            if t is not None and not t.is_contiguous():
                raise ValueError("codes, scales and biases must be contiguous")
        _same_device(self.codes.device, scales=self.scales, biases=self.biases)
        object.__setattr__(self, "device", self.codes.device)
        object.__setattr__(self, "_c", self.c())
        object.__setattr__(self, "_ref", ctypes.byref(self._c))

    def c(self) -> _CQ4:
        return _CQ4(self.rows, self.cols, self.group,
                    VQ_F16 if self.scales.dtype == torch.float16 else VQ_BF16,
                    self.codes.data_ptr(), self.scales.data_ptr(), _addr(self.biases))

    def stored_bytes(self) -> int:
        return self.codes.numel() * 4 + self.scales.numel() * (2 if self.biases is None else 4)


def _dense_x(name, x, cols, device):
    if x.requires_grad:
        _refuse_history(name)
    if x.dim() != 2 or x.shape[1] != cols:
        raise ValueError(f"x must be [n_tokens, {cols}], got {tuple(x.shape)}")
    if x.device != device:
        raise ValueError(f"x is on {x.device}, the weights on {device}")
    return x.contiguous()


def vq_q4_gemv(W: VQQ4Tensor, x: torch.Tensor, out: Optional[torch.Tensor] = None,
               accumulate: bool = False) -> torch.Tensor:
    """y[n] = W x[n] for up to 64 tokens, fp32 [n_tokens, rows]; with
    accumulate the product is added to what `out` holds."""
    x = _dense_x("vq_q4_gemv", x, W.cols, W.device)
    if accumulate and out is None:
        raise ValueError("accumulate needs out")
    n = x.shape[0]
    out = _out(out, (n, W.rows), _F32, W.device)
    _on_device(x, load_library().vq_q4_gemv, W._ref, n, x.data_ptr(), _dtype("x", x),
               out.data_ptr(), 1 if accumulate else 0)
    return out


def vq_q4_gate_up(gate: VQQ4Tensor, up: VQQ4Tensor, x: torch.Tensor,
                  out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """h[n] = silu(W_gate x[n]) * (W_up x[n]) for up to 64 tokens, fp32."""
    x = _dense_x("vq_q4_gate_up", x, gate.cols, gate.device)
    if up.device != gate.device:
        raise ValueError(f"up is on {up.device}, gate on {gate.device}")
    n = x.shape[0]
    out = _out(out, (n, gate.rows), _F32, gate.device)
    _on_device(x, load_library().vq_q4_gate_up, gate._ref, up._ref, n, x.data_ptr(),
               _dtype("x", x), out.data_ptr())
    return out


def vq_router_logits(w: torch.Tensor, x: torch.Tensor,
                     out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """logits[n][e] = w[e] . x[n] for a bf16 router w [n_experts, hidden] and
    up to 64 tokens, fp32."""
    if w.dtype != torch.bfloat16 or w.dim() != 2 or not w.is_contiguous():
        raise TypeError("w must be a contiguous bfloat16 tensor [n_experts, hidden]")
    if w.requires_grad:
        _refuse_history("vq_router_logits")
    e, hidden = w.shape
    x = _dense_x("vq_router_logits", x, hidden, w.device)
    n = x.shape[0]
    out = _out(out, (n, e), _F32, w.device)
    _on_device(x, load_library().vq_router_logits, e, hidden, w.data_ptr(), n, x.data_ptr(),
               _dtype("x", x), out.data_ptr())
    return out


@functools.lru_cache(maxsize=256)
def _route_config(n_experts, top_k, score, renormalize, scale):
    cfg = _CRoute(n_experts, top_k, score, 1 if renormalize else 0, scale)
    return cfg, ctypes.byref(cfg)


@functools.lru_cache(maxsize=4096)
def _route_workspace_size(n_experts, n_tokens):
    cfg = _CRoute(n_experts, 1, 0, 0, 1.0)
    return int(load_library().vq_moe_route_workspace_size(ctypes.byref(cfg), n_tokens))


def _check_logits(logits, mask):
    if logits.dim() != 2 or not logits.is_contiguous():
        raise ValueError("logits must be a contiguous tensor [n_tokens, n_experts]")
    if mask is not None and (mask.dtype not in (torch.bool, torch.uint8) or mask.dim() != 1 or
                             mask.shape[0] != logits.shape[0] or not mask.is_contiguous() or
                             mask.device != logits.device):
        raise ValueError(f"mask must be a contiguous bool or uint8 tensor [{logits.shape[0]}] "
                         f"on {logits.device}")


def vq_moe_route(logits: torch.Tensor, top_k: int, *, score: int = VQ_SCORE_SOFTMAX,
                 renormalize: bool = True, scale: float = 1.0,
                 bias: Optional[torch.Tensor] = None, mask: Optional[torch.Tensor] = None,
                 balance: bool = False, workspace: Optional[torch.Tensor] = None):
    """Each token's top_k experts and their weights (see vq.h, vq_moe_route):
    (ids int32, weights fp32), both [n_tokens, top_k]; with balance also
    (counts int32 [n_experts], loss fp32 [1])."""
    if logits.requires_grad:
        _refuse_history("vq_moe_route", "vq_moe_route_grad")
    _check_logits(logits, mask)
    n, e = logits.shape
    dev = logits.device
    _check_array("bias", bias, (e,), _F32, dev)
    _, cfg = _route_config(e, top_k, score, bool(renormalize), float(scale))
    ids = torch.empty((n, max(top_k, 0)), dtype=torch.int32, device=dev)
    weights = torch.empty((n, max(top_k, 0)), dtype=_F32, device=dev)
    lib = load_library()
    if not balance:
        _on_device(logits, lib.vq_moe_route, cfg, n, logits.data_ptr(), _dtype("logits", logits),
                   _addr(bias), _addr(mask), ids.data_ptr(), weights.data_ptr(), None, None,
                   None, 0)
        return ids, weights
    counts = torch.empty((e,), dtype=torch.int32, device=dev)
    loss = torch.empty((1,), dtype=_F32, device=dev)
    ws = _workspace(workspace, _route_workspace_size(e, n), dev)
    _on_device(logits, lib.vq_moe_route, cfg, n, logits.data_ptr(), _dtype("logits", logits),
               _addr(bias), _addr(mask), ids.data_ptr(), weights.data_ptr(), counts.data_ptr(),
               loss.data_ptr(), ws.data_ptr(), ws.numel() * ws.element_size())
    return ids, weights, counts, loss


def vq_moe_route_grad(logits: torch.Tensor, topk_ids: torch.Tensor,
                      d_weights: Optional[torch.Tensor], *, score: int = VQ_SCORE_SOFTMAX,
                      renormalize: bool = True, scale: float = 1.0,
                      mask: Optional[torch.Tensor] = None,
                      counts: Optional[torch.Tensor] = None,
                      d_loss: Optional[torch.Tensor] = None,
                      out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Gradient of sum(d_weights * weights) + d_loss * loss by the logits, in
    their type; the choice and the counts are held fixed."""
    _check_logits(logits, mask)
    n, e = logits.shape
    if topk_ids.dim() != 2:
        raise ValueError("topk_ids must be [n_tokens, top_k]")
    k = topk_ids.shape[1]
    dev = logits.device
    _check_array("topk_ids", topk_ids, (n, k), torch.int32, dev)
    _check_array("d_weights", d_weights, (n, k), _F32, dev)
    _check_array("counts", counts, (e,), torch.int32, dev)
    _check_array("d_loss", d_loss, (1,), _F32, dev)
    out = _out(out, (n, e), logits.dtype, dev)
    _, cfg = _route_config(e, k, score, bool(renormalize), float(scale))
    _on_device(logits, load_library().vq_moe_route_grad, cfg, n, logits.data_ptr(),
               _dtype("logits", logits), _addr(mask), topk_ids.data_ptr(), _addr(d_weights),
               _addr(counts), _addr(d_loss), out.data_ptr())
    return out


_NORM = struct.Struct("6i4q5Pi4f2P")   # vq_block_norm_args (_CNorm, packed in one step)


def _row_stride(name, t, n, hidden, device):
    """Elements between the rows of a [n_tokens, hidden] tensor with unit column stride."""
    if t is None:
        return hidden
    if t.shape != (n, hidden) or t.stride(1) != 1 or t.device != device:
        raise ValueError(f"{name} must be [{n}, {hidden}] with consecutive columns, on {device}")
    return hidden if n <= 1 else t.stride(0)


def _norm_weights(post_weight, pre_weight, gate, n, hidden, device):
    """The three's common type, and the gate's kind."""
    kind, first = VQ_GATE_NONE, None
    for name, w in (("post_weight", post_weight), ("pre_weight", pre_weight), ("gate", gate)):
        if w is None:
            continue
        if first is None:
            first = w.dtype
        if w.dtype != first or not w.is_contiguous() or w.device != device:
            raise ValueError("post_weight, pre_weight and gate must be contiguous, of one type "
                             "and on h's device")
        if name == "gate":
            kind = VQ_GATE_TOKEN if w.shape == (n, 1) else VQ_GATE_CHANNEL
        if w.shape != (hidden,) and kind != VQ_GATE_TOKEN:
            raise ValueError(f"{name} must be [{hidden}]" +
                             (f" or [{n}, 1]" if name == "gate" else ""))
    if first is None:
        return VQ_F32, kind
    if first not in _DTYPE:
        raise TypeError("post_weight, pre_weight and gate must be float32 or bfloat16")
    return _DTYPE[first], kind


def vq_block_norm(h: torch.Tensor, y: Optional[torch.Tensor] = None, *,
                  post_weight: Optional[torch.Tensor] = None,
                  pre_weight: Optional[torch.Tensor] = None,
                  gate: Optional[torch.Tensor] = None, eps: float = 1e-6,
                  weight_offset: float = 0.0, skip_scale: float = 1.0,
                  block_scale: float = 1.0, x_dtype: torch.dtype = torch.bfloat16,
                  h_out: Optional[torch.Tensor] = None, x_out: Optional[torch.Tensor] = None):
    """A block's output y joins the residual stream h, and the next block's
    input is its norm (see vq.h, vq_block_norm): returns (h_out, x).

    h, y: [n_tokens, hidden] fp32 or bf16, rows may be strided; post_weight,
    pre_weight: [hidden]; gate: [hidden] (per channel) or [n_tokens, 1] (per
    token); the three share one type.  h_out may be h."""
    if (h.requires_grad or (y is not None and y.requires_grad) or
            (post_weight is not None and post_weight.requires_grad) or
            (pre_weight is not None and pre_weight.requires_grad) or
            (gate is not None and gate.requires_grad)):
        _refuse_history("vq_block_norm", "vq_block_norm_grad")
    if h.dim() != 2:
        raise ValueError("h must be [n_tokens, hidden]")
    n, hidden = h.shape
    dev = h.device
    w_code, kind = _norm_weights(post_weight, pre_weight, gate, n, hidden, dev)
    h_out_stride = x_stride = hidden
    if h_out is None:
        h_out = torch.empty((n, hidden), dtype=h.dtype, device=dev)
    else:
        if h_out.dtype != h.dtype:
            raise TypeError("h_out must have h's type")
        h_out_stride = _row_stride("h_out", h_out, n, hidden, dev)
    if x_out is None:
        x_out = torch.empty((n, hidden), dtype=x_dtype, device=dev)
    else:
        x_stride = _row_stride("x_out", x_out, n, hidden, dev)
    a = _NORM.pack(n, hidden, _dtype("h", h), VQ_F32 if y is None else _dtype("y", y),
                   _dtype("x", x_out), w_code, _row_stride("h", h, n, hidden, dev),
                   _row_stride("y", y, n, hidden, dev), h_out_stride, x_stride, h.data_ptr(),
                   0 if y is None else y.data_ptr(),
                   0 if post_weight is None else post_weight.data_ptr(),
                   0 if pre_weight is None else pre_weight.data_ptr(),
                   0 if gate is None else gate.data_ptr(), kind, eps,
                   weight_offset, skip_scale, block_scale, h_out.data_ptr(), x_out.data_ptr())
    _on_device(h, load_library().vq_block_norm, a)
    return h_out, x_out


def vq_block_norm_grad(h_out: torch.Tensor, y: Optional[torch.Tensor],
                       d_h_out: Optional[torch.Tensor], d_x: Optional[torch.Tensor], *,
                       post_weight: Optional[torch.Tensor] = None,
                       pre_weight: Optional[torch.Tensor] = None,
                       gate: Optional[torch.Tensor] = None, eps: float = 1e-6,
                       weight_offset: float = 0.0, skip_scale: float = 1.0,
                       block_scale: float = 1.0, workspace: Optional[torch.Tensor] = None):
    """Gradients of vq_block_norm from those of its two outputs (either may be
    None): (d_h, d_y, d_post_weight, d_pre_weight, d_gate), the last three
    fp32; None for what the forward did not have.  h_out is the forward's
    output, y its input."""
    if h_out.dim() != 2:
        raise ValueError("h_out must be [n_tokens, hidden]")
    n, hidden = h_out.shape
    dev = h_out.device
    w_code, kind = _norm_weights(post_weight, pre_weight, gate, n, hidden, dev)
    h_code = _dtype("h_out", h_out)
    h_stride = _row_stride("h_out", h_out, n, hidden, dev)
    if d_h_out is not None:
        if d_h_out.dtype != h_out.dtype:
            raise TypeError("d_h_out must have h_out's type")
        if _row_stride("d_h_out", d_h_out, n, hidden, dev) != h_stride:   # one stride for both
            d_h_out = torch.empty_strided(h_out.shape, h_out.stride(), dtype=h_out.dtype,
                                          device=dev).copy_(d_h_out)
    y_stride = _row_stride("y", y, n, hidden, dev)
    d_h = torch.empty((n, hidden), dtype=h_out.dtype, device=dev)
    d_y = None
    if y is not None:
        d_y = torch.empty((n, hidden), dtype=y.dtype, device=dev) if y_stride == hidden else \
            torch.empty_strided(y.shape, y.stride(), dtype=y.dtype, device=dev)
    d_post = None if post_weight is None else torch.empty(hidden, dtype=_F32, device=dev)
    d_pre = None if pre_weight is None else torch.empty(hidden, dtype=_F32, device=dev)
    d_gate = None if gate is None else torch.empty(gate.shape, dtype=_F32, device=dev)
    a = _NORM.pack(n, hidden, h_code, VQ_F32 if y is None else _dtype("y", y),
                   h_code if d_x is None else _dtype("d_x", d_x), w_code, hidden, y_stride,
                   h_stride, _row_stride("d_x", d_x, n, hidden, dev), 0, _addr(y) or 0,
                   _addr(post_weight) or 0, _addr(pre_weight) or 0, _addr(gate) or 0, kind, eps,
                   weight_offset, skip_scale, block_scale, h_out.data_ptr(), 0)
    lib = load_library()
    ws = _workspace(workspace, int(lib.vq_block_norm_grad_workspace_size(a)), dev)
    _on_device(h_out, lib.vq_block_norm_grad, a, _addr(d_h_out), _addr(d_x), d_h.data_ptr(),
               _addr(d_y), _addr(d_post), _addr(d_pre), _addr(d_gate), ws.data_ptr(),
               ws.numel() * ws.element_size())
    return d_h, d_y, d_post, d_pre, d_gate


@dataclass(frozen=True)
class VQMoEBlock:
    """What one MoE block holds (see vq.h, vq_moe_block): the routed VQ experts
    gate, up, down; router bf16 [n_experts, hidden] with an optional selection
    bias; the norms' weights and the channel gate (one type); optionally a
    shared expert as three VQQ4Tensor.  Its descriptor is built once: the
    tensors may change in place and must not be given other storage."""

    gate: VQTensor
    up: VQTensor
    down: VQTensor
    router: torch.Tensor
    top_k: int
    pre_weight: torch.Tensor
    post_weight: Optional[torch.Tensor] = None
    channel_gate: Optional[torch.Tensor] = None
    route_bias: Optional[torch.Tensor] = None
    shared: Optional[tuple] = None
    score: int = VQ_SCORE_SOFTMAX
    renormalize: bool = True
    route_scale: float = 1.0
    x_dtype: torch.dtype = torch.bfloat16
    eps: float = 1e-6
    weight_offset: float = 0.0
    skip_scale: float = 1.0
    block_scale: float = 1.0

    def __post_init__(self):
        e, hidden = self.gate.n_experts, self.gate.cols
        dev = self.router.device
        _check_array("router", self.router, (e, hidden), torch.bfloat16, dev)
        _check_array("route_bias", self.route_bias, (e,), _F32, dev)
        w_code = _dtype("pre_weight", self.pre_weight)
        for name in ("pre_weight", "post_weight", "channel_gate"):
            _check_array(name, getattr(self, name), (hidden,), self.pre_weight.dtype, dev)
        experts = [t.c() for t in (self.gate, self.up, self.down)]
        for t in (self.gate, self.up, self.down):
            _same_device(dev, **{"a routed expert": t.codes})
        shared = [None] * 3
        if self.shared is not None:
            if len(self.shared) != 3:
                raise ValueError("shared must be the three tensors (gate, up, down)")
            for t in self.shared:
                if t.device != dev:
                    raise ValueError("the shared expert must be on the router's device")
            shared = [ctypes.pointer(t._c) for t in self.shared]
        if self.x_dtype not in _DTYPE:
            raise TypeError("x_dtype must be torch.float32 or torch.bfloat16")
        c = _CBlock(*(ctypes.pointer(t) for t in experts), *shared, self.router.data_ptr(),
                    _addr(self.route_bias),
                    _CRoute(e, self.top_k, self.score, 1 if self.renormalize else 0,
                            self.route_scale),
                    _DTYPE[self.x_dtype], w_code, self.pre_weight.data_ptr(),
                    _addr(self.post_weight), _addr(self.channel_gate), self.eps,
                    self.weight_offset, self.skip_scale, self.block_scale)
        object.__setattr__(self, "device", dev)
        object.__setattr__(self, "_c", c)
        object.__setattr__(self, "_ref", ctypes.byref(c))

    def workspace_size(self, n_tokens: int) -> int:
        size = int(load_library().vq_moe_block_workspace_size(self._ref, n_tokens))
        if size == 0 and n_tokens != 0:
            _check(load_library().vq_moe_block(self._ref, n_tokens, *[None] * 6, 0, None))
        return size


def vq_moe_block(block: VQMoEBlock, h: torch.Tensor, attn: Optional[torch.Tensor] = None, *,
                 attn_weight: Optional[torch.Tensor] = None,
                 next_weight: Optional[torch.Tensor] = None,
                 x_out: Optional[torch.Tensor] = None,
                 workspace: Optional[torch.Tensor] = None):
    """One MoE block on the fp32 residual stream h [n_tokens, hidden], in place
    (up to 64 tokens): attn (fp32) joins it first if given; returns (h, x), x
    the next block's normalised input if next_weight is given, else None."""
    if any(t is not None and t.requires_grad
           for t in (h, attn, attn_weight, next_weight, block.router, block.pre_weight,
                     block.post_weight, block.channel_gate)):
        _refuse_history("vq_moe_block")
    hidden = block.gate.cols
    if h.dim() != 2:
        raise ValueError("h must be [n_tokens, hidden]")
    n = h.shape[0]
    dev = block.device
    _check_array("h", h, (n, hidden), _F32, dev)
    _check_array("attn", attn, (n, hidden), _F32, dev)
    for name, w in (("attn_weight", attn_weight), ("next_weight", next_weight)):
        _check_array(name, w, (hidden,), block.pre_weight.dtype, dev)
    if next_weight is not None:
        x_out = _out(x_out, (n, hidden), block.x_dtype, dev)
    elif x_out is not None:
        raise ValueError("x_out needs next_weight")
    ws = workspace
    if ws is None:
        ws = torch.empty(max(block.workspace_size(n), 1), dtype=torch.uint8, device=dev)
    _same_device(dev, workspace=ws)
    _on_device(h, load_library().vq_moe_block, block._ref, n, h.data_ptr(), _addr(attn),
               _addr(attn_weight), _addr(next_weight), _addr(x_out), ws.data_ptr(),
               ws.numel() * ws.element_size())
    return h, x_out


def vq_set_kernel_events(start, stop) -> None:
    """Record HIP events `start` / `stop` (raw hipEvent_t handles, or None to
    clear) around the dominant kernel of the following calls on this thread."""
    _check(load_library().vq_set_kernel_events(start, stop))


__all__ = [
    "VQError", "VQTensor", "build", "load_library", "vq_validate", "vq_dequantize",
    "vq_row_gather", "vq_fit",
    "vq_expert_gemv", "vq_expert_gemm", "vq_expert_gemm_workspace_size", "vq_moe_ffn",
    "vq_moe_ffn_workspace_size", "vq_moe_ffn_noalloc", "vq_moe_ffn_engine",
    "VQ_ENGINE_DECODE", "VQ_ENGINE_MFMA", "vq_moe_gate_up", "vq_moe_down", "vq_moe_combine",
    "vq_probe_read", "vq_probe_mfma",
    "vq_set_kernel_events", "vq_moe_stack", "vq_moe_stack_workspace_size",
    "VQ_F32", "VQ_BF16", "VQ_F16", "VQQ4Tensor", "vq_q4_gemv", "vq_q4_gate_up",
    "vq_router_logits", "vq_moe_route", "vq_moe_route_grad", "VQ_SCORE_SOFTMAX",
    "VQ_SCORE_SIGMOID", "vq_block_norm", "vq_block_norm_grad", "VQMoEBlock", "vq_moe_block",
]
