"""GB300 (sm_103a) routed MoE SwiGLU expert FFN with rank-r side-LoRA adapters.

Thin Python binding over ``libmoelora.so`` (C ABI, ``include/moe_lora.h``).  The
functions below carry the C names and only marshal arguments: torch CUDA tensors
become device pointers, the current torch stream becomes the ``cudaStream_t``.
Every step of the path runs in the library's CUDA kernels; there is no CPU or
PyTorch fallback, and importing a function fails loudly if the library is
missing (build it with ``moe_expert_ffn_top_gb300._build.build()``).

The method ("feat(mega): add fused shared side-LoRA kernels", DeepGEMM PR #9,
Summary): shared A1/A3/B2 side factors, expert-local B1/B3/A2, frozen W1/W2/W3;
the backward returns grad-x, router-weight gradients and the six adapter
gradients.
"""
from __future__ import annotations

import array
import ctypes
import os
from dataclasses import dataclass
from typing import Dict, Optional, Sequence

import torch

from . import _build

LIB_PATH = _build.LIB

MOE_LORA_WS_PLAN, MOE_LORA_WS_SAVED, MOE_LORA_WS_FWD_SCRATCH, MOE_LORA_WS_BWD_SCRATCH = 0, 1, 2, 3
MOE_LORA_WS_ROUTER_SCRATCH = 4
MOE_LORA_WS_BALANCE_SCRATCH = 5
MOE_LORA_DEV_BAD_ID, MOE_LORA_DEV_TIMEOUT = 1, 2


class MoeLoraError(RuntimeError):
    def __init__(self, code: int, what: str):
        super().__init__(f"{what}: {moe_lora_strerror(code)} (code {code})")
        self.code = code


class Dims(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int64), ("H", ctypes.c_int32), ("I", ctypes.c_int32), ("E", ctypes.c_int32),
                ("k", ctypes.c_int32), ("r", ctypes.c_int32), ("A", ctypes.c_int32), ("block_m", ctypes.c_int32),
                ("scale", ctypes.c_float), ("act", ctypes.c_int32), ("base_fmt", ctypes.c_int32),
                ("act_clamp", ctypes.c_float)]


class Weights(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("W1", "W3", "W2", "A1", "A3", "B1", "B3", "A2", "B2",
                                                 "S1", "S3", "S2")]


class Norm(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("ldx", ctypes.c_int64), ("ldy", ctypes.c_int64), ("lddx", ctypes.c_int64),
                ("lddres", ctypes.c_int64), ("n", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("wdtype", ctypes.c_int32), ("eps", ctypes.c_float)]


class AdamWTensor(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("p", "master", "g", "m", "v", "m_scale", "v_scale")] + [
        ("numel", ctypes.c_int64), ("p_dtype", ctypes.c_int32), ("g_dtype", ctypes.c_int32), ("state", ctypes.c_int32),
        ("lr", ctypes.c_double), ("weight_decay", ctypes.c_double)]


class AdamW(ctypes.Structure):
    _fields_ = [("beta1", ctypes.c_double), ("beta2", ctypes.c_double), ("eps", ctypes.c_double),
                ("step", ctypes.c_int64), ("grad_scale", ctypes.c_void_p)]


class Rows(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("ld", ctypes.c_int64), ("ldd", ctypes.c_int64), ("n", ctypes.c_int32),
                ("dtype", ctypes.c_int32), ("inv_temp", ctypes.c_float)]


class Policy(ctypes.Structure):
    _fields_ = [("clip_low", ctypes.c_float), ("clip_high", ctypes.c_float), ("kl_coef", ctypes.c_float),
                ("adapters", ctypes.c_int32)]


class Preference(ctypes.Structure):
    _fields_ = [("tokens", ctypes.c_int64), ("pairs", ctypes.c_int64), ("beta", ctypes.c_float),
                ("margin", ctypes.c_float), ("label_smoothing", ctypes.c_float), ("kind", ctypes.c_int32),
                ("average", ctypes.c_int32), ("adapters", ctypes.c_int32)]


class MuonTensor(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("p", "master", "g", "m")] + [
        ("batch", ctypes.c_int64), ("rows", ctypes.c_int32), ("cols", ctypes.c_int32), ("p_dtype", ctypes.c_int32),
        ("g_dtype", ctypes.c_int32), ("lr", ctypes.c_double), ("weight_decay", ctypes.c_double), ("scale", ctypes.c_double)]


class Muon(ctypes.Structure):
    _fields_ = [(n, ctypes.c_double) for n in ("momentum", "eps", "a", "b", "c")] + [
        ("nesterov", ctypes.c_int32), ("steps", ctypes.c_int32), ("grad_scale", ctypes.c_void_p)]


class Grads(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("dA1", "dA3", "dB1", "dB3", "dA2", "dB2")]


_lib: Optional[ctypes.CDLL] = None


def lib() -> ctypes.CDLL:
    """The loaded CUDA library (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: run moe_expert_ffn_top_gb300._build.build() first")
        L = ctypes.CDLL(LIB_PATH)
        P = ctypes.c_void_p
        L.moe_lora_workspace_bytes.restype = ctypes.c_size_t
        L.moe_lora_workspace_bytes.argtypes = [ctypes.POINTER(Dims), ctypes.c_int]
        L.moe_lora_plan.restype = ctypes.c_int
        L.moe_lora_plan.argtypes = [ctypes.POINTER(Dims), P, P, P, ctypes.c_size_t, P]
        L.moe_lora_forward.restype = ctypes.c_int
        L.moe_lora_forward.argtypes = [ctypes.POINTER(Dims), P, P, P, ctypes.POINTER(Weights), P, P,
                                       ctypes.c_size_t, P, ctypes.c_size_t, P]
        L.moe_lora_backward.restype = ctypes.c_int
        L.moe_lora_backward.argtypes = [ctypes.POINTER(Dims), P, P, P, P, P, ctypes.POINTER(Weights), P, P,
                                        ctypes.POINTER(Grads), P, ctypes.c_size_t, P]
        L.moe_lora_get_error.restype = ctypes.c_int
        L.moe_lora_get_error.argtypes = [ctypes.POINTER(Dims), P, P]
        L.moe_lora_plan_noalloc.restype = ctypes.c_int
        L.moe_lora_plan_noalloc.argtypes = [ctypes.POINTER(Dims), P, P, P, ctypes.c_size_t, P]
        L.moe_lora_plan_readback.restype = ctypes.c_int
        L.moe_lora_plan_readback.argtypes = [ctypes.POINTER(Dims), P, P, P, P, P, ctypes.c_int64, P]
        L.moe_lora_strerror.restype = ctypes.c_char_p
        L.moe_lora_strerror.argtypes = [ctypes.c_int]
        L.moe_lora_gemm_selftest.restype = ctypes.c_int
        L.moe_lora_gemm_selftest.argtypes = [ctypes.c_int32, ctypes.c_int32, ctypes.c_int32, P, ctypes.c_int32, P,
                                             ctypes.c_int32, P, P]
        L.moe_lora_gemm_pair_selftest.restype = ctypes.c_int
        L.moe_lora_gemm_pair_selftest.argtypes = [ctypes.c_int32, ctypes.c_int32, ctypes.c_int32, P, ctypes.c_int32,
                                                  P, ctypes.c_int32, P, P]
        L.moe_lora_gemm_starved_selftest.restype = ctypes.c_int
        L.moe_lora_gemm_starved_selftest.argtypes = [ctypes.c_int32, ctypes.c_int32, ctypes.c_int32, P,
                                                     ctypes.c_int32, P, ctypes.c_int32, P, ctypes.c_int32, P]
        L.moe_lora_native_selftest.restype = ctypes.c_int
        L.moe_lora_native_selftest.argtypes = [ctypes.c_int32, ctypes.c_int32, ctypes.c_int32, P, P, P, P, P,
                                               ctypes.c_int32, P]
        L.moe_lora_mxfp8_quantize.restype = ctypes.c_int
        L.moe_lora_mxfp8_quantize.argtypes = [P, ctypes.c_int64, ctypes.c_int32, P, P, P]
        L.moe_lora_mxfp4_decode.restype = ctypes.c_int
        L.moe_lora_mxfp4_decode.argtypes = [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int64,
                                             ctypes.c_void_p]
        L.moe_lora_profile_enable.restype = ctypes.c_int
        L.moe_lora_profile_enable.argtypes = [ctypes.c_int]
        L.moe_lora_profile_select.restype = ctypes.c_int
        L.moe_lora_profile_select.argtypes = [ctypes.c_char_p]
        L.moe_lora_profile_read.restype = ctypes.c_int
        L.moe_lora_profile_read.argtypes = [P, P, P, ctypes.c_int]
        L.moe_lora_launch_count.restype = ctypes.c_int64
        L.moe_lora_launch_count.argtypes = [ctypes.c_int]
        L.moe_lora_gemm_selftest_error.restype = ctypes.c_int
        L.moe_lora_gemm_selftest_error.argtypes = [P]
        L.moe_lora_router_forward.restype = ctypes.c_int
        L.moe_lora_router_forward.argtypes = [ctypes.POINTER(Dims), P, P, P, P, P, P, P, ctypes.c_size_t, P]
        L.moe_lora_router_backward.restype = ctypes.c_int
        L.moe_lora_router_backward.argtypes = [ctypes.POINTER(Dims), P, P, P, P, P, P, P, P, P, P, ctypes.c_size_t,
                                               P]
        L.moe_lora_router_get_error.restype = ctypes.c_int
        L.moe_lora_router_get_error.argtypes = [P, P]
        L.moe_lora_layernorm_forward.restype = ctypes.c_int
        L.moe_lora_layernorm_forward.argtypes = [ctypes.POINTER(Norm), P, P, P, P, P, P, P]
        L.moe_lora_layernorm_scratch_bytes.restype = ctypes.c_size_t
        L.moe_lora_layernorm_scratch_bytes.argtypes = [ctypes.POINTER(Norm)]
        L.moe_lora_layernorm_backward.restype = ctypes.c_int
        L.moe_lora_layernorm_backward.argtypes = [ctypes.POINTER(Norm), P, P, P, P, P, P, P, P, P, P, ctypes.c_size_t,
                                                  P]
        L.moe_lora_balance_loss.restype = ctypes.c_int
        L.moe_lora_balance_loss.argtypes = [ctypes.POINTER(Dims), P, ctypes.c_int32, ctypes.c_int64, P, P,
                                            ctypes.c_float, P, P, P, P, P, P, ctypes.c_size_t, P]
        L.moe_lora_balance_get_error.restype = ctypes.c_int
        L.moe_lora_balance_get_error.argtypes = [ctypes.POINTER(Dims), P, P]
        L.moe_lora_router_backward_aux.restype = ctypes.c_int
        L.moe_lora_router_backward_aux.argtypes = [ctypes.POINTER(Dims), P, P, P, P, P, P, P, P, P, P, P,
                                                   ctypes.c_size_t, P]
        L.moe_lora_adamw_step.restype = ctypes.c_int
        L.moe_lora_adamw_step.argtypes = [ctypes.POINTER(AdamW), P, ctypes.c_int32, P]
        L.moe_lora_token_logp_forward.restype = ctypes.c_int
        L.moe_lora_token_logp_forward.argtypes = [ctypes.POINTER(Rows), P, P, P, P, P, P, P]
        L.moe_lora_token_logp_backward.restype = ctypes.c_int
        L.moe_lora_token_logp_backward.argtypes = [ctypes.POINTER(Rows), P, P, P, P, P, P, P]
        L.moe_lora_policy_scratch_bytes.restype = ctypes.c_size_t
        L.moe_lora_policy_scratch_bytes.argtypes = [ctypes.c_int64, ctypes.c_int32]
        L.moe_lora_policy_loss.restype = ctypes.c_int
        L.moe_lora_policy_loss.argtypes = [ctypes.POINTER(Rows), ctypes.POINTER(Policy)] + [P] * 14 + [ctypes.c_size_t, P]
        L.moe_lora_preference_scratch_bytes.restype = ctypes.c_size_t
        L.moe_lora_preference_scratch_bytes.argtypes = [ctypes.c_int64]
        L.moe_lora_preference_loss.restype = ctypes.c_int
        L.moe_lora_preference_loss.argtypes = [ctypes.POINTER(Preference)] + [P] * 12 + [ctypes.c_size_t, P]
        L.moe_lora_muon_scratch_bytes.restype = ctypes.c_size_t
        L.moe_lora_muon_scratch_bytes.argtypes = [P, ctypes.c_int32]
        L.moe_lora_muon_step.restype = ctypes.c_int
        L.moe_lora_muon_step.argtypes = [ctypes.POINTER(Muon), P, ctypes.c_int32, P, ctypes.c_size_t, P]
        L.moe_lora_muon_get_error.restype = ctypes.c_int
        L.moe_lora_muon_get_error.argtypes = [P, P]
        _lib = L
    return _lib


def make_dims(T: int, H: int, I: int, E: int, k: int, r: int, A: int = 1, scale: float = 1.0,
              base_fmt: int = 0, act: int = 0, act_clamp: float = 0.0) -> Dims:
    """base_fmt: 0 = bf16 base weights; MXFP4 (packed E2M1 codes + UE8M0 scales S1/S3/S2) decoded
    inside the GEMMs (1) or once per pass into the saved workspace (2); 3 / 4 = the native FP4
    forward (gate/up base products on block-scaled FP4 tensor cores from MXFP8 activations,
    the rest as 1 / as 2; H and I multiples of 128);
    act: 0 = SwiGLU, 1 = GeGLU; act_clamp: clamp of the gate/up pre-activations (0 = none)."""
    return Dims(T, H, I, E, k, r, A, 128, float(scale), int(act), int(base_fmt), float(act_clamp))


def _ptr(t: Optional[torch.Tensor], dtype=None, name: str = "") -> Optional[int]:
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    return t.data_ptr()


def _stream(stream) -> int:
    if stream is None:  # the current stream's handle, without the 3 us of building a Stream object
        return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _check(rc: int, what: str) -> None:
    if rc != 0:
        raise MoeLoraError(rc, what)


def moe_lora_strerror(code: int) -> str:
    return lib().moe_lora_strerror(code).decode()


def moe_lora_workspace_bytes(dims: Dims, which: int) -> int:
    return int(lib().moe_lora_workspace_bytes(ctypes.byref(dims), which))


def moe_lora_plan(dims: Dims, topk_ids: torch.Tensor, adapter_offsets: Optional[Sequence[int]],
                  plan_ws: torch.Tensor, stream=None) -> None:
    offs = None
    if adapter_offsets is not None:
        vals = [int(v) for v in adapter_offsets]
        offs = (ctypes.c_int64 * len(vals))(*vals)
    rc = lib().moe_lora_plan(ctypes.byref(dims), _ptr(topk_ids, torch.int32, "topk_ids"),
                             ctypes.cast(offs, ctypes.c_void_p) if offs is not None else None,
                             _ptr(plan_ws, None, "plan_ws"), plan_ws.numel() * plan_ws.element_size(),
                             _stream(stream))
    _check(rc, "moe_lora_plan")


def moe_lora_plan_noalloc(dims: Dims, topk_ids: torch.Tensor, adapter_offsets: Optional[Sequence[int]],
                          plan_ws: torch.Tensor, plan_bytes: Optional[int] = None, stream=None) -> None:
    """The routing plan without caller-provided temporary space (see the C header):
    plan_ws only needs to hold the plan itself."""
    offs = None
    if adapter_offsets is not None:
        vals = [int(v) for v in adapter_offsets]
        offs = (ctypes.c_int64 * len(vals))(*vals)
    nbytes = plan_ws.numel() * plan_ws.element_size() if plan_bytes is None else plan_bytes
    rc = lib().moe_lora_plan_noalloc(ctypes.byref(dims), _ptr(topk_ids, torch.int32, "topk_ids"),
                                     ctypes.cast(offs, ctypes.c_void_p) if offs is not None else None,
                                     _ptr(plan_ws, None, "plan_ws"), nbytes, _stream(stream))
    _check(rc, "moe_lora_plan_noalloc")


def moe_lora_plan_readback(dims: Dims, plan_ws: torch.Tensor, stream=None) -> Dict[str, torch.Tensor]:
    """Host copies of the plan: counts, offsets, row_of_route, route_of_row."""
    G = dims.A * dims.E
    counts = torch.zeros(G, dtype=torch.int32)
    offsets = torch.zeros(G + 1, dtype=torch.int32)
    ror = torch.zeros(max(dims.T * dims.k, 1), dtype=torch.int32)
    cap = dims.T * dims.k + G * 128
    rrow = torch.zeros(max(cap, 1), dtype=torch.int32)
    rc = lib().moe_lora_plan_readback(ctypes.byref(dims), _ptr(plan_ws), counts.data_ptr(), offsets.data_ptr(),
                                      ror.data_ptr(), rrow.data_ptr(), cap, _stream(stream))
    _check(rc, "moe_lora_plan_readback")
    P = int(offsets[-1])
    return {"counts": counts, "offsets": offsets, "row_of_route": ror[:dims.T * dims.k],
            "route_of_row": rrow[:P].clone()}


def _weights(w: Dict[str, torch.Tensor], dims: Dims) -> Weights:
    mx = dims.base_fmt in (1, 2, 3, 4)
    base = [_ptr(w[n], torch.uint8 if mx else torch.bfloat16, n) for n in ("W1", "W3", "W2")]
    side = [_ptr(w[n], torch.bfloat16, n) for n in ("A1", "A3", "B1", "B3", "A2", "B2")]
    scales = [_ptr(w[n], torch.uint8, n) if mx else None for n in ("S1", "S3", "S2")]
    return Weights(*(base + side + scales))


def moe_lora_forward(dims: Dims, plan_ws: torch.Tensor, x: torch.Tensor, topk_w: torch.Tensor,
                     weights: Dict[str, torch.Tensor], y: torch.Tensor, saved: torch.Tensor,
                     scratch: torch.Tensor, stream=None) -> None:
    W = _weights(weights, dims)
    rc = lib().moe_lora_forward(ctypes.byref(dims), _ptr(plan_ws), _ptr(x, torch.bfloat16, "x"),
                                _ptr(topk_w, torch.float32, "topk_w"), ctypes.byref(W),
                                _ptr(y, torch.bfloat16, "y"), _ptr(saved), saved.numel() * saved.element_size(),
                                _ptr(scratch), scratch.numel() * scratch.element_size(), _stream(stream))
    _check(rc, "moe_lora_forward")


def moe_lora_backward(dims: Dims, plan_ws: torch.Tensor, saved: torch.Tensor, x: torch.Tensor,
                      topk_w: torch.Tensor, dy: torch.Tensor, weights: Dict[str, torch.Tensor],
                      dx: torch.Tensor, dw: torch.Tensor, grads: Dict[str, torch.Tensor],
                      scratch: torch.Tensor, stream=None) -> None:
    W = _weights(weights, dims)
    Gr = Grads(*[_ptr(grads[n], torch.float32, n) for n in ("dA1", "dA3", "dB1", "dB3", "dA2", "dB2")])
    rc = lib().moe_lora_backward(ctypes.byref(dims), _ptr(plan_ws), _ptr(saved), _ptr(x, torch.bfloat16, "x"),
                                 _ptr(topk_w, torch.float32, "topk_w"), _ptr(dy, torch.bfloat16, "dy"),
                                 ctypes.byref(W), _ptr(dx, torch.bfloat16, "dx"), _ptr(dw, torch.float32, "dw"),
                                 ctypes.byref(Gr), _ptr(scratch), scratch.numel() * scratch.element_size(),
                                 _stream(stream))
    _check(rc, "moe_lora_backward")


def moe_lora_get_error(dims: Dims, plan_ws: torch.Tensor, stream=None) -> int:
    rc = lib().moe_lora_get_error(ctypes.byref(dims), _ptr(plan_ws), _stream(stream))
    if rc < 0:
        raise MoeLoraError(rc, "moe_lora_get_error")
    return rc


def _offsets(adapter_offsets: Optional[Sequence[int]]):
    if adapter_offsets is None:
        return None
    vals = [int(v) for v in adapter_offsets]
    return (ctypes.c_int64 * len(vals))(*vals)


def moe_lora_router_forward(dims: Dims, x: torch.Tensor, Wr: torch.Tensor, topk_ids: torch.Tensor,
                            topk_w: torch.Tensor, logits: Optional[torch.Tensor], scratch: torch.Tensor,
                            stream=None, adapter_offsets: Optional[Sequence[int]] = None) -> None:
    """Softmax top-k router: topk_ids [T,k] int32, topk_w [T,k] fp32 (and logits [T,E] fp32 if given).
    W_r is [E,H] or [A,E,H]; adapter_offsets [A+1] (host) splits the tokens between adapters."""
    offs = _offsets(adapter_offsets)
    rc = lib().moe_lora_router_forward(ctypes.byref(dims), _ptr(x, torch.bfloat16, "x"),
                                       _ptr(Wr, torch.bfloat16, "Wr"),
                                       ctypes.cast(offs, ctypes.c_void_p) if offs is not None else None,
                                       _ptr(topk_ids, torch.int32, "topk_ids"),
                                       _ptr(topk_w, torch.float32, "topk_w"), _ptr(logits, torch.float32, "logits"),
                                       _ptr(scratch), scratch.numel() * scratch.element_size(), _stream(stream))
    _check(rc, "moe_lora_router_forward")


def moe_lora_router_backward(dims: Dims, x: torch.Tensor, Wr: torch.Tensor, topk_ids: torch.Tensor,
                             topk_w: torch.Tensor, dw: torch.Tensor, dlogits: Optional[torch.Tensor],
                             dWr: torch.Tensor, dx: torch.Tensor, scratch: torch.Tensor, stream=None,
                             adapter_offsets: Optional[Sequence[int]] = None) -> None:
    """Router backward: dWr [E,H] or [A,E,H] fp32 (and dlogits [T,E] fp32 if given); dx [T,H]
    bf16 is updated in place, dx <- bf16(dx + dlogits W_r)."""
    offs = _offsets(adapter_offsets)
    rc = lib().moe_lora_router_backward(ctypes.byref(dims), _ptr(x, torch.bfloat16, "x"),
                                        _ptr(Wr, torch.bfloat16, "Wr"),
                                        ctypes.cast(offs, ctypes.c_void_p) if offs is not None else None,
                                        _ptr(topk_ids, torch.int32, "topk_ids"),
                                        _ptr(topk_w, torch.float32, "topk_w"), _ptr(dw, torch.float32, "dw"),
                                        _ptr(dlogits, torch.float32, "dlogits"), _ptr(dWr, torch.float32, "dWr"),
                                        _ptr(dx, torch.bfloat16, "dx"), _ptr(scratch),
                                        scratch.numel() * scratch.element_size(), _stream(stream))
    _check(rc, "moe_lora_router_backward")


def moe_lora_router_get_error(scratch: torch.Tensor, stream=None) -> int:
    rc = lib().moe_lora_router_get_error(_ptr(scratch), _stream(stream))
    if rc < 0:
        raise MoeLoraError(rc, "moe_lora_router_get_error")
    return rc


def router_scratch(dims: Dims, device="cuda") -> torch.Tensor:
    n = moe_lora_workspace_bytes(dims, MOE_LORA_WS_ROUTER_SCRATCH)
    if n == 0:
        raise MoeLoraError(-5, "moe_lora_workspace_bytes(ROUTER_SCRATCH)")
    return torch.empty(n, dtype=torch.uint8, device=device)


def moe_lora_gemm_selftest(A: torch.Tensor, a_mn: bool, B: torch.Tensor, b_mn: bool, C: torch.Tensor,
                           stream=None) -> None:
    """C[M,N] = A(m,k) B(n,k) on the GEMM engine; A is [M,K] or, if a_mn, [K,M]; B is [N,K] or [K,N]."""
    M, N = C.shape
    K = A.shape[0] if a_mn else A.shape[1]
    rc = lib().moe_lora_gemm_selftest(M, N, K, _ptr(A, torch.bfloat16, "A"), int(a_mn),
                                      _ptr(B, torch.bfloat16, "B"), int(b_mn), _ptr(C, torch.float32, "C"),
                                      _stream(stream))
    _check(rc, "moe_lora_gemm_selftest")


def moe_lora_gemm_pair_selftest(A: torch.Tensor, a_mn: bool, B: torch.Tensor, b_mn: bool, C: torch.Tensor,
                                stream=None) -> None:
    """As moe_lora_gemm_selftest, on the two-SM (cta_group::2) engine."""
    M, N = C.shape
    K = A.shape[0] if a_mn else A.shape[1]
    rc = lib().moe_lora_gemm_pair_selftest(M, N, K, _ptr(A, torch.bfloat16, "A"), int(a_mn),
                                           _ptr(B, torch.bfloat16, "B"), int(b_mn), _ptr(C, torch.float32, "C"),
                                           _stream(stream))
    _check(rc, "moe_lora_gemm_pair_selftest")


def moe_lora_gemm_starved_selftest(A: torch.Tensor, a_mn: bool, B: torch.Tensor, b_mn: bool, C: torch.Tensor,
                                   pair: bool, stream=None) -> None:
    """The self-test GEMM with every operand copy withheld: its bounded waits must expire
    and set MOE_LORA_DEV_TIMEOUT (read with moe_lora_gemm_selftest_error)."""
    M, N = C.shape
    K = A.shape[0] if a_mn else A.shape[1]
    rc = lib().moe_lora_gemm_starved_selftest(M, N, K, _ptr(A, torch.bfloat16, "A"), int(a_mn),
                                              _ptr(B, torch.bfloat16, "B"), int(b_mn), _ptr(C, torch.float32, "C"),
                                              int(pair), _stream(stream))
    _check(rc, "moe_lora_gemm_starved_selftest")


def moe_lora_native_selftest(Aq: torch.Tensor, As: torch.Tensor, Bq: torch.Tensor, Bs: torch.Tensor,
                             C: torch.Tensor, layout: int = 0, stream=None) -> None:
    """Block-scaled FP4 self-test GEMM: C [M,N] fp32 from E4M3 codes Aq [M,K], packed
    E2M1 codes Bq [N,K/2] and UE8M0 scale bytes As, Bs in the tile-major layout
    [rows/128][K/128][128][4] (all uint8)."""
    M, K = Aq.shape
    N = Bq.shape[0]
    rc = lib().moe_lora_native_selftest(M, N, K, _ptr(Aq, torch.uint8, "Aq"), _ptr(As, torch.uint8, "As"),
                                        _ptr(Bq, torch.uint8, "Bq"), _ptr(Bs, torch.uint8, "Bs"),
                                        _ptr(C, torch.float32, "C"), int(layout), _stream(stream))
    _check(rc, "moe_lora_native_selftest")


def moe_lora_mxfp8_quantize(x: torch.Tensor, codes: torch.Tensor, scales: torch.Tensor, stream=None) -> None:
    """MXFP8 (E4M3 codes, one UE8M0 scale byte per 32 along a row) of a bf16 matrix
    x [rows, n] into codes [rows, n] and scales [rows, n/32] (uint8, device)."""
    rows, n = x.shape
    rc = lib().moe_lora_mxfp8_quantize(_ptr(x, torch.bfloat16, "x"), rows, n, _ptr(codes, torch.uint8, "codes"),
                                       _ptr(scales, torch.uint8, "scales"), _stream(stream))
    _check(rc, "moe_lora_mxfp8_quantize")


def moe_lora_gemm_selftest_error(stream=None) -> int:
    return lib().moe_lora_gemm_selftest_error(_stream(stream))


def moe_lora_mxfp4_decode(packed: torch.Tensor, scales: torch.Tensor, out: torch.Tensor, stream=None) -> None:
    """MXFP4 (packed E2M1 pairs + one UE8M0 per 32) -> bf16 `out`, exactly, on the device."""
    elems = out.numel()
    if packed.numel() * 2 != elems or scales.numel() * 32 != elems:
        raise ValueError("packed must hold elems/2 bytes and scales elems/32 bytes")
    _check(lib().moe_lora_mxfp4_decode(_ptr(packed, torch.uint8, "packed"), _ptr(scales, torch.uint8, "scales"),
                                       _ptr(out, torch.bfloat16, "out"), elems, _stream(stream)),
           "moe_lora_mxfp4_decode")


def moe_lora_profile_enable(on: bool) -> None:
    lib().moe_lora_profile_enable(1 if on else 0)


def moe_lora_profile_select(kernel: Optional[str]) -> None:
    """Time only `kernel`'s launches (None: every kernel)."""
    rc = lib().moe_lora_profile_select(kernel.encode() if kernel is not None else None)
    _check(rc, "moe_lora_profile_select")


def moe_lora_profile_read() -> Dict[str, tuple]:
    """{kernel name: (total ms, launches)} since the last read (then reset)."""
    cap = 64
    names = (ctypes.c_char_p * cap)()
    ms = (ctypes.c_double * cap)()
    cnt = (ctypes.c_int64 * cap)()
    n = lib().moe_lora_profile_read(ctypes.cast(names, ctypes.c_void_p), ctypes.cast(ms, ctypes.c_void_p),
                                    ctypes.cast(cnt, ctypes.c_void_p), cap)
    if n < 0:
        raise MoeLoraError(n, "moe_lora_profile_read")
    return {names[i].decode(): (ms[i], int(cnt[i])) for i in range(n)}


def moe_lora_launch_count(reset: bool = False) -> int:
    return int(lib().moe_lora_launch_count(1 if reset else 0))


# ------------------------------------------------------------------ training step
DTYPES = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}


def _dtype(t: torch.Tensor, name: str) -> int:
    code = DTYPES.get(t.dtype)
    if code is None:
        raise ValueError(f"{name} must be float32, bfloat16 or float16, got {t.dtype}")
    return code


def _rows(t: torch.Tensor, name: str, like: Optional[torch.Tensor] = None):
    """Pointer and row stride (0 = dense) of a [rows, n] tensor whose rows are contiguous."""
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if like is None:
        if t.dim() != 2 or t.size(1) < 1:
            raise ValueError(f"{name} must be [rows, n] with n >= 1")
    elif t.shape != like.shape or t.dtype is not like.dtype:
        raise ValueError(f"{name} must be {tuple(like.shape)} {like.dtype}, got {tuple(t.shape)} {t.dtype}")
    if t.is_contiguous():
        return t.data_ptr(), 0
    rows, n = t.shape
    ld, step = t.stride()
    if (n > 1 and step != 1) or (rows > 1 and ld < n):
        raise ValueError(f"{name} must have contiguous rows that do not overlap")
    return t.data_ptr(), ld if rows > 1 else 0


def _vec(t: Optional[torch.Tensor], n: int, name: str, dtype=None) -> Optional[int]:
    """Pointer of a contiguous CUDA tensor of n elements (None passes through)."""
    if t is None:
        return None
    if t.numel() != n:
        raise ValueError(f"{name} must have {n} elements, got {t.numel()}")
    if dtype is not None and t.dtype is not dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def moe_lora_layernorm_forward(x: torch.Tensor, gamma: Optional[torch.Tensor], beta: Optional[torch.Tensor],
                               y: torch.Tensor, mean: Optional[torch.Tensor] = None,
                               rstd: Optional[torch.Tensor] = None, eps: float = 1e-5, stream=None) -> None:
    """Layer norm of the rows of x [rows, n] (fp32, bf16 or fp16; rows may be strided) into y;
    gamma / beta [n] of one type or None; mean, rstd [rows] fp32 kept for the backward if given."""
    px, ldx = _rows(x, "x")
    py, ldy = _rows(y, "y", x)
    rows, n = x.shape
    w = gamma if gamma is not None else beta
    if beta is not None and beta.dtype != w.dtype:
        raise ValueError("gamma and beta must have one type")
    nm = Norm(rows, ldx, ldy, 0, 0, n, _dtype(x, "x"), 0 if w is None else _dtype(w, "gamma"), eps)
    rc = lib().moe_lora_layernorm_forward(nm, px, _vec(gamma, n, "gamma"), _vec(beta, n, "beta"), py,
                                          _vec(mean, rows, "mean", torch.float32),
                                          _vec(rstd, rows, "rstd", torch.float32), _stream(stream))
    _check(rc, "moe_lora_layernorm_forward")


def layernorm_scratch(rows: int, n: int, device="cuda") -> torch.Tensor:
    """Workspace of moe_lora_layernorm_backward's weight gradients."""
    b = int(lib().moe_lora_layernorm_scratch_bytes(Norm(rows, 0, 0, 0, 0, n, 0, 0, 1.0)))
    if b == 0:
        raise MoeLoraError(-2, "moe_lora_layernorm_scratch_bytes")
    return torch.empty(b, dtype=torch.uint8, device=device)


def moe_lora_layernorm_backward(x: torch.Tensor, gamma: Optional[torch.Tensor], mean: torch.Tensor,
                                rstd: torch.Tensor, dy: torch.Tensor, dres: Optional[torch.Tensor], dx: torch.Tensor,
                                dgamma: Optional[torch.Tensor] = None, dbeta: Optional[torch.Tensor] = None,
                                scratch: Optional[torch.Tensor] = None, stream=None) -> None:
    """dx of the layer norm (plus dres, a gradient that reaches x on another path, if given) and,
    where given, its weights' gradients dgamma, dbeta [n] fp32 (these need `scratch`)."""
    px, ldx = _rows(x, "x")
    pdy, ldy = _rows(dy, "dy", x)
    pdx, lddx = _rows(dx, "dx", x)
    pdr, lddr = (None, 0) if dres is None else _rows(dres, "dres", x)
    rows, n = x.shape
    nm = Norm(rows, ldx, ldy, lddx, lddr, n, _dtype(x, "x"), 0 if gamma is None else _dtype(gamma, "gamma"), 1.0)
    rc = lib().moe_lora_layernorm_backward(nm, px, _vec(gamma, n, "gamma"), _vec(mean, rows, "mean", torch.float32),
                                           _vec(rstd, rows, "rstd", torch.float32), pdy, pdr, pdx,
                                           _vec(dgamma, n, "dgamma", torch.float32),
                                           _vec(dbeta, n, "dbeta", torch.float32), _ptr(scratch, None, "scratch"),
                                           0 if scratch is None else scratch.numel() * scratch.element_size(),
                                           _stream(stream))
    _check(rc, "moe_lora_layernorm_backward")


def balance_scratch(dims: Dims, device="cuda") -> torch.Tensor:
    n = moe_lora_workspace_bytes(dims, MOE_LORA_WS_BALANCE_SCRATCH)
    if n == 0:
        raise MoeLoraError(-5, "moe_lora_workspace_bytes(BALANCE_SCRATCH)")
    return torch.empty(n, dtype=torch.uint8, device=device)


def moe_lora_balance_loss(dims: Dims, logits: torch.Tensor, topk_ids: torch.Tensor,
                          adapter_offsets: Optional[Sequence[int]], coef: float, loss: torch.Tensor,
                          counts: torch.Tensor, prob: torch.Tensor, scratch: torch.Tensor,
                          dlogits: Optional[torch.Tensor] = None, dloss: Optional[torch.Tensor] = None,
                          stream=None) -> None:
    """Balance loss [A] of the routes topk_ids [T,k] int32 (-1 = masked) under the router's logits
    [T,E], with counts [A,E] int32 and mean probabilities prob [A,E]; dlogits [T,E] fp32 receives
    its gradient (for the upstream gradient dloss [A], None = 1) in the same pass if given.
    moe_lora_balance_get_error(dims, scratch) reads the device error bits."""
    pl, ld = _rows(logits, "logits")
    T, E, A = dims.T, dims.E, dims.A
    if logits.size(0) != T or logits.size(1) != E:
        raise ValueError(f"logits must be [{T}, {E}], got {tuple(logits.shape)}")
    offs = None if adapter_offsets is None else array.array("q", adapter_offsets)
    if offs is not None and len(offs) != A + 1:
        raise ValueError(f"adapter_offsets must have {A + 1} entries")
    rc = lib().moe_lora_balance_loss(dims, pl, _dtype(logits, "logits"), ld,
                                     _vec(topk_ids, T * dims.k, "topk_ids", torch.int32),
                                     None if offs is None else offs.buffer_info()[0], coef,
                                     _vec(dloss, A, "dloss", torch.float32),
                                     _vec(loss, A, "loss", torch.float32), _vec(counts, A * E, "counts", torch.int32),
                                     _vec(prob, A * E, "prob", torch.float32),
                                     _vec(dlogits, T * E, "dlogits", torch.float32),
                                     _ptr(scratch, None, "scratch"), scratch.numel() * scratch.element_size(),
                                     _stream(stream))
    _check(rc, "moe_lora_balance_loss")


def moe_lora_balance_get_error(dims: Dims, scratch: torch.Tensor, stream=None) -> int:
    rc = lib().moe_lora_balance_get_error(dims, _ptr(scratch), _stream(stream))
    if rc < 0:
        raise MoeLoraError(rc, "moe_lora_balance_get_error")
    return rc


def moe_lora_router_backward_aux(dims: Dims, x: torch.Tensor, Wr: torch.Tensor, topk_ids: torch.Tensor,
                                 topk_w: torch.Tensor, dw: torch.Tensor, dlogits_aux: Optional[torch.Tensor],
                                 dlogits: Optional[torch.Tensor], dWr: torch.Tensor, dx: torch.Tensor,
                                 scratch: torch.Tensor, stream=None,
                                 adapter_offsets: Optional[Sequence[int]] = None) -> None:
    """moe_lora_router_backward with dlogits_aux [T,E] fp32 (e.g. moe_lora_balance_loss's dlogits)
    added to the routes' logit gradient."""
    rc = lib().moe_lora_router_backward_aux(dims, _ptr(x, torch.bfloat16, "x"), _ptr(Wr, torch.bfloat16, "Wr"),
                                            _offsets(adapter_offsets), _ptr(topk_ids, torch.int32, "topk_ids"),
                                            _ptr(topk_w, torch.float32, "topk_w"), _ptr(dw, torch.float32, "dw"),
                                            _vec(dlogits_aux, dims.T * dims.E, "dlogits_aux", torch.float32),
                                            _ptr(dlogits, torch.float32, "dlogits"), _ptr(dWr, torch.float32, "dWr"),
                                            _ptr(dx, torch.bfloat16, "dx"), _ptr(scratch),
                                            scratch.numel() * scratch.element_size(), _stream(stream))
    _check(rc, "moe_lora_router_backward_aux")


_CODES = (torch.uint8, torch.float8_e4m3fn)  # 8-bit moments


class AdamWTensors:
    """The tensors of an AdamW step, listed once and kept between steps.  Each entry is a dict:
    p (fp32, bf16 or fp16), g, m, v, and optionally master (fp32, for a 16-bit p), m_scale and
    v_scale (fp32, one per 256 elements, started at zero; with them m and v are 8-bit codes,
    uint8 or float8_e4m3fn, v holding sqrt(v)), lr (1e-3) and weight_decay (0).  All contiguous;
    no two overlap.  The entries hold the tensors alive."""

    def __init__(self, entries: Sequence[Dict]):
        self.entries = [dict(e) for e in entries]
        self.table = (AdamWTensor * max(1, len(self.entries)))()
        for d, e in zip(self.table, self.entries):
            p, n = e["p"], e["p"].numel()
            eight = e.get("m_scale") is not None
            if eight != (e.get("v_scale") is not None):
                raise ValueError("m_scale and v_scale come together")
            blocks = (n + 255) // 256
            for name in ("m", "v"):
                if eight and e[name].dtype not in _CODES:
                    raise ValueError(f"{name} must be uint8 or float8_e4m3fn codes, got {e[name].dtype}")
            state = None if eight else torch.float32
            d.p, d.g = _vec(p, n, "p"), _vec(e["g"], n, "g")
            d.master = _vec(e.get("master"), n, "master", torch.float32)
            d.m, d.v = _vec(e["m"], n, "m", state), _vec(e["v"], n, "v", state)
            d.m_scale = _vec(e.get("m_scale"), blocks, "m_scale", torch.float32)
            d.v_scale = _vec(e.get("v_scale"), blocks, "v_scale", torch.float32)
            d.numel, d.p_dtype, d.g_dtype, d.state = n, _dtype(p, "p"), _dtype(e["g"], "g"), int(eight)
            d.lr, d.weight_decay = e.get("lr", 1e-3), e.get("weight_decay", 0.0)

    def set_lr(self, lr: float) -> None:
        for d in self.table:
            d.lr = lr


def moe_lora_adamw_step(tensors: AdamWTensors, step: int, beta1: float = 0.9, beta2: float = 0.999,
                        eps: float = 1e-8, grad_scale: Optional[torch.Tensor] = None, stream=None) -> None:
    """One AdamW step (number `step`, from 1) over all tensors; grad_scale: a device fp32 scalar that
    multiplies every gradient (e.g. a clipping factor)."""
    opt = AdamW(beta1, beta2, eps, step, _vec(grad_scale, 1, "grad_scale", torch.float32))
    rc = lib().moe_lora_adamw_step(opt, tensors.table, len(tensors.entries), _stream(stream))
    _check(rc, "moe_lora_adamw_step")


# ------------------------------------------------------------------ post-training
def _stream_of(t: torch.Tensor, name: str, stream) -> int:
    """The stream's handle.  Launches go to the current device, which does not hold another device's tensors."""
    device = torch._C._cuda_getDevice()
    if t.get_device() != device:
        raise ValueError(f"{name} must be on the current device, cuda:{device}, got {t.device}")
    return torch._C._cuda_getCurrentRawStream(device) if stream is None else _stream(stream)


def _logit_rows(logits: torch.Tensor, dlogits: Optional[torch.Tensor], inv_temp: float):
    """The row description of logits [rows, n] and their gradient, and both pointers."""
    px, ld = _rows(logits, "logits")
    pd, ldd = (None, 0) if dlogits is None else _rows(dlogits, "dlogits", logits)
    rows, n = logits.shape
    return Rows(rows, ld, ldd, n, _dtype(logits, "logits"), inv_temp), px, pd


def moe_lora_token_logp_forward(logits: torch.Tensor, targets: torch.Tensor, logp: Optional[torch.Tensor],
                                lse: Optional[torch.Tensor] = None, entropy: Optional[torch.Tensor] = None,
                                inv_temp: float = 1.0, err: Optional[torch.Tensor] = None, stream=None) -> None:
    """Log probability of targets [rows] int32 (-1 = none, gives 0) under softmax(inv_temp * logits) of
    logits [rows, n] (fp32, bf16 or fp16; rows may be strided), with lse and entropy if given, all
    [rows] fp32.  err: a device int32 word that collects MOE_LORA_DEV_BAD_ID."""
    r, px, _ = _logit_rows(logits, None, inv_temp)
    T = r.rows
    rc = lib().moe_lora_token_logp_forward(r, px, _vec(targets, T, "targets", torch.int32),
                                           _vec(logp, T, "logp", torch.float32), _vec(lse, T, "lse", torch.float32),
                                           _vec(entropy, T, "entropy", torch.float32), _vec(err, 1, "err", torch.int32),
                                           _stream_of(logits, "logits", stream))
    _check(rc, "moe_lora_token_logp_forward")


def moe_lora_token_logp_backward(logits: torch.Tensor, targets: torch.Tensor, lse: torch.Tensor, dlogp: torch.Tensor,
                                 dlogits: torch.Tensor, inv_temp: float = 1.0, err: Optional[torch.Tensor] = None,
                                 stream=None) -> None:
    """dlogits [rows, n] (the logits' type; may be logits) of the log probabilities, from the forward's
    lse [rows] and the gradient dlogp [rows] that reaches them."""
    r, px, pd = _logit_rows(logits, dlogits, inv_temp)
    T = r.rows
    rc = lib().moe_lora_token_logp_backward(r, px, _vec(targets, T, "targets", torch.int32),
                                            _vec(lse, T, "lse", torch.float32), _vec(dlogp, T, "dlogp", torch.float32),
                                            pd, _vec(err, 1, "err", torch.int32), _stream_of(logits, "logits", stream))
    _check(rc, "moe_lora_token_logp_backward")


def _ticket_scratch(nbytes: int, device) -> torch.Tensor:
    """A workspace whose first 16 bytes are cleared, once."""
    t = torch.empty(nbytes, dtype=torch.uint8, device=device)
    t[:16].zero_()
    return t


def policy_scratch(rows: int, adapters: int = 1, device="cuda") -> torch.Tensor:
    """Workspace of moe_lora_policy_loss."""
    b = int(lib().moe_lora_policy_scratch_bytes(rows, adapters))
    if b == 0:
        raise MoeLoraError(-2, "moe_lora_policy_scratch_bytes")
    return _ticket_scratch(b, device)


def _host_offsets(offsets: Optional[Sequence[int]], adapters: int, name: str):
    if offsets is None:
        return None
    a = array.array("q", offsets)
    if len(a) != adapters + 1:
        raise ValueError(f"{name} must have {adapters + 1} entries")
    return a


def moe_lora_policy_loss(logits: torch.Tensor, targets: torch.Tensor, advantages: torch.Tensor, old_logp: torch.Tensor,
                         ref_logp: Optional[torch.Tensor], loss: torch.Tensor, stats: torch.Tensor,
                         scratch: torch.Tensor, clip_low: float = 0.2, clip_high: float = 0.2, kl_coef: float = 0.0,
                         weight: Optional[torch.Tensor] = None, adapter_offsets: Optional[Sequence[int]] = None,
                         logp: Optional[torch.Tensor] = None, dlogits: Optional[torch.Tensor] = None,
                         dloss: Optional[torch.Tensor] = None, inv_temp: float = 1.0,
                         err: Optional[torch.Tensor] = None, stream=None) -> None:
    """Clipped policy loss [A] with a KL term to ref_logp, for targets [rows] int32 (-1 = none) under
    logits [rows, n]; advantages, old_logp, ref_logp and weight (None: each adapter's mean) [rows] fp32.
    stats [A,4]: weighted KL, clipped share, ratio, entropy.  dlogits [rows, n] (may be logits) receives
    the gradient (for the upstream gradient dloss [A], None = 1) in the same pass if given.
    adapter_offsets [A+1] (host) splits the tokens between adapters."""
    r, px, pd = _logit_rows(logits, dlogits, inv_temp)
    T, A, f32 = r.rows, loss.numel(), torch.float32
    offs = _host_offsets(adapter_offsets, A, "adapter_offsets")
    rc = lib().moe_lora_policy_loss(r, Policy(clip_low, clip_high, kl_coef, A), px,
                                    _vec(targets, T, "targets", torch.int32), _vec(advantages, T, "advantages", f32),
                                    _vec(old_logp, T, "old_logp", f32), _vec(ref_logp, T, "ref_logp", f32),
                                    _vec(weight, T, "weight", f32), None if offs is None else offs.buffer_info()[0],
                                    _vec(dloss, A, "dloss", f32), _vec(loss, A, "loss", f32),
                                    _vec(stats, 4 * A, "stats", f32), _vec(logp, T, "logp", f32), pd,
                                    _vec(err, 1, "err", torch.int32), _ptr(scratch, None, "scratch"),
                                    scratch.numel() * scratch.element_size(), _stream_of(logits, "logits", stream))
    _check(rc, "moe_lora_policy_loss")


PREFERENCE_KINDS = {"sigmoid": 0, "squared": 1, "hinge": 2}


def preference_scratch(pairs: int, adapters: int = 1, device="cuda") -> torch.Tensor:
    """Workspace of moe_lora_preference_loss (its size does not depend on the adapters)."""
    b = int(lib().moe_lora_preference_scratch_bytes(pairs))
    if b == 0 or not 1 <= adapters <= 64:
        raise MoeLoraError(-2, "moe_lora_preference_scratch_bytes")
    return _ticket_scratch(b, device)


def moe_lora_preference_loss(logp: torch.Tensor, targets: torch.Tensor, seq_offsets: torch.Tensor,
                             ref: Optional[torch.Tensor], loss: torch.Tensor, stats: torch.Tensor,
                             scratch: torch.Tensor, beta: float = 0.1, kind: str = "sigmoid",
                             label_smoothing: float = 0.0, margin: float = 0.0, average: bool = False,
                             pair_offsets: Optional[Sequence[int]] = None, seq_logp: Optional[torch.Tensor] = None,
                             dlogp: Optional[torch.Tensor] = None, dloss: Optional[torch.Tensor] = None,
                             err: Optional[torch.Tensor] = None, stream=None) -> None:
    """Preference loss [A] over pairs of packed sequences (2i chosen, 2i + 1 rejected; seq_offsets
    [2 pairs + 1] int64 on the device) of token log probabilities logp [tokens], live where targets
    [tokens] int32 is not negative; ref [2 pairs] holds the reference model's sums.  stats [A,4]: share
    of pairs the right way round, rewards of chosen and rejected, their distance.  dlogp [tokens]
    receives the gradient, seq_logp [2 pairs] the sums (means with `average`)."""
    if seq_offsets.numel() % 2 != 1:
        raise ValueError("seq_offsets must have 2 * pairs + 1 entries")
    if kind not in PREFERENCE_KINDS:
        raise ValueError(f"kind must be one of {sorted(PREFERENCE_KINDS)}, got {kind!r}")
    P, T, A, f32 = seq_offsets.numel() // 2, logp.numel(), loss.numel(), torch.float32
    offs = _host_offsets(pair_offsets, A, "pair_offsets")
    opt = Preference(T, P, beta, margin, label_smoothing, PREFERENCE_KINDS[kind], int(average), A)
    rc = lib().moe_lora_preference_loss(opt, _vec(logp, T, "logp", f32), _vec(targets, T, "targets", torch.int32),
                                        _vec(seq_offsets, 2 * P + 1, "seq_offsets", torch.int64),
                                        _vec(ref, 2 * P, "ref", f32), None if offs is None else offs.buffer_info()[0],
                                        _vec(dloss, A, "dloss", f32), _vec(loss, A, "loss", f32),
                                        _vec(stats, 4 * A, "stats", f32), _vec(seq_logp, 2 * P, "seq_logp", f32),
                                        _vec(dlogp, T, "dlogp", f32), _vec(err, 1, "err", torch.int32),
                                        _ptr(scratch, None, "scratch"), scratch.numel() * scratch.element_size(),
                                        _stream_of(logp, "logp", stream))
    _check(rc, "moe_lora_preference_loss")


class MuonTensors:
    """The tensors of a Muon step, listed once and kept between steps, with their workspace.  Each entry
    is a dict: p (fp32, bf16 or fp16; its last two axes are a matrix, one of them at most 128, all others
    count matrices), g of p's shape, m (fp32 momentum, started at zero), and optionally master (fp32, for
    a 16-bit p), lr (1e-3), weight_decay (0) and scale (sqrt(max(1, rows / cols))), which multiplies the
    update.  All contiguous, on one device; no two overlap.  The entries hold the tensors alive.  Steps
    that may run at the same time need an object each."""

    def __init__(self, entries: Sequence[Dict]):
        self.entries = [dict(e) for e in entries]
        self.table = (MuonTensor * max(1, len(self.entries)))()
        for d, e in zip(self.table, self.entries):
            p, n = e["p"], e["p"].numel()
            if p.dim() < 2:
                raise ValueError("p must have at least two axes")
            if e["g"].shape != p.shape:
                raise ValueError(f"g must be {tuple(p.shape)}, got {tuple(e['g'].shape)}")
            d.rows, d.cols = p.shape[-2:]
            d.batch = n // (d.rows * d.cols) if n else 0
            d.p, d.g, d.m = _vec(p, n, "p"), _vec(e["g"], n, "g"), _vec(e["m"], n, "m", torch.float32)
            d.master = _vec(e.get("master"), n, "master", torch.float32)
            d.p_dtype, d.g_dtype = _dtype(p, "p"), _dtype(e["g"], "g")
            d.lr, d.weight_decay = e.get("lr", 1e-3), e.get("weight_decay", 0.0)
            scale = e.get("scale")
            d.scale = max(1.0, d.rows / max(1, d.cols)) ** 0.5 if scale is None else scale
        b = int(lib().moe_lora_muon_scratch_bytes(self.table, len(self.entries)))
        if b == 0:
            raise MoeLoraError(-5, "moe_lora_muon_scratch_bytes")
        devices = {e[k].device for e in self.entries for k in ("p", "g", "m", "master") if e.get(k) is not None}
        if len(devices) > 1:
            raise ValueError(f"tensors must be on one device, got {sorted(map(str, devices))}")
        self.scratch = _ticket_scratch(b, devices.pop() if devices else "cuda")  # starts with the error word

    def set_lr(self, lr: float) -> None:
        for d in self.table:
            d.lr = lr


def moe_lora_muon_step(tensors: MuonTensors, momentum: float = 0.95, nesterov: bool = True, steps: int = 5,
                       coefs: Sequence[float] = (3.4445, -4.7750, 2.0315), eps: float = 1e-7,
                       grad_scale: Optional[torch.Tensor] = None, stream=None) -> None:
    """One Muon step over all tensors: momentum, `steps` Newton-Schulz steps with the coefficients (a, b, c)
    on every matrix, weights.  grad_scale: a device fp32 scalar that multiplies every gradient."""
    a, b, c = coefs
    opt = Muon(momentum, eps, a, b, c, int(nesterov), steps, _vec(grad_scale, 1, "grad_scale", torch.float32))
    rc = lib().moe_lora_muon_step(opt, tensors.table, len(tensors.entries), tensors.scratch.data_ptr(),
                                  tensors.scratch.numel(), _stream_of(tensors.scratch, "the tensors", stream))
    _check(rc, "moe_lora_muon_step")


def moe_lora_muon_get_error(tensors: MuonTensors, stream=None) -> int:
    rc = lib().moe_lora_muon_get_error(tensors.scratch.data_ptr(), _stream(stream))
    if rc < 0:
        raise MoeLoraError(rc, "moe_lora_muon_get_error")
    return rc


# ------------------------------------------------------------------ convenience
@dataclass
class Workspaces:
    """Device buffers for one problem size (allocated by torch, owned by the caller)."""
    plan: torch.Tensor
    saved: torch.Tensor
    fwd: torch.Tensor
    bwd: torch.Tensor

    @staticmethod
    def allocate(dims: Dims, device="cuda") -> "Workspaces":
        def buf(which):
            n = moe_lora_workspace_bytes(dims, which)
            if n == 0:
                raise MoeLoraError(-2, "moe_lora_workspace_bytes")
            return torch.empty(n, dtype=torch.uint8, device=device)
        return Workspaces(buf(MOE_LORA_WS_PLAN), buf(MOE_LORA_WS_SAVED), buf(MOE_LORA_WS_FWD_SCRATCH),
                          buf(MOE_LORA_WS_BWD_SCRATCH))


def alloc_grads(dims: Dims, device="cuda") -> Dict[str, torch.Tensor]:
    A, E, H, I, r = dims.A, dims.E, dims.H, dims.I, dims.r
    f = dict(dtype=torch.float32, device=device)
    return {"dA1": torch.empty(A, r, H, **f), "dA3": torch.empty(A, r, H, **f),
            "dB1": torch.empty(A, E, I, r, **f), "dB3": torch.empty(A, E, I, r, **f),
            "dA2": torch.empty(A, E, r, I, **f), "dB2": torch.empty(A, H, r, **f)}
