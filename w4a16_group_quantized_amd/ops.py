"""Thin Python binding over libmoe_w4a16.so (C ABI in include/moe_w4a16.h).

Argument marshalling only: each function takes torch tensors, allocates its
outputs with torch (device memory is the caller's), and passes raw device
pointers plus torch's current HIP stream to the library.  Every step of the
layer runs in the library's HIP kernels; there is no fallback, and a missing
library or a non-OK status raises.
"""

from __future__ import annotations

import ctypes
import os

import torch

_PKG_DIR = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG_DIR, "libmoe_w4a16.so")

MOE_OK = 0
MOE_ERR_INVALID_ARG = 1
MOE_ERR_UNSUPPORTED = 2
MOE_ERR_WORKSPACE = 3
MOE_ERR_HIP = 4

GROUP_SIZE = 32

EXPORTED = (
    "moe_status_string",
    "moe_abi_version",
    "moe_route",
    "moe_permute_workspace_bytes",
    "moe_permute",
    "moe_route_permute",
    "moe_ffn_workspace_bytes",
    "moe_w4a16_grouped_ffn",
    "moe_w4a16_gate_up",
    "moe_w4a16_down",
    "moe_route_gate_up",
    "moe_combine",
    "moe_layer_workspace_bytes",
    "moe_layer_forward",
    "moe_layer_forward_noalloc",
    "moe_router_gate",
    "moe_route_shared",
    "moe_block_workspace_bytes",
    "moe_block_forward",
    "moe_plan_default",
    "moe_layer_forward_plan",
    "moe_block_forward_plan",
    "moe_mxfp4_scale_bytes",
    "moe_mxfp4_quantize",
    "moe_mxfp4_dequantize",
    "moe_mxfp4_grouped_gemm",
    "moe_mxfp4_gate_up",
    "moe_mxfp4_layer_workspace_bytes",
    "moe_mxfp4_layer_forward",
    "moe_permute_masked_workspace_bytes",
    "moe_permute_masked",
    "moe_dispatch",
    "moe_dispatch_backward",
    "moe_combine_masked",
    "moe_combine_backward",
)

FFN_GEMV, FFN_MFMA = 0, 1
ROUTE_IN_GATE_UP, ROUTE_ONE_LAUNCH, ROUTE_SEPARATE = 0, 1, 2


class Plan(ctypes.Structure):
    """moe_plan: kernel variant and tile profile of a layer call."""

    _fields_ = [("ffn", ctypes.c_int32), ("route", ctypes.c_int32), ("msub", ctypes.c_int32),
                ("lanes_gate_up", ctypes.c_int32), ("lanes_down", ctypes.c_int32),
                ("rows_per_pass", ctypes.c_int32), ("cost_split", ctypes.c_int32),
                ("router_gemv", ctypes.c_int32), ("shared_mfma", ctypes.c_int32),
                ("combine_in_down", ctypes.c_int32), ("one_launch", ctypes.c_int32)]

    def as_dict(self) -> dict:
        return {name: int(getattr(self, name)) for name, _ in self._fields_}

    def __repr__(self):
        return f"Plan({self.as_dict()})"

NOALLOC_SCRATCH_BYTES = 32 << 20


class MoEError(RuntimeError):
    def __init__(self, fn: str, status: int, msg: str):
        super().__init__(f"{fn} failed with status {status}: {msg}")
        self.status = status


_lib = None

_P = ctypes.c_void_p
_I64 = ctypes.c_int64
_I32 = ctypes.c_int32
_SZ = ctypes.c_size_t

_SIGNATURES = {
    "moe_mxfp4_scale_bytes": (ctypes.c_int, [_I32]),
    "moe_mxfp4_quantize": (ctypes.c_int, [_P, _I32, _I64, _I32, _I64, _P, _P, _P]),
    "moe_mxfp4_dequantize": (ctypes.c_int, [_P, _P, _I64, _I32, _P, _I32, _I64, _P]),
    "moe_mxfp4_grouped_gemm": (
        ctypes.c_int,
        [_P, _P, _I64, _P, _I32, _I64, _P, _I32, _P, _P, _I32, _I32, _P, _I32, _I64, _P]),
    "moe_mxfp4_gate_up": (
        ctypes.c_int,
        [_P, _P, _I64, _P, _I32, _I64, _P, _I32, _P, _P, _I32, _I32, _P, _P, _P]),
    "moe_mxfp4_layer_workspace_bytes": (_SZ, [_I64, _I32, _I32, _I32, _I32]),
    "moe_mxfp4_layer_forward": (
        ctypes.c_int,
        [_P, _P, _I32, _I64, _I32, _I32, _P, _P, _P, _P, _I32, _I32, _P, _P, _SZ, _P]),
    "moe_permute_masked_workspace_bytes": (_SZ, [_I64, _I32, _I32]),
    "moe_permute_masked": (
        ctypes.c_int, [_P, _I64, _I32, _I32, _I32, _P, _P, _P, _P, _P, _P, _SZ, _P]),
    "moe_dispatch": (
        ctypes.c_int, [_P, _I32, _I64, _I32, _I32, _I64, _P, _I64, _P, _I64, _P]),
    "moe_dispatch_backward": (
        ctypes.c_int, [_P, _I32, _I64, _I32, _I32, _I64, _P, _I64, _P, _I64, _P]),
    "moe_combine_masked": (
        ctypes.c_int,
        [_P, _I32, _I64, _I32, _I32, _I64, _P, _P, _I64, _P, _I32, _I64, _P]),
    "moe_combine_backward": (
        ctypes.c_int,
        [_P, _I32, _I64, _P, _I32, _I64, _P, _P, _I64, _I32, _I32, _I64, _P, _I64, _P, _P]),
    "moe_status_string": (ctypes.c_char_p, [ctypes.c_int]),
    "moe_abi_version": (ctypes.c_int, []),
    "moe_route": (ctypes.c_int, [_P, _I64, _I32, _I32, _P, _P, _P]),
    "moe_permute_workspace_bytes": (_SZ, [_I64, _I32, _I32]),
    "moe_permute": (ctypes.c_int, [_P, _I64, _I32, _I32, _P, _P, _P, _P, _P, _P, _SZ, _P]),
    "moe_route_permute": (
        ctypes.c_int, [_P, _I64, _I32, _I32, _P, _P, _P, _P, _P, _P, _P, _P, _SZ, _P]),
    "moe_ffn_workspace_bytes": (_SZ, [_I64, _I32, _I32, _I32, _I32]),
    "moe_w4a16_grouped_ffn": (
        ctypes.c_int,
        [_P, _I64, _I32, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _I32, _I32, _I32, _I32, _P, _P,
         _SZ, _P],
    ),
    "moe_w4a16_gate_up": (
        ctypes.c_int,
        [_P, _I64, _I32, _P, _P, _P, _P, _P, _P, _P, _I32, _I32, _I32, _I32, _P, _SZ, _P],
    ),
    "moe_w4a16_down": (
        ctypes.c_int,
        [_I64, _I32, _P, _P, _P, _P, _P, _P, _I32, _I32, _I32, _I32, _P, _P, _SZ, _P],
    ),
    "moe_combine": (ctypes.c_int, [_P, _P, _P, _I64, _I32, _I32, _P, _P]),
    "moe_route_gate_up": (
        ctypes.c_int,
        [_P, _P, _I64, _I32, _I32, _P, _P, _P, _I32, _I32, _I32, _P, _P, _P, _P, _P, _P, _P, _P,
         _SZ, _P]),
    "moe_layer_workspace_bytes": (_SZ, [_I64, _I32, _I32, _I32, _I32]),
    "moe_layer_forward": (
        ctypes.c_int,
        [_P, _P, _I64, _I32, _I32, _P, _P, _P, _P, _P, _P, _I32, _I32, _I32, _P, _P, _SZ, _P]),
    "moe_layer_forward_noalloc": (
        ctypes.c_int,
        [_P, _P, _I64, _I32, _I32, _P, _P, _P, _P, _P, _P, _I32, _I32, _I32, _P, _P]),
    "moe_router_gate": (ctypes.c_int, [_P, _I64, _I32, _P, _I32, _P, _P]),
    "moe_route_shared": (ctypes.c_int, [_P, _I64, _I32, _I32, _P, _P, _P]),
    "moe_block_workspace_bytes": (_SZ, [_I64, _I32, _I32, _I32, _I32, _I32]),
    "moe_plan_default": (ctypes.c_int, [_I64, _I32, _I32, _I32, _I32, _I32, _P]),
    "moe_layer_forward_plan": (
        ctypes.c_int,
        [_P, _P, _I64, _I32, _I32, _P, _P, _P, _P, _P, _P, _I32, _I32, _I32, _P, _P, _SZ, _P,
         _P]),
    "moe_block_forward_plan": (
        ctypes.c_int,
        [_P, _I64, _P, _I32, _I32, _I32, _P, _P, _P, _P, _P, _P, _I32, _I32, _I32, _P, _P, _P,
         _SZ, _P, _P]),
    "moe_block_forward": (
        ctypes.c_int,
        [_P, _I64, _P, _I32, _I32, _I32, _P, _P, _P, _P, _P, _P, _I32, _I32, _I32, _P, _P, _P,
         _SZ, _P]),
}


def load_library(path: str = LIB_PATH) -> ctypes.CDLL:
    """Open the HIP library (once); raises if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(
            f"{path} is missing: build it with `python -m w4a16_group_quantized_amd.build_lib`"
        )
    lib = ctypes.CDLL(path)
    for name, (res, args) in _SIGNATURES.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    _lib = lib
    return lib


def status_string(status: int) -> str:
    return load_library().moe_status_string(status).decode()


def _check(fn: str, status: int) -> None:
    if status != MOE_OK:
        raise MoEError(fn, status, status_string(status))


def _ptr(t: torch.Tensor | None) -> int | None:
    if t is None:
        return None
    if not t.is_contiguous():
        raise ValueError("tensors passed to the library must be contiguous")
    return t.data_ptr() or None


def _stream() -> int | None:
    return torch.cuda.current_stream().cuda_stream or None


# --------------------------------------------------------------------------- #
# size queries
# --------------------------------------------------------------------------- #
def permute_workspace_bytes(T: int, top_k: int, E: int) -> int:
    return int(load_library().moe_permute_workspace_bytes(T, top_k, E))


def ffn_workspace_bytes(T: int, top_k: int, E: int, H: int, I: int) -> int:
    return int(load_library().moe_ffn_workspace_bytes(T, top_k, E, H, I))


def _workspace(nbytes: int, device) -> torch.Tensor:
    return torch.empty(max(nbytes, 1), dtype=torch.uint8, device=device)


# --------------------------------------------------------------------------- #
# the four layer calls (plus the two halves of the FFN)
# --------------------------------------------------------------------------- #
def moe_route(logits: torch.Tensor, top_k: int, out_ids=None, out_weights=None):
    """fp32 logits [T, E] -> (topk_ids int32 [T, k], topk_weights fp32 [T, k])."""
    lib = load_library()
    T, E = logits.shape
    dev = logits.device
    ids = out_ids if out_ids is not None else torch.empty((T, top_k), dtype=torch.int32, device=dev)
    w = out_weights if out_weights is not None else torch.empty((T, top_k), dtype=torch.float32, device=dev)
    _check("moe_route", lib.moe_route(_ptr(logits), T, E, top_k, _ptr(ids), _ptr(w), _stream()))
    return ids, w


def moe_permute(topk_ids: torch.Tensor, E: int, workspace: torch.Tensor | None = None,
                out: dict | None = None) -> dict:
    """topk_ids [T, k] -> dict of expert_offsets, sorted_slots, slot_rows, active_experts, num_active."""
    lib = load_library()
    T, k = topk_ids.shape
    dev = topk_ids.device
    S = T * k
    if out is None:
        out = {
            "expert_offsets": torch.empty(E + 1, dtype=torch.int32, device=dev),
            "sorted_slots": torch.empty(S, dtype=torch.int32, device=dev),
            "slot_rows": torch.empty(S, dtype=torch.int32, device=dev),
            "active_experts": torch.empty(E, dtype=torch.int32, device=dev),
            "num_active": torch.empty(1, dtype=torch.int32, device=dev),
        }
    need = permute_workspace_bytes(T, k, E)
    if workspace is None:
        workspace = _workspace(need, dev)
    _check("moe_permute", lib.moe_permute(
        _ptr(topk_ids), T, k, E, _ptr(out["expert_offsets"]), _ptr(out["sorted_slots"]),
        _ptr(out["slot_rows"]), _ptr(out["active_experts"]), _ptr(out["num_active"]),
        _ptr(workspace), workspace.numel(), _stream()))
    return out


def moe_route_permute(logits: torch.Tensor, top_k: int, workspace: torch.Tensor | None = None,
                      out_ids=None, out_weights=None, out: dict | None = None):
    """moe_route then moe_permute in one call (one launch for small T): (ids, weights, perm dict)."""
    lib = load_library()
    T, E = logits.shape
    dev = logits.device
    S = T * top_k
    ids = out_ids if out_ids is not None else torch.empty((T, top_k), dtype=torch.int32, device=dev)
    w = out_weights if out_weights is not None else torch.empty((T, top_k), dtype=torch.float32, device=dev)
    if out is None:
        out = {
            "expert_offsets": torch.empty(E + 1, dtype=torch.int32, device=dev),
            "sorted_slots": torch.empty(S, dtype=torch.int32, device=dev),
            "slot_rows": torch.empty(S, dtype=torch.int32, device=dev),
            "active_experts": torch.empty(E, dtype=torch.int32, device=dev),
            "num_active": torch.empty(1, dtype=torch.int32, device=dev),
        }
    need = permute_workspace_bytes(T, top_k, E)
    if workspace is None:
        workspace = _workspace(need, dev)
    _check("moe_route_permute", lib.moe_route_permute(
        _ptr(logits), T, E, top_k, _ptr(ids), _ptr(w), _ptr(out["expert_offsets"]),
        _ptr(out["sorted_slots"]), _ptr(out["slot_rows"]), _ptr(out["active_experts"]),
        _ptr(out["num_active"]), _ptr(workspace), workspace.numel(), _stream()))
    return ids, w, out


def _ffn_ws(T, k, E, H, I, workspace, dev):
    need = ffn_workspace_bytes(T, k, E, H, I)
    if workspace is None:
        workspace = _workspace(need, dev)
    return workspace


def moe_w4a16_grouped_ffn(x: torch.Tensor, top_k: int, perm: dict, w: dict,
                          y_sorted: torch.Tensor | None = None,
                          workspace: torch.Tensor | None = None) -> torch.Tensor:
    """x fp16 [T, H] -> y_sorted fp32 [T*k, H] (sorted-row order)."""
    lib = load_library()
    T, H = x.shape
    E = w["w13_q"].shape[0]
    I = w["w2_q"].shape[2] * 8
    dev = x.device
    if y_sorted is None:
        y_sorted = torch.empty((T * top_k, H), dtype=torch.float32, device=dev)
    workspace = _ffn_ws(T, top_k, E, H, I, workspace, dev)
    _check("moe_w4a16_grouped_ffn", lib.moe_w4a16_grouped_ffn(
        _ptr(x), T, top_k, _ptr(perm["expert_offsets"]), _ptr(perm["sorted_slots"]),
        _ptr(perm["active_experts"]), _ptr(perm["num_active"]),
        _ptr(w["w13_q"]), _ptr(w["w13_s"]), _ptr(w["w13_z"]),
        _ptr(w["w2_q"]), _ptr(w["w2_s"]), _ptr(w["w2_z"]),
        E, H, I, GROUP_SIZE, _ptr(y_sorted), _ptr(workspace), workspace.numel(), _stream()))
    return y_sorted


def moe_w4a16_gate_up(x: torch.Tensor, top_k: int, perm: dict, w: dict,
                      workspace: torch.Tensor) -> None:
    lib = load_library()
    T, H = x.shape
    E = w["w13_q"].shape[0]
    I = w["w2_q"].shape[2] * 8
    _check("moe_w4a16_gate_up", lib.moe_w4a16_gate_up(
        _ptr(x), T, top_k, _ptr(perm["expert_offsets"]), _ptr(perm["sorted_slots"]),
        _ptr(perm["active_experts"]), _ptr(perm["num_active"]),
        _ptr(w["w13_q"]), _ptr(w["w13_s"]), _ptr(w["w13_z"]),
        E, H, I, GROUP_SIZE, _ptr(workspace), workspace.numel(), _stream()))


def moe_w4a16_down(T: int, top_k: int, perm: dict, w: dict, y_sorted: torch.Tensor,
                   workspace: torch.Tensor) -> None:
    lib = load_library()
    E, H = w["w2_q"].shape[0], w["w2_q"].shape[1]
    I = w["w2_q"].shape[2] * 8
    _check("moe_w4a16_down", lib.moe_w4a16_down(
        T, top_k, _ptr(perm["expert_offsets"]), _ptr(perm["active_experts"]),
        _ptr(perm["num_active"]), _ptr(w["w2_q"]), _ptr(w["w2_s"]), _ptr(w["w2_z"]),
        E, H, I, GROUP_SIZE, _ptr(y_sorted), _ptr(workspace), workspace.numel(), _stream()))


def moe_route_gate_up(logits: torch.Tensor, x: torch.Tensor, top_k: int, w: dict,
                      ids: torch.Tensor, weights: torch.Tensor, perm: dict,
                      workspace: torch.Tensor) -> None:
    """Decode sizes (T <= 8): router, permutation and gate/up in one launch; the routing
    goes to ids, weights and perm (as moe_route_permute), act to the FFN workspace."""
    lib = load_library()
    T, E = logits.shape
    H = x.shape[1]
    I = w["w13_q"].shape[1] // 2
    _check("moe_route_gate_up", lib.moe_route_gate_up(
        _ptr(logits), _ptr(x), T, E, top_k, _ptr(w["w13_q"]), _ptr(w["w13_s"]), _ptr(w["w13_z"]),
        H, I, GROUP_SIZE, _ptr(ids), _ptr(weights), _ptr(perm["expert_offsets"]),
        _ptr(perm["sorted_slots"]), _ptr(perm["slot_rows"]), _ptr(perm["active_experts"]),
        _ptr(perm["num_active"]), _ptr(workspace), workspace.numel(), _stream()))


def moe_combine(y_sorted: torch.Tensor, topk_weights: torch.Tensor, slot_rows: torch.Tensor,
                out: torch.Tensor | None = None) -> torch.Tensor:
    """y_sorted fp32 [T*k, H] -> out fp16 [T, H]."""
    lib = load_library()
    T, k = topk_weights.shape
    H = y_sorted.shape[1]
    if out is None:
        out = torch.empty((T, H), dtype=torch.float16, device=y_sorted.device)
    _check("moe_combine", lib.moe_combine(
        _ptr(y_sorted), _ptr(topk_weights), _ptr(slot_rows), T, k, H, _ptr(out), _stream()))
    return out


def layer_workspace_bytes(T: int, top_k: int, E: int, H: int, I: int) -> int:
    return int(load_library().moe_layer_workspace_bytes(T, top_k, E, H, I))


def layer_workspace_views(ws: torch.Tensor, T: int, top_k: int, E: int, H: int, I: int) -> dict:
    """The routing and y_sorted inside a moe_layer_forward workspace (layout of the header)."""
    S = T * top_k

    def a256(n):
        return (n + 255) & ~255

    sizes = [("topk_ids", 4 * S), ("topk_weights", 4 * S), ("expert_offsets", 4 * (E + 1)),
             ("sorted_slots", 4 * S), ("slot_rows", 4 * S), ("active_experts", 4 * E),
             ("num_active", 4), ("perm_ws", permute_workspace_bytes(T, top_k, E)),
             ("ffn_ws", ffn_workspace_bytes(T, top_k, E, H, I)), ("y_sorted", 4 * S * H)]
    views, at = {}, 0
    for name, n in sizes:
        views[name] = ws[at:at + n]
        at += a256(n)
    out = {k: views[k].view(torch.int32) for k in ("topk_ids", "sorted_slots", "slot_rows",
                                                   "expert_offsets", "active_experts", "num_active")}
    out["topk_ids"] = out["topk_ids"].view(T, top_k)
    out["topk_weights"] = views["topk_weights"].view(torch.float32).view(T, top_k)
    out["y_sorted"] = views["y_sorted"].view(torch.float32).view(S, H)
    return out


def moe_layer_forward(logits: torch.Tensor, x: torch.Tensor, top_k: int, w: dict,
                      workspace: torch.Tensor | None = None, out: torch.Tensor | None = None):
    """The whole layer in one call: logits fp32 [T, E], x fp16 [T, H] -> out fp16 [T, H]."""
    lib = load_library()
    T, E = logits.shape
    H = x.shape[1]
    I = w["w2_q"].shape[2] * 8
    dev = x.device
    if workspace is None:
        workspace = _workspace(layer_workspace_bytes(T, top_k, E, H, I), dev)
    if out is None:
        out = torch.empty((T, H), dtype=torch.float16, device=dev)
    _check("moe_layer_forward", lib.moe_layer_forward(
        _ptr(logits), _ptr(x), T, E, top_k, _ptr(w["w13_q"]), _ptr(w["w13_s"]), _ptr(w["w13_z"]),
        _ptr(w["w2_q"]), _ptr(w["w2_s"]), _ptr(w["w2_z"]), H, I, GROUP_SIZE, _ptr(out),
        _ptr(workspace), workspace.numel(), _stream()))
    return out


def moe_layer_forward_noalloc(logits: torch.Tensor, x: torch.Tensor, top_k: int, w: dict,
                              out: torch.Tensor) -> torch.Tensor:
    """moe_layer_forward without a workspace: the library's per-device scratch is used.
    `out` fp16 [T, H] is the caller's (this call allocates nothing)."""
    lib = load_library()
    T, E = logits.shape
    H = x.shape[1]
    I = w["w2_q"].shape[2] * 8
    _check("moe_layer_forward_noalloc", lib.moe_layer_forward_noalloc(
        _ptr(logits), _ptr(x), T, E, top_k, _ptr(w["w13_q"]), _ptr(w["w13_s"]), _ptr(w["w13_z"]),
        _ptr(w["w2_q"]), _ptr(w["w2_s"]), _ptr(w["w2_z"]), H, I, GROUP_SIZE, _ptr(out), _stream()))
    return out


# --------------------------------------------------------------------------- #
# the MoE block: router gate projection, shared expert
# --------------------------------------------------------------------------- #
def moe_router_gate(x: torch.Tensor, gate_weight: torch.Tensor, out: torch.Tensor | None = None):
    """fp16 x [T, H], fp16 gate_weight [E, H] -> fp32 logits [T, E]."""
    lib = load_library()
    T, H = x.shape
    E = gate_weight.shape[0]
    if out is None:
        out = torch.empty((T, E), dtype=torch.float32, device=x.device)
    _check("moe_router_gate", lib.moe_router_gate(_ptr(x), T, H, _ptr(gate_weight), E, _ptr(out),
                                                  _stream()))
    return out


def moe_route_shared(logits: torch.Tensor, top_k: int):
    """fp32 logits [T, E] -> (ids int32 [T, k+1], weights fp32 [T, k+1]); column k is the
    shared expert E with weight 1."""
    lib = load_library()
    T, E = logits.shape
    dev = logits.device
    ids = torch.empty((T, top_k + 1), dtype=torch.int32, device=dev)
    w = torch.empty((T, top_k + 1), dtype=torch.float32, device=dev)
    _check("moe_route_shared", lib.moe_route_shared(_ptr(logits), T, E, top_k, _ptr(ids), _ptr(w),
                                                    _stream()))
    return ids, w


def block_workspace_bytes(T: int, top_k: int, E: int, shared: bool, H: int, I: int) -> int:
    return int(load_library().moe_block_workspace_bytes(T, top_k, E, int(shared), H, I))


def moe_block_forward(x: torch.Tensor, gate_weight: torch.Tensor, top_k: int, w: dict,
                      shared: bool = True, workspace: torch.Tensor | None = None,
                      logits: torch.Tensor | None = None, out: torch.Tensor | None = None):
    """The MoE block: projection, routed layer and (when ``shared``) the shared expert,
    stored as expert E of the weight arrays.  Returns (out fp16 [T, H], logits fp32 [T, E])."""
    lib = load_library()
    T, H = x.shape
    E = gate_weight.shape[0]
    I = w["w2_q"].shape[2] * 8
    dev = x.device
    if workspace is None:
        workspace = _workspace(block_workspace_bytes(T, top_k, E, shared, H, I), dev)
    if logits is None:
        logits = torch.empty((T, E), dtype=torch.float32, device=dev)
    if out is None:
        out = torch.empty((T, H), dtype=torch.float16, device=dev)
    _check("moe_block_forward", lib.moe_block_forward(
        _ptr(x), T, _ptr(gate_weight), E, top_k, int(shared), _ptr(w["w13_q"]), _ptr(w["w13_s"]),
        _ptr(w["w13_z"]), _ptr(w["w2_q"]), _ptr(w["w2_s"]), _ptr(w["w2_z"]), H, I, GROUP_SIZE,
        _ptr(logits), _ptr(out), _ptr(workspace), workspace.numel(), _stream()))
    return out, logits


def plan_default(T: int, top_k: int, E: int, H: int, I: int, shared: bool = False) -> Plan:
    """The plan the library uses for these sizes (routed top_k and E; `shared`: a shared expert)."""
    p = Plan()
    _check("moe_plan_default", load_library().moe_plan_default(T, top_k, E, int(shared), H, I,
                                                               ctypes.addressof(p)))
    return p


def _plan_ptr(plan):
    return None if plan is None else ctypes.addressof(plan)


def moe_layer_forward_plan(logits: torch.Tensor, x: torch.Tensor, top_k: int, w: dict,
                           plan: Plan | None, workspace: torch.Tensor | None = None,
                           out: torch.Tensor | None = None):
    """moe_layer_forward with an explicit plan (None: the default)."""
    lib = load_library()
    T, E = logits.shape
    H = x.shape[1]
    I = w["w2_q"].shape[2] * 8
    dev = x.device
    if workspace is None:
        workspace = _workspace(layer_workspace_bytes(T, top_k, E, H, I), dev)
    if out is None:
        out = torch.empty((T, H), dtype=torch.float16, device=dev)
    _check("moe_layer_forward_plan", lib.moe_layer_forward_plan(
        _ptr(logits), _ptr(x), T, E, top_k, _ptr(w["w13_q"]), _ptr(w["w13_s"]), _ptr(w["w13_z"]),
        _ptr(w["w2_q"]), _ptr(w["w2_s"]), _ptr(w["w2_z"]), H, I, GROUP_SIZE, _ptr(out),
        _ptr(workspace), workspace.numel(), _plan_ptr(plan), _stream()))
    return out


def moe_block_forward_plan(x: torch.Tensor, gate_weight: torch.Tensor, top_k: int, w: dict,
                           shared: bool, plan: Plan | None, workspace: torch.Tensor,
                           logits: torch.Tensor, out: torch.Tensor):
    """moe_block_forward with an explicit plan (None: the default)."""
    lib = load_library()
    T, H = x.shape
    E = gate_weight.shape[0]
    I = w["w2_q"].shape[2] * 8
    _check("moe_block_forward_plan", lib.moe_block_forward_plan(
        _ptr(x), T, _ptr(gate_weight), E, top_k, int(shared), _ptr(w["w13_q"]), _ptr(w["w13_s"]),
        _ptr(w["w13_z"]), _ptr(w["w2_q"]), _ptr(w["w2_s"]), _ptr(w["w2_z"]), H, I, GROUP_SIZE,
        _ptr(logits), _ptr(out), _ptr(workspace), workspace.numel(), _plan_ptr(plan), _stream()))
    return out


class MoEBlock:
    """Device-resident buffers for repeated block calls at one size (graph-capturable):
    the projection, the routed experts and the shared expert in one entry point."""

    def __init__(self, T: int, E: int, top_k: int, H: int, I: int, shared: bool = True,
                 device="cuda"):
        self.T, self.E, self.top_k, self.H, self.I, self.shared = T, E, top_k, H, I, shared
        dev = torch.device(device)
        self.ws = _workspace(block_workspace_bytes(T, top_k, E, shared, H, I), dev)
        self.logits = torch.empty((T, E), dtype=torch.float32, device=dev)
        self.out = torch.empty((T, H), dtype=torch.float16, device=dev)

    def __call__(self, x: torch.Tensor, gate_weight: torch.Tensor, w: dict) -> torch.Tensor:
        moe_block_forward(x, gate_weight, self.top_k, w, self.shared, self.ws, self.logits,
                          self.out)
        return self.out

    def views(self) -> dict:
        k, E = self.top_k + int(self.shared), self.E + int(self.shared)
        return layer_workspace_views(self.ws, self.T, k, E, self.H, self.I)


# --------------------------------------------------------------------------- #
# one whole layer call
# --------------------------------------------------------------------------- #
class MoELayer:
    """Device-resident buffers for repeated layer calls at one size (graph-capturable)."""

    def __init__(self, T: int, E: int, top_k: int, H: int, I: int, device="cuda"):
        self.T, self.E, self.top_k, self.H, self.I = T, E, top_k, H, I
        S = T * top_k
        dev = torch.device(device)
        self.ids = torch.empty((T, top_k), dtype=torch.int32, device=dev)
        self.weights = torch.empty((T, top_k), dtype=torch.float32, device=dev)
        self.perm = {
            "expert_offsets": torch.empty(E + 1, dtype=torch.int32, device=dev),
            "sorted_slots": torch.empty(S, dtype=torch.int32, device=dev),
            "slot_rows": torch.empty(S, dtype=torch.int32, device=dev),
            "active_experts": torch.empty(E, dtype=torch.int32, device=dev),
            "num_active": torch.empty(1, dtype=torch.int32, device=dev),
        }
        self.perm_ws = _workspace(permute_workspace_bytes(T, top_k, E), dev)
        self.ffn_ws = _workspace(ffn_workspace_bytes(T, top_k, E, H, I), dev)
        self.y_sorted = torch.empty((S, H), dtype=torch.float32, device=dev)
        self.out = torch.empty((T, H), dtype=torch.float16, device=dev)
        self.layer_ws = _workspace(layer_workspace_bytes(T, top_k, E, H, I), dev)
        self.fused_out = torch.empty((T, H), dtype=torch.float16, device=dev)

    def __call__(self, logits: torch.Tensor, x: torch.Tensor, w: dict) -> torch.Tensor:
        moe_route_permute(logits, self.top_k, self.perm_ws, self.ids, self.weights, self.perm)
        moe_w4a16_grouped_ffn(x, self.top_k, self.perm, w, self.y_sorted, self.ffn_ws)
        moe_combine(self.y_sorted, self.weights, self.perm["slot_rows"], self.out)
        return self.out

    def forward(self, logits: torch.Tensor, x: torch.Tensor, w: dict) -> torch.Tensor:
        """The same layer through moe_layer_forward (one call; routing kept in layer_ws)."""
        return moe_layer_forward(logits, x, self.top_k, w, self.layer_ws, self.fused_out)

    def forward_views(self) -> dict:
        return layer_workspace_views(self.layer_ws, self.T, self.top_k, self.E, self.H, self.I)


def weights_to_device(host: dict, device="cuda") -> dict:
    """numpy weight arrays -> device tensors (int32 and fp16 bit-compatible dtypes)."""
    out = {}
    for key in ("w13_q", "w13_z", "w2_q", "w2_z"):
        out[key] = torch.from_numpy(host[key]).to(device)
    for key in ("w13_s", "w2_s"):
        out[key] = torch.from_numpy(host[key]).to(device)
    return out


# --------------------------------------------------------------------------- #
# MXFP4 experts, and token rows to expert order and back
#
# These calls check their tensors (device, type, shape, layout) and run on the
# tensors' own device, on that device's current stream.  Gradients are calls of
# their own: nothing here records an autograd graph.
# --------------------------------------------------------------------------- #
_DTYPE = {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2}

# The checks below run on every call of a few microseconds, so each asks a
# tensor as little as it can; what went wrong is worked out only for a refusal.


def _device_of(*tensors) -> int:
    """Index of the one GPU that all the given tensors (None: absent) are on."""
    dev = tensors[0].get_device()
    for t in tensors:
        if t is not None and (t.get_device() != dev or dev < 0):
            where = "not on a GPU" if t.get_device() < 0 else f"others are on {tensors[0].device}"
            raise ValueError(f"a tensor of shape {tuple(t.shape)} is on {t.device}, {where}")
    return dev


_fns: dict = {}


def _run(fn: str, dev: int, *args) -> None:
    f = _fns.get(fn)
    if f is None:
        f = _fns[fn] = getattr(load_library(), fn)
    # the device's current stream as torch keeps it, without an object around it
    if dev == torch._C._cuda_getDevice():
        status = f(*args, torch._C._cuda_getCurrentRawStream(dev))
    else:
        with torch.cuda.device(dev):
            status = f(*args, torch._C._cuda_getCurrentRawStream(dev))
    if status != MOE_OK:
        _check(fn, status)


def _dense(name: str, t: torch.Tensor, dtype: torch.dtype, *shape) -> int:
    """Pointer of a contiguous tensor of this type and shape."""
    if t.dtype is not dtype:
        raise ValueError(f"{name} is {t.dtype}, not {dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, not {shape}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _bytes(name: str, t: torch.Tensor | None):
    """(pointer, bytes) of a workspace (None: none)."""
    if t is None:
        return None, 0
    n = t.numel()
    return _dense(name, t, torch.uint8, n), n


def _matrix(name: str, t: torch.Tensor):
    """(pointer, dtype code, row stride, rows, columns) of a matrix with contiguous rows."""
    code = _DTYPE.get(t.dtype)
    if code is None:
        raise ValueError(f"{name} is {t.dtype}, not float32, float16 or bfloat16")
    if t.dim() != 2:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, not two dimensions")
    rows, cols = t.shape
    if t.is_contiguous():
        return t.data_ptr(), code, cols, rows, cols
    if cols > 1 and t.stride(1) != 1:
        raise ValueError(f"{name} must have contiguous rows")
    stride = t.stride(0) if rows > 1 else max(t.stride(0), cols)
    if stride < cols:
        raise ValueError(f"{name} has rows that overlap (stride {stride})")
    return t.data_ptr(), code, stride, rows, cols


def _sized(name: str, t: torch.Tensor, rows: int, cols: int, code: int | None = None):
    """(pointer, dtype code, row stride) of such a matrix of a given shape (and type)."""
    ptr, got, stride, r, c = _matrix(name, t)
    if r != rows or c != cols:
        raise ValueError(f"{name} has shape {(r, c)}, not {(rows, cols)}")
    if code is not None and got != code:
        raise ValueError(f"{name} is {t.dtype}, not the type of the tensor that it goes with")
    return ptr, got, stride


def _made(like: torch.Tensor, rows: int, cols: int, dtype: torch.dtype):
    """(matrix, pointer, dtype code, row stride) of an output made here."""
    code = _DTYPE.get(dtype)
    if code is None:
        raise ValueError(f"dtype {dtype} is not float32, float16 or bfloat16")
    out = like.new_empty((rows, cols), dtype=dtype)
    return out, out.data_ptr(), code, cols


def _apart(name: str, out: torch.Tensor, **inputs) -> None:
    """Refuses an output matrix that shares memory with an input matrix.  Column ranges of one
    buffer (equal row strides) may interleave as long as they do not meet."""
    def place(t):
        size, rows, cols = t.element_size(), t.shape[0], t.shape[1]
        stride = (t.stride(0) if rows > 1 else cols) * size
        return t.data_ptr(), stride, cols * size, (rows - 1) * stride + cols * size

    a, dense = out.data_ptr(), out.is_contiguous()
    for other, t in inputs.items():
        if dense and t.is_contiguous():  # the usual case, at the least cost
            b = t.data_ptr()
            if a + out.nbytes <= b or b + t.nbytes <= a:
                continue
        if out.numel() == 0 or t.numel() == 0:
            continue
        a, a_stride, a_cols, a_span = place(out)
        b, b_stride, b_cols, b_span = place(t)
        if a + a_span <= b or b + b_span <= a:
            continue
        d = (b - a) % a_stride
        if a_stride == b_stride and a_cols <= d and d + b_cols <= a_stride:
            continue
        raise ValueError(f"{name} overlaps {other}")


def mxfp4_scale_bytes(K: int) -> int:
    """Bytes of one row's scales for K columns: one per 32, rows padded to whole 32-bit words."""
    if K < 32 or K % 32 or K > 65536:
        raise ValueError(f"K = {K} is not a multiple of 32 in [32, 65536]")
    return (K + 127) // 128 * 4


def _mx(name: str, codes: torch.Tensor, scales: torch.Tensor, dims: int):
    """(codes pointer, scales pointer, shape with K in place of its words) of an MXFP4 tensor."""
    if codes.dim() == dims:  # the usual case, at the least cost
        if dims == 2:
            rows, words = codes.shape
            want = (rows, (words + 15) // 16 * 4)
            shape = (rows, words * 8)
        else:
            experts, rows, words = codes.shape
            want = (experts, rows, (words + 15) // 16 * 4)
            shape = (experts, rows, words * 8)
        if (codes.dtype is torch.int32 and scales.dtype is torch.uint8 and scales.shape == want
                and not words % 4 and 0 < words <= 8192 and codes.is_contiguous()
                and scales.is_contiguous()):
            return codes.data_ptr(), scales.data_ptr(), shape
    shape = codes.shape
    if len(shape) != dims:
        raise ValueError(f"{name} codes have shape {tuple(shape)}, not {dims} dimensions")
    lead, words = shape[:-1], shape[-1]
    return (_dense(name, codes, torch.int32, *shape),
            _dense(name + " scales", scales, torch.uint8, *lead, mxfp4_scale_bytes(words * 8)),
            (*lead, words * 8))


def _mx_out(out: tuple | None, rows: int, K: int, like: torch.Tensor):
    """(codes, scales, their pointers) of an MXFP4 output, made here unless given."""
    sbytes = mxfp4_scale_bytes(K)
    if out is None:
        codes = like.new_empty((rows, K // 8), dtype=torch.int32)
        scales = like.new_empty((rows, sbytes), dtype=torch.uint8)
        return codes, scales, codes.data_ptr(), scales.data_ptr()
    codes, scales = out
    return (codes, scales, _dense("codes", codes, torch.int32, rows, K // 8),
            _dense("scales", scales, torch.uint8, rows, sbytes))


def moe_mxfp4_quantize(x: torch.Tensor, out: tuple | None = None):
    """x [R, K] -> (codes int32 [R, K/8], scales uint8 [R, mxfp4_scale_bytes(K)])."""
    ptr, dtype, stride, R, K = _matrix("x", x)
    codes, scales, pc, ps = _mx_out(out, R, K, x)
    _run("moe_mxfp4_quantize", _device_of(x, codes, scales), ptr, dtype, R, K, stride, pc, ps)
    return codes, scales


def moe_mxfp4_dequantize(codes: torch.Tensor, scales: torch.Tensor,
                         dtype: torch.dtype = torch.float32, out: torch.Tensor | None = None):
    """The values of MXFP4 rows, rounded to dtype (or out's type): [R, K]."""
    pc, ps, (R, K) = _mx("x", codes, scales, 2)
    if out is None:
        out, ptr, code, stride = _made(codes, R, K, dtype)
    else:
        ptr, code, stride = _sized("out", out, R, K)
    _run("moe_mxfp4_dequantize", _device_of(codes, scales, out), pc, ps, R, K, ptr, code, stride)
    return out


def _product_args(a_codes, a_scales, w_codes, w_scales, expert_offsets, row_slots, top_k):
    pa, sa, (rows, K) = _mx("a", a_codes, a_scales, 2)
    pw, sw, (E, N, Kw) = _mx("w", w_codes, w_scales, 3)
    if K != Kw:
        raise ValueError(f"a has {K} columns, w has {Kw}")
    a_rows, po, pr = rows, None, None
    if row_slots is not None:
        rows = row_slots.numel()
        pr = _dense("row_slots", row_slots, torch.int32, rows)
    if expert_offsets is not None:
        po = _dense("expert_offsets", expert_offsets, torch.int32, E + 1)
    return (pa, sa, a_rows, pr, top_k, rows, po, E, pw, sw), rows, N, K


def moe_mxfp4_grouped_gemm(a_codes: torch.Tensor, a_scales: torch.Tensor, w_codes: torch.Tensor,
                           w_scales: torch.Tensor, expert_offsets: torch.Tensor | None = None,
                           row_slots: torch.Tensor | None = None, top_k: int = 1,
                           dtype: torch.dtype = torch.float32, out: torch.Tensor | None = None):
    """MXFP4 rows times their expert's MXFP4 weights [E, N, K]: out [rows, N].  Rows are a's, or
    a's row_slots[r] // top_k; without expert_offsets (E == 1) all belong to the one expert.  Rows
    outside the experts' segments are left as they were (undefined when out is made here)."""
    args, rows, N, K = _product_args(a_codes, a_scales, w_codes, w_scales, expert_offsets,
                                     row_slots, top_k)
    if out is None:
        out, ptr, code, stride = _made(a_codes, rows, N, dtype)
    else:
        ptr, code, stride = _sized("out", out, rows, N)
    _run("moe_mxfp4_grouped_gemm",
         _device_of(a_codes, a_scales, w_codes, w_scales, expert_offsets, row_slots, out), *args, N,
         K, ptr, code, stride)
    return out


def moe_mxfp4_gate_up(a_codes: torch.Tensor, a_scales: torch.Tensor, w13_codes: torch.Tensor,
                      w13_scales: torch.Tensor, expert_offsets: torch.Tensor | None = None,
                      row_slots: torch.Tensor | None = None, top_k: int = 1,
                      out: tuple | None = None):
    """SiLU(gate) * up of MXFP4 rows and W13 [E, 2I, H], stored as MXFP4: (codes, scales) [rows, I]."""
    args, rows, N, H = _product_args(a_codes, a_scales, w13_codes, w13_scales, expert_offsets,
                                     row_slots, top_k)
    if N % 64:
        raise ValueError(f"w13 has {N} rows per expert, not a multiple of 64")
    codes, scales, pc, ps = _mx_out(out, rows, N // 2, a_codes)
    _run("moe_mxfp4_gate_up",
         _device_of(a_codes, a_scales, w13_codes, w13_scales, expert_offsets, row_slots, codes,
                    scales), *args, N // 2, H, pc, ps)
    return codes, scales


def mxfp4_layer_workspace_bytes(T: int, top_k: int, E: int, H: int, I: int) -> int:
    return int(load_library().moe_mxfp4_layer_workspace_bytes(T, top_k, E, H, I))


def moe_mxfp4_layer_forward(logits: torch.Tensor, x: torch.Tensor, top_k: int, w: dict,
                            workspace: torch.Tensor | None = None, out: torch.Tensor | None = None):
    """The routed-expert layer on MXFP4 experts: logits fp32 [T, E], x [T, H] -> out [T, H] of
    x's type.  w: w13_codes, w13_scales [E, 2I, H] and w2_codes, w2_scales [E, H, I]."""
    w13, w13_s, w2, w2_s = w["w13_codes"], w["w13_scales"], w["w2_codes"], w["w2_scales"]
    pw13, sw13, (E, N, H) = _mx("w13", w13, w13_s, 3)
    pw2, sw2, (E2, H2, I) = _mx("w2", w2, w2_s, 3)
    if (E2, H2, 2 * I) != (E, H, N):
        raise ValueError(f"w13 is {(E, N, H)}, w2 is {(E2, H2, I)}: not [E, 2I, H] and [E, H, I]")
    dtype = x.dtype
    code = _DTYPE.get(dtype)
    if code is None:
        raise ValueError(f"x is {dtype}, not float32, float16 or bfloat16")
    T = x.shape[0] if x.dim() == 2 else 0
    px, pl = _dense("x", x, dtype, T, H), _dense("logits", logits, torch.float32, T, E)
    if out is None:
        out = x.new_empty((T, H))
    if workspace is None:
        workspace = x.new_empty(mxfp4_layer_workspace_bytes(T, top_k, E, H, I), dtype=torch.uint8)
    _run("moe_mxfp4_layer_forward", _device_of(logits, x, w13, w13_s, w2, w2_s, out, workspace), pl,
         px, code, T, E, top_k, pw13, sw13, pw2, sw2, H, I, _dense("out", out, dtype, T, H),
         *_bytes("workspace", workspace))
    return out


def permute_masked_workspace_bytes(T: int, top_k: int, E: int) -> int:
    return int(load_library().moe_permute_masked_workspace_bytes(T, top_k, E))


def moe_permute_masked(topk_ids: torch.Tensor, E: int, first_expert: int = 0,
                       workspace: torch.Tensor | None = None, out: dict | None = None) -> dict:
    """moe_permute for ids that may leave slots out: an id outside [first_expert, first_expert + E)
    drops its slot (slot_rows -1); sorted_slots ends with -1 for each dropped slot.  No tokens
    give empty segments, in buffers given too."""
    if topk_ids.dim() != 2:
        raise ValueError(f"topk_ids has shape {tuple(topk_ids.shape)}, not [T, top_k]")
    T, k = topk_ids.shape
    S = T * k
    if out is None:
        made = topk_ids.new_empty  # int32, or the ids are refused below
        out = {"expert_offsets": made(E + 1), "sorted_slots": made(S), "slot_rows": made(S),
               "active_experts": made(E), "num_active": made(1)}
    if workspace is None:
        need = permute_masked_workspace_bytes(T, k, E)
        if need:
            workspace = topk_ids.new_empty(need, dtype=torch.uint8)
    offsets, slots, rows = out["expert_offsets"], out["sorted_slots"], out["slot_rows"]
    active, count = out["active_experts"], out["num_active"]
    _run("moe_permute_masked", _device_of(topk_ids, offsets, slots, rows, active, count, workspace),
         _dense("topk_ids", topk_ids, torch.int32, T, k), T, k, first_expert, E,
         _dense("expert_offsets", offsets, torch.int32, E + 1),
         _dense("sorted_slots", slots, torch.int32, S), _dense("slot_rows", rows, torch.int32, S),
         _dense("active_experts", active, torch.int32, E),
         _dense("num_active", count, torch.int32, 1), *_bytes("workspace", workspace))
    if T == 0:  # the call writes nothing then
        for t, value in ((offsets, 0), (active, -1), (count, 0)):
            t.fill_(value)
    return out


def _slots(slot_rows: torch.Tensor, top_k: int):
    """(pointer, tokens) of slot_rows [T * top_k]."""
    S = slot_rows.numel()
    if top_k < 1 or S % top_k:
        raise ValueError(f"slot_rows has shape {tuple(slot_rows.shape)}, not [T * {top_k}]")
    return _dense("slot_rows", slot_rows, torch.int32, S), S // top_k


def _weights(topk_weights: torch.Tensor):
    """(pointer, T, top_k) of router weights fp32 [T, top_k]."""
    if topk_weights.dim() != 2:
        raise ValueError(f"topk_weights has shape {tuple(topk_weights.shape)}, not [T, top_k]")
    T, k = topk_weights.shape
    if topk_weights.dtype is not torch.float32 or not topk_weights.is_contiguous():
        raise ValueError(f"topk_weights must be contiguous float32, is {topk_weights.dtype}")
    return topk_weights.data_ptr(), T, k


def moe_dispatch(x: torch.Tensor, slot_rows: torch.Tensor, top_k: int,
                 out: torch.Tensor | None = None) -> torch.Tensor:
    """Token rows to expert order: out[slot_rows[s]] = x[s // top_k].  out has T * top_k rows, or
    any number when given; rows that no slot points at are left as they were (zero when out is
    made here).  No two slots may hold one row."""
    pr, T = _slots(slot_rows, top_k)
    px, dtype, sx, rows_x, H = _matrix("x", x)
    if rows_x != T:
        raise ValueError(f"x has {rows_x} rows, slot_rows {T} tokens")
    if out is None:
        out = x.new_zeros((T * top_k, H))
    rows = out.shape[0] if out.dim() == 2 else 0
    po, _, so = _sized("out", out, rows, H, dtype)
    _apart("out", out, x=x)
    _run("moe_dispatch", _device_of(x, slot_rows, out), px, dtype, T, top_k, H, sx, pr, rows, po, so)
    return out


def moe_dispatch_backward(grad_sorted: torch.Tensor, slot_rows: torch.Tensor, top_k: int,
                          out: torch.Tensor | None = None) -> torch.Tensor:
    """moe_dispatch's gradient: grad_x [T, H], the sum of a token's rows (zeros without one)."""
    pr, T = _slots(slot_rows, top_k)
    pg, dtype, sg, rows, H = _matrix("grad_sorted", grad_sorted)
    if out is None:
        out = grad_sorted.new_empty((T, H))
        po, so = out.data_ptr(), H
    else:
        po, _, so = _sized("out", out, T, H, dtype)
        _apart("out", out, grad_sorted=grad_sorted)
    _run("moe_dispatch_backward", _device_of(grad_sorted, slot_rows, out), pg, dtype, T, top_k, H,
         sg, pr, rows, po, so)
    return out


def moe_combine_masked(y_sorted: torch.Tensor, topk_weights: torch.Tensor, slot_rows: torch.Tensor,
                       dtype: torch.dtype | None = None, out: torch.Tensor | None = None):
    """The router-weighted sum of a token's rows, dropped slots left out: out [T, H] of `dtype`
    (default: y_sorted's)."""
    pw, T, k = _weights(topk_weights)
    py, y_code, sy, rows, H = _matrix("y_sorted", y_sorted)
    if out is None:
        out, po, o_code, so = _made(y_sorted, T, H, dtype or y_sorted.dtype)
    else:
        po, o_code, so = _sized("out", out, T, H)
        _apart("out", out, y_sorted=y_sorted)
    _run("moe_combine_masked", _device_of(y_sorted, topk_weights, slot_rows, out), py, y_code, T, k,
         H, sy, pw, _dense("slot_rows", slot_rows, torch.int32, T * k), rows, po, o_code, so)
    return out


def moe_combine_backward(grad_out: torch.Tensor, y_sorted: torch.Tensor,
                         topk_weights: torch.Tensor, slot_rows: torch.Tensor,
                         out: torch.Tensor | None = None, grad_weights: torch.Tensor | None = None):
    """moe_combine_masked's gradients: (grad_y of y_sorted's type and shape, grad_weights fp32
    [T, top_k]).  Rows of grad_y that no slot points at are left as they were (zero when made here);
    no two slots may hold one row."""
    pw, T, k = _weights(topk_weights)
    py, y_code, sy, rows, H = _matrix("y_sorted", y_sorted)
    pg, g_code, sg = _sized("grad_out", grad_out, T, H)
    if out is None:
        out = y_sorted.new_zeros((rows, H))
    po, _, so = _sized("out", out, rows, H, y_code)
    if grad_weights is None:
        grad_weights = topk_weights.new_empty((T, k))
    _apart("out", out, y_sorted=y_sorted, grad_out=grad_out)
    _run("moe_combine_backward",
         _device_of(grad_out, y_sorted, topk_weights, slot_rows, out, grad_weights), pg, g_code, sg,
         py, y_code, sy, pw, _dense("slot_rows", slot_rows, torch.int32, T * k), T, k, H, rows, po, so,
         _dense("grad_weights", grad_weights, torch.float32, T, k))
    return out, grad_weights
