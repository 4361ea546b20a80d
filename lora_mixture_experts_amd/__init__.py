"""Fused MoE + multi-LoRA layer for AMD Instinct MI355X (gfx950).

Thin ctypes binding over libmoelora.so (include/moelora.h). Every step of the layer runs in
the library's HIP kernels; this module only checks tensor shapes, allocates outputs and the
workspace with torch when the caller does not pass them, and hands raw device pointers and
torch's current HIP stream to the C ABI. For the operators whose kernels take a few microseconds
(route, linear, linear_lora, block_norm, forward_few) a compiled module (csrc/binding.cpp) does the same. There is no fallback: without
the built library or a gfx950 device every call raises.
"""
from __future__ import annotations

import ctypes
import os

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libmoelora.so")

OK, EINVAL_DIMS, ENULL, EALIGN, EWORKSPACE, EHIP, EDEVICE, EUNSUPPORTED, ESCRATCH = 0, -1, -2, -3, -4, -5, -6, -7, -8
FLAG_NONFINITE_LOGIT, FLAG_ADAPTER_RANGE, FLAG_EXPERT_RANGE = 1, 2, 4

EXPORTS = ("moe_lora_workspace_size", "moe_lora_forward", "moe_lora_forward_timed", "moe_lora_forward_fp8",
           "moe_lora_sorted_capacity", "moe_lora_route_align", "moe_lora_strerror",
           "moe_lora_debug_status", "moe_lora_sgmv_workspace_size", "moe_lora_sgmv",
           "moe_lora_router_logits", "moe_lora_forward_routed", "moe_lora_workspace_layout",
           "moe_lora_route", "moe_lora_forward_topk", "moe_lora_linear", "moe_lora_linear_workspace_size",
           "moe_lora_linear_plan", "moe_lora_linear_lora", "moe_lora_linear_lora_workspace_size",
           "moe_lora_linear_lora_plan", "moe_lora_block_norm", "moe_lora_forward_few",
           "moe_lora_few_workspace_size", "moe_lora_forward_noalloc", "moe_lora_probe_read", "moe_lora_probe_mfma")
N_STAGES = 7
STAGES = ("route", "align", "shrink_gate_up", "gate_up", "shrink_down", "down", "combine")


class MoeLoraError(RuntimeError):
    def __init__(self, code: int, what: str):
        super().__init__(f"{what}: {strerror(code)} (code {code})")
        self.code = code


class Dims(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("T", "hidden", "inter", "n_experts", "n_adapters", "rank")]


class LayoutInfo(ctypes.Structure):
    _fields_ = [("tiled", ctypes.c_int32), ("block_m", ctypes.c_int32)] + [
        (n, ctypes.c_int64) for n in ("capacity", "workspace_bytes", "topk_ids", "topk_w", "sorted_pairs",
                                      "expert_offsets", "seg_table", "n_seg", "n_blocks", "block_expert",
                                      "block_seg", "pair_row", "sorted_ad")]


class SgmvDims(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("T", "in_features", "out_features", "n_adapters", "rank")]


class Router(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("T", "n_experts", "topk", "scoring", "n_groups", "topk_groups",
                                              "group_score", "renormalize")] + [
        ("scale", ctypes.c_float), ("logits_stride", ctypes.c_int64)]


class LinearDims(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("T", "in_features", "out_features", "act", "w_type")] + [
        (n, ctypes.c_int64) for n in ("x_stride", "w_stride", "y_stride", "residual_stride")]


class LinearLoraDims(ctypes.Structure):
    _fields_ = [("linear", LinearDims), ("n_adapters", ctypes.c_int32), ("rank", ctypes.c_int32)]


class BlockNormDims(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("T", "hidden", "norm", "gate")] + [
        (n, ctypes.c_float) for n in ("eps", "residual_scale", "branch_scale")] + [
        (n, ctypes.c_int64) for n in ("y_stride", "residual_stride", "gate_stride", "sum_stride", "out_stride")]


class LinearPlanInfo(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("streamed", "tile_rows", "tile_cols", "k_groups", "splits")]


SCORINGS = {"softmax": 0, "sigmoid": 1}
GROUP_SCORES = {"max": 0, "top2": 1}
ACTIVATIONS = {"none": 0, "relu": 1, "silu": 2, "gelu": 3, "gelu_tanh": 4, "swiglu": 5}

NORMS = {"rms": 0, "layer": 1}

_lib = None
_compiled = None


def lib() -> ctypes.CDLL:
    """The loaded library (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with lora_mixture_experts_amd.build.build()")
        L = ctypes.CDLL(LIB_PATH)
        P, i32, i64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64
        D = ctypes.POINTER(Dims)
        L.moe_lora_workspace_size.argtypes = [D, i32]
        L.moe_lora_workspace_size.restype = ctypes.c_size_t
        L.moe_lora_forward.argtypes = [P, P, P, P, P, P, P, P, P, i32, D, P, P, ctypes.c_size_t, P]
        L.moe_lora_forward.restype = ctypes.c_int
        L.moe_lora_forward_timed.argtypes = [P, P, P, P, P, P, P, P, P, i32, D, P, P, ctypes.c_size_t, P,
                                             ctypes.POINTER(ctypes.c_void_p)]
        L.moe_lora_forward_timed.restype = ctypes.c_int
        L.moe_lora_forward_fp8.argtypes = [P, P, P, P, P, P, P, P, P, P, P, i32, D, P, P, ctypes.c_size_t, P,
                                           ctypes.POINTER(ctypes.c_void_p)]
        L.moe_lora_forward_fp8.restype = ctypes.c_int
        L.moe_lora_probe_read.argtypes = [P, ctypes.c_size_t, P, P]
        L.moe_lora_probe_read.restype = ctypes.c_int
        L.moe_lora_probe_mfma.argtypes = [i32, i32, P, P]
        L.moe_lora_probe_mfma.restype = ctypes.c_int
        L.moe_lora_forward_noalloc.argtypes = [P, P, P, P, P, P, P, P, P, i32, D, P, P]
        L.moe_lora_forward_noalloc.restype = ctypes.c_int
        L.moe_lora_router_logits.argtypes = [P, P, i32, i32, i32, P, P]
        L.moe_lora_router_logits.restype = ctypes.c_int
        L.moe_lora_forward_routed.argtypes = [P, P, P, P, P, P, P, P, P, i32, D, P, P, ctypes.c_size_t, P]
        L.moe_lora_forward_routed.restype = ctypes.c_int
        L.moe_lora_sgmv_workspace_size.argtypes = [ctypes.POINTER(SgmvDims)]
        L.moe_lora_sgmv_workspace_size.restype = ctypes.c_size_t
        L.moe_lora_sgmv.argtypes = [P, P, P, P, ctypes.POINTER(SgmvDims), P, P, ctypes.c_size_t, P]
        L.moe_lora_sgmv.restype = ctypes.c_int
        L.moe_lora_sorted_capacity.argtypes = [D, i32, i32, i32]
        L.moe_lora_sorted_capacity.restype = i64
        L.moe_lora_route_align.argtypes = [P, P, i32, D, i32, i32, P, P, P, i64, P, P, P, P,
                                           ctypes.c_size_t, P]
        L.moe_lora_route_align.restype = ctypes.c_int
        L.moe_lora_workspace_layout.argtypes = [D, i32, ctypes.POINTER(LayoutInfo)]
        L.moe_lora_workspace_layout.restype = ctypes.c_int
        L.moe_lora_route.argtypes = [P, P, P, ctypes.POINTER(Router), P, P, P, P]
        L.moe_lora_route.restype = ctypes.c_int
        L.moe_lora_forward_topk.argtypes = [P, P, P, P, P, P, P, P, P, P, P, P, i32, D, P, P, ctypes.c_size_t, P]
        L.moe_lora_forward_topk.restype = ctypes.c_int
        L.moe_lora_linear_workspace_size.argtypes = [ctypes.POINTER(LinearDims)]
        L.moe_lora_linear_workspace_size.restype = ctypes.c_size_t
        L.moe_lora_linear_plan.argtypes = [ctypes.POINTER(LinearDims), ctypes.POINTER(LinearPlanInfo)]
        L.moe_lora_linear_plan.restype = ctypes.c_int
        L.moe_lora_linear.argtypes = [P, P, P, P, P, ctypes.POINTER(LinearDims), P, P, ctypes.c_size_t, P]
        L.moe_lora_linear.restype = ctypes.c_int
        L.moe_lora_linear_lora_workspace_size.argtypes = [ctypes.POINTER(LinearLoraDims)]
        L.moe_lora_linear_lora_workspace_size.restype = ctypes.c_size_t
        L.moe_lora_linear_lora_plan.argtypes = [ctypes.POINTER(LinearLoraDims), ctypes.POINTER(LinearPlanInfo)]
        L.moe_lora_linear_lora_plan.restype = ctypes.c_int
        L.moe_lora_linear_lora.argtypes = [P, P, P, P, P, P, P, P, ctypes.POINTER(LinearLoraDims), P, P,
                                           ctypes.c_size_t, P]
        L.moe_lora_linear_lora.restype = ctypes.c_int
        L.moe_lora_block_norm.argtypes = [P, P, P, P, P, P, P, ctypes.POINTER(BlockNormDims), P, P, P]
        L.moe_lora_block_norm.restype = ctypes.c_int
        L.moe_lora_few_workspace_size.argtypes = [D, i32]
        L.moe_lora_few_workspace_size.restype = ctypes.c_size_t
        L.moe_lora_forward_few.argtypes = [P, P, P, P, P, P, P, P, P, P, P, P, P, i32, D, P, P, ctypes.c_size_t, P]
        L.moe_lora_forward_few.restype = ctypes.c_int
        L.moe_lora_strerror.argtypes = [ctypes.c_int]
        L.moe_lora_strerror.restype = ctypes.c_char_p
        L.moe_lora_debug_status.argtypes = [P, ctypes.c_size_t, P, ctypes.POINTER(ctypes.c_uint32)]
        L.moe_lora_debug_status.restype = ctypes.c_int
        _lib = L
    return _lib


def _native():
    """The compiled half of the binding (raises if it has not been built)."""
    global _compiled
    if _compiled is None:
        lib()  # (its message, if the library is missing)
        try:
            from . import _binding
        except ImportError as e:
            raise RuntimeError(f"_binding.so is missing or does not load ({e}): build it with "
                               "lora_mixture_experts_amd.build.build()") from e
        _compiled = _binding
    return _compiled


def strerror(code: int) -> str:
    return lib().moe_lora_strerror(code).decode()


def _check(code: int, what: str):
    if code != OK:
        raise MoeLoraError(code, what)


def dims_of(x: torch.Tensor, W1: torch.Tensor, A1: torch.Tensor) -> Dims:
    T, h = x.shape
    E, twoI, _ = W1.shape
    nA, _, r, _ = A1.shape
    return Dims(T, h, twoI // 2, E, nA, r)


def workspace_size(d: Dims, topk: int) -> int:
    return int(lib().moe_lora_workspace_size(ctypes.byref(d), topk))


def sorted_capacity(d: Dims, topk: int, seg_pad: int, block_m: int) -> int:
    return int(lib().moe_lora_sorted_capacity(ctypes.byref(d), topk, seg_pad, block_m))


def new_workspace(d: Dims, topk: int, device) -> torch.Tensor:
    n = workspace_size(d, topk)
    if n == 0:
        raise MoeLoraError(EINVAL_DIMS, "workspace_size")
    return torch.empty(n, dtype=torch.uint8, device=device)


def workspace_layout(d: Dims, topk: int) -> dict:
    """Where the forward keeps its sorted layout in the workspace (moe_lora_workspace_layout)."""
    info = LayoutInfo()
    _check(lib().moe_lora_workspace_layout(ctypes.byref(d), topk, ctypes.byref(info)),
           "moe_lora_workspace_layout")
    return {name: getattr(info, name) for name, _ in LayoutInfo._fields_}


def read_layout_tables(workspace: torch.Tensor, d: Dims, topk: int) -> dict:
    """The forward's routing and sorted-layout tables, copied to the host from the workspace of
    the last call that used it (int32 numpy arrays; topk_w float32). Synchronises."""
    info = workspace_layout(d, topk)
    host = workspace.cpu()
    P = d.T * topk

    def region(name, n, dtype=torch.int32):
        off = info[name]
        return host[off:off + 4 * n].view(dtype).numpy()

    n_blocks = int(region("n_blocks", 1)[0])
    n_seg = int(region("n_seg", 1)[0])
    total = n_blocks * info["block_m"]
    return {
        "info": info, "n_blocks": n_blocks, "n_seg": n_seg,
        "topk_ids": region("topk_ids", P).reshape(d.T, topk),
        "topk_w": region("topk_w", P, torch.float32).reshape(d.T, topk),
        "sorted_pairs": region("sorted_pairs", total),
        "expert_offsets": region("expert_offsets", d.n_experts + 1),
        "seg_table": region("seg_table", 4 * n_seg).reshape(n_seg, 4),
        "block_expert": region("block_expert", n_blocks),
        "block_seg": region("block_seg", n_blocks),
        "pair_row": region("pair_row", P),
        "sorted_ad": region("sorted_ad", total),
    }


def _ptr(t) -> int | None:
    return None if t is None else t.data_ptr()


def _stream(device) -> int:
    return torch.cuda.current_stream(device).cuda_stream


def _expect(t: torch.Tensor, name: str, dtype, shape):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if t.device.type != "cuda":
        raise ValueError(f"{name} must be on a GPU")


def forward(x, router_logits, W1, W2, A1, B1, A2, B2, adapter_ids, topk: int, y=None,
            workspace=None, stage_events=None) -> torch.Tensor:
    """y[T][h] (bf16) of the fused MoE + multi-LoRA layer; see include/moelora.h.

    stage_events: optional list of N_STAGES + 1 torch.cuda.Event(enable_timing=True) (or None
    for a boundary not to record) that the library records at the stage boundaries on the
    current stream (moe_lora_forward_timed)."""
    d = dims_of(x, W1, A1)
    T, h, I, E, nA, r = d.T, d.hidden, d.inter, d.n_experts, d.n_adapters, d.rank
    bf = torch.bfloat16
    _expect(x, "x", bf, (T, h))
    _expect(router_logits, "router_logits", torch.float32, (T, E))
    _expect(W1, "W1", bf, (E, 2 * I, h))
    _expect(W2, "W2", bf, (E, h, I))
    _expect(A1, "A1", bf, (nA, E, r, h))
    _expect(B1, "B1", bf, (nA, E, 2 * I, r))
    _expect(A2, "A2", bf, (nA, E, r, I))
    _expect(B2, "B2", bf, (nA, E, h, r))
    _expect(adapter_ids, "adapter_ids", torch.int32, (T,))
    if y is None:
        y = torch.empty((T, h), dtype=bf, device=x.device)
    _expect(y, "y", bf, (T, h))
    if workspace is None:
        workspace = new_workspace(d, topk, x.device)
    args = (_ptr(x), _ptr(router_logits), _ptr(W1), _ptr(W2), _ptr(A1), _ptr(B1), _ptr(A2), _ptr(B2),
            _ptr(adapter_ids), topk, ctypes.byref(d), _ptr(y), _ptr(workspace), workspace.numel(),
            _stream(x.device))
    if stage_events is None:
        _check(lib().moe_lora_forward(*args), "moe_lora_forward")
    else:
        if len(stage_events) != N_STAGES + 1:
            raise ValueError(f"need {N_STAGES + 1} events")
        for ev in stage_events:
            if ev is not None and not ev.cuda_event:  # torch creates the HIP event on its first record
                ev.record()
        handles = (ctypes.c_void_p * (N_STAGES + 1))(
            *[ev.cuda_event if ev is not None else None for ev in stage_events])
        _check(lib().moe_lora_forward_timed(*args, handles), "moe_lora_forward_timed")
    return y


def forward_noalloc(x, router_logits, W1, W2, A1, B1, A2, B2, adapter_ids, topk: int,
                    y=None) -> torch.Tensor:
    """forward without a workspace argument (moe_lora_forward_noalloc): the library uses its
    static 128 MiB device scratch. Raises MoeLoraError(ESCRATCH) when the sizes need more.
    Calls on one GPU share that scratch and must be ordered on one stream."""
    d = dims_of(x, W1, A1)
    T, h, I, E, nA, r = d.T, d.hidden, d.inter, d.n_experts, d.n_adapters, d.rank
    bf = torch.bfloat16
    _expect(x, "x", bf, (T, h))
    _expect(router_logits, "router_logits", torch.float32, (T, E))
    _expect(W1, "W1", bf, (E, 2 * I, h))
    _expect(W2, "W2", bf, (E, h, I))
    _expect(A1, "A1", bf, (nA, E, r, h))
    _expect(B1, "B1", bf, (nA, E, 2 * I, r))
    _expect(A2, "A2", bf, (nA, E, r, I))
    _expect(B2, "B2", bf, (nA, E, h, r))
    _expect(adapter_ids, "adapter_ids", torch.int32, (T,))
    if y is None:
        y = torch.empty((T, h), dtype=bf, device=x.device)
    _expect(y, "y", bf, (T, h))
    _check(lib().moe_lora_forward_noalloc(_ptr(x), _ptr(router_logits), _ptr(W1), _ptr(W2), _ptr(A1),
                                          _ptr(B1), _ptr(A2), _ptr(B2), _ptr(adapter_ids), topk,
                                          ctypes.byref(d), _ptr(y), _stream(x.device)),
           "moe_lora_forward_noalloc")
    return y


def router_logits(x, W_router, out=None) -> torch.Tensor:
    """logits [T][E] float32 = x W_router^T (moe_lora_router_logits), into `out` if given."""
    T, h = x.shape
    E = W_router.shape[0]
    _expect(x, "x", torch.bfloat16, (T, h))
    _expect(W_router, "W_router", torch.bfloat16, (E, h))
    if out is None:
        out = torch.empty((T, E), dtype=torch.float32, device=x.device)
    _expect(out, "out", torch.float32, (T, E))
    _check(lib().moe_lora_router_logits(_ptr(x), _ptr(W_router), T, h, E, _ptr(out), _stream(x.device)),
           "moe_lora_router_logits")
    return out


def forward_routed(x, W_router, W1, W2, A1, B1, A2, B2, adapter_ids, topk: int, y=None,
                   workspace=None) -> torch.Tensor:
    """forward starting from the router weights W_router [E][h] (moe_lora_forward_routed)."""
    d = dims_of(x, W1, A1)
    T, h, I, E, nA, r = d.T, d.hidden, d.inter, d.n_experts, d.n_adapters, d.rank
    bf = torch.bfloat16
    _expect(x, "x", bf, (T, h))
    _expect(W_router, "W_router", bf, (E, h))
    _expect(W1, "W1", bf, (E, 2 * I, h))
    _expect(W2, "W2", bf, (E, h, I))
    _expect(A1, "A1", bf, (nA, E, r, h))
    _expect(B1, "B1", bf, (nA, E, 2 * I, r))
    _expect(A2, "A2", bf, (nA, E, r, I))
    _expect(B2, "B2", bf, (nA, E, h, r))
    _expect(adapter_ids, "adapter_ids", torch.int32, (T,))
    if y is None:
        y = torch.empty((T, h), dtype=bf, device=x.device)
    _expect(y, "y", bf, (T, h))
    if workspace is None:
        workspace = new_workspace(d, topk, x.device)
    _check(lib().moe_lora_forward_routed(_ptr(x), _ptr(W_router), _ptr(W1), _ptr(W2), _ptr(A1), _ptr(B1),
                                         _ptr(A2), _ptr(B2), _ptr(adapter_ids), topk, ctypes.byref(d),
                                         _ptr(y), _ptr(workspace), workspace.numel(), _stream(x.device)),
           "moe_lora_forward_routed")
    return y


def sgmv(x, A, B, adapter_ids, y, workspace=None) -> torch.Tensor:
    """Dense multi-LoRA, in place: y[t] += (x[t] A[a]^T) B[a]^T for a = adapter_ids[t] (-1: y[t]
    unchanged); moe_lora_sgmv. x [T][K], A [nA][r][K], B [nA][N][r], y [T][N] bf16,
    adapter_ids [T] int32."""
    T, K = x.shape
    nA, r, _ = A.shape
    N = B.shape[1]
    d = SgmvDims(T, K, N, nA, r)
    bf = torch.bfloat16
    _expect(x, "x", bf, (T, K))
    _expect(A, "A", bf, (nA, r, K))
    _expect(B, "B", bf, (nA, N, r))
    _expect(adapter_ids, "adapter_ids", torch.int32, (T,))
    _expect(y, "y", bf, (T, N))
    if workspace is None:
        n = int(lib().moe_lora_sgmv_workspace_size(ctypes.byref(d)))
        if n == 0:
            raise MoeLoraError(EINVAL_DIMS, "moe_lora_sgmv_workspace_size")
        workspace = torch.empty(n, dtype=torch.uint8, device=x.device)
    _check(lib().moe_lora_sgmv(_ptr(x), _ptr(A), _ptr(B), _ptr(adapter_ids), ctypes.byref(d), _ptr(y),
                               _ptr(workspace), workspace.numel(), _stream(x.device)), "moe_lora_sgmv")
    return y


def _dense(t, name: str, dtype, shape, device: int):
    """Pointer of a contiguous tensor on GPU `device`, None for None."""
    if t is None:
        return None
    _expect(t, name, dtype, shape)
    if t.get_device() != device:
        raise ValueError(f"{name} is on cuda:{t.get_device()}, expected cuda:{device}")
    return t.data_ptr()


def _on(device: int, call, what: str, *args):
    """call(*args, stream) with GPU `device` current, on torch's current stream of it."""
    if torch.cuda.current_device() == device:
        rc = call(*args, torch._C._cuda_getCurrentRawStream(device))
    else:
        with torch.cuda.device(device):
            rc = call(*args, torch._C._cuda_getCurrentRawStream(device))
    if rc != OK:
        raise MoeLoraError(rc, what)


def route(logits, topk: int, *, scoring: str = "softmax", bias=None, n_groups: int = 1, topk_groups: int = 1,
          group_score: str = "max", renormalize: bool = True, scale: float = 1.0, token_mask=None,
          topk_ids=None, topk_w=None, token_flags=None):
    """Expert choice of a router (moe_lora_route): (topk_ids [T][topk] int32, topk_w [T][topk]
    float32) of logits [T][E] float32 (rows may lie apart), the arguments of forward_topk.

    scoring: "softmax" over the experts or "sigmoid"; bias [E] float32 steers the choice only;
    n_groups, topk_groups, group_score ("max" or "top2"): only the best groups' experts are
    chosen from; renormalize: weights over the sum of the chosen; token_mask [T] bool: False for
    rows of padding. Empty slots hold expert -1 and weight 0. token_flags [T] int32, when given,
    receives 1 where a token's logits were not all finite. An output that shares a byte with another
    argument is refused."""
    if scoring not in SCORINGS:
        raise ValueError(f"scoring must be one of {sorted(SCORINGS)}")
    if group_score not in GROUP_SCORES:
        raise ValueError(f"group_score must be one of {sorted(GROUP_SCORES)}")
    out = (_compiled or _native()).route(logits, topk, SCORINGS[scoring], bias, n_groups, topk_groups,
                                         GROUP_SCORES[group_score], 1 if renormalize else 0, scale, token_mask,
                                         topk_ids, topk_w, token_flags)
    if type(out) is int:
        raise MoeLoraError(out, "moe_lora_route")
    return out


def forward_topk(x, topk_ids, topk_w, W1, W2, A1, B1, A2, B2, adapter_ids, *, W1_scale=None, W2_scale=None,
                 y=None, workspace=None) -> torch.Tensor:
    """forward with the tokens' experts and weights given (moe_lora_forward_topk): topk_ids [T][k]
    int32 (-1: an empty slot) and topk_w [T][k] float32, as route returns them. With W1_scale
    [E][2I] and W2_scale [E][h] (float32), W1 and W2 are uint8 E4M3 codes as in forward_fp8."""
    d = dims_of(x, W1, A1)
    T, h, I, E, nA, r = d.T, d.hidden, d.inter, d.n_experts, d.n_adapters, d.rank
    if not isinstance(topk_ids, torch.Tensor) or topk_ids.dim() != 2:
        raise ValueError("topk_ids must be a [T][k] tensor")
    if (W1_scale is None) != (W2_scale is None):
        raise ValueError("W1_scale and W2_scale go together")
    k = topk_ids.shape[1]
    dev, bf = x.get_device(), torch.bfloat16
    wt = bf if W1_scale is None else torch.uint8
    if y is None:
        y = torch.empty((T, h), dtype=bf, device=x.device)
    args = (_dense(x, "x", bf, (T, h), dev), _dense(topk_ids, "topk_ids", torch.int32, (T, k), dev),
            _dense(topk_w, "topk_w", torch.float32, (T, k), dev), _dense(W1, "W1", wt, (E, 2 * I, h), dev),
            _dense(W1_scale, "W1_scale", torch.float32, (E, 2 * I), dev), _dense(W2, "W2", wt, (E, h, I), dev),
            _dense(W2_scale, "W2_scale", torch.float32, (E, h), dev), _dense(A1, "A1", bf, (nA, E, r, h), dev),
            _dense(B1, "B1", bf, (nA, E, 2 * I, r), dev), _dense(A2, "A2", bf, (nA, E, r, I), dev),
            _dense(B2, "B2", bf, (nA, E, h, r), dev), _dense(adapter_ids, "adapter_ids", torch.int32, (T,), dev))
    if workspace is None:
        workspace = new_workspace(d, k, x.device)
    _on(dev, lib().moe_lora_forward_topk, "moe_lora_forward_topk", *args, k, ctypes.byref(d),
        _dense(y, "y", bf, (T, h), dev), _dense(workspace, "workspace", torch.uint8, workspace.shape, dev),
        workspace.numel())
    return y


def linear_plan(T: int, in_features: int, out_features: int, act: str = "none", e4m3: bool = False) -> dict:
    """Kernel, tile and splits that linear takes for these sizes (moe_lora_linear_plan), host-only."""
    if act not in ACTIVATIONS:
        raise ValueError(f"act must be one of {sorted(ACTIVATIONS)}")
    d = LinearDims(T, in_features, out_features, ACTIVATIONS[act], 1 if e4m3 else 0, in_features, in_features,
                   out_features, out_features)
    out = LinearPlanInfo()
    _check(lib().moe_lora_linear_plan(ctypes.byref(d), ctypes.byref(out)), "moe_lora_linear_plan")
    return {n: getattr(out, n) for n, _ in LinearPlanInfo._fields_}


def linear(x, W, *, w_scale=None, bias=None, act: str = "none", residual=None, y=None,
           workspace=None) -> torch.Tensor:
    """Dense projection y = act(x W^T + bias) + residual (moe_lora_linear), bf16 [T][N].

    x [T][K] bf16; W [N][K] bf16, or uint8 E4M3 codes with w_scale [N] float32; bias [N] and
    residual [T][N] bf16. act: "none", "relu", "silu", "gelu", "gelu_tanh", or "swiglu", for which
    W (w_scale, bias) has 2 N rows, gate then up. Rows of x, W, residual and y may lie apart (x
    and W rows 16-byte aligned). y may be the residual; a y or a workspace in use that shares a byte
    with another argument is refused.
    sgmv(x, A, B, adapter_ids, y) adds a batch's adapters to a projection without an activation,
    linear_lora takes them inside the epilogue."""
    if act not in ACTIVATIONS:
        raise ValueError(f"act must be one of {sorted(ACTIVATIONS)}")
    out = (_compiled or _native()).linear(x, W, w_scale, bias, ACTIVATIONS[act], residual, y, workspace)
    if type(out) is int:
        raise MoeLoraError(out, "moe_lora_linear")
    return out


def linear_lora(x, W, A, B, adapter_ids, *, w_scale=None, bias=None, act: str = "none", residual=None, y=None,
                workspace=None) -> torch.Tensor:
    """Dense projection with a batch's adapters inside its epilogue (moe_lora_linear_lora), bf16 [T][N]:
    y[t] = act(x[t] W^T + (x[t] A_a^T) B_a^T + bias) + residual[t], a = adapter_ids[t] (-1: none).

    A [nA][r][K] and B [nA][rows of W][r] bf16, contiguous, rank r 8, 16, 32 or 64; adapter_ids [T]
    int32. The rest as in linear. debug_status(workspace) of a workspace given here tells of adapter ids
    out of range."""
    if act not in ACTIVATIONS:
        raise ValueError(f"act must be one of {sorted(ACTIVATIONS)}")
    out = (_compiled or _native()).linear_lora(x, W, w_scale, bias, ACTIVATIONS[act], residual, y, workspace, A, B,
                                               adapter_ids)
    if type(out) is int:
        raise MoeLoraError(out, "moe_lora_linear_lora")
    return out


def linear_lora_plan(T: int, in_features: int, out_features: int, n_adapters: int, rank: int, act: str = "none",
                     e4m3: bool = False) -> dict:
    """linear_plan for linear_lora (moe_lora_linear_lora_plan), host-only."""
    if act not in ACTIVATIONS:
        raise ValueError(f"act must be one of {sorted(ACTIVATIONS)}")
    d = LinearLoraDims(LinearDims(T, in_features, out_features, ACTIVATIONS[act], 1 if e4m3 else 0, in_features,
                                  in_features, out_features, out_features), n_adapters, rank)
    out = LinearPlanInfo()
    _check(lib().moe_lora_linear_lora_plan(ctypes.byref(d), ctypes.byref(out)), "moe_lora_linear_lora_plan")
    return {n: getattr(out, n) for n, _ in LinearPlanInfo._fields_}


def block_norm(y, residual, weight=None, *, bias=None, post_weight=None, post_bias=None, gate=None,
               sigmoid_gate: bool = False, residual_scale: float = 1.0, branch_scale: float = 1.0,
               norm: str = "rms", eps: float = 1e-6, total=None, out=None):
    """The norms around a block (moe_lora_block_norm): (total, out), bf16 [T][h], of what the block gave,
    y [T][h], and the residual stream [T][h] (bf16, rows may lie apart):
    total = residual_scale * residual + branch_scale * gate * b, b = y or, with post_weight [h], its norm;
    out = the norm of total (before its rounding) with weight [h].

    norm: "rms" or "layer", both with an optional bias [h]; gate: None, [T] float32 (through a sigmoid with
    sigmoid_gate, which no gate of features takes) or [T][h] bf16 (an expanded row is read as one). Without
    weight out is None; with y None total is residual_scale * residual and only written where it is given.
    total and out may be y or the residual; an output that shares other bytes with an argument is refused."""
    if norm not in NORMS:
        raise ValueError(f"norm must be one of {sorted(NORMS)}")
    pair = (_compiled or _native()).block_norm(y, residual, gate, 1 if sigmoid_gate else 0, post_weight, post_bias,
                                               weight, bias, NORMS[norm], eps, residual_scale, branch_scale, total,
                                               out)
    if type(pair) is int:
        raise MoeLoraError(pair, "moe_lora_block_norm")
    return pair


FEW_TOKENS = 16  # the most that forward_few takes


def forward_few(x, W1, W2, A1, B1, A2, B2, adapter_ids, *, router_logits=None, topk=None, topk_ids=None, topk_w=None,
                W1_scale=None, W2_scale=None, y=None, workspace=None) -> torch.Tensor:
    """The layer for up to 16 tokens in three launches (moe_lora_forward_few): forward's function with
    router_logits [T][E] float32 and topk, forward_topk's with topk_ids [T][k] int32 (-1: an empty slot) and
    topk_w [T][k] float32. With W1_scale [E][2I] and W2_scale [E][h] (float32), W1 and W2 are uint8 E4M3
    codes as in forward_fp8. debug_status(workspace) of a workspace given here tells of logits that were not
    finite and of ids out of range."""
    out = (_compiled or _native()).forward_few(x, W1, W2, A1, B1, A2, B2, adapter_ids, router_logits, topk, topk_ids,
                                               topk_w, W1_scale, W2_scale, y, workspace)
    if type(out) is int:
        raise MoeLoraError(out, "moe_lora_forward_few")
    return out


def forward_fp8(x, router_logits, W1q, W1_scale, W2q, W2_scale, A1, B1, A2, B2, adapter_ids,
                topk: int, y=None, workspace=None, stage_events=None) -> torch.Tensor:
    """forward with E4M3 expert weights (moe_lora_forward_fp8): W1q [E][2I][h] and W2q [E][h][I]
    as uint8 codes, W1_scale [E][2I] and W2_scale [E][h] float32 per-row scales; the rest as
    in forward."""
    T, h = x.shape
    E, twoI, _ = W1q.shape
    nA, _, r, _ = A1.shape
    I = twoI // 2
    d = Dims(T, h, I, E, nA, r)
    bf = torch.bfloat16
    _expect(x, "x", bf, (T, h))
    _expect(router_logits, "router_logits", torch.float32, (T, E))
    _expect(W1q, "W1q", torch.uint8, (E, 2 * I, h))
    _expect(W1_scale, "W1_scale", torch.float32, (E, 2 * I))
    _expect(W2q, "W2q", torch.uint8, (E, h, I))
    _expect(W2_scale, "W2_scale", torch.float32, (E, h))
    _expect(A1, "A1", bf, (nA, E, r, h))
    _expect(B1, "B1", bf, (nA, E, 2 * I, r))
    _expect(A2, "A2", bf, (nA, E, r, I))
    _expect(B2, "B2", bf, (nA, E, h, r))
    _expect(adapter_ids, "adapter_ids", torch.int32, (T,))
    if y is None:
        y = torch.empty((T, h), dtype=bf, device=x.device)
    _expect(y, "y", bf, (T, h))
    if workspace is None:
        workspace = new_workspace(d, topk, x.device)
    handles = None
    if stage_events is not None:
        if len(stage_events) != N_STAGES + 1:
            raise ValueError(f"need {N_STAGES + 1} events")
        for ev in stage_events:
            if ev is not None and not ev.cuda_event:
                ev.record()
        handles = (ctypes.c_void_p * (N_STAGES + 1))(
            *[ev.cuda_event if ev is not None else None for ev in stage_events])
    _check(lib().moe_lora_forward_fp8(_ptr(x), _ptr(router_logits), _ptr(W1q), _ptr(W1_scale),
                                      _ptr(W2q), _ptr(W2_scale), _ptr(A1), _ptr(B1), _ptr(A2),
                                      _ptr(B2), _ptr(adapter_ids), topk, ctypes.byref(d), _ptr(y),
                                      _ptr(workspace), workspace.numel(), _stream(x.device), handles),
           "moe_lora_forward_fp8")
    return y


def route_align(router_logits, adapter_ids, topk: int, d: Dims, seg_pad: int = 1, block_m: int = 1,
                workspace=None) -> dict:
    """Routing and align outputs as device tensors; see moe_lora_route_align."""
    dev = router_logits.device
    _expect(router_logits, "router_logits", torch.float32, (d.T, d.n_experts))
    _expect(adapter_ids, "adapter_ids", torch.int32, (d.T,))
    cap = sorted_capacity(d, topk, seg_pad, block_m)
    if cap < 0:
        raise MoeLoraError(EINVAL_DIMS, "sorted_capacity")
    P = d.T * topk
    out = {
        "topk_ids": torch.empty((d.T, topk), dtype=torch.int32, device=dev),
        "topk_w": torch.empty((d.T, topk), dtype=torch.float32, device=dev),
        "sorted_pairs": torch.full((max(cap, 1),), -7, dtype=torch.int32, device=dev),
        "expert_offsets": torch.empty(d.n_experts + 1, dtype=torch.int32, device=dev),
        "seg_table": torch.empty((max(P, 1), 4), dtype=torch.int32, device=dev),
        "n_seg": torch.empty(1, dtype=torch.int32, device=dev),
    }
    if workspace is None:
        workspace = new_workspace(d, topk, dev)
    rc = lib().moe_lora_route_align(_ptr(router_logits), _ptr(adapter_ids), topk, ctypes.byref(d),
                                    seg_pad, block_m, _ptr(out["topk_ids"]), _ptr(out["topk_w"]),
                                    _ptr(out["sorted_pairs"]), cap, _ptr(out["expert_offsets"]),
                                    _ptr(out["seg_table"]), _ptr(out["n_seg"]), _ptr(workspace),
                                    workspace.numel(), _stream(dev))
    _check(rc, "moe_lora_route_align")
    out["workspace"] = workspace
    return out


PROBE_READ_SINK = 2048 * 256  # uint32 words the read probe writes


def probe_read(src: torch.Tensor, sink: torch.Tensor):
    """Streaming read of src's bytes (moe_lora_probe_read) on the current stream."""
    _check(lib().moe_lora_probe_read(_ptr(src), src.numel() * src.element_size(), _ptr(sink),
                                     _stream(src.device)), "moe_lora_probe_read")


def probe_mfma(iters: int, n_workgroups: int, sink: torch.Tensor) -> int:
    """Loop of bf16 MFMAs (moe_lora_probe_mfma) on the current stream; returns its flops."""
    _check(lib().moe_lora_probe_mfma(iters, n_workgroups, _ptr(sink), _stream(sink.device)),
           "moe_lora_probe_mfma")
    return n_workgroups * 4 * iters * 8 * 32768


def debug_status(workspace: torch.Tensor) -> int:
    """Device flags (FLAG_* bits) of the last call that used `workspace`; synchronises."""
    flags = ctypes.c_uint32(0)
    rc = lib().moe_lora_debug_status(_ptr(workspace), workspace.numel(), _stream(workspace.device),
                                     ctypes.byref(flags))
    _check(rc, "moe_lora_debug_status")
    return int(flags.value)
