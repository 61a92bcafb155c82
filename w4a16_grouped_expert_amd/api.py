"""Thin torch-facing binding of the C ABI (same names as the entry points).

PyTorch provides device memory and streams; every step of the layer runs in the
HIP library.  Functions check dtypes, devices and shapes, marshal pointers and
raise MoeError on a non-zero status.  The ``*_into`` forms write into
caller-provided buffers and allocate nothing, for use in timed loops and graphs.
"""
from __future__ import annotations

import ctypes
from dataclasses import dataclass
from typing import Optional

import torch

from . import _lib
from ._lib import check, lib

MODE_AUTO, MODE_DECODE, MODE_PREFILL = 0, 1, 2
GROUP = 128


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream=None):
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _need(t, dtype, name, device=True):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if device and not t.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor")


def expert_layout(d: int, I: int) -> dict:
    lay = _lib.ExpertLayout()
    check("moe_expert_layout_get", lib().moe_expert_layout_get(d, I, ctypes.byref(lay)))
    return {f: getattr(lay, f) for f, _ in _lib.ExpertLayout._fields_}


# ---------------------------------------------------------------- pack

def pack_w4_g128(w: torch.Tensor, gateup_interleave: bool, codes: torch.Tensor, codes_stride: int,
                 scales: torch.Tensor, scales_stride: int, codes_offset: int = 0, scales_offset: int = 0,
                 stream=None):
    """Quantise + pack bf16 w [E, N, K] into codes/scales (uint8 device buffers, byte strides/offsets)."""
    _need(w, torch.bfloat16, "w")
    _need(codes, torch.uint8, "codes")
    _need(scales, torch.uint8, "scales")
    E, N, K = w.shape
    check("pack_w4_g128", lib().pack_w4_g128(
        _ptr(w), E, N, K, int(bool(gateup_interleave)),
        ctypes.c_void_p(codes.data_ptr() + codes_offset), codes_stride,
        ctypes.c_void_p(scales.data_ptr() + scales_offset), scales_stride, _stream(stream)))


def pack_experts(w13: torch.Tensor, w2: torch.Tensor, bank: Optional[torch.Tensor] = None, stream=None):
    """Quantise + pack experts into a bank of blobs: w13 [E, 2I, d], w2 [E, d, I] (bf16, GPU).

    Returns (bank uint8 [E, blob_bytes], layout dict).  Packing may be split over
    calls by passing slices of the expert axis and the matching bank rows.
    """
    E, twoI, d = w13.shape
    I = twoI // 2
    lay = expert_layout(d, I)
    if bank is None:
        bank = torch.empty((E, lay["blob_bytes"]), dtype=torch.uint8, device=w13.device)
    stride = bank.stride(0)
    pack_w4_g128(w13, True, bank, stride, bank, stride, lay["w13_codes"], lay["w13_scales"], stream)
    pack_w4_g128(w2, False, bank, stride, bank, stride, lay["w2_codes"], lay["w2_scales"], stream)
    return bank, lay


# ---------------------------------------------------------------- route

@dataclass
class RouteOut:
    logits: torch.Tensor   # [T, E] fp32
    ids: torch.Tensor      # [T, k] int32
    weights: torch.Tensor  # [T, k] fp32


def alloc_route(T: int, E: int, k: int, device) -> RouteOut:
    return RouteOut(torch.empty((T, E), dtype=torch.float32, device=device),
                    torch.empty((T, k), dtype=torch.int32, device=device),
                    torch.empty((T, k), dtype=torch.float32, device=device))


def moe_route_into(x, w_router, k, out: RouteOut, renormalize=True, stream=None) -> RouteOut:
    _need(x, torch.bfloat16, "x")
    _need(w_router, torch.bfloat16, "w_router")
    T, d = x.shape
    E = w_router.shape[0]
    check("moe_route", lib().moe_route(_ptr(x), _ptr(w_router), T, d, E, k, int(bool(renormalize)),
                                       _ptr(out.logits), _ptr(out.ids), _ptr(out.weights), _stream(stream)))
    return out


def moe_route(x, w_router, k, renormalize=True, stream=None) -> RouteOut:
    return moe_route_into(x, w_router, k, alloc_route(x.shape[0], w_router.shape[0], k, x.device),
                          renormalize, stream)


# ---------------------------------------------------------------- align

@dataclass
class AlignOut:
    offsets: torch.Tensor        # [E+1]
    sorted_pairs: torch.Tensor   # [T*k]
    pair_pos: torch.Tensor       # [T*k]
    active: torch.Tensor         # [4 + 4E] work list: U, then {expert, first position, count, 0}
    tile_offsets: Optional[torch.Tensor]  # [E+1] or None
    block_m: int = 0


def alloc_align(T: int, k: int, E: int, device, block_m: int = 0) -> AlignOut:
    i32 = dict(dtype=torch.int32, device=device)
    return AlignOut(torch.empty(E + 1, **i32), torch.empty(max(T * k, 1), **i32), torch.empty(max(T * k, 1), **i32),
                    torch.empty(4 + 4 * E, **i32), torch.empty(E + 1, **i32) if block_m > 0 else None, block_m)


def active_experts(al: AlignOut):
    """Host copy of the active-expert work list: list of (expert, first position, count)."""
    w = al.active.cpu()
    U = int(w[0])
    return [tuple(int(v) for v in w[4 + 4 * u: 7 + 4 * u]) for u in range(U)]


def moe_align_into(ids, E, out: AlignOut, stream=None) -> AlignOut:
    _need(ids, torch.int32, "topk_ids")
    T, k = ids.shape
    check("moe_align", lib().moe_align(_ptr(ids), T, k, E, out.block_m, _ptr(out.offsets), _ptr(out.sorted_pairs),
                                       _ptr(out.pair_pos), _ptr(out.active), _ptr(out.tile_offsets),
                                       _stream(stream)))
    return out


def moe_align(ids, E, block_m=0, stream=None) -> AlignOut:
    T, k = ids.shape
    return moe_align_into(ids, E, alloc_align(T, k, E, ids.device, block_m), stream)


ROUTE_ALIGN_COUNTERS = 256  # MOE_ROUTE_ALIGN_COUNTERS in w4a16_moe.h


def alloc_counter(device) -> torch.Tensor:
    """Zeroed device counters for moe_route_align (each call leaves them zero)."""
    return torch.zeros(ROUTE_ALIGN_COUNTERS, dtype=torch.int32, device=device)


def moe_route_align_into(x, w_router, k, route: RouteOut, al: AlignOut, counter: torch.Tensor, renormalize=True,
                         stream=None):
    """moe_route + moe_align in one launch for T <= 128 (bit-identical outputs)."""
    _need(x, torch.bfloat16, "x")
    _need(w_router, torch.bfloat16, "w_router")
    _need(counter, torch.int32, "counter")
    if counter.numel() < ROUTE_ALIGN_COUNTERS:
        raise ValueError(f"moe_route_align needs {ROUTE_ALIGN_COUNTERS} counters, got {counter.numel()}")
    T, d = x.shape
    E = w_router.shape[0]
    check("moe_route_align", lib().moe_route_align(
        _ptr(x), _ptr(w_router), T, d, E, k, int(bool(renormalize)), al.block_m, _ptr(route.logits),
        _ptr(route.ids), _ptr(route.weights), _ptr(al.offsets), _ptr(al.sorted_pairs), _ptr(al.pair_pos),
        _ptr(al.active), _ptr(al.tile_offsets), _ptr(counter), _stream(stream)))
    return route, al


# ---------------------------------------------------------------- grouped FFN

def ffn_workspace_bytes(T, d, I, E, k, mode=MODE_AUTO) -> int:
    return int(lib().moe_ffn_workspace_bytes(T, d, I, E, k, mode))


def alloc_workspace(T, d, I, E, k, mode=MODE_AUTO, device="cuda") -> torch.Tensor:
    return torch.empty(max(ffn_workspace_bytes(T, d, I, E, k, mode), 256), dtype=torch.uint8, device=device)


def _ffn_args(x, route: RouteOut, al: AlignOut, bank: torch.Tensor, I: int, out, workspace, mode, combine,
              slot_of_expert, bank_stride):
    _need(x, torch.bfloat16, "x")
    _need(bank, torch.uint8, "bank")
    if workspace is not None:
        _need(workspace, torch.uint8, "workspace")
    if combine:
        _need(out, torch.bfloat16, "out")
    if slot_of_expert is not None:
        _need(slot_of_expert, torch.int32, "slot_of_expert")
    T, d = x.shape
    E = route.logits.shape[1]
    k = route.ids.shape[1]
    a = _lib.FfnArgs()
    a.x, a.T, a.d, a.I, a.E, a.k = x.data_ptr(), T, d, I, E, k
    a.topk_ids, a.topk_weights = route.ids.data_ptr(), route.weights.data_ptr()
    a.expert_offsets, a.sorted_pairs = al.offsets.data_ptr(), al.sorted_pairs.data_ptr()
    a.pair_pos, a.active_experts = al.pair_pos.data_ptr(), al.active.data_ptr()
    a.tile_offsets = al.tile_offsets.data_ptr() if al.tile_offsets is not None else None
    a.bank = bank.data_ptr()
    a.bank_stride = bank.stride(0) if bank_stride is None else bank_stride
    a.slot_of_expert = slot_of_expert.data_ptr() if slot_of_expert is not None else None
    a.mode, a.combine = mode, int(bool(combine))
    a.out = out.data_ptr() if out is not None else None
    a.workspace = workspace.data_ptr() if workspace is not None else None
    a.workspace_bytes = workspace.numel() if workspace is not None else 0
    return a


def moe_w4a16_grouped_ffn_into(x, route: RouteOut, al: AlignOut, bank: torch.Tensor, I: int, out: torch.Tensor,
                               workspace: torch.Tensor, mode=MODE_AUTO, combine=True,
                               slot_of_expert: Optional[torch.Tensor] = None, bank_stride: Optional[int] = None,
                               stream=None):
    if workspace is None:
        raise ValueError("workspace is required (moe_w4a16_grouped_ffn_noalloc_into uses the library's scratch)")
    a = _ffn_args(x, route, al, bank, I, out, workspace, mode, combine, slot_of_expert, bank_stride)
    check("moe_w4a16_grouped_ffn", lib().moe_w4a16_grouped_ffn(ctypes.byref(a), _stream(stream)))
    return out


NOALLOC_SCRATCH_BYTES = 64 << 20  # MOE_NOALLOC_SCRATCH_BYTES in w4a16_moe.h


def moe_w4a16_grouped_ffn_noalloc_into(x, route: RouteOut, al: AlignOut, bank: torch.Tensor, I: int,
                                       out: torch.Tensor, mode=MODE_AUTO, combine=True,
                                       slot_of_expert: Optional[torch.Tensor] = None,
                                       bank_stride: Optional[int] = None, stream=None):
    """moe_w4a16_grouped_ffn with the library's per-GPU scratch as its workspace
    (no workspace argument, no allocation); calls on one GPU must not overlap."""
    a = _ffn_args(x, route, al, bank, I, out, None, mode, combine, slot_of_expert, bank_stride)
    check("moe_w4a16_grouped_ffn_noalloc", lib().moe_w4a16_grouped_ffn_noalloc(ctypes.byref(a), _stream(stream)))
    return out


# ---------------------------------------------------------------- whole decode layer

DECODE_LAYER_COUNTERS = 1024  # MOE_DECODE_LAYER_COUNTERS in w4a16_moe.h


def alloc_layer_counters(device) -> torch.Tensor:
    """Zeroed device counters for moe_decode_layer (each call leaves them zero,
    the last one excepted: a timeout flag)."""
    return torch.zeros(DECODE_LAYER_COUNTERS, dtype=torch.int32, device=device)


def decode_layer_workspace_bytes(T, d, I, E, k) -> int:
    return int(lib().moe_decode_layer_workspace_bytes(T, d, I, E, k))


def _layer_args(x, w_router, bank, I, k, route, out, workspace, counters, renormalize, bank_stride, name):
    _need(x, torch.bfloat16, "x")
    _need(w_router, torch.bfloat16, "w_router")
    _need(bank, torch.uint8, "bank")
    _need(out, torch.bfloat16, "out")
    _need(workspace, torch.uint8, "workspace")
    _need(counters, torch.int32, "counters")
    if counters.numel() < DECODE_LAYER_COUNTERS:
        raise ValueError(f"{name} needs {DECODE_LAYER_COUNTERS} counters, got {counters.numel()}")
    T, d = x.shape
    E = w_router.shape[0]
    a = _lib.LayerArgs()
    a.x, a.w_router, a.T, a.d, a.I, a.E, a.k = x.data_ptr(), w_router.data_ptr(), T, d, I, E, k
    a.renormalize = int(bool(renormalize))
    a.bank = bank.data_ptr()
    a.bank_stride = bank.stride(0) if bank_stride is None else bank_stride
    a.logits, a.topk_ids, a.topk_weights = route.logits.data_ptr(), route.ids.data_ptr(), route.weights.data_ptr()
    a.out = out.data_ptr()
    a.workspace, a.workspace_bytes = workspace.data_ptr(), workspace.numel()
    a.counters = counters.data_ptr()
    return a


def moe_decode_layer_into(x, w_router, bank: torch.Tensor, I: int, k: int, route: RouteOut, out: torch.Tensor,
                          workspace: torch.Tensor, counters: torch.Tensor, renormalize=True,
                          bank_stride: Optional[int] = None, stream=None):
    """Router, top-k, grouped gate/up, down and combine of one decode step (T <= 16)
    in two launches; outputs bit-identical to moe_route_align + moe_w4a16_grouped_ffn."""
    a = _layer_args(x, w_router, bank, I, k, route, out, workspace, counters, renormalize, bank_stride,
                    "moe_decode_layer")
    check("moe_decode_layer", lib().moe_decode_layer(ctypes.byref(a), _stream(stream)))
    return out


def moe_mat_decode_layer_into(x, w_router, bank: torch.Tensor, I: int, k: int, route: RouteOut, out: torch.Tensor,
                              workspace: torch.Tensor, counters: torch.Tensor, tau: float, renormalize=True,
                              bank_stride: Optional[int] = None, stream=None):
    """moe_decode_layer_into on nested two/four-bit blobs (layout m1, from mat_from_w4):
    each expert at four bits when the largest routing weight of its pairs reaches tau."""
    a = _layer_args(x, w_router, bank, I, k, route, out, workspace, counters, renormalize, bank_stride,
                    "moe_mat_decode_layer")
    check("moe_mat_decode_layer", lib().moe_mat_decode_layer(ctypes.byref(a), float(tau), _stream(stream)))
    return out


def layer_routing_timed_out(counters: torch.Tensor) -> bool:
    """Whether a moe_decode_layer call on these counters gave up its bounded wait
    for the routing (the last counter; the outputs of that call are invalid).
    Synchronises the device (every stream) before reading the flag."""
    torch.cuda.synchronize(counters.device)
    return bool(int(counters[DECODE_LAYER_COUNTERS - 1].item()))


def moe_decode_layer(x, w_router, bank: torch.Tensor, I: int, k: int, renormalize=True, stream=None):
    """Allocating convenience form of moe_decode_layer_into: returns (out, route).
    It reads the routing-wait flag after the call (a device round trip) and raises
    MoeError if the wait timed out."""
    T, d = x.shape
    E = w_router.shape[0]
    route = alloc_route(T, E, k, x.device)
    out = torch.empty((T, d), dtype=torch.bfloat16, device=x.device)
    ws = torch.empty(max(decode_layer_workspace_bytes(T, d, I, E, k), 256), dtype=torch.uint8, device=x.device)
    ctr = alloc_layer_counters(x.device)
    moe_decode_layer_into(x, w_router, bank, I, k, route, out, ws, ctr, renormalize, stream=stream)
    if layer_routing_timed_out(ctr):
        raise _lib.MoeError("moe_decode_layer", 5, "the bounded wait for the routing timed out; outputs are invalid")
    return out, route


def bf16_expert_bytes(d: int, I: int) -> int:
    return int(lib().moe_bf16_expert_bytes(d, I))


def pack_bf16_experts(w13: torch.Tensor, w2: torch.Tensor, bank: Optional[torch.Tensor] = None, stream=None):
    """BF16 expert bank: w13 [E, 2I, d], w2 [E, d, I] (bf16, GPU) copied into blobs
    (uint8 [E, stride], stride = bf16 blob bytes rounded up to 256)."""
    _need(w13, torch.bfloat16, "w13")
    _need(w2, torch.bfloat16, "w2")
    E, twoI, d = w13.shape
    I = twoI // 2
    stride = (bf16_expert_bytes(d, I) + 255) // 256 * 256
    if bank is None:
        bank = torch.empty((E, stride), dtype=torch.uint8, device=w13.device)
    check("moe_bf16_pack", lib().moe_bf16_pack(_ptr(w13.contiguous()), _ptr(w2.contiguous()), E, d, I, _ptr(bank),
                                               bank.stride(0), _stream(stream)))
    return bank


def moe_bf16_grouped_ffn_into(x, route: RouteOut, al: AlignOut, bank: torch.Tensor, I: int, out: torch.Tensor,
                              workspace: torch.Tensor, combine=True, slot_of_expert: Optional[torch.Tensor] = None,
                              stream=None):
    """The grouped pass over BF16 expert blobs (pack_bf16_experts); workspace sized
    with mode=MODE_DECODE."""
    _need(x, torch.bfloat16, "x")
    _need(bank, torch.uint8, "bank")
    _need(workspace, torch.uint8, "workspace")
    if combine:
        _need(out, torch.bfloat16, "out")
    if slot_of_expert is not None:
        _need(slot_of_expert, torch.int32, "slot_of_expert")
    T, d = x.shape
    a = _lib.FfnArgs()
    a.x, a.T, a.d, a.I, a.E, a.k = x.data_ptr(), T, d, I, route.logits.shape[1], route.ids.shape[1]
    a.topk_ids, a.topk_weights = route.ids.data_ptr(), route.weights.data_ptr()
    a.expert_offsets, a.sorted_pairs = al.offsets.data_ptr(), al.sorted_pairs.data_ptr()
    a.pair_pos, a.active_experts = al.pair_pos.data_ptr(), al.active.data_ptr()
    a.tile_offsets = al.tile_offsets.data_ptr() if al.tile_offsets is not None else None
    a.bank, a.bank_stride = bank.data_ptr(), bank.stride(0)
    a.slot_of_expert = slot_of_expert.data_ptr() if slot_of_expert is not None else None
    a.mode, a.combine = MODE_DECODE, int(bool(combine))
    a.out = out.data_ptr() if out is not None else None
    a.workspace, a.workspace_bytes = workspace.data_ptr(), workspace.numel()
    check("moe_bf16_grouped_ffn", lib().moe_bf16_grouped_ffn(ctypes.byref(a), _stream(stream)))
    return out


def moe_bf16_grouped_ffn(x, route, al, bank, I, stream=None):
    T, d = x.shape
    E, k = route.logits.shape[1], route.ids.shape[1]
    out = torch.empty((T, d), dtype=torch.bfloat16, device=x.device)
    ws = alloc_workspace(T, d, I, E, k, MODE_DECODE, x.device)
    return moe_bf16_grouped_ffn_into(x, route, al, bank, I, out, ws, True, stream=stream)


def mat_layout(d: int, I: int) -> dict:
    lay = _lib.MatLayout()
    check("moe_mat_layout_get", lib().moe_mat_layout_get(d, I, ctypes.byref(lay)))
    return {f: getattr(lay, f) for f, _ in _lib.MatLayout._fields_}


def mat_from_w4(w4_bank: torch.Tensor, d: int, I: int, stream=None) -> torch.Tensor:
    """Nested two/four-bit bank (layout m1) from a four-bit bank (pack_experts)."""
    _need(w4_bank, torch.uint8, "w4_bank")
    E = w4_bank.shape[0]
    stride = mat_layout(d, I)["blob_bytes"]
    bank = torch.empty((E, stride), dtype=torch.uint8, device=w4_bank.device)
    check("moe_mat_from_w4", lib().moe_mat_from_w4(_ptr(w4_bank), w4_bank.stride(0), E, d, I, _ptr(bank), stride,
                                                   _stream(stream)))
    return bank


def moe_mat_grouped_ffn_into(x, route: RouteOut, al: AlignOut, bank: torch.Tensor, I: int, out: torch.Tensor,
                             workspace: torch.Tensor, tau: float, combine=True,
                             slot_of_expert: Optional[torch.Tensor] = None, stream=None):
    """The grouped pass over nested two/four-bit blobs (mat_from_w4): an expert runs
    at four bits when its largest routing weight in the step is >= tau, else at two."""
    _need(x, torch.bfloat16, "x")
    _need(bank, torch.uint8, "bank")
    _need(workspace, torch.uint8, "workspace")
    if combine:
        _need(out, torch.bfloat16, "out")
    T, d = x.shape
    a = _lib.FfnArgs()
    a.x, a.T, a.d, a.I, a.E, a.k = x.data_ptr(), T, d, I, route.logits.shape[1], route.ids.shape[1]
    a.topk_ids, a.topk_weights = route.ids.data_ptr(), route.weights.data_ptr()
    a.expert_offsets, a.sorted_pairs = al.offsets.data_ptr(), al.sorted_pairs.data_ptr()
    a.pair_pos, a.active_experts = al.pair_pos.data_ptr(), al.active.data_ptr()
    a.tile_offsets = al.tile_offsets.data_ptr() if al.tile_offsets is not None else None
    a.bank, a.bank_stride = bank.data_ptr(), bank.stride(0)
    a.slot_of_expert = slot_of_expert.data_ptr() if slot_of_expert is not None else None
    a.mode, a.combine = MODE_DECODE, int(bool(combine))
    a.out = out.data_ptr() if out is not None else None
    a.workspace, a.workspace_bytes = workspace.data_ptr(), workspace.numel()
    check("moe_mat_grouped_ffn", lib().moe_mat_grouped_ffn(ctypes.byref(a), float(tau), _stream(stream)))
    return out


def moe_w4a16_grouped_ffn(x, route, al, bank, I, mode=MODE_AUTO, slot_of_expert=None, stream=None):
    T, d = x.shape
    E, k = route.logits.shape[1], route.ids.shape[1]
    out = torch.empty((T, d), dtype=torch.bfloat16, device=x.device)
    ws = alloc_workspace(T, d, I, E, k, mode, x.device)
    return moe_w4a16_grouped_ffn_into(x, route, al, bank, I, out, ws, mode, True, slot_of_expert, stream=stream)


# ---------------------------------------------------------------- rows sorted by expert and back

DTYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}  # moe_dtype in w4a16_moe.h


def _launch(fn, device, stream, *args):
    """fn(*args, stream handle) with GPU `device` (an index) current; the stream defaults to
    that GPU's current one (whose handle alone is asked for: a Stream object costs 1.6 us)."""
    if stream is None:
        handle = torch._C._cuda_getCurrentRawStream(device)
    elif stream.device.index != device:
        raise ValueError(f"stream on {stream.device} for tensors on GPU {device}")
    else:
        handle = stream.cuda_stream
    if torch._C._cuda_getDevice() == device:  # (a tensor is on it: the GPU is initialised)
        return fn(*args, handle)
    with torch.cuda.device(device):
        return fn(*args, handle)


def _like(t, name, dtype, shape, device):
    """A contiguous tensor of this type and shape on GPU `device`: its address."""
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.get_device() != device:
        raise ValueError(f"{name} must be on GPU {device}, got {t.device}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _rows(t, name, dtype, T, d, device, output=False):
    """A [T, d] tensor with contiguous rows at any stride: its address and row stride."""
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != (T, d):
        raise ValueError(f"{name} must have shape ({T}, {d}), got {tuple(t.shape)}")
    if t.get_device() != device:
        raise ValueError(f"{name} must be on GPU {device}, got {t.device}")
    stride, inner = t.stride()
    if inner != 1 and d > 1:
        raise ValueError(f"{name} must have contiguous rows")
    if T <= 1:
        stride = d
    elif output and stride < d:
        raise ValueError(f"{name} must have rows that do not overlap")
    return t.data_ptr(), stride


def _row_type(t, name):
    """Type, GPU index, and the two sizes of a row tensor."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    dtype = t.dtype
    if dtype not in DTYPES:
        raise TypeError(f"{name} must be bfloat16, float16 or float32, got {dtype}")
    shape = t.shape
    if len(shape) != 2:
        raise ValueError(f"{name} must have two dimensions, got {tuple(shape)}")
    device = t.get_device()
    if device < 0:
        raise ValueError(f"{name} must be a GPU tensor")
    return dtype, device, *shape


def _first_rows(t, name):
    """_row_type and _rows of a call's first input: type, GPU index, sizes, address and row
    stride."""
    dtype, device, T, d = _row_type(t, name)
    stride, inner = t.stride()
    if inner != 1 and d > 1:
        raise ValueError(f"{name} must have contiguous rows")
    return dtype, device, T, d, t.data_ptr(), stride if T > 1 else d


def _pairs(pair_pos, weights, dweights, T, k, device):
    """Addresses of pair_pos (at least T*k positions), weights and dweights ([T, k])."""
    if pair_pos.dtype is not torch.int32:
        raise TypeError(f"pair_pos must be torch.int32, got {pair_pos.dtype}")
    if pair_pos.numel() < T * k or not pair_pos.is_contiguous():
        raise ValueError(f"pair_pos must be contiguous with at least {T * k} positions")
    if pair_pos.get_device() != device:
        raise ValueError(f"pair_pos must be on GPU {device}, got {pair_pos.device}")
    w = None if weights is None else _like(weights, "weights", torch.float32, (T, k), device)
    dw = None if dweights is None else _like(dweights, "dweights", torch.float32, (T, k), device)
    return pair_pos.data_ptr(), w, dw


def moe_permute_into(x, pair_pos, k, rows, weights: Optional[torch.Tensor] = None, stream=None):
    """rows[pair_pos[t*k + j]] = x[t], times weights[t, j] if given.

    x [T, d] and rows [num_rows, d] bf16, fp16 or fp32 with any row stride; pair_pos from
    moe_align (AlignOut.pair_pos).  Pairs whose position is negative or past the last row
    are dropped; rows that no pair names keep their contents."""
    dtype, dev, T, d, xp, xs = _first_rows(x, "x")
    R = rows.shape[0]
    rp, rs = _rows(rows, "rows", dtype, R, d, dev, True)
    pp, wp, _ = _pairs(pair_pos, weights, None, T, k, dev)
    check("moe_permute", _launch(
        lib().moe_permute, dev, stream, xp, xs, DTYPES[dtype], T, d, k, pp, wp, rp, rs, R))
    return rows


def moe_unpermute_into(rows, pair_pos, k, out, weights: Optional[torch.Tensor] = None, stream=None):
    """out[t] = sum over j of rows[pair_pos[t*k + j]], times weights[t, j] if given
    (float32 sums in slot order, one rounding; dropped pairs add nothing)."""
    dtype, dev, R, d, rp, rs = _first_rows(rows, "rows")
    T = out.shape[0]
    op, os = _rows(out, "out", dtype, T, d, dev, True)
    pp, wp, _ = _pairs(pair_pos, weights, None, T, k, dev)
    check("moe_unpermute", _launch(
        lib().moe_unpermute, dev, stream, rp, rs, R, DTYPES[dtype], T, d, k, pp, wp, op, os))
    return out


def moe_permute_backward_into(drows, pair_pos, k, dx, weights: Optional[torch.Tensor] = None,
                              x: Optional[torch.Tensor] = None, dweights: Optional[torch.Tensor] = None, stream=None):
    """Gradient of moe_permute: dx[t] = sum over j of w drows[pos]; with x and dweights
    also dweights[t, j] = <x[t], drows[pos]> (0 for dropped pairs)."""
    dtype, dev, R, d, rp, rs = _first_rows(drows, "drows")
    if (x is None) != (dweights is None):
        raise ValueError("x and dweights go together")
    T = dx.shape[0]
    op, os = _rows(dx, "dx", dtype, T, d, dev, True)
    xp, xs = (None, 0) if x is None else _rows(x, "x", dtype, T, d, dev)
    pp, wp, dwp = _pairs(pair_pos, weights, dweights, T, k, dev)
    check("moe_permute_backward", _launch(
        lib().moe_permute_backward, dev, stream, rp, rs, R, xp, xs, DTYPES[dtype], T, d, k, pp, wp, op, os, dwp))
    return dx


def moe_unpermute_backward_into(dout, pair_pos, k, drows, weights: Optional[torch.Tensor] = None,
                                rows: Optional[torch.Tensor] = None, dweights: Optional[torch.Tensor] = None,
                                stream=None):
    """Gradient of moe_unpermute: drows[pos] = w dout[t]; with rows and dweights also
    dweights[t, j] = <dout[t], rows[pos]> (0 for dropped pairs).  Rows of drows that no
    pair names keep their contents."""
    dtype, dev, T, d, op, os = _first_rows(dout, "dout")
    if (rows is None) != (dweights is None):
        raise ValueError("rows and dweights go together")
    R = drows.shape[0]
    dp, ds = _rows(drows, "drows", dtype, R, d, dev, True)
    rp, rs = (None, 0) if rows is None else _rows(rows, "rows", dtype, R, d, dev)
    pp, wp, dwp = _pairs(pair_pos, weights, dweights, T, k, dev)
    check("moe_unpermute_backward", _launch(
        lib().moe_unpermute_backward, dev, stream, op, os, rp, rs, DTYPES[dtype], T, d, k, pp, wp, dp, ds, R, dwp))
    return drows


def _alloc_on(device, stream):
    """Context in which allocations belong to the stream that the call runs on."""
    return torch.cuda.stream(torch.cuda.current_stream(device) if stream is None else stream)


def moe_permute(x, pair_pos, k, weights=None, stream=None):
    """Allocating form of moe_permute_into: rows [T*k, d].  Rows behind the last placed
    pair (there are some when pairs were dropped) are uninitialised."""
    _row_type(x, "x")
    with _alloc_on(x.device, stream):
        rows = torch.empty((x.shape[0] * k, x.shape[1]), dtype=x.dtype, device=x.device)
    return moe_permute_into(x, pair_pos, k, rows, weights, stream)


def moe_unpermute(rows, pair_pos, k, T, weights=None, stream=None):
    """Allocating form of moe_unpermute_into: out [T, d]."""
    _row_type(rows, "rows")
    with _alloc_on(rows.device, stream):
        out = torch.empty((T, rows.shape[1]), dtype=rows.dtype, device=rows.device)
    return moe_unpermute_into(rows, pair_pos, k, out, weights, stream)


# ---------------------------------------------------------------- router gradient

def route_backward_workspace_bytes(T, d, E, k) -> int:
    return int(lib().moe_route_backward_workspace_bytes(T, d, E, k))


def alloc_route_backward_workspace(T, d, E, k, device) -> torch.Tensor:
    return torch.empty(max(route_backward_workspace_bytes(T, d, E, k), 256), dtype=torch.uint8, device=device)


def moe_route_backward_into(x, w_router, route: RouteOut, dweights, dx: Optional[torch.Tensor],
                            dw_router: Optional[torch.Tensor], workspace, renormalize=True,
                            dlogits: Optional[torch.Tensor] = None, dx_add: Optional[torch.Tensor] = None,
                            stream=None):
    """Gradient of moe_route from that of its weights, dweights [T, k] float32 (e.g. from
    moe_unpermute_backward): dx [T, d] bf16 (plus dx_add, which may be dx itself) and
    dw_router [E, d] float32; either may be None.  dlogits [T, E] float32 adds the
    gradient of a loss on the logits themselves.  `route` and `renormalize` as moe_route
    had them."""
    _, dev, T, d = _row_type(x, "x")
    E, k = w_router.shape[0], route.ids.shape[1]
    bf, f32 = torch.bfloat16, torch.float32
    a = _lib.RouteBackwardArgs()
    a.x, a.w_router = _like(x, "x", bf, (T, d), dev), _like(w_router, "w_router", bf, (E, d), dev)
    a.T, a.d, a.E, a.k, a.renormalize = T, d, E, k, int(bool(renormalize))
    a.logits = _like(route.logits, "route.logits", f32, (T, E), dev)
    a.topk_ids = _like(route.ids, "route.ids", torch.int32, (T, k), dev)
    a.topk_weights = _like(route.weights, "route.weights", f32, (T, k), dev)
    a.dweights = _like(dweights, "dweights", f32, (T, k), dev)
    a.dlogits = None if dlogits is None else _like(dlogits, "dlogits", f32, (T, E), dev)
    a.dx_add = None if dx_add is None else _like(dx_add, "dx_add", bf, (T, d), dev)
    a.dx = None if dx is None else _like(dx, "dx", bf, (T, d), dev)
    a.dw_router = None if dw_router is None else _like(dw_router, "dw_router", f32, (E, d), dev)
    a.workspace = _like(workspace, "workspace", torch.uint8, workspace.shape, dev)
    a.workspace_bytes = workspace.numel()
    check("moe_route_backward", _launch(
        lib().moe_route_backward, dev, stream, ctypes.byref(a)))
    return dx, dw_router


def moe_route_backward(x, w_router, route: RouteOut, dweights, renormalize=True, dlogits=None, dx_add=None,
                       stream=None):
    """Allocating form of moe_route_backward_into: (dx, dw_router)."""
    _row_type(x, "x")
    (T, d), E = x.shape, w_router.shape[0]
    with _alloc_on(x.device, stream):
        dx = torch.empty((T, d), dtype=torch.bfloat16, device=x.device)
        dw = torch.empty((E, d), dtype=torch.float32, device=x.device)
        ws = alloc_route_backward_workspace(T, d, E, route.ids.shape[1], x.device)
    return moe_route_backward_into(x, w_router, route, dweights, dx, dw, ws, renormalize, dlogits, dx_add, stream)


# ---------------------------------------------------------------- norms around a block

GATE_NONE, GATE_CHANNEL, GATE_TOKEN, GATE_FULL = 0, 1, 2, 3


@dataclass
class BlockNorm:
    """Parameters of moe_block_norm (all of the residual stream's type):
    z = rms(y) norm_out, h = residual_scale x + gate z, n = rms(h) norm_in."""
    norm_in: Optional[torch.Tensor] = None   # [d] weights of the norm before the next block
    norm_out: Optional[torch.Tensor] = None  # [d] weights of the norm behind this block
    gate: Optional[torch.Tensor] = None      # [d] per channel, [T, 1] per token, or [T, d]
    residual_scale: float = 1.0
    eps: float = 1e-6


@dataclass
class BlockNormGrads:
    """Outputs of moe_block_norm_backward; None: not wanted."""
    dx: Optional[torch.Tensor] = None         # [T, d]
    dy: Optional[torch.Tensor] = None         # [T, d]
    dgate: Optional[torch.Tensor] = None      # [d] or [T, 1] float32, or [T, d] of the rows' type
    dnorm_out: Optional[torch.Tensor] = None  # [d] float32
    dnorm_in: Optional[torch.Tensor] = None   # [d] float32


def _block_norm_args(norm: BlockNorm, x, y):
    a = _lib.BlockNormArgs()
    dtype, dev, T, d, a.x, a.x_stride = _first_rows(x, "x")
    a.dtype, a.T, a.d = DTYPES[dtype], T, d
    if y is not None:
        a.y, a.y_stride = _rows(y, "y", dtype, T, d, dev)
    if norm.norm_out is not None:
        a.norm_out = _like(norm.norm_out, "norm_out", dtype, (d,), dev)
    if norm.norm_in is not None:
        a.norm_in = _like(norm.norm_in, "norm_in", dtype, (d,), dev)
    g = norm.gate
    if g is not None:
        if g.dim() == 1:
            a.gate_kind, a.gate = GATE_CHANNEL, _like(g, "gate", dtype, (d,), dev)
        elif g.dim() == 2 and g.shape[1] == 1:
            a.gate_kind = GATE_TOKEN
            a.gate, a.gate_stride = _rows(g, "gate", dtype, T, 1, dev)
        else:
            a.gate_kind = GATE_FULL
            a.gate, a.gate_stride = _rows(g, "gate", dtype, T, d, dev)
    a.residual_scale, a.eps = norm.residual_scale, norm.eps
    return a, dtype, T, d, dev


def moe_block_norm_into(norm: BlockNorm, x, y: Optional[torch.Tensor] = None, h: Optional[torch.Tensor] = None,
                        n: Optional[torch.Tensor] = None, stream=None):
    """What stands between two blocks, in one pass: h (residual stream behind this block)
    and n (input of the next one, exactly when norm.norm_in is given); x [T, d] residual
    stream, y [T, d] this block's output or None.  h may be x or y itself, n may be y."""
    a, dtype, T, d, dev = _block_norm_args(norm, x, y)
    hp, hs = (None, 0) if h is None else _rows(h, "h", dtype, T, d, dev, True)
    np_, ns = (None, 0) if n is None else _rows(n, "n", dtype, T, d, dev, True)
    check("moe_block_norm", _launch(
        lib().moe_block_norm, dev, stream, ctypes.byref(a), hp, hs, np_, ns))
    return h, n


def moe_block_norm(norm: BlockNorm, x, y: Optional[torch.Tensor] = None, stream=None):
    """Allocating form of moe_block_norm_into: (h, n).  Without y, h is None where
    norm.norm_in is given and the residual scale is 1 (h is x then)."""
    _row_type(x, "x")
    with _alloc_on(x.device, stream):
        alone = y is None and norm.norm_in is not None and norm.residual_scale == 1.0
        h = None if alone else torch.empty(x.shape, dtype=x.dtype, device=x.device)
        n = None if norm.norm_in is None else torch.empty(x.shape, dtype=x.dtype, device=x.device)
    return moe_block_norm_into(norm, x, y, h, n, stream)


def block_norm_workspace_bytes(T, d) -> int:
    return int(lib().moe_block_norm_backward_workspace_bytes(T, d))


def alloc_block_norm_workspace(T, d, device) -> torch.Tensor:
    return torch.empty(max(block_norm_workspace_bytes(T, d), 256), dtype=torch.uint8, device=device)


def moe_block_norm_backward_into(norm: BlockNorm, x, y: Optional[torch.Tensor], grads: BlockNormGrads,
                                 workspace: Optional[torch.Tensor], dh: Optional[torch.Tensor] = None,
                                 dn: Optional[torch.Tensor] = None, stream=None) -> BlockNormGrads:
    """Gradient of moe_block_norm from those of h and n (None: zero), on the x and y of
    the forward call.  dx may be dh itself, dy may be y or dn itself.  The workspace
    (alloc_block_norm_workspace) is needed for the [d] gradients only."""
    a, dtype, T, d, dev = _block_norm_args(norm, x, y)
    g = _lib.BlockNormGradArgs()
    if dh is not None:
        g.dh, g.dh_stride = _rows(dh, "dh", dtype, T, d, dev)
    if dn is not None:
        g.dn, g.dn_stride = _rows(dn, "dn", dtype, T, d, dev)
    if grads.dx is not None:
        g.dx, g.dx_stride = _rows(grads.dx, "dx", dtype, T, d, dev, True)
    if grads.dy is not None:
        g.dy, g.dy_stride = _rows(grads.dy, "dy", dtype, T, d, dev, True)
    f32 = torch.float32
    if grads.dgate is not None:
        if a.gate_kind == GATE_FULL:
            g.dgate, g.dgate_stride = _rows(grads.dgate, "dgate", dtype, T, d, dev, True)
        else:
            shape = (d,) if a.gate_kind == GATE_CHANNEL else (T, 1)
            g.dgate = _like(grads.dgate, "dgate", f32, shape, dev)
    if grads.dnorm_out is not None:
        g.dnorm_out = _like(grads.dnorm_out, "dnorm_out", f32, (d,), dev)
    if grads.dnorm_in is not None:
        g.dnorm_in = _like(grads.dnorm_in, "dnorm_in", f32, (d,), dev)
    if workspace is not None:
        g.workspace = _like(workspace, "workspace", torch.uint8, workspace.shape, dev)
        g.workspace_bytes = workspace.numel()
    check("moe_block_norm_backward", _launch(
        lib().moe_block_norm_backward, dev, stream, ctypes.byref(a), ctypes.byref(g)))
    return grads


def moe_block_norm_backward(norm: BlockNorm, x, y: Optional[torch.Tensor] = None,
                            dh: Optional[torch.Tensor] = None, dn: Optional[torch.Tensor] = None,
                            stream=None) -> BlockNormGrads:
    """Allocating form of moe_block_norm_backward_into: every gradient there is."""
    _row_type(x, "x")
    (T, d), dev = x.shape, x.device
    with _alloc_on(dev, stream):
        def vec(p):
            return None if p is None else torch.empty(d, dtype=torch.float32, device=dev)

        grads = BlockNormGrads(torch.empty(x.shape, dtype=x.dtype, device=dev),
                               None if y is None else torch.empty(x.shape, dtype=x.dtype, device=dev),
                               None, vec(norm.norm_out), vec(norm.norm_in))
        if norm.gate is not None:
            full = norm.gate.dim() == 2 and norm.gate.shape[1] != 1
            grads.dgate = torch.empty(norm.gate.shape, dtype=x.dtype if full else torch.float32, device=dev)
        ws = alloc_block_norm_workspace(T, d, dev)
    return moe_block_norm_backward_into(norm, x, y, grads, ws, dh, dn, stream)


class MoELayer:
    """One W4A16 MoE layer step with preallocated buffers (no allocation per call).

    forward(x) = moe_route -> moe_align -> moe_w4a16_grouped_ffn on the current stream.
    block(x) = the whole block around it: norm before (norm_before [d]), forward, and
    what follows (after, a BlockNorm whose norm_in is the next block's norm before).
    """

    def __init__(self, w_router: torch.Tensor, bank: torch.Tensor, I: int, k: int, T_max: int,
                 mode=MODE_AUTO, renormalize=True, norm_before: Optional[torch.Tensor] = None,
                 after: Optional[BlockNorm] = None):
        self.w_router, self.bank, self.I, self.k, self.mode = w_router, bank, I, k, mode
        self.renormalize = renormalize
        self.E, self.d = w_router.shape
        dev = w_router.device
        self.T_max = T_max
        self.route = alloc_route(T_max, self.E, k, dev)
        self.align = alloc_align(T_max, k, self.E, dev)
        self.counter = alloc_counter(dev)
        self.out = torch.empty((T_max, self.d), dtype=torch.bfloat16, device=dev)
        need = max(ffn_workspace_bytes(t, self.d, I, self.E, k, mode) for t in range(1, T_max + 1))
        self.ws = torch.empty(max(need, 256), dtype=torch.uint8, device=dev)
        self.after = after
        self.before = None
        if after is not None or norm_before is not None:
            after = self.after = BlockNorm() if after is None else after
            self.n, self.h, self.n_next = (torch.empty_like(self.out) for _ in range(3))
            if norm_before is not None:
                self.before = BlockNorm(norm_in=norm_before, eps=after.eps)

    def views(self, T):
        r = RouteOut(self.route.logits[:T], self.route.ids[:T], self.route.weights[:T])
        a = AlignOut(self.align.offsets, self.align.sorted_pairs[:max(T * self.k, 1)],
                     self.align.pair_pos[:max(T * self.k, 1)], self.align.active, None, 0)
        return r, a

    def forward(self, x: torch.Tensor, out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
        T = x.shape[0]
        if T > self.T_max:
            raise ValueError(f"T={T} exceeds T_max={self.T_max}")
        r, a = self.views(T)
        moe_route_align_into(x, self.w_router, self.k, r, a, self.counter, self.renormalize, stream)
        o = self.out[:T] if out is None else out
        ws_need = ffn_workspace_bytes(T, self.d, self.I, self.E, self.k, self.mode)
        moe_w4a16_grouped_ffn_into(x, r, a, self.bank, self.I, o, self.ws[:max(ws_need, 256)], self.mode, True,
                                   stream=stream)
        return o

    def block(self, x: torch.Tensor, n: Optional[torch.Tensor] = None, stream=None):
        """One block on the residual stream x [T, d]: (h, n_next) with y = forward(n) and
        moe_block_norm's h and n behind it (n_next is None without after.norm_in).  n, if
        given, is the normed x that the block before returned; else norm_before is
        applied here.  The results lie in the layer's own buffers, which the next call
        overwrites; x and n may be another layer's."""
        if self.after is None:
            raise ValueError("block needs norm_before or after")
        T = x.shape[0]
        if T > self.T_max:
            raise ValueError(f"T={T} exceeds T_max={self.T_max}")
        if n is None:
            if self.before is None:
                raise ValueError("block needs n or norm_before")
            _, n = moe_block_norm_into(self.before, x, None, None, self.n[:T], stream)
        y = self.forward(n, stream=stream)
        n_next = self.n_next[:T] if self.after.norm_in is not None else None
        return moe_block_norm_into(self.after, x, y, self.h[:T], n_next, stream)


# ---------------------------------------------------------------- slot cache

class SlotCache:
    """Host LRU bookkeeping for S device slots over a pinned host expert store."""

    def __init__(self, E: int, S: int, blob_bytes: int, host_store: torch.Tensor, device_slots: torch.Tensor):
        _need(host_store, torch.uint8, "host_store", device=False)
        _need(device_slots, torch.uint8, "device_slots")
        if not host_store.is_pinned():
            raise ValueError("host_store must be pinned host memory")
        self.E, self.S, self.blob_bytes = E, S, blob_bytes
        self.host_store, self.device_slots = host_store, device_slots
        h = ctypes.c_void_p()
        check("moe_slot_cache_create", lib().moe_slot_cache_create(E, S, blob_bytes, _ptr(host_store),
                                                                   _ptr(device_slots), ctypes.byref(h)))
        self._h = h
        self.words = (E + 63) // 64

    def close(self):
        if getattr(self, "_h", None):
            lib().moe_slot_cache_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def load(self, pending: set, slot_table_dev: torch.Tensor, copy_stream, wait_event, done_event):
        """One round: returns (round experts set, hits, misses)."""
        # torch creates an event's HIP handle on its first record; make sure both exist
        if done_event.cuda_event == 0:
            done_event.record(copy_stream)
        if wait_event is not None and wait_event.cuda_event == 0:
            wait_event.record(torch.cuda.current_stream())
        pm = (ctypes.c_uint64 * self.words)()
        for e in pending:
            pm[e >> 6] |= 1 << (e & 63)
        rm = (ctypes.c_uint64 * self.words)()
        nh, nm = ctypes.c_int32(), ctypes.c_int32()
        check("slot_cache_load", lib().slot_cache_load(
            self._h, pm, rm, _ptr(slot_table_dev), ctypes.byref(nh), ctypes.byref(nm),
            ctypes.c_void_p(copy_stream.cuda_stream),
            ctypes.c_void_p(wait_event.cuda_event) if wait_event is not None else None,
            ctypes.c_void_p(done_event.cuda_event)))
        got = {e for e in range(self.E) if (rm[e >> 6] >> (e & 63)) & 1}
        return got, nh.value, nm.value

    POLICY_LRU, POLICY_COST = 0, 1

    def configure(self, policy: int = 0, decay: float = 0.9, copy_streams: int = 1):
        """Replacement policy (POLICY_LRU / POLICY_COST), usage decay and 1 or 2 copy streams."""
        check("moe_slot_cache_configure", lib().moe_slot_cache_configure(self._h, int(policy), float(decay),
                                                                         int(copy_streams)))

    def _mask(self, experts):
        m = (ctypes.c_uint64 * self.words)()
        for e in experts:
            m[e >> 6] |= 1 << (e & 63)
        return m

    def begin_step(self, needed: set):
        """The needed experts of a new step (usage averages of the cost-aware policy)."""
        check("slot_cache_begin_step", lib().slot_cache_begin_step(self._h, self._mask(needed)))

    def set_prefix(self, prefix_bytes: int):
        """Precision-aware loads: the blobs' first prefix_bytes are their two-bit part."""
        check("moe_slot_cache_set_prefix", lib().moe_slot_cache_set_prefix(self._h, int(prefix_bytes)))

    def load_precision(self, pending: set, full: set, slot_table_dev: torch.Tensor, copy_stream, wait_event,
                       done_event):
        """One round with per-expert precision (full: experts needed at four bits):
        returns (round experts set, hits, misses, bytes copied)."""
        if done_event.cuda_event == 0:
            done_event.record(copy_stream)
        if wait_event is not None and wait_event.cuda_event == 0:
            wait_event.record(torch.cuda.current_stream())
        rm = (ctypes.c_uint64 * self.words)()
        nh, nm, nb = ctypes.c_int32(), ctypes.c_int32(), ctypes.c_int64()
        check("slot_cache_load_precision", lib().slot_cache_load_precision(
            self._h, self._mask(pending), self._mask(full), rm, _ptr(slot_table_dev), ctypes.byref(nh),
            ctypes.byref(nm), ctypes.byref(nb), ctypes.c_void_p(copy_stream.cuda_stream),
            ctypes.c_void_p(wait_event.cuda_event) if wait_event is not None else None,
            ctypes.c_void_p(done_event.cuda_event)))
        got = {e for e in range(self.E) if (rm[e >> 6] >> (e & 63)) & 1}
        return got, nh.value, nm.value, nb.value

    def planes(self):
        """([S] 1 where the slot holds the whole blob, low-plane completions, bytes copied so far)."""
        sf = (ctypes.c_int32 * self.S)()
        up, nb = ctypes.c_int64(), ctypes.c_int64()
        check("moe_slot_cache_planes", lib().moe_slot_cache_planes(self._h, sf, ctypes.byref(up), ctypes.byref(nb)))
        return list(sf), up.value, nb.value

    def prefetch(self, predicted: set, max_copies: int, copy_stream, wait_event=None) -> int:
        """Copy predicted experts ahead of their round; returns the number of copies."""
        if wait_event is not None and wait_event.cuda_event == 0:
            wait_event.record(torch.cuda.current_stream())
        pm = (ctypes.c_uint64 * self.words)()
        for e in predicted:
            pm[e >> 6] |= 1 << (e & 63)
        n = ctypes.c_int32()
        check("slot_cache_prefetch", lib().slot_cache_prefetch(
            self._h, pm, int(max_copies), ctypes.byref(n), ctypes.c_void_p(copy_stream.cuda_stream),
            ctypes.c_void_p(wait_event.cuda_event) if wait_event is not None else None))
        return n.value

    def state(self):
        se = (ctypes.c_int32 * self.S)()
        h, m = ctypes.c_int64(), ctypes.c_int64()
        check("moe_slot_cache_state", lib().moe_slot_cache_state(self._h, se, ctypes.byref(h), ctypes.byref(m)))
        return list(se), h.value, m.value


# ---------------------------------------------------------------- timing

KERNELS = {"gateup_decode": 0, "down_decode": 1, "gateup_prefill": 2, "down_prefill": 3, "combine": 4,
           "gateup_bf16": 7, "down_bf16": 8, "gateup_mat": 9, "down_mat": 10,
           "route": 5, "align": 6, "permute": 11, "unpermute": 12, "route_backward": 13, "block_norm": 14,
           "block_norm_backward": 15}


def timing_enable(on: bool):
    check("moe_timing_enable", lib().moe_timing_enable(int(on)))


def timing_reset():
    check("moe_timing_reset", lib().moe_timing_reset())


def timing_read(kernel: str):
    ms, n = ctypes.c_double(), ctypes.c_int64()
    check("moe_timing_read", lib().moe_timing_read(KERNELS[kernel], ctypes.byref(ms), ctypes.byref(n)))
    return ms.value, n.value
