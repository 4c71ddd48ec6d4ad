"""Torch-tensor front end of libplmla (argument marshalling only).

Every step of the decode runs in the CUDA library; these functions check
shapes, dtypes and devices, then pass raw device pointers and sizes through the
C ABI.  PyTorch only supplies device memory and the current stream.
"""
from __future__ import annotations

import ctypes
import math

import torch

from . import _native

LATENT = 512
ROPE = 64
ROW = LATENT + ROPE
PAGE_TOKENS = 1536
DEFAULT_SCALE = 1.0 / math.sqrt(192.0)   # a 128-wide nope + 64-wide rope head


def _stream_ptr(stream, device):
    s = stream if stream is not None else torch.cuda.current_stream(device)
    return ctypes_void(s.cuda_stream)


def ctypes_void(v):
    return None if v in (0, None) else int(v)


def _require(cond, msg):
    if not cond:
        raise ValueError(msg)


def _check_bf16(t, name, shape=None):
    _require(isinstance(t, torch.Tensor), f"{name} must be a tensor")
    _require(t.is_cuda, f"{name} must be a CUDA tensor")
    _require(t.dtype == torch.bfloat16, f"{name} must be bfloat16")
    _require(t.is_contiguous(), f"{name} must be contiguous")
    if shape is not None:
        _require(tuple(t.shape) == tuple(shape), f"{name} has shape {tuple(t.shape)}, "
                                                 f"expected {tuple(shape)}")


def mla_split_budget(num_reqs, n_q, num_heads, cta_budget=0, min_splits=1) -> int:
    b = _native.lib().mla_split_budget(num_reqs, n_q, num_heads, cta_budget, min_splits)
    if b < 1:
        raise ValueError("invalid shape for mla_split_budget")
    return int(b)


def mla_workspace_size(num_reqs, n_q, num_heads, cta_budget=0, min_splits=1) -> int:
    n = _native.lib().mla_workspace_size(num_reqs, n_q, num_heads, cta_budget, min_splits)
    if n == 0:
        raise ValueError("invalid shape for mla_workspace_size")
    return int(n)


def mla_workspace_size_fp8(num_reqs, n_q, num_heads, cta_budget=0, min_splits=1) -> int:
    n = _native.lib().mla_workspace_size_fp8(num_reqs, n_q, num_heads, cta_budget, min_splits)
    if n == 0:
        raise ValueError("invalid shape for mla_workspace_size_fp8")
    return int(n)


def allocate_workspace(num_reqs, n_q, num_heads, cta_budget=0, min_splits=1, device=None,
                       fp8=False):
    """A caller-owned workspace tensor (uint8) of the size mla_decode (or, with
    ``fp8``, mla_decode_fp8) needs."""
    size = mla_workspace_size_fp8 if fp8 else mla_workspace_size
    n = size(num_reqs, n_q, num_heads, cta_budget, min_splits)
    return torch.empty(n, dtype=torch.uint8, device=device or "cuda")


def _byte_view(slab):
    """An E4M3 slab as uint8 (float8_e4m3fn tensors are viewed, not copied)."""
    if slab.dtype == torch.uint8:
        return slab
    _require(slab.dtype == getattr(torch, "float8_e4m3fn", None),
             "an FP8 slab must be uint8 or float8_e4m3fn")
    return slab.view(torch.uint8)


def mla_decode(q_nope_absorbed, q_rope, gate, slab, page_table, seq_lens, *, n_q=1,
               scale=DEFAULT_SCALE, out=None, lse=None, workspace=None, cta_budget=0,
               min_splits=1, stream=None, with_lse=True, events=None):
    """One gated-MLA decode step; returns (out, lse).

    ``events`` (optional): four torch.cuda.Event (or None) recorded before the
    plan kernel, before the split-decode kernel, before the combine kernel and
    after it, on the launch stream.  Each event must have been recorded once
    already, so that torch has created its handle.

    q_nope_absorbed, gate: [R*n_q, H, 512] bf16; q_rope: [R*n_q, H, 64] bf16.
    slab: [num_pages, page_stride] bf16 (page_stride >= 1536*576; row r of a
    page at r*576).  page_table: [R, ld] int32 with unit column stride (its row
    stride is passed through, so a strided view works).  seq_lens: [R] int32.
    """
    return _decode(q_nope_absorbed, q_rope, gate, slab, page_table, seq_lens, None, n_q, scale,
                   out, lse, workspace, cta_budget, min_splits, stream, with_lse, events)


def mla_decode_fp8(q_nope_absorbed, q_rope, gate, slab, page_table, seq_lens, *, kv_scale,
                   n_q=1, scale=DEFAULT_SCALE, out=None, lse=None, workspace=None, cta_budget=0,
                   min_splits=1, stream=None, with_lse=True, events=None):
    """mla_decode over E4M3 pages: slab is [num_pages, page_stride] uint8 (or
    float8_e4m3fn) holding E4M3 codes of value / kv_scale, 576 bytes per token
    row (page_stride >= 1536*576, a multiple of 16).  The queries stay bf16;
    the library splits each query row into two E4M3 parts with a power-of-two
    scale (exact for elements above 2^-2 of the scale).
    The workspace must come from allocate_workspace(..., fp8=True)."""
    _require(math.isfinite(kv_scale) and kv_scale > 0, "kv_scale must be finite and > 0")
    return _decode(q_nope_absorbed, q_rope, gate, _byte_view(slab), page_table, seq_lens,
                   float(kv_scale), n_q, scale, out, lse, workspace, cta_budget, min_splits,
                   stream, with_lse, events)


def _decode(q_nope_absorbed, q_rope, gate, slab, page_table, seq_lens, kv_scale, n_q, scale,
            out, lse, workspace, cta_budget, min_splits, stream, with_lse, events):
    fp8 = kv_scale is not None
    _require(q_nope_absorbed.dim() == 3, "q_nope_absorbed must be [R*n_q, H, 512]")
    T, H, _ = q_nope_absorbed.shape
    _require(T % n_q == 0, "first dimension must be num_reqs * n_q")
    R = T // n_q
    device = q_nope_absorbed.device
    _check_bf16(q_nope_absorbed, "q_nope_absorbed", (T, H, LATENT))
    _check_bf16(q_rope, "q_rope", (T, H, ROPE))
    _check_bf16(gate, "gate", (T, H, LATENT))
    want = torch.uint8 if fp8 else torch.bfloat16
    _require(slab.is_cuda and slab.dtype == want and slab.dim() == 2,
             f"slab must be a 2-D CUDA {want} tensor [num_pages, page_stride]")
    _require(slab.stride(1) == 1, "slab pages must be contiguous")
    num_pages, page_stride = slab.shape[0], slab.stride(0)
    _require(slab.shape[1] >= PAGE_TOKENS * ROW, "slab page too small")
    _require(page_table.is_cuda and page_table.dtype == torch.int32 and page_table.dim() == 2,
             "page_table must be a 2-D CUDA int32 tensor")
    _require(page_table.shape[0] == R and page_table.stride(1) == 1,
             "page_table must be [R, ld] with unit column stride")
    _require(seq_lens.is_cuda and seq_lens.dtype == torch.int32 and seq_lens.is_contiguous()
             and tuple(seq_lens.shape) == (R,), "seq_lens must be a contiguous CUDA int32 [R]")
    if out is None:
        out = torch.empty_like(q_nope_absorbed)
    _check_bf16(out, "out", (T, H, LATENT))
    if lse is None and with_lse:
        lse = torch.empty(T, H, dtype=torch.float32, device=device)
    if lse is not None:
        _require(lse.is_cuda and lse.dtype == torch.float32 and lse.is_contiguous()
                 and tuple(lse.shape) == (T, H), "lse must be a contiguous CUDA fp32 [T, H]")
    if workspace is None:
        workspace = allocate_workspace(R, n_q, H, cta_budget, min_splits, device, fp8=fp8)
    _require(workspace.is_cuda and workspace.is_contiguous(), "workspace must be CUDA memory")
    nbytes = workspace.numel() * workspace.element_size()
    ev = None
    if events is not None:
        handles = []
        for e in events:
            h = None if e is None else int(e.cuda_event)
            _require(h != 0, "stage events must have been recorded once before use")
            handles.append(h)
        ev = _native.StageEvents(*handles)
    lib = _native.lib()
    head = (q_nope_absorbed.data_ptr(), q_rope.data_ptr(), gate.data_ptr(), slab.data_ptr(),
            num_pages, page_stride)
    tail = (page_table.data_ptr(), page_table.stride(0), seq_lens.data_ptr(), R, n_q, H,
            float(scale), out.data_ptr(), lse.data_ptr() if lse is not None else None,
            workspace.data_ptr(), nbytes, int(cta_budget), int(min_splits),
            _stream_ptr(stream, device), ctypes.byref(ev) if ev is not None else None)
    if fp8:
        status = lib.mla_decode_fp8_ex(*head, kv_scale, *tail)
    else:
        status = lib.mla_decode_ex(*head, *tail)
    _native.check(status, "mla_decode_fp8" if fp8 else "mla_decode")
    return out, lse


def mla_decode_layers(q_nope_absorbed, q_rope, gate, slabs, page_table, seq_lens, *, n_q=1,
                      scale=DEFAULT_SCALE, kv_scale=None, out=None, lse=None, workspace=None,
                      cta_budget=0, min_splits=1, stream=None, with_lse=True):
    """The decode step of several MLA layers that share the page table and the
    history lengths (every layer's pool is paged by the same global page IDs):
    one split plan for the step, then each layer's split decode and combine.
    q_nope_absorbed, q_rope, gate and slabs are lists with one tensor per layer,
    each as in mla_decode (E4M3 slabs with `kv_scale`, a float or one per
    layer); returns (outs, lses), lists (lses of None without LSE).  Layer l's
    results equal mla_decode's (or mla_decode_fp8's) on layer l's tensors."""
    L = len(slabs)
    _require(L >= 1 and len(q_nope_absorbed) == L and len(q_rope) == L and len(gate) == L,
             "one query, rope, gate and slab tensor per layer")
    fp8 = kv_scale is not None
    scales = None
    if fp8:
        scales = list(kv_scale) if isinstance(kv_scale, (list, tuple)) else [kv_scale] * L
        _require(len(scales) == L and all(math.isfinite(v) and v > 0 for v in scales),
                 "kv_scale must be finite and > 0 (one value, or one per layer)")
        slabs = [_byte_view(s) for s in slabs]
    qn0 = q_nope_absorbed[0]
    _require(qn0.dim() == 3, "q_nope_absorbed must be [R*n_q, H, 512]")
    T, H, _ = qn0.shape
    _require(T % n_q == 0, "first dimension must be num_reqs * n_q")
    R = T // n_q
    device = qn0.device
    want = torch.uint8 if fp8 else torch.bfloat16
    num_pages, page_stride = slabs[0].shape[0], slabs[0].stride(0)
    for l in range(L):
        _check_bf16(q_nope_absorbed[l], "q_nope_absorbed", (T, H, LATENT))
        _check_bf16(q_rope[l], "q_rope", (T, H, ROPE))
        _check_bf16(gate[l], "gate", (T, H, LATENT))
        s = slabs[l]
        _require(s.is_cuda and s.dtype == want and s.dim() == 2 and s.stride(1) == 1,
                 f"each slab must be a 2-D CUDA {want} tensor with contiguous pages")
        _require(s.shape[0] == num_pages and s.stride(0) == page_stride,
                 "the layers' slabs must share the page count and page stride")
    _require(slabs[0].shape[1] >= PAGE_TOKENS * ROW, "slab page too small")
    _require(page_table.is_cuda and page_table.dtype == torch.int32 and page_table.dim() == 2,
             "page_table must be a 2-D CUDA int32 tensor")
    _require(page_table.shape[0] == R and page_table.stride(1) == 1,
             "page_table must be [R, ld] with unit column stride")
    _require(seq_lens.is_cuda and seq_lens.dtype == torch.int32 and seq_lens.is_contiguous()
             and tuple(seq_lens.shape) == (R,), "seq_lens must be a contiguous CUDA int32 [R]")
    if out is None:
        out = [torch.empty_like(q) for q in q_nope_absorbed]
    _require(len(out) == L, "one output tensor per layer")
    for o in out:
        _check_bf16(o, "out", (T, H, LATENT))
    if lse is None and with_lse:
        lse = [torch.empty(T, H, dtype=torch.float32, device=device) for _ in range(L)]
    if lse is not None:
        _require(len(lse) == L, "one lse tensor per layer")
        for v in lse:
            _require(v is None or (v.is_cuda and v.dtype == torch.float32 and v.is_contiguous()
                                   and tuple(v.shape) == (T, H)),
                     "lse must be a contiguous CUDA fp32 [T, H] (or None)")
    if workspace is None:
        workspace = allocate_workspace(R, n_q, H, cta_budget, min_splits, device, fp8=fp8)
    _require(workspace.is_cuda and workspace.is_contiguous(), "workspace must be CUDA memory")
    nbytes = workspace.numel() * workspace.element_size()

    def ptrs(ts):
        arr = (ctypes.c_void_p * L)(*[None if t is None else t.data_ptr() for t in ts])
        return arr, ctypes.cast(arr, ctypes.c_void_p)

    keep = [ptrs(q_nope_absorbed), ptrs(q_rope), ptrs(gate), ptrs(slabs), ptrs(out)]
    lse_arr = ptrs(lse) if lse is not None else (None, None)
    lib = _native.lib()
    head = [L] + [k[1] for k in keep[:4]]
    tail = [num_pages, page_stride, page_table.data_ptr(), page_table.stride(0),
            seq_lens.data_ptr(), R, n_q, H, float(scale), keep[4][1], lse_arr[1],
            workspace.data_ptr(), nbytes, int(cta_budget), int(min_splits),
            _stream_ptr(stream, device)]
    if fp8:
        sc = (ctypes.c_float * L)(*[float(v) for v in scales])
        status = lib.mla_decode_layers_fp8(*head, ctypes.cast(sc, ctypes.c_void_p), *tail)
    else:
        status = lib.mla_decode_layers(*head, *tail)
    _native.check(status, "mla_decode_layers_fp8" if fp8 else "mla_decode_layers")
    return out, (lse if lse is not None else [None] * L)


def mla_quantize_queries_fp8(q_nope_absorbed, q_rope, stream=None):
    """The FP8 decode's query step: (hi [rows, 576] uint8, lo [rows, 576] uint8,
    exps [rows] int32) for the rows of [q_nope | q_rope] (any leading shape,
    flattened): q = (decode(hi) + decode(lo)) * 2^exp, exactly where
    |q| >= 2^(exp - 2)."""
    _require(q_nope_absorbed.is_cuda and q_nope_absorbed.dtype == torch.bfloat16
             and q_nope_absorbed.is_contiguous() and q_nope_absorbed.shape[-1] == LATENT,
             "q_nope_absorbed must be contiguous CUDA bf16 [..., 512]")
    rows = q_nope_absorbed.numel() // LATENT
    _require(q_rope.is_cuda and q_rope.dtype == torch.bfloat16 and q_rope.is_contiguous()
             and q_rope.numel() == rows * ROPE, "q_rope must be contiguous CUDA bf16 [..., 64]")
    codes = torch.empty(2, rows, ROW, dtype=torch.uint8, device=q_nope_absorbed.device)
    exps = torch.empty(rows, dtype=torch.int32, device=q_nope_absorbed.device)
    status = _native.lib().mla_quantize_queries_fp8(
        q_nope_absorbed.data_ptr(), q_rope.data_ptr(), rows, codes.data_ptr(), exps.data_ptr(),
        _stream_ptr(stream, q_nope_absorbed.device))
    _native.check(status, "mla_quantize_queries_fp8")
    return codes[0], codes[1], exps


def set_page_checks(on: bool) -> None:
    """Process-wide: check every page-table entry a decode step uses after the
    step (status 40 in the workspace's status word if one is out of range)."""
    _native.lib().mla_set_page_checks(1 if on else 0)


def get_page_checks() -> bool:
    return bool(_native.lib().mla_get_page_checks())


SPLIT_MODES = {"per-request": 0, "uniform": 1}


def set_split_mode(mode: str) -> None:
    """Process-wide split rule of the planner: "per-request" (the default) or
    "uniform" (the same split count for every request, the baseline of the
    pages' Figure 5 comparison)."""
    _require(mode in SPLIT_MODES, f"split mode must be one of {sorted(SPLIT_MODES)}")
    _native.check(_native.lib().mla_set_split_mode(SPLIT_MODES[mode]), "mla_set_split_mode")


def get_split_mode() -> str:
    m = int(_native.lib().mla_get_split_mode())
    return {v: k for k, v in SPLIT_MODES.items()}[m]


def set_team_clusters(max_teams: int) -> None:
    """Process-wide widest cluster (1, 2 or 4; default 2) of 64-row query teams
    that share each KV tile's load (TMA multicast) in the bf16 decode; the
    outputs do not depend on it."""
    _require(max_teams in (1, 2, 4), "max_teams must be 1, 2 or 4")
    _native.check(_native.lib().mla_set_team_clusters(int(max_teams)), "mla_set_team_clusters")


def get_team_clusters() -> int:
    return int(_native.lib().mla_get_team_clusters())


def device_status(workspace) -> int:
    """The decode kernel's status word from the workspace of the last step
    (0 = ok).  Reads device memory: synchronises with the workspace's stream."""
    return int(workspace[:4].view(torch.int32).item())


def mla_plan_splits(seq_lens, split_budget, stream=None):
    """Device split plan: (split_indptr [R+1] int32, chunk [1] int64)."""
    _require(seq_lens.is_cuda and seq_lens.dtype == torch.int32 and seq_lens.is_contiguous()
             and seq_lens.dim() == 1, "seq_lens must be a contiguous CUDA int32 vector")
    R = seq_lens.shape[0]
    indptr = torch.empty(R + 1, dtype=torch.int32, device=seq_lens.device)
    chunk = torch.empty(1, dtype=torch.int64, device=seq_lens.device)
    status = _native.lib().mla_plan_splits(seq_lens.data_ptr(), R, int(split_budget),
                                           indptr.data_ptr(), chunk.data_ptr(),
                                           _stream_ptr(stream, seq_lens.device))
    _native.check(status, "mla_plan_splits")
    return indptr, chunk


def mla_dcp_shard(page_table, seq_lens, world, rank, stream=None):
    """Rank `rank`'s page table and history lengths for decode context
    parallelism over `world` ranks (page column c of request r belongs to rank
    (c + r) mod world): (table_k [R, ceil(ld / world)] int32, lens_k [R] int32),
    computed on the device."""
    _require(page_table.is_cuda and page_table.dtype == torch.int32 and page_table.dim() == 2
             and page_table.stride(1) == 1, "page_table must be a CUDA int32 [R, ld] view")
    _require(seq_lens.is_cuda and seq_lens.dtype == torch.int32 and seq_lens.is_contiguous(),
             "seq_lens must be a contiguous CUDA int32 vector")
    R = seq_lens.shape[0]
    ld = page_table.stride(0)
    out_ld = max(1, -(-ld // world))
    table_k = torch.empty(R, out_ld, dtype=torch.int32, device=page_table.device)
    lens_k = torch.empty(R, dtype=torch.int32, device=page_table.device)
    _native.check(_native.lib().mla_dcp_shard(page_table.data_ptr(), ld, seq_lens.data_ptr(), R,
                                              int(world), int(rank), table_k.data_ptr(), out_ld,
                                              lens_k.data_ptr(),
                                              _stream_ptr(stream, page_table.device)),
                  "mla_dcp_shard")
    return table_k, lens_k


def mla_split_combine(o_part, lse_part, split_indptr, gate, *, n_q=1, out=None, lse=None,
                      stream=None, with_lse=True):
    """Merge chunk partials and apply the sigmoid gate; returns (out, lse)."""
    _check_bf16(gate, "gate")
    T, H, _ = gate.shape
    R = T // n_q
    rows = n_q * H
    _require(o_part.is_cuda and o_part.dtype == torch.float32 and o_part.is_contiguous()
             and o_part.dim() == 3 and o_part.shape[1:] == (rows, LATENT),
             "o_part must be contiguous CUDA fp32 [splits, n_q*H, 512]")
    _require(lse_part.is_cuda and lse_part.dtype == torch.float32 and lse_part.is_contiguous()
             and tuple(lse_part.shape) == (o_part.shape[0], rows),
             "lse_part must be contiguous CUDA fp32 [splits, n_q*H]")
    _require(split_indptr.is_cuda and split_indptr.dtype == torch.int32
             and tuple(split_indptr.shape) == (R + 1,), "split_indptr must be CUDA int32 [R+1]")
    if out is None:
        out = torch.empty_like(gate)
    if lse is None and with_lse:
        lse = torch.empty(T, H, dtype=torch.float32, device=gate.device)
    status = _native.lib().mla_split_combine(
        o_part.data_ptr(), lse_part.data_ptr(), split_indptr.data_ptr(), gate.data_ptr(), R,
        n_q, H, out.data_ptr(), lse.data_ptr() if lse is not None else None,
        _stream_ptr(stream, gate.device))
    _native.check(status, "mla_split_combine")
    return out, lse


def mla_merge_partials(out_parts, lse_parts, *, out=None, lse=None, stream=None, with_lse=True):
    """Merge the gated outputs of ranks that each decoded a disjoint part of the
    histories (decode context parallelism).  out_parts is bf16 [world, T, H, 512]
    (rank k's mla_decode output), lse_parts fp32 [world, T, H]; returns the
    merged (out [T, H, 512] bf16, lse [T, H] fp32)."""
    _require(out_parts.is_cuda and out_parts.dtype == torch.bfloat16 and out_parts.is_contiguous()
             and out_parts.dim() == 4 and out_parts.shape[-1] == LATENT,
             "out_parts must be contiguous CUDA bf16 [world, T, H, 512]")
    world, T, H, _ = out_parts.shape
    _require(lse_parts.is_cuda and lse_parts.dtype == torch.float32 and lse_parts.is_contiguous()
             and tuple(lse_parts.shape) == (world, T, H),
             "lse_parts must be contiguous CUDA fp32 [world, T, H]")
    if out is None:
        out = torch.empty(T, H, LATENT, dtype=torch.bfloat16, device=out_parts.device)
    _check_bf16(out, "out", (T, H, LATENT))
    if lse is None and with_lse:
        lse = torch.empty(T, H, dtype=torch.float32, device=out_parts.device)
    if lse is not None:
        _require(lse.is_cuda and lse.dtype == torch.float32 and lse.is_contiguous()
                 and tuple(lse.shape) == (T, H), "lse must be a contiguous CUDA fp32 [T, H]")
    status = _native.lib().mla_merge_partials(
        out_parts.data_ptr(), lse_parts.data_ptr(), world, T * H, out.data_ptr(),
        lse.data_ptr() if lse is not None else None, _stream_ptr(stream, out_parts.device))
    _native.check(status, "mla_merge_partials")
    return out, lse


def mla_kv_append_fp8(latent_new, rope_new, slab, page_table, seq_lens, n_new, *, kv_scale,
                      status=None, stream=None):
    """mla_kv_append into E4M3 pages (slab uint8 or float8_e4m3fn [num_pages,
    page_stride]): each value is stored as the E4M3 code of value / kv_scale."""
    return _append(latent_new, rope_new, _byte_view(slab), page_table, seq_lens, n_new, status,
                   stream, float(kv_scale))


def mla_kv_append(latent_new, rope_new, slab, page_table, seq_lens, n_new, *, status=None,
                  stream=None):
    """Write each request's n_new new latent / rope rows into the page pool.

    latent_new [R*n_new, 512] and rope_new [R*n_new, 64] bf16 (row r*n_new + j is
    request r's new token j); slab, page_table as for mla_decode; seq_lens [R]
    int32 histories after the append, so token j lands at position
    seq_lens[r] - n_new + j.  ``status``: optional CUDA int32 tensor of one
    element that the kernel sets to 32 (a history shorter than n_new) or 33 (a
    page ID outside the pool); such rows are skipped.  Asynchronous.
    """
    return _append(latent_new, rope_new, slab, page_table, seq_lens, n_new, status, stream,
                   None)


def _append(latent_new, rope_new, slab, page_table, seq_lens, n_new, status, stream, kv_scale):
    fp8 = kv_scale is not None
    R = int(seq_lens.shape[0]) if hasattr(seq_lens, "shape") else 0
    _require(seq_lens.is_cuda and seq_lens.dtype == torch.int32 and seq_lens.is_contiguous()
             and seq_lens.dim() == 1, "seq_lens must be a contiguous CUDA int32 vector")
    _check_bf16(latent_new, "latent_new", (R * n_new, 512))
    _check_bf16(rope_new, "rope_new", (R * n_new, 64))
    want = torch.uint8 if fp8 else torch.bfloat16
    _require(slab.is_cuda and slab.dtype == want and slab.dim() == 2 and slab.stride(1) == 1,
             f"slab must be a CUDA {want} [num_pages, page_stride] view")
    _require(slab.shape[1] >= PAGE_TOKENS * ROW, "slab page too small")
    _require(page_table.is_cuda and page_table.dtype == torch.int32 and page_table.dim() == 2
             and page_table.shape[0] == R and page_table.stride(1) == 1,
             "page_table must be a CUDA int32 [R, >= pages] view with unit column stride")
    if status is not None:
        _require(status.is_cuda and status.dtype == torch.int32 and status.numel() >= 1,
                 "status must be a CUDA int32 tensor")
    lib = _native.lib()
    head = (latent_new.data_ptr(), rope_new.data_ptr(), slab.data_ptr(), slab.shape[0],
            slab.stride(0))
    tail = (page_table.data_ptr(), page_table.stride(0), seq_lens.data_ptr(), R, int(n_new),
            None if status is None else status.data_ptr(), _stream_ptr(stream, slab.device))
    if fp8:
        rc = lib.mla_kv_append_fp8(*head, kv_scale, *tail)
    else:
        rc = lib.mla_kv_append(*head, *tail)
    _native.check(rc, "mla_kv_append_fp8" if fp8 else "mla_kv_append")


# ---------------------------------------------------------------------------
# rotary positions, accumulated weights, eviction
# ---------------------------------------------------------------------------
#
# A decode step's calls of these take a few microseconds on the device, so their
# checks are written to be quick: messages are only formatted on failure, a
# tensor's device is read as an index (-1 for host memory), and the current device
# and stream come from torch's raw accessors instead of the wrapping objects.

ROPE_LAYOUTS = {"half": 0, "interleaved": 1}
ROPE_SCALINGS = {"none": 0, "linear": 1, "by_parts": 2}
_ROPE_TYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}
_BF16, _I32, _F32, _U8 = torch.bfloat16, torch.int32, torch.float32, torch.uint8
_E4M3 = torch.float8_e4m3fn


def _fail(message):
    raise ValueError(message)


def _launch(dev, fn, where, stream, *args):
    """Calls the library with the stream as last argument, device `dev` current."""
    s = torch._C._cuda_getCurrentRawStream(dev) if stream is None else stream.cuda_stream
    if dev == torch._C._cuda_getDevice():
        status = fn(*args, s)
    else:
        with torch.cuda.device(dev):
            status = fn(*args, s)
    if status != 0:
        raise _native.PlmlaError(status, where)


def _empty(shape, dtype, device, stream):
    """New memory for a call on `stream`.  It comes from that stream's own blocks: one of
    the current stream's may still be in use there by work queued before it was freed.
    Once freed, the allocator keeps it until the caller's stream has passed too."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        t = torch.empty(shape, dtype=dtype, device=device)
    t.record_stream(torch.cuda.current_stream(device))
    return t


def _vector(t, name, dev, n):
    """A contiguous int32 vector of n elements on device `dev`."""
    if not (t.dtype is _I32 and t.get_device() == dev and t.dim() == 1 and t.shape[0] == n
            and t.is_contiguous()):
        _fail(f"{name} must be a contiguous int32 tensor [{n}] on cuda:{dev}")
    return t.data_ptr()


def _rows(t, name, dev, dtype, n):
    """(address, row stride, columns) of an [n, columns] view with unit column
    stride and rows that do not overlap."""
    shape = t.shape
    if not (t.dtype is dtype and t.get_device() == dev and len(shape) == 2 and shape[0] == n
            and shape[1] >= 1):
        _fail(f"{name} must be a {dtype} tensor [{n}, columns] on cuda:{dev}")
    ld, unit = t.stride()
    cols = shape[1]
    if n == 1:
        ld = cols
    if (unit != 1 and cols > 1) or ld < cols:
        _fail(f"{name} must have unit column stride and rows that do not overlap")
    return t.data_ptr(), ld, cols


def _dense(t, name, dev, shape, dtype=_BF16):
    if not (t.dtype is dtype and t.get_device() == dev and t.shape == shape
            and t.is_contiguous()):
        _fail(f"{name} must be a contiguous {dtype} tensor {tuple(shape)} on cuda:{dev}")
    return t.data_ptr()


def _pool(slab, fp8):
    """(address, pages, page stride) of a pool [num_pages, page_stride]."""
    shape = slab.shape
    dtype = slab.dtype
    if not ((dtype is _E4M3 or dtype is _U8 if fp8 else dtype is _BF16) and slab.is_cuda
            and len(shape) == 2 and shape[1] >= PAGE_TOKENS * ROW and slab.stride(1) == 1):
        _fail(f"slab must be a CUDA {'E4M3 (uint8 or float8_e4m3fn)' if fp8 else 'bf16'} view "
              f"[num_pages, page_stride >= {PAGE_TOKENS * ROW}] with contiguous pages")
    return slab.data_ptr(), shape[0], slab.stride(0) if shape[0] > 1 else shape[1]


def _flag(status, dev):
    if status is None:
        return None
    if not (status.dtype is _I32 and status.get_device() == dev and status.numel() >= 1):
        _fail(f"status must be an int32 tensor on cuda:{dev}")
    return status.data_ptr()


def _heads(t):
    """(token stride, head stride) of a [T, H, D] view, 0 along extents of one."""
    T, H, _ = t.shape
    ts, hs, _ = t.stride()
    return (ts if T > 1 else 0), (hs if H > 1 else 0)


def _check_apart(a, b, message):
    """Refuses two views (of one type, with contiguous rows) that share elements, or whose
    address ranges meet and whose strides do not show that they share none."""
    def span(t):
        first = t.data_ptr()
        last = sum((n - 1) * s for n, s in zip(t.shape, t.stride()))
        return first, first + (last + 1) * t.element_size()
    (a0, a1), (b0, b1) = span(a), span(b)
    if a0 >= b1 or b0 >= a1:
        return
    # rows in columns of one grid: [0, width of a) and [off, off + width of b) modulo the
    # shortest stride, of which the others are multiples
    strides = [s for t in (a, b) for n, s in zip(t.shape[:-1], t.stride()) if n > 1 and s > 0]
    step = min(strides, default=0)
    if step and all(s % step == 0 for s in strides) and (b0 - a0) % a.element_size() == 0:
        off = (b0 - a0) // a.element_size() % step
        if a.shape[-1] <= off <= step - b.shape[-1]:
            return
    _fail(message)


class RopeTable:
    """Rotary frequencies on a device (see rope_table): `turns` int64 [dim / 2],
    2^-64 turns per position; `magnitude` scales the rotated pairs."""

    def __init__(self, turns, magnitude):
        if not (turns.dtype is torch.int64 and turns.dim() == 1 and turns.is_contiguous()):
            _fail("turns must be a contiguous int64 tensor [dim / 2]")
        if not math.isfinite(magnitude):
            _fail("magnitude must be finite")
        self.turns, self.magnitude, self.dim = turns, float(magnitude), 2 * turns.numel()

    def address(self, dev, dim):
        if self.dim != dim or self.turns.get_device() != dev:
            _fail(f"the rotary table must have dim {dim} and lie on cuda:{dev}")
        return self.turns.data_ptr()


def rope_table(dim=ROPE, *, base=10000.0, scaling="none", factor=1.0, original_len=0, low=1.0,
               high=32.0, magnitude=None, device=None) -> RopeTable:
    """The rotary frequencies f_i = base^(-2 i / dim) of mla_rope and
    mla_kv_append_rope, for a context longer than the trained one divided by
    ``factor``: every one ("linear"), or by parts ("by_parts") -- pairs that turn
    fewer than ``low`` times over ``original_len`` positions are divided, those
    that turn more than ``high`` times kept, and a ramp joins the two.
    The ramp is linear in turns; some models' code has one in the pair index between
    rounded bounds.  ``magnitude`` scales the rotated pairs; by default 1, and 0.1
    ln(factor) + 1 by parts, which is meant for heads that are rotated whole: a head of
    this library has 512 elements without a position, which that factor leaves alone,
    so models with a latent part usually want ``magnitude=1`` and put the factor, squared,
    into the softmax ``scale`` of mla_decode.  Make the table once and keep it: it is
    copied to the device here."""
    if scaling not in ROPE_SCALINGS:
        _fail(f"scaling must be one of {sorted(ROPE_SCALINGS)}")
    host = torch.empty(max(dim, 0) // 2, dtype=torch.int64)
    status = _native.lib().mla_rope_turns(int(dim), float(base), ROPE_SCALINGS[scaling],
                                          float(factor), float(original_len), float(low),
                                          float(high), host.data_ptr())
    if status != 0:
        _fail(f"invalid rotary table: {_native.strerror(status)}")
    if magnitude is None:
        magnitude = 0.1 * math.log(factor) + 1.0 if scaling == "by_parts" else 1.0
    return RopeTable(host.to(device or "cuda"), magnitude)


def _no_grad(name, *tensors):
    """Refuses tensors whose gradients the call would lose without a word."""
    if torch.is_grad_enabled():
        for t in tensors:
            if t is not None and t.requires_grad:
                _fail(f"{name} is not recorded by autograd: call it under torch.no_grad() or on "
                      "detached tensors (the gradient of a rotation is mla_rope with inverse)")


def _layout(layout):
    code = ROPE_LAYOUTS.get(layout)
    if code is None:
        _fail(f"layout must be one of {sorted(ROPE_LAYOUTS)}")
    return code


def mla_rope(x, positions, table, *, layout="half", inverse=False, out=None, stream=None):
    """Rotary positions: x [T, H, D] (bf16, fp16 or fp32; any token and head
    strides, so ``q[..., 128:]`` rotates the last part of wider heads) turned by
    positions [T] int32.  ``layout`` pairs element i with i + D/2 ("half") or 2i
    with 2i + 1 ("interleaved"); ``inverse`` negates the angles, which is the
    gradient of the forward call: autograd does not record the call, so a tensor
    that requires grad is refused while gradients are recorded.  ``out`` may be x
    itself (in place); returns it (a new contiguous tensor by default)."""
    _no_grad("mla_rope", x, out)
    kind = _ROPE_TYPES.get(x.dtype)
    dev = x.get_device()
    if kind is None or dev < 0 or x.dim() != 3 or x.stride(2) != 1:
        _fail("x must be a CUDA bf16, fp16 or fp32 tensor [T, H, D] with contiguous heads")
    T, H, D = x.shape
    code = _layout(layout)
    at, turns = _vector(positions, "positions", dev, T), table.address(dev, D)
    if out is None:
        out = _empty((T, H, D), x.dtype, x.device, stream)
    else:
        _check_rope_out(x, out, dev)
    if T and H:
        _launch(dev, _native.lib().mla_rope, "mla_rope", stream, x.data_ptr(), *_heads(x), at,
                turns, table.magnitude, T, H, D, kind, code, bool(inverse), out.data_ptr(),
                *_heads(out))
    return out


def _check_rope_out(x, out, dev):
    if not (out.dtype is x.dtype and out.get_device() == dev and out.shape == x.shape
            and out.stride(2) == 1):
        _fail("out must be like x, each head contiguous")
    T, H, D = out.shape
    if T == 0 or H == 0:
        return
    ts, hs = _heads(out)
    if not ((H == 1 or hs >= D) and (T == 1 or ts >= D)
            and (T == 1 or H == 1 or ts >= (H - 1) * hs + D or hs >= (T - 1) * ts + D)):
        _fail("heads of out overlap")
    if not (out.data_ptr() == x.data_ptr() and _heads(out) == _heads(x)):
        _check_apart(x, out, "out must be x or not overlap it")


def mla_kv_append_rope(latent_new, rope_new, slab, page_table, seq_lens, n_new, table, *,
                       positions=None, layout="half", q_rope=None, q_out=None, status=None,
                       stream=None):
    """mla_kv_append of rope keys that are not rotated yet, and in the same launch
    the rotation of the same tokens' queries.  ``positions`` [R*n_new] int32 (by
    default each token's index in its history; give the true positions where a
    history has lost tokens).  ``q_rope`` bf16 [R*n_new, H, 64], any token and head
    strides, is rotated into ``q_out`` (contiguous, new by default), mla_decode's
    q_rope; returns it (None without q_rope).  As in mla_rope, a q_rope that
    requires grad is refused while gradients are recorded."""
    return _append_rope(latent_new, rope_new, slab, page_table, seq_lens, n_new, table, positions,
                        layout, q_rope, q_out, status, stream, None)


def mla_kv_append_rope_fp8(latent_new, rope_new, slab, page_table, seq_lens, n_new, table, *,
                           kv_scale, positions=None, layout="half", q_rope=None, q_out=None,
                           status=None, stream=None):
    """mla_kv_append_rope into E4M3 pages (slab and kv_scale as in
    mla_kv_append_fp8)."""
    return _append_rope(latent_new, rope_new, slab, page_table, seq_lens, n_new, table,
                        positions, layout, q_rope, q_out, status, stream, _kv_scale(kv_scale))


def _kv_scale(kv_scale):
    if not (math.isfinite(kv_scale) and kv_scale > 0):
        _fail("kv_scale must be finite and > 0")
    return float(kv_scale)


def _append_rope(latent_new, rope_new, slab, page_table, seq_lens, n_new, table, positions, layout,
                 q_rope, q_out, status, stream, kv_scale):
    _no_grad("the rotating append", q_rope, q_out)
    base, pages, page_stride = _pool(slab, kv_scale is not None)
    dev, n_new = slab.get_device(), int(n_new)
    R = seq_lens.shape[0] if seq_lens.dim() == 1 else 0
    rows = R * n_new
    lens = _vector(seq_lens, "seq_lens", dev, R)
    latent = _dense(latent_new, "latent_new", dev, (rows, LATENT))
    rope = _dense(rope_new, "rope_new", dev, (rows, ROPE))
    ids = _rows(page_table, "page_table", dev, _I32, R)
    at = None if positions is None else _vector(positions, "positions", dev, rows)
    q = (None, 0, 0, 0, None)
    if q_rope is None:
        if q_out is not None:
            _fail("q_out needs q_rope")
    else:
        shape = q_rope.shape
        if not (q_rope.dtype is _BF16 and q_rope.get_device() == dev and len(shape) == 3
                and shape[0] == rows and shape[2] == ROPE and q_rope.stride(2) == 1):
            _fail(f"q_rope must be a bf16 view [{rows}, H, {ROPE}] on cuda:{dev} with contiguous "
                  "heads")
        if q_out is None:
            q_out = _empty(shape, _BF16, q_rope.device, stream)
        else:
            _dense(q_out, "q_out", dev, shape)
            if q_out.numel():
                _check_apart(q_rope, q_out, "q_out must not overlap q_rope")
        if rows and shape[1]:
            q = (q_rope.data_ptr(), *_heads(q_rope), shape[1], q_out.data_ptr())
    tail = (*ids, lens, R, n_new, at, table.address(dev, ROPE), table.magnitude,
            _layout(layout), *q, _flag(status, dev))
    lib = _native.lib()
    if kv_scale is not None:
        _launch(dev, lib.mla_kv_append_rope_fp8_ex, "mla_kv_append_rope_fp8", stream, latent, rope,
                base, pages, page_stride, kv_scale, *tail)
    else:
        _launch(dev, lib.mla_kv_append_rope_ex, "mla_kv_append_rope", stream, latent, rope, base,
                pages, page_stride, *tail)
    return q_out


def allocate_mass_workspace(num_reqs, n_q, num_heads, device=None):
    """A workspace tensor (uint8) of the size mla_attention_mass_fp8 needs."""
    n = _native.lib().mla_mass_workspace_size_fp8(num_reqs, n_q, num_heads)
    if n == 0:
        _fail("invalid shape for mla_mass_workspace_size_fp8")
    return torch.empty(n, dtype=_U8, device=device or "cuda")


def mla_attention_mass(q_nope_absorbed, q_rope, lse, slab, page_table, seq_lens, mass, *, n_q=1,
                       scale=DEFAULT_SCALE, decay=1.0, status=None, stream=None):
    """Adds to mass [R, tokens] fp32 the attention weight that this step's query
    rows gave every cached token (decay * mass + the sum over drafts and heads);
    returns mass.  The entry of a token that is new in its history must hold 0: make
    mass with zeros, as wide as the histories may become.  The queries, pool and histories are mla_decode's, ``lse`` is
    what it returned.  Layers that share a page table accumulate into one mass, a
    call each (with the step's decay in the first of
    these calls and 1 in the others); ``decay`` 0 overwrites.  Scores are fp32 sums: the
    weights are within 3e-7 (2-norm, N(0, 1) rows) of 64-bit arithmetic.  ``status``: optional CUDA int32 tensor of
    one element that the kernel sets to 33 or 34 where a history leaves the page
    table, the pool or its row of mass.  Asynchronous."""
    return _mass(q_nope_absorbed, q_rope, lse, slab, page_table, seq_lens, mass, n_q, scale, decay,
                 None, None, status, stream)


def mla_attention_mass_fp8(q_nope_absorbed, q_rope, lse, slab, page_table, seq_lens, mass, *,
                           kv_scale, n_q=1, scale=DEFAULT_SCALE, decay=1.0, workspace=None,
                           status=None, stream=None):
    """mla_attention_mass over E4M3 pages (slab and kv_scale as in mla_decode_fp8).
    The queries are taken in two E4M3 parts, as in mla_decode_fp8: exact for elements
    above 2^-2 of their row's scale, within 2^-10 of it below.
    The workspace comes from allocate_mass_workspace (a new one by default); calls
    that may run at once need one each."""
    return _mass(q_nope_absorbed, q_rope, lse, slab, page_table, seq_lens, mass, n_q,
                 scale, decay, _kv_scale(kv_scale), workspace, status, stream)


def _mass(q_nope_absorbed, q_rope, lse, slab, page_table, seq_lens, mass, n_q, scale, decay,
          kv_scale, workspace, status, stream):
    base, pages, page_stride = _pool(slab, kv_scale is not None)
    dev, n_q = slab.get_device(), int(n_q)
    shape = q_nope_absorbed.shape
    if len(shape) != 3 or n_q < 1 or shape[0] % n_q != 0:
        _fail("q_nope_absorbed must be [R*n_q, H, 512]")
    T, H, _ = shape
    R = T // n_q
    qn = _dense(q_nope_absorbed, "q_nope_absorbed", dev, (T, H, LATENT))
    qr = _dense(q_rope, "q_rope", dev, (T, H, ROPE))
    l = _dense(lse, "lse", dev, (T, H), _F32)
    ids = _rows(page_table, "page_table", dev, _I32, R)
    lens = _vector(seq_lens, "seq_lens", dev, R)
    out = _rows(mass, "mass", dev, _F32, R)
    flag = _flag(status, dev)
    lib = _native.lib()
    tail = (*ids, lens, R, n_q, H, float(scale), float(decay), *out)
    if kv_scale is None:
        _launch(dev, lib.mla_attention_mass_ex, "mla_attention_mass", stream, qn, qr, l, base,
                pages, page_stride, *tail, flag)
    else:
        if workspace is None:
            size = lib.mla_mass_workspace_size_fp8(R, n_q, H)
            workspace = _empty(size, _U8, slab.device, stream)
        if workspace.get_device() != dev or not workspace.is_contiguous():
            _fail(f"workspace must be contiguous memory on cuda:{dev}")
        _launch(dev, lib.mla_attention_mass_fp8_ex, "mla_attention_mass_fp8", stream, qn, qr, l,
                base, pages, page_stride, kv_scale, *tail, workspace.data_ptr(),
                workspace.numel() * workspace.element_size(), flag)
    return mass


def _evict_workspace_size(dev, num_reqs, tokens):
    """The size depends on the device that the call will run on."""
    size = _native.lib().mla_evict_workspace_size
    if dev == torch._C._cuda_getDevice():
        return size(num_reqs, tokens)
    with torch.cuda.device(dev):
        return size(num_reqs, tokens)


def allocate_evict_workspace(num_reqs, tokens, device=None):
    """A workspace tensor (uint8) for mla_evict_select on mass [num_reqs, tokens] (of
    no bytes where that shape makes no use of one)."""
    device = torch.device(device or "cuda")
    dev = torch.cuda.current_device() if device.index is None else device.index
    return torch.empty(_evict_workspace_size(dev, num_reqs, tokens), dtype=_U8, device=device)


def mla_evict_select(mass, seq_lens, keep, *, sink=0, recent=0, kept=None, kept_lens=None,
                     workspace=None, status=None, stream=None):
    """Which tokens of each history stay within ``keep``: the first ``sink``, the
    last ``recent`` and the heaviest of the rest by mass [R, tokens] fp32 (ties to
    the lower index).  Returns (kept [R, min(keep, tokens)] int32 ascending
    indices, kept_lens [R] int32 = min(keep, seq_lens)); entries of kept past a
    row's count are not written, and neither may overlap an input.  A history longer than its row of mass is taken as
    ``tokens`` long and loses its newest tokens, ``recent`` or not: ``status``, an
    optional CUDA int32 tensor of one element, is then set to 34.  The workspace
    comes from allocate_evict_workspace (a new one by default); calls that may run
    at once need one each.  Asynchronous."""
    dev = mass.get_device()
    if mass.dim() != 2 or dev < 0:
        _fail("mass must be a CUDA tensor [R, tokens]")
    R, tokens = mass.shape
    keep, sink, recent = int(keep), int(sink), int(recent)
    weights = _rows(mass, "mass", dev, _F32, R)
    lens = _vector(seq_lens, "seq_lens", dev, R)
    if not (1 <= keep < 1 << 31 and sink >= 0 and recent >= 0 and sink + recent <= keep):
        _fail("keep >= 1, sink and recent >= 0, and sink + recent <= keep are needed")
    cols = min(keep, tokens)
    if kept is None:
        kept = _empty((R, cols), _I32, mass.device, stream)
    if kept_lens is None:
        kept_lens = _empty(R, _I32, mass.device, stream)
    counts = _vector(kept_lens, "kept_lens", dev, R)
    if abs(counts - lens) < 4 * R:
        _fail("kept_lens must not overlap seq_lens")
    ids, ids_ld, have = _rows(kept, "kept", dev, _I32, R)
    if have < cols:
        _fail(f"kept needs {cols} columns")
    lib, scratch, size = _native.lib(), None, 0
    if workspace is None:
        size = _evict_workspace_size(dev, R, tokens)
        if size:
            workspace = _empty(size, _U8, mass.device, stream)
    elif workspace.get_device() != dev or not workspace.is_contiguous():
        _fail(f"workspace must be contiguous memory on cuda:{dev}")
    if workspace is not None and workspace.numel():
        scratch, size = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    _launch(dev, lib.mla_evict_select_ex, "mla_evict_select", stream, *weights, lens, R, keep,
            sink, recent, ids, ids_ld, counts, scratch, size, _flag(status, dev))
    return kept, kept_lens


def mla_kv_compact(slabs, page_table, seq_lens, out_table, kept, kept_lens, *, mass=None,
                   mass_out=None, status=None, stream=None):
    """Copies each history's kept rows (kept, kept_lens from mla_evict_select), for
    every layer's pool in ``slabs`` (bf16, or uint8 / float8_e4m3fn), into the
    fresh pages of out_table [R, columns]: row i of the new history is token
    kept[r, i].  The fresh pages must be distinct and none of those read.  ``mass``
    rows are carried into ``mass_out`` (by default a new tensor as wide as mass, so
    that the histories can grow again, with zeros where the next tokens' weights
    come; in a given one those entries stay as they are and have to be 0); returns
    mass_out (None without mass).  ``status``: optional CUDA int32 tensor of one
    element, set to 33 where an index or page is out of range (such rows are
    skipped), to 34 where a kept token has no weight in mass (its row is copied).
    The old pages are not changed.  Asynchronous."""
    if not isinstance(slabs, (list, tuple)) or not slabs:
        _fail("slabs must be a list of pools")
    first = slabs[0]
    dtype, fp8 = first.dtype, first.dtype is not _BF16
    base, pages, page_stride = _pool(first, fp8)
    dev, layers = first.get_device(), len(slabs)
    bases = (ctypes.c_void_p * layers)(base)
    shape, strides = first.shape, first.stride()
    for i in range(1, layers):
        s = slabs[i]
        if not (s.dtype is dtype and s.get_device() == dev and s.shape == shape
                and s.stride() == strides):
            _fail("the layers' slabs must share their type, shape and strides")
        bases[i] = s.data_ptr()
    if kept.dim() != 2:
        _fail("kept must be [R, columns]")
    R = kept.shape[0]
    idx, idx_ld, cols = _rows(kept, "kept", dev, _I32, R)
    ids = _rows(page_table, "page_table", dev, _I32, R)
    outs = _rows(out_table, "out_table", dev, _I32, R)
    carried = (None, 0, 0, None, 0)
    if mass is None:
        if mass_out is not None:
            _fail("mass_out needs mass")
    else:
        weights = _rows(mass, "mass", dev, _F32, R)
        if mass_out is None:
            mass_out = _empty((R, max(cols, weights[2])), _F32, mass.device, stream)
            with torch.cuda.stream(stream):
                mass_out.zero_()
        dst, dst_ld, have = _rows(mass_out, "mass_out", dev, _F32, R)
        if have < cols:
            _fail(f"mass_out needs {cols} columns")
        _check_apart(mass, mass_out, "mass_out must not overlap mass")
        carried = (*weights, dst, dst_ld)
    _launch(dev, _native.lib().mla_kv_compact_ex, "mla_kv_compact", stream, layers, bases,
            1 if fp8 else 2, pages, page_stride, *ids,
            _vector(seq_lens, "seq_lens", dev, R), *outs, idx, idx_ld,
            _vector(kept_lens, "kept_lens", dev, R), R, cols, *carried, _flag(status, dev))
    return mass_out
