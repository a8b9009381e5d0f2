"""Flash-dLLM per-layer hot path on NVIDIA B200 (sm_100a).

Python binding over the C ABI of libfdllm.so (include/fdllm.h). Functions
carry the C names; they only marshal torch tensors (device memory and the
current CUDA stream) into pointers. The layer step itself, the attention
mass and the top-k selection all run in the library's CUDA kernels; if the
library is missing or no GPU is present the calls raise.

Sources: "Flash-dLLM: I/O-Aware KV Caching and Parallel Decoding for Fast,
Memory-Efficient Diffusion LLMs" (ai4snews summary of the full text),
paragraphs 1-3 (Flash-Cache fusion, scheduled attention with a block table,
tracking budget, Flash-Verify two-view mask).
"""
from __future__ import annotations

import ctypes
from typing import Optional, Sequence

import numpy as np
import torch

from . import _lib
from ._lib import (FDLLM_BF16, FDLLM_F32, FDLLM_OK, CacheConfig, FdllmError, Step,  # noqa: F401
                   check_status, load)

__all__ = [
    "fdllm_cache_create", "fdllm_cache_destroy", "fdllm_layer_step", "fdllm_layer_step_noalloc",
    "fdllm_select_tracked", "fdllm_verify_accept", "fdllm_plan_tile_schedule", "fdllm_oproj",
    "fdllm_plan_blocks", "fdllm_release_blocks", "fdllm_plan_buffers", "fdllm_decode_attention",
    "fdllm_rope_tables", "fdllm_linear",
    "fdllm_check", "fdllm_inject_fault", "fdllm_inject_tile_timeout", "fdllm_last_launch_count",
    "FlashCache", "FdllmError",
    "load",
]


def _stream_ptr(stream) -> int:
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def _dev_ptr(t: Optional[torch.Tensor], dtype=None, name="tensor") -> Optional[int]:
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    return t.data_ptr()


def _out_bf16(out: Optional[torch.Tensor]) -> int:
    """1 for a bf16 `out`, 0 for fp32; anything else is refused."""
    if out is None or out.dtype == torch.float32:
        return 0
    if out.dtype == torch.bfloat16:
        return 1
    raise ValueError(f"out must be float32 or bfloat16, got {out.dtype}")


def _host_i32(a) -> np.ndarray:
    return np.ascontiguousarray(np.asarray(a, dtype=np.int32))


def fdllm_cache_create(n_layers: int, n_heads: int, head_dim: int, page_size: int,
                       num_pages: int, max_position: int, rope_theta: float, dtype: str,
                       k_pool: torch.Tensor, v_pool: torch.Tensor, max_batch: int,
                       max_slots_per_seq: int, stream=None) -> int:
    """Returns an opaque handle (int) over the caller's K/V pools."""
    lib = load()
    tdt = torch.bfloat16 if dtype == "bf16" else torch.float32
    cfg = CacheConfig(n_layers, n_heads, head_dim, page_size, num_pages, max_position, max_batch,
                      max_slots_per_seq, float(rope_theta),
                      FDLLM_BF16 if dtype == "bf16" else FDLLM_F32)
    shape = (n_layers, num_pages, n_heads, page_size, head_dim)
    for nm, p in (("k_pool", k_pool), ("v_pool", v_pool)):
        if tuple(p.shape) != shape:
            raise ValueError(f"{nm} must have shape {shape}, got {tuple(p.shape)}")
    out = ctypes.c_void_p()
    check_status(lib.fdllm_cache_create(ctypes.byref(cfg), _dev_ptr(k_pool, tdt, "k_pool"),
                                        _dev_ptr(v_pool, tdt, "v_pool"), _stream_ptr(stream),
                                        ctypes.byref(out)))
    return out.value


def fdllm_cache_destroy(handle: int) -> None:
    if handle:
        load().fdllm_cache_destroy(handle)


def fdllm_layer_step(handle: int, layer: int, cu_rows: Sequence[int], seq_lens: Sequence[int],
                     max_blocks_per_seq: int, x: torch.Tensor, wqkv: torch.Tensor,
                     positions: torch.Tensor, block_table: torch.Tensor,
                     view_mask: Optional[torch.Tensor], out: torch.Tensor,
                     attn_mass: Optional[torch.Tensor], slots: Optional[torch.Tensor] = None,
                     validate: bool = False, stream=None) -> None:
    """One Flash-Cache + scheduled-attention layer step (see include/fdllm.h).

    cu_rows, seq_lens: host integer sequences; all tensors on the device."""
    lib = load()
    cu = _host_i32(cu_rows)
    sl = _host_i32(seq_lens)
    st = Step(len(sl), int(cu[-1]), int(max_blocks_per_seq),
              cu.ctypes.data_as(ctypes.POINTER(ctypes.c_int32)),
              sl.ctypes.data_as(ctypes.POINTER(ctypes.c_int32)),
              _dev_ptr(slots, torch.int32, "slots"), 1 if validate else 0, _out_bf16(out))
    check_status(lib.fdllm_layer_step(
        handle, int(layer), ctypes.byref(st), _dev_ptr(x, None, "x"), _dev_ptr(wqkv, None, "wqkv"),
        _dev_ptr(positions, torch.int32, "positions"), _dev_ptr(block_table, torch.int32, "block_table"),
        _dev_ptr(view_mask, torch.int8, "view_mask"), _dev_ptr(out, None, "out"),
        _dev_ptr(attn_mass, torch.float32, "attn_mass"), _stream_ptr(stream)))


def fdllm_layer_step_noalloc(n_layers: int, n_heads: int, head_dim: int, page_size: int,
                             num_pages: int, max_position: int, rope_theta: float, dtype: str,
                             max_batch: int, max_slots_per_seq: int, k_pool: torch.Tensor,
                             v_pool: torch.Tensor, rope_cos: torch.Tensor, rope_sin: torch.Tensor,
                             layer: int, cu_rows: Sequence[int], seq_lens: Sequence[int],
                             max_blocks_per_seq: int, x: torch.Tensor, wqkv: torch.Tensor,
                             positions: torch.Tensor, block_table: torch.Tensor,
                             view_mask: Optional[torch.Tensor], out: torch.Tensor,
                             attn_mass: Optional[torch.Tensor],
                             slots: Optional[torch.Tensor] = None, validate: bool = False,
                             stream=None) -> None:
    """The layer step without a handle or any device allocation, for callers
    that cannot call cudaMalloc when they step (their HBM is already handed
    to a KV pool or to their own allocator). The library keeps its scratch
    in a fixed per-device array; overlapping calls on one GPU race on it.
    rope_cos / rope_sin: caller-owned fp64 [max_position][head_dim / 2]
    tables (see include/fdllm.h)."""
    lib = load()
    tdt = torch.bfloat16 if dtype == "bf16" else torch.float32
    cfg = CacheConfig(n_layers, n_heads, head_dim, page_size, num_pages, max_position, max_batch,
                      max_slots_per_seq, float(rope_theta),
                      FDLLM_BF16 if dtype == "bf16" else FDLLM_F32)
    half = head_dim // 2
    for nm, t in (("rope_cos", rope_cos), ("rope_sin", rope_sin)):
        if tuple(t.shape) != (max_position, half):
            raise ValueError(f"{nm} must have shape {(max_position, half)}, got {tuple(t.shape)}")
    cu = _host_i32(cu_rows)
    sl = _host_i32(seq_lens)
    st = Step(len(sl), int(cu[-1]), int(max_blocks_per_seq),
              cu.ctypes.data_as(ctypes.POINTER(ctypes.c_int32)),
              sl.ctypes.data_as(ctypes.POINTER(ctypes.c_int32)),
              _dev_ptr(slots, torch.int32, "slots"), 1 if validate else 0, _out_bf16(out))
    check_status(lib.fdllm_layer_step_noalloc(
        ctypes.byref(cfg), _dev_ptr(k_pool, tdt, "k_pool"), _dev_ptr(v_pool, tdt, "v_pool"),
        _dev_ptr(rope_cos, torch.float64, "rope_cos"), _dev_ptr(rope_sin, torch.float64, "rope_sin"),
        int(layer), ctypes.byref(st), _dev_ptr(x, None, "x"), _dev_ptr(wqkv, None, "wqkv"),
        _dev_ptr(positions, torch.int32, "positions"), _dev_ptr(block_table, torch.int32, "block_table"),
        _dev_ptr(view_mask, torch.int8, "view_mask"), _dev_ptr(out, None, "out"),
        _dev_ptr(attn_mass, torch.float32, "attn_mass"), _stream_ptr(stream)))


def fdllm_select_tracked(attn_mass: torch.Tensor, seq_lens: torch.Tensor, k: int,
                         exclude_cu: Optional[torch.Tensor] = None,
                         exclude_slots: Optional[torch.Tensor] = None,
                         tracked: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Top-k most attended slots per sequence (see include/fdllm.h)."""
    lib = load()
    B, stride = attn_mass.shape
    if tracked is None:
        tracked = torch.empty(B, k, dtype=torch.int32, device=attn_mass.device)
    check_status(lib.fdllm_select_tracked(
        _dev_ptr(attn_mass, torch.float32, "attn_mass"), _dev_ptr(seq_lens, torch.int32, "seq_lens"),
        int(B), int(stride), int(k), _dev_ptr(exclude_cu, torch.int32, "exclude_cu"),
        _dev_ptr(exclude_slots, torch.int32, "exclude_slots"), _dev_ptr(tracked, torch.int32, "tracked"),
        _stream_ptr(stream)))
    return tracked


def fdllm_verify_accept(mask_logits: torch.Tensor, cu_rows: torch.Tensor,
                        draft_tokens: torch.Tensor, tau: float, pred: Optional[torch.Tensor] = None,
                        conf: Optional[torch.Tensor] = None,
                        n_accepted: Optional[torch.Tensor] = None, stream=None):
    """Flash-Verify acceptance (see include/fdllm.h): returns (pred, conf,
    n_accepted) for mask-view logits [rows, vocab] (bf16 or fp32)."""
    lib = load()
    if mask_logits.dtype not in (torch.bfloat16, torch.float32):
        raise ValueError("mask_logits must be bf16 or fp32")
    rows, vocab = mask_logits.shape
    batch = int(cu_rows.numel()) - 1
    dev = mask_logits.device
    if pred is None:
        pred = torch.empty(rows, dtype=torch.int32, device=dev)
    if conf is None:
        conf = torch.empty(rows, dtype=torch.float32, device=dev)
    if n_accepted is None:
        n_accepted = torch.empty(batch, dtype=torch.int32, device=dev)
    check_status(lib.fdllm_verify_accept(
        _dev_ptr(mask_logits, None, "mask_logits"),
        FDLLM_BF16 if mask_logits.dtype == torch.bfloat16 else FDLLM_F32, int(rows), int(vocab),
        _dev_ptr(cu_rows, torch.int32, "cu_rows"), batch,
        _dev_ptr(draft_tokens, torch.int32, "draft_tokens"), float(tau),
        _dev_ptr(pred, torch.int32, "pred"), _dev_ptr(conf, torch.float32, "conf"),
        _dev_ptr(n_accepted, torch.int32, "n_accepted"), _stream_ptr(stream)))
    return pred, conf, n_accepted


def fdllm_plan_tile_schedule(group_cost: Sequence[float], n_heads: int, n_bins: int):
    """The bf16 step's static tile schedule (see include/fdllm.h): returns
    (bin_start [n_bins + 1], tiles [n_groups * n_heads]) as int32 arrays;
    tile t is group t // n_heads, head t % n_heads. Host only."""
    lib = load()
    cost = np.ascontiguousarray(np.asarray(group_cost, dtype=np.float64))
    n_groups = int(cost.size)
    bin_start = np.zeros(max(int(n_bins), 0) + 1, np.int32)
    tiles = np.zeros(max(n_groups * int(n_heads), 0), np.int32)
    check_status(lib.fdllm_plan_tile_schedule(
        cost.ctypes.data if n_groups else None, n_groups, int(n_heads), int(n_bins),
        bin_start.ctypes.data, tiles.ctypes.data if tiles.size else None))
    return bin_start, tiles


def fdllm_oproj(attn_out: torch.Tensor, w_o: torch.Tensor, y: Optional[torch.Tensor] = None,
                status: Optional[torch.Tensor] = None, stream=None,
                residual: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Output projection y = residual + attn_out W_o (see include/fdllm.h):
    bf16 [rows, hidden] times bf16 [hidden, hidden], bf16 result; residual
    is optional and may be y itself."""
    lib = load()
    rows, hidden = attn_out.shape
    if tuple(w_o.shape) != (hidden, hidden):
        raise ValueError(f"w_o must be [{hidden}, {hidden}], got {tuple(w_o.shape)}")
    if residual is not None and tuple(residual.shape) != (rows, hidden):
        raise ValueError(f"residual must be [{rows}, {hidden}], got {tuple(residual.shape)}")
    if y is None:
        y = torch.empty(rows, hidden, dtype=torch.bfloat16, device=attn_out.device)
    check_status(lib.fdllm_oproj(
        _dev_ptr(attn_out, torch.bfloat16, "attn_out"), _dev_ptr(w_o, torch.bfloat16, "w_o"),
        _dev_ptr(residual, torch.bfloat16, "residual"), _dev_ptr(y, torch.bfloat16, "y"),
        int(rows), int(hidden), _dev_ptr(status, torch.int32, "status"), _stream_ptr(stream)))
    return y


# ---------------------------------------------------------------- single-token serving
_ACTS = {"none": 0, "relu": 1, "silu": 2, "gelu": 3, "gelu_tanh": 4}
_bound = None


def _native():
    """The native marshalling module over the loaded library."""
    global _bound, _serve
    lib = load()
    if _bound is not lib:
        try:
            from . import _serve
        except ImportError as e:
            raise ImportError("_serve.so is missing or does not load: build it with "
                              "`python -m kv_cache_attention_flash_b200.build`") from e
        _serve.bind(*(ctypes.cast(getattr(lib, n), ctypes.c_void_p).value for n in (
            "fdllm_plan_step", "fdllm_release_blocks", "fdllm_decode_workspace_bytes",
            "fdllm_decode_attention", "fdllm_linear")))
        _bound = lib
    return _serve


def _on(stream, t: torch.Tensor):
    """The context in which `stream` is current on t's device, so that what a
    call allocates belongs to the stream that uses it."""
    if not t.is_cuda:
        raise ValueError("the tensors must be CUDA tensors")
    if isinstance(stream, torch.cuda.Stream):
        s = stream
    elif int(stream) == 0:
        s = torch.cuda.default_stream(t.device)
    else:
        s = torch.cuda.ExternalStream(int(stream), t.device)
    if s.device != t.device:
        raise ValueError(f"stream is on {s.device}, the tensors on {t.device}")
    return torch.cuda.stream(s)


def _is_f32(dtype) -> bool:
    if dtype is torch.float32:
        return True
    if dtype is torch.bfloat16:
        return False
    raise ValueError(f"out_dtype must be float32 or bfloat16, got {dtype}")


def fdllm_plan_buffers(batch: int, capacity: int, device="cuda") -> dict:
    """The outputs of fdllm_plan_blocks for `batch` requests (no more and no
    fewer: slices of larger ones will do) and up to `capacity` rows, to be kept
    and passed as `out`."""
    i32 = dict(dtype=torch.int32, device=device)
    return {"cu_rows": torch.empty(batch + 1, **i32), "positions": torch.empty(capacity, **i32),
            "slots": torch.empty(capacity, **i32), "row_seq": torch.empty(capacity, **i32),
            "slot_map": torch.empty(capacity, dtype=torch.int64, device=device),
            "seq_lens": torch.empty(batch, **i32), "granted": torch.empty(batch, **i32),
            "n_free": torch.empty(1, **i32), "headroom": torch.empty(1, **i32),
            "seq_positions": torch.empty(batch, **i32), "seq_slots": torch.empty(batch, **i32)}


def fdllm_plan_blocks(seq_lens: torch.Tensor, new_lens: torch.Tensor, block_table: torch.Tensor,
                      page_size: int, free_pages: torch.Tensor, n_free: torch.Tensor,
                      capacity: Optional[int] = None, out: Optional[dict] = None,
                      status: Optional[torch.Tensor] = None, stream=None) -> dict:
    """Block tables, positions and slot maps of a step, pages taken from the
    free list (see include/fdllm.h); block_table is updated in place.

    out: buffers as fdllm_plan_buffers gives them ("headroom", "seq_positions"
    and "seq_slots" may be left out); without it, `capacity` (room for the
    step's rows) is needed. Returns them. "positions" and "slots" have an entry
    for each new row; for fdllm_decode_attention take "seq_positions" and
    "seq_slots", which have one for each request, also for one without a row."""
    if stream is not None:
        with _on(stream, block_table):
            return fdllm_plan_blocks(seq_lens, new_lens, block_table, page_size, free_pages, n_free,
                                     capacity, out, status)
    if out is None:
        if capacity is None:
            raise ValueError("capacity (room for the step's rows) or out is needed")
        out = fdllm_plan_buffers(block_table.shape[0], capacity, block_table.device)
    r = _native().plan_blocks(seq_lens, new_lens, block_table, page_size, free_pages, n_free, out,
                              status)
    if r:
        check_status(r)
    return out


def fdllm_release_blocks(seq_lens: torch.Tensor, keep_lens: torch.Tensor,
                         block_table: torch.Tensor, page_size: int, free_pages: torch.Tensor,
                         n_free: torch.Tensor, out: Optional[dict] = None,
                         status: Optional[torch.Tensor] = None, stream=None) -> dict:
    """Pages past each request's first keep_lens tokens go back onto the free
    list (see include/fdllm.h); free_pages is updated in place. Returns the
    new "seq_lens" and "n_free" (in `out`, when given)."""
    if stream is not None:
        with _on(stream, block_table):
            return fdllm_release_blocks(seq_lens, keep_lens, block_table, page_size, free_pages,
                                        n_free, out, status)
    if out is None:
        dev = block_table.device
        out = {"seq_lens": torch.empty(block_table.shape[0], dtype=torch.int32, device=dev),
               "n_free": torch.empty(1, dtype=torch.int32, device=dev)}
    r = _native().release_blocks(seq_lens, keep_lens, block_table, page_size, free_pages, n_free,
                                 out, status)
    if r:
        check_status(r)
    return out


def fdllm_rope_tables(max_position: int, head_dim: int, rope_theta: float, device="cuda"):
    """(cos, sin), fp64 [max_position, head_dim / 2], of the angles
    p * rope_theta^(-2i / head_dim): the tables that fdllm_cache_create
    builds."""
    inv = float(rope_theta) ** (-2.0 * np.arange(head_dim // 2) / head_dim)
    angle = np.arange(max_position, dtype=np.float64)[:, None] * inv
    return (torch.from_numpy(np.cos(angle)).to(device), torch.from_numpy(np.sin(angle)).to(device))


def fdllm_decode_attention(q: torch.Tensor, k_pool: torch.Tensor, v_pool: torch.Tensor, layer: int,
                           block_table: torch.Tensor, seq_lens: torch.Tensor,
                           k: Optional[torch.Tensor] = None, v: Optional[torch.Tensor] = None,
                           positions: Optional[torch.Tensor] = None,
                           slots: Optional[torch.Tensor] = None,
                           rope_cos: Optional[torch.Tensor] = None,
                           rope_sin: Optional[torch.Tensor] = None,
                           starts: Optional[torch.Tensor] = None, scale: Optional[float] = None,
                           out: Optional[torch.Tensor] = None, out_dtype=torch.float32,
                           lse: Optional[torch.Tensor] = None, with_lse: bool = False,
                           workspace: Optional[torch.Tensor] = None,
                           status: Optional[torch.Tensor] = None, stream=None):
    """Attention of one new token a sequence over its pages, with RoPE and
    the cache write of its k and v (see include/fdllm.h).

    q: [B, n_heads * D]; k, v: [B, n_kv_heads * D] (rows may be strided, so
    that the three can be slices of one projection). The pools give the
    layout [n_layers, num_pages, n_kv_heads, page_size, D]. positions, slots:
    [B], "seq_positions" and "seq_slots" of fdllm_plan_blocks. scale: default
    1 / sqrt(D). Returns (out [B, n_heads * D], lse [B, n_heads] or None).
    workspace: a uint8 tensor of fdllm_decode_workspace_bytes, else one is
    allocated for the call."""
    if stream is not None:
        with _on(stream, k_pool):
            return fdllm_decode_attention(q, k_pool, v_pool, layer, block_table, seq_lens, k, v,
                                          positions, slots, rope_cos, rope_sin, starts, scale, out,
                                          out_dtype, lse, with_lse, workspace, status)
    r, out, lse = _native().decode_attention(
        q, k_pool, v_pool, layer, block_table, seq_lens, k, v, positions, slots, rope_cos, rope_sin,
        starts, scale, out, _is_f32(out_dtype), lse, bool(with_lse), workspace, status)
    if r:
        check_status(r)
    return out, lse


def fdllm_linear(x: torch.Tensor, w: torch.Tensor, bias: Optional[torch.Tensor] = None,
                 act: str = "none", w_gate: Optional[torch.Tensor] = None,
                 bias_gate: Optional[torch.Tensor] = None,
                 residual: Optional[torch.Tensor] = None, y: Optional[torch.Tensor] = None,
                 out_dtype=torch.bfloat16, status: Optional[torch.Tensor] = None,
                 stream=None) -> torch.Tensor:
    """y = residual + act(x w + bias), or with w_gate
    y = residual + act(x w_gate + bias_gate) * (x w + bias) (see
    include/fdllm.h): bf16 x [rows, n_in] and w [n_in, n_out]; act one of
    none, relu, silu, gelu, gelu_tanh; rows of x, residual and y may be
    strided; residual may be y itself. y is bf16 or fp32."""
    if stream is not None:
        with _on(stream, x):
            return fdllm_linear(x, w, bias, act, w_gate, bias_gate, residual, y, out_dtype, status)
    if act not in _ACTS:
        raise ValueError(f"act must be one of {sorted(_ACTS)}, got {act!r}")
    r, y = _native().linear(x, w, bias, _ACTS[act], w_gate, bias_gate, residual, y,
                            _is_f32(out_dtype), status)
    if r:
        check_status(r)
    return y


def fdllm_check(handle: int, stream=None) -> None:
    """Synchronises the stream and raises FdllmError on a device-side error."""
    check_status(load().fdllm_check(handle, _stream_ptr(stream)))


def fdllm_inject_fault(handle: int, kind: int, wait_ns: int = 0) -> None:
    """Arms a host-made failure for the handle's next split-tile step (see
    include/fdllm.h: the attending CTAs' bounded flag wait runs out after
    wait_ns and the step records FDLLM_ERR_TIMEOUT)."""
    check_status(load().fdllm_inject_fault(handle, int(kind), int(wait_ns)))


def fdllm_inject_tile_timeout(wait_ns: int = 0) -> None:
    """Makes the waits of this thread's next fdllm_decode_attention or
    fdllm_linear run out after wait_ns (see include/fdllm.h); 0 cancels it."""
    check_status(load().fdllm_inject_tile_timeout(int(wait_ns)))


def fdllm_last_launch_count() -> int:
    return int(load().fdllm_last_launch_count())


class FlashCache:
    """Owns K/V pools (torch device memory) and the library handle."""

    def __init__(self, n_layers: int, n_heads: int, head_dim: int, page_size: int,
                 num_pages: int, max_position: int, rope_theta: float, dtype: str,
                 max_batch: int, max_slots_per_seq: int, k_pool: Optional[torch.Tensor] = None,
                 v_pool: Optional[torch.Tensor] = None, device="cuda"):
        tdt = torch.bfloat16 if dtype == "bf16" else torch.float32
        shape = (n_layers, num_pages, n_heads, page_size, head_dim)
        self.k_pool = k_pool if k_pool is not None else torch.zeros(shape, dtype=tdt, device=device)
        self.v_pool = v_pool if v_pool is not None else torch.zeros(shape, dtype=tdt, device=device)
        self.page_size = page_size
        self.n_heads = n_heads
        self.head_dim = head_dim
        self.max_position = max_position
        self.rope_theta = rope_theta
        self._rope = None
        # what decode() meets on the device, for check()
        self.status = torch.zeros(1, dtype=torch.int32, device=self.k_pool.device)
        self.handle = fdllm_cache_create(n_layers, n_heads, head_dim, page_size, num_pages,
                                         max_position, rope_theta, dtype, self.k_pool, self.v_pool,
                                         max_batch, max_slots_per_seq)

    def step(self, layer, cu_rows, seq_lens, x, wqkv, positions, block_table, view_mask=None,
             slots=None, with_mass=True, out=None, attn_mass=None, validate=False, stream=None):
        R = int(cu_rows[-1])
        B = len(seq_lens)
        mb = int(block_table.shape[1])
        if out is None:
            out = torch.empty(R, self.n_heads * self.head_dim, dtype=torch.float32, device=x.device)
        if with_mass and attn_mass is None:
            attn_mass = torch.empty(B, mb * self.page_size, dtype=torch.float32, device=x.device)
        fdllm_layer_step(self.handle, layer, cu_rows, seq_lens, mb, x, wqkv, positions, block_table,
                         view_mask, out, attn_mass if with_mass else None, slots, validate, stream)
        return out, (attn_mass if with_mass else None)

    def rope_tables(self):
        """The cache's RoPE tables as tensors (built at the first call)."""
        if self._rope is None:
            self._rope = fdllm_rope_tables(self.max_position, self.head_dim, self.rope_theta,
                                           self.k_pool.device)
        return self._rope

    def decode(self, layer, q, k, v, positions, block_table, seq_lens, slots=None, starts=None,
               out=None, out_dtype=torch.float32, lse=None, with_lse=False, workspace=None,
               status=None, stream=None):
        """One new token a sequence: RoPE, the write of k and v, attention
        over the visible slots (fdllm_decode_attention on this cache).
        Device-side errors are raised by the next check(), or written to
        `status` alone when that is given."""
        status = self.status if status is None else status
        cos, sin = self.rope_tables()
        return fdllm_decode_attention(q, self.k_pool, self.v_pool, layer, block_table, seq_lens, k,
                                      v, positions, slots, cos, sin, starts, None, out, out_dtype,
                                      lse, with_lse, workspace, status, stream)

    def check(self, stream=None):
        """Synchronises the stream and raises FdllmError on an error that a
        step, or a decode() without a status of its own, met on the device
        since the last check."""
        fdllm_check(self.handle, stream)
        if stream is None:
            code = int(self.status.item())
            if code:
                self.status.zero_()
                raise FdllmError(code, load().fdllm_status_string(code).decode())
        else:
            with _on(stream, self.status):
                self.check()

    def close(self):
        if self.handle:
            fdllm_cache_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass
