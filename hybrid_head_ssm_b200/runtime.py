"""Device-memory plumbing around the C ABI: uploads a layer's weights, allocates the
KV buffers, SSM state and workspace as torch CUDA tensors, and calls
hymba_mixer_prefill / hymba_mixer_decode on torch's current stream. No arithmetic
of the mixer happens here.
"""
from __future__ import annotations

import ctypes
from typing import Dict, Optional

import numpy as np
import torch

from . import (HYMBA_BF16, HYMBA_F16, HYMBA_F32, HYMBA_MODE_DECODE, HYMBA_MODE_PREFILL, check, cfg_struct,
               current_stream_ptr, hymba_attn_decode_paged, hymba_attn_decode_paged_workspace,
               hymba_attn_prefill_packed, hymba_kv_append_paged, hymba_linattn_prefill, hymba_linattn_step,
               hymba_linattn_workspace, hymba_mixer_decode, hymba_mixer_prefill, hymba_paged_kv,
               hymba_workspace_bytes, kv_struct, state_struct, weights_struct)

BIG = ("w_in", "w_dt", "w_out", "meta")
NAMES = ("w_in", "w_dt", "b_dt", "conv_w", "conv_b", "A_log", "D", "norm_attn_w", "norm_ssm_w",
         "beta1", "beta2", "w_out", "meta", "kv_scale", "kv_bias", "pre_norm_w")
# a consumer's affine adaptation of the shared K/V; the block's pre-mixer norm gain
OPTIONAL = ("kv_scale", "kv_bias", "pre_norm_w")


def act_dtype(cfg):
    return torch.bfloat16 if cfg.dtype == HYMBA_BF16 else torch.float32


def mid_dtype(cfg):
    """Element type of K/V and the other intermediates (fp16 in bf16 layers)."""
    return torch.float16 if cfg.dtype == HYMBA_BF16 else torch.float32


class DeviceLayer:
    """One mixer layer's weights in device memory and its C structs."""

    def __init__(self, cfg, w: Dict[str, np.ndarray], device="cuda"):
        self.cfg = cfg
        self.c = cfg_struct(cfg)
        adt = act_dtype(cfg)
        self.t = {}
        for n in NAMES:
            a = w.get(n)
            if a is None and n in OPTIONAL:
                continue
            a = w[n]
            dt = adt if n in BIG else torch.float32
            self.t[n] = torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).to(device=device, dtype=dt)
        self.s = weights_struct(self.t)


class KV:
    """K/V buffers of a producer layer (and its consumers)."""

    def __init__(self, cfg, B: int, seq_cap: int = 0, cache_cap: int = 0, device="cuda"):
        adt = mid_dtype(cfg)
        G, dh, dv = cfg.n_kv_heads, cfg.head_dim, cfg.v_head_dim
        self.k_seq = torch.empty((B, G, seq_cap, dh), dtype=adt, device=device) if seq_cap else None
        self.v_seq = torch.empty((B, G, seq_cap, dv), dtype=adt, device=device) if seq_cap else None
        self.k_cache = torch.zeros((B, G, cache_cap, dh), dtype=adt, device=device) if cache_cap else None
        self.v_cache = torch.zeros((B, G, cache_cap, dv), dtype=adt, device=device) if cache_cap else None
        self.len = torch.zeros(B, dtype=torch.int32, device=device) if cache_cap else None
        self.s = kv_struct(cfg, B, self.k_seq, self.v_seq, self.k_cache, self.v_cache, self.len)


class State:
    def __init__(self, cfg, B: int, device="cuda"):
        self.h = torch.zeros((B, cfg.d_inner, cfg.d_state), dtype=torch.float32, device=device)
        self.conv = torch.zeros((B, cfg.d_inner, cfg.d_conv), dtype=torch.float32, device=device)
        self.s = state_struct(self.h, self.conv)


def workspace(cfg, B: int, T: int, mode: int, device="cuda") -> torch.Tensor:
    n = hymba_workspace_bytes(ctypes.byref(cfg_struct(cfg)), B, T, mode)
    if n == 0:
        raise ValueError("invalid layer configuration")
    return torch.empty(n, dtype=torch.uint8, device=device)


def prefill(layer: DeviceLayer, x: torch.Tensor, T: int, kv: KV, y: torch.Tensor, ws: torch.Tensor,
            state: Optional[State] = None, flags: int = 0, kv_struct_override=None) -> None:
    kvs = kv_struct_override if kv_struct_override is not None else kv.s
    check(hymba_mixer_prefill(ctypes.byref(layer.c), ctypes.byref(layer.s), x.data_ptr(), x.shape[0], T,
                              flags, y.data_ptr(), ctypes.byref(kvs),
                              ctypes.byref(state.s) if state is not None else None,
                              ws.data_ptr(), ws.numel(), current_stream_ptr()))


def decode(layer: DeviceLayer, x_t: torch.Tensor, kv_s, state: State, y_t: torch.Tensor,
           ws: torch.Tensor, flags: int = 0) -> None:
    check(hymba_mixer_decode(ctypes.byref(layer.c), ctypes.byref(layer.s), x_t.data_ptr(), x_t.shape[0],
                             flags, y_t.data_ptr(), ctypes.byref(kv_s), ctypes.byref(state.s),
                             ws.data_ptr(), ws.numel(), current_stream_ptr()))


def to_device(a: np.ndarray, cfg, device="cuda", io_f32: bool = False) -> torch.Tensor:
    dt = torch.float32 if io_f32 else act_dtype(cfg)
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).to(device=device, dtype=dt)


def stream_flags(cfg) -> int:
    """Flags of a layer inside a residual stack: fp32 residual stream for bf16 layers."""
    from . import HYMBA_ADD_RESIDUAL, HYMBA_IO_F32
    return HYMBA_ADD_RESIDUAL | (HYMBA_IO_F32 if cfg.dtype == HYMBA_BF16 else 0)


class DeviceMLP:
    """The block MLP's weights in device memory and their C struct."""

    def __init__(self, cfg, w: Dict[str, np.ndarray], device="cuda"):
        from . import hymba_mlp_weights
        self.cfg = cfg
        self.c = cfg_struct(cfg)
        self.d_ff = w["w_gate"].shape[0]
        adt = act_dtype(cfg)
        self.t = {n: torch.from_numpy(np.ascontiguousarray(w[n], dtype=np.float32)).to(
            device=device, dtype=torch.float32 if n == "norm_w" else adt) for n in ("norm_w", "w_gate", "w_up", "w_down")}
        self.s = hymba_mlp_weights(*[self.t[n].data_ptr() for n in ("norm_w", "w_gate", "w_up", "w_down")])


def mlp_workspace(mlp: DeviceMLP, rows: int, device="cuda") -> torch.Tensor:
    from . import hymba_mlp_workspace_bytes
    n = hymba_mlp_workspace_bytes(ctypes.byref(mlp.c), mlp.d_ff, rows)
    if n == 0:
        raise ValueError("invalid MLP configuration")
    return torch.empty(n, dtype=torch.uint8, device=device)


def mlp(m: DeviceMLP, h: torch.Tensor, ws: torch.Tensor) -> None:
    """h += MLP(RMSNorm(h)) in place on every row of the fp32 stream h."""
    from . import hymba_mlp
    assert h.dtype == torch.float32 and h.is_contiguous()
    rows = h.numel() // m.cfg.d_model
    check(hymba_mlp(ctypes.byref(m.c), m.d_ff, ctypes.byref(m.s), h.data_ptr(), rows, ws.data_ptr(), ws.numel(),
                    current_stream_ptr()))


# ---------------------------------------------------------------------------
# ragged batches: packed prompts, paged K/V, linear attention
# ---------------------------------------------------------------------------
TORCH_DTYPE = {HYMBA_F16: torch.float16, HYMBA_BF16: torch.bfloat16, HYMBA_F32: torch.float32}
_DTYPE_CODE = {v: k for k, v in TORCH_DTYPE.items()}
_F32, _I32 = torch.float32, torch.int32
# the current stream's handle without building a Stream object (2 us of the smallest calls)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


def _need(ok: bool, what: str) -> None:
    if not ok:
        raise ValueError(what)


def _misfit(name: str, t: torch.Tensor, what: str) -> ValueError:
    return ValueError(f"{name}: {what} wanted, got {tuple(t.shape)} with strides {t.stride()} of {t.dtype} on {t.device}")


def _rows(name: str, t: torch.Tensor, rows: int, width: int, dtype: torch.dtype, dev: torch.device) -> int:
    """Row stride of a [rows, width] tensor of one type on one device, its elements side by
    side within a row."""
    if t.shape != (rows, width) or t.dtype is not dtype or t.device != dev:
        raise _misfit(name, t, f"[{rows}, {width}] of {dtype} on {dev}")
    ld, step = t.stride()
    if step != 1 and width > 1:
        raise _misfit(name, t, "elements side by side within a row")
    # the stride of a single row is never used (and torch may report anything for it)
    return ld if rows > 1 else width


def _dense(name: str, t: torch.Tensor, shape, dtype: torch.dtype, dev: torch.device) -> None:
    if t.shape != shape or t.dtype is not dtype or t.device != dev or not t.is_contiguous():
        raise _misfit(name, t, f"contiguous {tuple(shape)} of {dtype} on {dev}")


def _scratch(ws: torch.Tensor, dev: torch.device) -> int:
    if ws.device != dev or not ws.is_contiguous():
        raise _misfit("workspace", ws, f"a contiguous tensor on {dev}")
    return ws.numel() * ws.element_size()


def _queue(dev: torch.device, fn, *args) -> None:
    """Call fn(*args, stream) with the tensors' device current, on torch's current stream
    of that device."""
    if dev.type != "cuda":
        raise ValueError(f"tensors on a CUDA device wanted, got {dev}")
    index = dev.index
    if index == torch.cuda.current_device():
        rc = fn(*args, _raw_stream(index))
    else:
        with torch.cuda.device(index):
            rc = fn(*args, _raw_stream(index))
    if rc:
        check(rc)


class PagedKV:
    """K and V in pages: k_pages [n_pages, n_kv_heads, page_size, head_dim], v_pages [n_pages,
    n_kv_heads, page_size, v_head_dim], page_table int32 [batch, max_pages], len int32
    [batch]; the tensors stay the caller's and are kept alive here."""

    def __init__(self, k_pages: torch.Tensor, v_pages: torch.Tensor, page_table: torch.Tensor, length: torch.Tensor):
        code, dev = _DTYPE_CODE.get(k_pages.dtype), k_pages.device
        if code is None or k_pages.dim() != 4 or not k_pages.is_contiguous():
            raise _misfit("k_pages", k_pages, "contiguous [n_pages, n_kv_heads, page_size, head_dim] of float16, "
                          "bfloat16 or float32")
        n_pages, G, page, dh = k_pages.shape
        _need(v_pages.dim() == 4 and page_table.dim() == 2, "v_pages of 4 dimensions, page_table [batch, max_pages]")
        _dense("v_pages", v_pages, (n_pages, G, page, v_pages.shape[3]), k_pages.dtype, dev)
        _dense("page_table", page_table, page_table.shape, _I32, dev)
        _dense("len", length, (page_table.shape[0],), _I32, dev)
        self.k_pages, self.v_pages, self.page_table, self.len = k_pages, v_pages, page_table, length
        self.device, self.dtype, self.batch = dev, k_pages.dtype, page_table.shape[0]
        self.k_width, self.v_width = G * dh, G * v_pages.shape[3]
        self.s = hymba_paged_kv(k_pages.data_ptr(), v_pages.data_ptr(), page_table.data_ptr(), length.data_ptr(),
                                n_pages, page, page_table.shape[1], self.batch, G, dh, v_pages.shape[3], code)
        self.ref = ctypes.byref(self.s)


def attn_prefill_packed(shape, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, cu_seqlens: torch.Tensor,
                        o: torch.Tensor) -> None:
    """o [rows, H * dv] = causal attention of the packed prompts q [rows, H * dh], k [rows,
    G * dh], v [rows, G * dv]; cu_seqlens int32 [sequences + 1]."""
    H, G, dh, dv = shape.n_q_heads, shape.n_kv_heads, shape.head_dim, shape.v_head_dim
    rows, dev, dtype = q.shape[0], q.device, TORCH_DTYPE.get(shape.dtype)
    ldq, ldk = _rows("q", q, rows, H * dh, dtype, dev), _rows("k", k, rows, G * dh, dtype, dev)
    ldv, ldo = _rows("v", v, rows, G * dv, dtype, dev), _rows("o", o, rows, H * dv, dtype, dev)
    n = cu_seqlens.numel()
    _dense("cu_seqlens", cu_seqlens, (n,), _I32, dev)
    _queue(dev, hymba_attn_prefill_packed, ctypes.byref(shape), q.data_ptr(), ldq, k.data_ptr(), ldk, v.data_ptr(),
           ldv, cu_seqlens.data_ptr(), n - 1, rows, o.data_ptr(), ldo)


def kv_append_paged(kv: PagedKV, k: torch.Tensor, v: torch.Tensor, cu_seqlens: Optional[torch.Tensor] = None) -> None:
    """The rows of k [rows, G * dh] and v [rows, G * dv] become their sequences' newest
    positions (kv.len counts them already); cu_seqlens None: one row per sequence."""
    rows, dev, cu = k.shape[0], kv.device, None
    ldk, ldv = _rows("k", k, rows, kv.k_width, kv.dtype, dev), _rows("v", v, rows, kv.v_width, kv.dtype, dev)
    if cu_seqlens is not None:
        _dense("cu_seqlens", cu_seqlens, (kv.batch + 1,), _I32, dev)
        cu = cu_seqlens.data_ptr()
    _queue(dev, hymba_kv_append_paged, kv.ref, k.data_ptr(), ldk, v.data_ptr(), ldv, cu, rows)


def decode_paged_workspace(shape, batch: int, max_len: int, device="cuda") -> torch.Tensor:
    n = hymba_attn_decode_paged_workspace(ctypes.byref(shape), batch, max_len)
    _need(n > 0, "invalid attention shape, batch or length")
    return torch.empty(n, dtype=torch.uint8, device=device)


def attn_decode_paged(shape, q: torch.Tensor, kv: PagedKV, o: torch.Tensor, ws: torch.Tensor, max_len: int = 0) -> None:
    """o [batch, H * dv] = attention of the newest position of every sequence (q [batch, H *
    dh]) over its pages. max_len: a bound on every length (0: the page table's capacity);
    ws from decode_paged_workspace with that bound."""
    H, dev = shape.n_q_heads, kv.device
    ldq = _rows("q", q, kv.batch, H * shape.head_dim, kv.dtype, dev)
    ldo = _rows("o", o, kv.batch, H * shape.v_head_dim, kv.dtype, dev)
    _queue(dev, hymba_attn_decode_paged, ctypes.byref(shape), q.data_ptr(), ldq, kv.ref, max_len, o.data_ptr(), ldo,
           ws.data_ptr(), _scratch(ws, dev))


def _decays(g: torch.Tensor, rows: int, heads: int, dev: torch.device) -> int:
    """Row stride of the log decays: float32 [rows, heads], or [heads] (0: the same for every
    row, as for rows expanded from one)."""
    if g.dim() == 1:
        _dense("g", g, (heads,), _F32, dev)
        return 0
    if rows > 1 and g.stride(0) == 0 and g.shape[0] == rows:
        _rows("g", g[:1], 1, heads, _F32, dev)
        return 0
    return _rows("g", g, rows, heads, _F32, dev)


def linattn_workspace(shape, n_seqs: int, rows: int, device="cuda") -> torch.Tensor:
    """Scratch for linattn_prefill calls with just these numbers of sequences and rows (fewer may
    need more: few long prompts are cut into segments)."""
    n = hymba_linattn_workspace(ctypes.byref(shape), n_seqs, rows)
    _need(n > 0, "invalid linear-attention shape, sequence count or row count")
    return torch.empty(n, dtype=torch.uint8, device=device)


def linattn_prefill(shape, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, g: torch.Tensor, cu_seqlens: torch.Tensor,
                    o: torch.Tensor, ws: torch.Tensor, state_in: Optional[torch.Tensor] = None,
                    state_out: Optional[torch.Tensor] = None) -> None:
    """o [rows, H * dv] of the packed prompts q, k [rows, Hk * dk], v [rows, H * dv] with log
    decays g float32 [rows, H] or [H]; states float32 [sequences, H, dv, dk] before and
    after the prompts."""
    Hk, H, dk, dv = shape.n_qk_heads, shape.n_heads, shape.key_dim, shape.v_head_dim
    rows, dev, dtype = q.shape[0], q.device, TORCH_DTYPE.get(shape.dtype)
    ldq, ldk = _rows("q", q, rows, Hk * dk, dtype, dev), _rows("k", k, rows, Hk * dk, dtype, dev)
    ldv, ldo = _rows("v", v, rows, H * dv, dtype, dev), _rows("o", o, rows, H * dv, dtype, dev)
    n = cu_seqlens.numel() - 1
    _dense("cu_seqlens", cu_seqlens, (n + 1,), _I32, dev)
    first = last = None
    if state_in is not None:
        _dense("state_in", state_in, (n, H, dv, dk), _F32, dev)
        first = state_in.data_ptr()
    if state_out is not None:
        _dense("state_out", state_out, (n, H, dv, dk), _F32, dev)
        last = state_out.data_ptr()
    _queue(dev, hymba_linattn_prefill, ctypes.byref(shape), q.data_ptr(), ldq, k.data_ptr(), ldk, v.data_ptr(), ldv,
           g.data_ptr(), _decays(g, rows, H, dev), cu_seqlens.data_ptr(), n, rows, first, last, o.data_ptr(), ldo,
           ws.data_ptr(), _scratch(ws, dev))


def linattn_step(shape, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, g: torch.Tensor, state: torch.Tensor,
                 o: torch.Tensor) -> None:
    """One token per sequence: state float32 [batch, H, dv, dk] is updated in place, o [batch,
    H * dv] is its product with the token's query."""
    Hk, H, dk, dv = shape.n_qk_heads, shape.n_heads, shape.key_dim, shape.v_head_dim
    rows, dev, dtype = q.shape[0], q.device, TORCH_DTYPE.get(shape.dtype)
    ldq, ldk = _rows("q", q, rows, Hk * dk, dtype, dev), _rows("k", k, rows, Hk * dk, dtype, dev)
    ldv, ldo = _rows("v", v, rows, H * dv, dtype, dev), _rows("o", o, rows, H * dv, dtype, dev)
    _dense("state", state, (rows, H, dv, dk), _F32, dev)
    _queue(dev, hymba_linattn_step, ctypes.byref(shape), q.data_ptr(), ldq, k.data_ptr(), ldk, v.data_ptr(), ldv,
           g.data_ptr(), _decays(g, rows, H, dev), state.data_ptr(), rows, o.data_ptr(), ldo)
