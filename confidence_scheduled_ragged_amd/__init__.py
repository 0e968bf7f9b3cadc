"""Python binding of libdspark, the MI355X verify hot path (argument marshalling only).

Every function here has the name of a C entry point declared in
``include/dspark.h`` and does nothing but check that tensors are on the GPU
with the expected dtype and layout, allocate missing outputs with torch, and
pass raw device pointers plus torch's current HIP stream to the library. All
computation happens in the HIP kernels of ``libdspark.so``; there is no CPU
fallback, and every entry point raises ImportError when the library is not
built.
"""
from __future__ import annotations

import ctypes
import functools
import os
from typing import Dict, Optional

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libdspark.so")

DSPARK_CUT_THRESHOLD = 0
DSPARK_CUT_BUDGET = 1
DSPARK_CUT_STATIC = 2
DSPARK_CUT_COMBINED = 3
MODES = {"threshold": DSPARK_CUT_THRESHOLD, "budget": DSPARK_CUT_BUDGET,
         "static": DSPARK_CUT_STATIC, "combined": DSPARK_CUT_COMBINED}

_lib = None


class DsparkError(RuntimeError):
    def __init__(self, fn: str, status: int):
        msg = lib().dspark_status_string(status).decode()
        super().__init__(f"{fn}: status {status} ({msg})")
        self.status = status


def lib() -> ctypes.CDLL:
    """Load libdspark.so (built in-tree); raise if it is missing."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(
                f"{LIB_PATH} is not built; run `python -m confidence_scheduled_ragged_amd.build` "
                "or `python -c 'import __graft_entry__; __graft_entry__.build()'`")
        L = ctypes.CDLL(LIB_PATH)
        P, I, F, LL, S = (ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_longlong,
                          ctypes.c_size_t)
        L.dspark_confidence.argtypes = [P, P, F, P, I, I, I, P, P, P]
        L.dspark_schedule.argtypes = [P, I, I, I, P, LL, P, P]
        L.dspark_compact.argtypes = [P, P, I, I, P, P, P, P, I, P, P]
        L.dspark_accept.argtypes = [P, P, P, P, I, I, I, P, P, P, P, S, P]
        L.dspark_step.argtypes = [P, P, F, P, P, P, I, I, I, I, I, P, LL, P, P, P, P, P, P, P, P,
                                  P, P, S, P]
        L.dspark_cap_accept.argtypes = [P, P, P, I, I, P, P, P, P, P]
        L.dspark_gather_rows.argtypes = [P, P, P, I, I, LL, P, P]
        L.dspark_tier_select.argtypes = [P, I, I, P, I, ctypes.c_int32, P, P, P, P, P]
        L.dspark_cost_cutoff.argtypes = [P, I, P, I, P, P]
        L.dspark_step_ex.argtypes = L.dspark_step.argtypes + [P, P, I, ctypes.c_ulonglong]
        L.dspark_step_status.argtypes = [P, P, P]
        L.dspark_step_noalloc.argtypes = L.dspark_step.argtypes[:22] + [P, P]
        L.dspark_workspace_bytes.argtypes = [I, I, I]
        L.dspark_workspace_bytes.restype = S
        L.dspark_workspace_init.argtypes = [P, S, P]
        L.dspark_append_kv.argtypes = [P, P, P, LL, LL, LL, P, P, I, I, I, P, P, I, I, I, I, I, P,
                                       P, I, I, I, LL, LL, LL, F, F, P, I, P, P]
        L.dspark_verify_attention.argtypes = [P, LL, LL, P, P, I, I, I, LL, LL, LL, F, F, P, I, P,
                                              P, I, I, I, I, I, I, I, F, P, P, S, P]
        L.dspark_attention_workspace_bytes.argtypes = [I, I, I, I, I]
        L.dspark_attention_workspace_bytes.restype = S
        L.dspark_sample_accept.argtypes = [P, P, P, P, P, P, P, P, P, I, I, I, P, P, P, P, S, P]
        L.dspark_tree_masks.argtypes = [P, P, P, I, I, I, I, I, I, P, P, P]
        L.dspark_append_tree_kv.argtypes = (L.dspark_append_kv.argtypes[:11] + [P]
                                            + L.dspark_append_kv.argtypes[11:])
        L.dspark_tree_attention.argtypes = (L.dspark_verify_attention.argtypes[:24]
                                            + [I, P, P, I] + L.dspark_verify_attention.argtypes[24:])
        L.dspark_tree_accept.argtypes = [P, P, P, P, I, I, I, I, P, P, P, P]
        L.dspark_move_kv.argtypes = [P, P, I, I, LL, I, I, LL, LL, LL, I, I, P, P, I, P, P, I, I, P]
        L.dspark_resize_pages.argtypes = [P, P, P, I, I, I, P, I, P, P]
        L.dspark_fork_pages.argtypes = [P, P, P, I, I, I, P, I, P, P, I, P, P, P, P, P]
        L.dspark_copy_pages.argtypes = [P, P, I, I, LL, I, I, LL, LL, LL, I, I, P, P, P, I, P]
        L.dspark_status_string.argtypes = [I]
        L.dspark_status_string.restype = ctypes.c_char_p
        for f in (L.dspark_confidence, L.dspark_schedule, L.dspark_compact, L.dspark_accept,
                  L.dspark_step, L.dspark_workspace_init, L.dspark_cap_accept,
                  L.dspark_gather_rows, L.dspark_tier_select, L.dspark_cost_cutoff,
                  L.dspark_step_ex, L.dspark_step_status, L.dspark_step_noalloc,
                  L.dspark_append_kv, L.dspark_verify_attention, L.dspark_sample_accept,
                  L.dspark_tree_masks, L.dspark_append_tree_kv, L.dspark_tree_attention,
                  L.dspark_tree_accept, L.dspark_move_kv, L.dspark_resize_pages,
                  L.dspark_fork_pages, L.dspark_copy_pages):
            f.restype = ctypes.c_int
        _lib = L
    return _lib


# ------------------------------------------------------------------ helpers

def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _need(t: torch.Tensor, name: str, dtype: torch.dtype, shape=None, gpu=None) -> torch.Tensor:
    if (isinstance(t, torch.Tensor) and t.is_cuda and t.dtype is dtype and t.is_contiguous()
            and (shape is None or t.shape == shape) and (gpu is None or t.get_device() == gpu)):
        return t
    # what of it is wrong
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device.type != "cuda":
        raise ValueError(f"{name} must be a GPU tensor (got {t.device})")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype} (got {t.dtype})")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)} (got {tuple(t.shape)})")
    if gpu is not None and t.get_device() != gpu:
        raise ValueError(f"{name} must be on GPU {gpu} as the call's other tensors (got {t.device})")
    return t


def _stream(device: torch.device):
    return ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)


def _raw_stream(index: int) -> int:
    """The current stream's handle without a Stream object in between."""
    return torch._C._cuda_getCurrentRawStream(index)


@functools.lru_cache(maxsize=None)
def _gpus() -> int:
    """How many there are, fixed once a process has used one."""
    return torch.cuda.device_count()


def _launch(gpu: int, name: str, args) -> None:
    """Calls an entry point on GPU `gpu`, which need not be the current one. args end
    with the stream: passed on as they are, and the GPUs counted once, a call takes
    as long as one without this did."""
    fn = getattr(lib(), name)
    if gpu or _gpus() > 1:
        with torch.cuda.device(gpu):
            status = fn(*args)
    else:
        status = fn(*args)
    if status:
        _ok(name, status)


def _ok(fn: str, status: int):
    if status != 0:
        raise DsparkError(fn, status)


def _mode(mode) -> int:
    return MODES[mode] if isinstance(mode, str) else int(mode)


def dspark_status_string(status: int) -> str:
    return lib().dspark_status_string(int(status)).decode()


# --------------------------------------------------------------- workspace

def dspark_workspace_bytes(B: int, gamma: int, V: int) -> int:
    return int(lib().dspark_workspace_bytes(B, gamma, V))


def dspark_workspace_init(ws: torch.Tensor) -> None:
    _need(ws, "ws", torch.uint8)
    gpu = ws.get_device()
    _launch(gpu, "dspark_workspace_init", (ws.data_ptr(), ws.numel(), _raw_stream(gpu)))


class _Kept:
    """The workspaces of one device that calls without one of their own use."""

    def __init__(self):
        self.held = []         # zeroed outside of captures, by size
        self.capture = 0       # the last capture that had to make one, and that one
        self.captured = None
        self.used = None       # by the last call


_WS: Dict[tuple, _Kept] = {}


def _ws_key(device) -> tuple:
    device = device if isinstance(device, torch.device) else torch.device(device)
    idx = device.index if device.index is not None else torch.cuda.current_device()
    return (device.type, idx)


def _capture_id(device) -> int:
    """The capture that the current stream of `device` is in, 0 if in none."""
    with torch.cuda.device(device):
        if not torch.cuda.is_current_stream_capturing():
            return 0
    status, capture = ctypes.c_int(), ctypes.c_ulonglong()
    error = lib().hipStreamGetCaptureInfo(_stream(device), ctypes.byref(status),
                                          ctypes.byref(capture))
    if error:
        raise RuntimeError(f"hipStreamGetCaptureInfo: error {error}")
    return capture.value


def _kept_workspace(cache: Dict[tuple, _Kept], need: int, device) -> torch.Tensor:
    """A zero-filled workspace of at least `need` bytes. One that has become too
    small stays allocated: a captured graph may use it. One that a capture has to
    make is zeroed by the graph only, so it serves that capture alone."""
    key = _ws_key(device)
    kept = cache.get(key)
    if kept is None:
        kept = cache[key] = _Kept()
    if kept.held and kept.held[-1].numel() >= need:
        kept.used = kept.held[-1]
        return kept.used
    capture = _capture_id(device)
    if capture and kept.capture == capture and kept.captured.numel() >= need:
        kept.used = kept.captured
        return kept.used
    ws = torch.empty(need, dtype=torch.uint8, device=device)
    dspark_workspace_init(ws)
    if capture:
        kept.capture, kept.captured = capture, ws
    else:
        kept.held.append(ws)
    kept.used = ws
    return ws


def workspace(B: int, gamma: int, V: int, device) -> torch.Tensor:
    """A zero-initialised workspace of the required size, cached per device (a
    capture for which none is large enough gets its own). Calls sharing it must
    not overlap in time (one stream, or ordered)."""
    device = torch.device(device)
    need = dspark_workspace_bytes(B, gamma, V)
    if need == 0:
        raise ValueError(f"invalid sizes B={B} gamma={gamma} V={V}")
    return _kept_workspace(_WS, need, device)


# ------------------------------------------------------------- entry points

def dspark_confidence(hidden, w, bias, temps, conf=None, survival=None):
    """Steps 1-2: conf[b,i] and survival[b,i] ([B, gamma] fp32)."""
    B, g, d = hidden.shape
    _need(hidden, "hidden", torch.bfloat16)
    _need(w, "w", torch.bfloat16, (d,))
    _need(temps, "temps", torch.float32, (g,))
    dev = hidden.device
    conf = torch.empty((B, g), dtype=torch.float32, device=dev) if conf is None else conf
    survival = torch.empty((B, g), dtype=torch.float32, device=dev) if survival is None else survival
    _need(conf, "conf", torch.float32, (B, g))
    _need(survival, "survival", torch.float32, (B, g))
    _ok("dspark_confidence", lib().dspark_confidence(
        _ptr(hidden), _ptr(w), float(bias), _ptr(temps), B, g, d, _ptr(conf), _ptr(survival),
        _stream(dev)))
    return conf, survival


def dspark_schedule(survival, mode, cutoff=None, budget=0, lengths=None):
    """Step 3: lengths[B] int32 from the survival curves."""
    B, g = survival.shape
    _need(survival, "survival", torch.float32)
    m = _mode(mode)
    if cutoff is not None:
        _need(cutoff, "cutoff", torch.float32, (B,))
    dev = survival.device
    lengths = torch.empty(B, dtype=torch.int32, device=dev) if lengths is None else lengths
    _need(lengths, "lengths", torch.int32, (B,))
    _ok("dspark_schedule", lib().dspark_schedule(
        _ptr(survival), B, g, m, _ptr(cutoff), int(budget), _ptr(lengths), _stream(dev)))
    return lengths


def dspark_compact(lengths, tokens, logits=None, out=None):
    """Step 4: (cu_seqlens, packed_tokens, packed_src_row, packed_logits or None)."""
    B, g1 = tokens.shape
    g = g1 - 1
    _need(lengths, "lengths", torch.int32, (B,))
    _need(tokens, "tokens", torch.int32)
    dev = tokens.device
    cap = B * g1
    out = out or {}
    cu = out.get("cu_seqlens")
    ptok = out.get("packed_tokens")
    psrc = out.get("packed_src_row")
    cu = torch.empty(B + 1, dtype=torch.int32, device=dev) if cu is None else cu
    ptok = torch.full((cap,), -1, dtype=torch.int32, device=dev) if ptok is None else ptok
    psrc = torch.full((cap,), -1, dtype=torch.int32, device=dev) if psrc is None else psrc
    _need(cu, "cu_seqlens", torch.int32, (B + 1,))
    _need(ptok, "packed_tokens", torch.int32, (cap,))
    _need(psrc, "packed_src_row", torch.int32, (cap,))
    plog = None
    V = 0
    if logits is not None:
        _need(logits, "logits", torch.bfloat16)
        V = logits.shape[-1]
        if logits.numel() != cap * V:
            raise ValueError("logits must hold B*(gamma+1) rows")
        plog = out.get("packed_logits")
        plog = torch.zeros((cap, V), dtype=torch.bfloat16, device=dev) if plog is None else plog
        _need(plog, "packed_logits", torch.bfloat16, (cap, V))
    _ok("dspark_compact", lib().dspark_compact(
        _ptr(lengths), _ptr(tokens), B, g, _ptr(cu), _ptr(ptok), _ptr(psrc), _ptr(logits), V,
        _ptr(plog), _stream(dev)))
    return cu, ptok, psrc, plog


def dspark_accept(logits, packed_src_row, cu_seqlens, tokens, out=None, ws=None):
    """Steps 5-6: (packed_argmax, accepted, bonus). packed_src_row None means
    `logits` is already packed ([B*(gamma+1), V], rows past cu_seqlens[B] unused)."""
    B, g1 = tokens.shape
    g = g1 - 1
    _need(logits, "logits", torch.bfloat16)
    V = logits.shape[-1]
    _need(cu_seqlens, "cu_seqlens", torch.int32, (B + 1,))
    _need(tokens, "tokens", torch.int32)
    cap = B * g1
    # dense [B*(gamma+1), V] with source rows, or packed rows with capacity
    # B*(gamma+1) (the packed total is a device value, so the full capacity is
    # required for the reads to stay inside the buffer)
    if logits.numel() != cap * V:
        raise ValueError("logits must hold B*(gamma+1) rows of V entries")
    if packed_src_row is not None:
        _need(packed_src_row, "packed_src_row", torch.int32, (cap,))
    dev = tokens.device
    out = out or {}
    pam = out.get("packed_argmax")
    acc = out.get("accepted")
    bon = out.get("bonus")
    pam = torch.full((cap,), -1, dtype=torch.int32, device=dev) if pam is None else pam
    acc = torch.empty(B, dtype=torch.int32, device=dev) if acc is None else acc
    bon = torch.empty(B, dtype=torch.int32, device=dev) if bon is None else bon
    _need(pam, "packed_argmax", torch.int32, (cap,))
    _need(acc, "accepted", torch.int32, (B,))
    _need(bon, "bonus", torch.int32, (B,))
    ws = workspace(B, g, V, dev) if ws is None else _need(ws, "ws", torch.uint8)
    _ok("dspark_accept", lib().dspark_accept(
        _ptr(logits), _ptr(packed_src_row), _ptr(cu_seqlens), _ptr(tokens), B, g, V, _ptr(pam),
        _ptr(acc), _ptr(bon), _ptr(ws), ws.numel(), _stream(dev)))
    return pam, acc, bon


STEP_OUTPUTS = ("conf", "survival", "lengths", "cu_seqlens", "packed_tokens", "packed_src_row",
                "packed_argmax", "accepted", "bonus")


def dspark_gather_rows(src, packed_src_row, cu_seqlens, out=None):
    """Packed row gather: out[r] = src[packed_src_row[r]] for r < cu_seqlens[B].
    src is [B*(gamma+1), ...] (or [B, gamma+1, ...]) of any dtype; out has the
    same row shape and B*(gamma+1) rows (allocated when None)."""
    _need(cu_seqlens, "cu_seqlens", torch.int32)
    B = cu_seqlens.numel() - 1
    _need(packed_src_row, "packed_src_row", torch.int32)
    cap = packed_src_row.numel()
    if cap % B != 0:
        raise ValueError("packed_src_row must have B*(gamma+1) entries")
    g = cap // B - 1
    if not isinstance(src, torch.Tensor) or src.device.type != "cuda" or not src.is_contiguous():
        raise ValueError("src must be a contiguous GPU tensor")
    if src.numel() % cap != 0:
        raise ValueError("src must hold B*(gamma+1) rows")
    if src.shape[0] == cap:
        row_shape = (cap,) + tuple(src.shape[1:])
    elif src.dim() >= 2 and tuple(src.shape[:2]) == (B, g + 1):
        row_shape = (cap,) + tuple(src.shape[2:])
    else:
        raise ValueError("src must be [B*(gamma+1), ...] or [B, gamma+1, ...]")
    row_bytes = src.numel() // cap * src.element_size()
    if out is None:
        out = torch.empty(row_shape, dtype=src.dtype, device=src.device)
    if (out.dtype != src.dtype or not out.is_contiguous() or out.device != src.device
            or out.numel() * out.element_size() != cap * row_bytes):
        raise ValueError("out must be a contiguous GPU tensor of B*(gamma+1) rows like src")
    _ok("dspark_gather_rows", lib().dspark_gather_rows(
        _ptr(src), _ptr(packed_src_row), _ptr(cu_seqlens), B, g, row_bytes, _ptr(out),
        _stream(src.device)))
    return out


def dspark_cost_cutoff(table, load, B, cutoff=None):
    """Every request's cutoff from the cost table at the step's load level:
    table fp32 [n] and load int32 [1] on the device; returns cutoff fp32 [B]."""
    _need(table, "table", torch.float32)
    _need(load, "load", torch.int32, (1,))
    dev = table.device
    cutoff = torch.empty(B, dtype=torch.float32, device=dev) if cutoff is None else cutoff
    _need(cutoff, "cutoff", torch.float32, (B,))
    _ok("dspark_cost_cutoff", lib().dspark_cost_cutoff(
        _ptr(table), table.numel(), _ptr(load), int(B), _ptr(cutoff), _stream(dev)))
    return cutoff


def dspark_tier_select(cu_seqlens, gamma, tiers, pad_token=0, packed_tokens=None,
                       packed_src_row=None, out=None):
    """Graph tier of a packed batch: (padded_total [1], tier_index [1]) int32 on
    the device; pads packed_tokens / packed_src_row (when given) up to the
    tier. tiers: int32 device tensor, strictly ascending."""
    _need(cu_seqlens, "cu_seqlens", torch.int32)
    B = cu_seqlens.numel() - 1
    _need(tiers, "tiers", torch.int32)
    dev = cu_seqlens.device
    cap = B * (gamma + 1)
    for t, n in ((packed_tokens, "packed_tokens"), (packed_src_row, "packed_src_row")):
        if t is not None:
            _need(t, n, torch.int32, (cap,))
    out = out or {}
    padded = out.get("padded_total")
    idx = out.get("tier_index")
    padded = torch.empty(1, dtype=torch.int32, device=dev) if padded is None else padded
    idx = torch.empty(1, dtype=torch.int32, device=dev) if idx is None else idx
    _need(padded, "padded_total", torch.int32, (1,))
    _need(idx, "tier_index", torch.int32, (1,))
    _ok("dspark_tier_select", lib().dspark_tier_select(
        _ptr(cu_seqlens), B, int(gamma), _ptr(tiers), tiers.numel(), int(pad_token), _ptr(padded),
        _ptr(idx), _ptr(packed_tokens), _ptr(packed_src_row), _stream(dev)))
    return padded, idx


def dspark_cap_accept(packed_argmax_full, tokens, lengths, out=None, sums=None):
    """Cap-accept audit arm over a static verify: (accepted, bonus,
    accepted_full, sums). packed_argmax_full holds the argmax of every row of
    the full block (static packing, [B*(gamma+1)]); lengths is the cut's
    window. sums, when given (int64 [2]), receives (sum accepted, sum
    accepted_full)."""
    B, g1 = tokens.shape
    _need(tokens, "tokens", torch.int32)
    _need(packed_argmax_full, "packed_argmax_full", torch.int32, (B * g1,))
    _need(lengths, "lengths", torch.int32, (B,))
    dev = tokens.device
    out = out or {}
    acc = out.get("accepted")
    bon = out.get("bonus")
    full = out.get("accepted_full")
    acc = torch.empty(B, dtype=torch.int32, device=dev) if acc is None else acc
    bon = torch.empty(B, dtype=torch.int32, device=dev) if bon is None else bon
    full = torch.empty(B, dtype=torch.int32, device=dev) if full is None else full
    for t, n in ((acc, "accepted"), (bon, "bonus"), (full, "accepted_full")):
        _need(t, n, torch.int32, (B,))
    if sums is not None:
        _need(sums, "sums", torch.int64, (2,))
    _ok("dspark_cap_accept", lib().dspark_cap_accept(
        _ptr(packed_argmax_full), _ptr(tokens), _ptr(lengths), B, g1 - 1, _ptr(acc), _ptr(bon),
        _ptr(full), _ptr(sums), _stream(dev)))
    return acc, bon, full, sums


def alloc_step_outputs(B: int, gamma: int, device, with_conf: bool = True) -> Dict[str, torch.Tensor]:
    cap = B * (gamma + 1)
    i32 = dict(dtype=torch.int32, device=device)
    out = dict(lengths=torch.empty(B, **i32), cu_seqlens=torch.empty(B + 1, **i32),
               packed_tokens=torch.full((cap,), -1, **i32),
               packed_src_row=torch.full((cap,), -1, **i32),
               packed_argmax=torch.full((cap,), -1, **i32),
               accepted=torch.empty(B, **i32), bonus=torch.empty(B, **i32))
    if with_conf:
        out["conf"] = torch.empty((B, gamma), dtype=torch.float32, device=device)
        out["survival"] = torch.empty((B, gamma), dtype=torch.float32, device=device)
    return out


def _event_handle(ev):
    """Raw hipEvent_t of a torch.cuda.Event (created on first use) or a handle."""
    if ev is None:
        return None
    if isinstance(ev, torch.cuda.Event):
        if not ev.cuda_event:
            ev.record()                  # torch creates the event lazily
        return ctypes.c_void_p(ev.cuda_event)
    return ctypes.c_void_p(int(ev))


def dspark_step(hidden, w, bias, temps, tokens, logits, mode, cutoff=None, budget=0, out=None,
                ws=None, events=None, launches=0, wait_ticks=0):
    """Steps 1-6 in one call; returns the dict of output tensors. With any of
    `events` (a pair of timing events, recorded around the step's dominant
    kernel), `launches` (0 by size, 1 one launch where the cut allows it, 2 two
    launches) or `wait_ticks` (bound of the one-launch wait, 100 MHz ticks; 0 is
    the default) the call goes through dspark_step_ex."""
    args, out, ws = _step_args(hidden, w, bias, temps, tokens, logits, mode, cutoff, budget, out,
                               ws, None)
    if events is None and not launches and not wait_ticks:
        _ok("dspark_step", lib().dspark_step(*args))
    else:
        ev = events if events is not None else (None, None)
        _ok("dspark_step_ex", lib().dspark_step_ex(
            *args, _event_handle(ev[0]), _event_handle(ev[1]), int(launches), int(wait_ticks)))
    return out


def _step_args(hidden, w, bias, temps, tokens, logits, mode, cutoff, budget, out, ws, stream):
    """Checked, marshalled arguments of dspark_step (and the outputs)."""
    B, g, d = hidden.shape
    V = logits.shape[-1]
    _need(hidden, "hidden", torch.bfloat16)
    _need(w, "w", torch.bfloat16, (d,))
    _need(temps, "temps", torch.float32, (g,))
    _need(tokens, "tokens", torch.int32, (B, g + 1))
    _need(logits, "logits", torch.bfloat16, (B, g + 1, V))
    m = _mode(mode)
    if cutoff is not None:
        _need(cutoff, "cutoff", torch.float32, (B,))
    dev = hidden.device
    out = alloc_step_outputs(B, g, dev) if out is None else out
    cap = B * (g + 1)
    shapes = dict(conf=(B, g), survival=(B, g), lengths=(B,), cu_seqlens=(B + 1,),
                  packed_tokens=(cap,), packed_src_row=(cap,), packed_argmax=(cap,),
                  accepted=(B,), bonus=(B,))
    for k, shp in shapes.items():
        if out.get(k) is not None:
            _need(out[k], k, torch.float32 if k in ("conf", "survival") else torch.int32, shp)
    ws = workspace(B, g, V, dev) if ws is None else _need(ws, "ws", torch.uint8)
    st = _stream(dev) if stream is None else ctypes.c_void_p(int(stream))
    args = (
        _ptr(hidden), _ptr(w), float(bias), _ptr(temps), _ptr(tokens), _ptr(logits), B, g, d, V,
        m, _ptr(cutoff), int(budget), _ptr(out.get("conf")), _ptr(out.get("survival")),
        _ptr(out["lengths"]), _ptr(out["cu_seqlens"]), _ptr(out["packed_tokens"]),
        _ptr(out["packed_src_row"]), _ptr(out["packed_argmax"]), _ptr(out["accepted"]),
        _ptr(out["bonus"]), _ptr(ws), ws.numel(), st)
    return args, out, ws


class BoundStep:
    """dspark_step on fixed buffers: the arguments are checked and marshalled
    once, and each call is one C call (for serving loops that refill the same
    input buffers every step, where the per-call checks of dspark_step cost
    more host time than a small step takes on the GPU). The tensors must stay
    alive, in place and unresized while the object is used; calls run on the
    stream given at binding (the current stream by default)."""

    def __init__(self, hidden, w, bias, temps, tokens, logits, mode, cutoff=None, budget=0,
                 out=None, ws=None, launches=0, wait_ticks=0, stream=None):
        args, self.out, self.ws = _step_args(hidden, w, bias, temps, tokens, logits, mode, cutoff,
                                             budget, out, ws, stream)
        # the tensors the raw pointers point into
        self._keep = (hidden, w, temps, tokens, logits, cutoff, self.out, self.ws)
        self._fn = lib().dspark_step_ex
        self._args = args + (None, None, int(launches), int(wait_ticks))

    def __call__(self):
        status = self._fn(*self._args)
        if status != 0:
            raise DsparkError("dspark_step_ex", status)
        return self.out


def bind_step(hidden, w, bias, temps, tokens, logits, mode, cutoff=None, budget=0, out=None,
              ws=None, launches=0, wait_ticks=0, stream=None) -> BoundStep:
    """A BoundStep: dspark_step's arguments checked once, launched by calling it."""
    return BoundStep(hidden, w, bias, temps, tokens, logits, mode, cutoff=cutoff, budget=budget,
                     out=out, ws=ws, launches=launches, wait_ticks=wait_ticks, stream=stream)


def dspark_step_ex(hidden, w, bias, temps, tokens, logits, mode, cutoff=None, budget=0,
                   out=None, ws=None, events=None, launches=0, wait_ticks=0):
    """dspark_step with explicit controls: timing events around its dominant
    kernel, the form (launches) and the bound of the one-launch wait."""
    return dspark_step(hidden, w, bias, temps, tokens, logits, mode, cutoff=cutoff,
                       budget=budget, out=out, ws=ws, events=events, launches=launches,
                       wait_ticks=wait_ticks)


def dspark_step_noalloc(hidden, w, bias, temps, tokens, logits, mode, cutoff=None, budget=0,
                        out=None, status=None):
    """dspark_step without a workspace argument: the library's own per-device
    scratch array serves as the workspace, so the call allocates nothing on the
    device side (torch allocates the outputs here only when `out` is None).
    `status` (int32 [1], optional) receives the give-up flag of this call.
    Calls on one device share that scratch and must not overlap in time."""
    B, g, d = hidden.shape
    V = logits.shape[-1]
    _need(hidden, "hidden", torch.bfloat16)
    _need(w, "w", torch.bfloat16, (d,))
    _need(temps, "temps", torch.float32, (g,))
    _need(tokens, "tokens", torch.int32, (B, g + 1))
    _need(logits, "logits", torch.bfloat16, (B, g + 1, V))
    m = _mode(mode)
    if cutoff is not None:
        _need(cutoff, "cutoff", torch.float32, (B,))
    dev = hidden.device
    out = alloc_step_outputs(B, g, dev) if out is None else out
    if status is not None:
        _need(status, "status", torch.int32, (1,))
    _ok("dspark_step_noalloc", lib().dspark_step_noalloc(
        _ptr(hidden), _ptr(w), float(bias), _ptr(temps), _ptr(tokens), _ptr(logits), B, g, d, V,
        m, _ptr(cutoff), int(budget), _ptr(out.get("conf")), _ptr(out.get("survival")),
        _ptr(out["lengths"]), _ptr(out["cu_seqlens"]), _ptr(out["packed_tokens"]),
        _ptr(out["packed_src_row"]), _ptr(out["packed_argmax"]), _ptr(out["accepted"]),
        _ptr(out["bonus"]), _ptr(status), _stream(dev)))
    return out


def dspark_step_status(ws=None, status=None, device=None):
    """The fused step's give-up flag of a workspace, read and cleared on the
    device: an int32 [1] tensor, 0 when no call since the last read gave up its
    bounded wait. ws defaults to the binding's workspace of `device` that the last
    call without one of its own used."""
    if ws is None:
        kept = _WS.get(_ws_key(device if device is not None else "cuda"))
        if kept is None or kept.used is None:
            raise ValueError("no workspace has been used on this device")
        ws = kept.used
    _need(ws, "ws", torch.uint8)
    status = torch.empty(1, dtype=torch.int32, device=ws.device) if status is None else status
    _need(status, "status", torch.int32, (1,))
    _ok("dspark_step_status", lib().dspark_step_status(_ptr(ws), _ptr(status), _stream(ws.device)))
    return status


# ------------------------------------------- around the target's verify forward

_CACHE_TYPES = {torch.bfloat16: 0, torch.float8_e4m3fn: 1}


def _paged(k_cache, v_cache, cu_seqlens, ctx_lens, block_table):
    """Checks the paged cache and the packed batch's lengths; returns the index of
    their GPU, B, the cache's type, sizes and strides."""
    shape, strides, dtype = k_cache.shape, k_cache.stride(), k_cache.dtype
    if len(shape) != 4 or v_cache.shape != shape:
        raise ValueError("k_cache and v_cache must have one shape, [pages, Hkv, page_size, D]")
    gpu = k_cache.get_device()
    if not k_cache.is_cuda or not v_cache.is_cuda or v_cache.get_device() != gpu:
        raise ValueError(f"the caches must be on one GPU (got {k_cache.device}, {v_cache.device})")
    if dtype not in _CACHE_TYPES or v_cache.dtype is not dtype:
        raise TypeError(f"the caches must be bfloat16 or float8_e4m3fn (got {dtype}, "
                        f"{v_cache.dtype})")
    if v_cache.stride() != strides or strides[3] != 1:
        raise ValueError("k_cache and v_cache must share strides, with D contiguous")
    B = cu_seqlens.numel() - 1
    _need(cu_seqlens, "cu_seqlens", torch.int32, None, gpu)
    _need(ctx_lens, "ctx_lens", torch.int32, (B,), gpu)
    _need(block_table, "block_table", torch.int32, None, gpu)
    if block_table.dim() != 2 or block_table.shape[0] != B:
        raise ValueError(f"block_table must have shape ({B}, pages of a request)")
    return gpu, B, _CACHE_TYPES[dtype], shape, strides


def _packed_heads(t, name, rows, heads, D, gpu):
    """Checks packed [rows, heads, D] bf16 with rows at any stride; returns its strides."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor")
    if t.get_device() != gpu:
        raise ValueError(f"{name} must be on GPU {gpu} as the caches (got {t.device})")
    if t.dtype is not torch.bfloat16:
        raise TypeError(f"{name} must be {torch.bfloat16} (got {t.dtype})")
    if t.shape != (rows, heads, D):
        raise ValueError(f"{name} must have shape {(rows, heads, D)} (got {tuple(t.shape)})")
    strides = t.stride()
    if strides[2] != 1:
        raise ValueError(f"{name} must have its last axis contiguous")
    return strides


def dspark_append_kv(q, k, v, cos, sin, cu_seqlens, ctx_lens, block_table, k_cache, v_cache,
                     interleaved=False, k_scale=1.0, v_scale=1.0, out=None):
    """Rotates the packed rows' queries and keys by their positions and writes
    keys and values into the paged cache; returns the rotated queries.
    q [rows, Hq, D], k and v [rows, Hkv, D] bf16 (views of one projection, with
    heads side by side), cos and sin [positions, rot / 2] fp32, ctx_lens [B]
    tokens cached before the call, block_table [B, width] int32, k_cache and
    v_cache [pages, Hkv, page_size, D] bf16 or float8_e4m3fn."""
    return _append("dspark_append_kv", None, q, k, v, cos, sin, cu_seqlens, ctx_lens, block_table,
                   k_cache, v_cache, interleaved, k_scale, v_scale, out)


def _append(name, depths, q, k, v, cos, sin, cu_seqlens, ctx_lens, block_table, k_cache, v_cache,
            interleaved, k_scale, v_scale, out):
    """dspark_append_kv, or with depths dspark_append_tree_kv."""
    gpu, B, kind, (pages, Hkv, page, D), (ps, hs, ss, _) = _paged(
        k_cache, v_cache, cu_seqlens, ctx_lens, block_table)
    rows, Hq = q.shape[0], q.shape[1]
    qs = _packed_heads(q, "q", rows, Hq, D, gpu)
    ks = _packed_heads(k, "k", rows, Hkv, D, gpu)
    vs = _packed_heads(v, "v", rows, Hkv, D, gpu)
    if (qs[1] != D and Hq > 1) or ((ks[1] != D or vs[1] != D) and Hkv > 1):
        raise ValueError("q, k and v must have their heads side by side")
    _need(cos, "cos", torch.float32, None, gpu)
    angles = cos.shape
    _need(sin, "sin", torch.float32, angles, gpu)
    if len(angles) != 2:
        raise ValueError("cos must have shape (positions, rotated pairs)")
    if out is None:
        out = torch.empty((rows, Hq, D), dtype=torch.bfloat16, device=q.device)
    else:
        _need(out, "out", torch.bfloat16, (rows, Hq, D), gpu)
    args = [
        q.data_ptr(), k.data_ptr(), v.data_ptr(), qs[0], ks[0], vs[0], cos.data_ptr(),
        sin.data_ptr(), angles[0], angles[1], 1 if interleaved else 0, cu_seqlens.data_ptr(),
        ctx_lens.data_ptr(), B, rows, Hq, Hkv, D, k_cache.data_ptr(), v_cache.data_ptr(), kind,
        pages, page, ps, hs, ss, k_scale, v_scale, block_table.data_ptr(), block_table.shape[1],
        out.data_ptr(), _raw_stream(gpu)]
    if name == "dspark_append_tree_kv":
        _need(depths, "depths", torch.int32, (rows,), gpu)
        args.insert(11, depths.data_ptr())  # after `interleaved`
    _launch(gpu, name, args)
    return out


def dspark_attention_workspace_bytes(B: int, max_rows: int, Hq: int, Hkv: int, D: int) -> int:
    return int(lib().dspark_attention_workspace_bytes(B, max_rows, Hq, Hkv, D))


_ATTN_WS: Dict[tuple, _Kept] = {}


def attention_workspace(B: int, max_rows: int, Hq: int, Hkv: int, D: int, device) -> torch.Tensor:
    """A zero-initialised workspace of dspark_verify_attention, cached per
    device as by workspace(). Calls sharing it must not overlap in time (one
    stream, or ordered)."""
    need = lib().dspark_attention_workspace_bytes(B, max_rows, Hq, Hkv, D)
    if need == 0:
        raise ValueError(f"invalid sizes B={B} max_rows={max_rows} Hq={Hq} Hkv={Hkv} D={D}")
    return _kept_workspace(_ATTN_WS, need, device)


def dspark_verify_attention(q, k_cache, v_cache, cu_seqlens, ctx_lens, block_table, max_rows,
                            window=0, scale=None, k_scale=1.0, v_scale=1.0, out=None, ws=None):
    """Attention of the packed rows q [rows, Hq, D] bf16 over each request's
    pages, causal at the end of the request: row j of request b stands at
    position ctx_lens[b] + j, which the cache already holds. max_rows bounds the
    rows of a request (1 for plain decoding, gamma + 1 for a verify window, any
    number for a prompt chunk); window > 0 keeps the last `window` positions;
    scale defaults to D ** -0.5. Returns out [rows, Hq, D] bf16. Without ws the
    call uses attention_workspace(), one for all streams of the GPU: calls on
    several streams at a time need one each."""
    return _attend("dspark_verify_attention", None, q, k_cache, v_cache, cu_seqlens, ctx_lens,
                   block_table, max_rows, window, scale, k_scale, v_scale, out, ws)


def _attend(name, tree, q, k_cache, v_cache, cu_seqlens, ctx_lens, block_table, max_rows, window,
            scale, k_scale, v_scale, out, ws):
    """dspark_verify_attention, or with (depths, masks, sinks) dspark_tree_attention."""
    gpu, B, kind, (pages, Hkv, page, D), (ps, hs, ss, _) = _paged(
        k_cache, v_cache, cu_seqlens, ctx_lens, block_table)
    rows, Hq = q.shape[0], q.shape[1]
    qs = _packed_heads(q, "q", rows, Hq, D, gpu)
    if out is None:
        out = torch.empty((rows, Hq, D), dtype=torch.bfloat16, device=q.device)
    else:
        _need(out, "out", torch.bfloat16, (rows, Hq, D), gpu)
    max_rows = min(int(max_rows), rows)
    view = None
    if tree is not None:
        depths, masks, sinks = tree
        if (depths is None) != (masks is None):
            raise ValueError("depths and masks must be given together")
        if masks is None:
            view = (int(sinks), None, None, 0)
        else:
            _need(depths, "depths", torch.int32, (rows,), gpu)
            _need(masks, "masks", torch.int32, None, gpu)
            if masks.dim() != 2 or masks.shape[0] != rows:
                raise ValueError(f"masks must have shape ({rows}, words)")
            view = (int(sinks), depths.data_ptr(), masks.data_ptr(), masks.shape[1])
    if ws is None:
        ws = attention_workspace(B, max_rows, Hq, Hkv, D, q.device)
    else:
        _need(ws, "ws", torch.uint8, None, gpu)
    args = [
        q.data_ptr(), qs[0], qs[1], k_cache.data_ptr(), v_cache.data_ptr(), kind, pages, page, ps,
        hs, ss, k_scale, v_scale, block_table.data_ptr(), block_table.shape[1],
        cu_seqlens.data_ptr(), ctx_lens.data_ptr(), B, rows, max_rows, Hq, Hkv, D, int(window),
        D ** -0.5 if scale is None else scale, out.data_ptr(), ws.data_ptr(), ws.numel(),
        _raw_stream(gpu)]
    if view is not None:
        args[24:24] = view  # after the window
    _launch(gpu, name, args)
    return out


def dspark_sample_accept(logits, packed_src_row, cu_seqlens, tokens, uniforms, temperature=None,
                         top_k=None, top_p=None, min_p=None, out=None, ws=None):
    """dspark_accept with the target's tokens drawn: (packed_sample, accepted,
    bonus). uniforms fp32 [B*(gamma+1)] in [0, 1), one per packed row;
    temperature (<= 0: greedy), top_p, min_p fp32 [B] and top_k int32 [B] (0:
    off) per request, None for temperature 1 and no filter. packed_src_row None
    means `logits` is already packed. Without ws the call uses workspace(), one for
    all streams of the GPU: calls on several streams at a time need one each."""
    B, g1 = tokens.shape
    cap = B * g1
    _need(logits, "logits", torch.bfloat16)
    V = logits.shape[-1]
    if logits.numel() != cap * V:
        raise ValueError("logits must hold B*(gamma+1) rows of V entries")
    gpu = logits.get_device()
    _need(cu_seqlens, "cu_seqlens", torch.int32, (B + 1,), gpu)
    _need(tokens, "tokens", torch.int32, None, gpu)
    _need(uniforms, "uniforms", torch.float32, (cap,), gpu)
    if packed_src_row is not None:
        _need(packed_src_row, "packed_src_row", torch.int32, (cap,), gpu)
    for t, n in ((temperature, "temperature"), (top_p, "top_p"), (min_p, "min_p")):
        if t is not None:
            _need(t, n, torch.float32, (B,), gpu)
    if top_k is not None:
        _need(top_k, "top_k", torch.int32, (B,), gpu)
    dev = tokens.device
    out = out or {}
    smp = out.get("packed_sample")
    acc = out.get("accepted")
    bon = out.get("bonus")
    smp = torch.full((cap,), -1, dtype=torch.int32, device=dev) if smp is None else smp
    acc = torch.empty(B, dtype=torch.int32, device=dev) if acc is None else acc
    bon = torch.empty(B, dtype=torch.int32, device=dev) if bon is None else bon
    _need(smp, "packed_sample", torch.int32, (cap,), gpu)
    _need(acc, "accepted", torch.int32, (B,), gpu)
    _need(bon, "bonus", torch.int32, (B,), gpu)
    ws = workspace(B, g1 - 1, V, dev) if ws is None else _need(ws, "ws", torch.uint8, None, gpu)
    at = lambda t: None if t is None else t.data_ptr()  # noqa: E731
    status = lib().dspark_sample_accept(
        logits.data_ptr(), at(packed_src_row), cu_seqlens.data_ptr(), tokens.data_ptr(),
        uniforms.data_ptr(), at(temperature), at(top_k), at(top_p), at(min_p), B, g1 - 1, V,
        smp.data_ptr(), acc.data_ptr(), bon.data_ptr(), ws.data_ptr(), ws.numel(),
        _raw_stream(gpu))
    if status:
        _ok("dspark_sample_accept", status)
    return smp, acc, bon


# --------------------------------------------- drafted trees and shared pages

def dspark_tree_masks(parents, cu_seqlens, max_rows, ctx_lens=None, window=0, sinks=0, out=None):
    """(depths [rows], masks [rows, words]) int32 of drafted trees: parents [rows]
    int32, the place of each row's parent among its request's rows (below its own;
    anything else is a root), max_rows the most rows of a request, words as many as
    hold that many bits. ctx_lens [B] is needed with window and sinks. Rows past
    cu_seqlens[-1] are untouched."""
    _need(parents, "parents", torch.int32)
    gpu, rows = parents.get_device(), parents.numel()
    _need(cu_seqlens, "cu_seqlens", torch.int32, None, gpu)
    B = cu_seqlens.numel() - 1
    if ctx_lens is not None:
        _need(ctx_lens, "ctx_lens", torch.int32, (B,), gpu)
    elif window > 0 and sinks > 0:
        raise ValueError("ctx_lens must be given with window and sinks")
    words = -(-int(max_rows) // 32)
    depths, masks = (None, None) if out is None else out
    if depths is None:
        depths = torch.zeros(rows, dtype=torch.int32, device=parents.device)
    else:
        _need(depths, "depths", torch.int32, (rows,), gpu)
    if masks is None:
        masks = torch.zeros((rows, max(words, 1)), dtype=torch.int32, device=parents.device)
    else:
        _need(masks, "masks", torch.int32, None, gpu)
        if masks.dim() != 2 or masks.shape[0] != rows:
            raise ValueError(f"masks must have shape ({rows}, words)")
    _launch(gpu, "dspark_tree_masks", (
        parents.data_ptr(), cu_seqlens.data_ptr(), None if ctx_lens is None else ctx_lens.data_ptr(),
        B, rows, int(max_rows), int(window), int(sinks), masks.shape[1], depths.data_ptr(),
        masks.data_ptr(), _raw_stream(gpu)))
    return depths, masks


def dspark_append_tree_kv(q, k, v, cos, sin, depths, cu_seqlens, ctx_lens, block_table, k_cache,
                          v_cache, interleaved=False, k_scale=1.0, v_scale=1.0, out=None):
    """dspark_append_kv for the nodes of trees: a row is rotated by the position
    ctx_lens[b] + depths[row] (dspark_tree_masks) and keeps the slot that it has in a
    chain. Returns the rotated queries."""
    return _append("dspark_append_tree_kv", depths, q, k, v, cos, sin, cu_seqlens, ctx_lens,
                   block_table, k_cache, v_cache, interleaved, k_scale, v_scale, out)


def dspark_tree_attention(q, k_cache, v_cache, cu_seqlens, ctx_lens, block_table, max_rows,
                          depths=None, masks=None, window=0, sinks=0, scale=None, k_scale=1.0,
                          v_scale=1.0, out=None, ws=None):
    """dspark_verify_attention for the nodes of trees (depths [rows] and masks [rows,
    words] int32 of dspark_tree_masks; none for a chain), and with the first `sinks`
    positions visible beside a window. Without ws the call uses
    attention_workspace(), as dspark_verify_attention does."""
    return _attend("dspark_tree_attention", (depths, masks, sinks), q, k_cache, v_cache,
                   cu_seqlens, ctx_lens, block_table, max_rows, window, scale, k_scale, v_scale,
                   out, ws)


def dspark_tree_accept(packed_choice, packed_tokens, parents, cu_seqlens, max_rows, width, out=None):
    """(accepted [B], bonus [B], path [B, width]) int32: the walk down every request's
    tree by the target's choices (packed_argmax of dspark_accept or packed_sample of
    dspark_sample_accept), to the lowest of siblings that share the chosen token. path
    holds places among the request's rows, from row 0 on, then -1; at most width - 1
    drafts are accepted."""
    _need(packed_choice, "packed_choice", torch.int32)
    gpu, rows, dev = packed_choice.get_device(), packed_choice.numel(), packed_choice.device
    _need(packed_tokens, "packed_tokens", torch.int32, None, gpu)
    _need(parents, "parents", torch.int32, None, gpu)
    if packed_tokens.numel() != rows or parents.numel() != rows:
        raise ValueError("packed_choice, packed_tokens and parents must have one entry a row")
    _need(cu_seqlens, "cu_seqlens", torch.int32, None, gpu)
    B = cu_seqlens.numel() - 1
    if out is None:
        acc, bonus, path = torch.empty(B * (width + 2), dtype=torch.int32, device=dev).split(
            (B, B, B * width))
        path = path.view(B, width)
    else:
        acc, bonus, path = out
        _need(acc, "accepted", torch.int32, (B,), gpu)
        _need(bonus, "bonus", torch.int32, (B,), gpu)
        _need(path, "path", torch.int32, (B, width), gpu)
    _launch(gpu, "dspark_tree_accept", (
        packed_choice.data_ptr(), packed_tokens.data_ptr(), parents.data_ptr(),
        cu_seqlens.data_ptr(), B, rows, int(max_rows), int(width), acc.data_ptr(),
        bonus.data_ptr(), path.data_ptr(), _raw_stream(gpu)))
    return acc, bonus, path


def _layered(k_cache, v_cache):
    """Checks pools [layers, pages, Hkv, page_size, D] or [pages, Hkv, page_size, D];
    returns their GPU and the arguments from the pointers to D."""
    shape, strides, dtype = k_cache.shape, k_cache.stride(), k_cache.dtype
    if len(shape) not in (4, 5) or v_cache.shape != shape:
        raise ValueError("k_cache and v_cache must have one shape, [layers, pages, Hkv, page_size, "
                         "D] or [pages, Hkv, page_size, D]")
    gpu = k_cache.get_device()
    if not k_cache.is_cuda or not v_cache.is_cuda or v_cache.get_device() != gpu:
        raise ValueError(f"the caches must be on one GPU (got {k_cache.device}, {v_cache.device})")
    if dtype not in _CACHE_TYPES or v_cache.dtype is not dtype:
        raise TypeError(f"the caches must be bfloat16 or float8_e4m3fn (got {dtype}, "
                        f"{v_cache.dtype})")
    if v_cache.stride() != strides or strides[-1] != 1:
        raise ValueError("k_cache and v_cache must share strides, with D contiguous")
    layers, layer_stride = (shape[0], strides[0]) if len(shape) == 5 else (1, 0)
    pages, Hkv, page, D = shape[-4:]
    ps, hs, ss = strides[-4:-1]
    return gpu, (k_cache.data_ptr(), v_cache.data_ptr(), _CACHE_TYPES[dtype], layers, layer_stride,
                 pages, page, ps, hs, ss, Hkv, D)


def dspark_move_kv(k_cache, v_cache, path, accepted, ctx_lens, block_table):
    """Brings every request's accepted path (dspark_tree_accept) together in the
    cache: slot ctx_lens[b] + path[b, i] goes to slot ctx_lens[b] + i, keys and values.
    The caches are those of all layers, [layers, pages, Hkv, page_size, D], or of one."""
    gpu, pool = _layered(k_cache, v_cache)
    _need(path, "path", torch.int32, None, gpu)
    if path.dim() != 2:
        raise ValueError("path must have shape (B, width)")
    B, width = path.shape
    _need(accepted, "accepted", torch.int32, (B,), gpu)
    _need(ctx_lens, "ctx_lens", torch.int32, (B,), gpu)
    _need(block_table, "block_table", torch.int32, None, gpu)
    if block_table.dim() != 2 or block_table.shape[0] != B:
        raise ValueError(f"block_table must have shape ({B}, pages of a request)")
    _launch(gpu, "dspark_move_kv", (
        *pool, path.data_ptr(), accepted.data_ptr(), width, ctx_lens.data_ptr(),
        block_table.data_ptr(), block_table.shape[1], B, _raw_stream(gpu)))


def page_pool(pages: int, rows: int, width: int, device):
    """(table [rows, width], held [rows], refs [pages]) of a new pool: no row holds a page."""
    table = torch.full((rows, width), -1, dtype=torch.int32, device=device)
    return table, torch.zeros(rows, dtype=torch.int32, device=device), torch.zeros(
        pages, dtype=torch.int32, device=device)


def _pool(table, held, refs, lens):
    _need(table, "table", torch.int32)
    if table.dim() != 2:
        raise ValueError("table must have shape (rows, pages of a row)")
    gpu, (R, width) = table.get_device(), table.shape
    _need(held, "held", torch.int32, (R,), gpu)
    _need(refs, "refs", torch.int32, None, gpu)
    _need(lens, "lens", torch.int32, (R,), gpu)
    return gpu, R, width


def dspark_resize_pages(table, held, refs, lens, page_size, granted=None):
    """Every row of the table [R, width] gets and gives back pages until it holds
    ceil(lens[b] / page_size) of them (page_pool() makes the state: table, held [R],
    refs [pages], all changed in place). Returns granted [R] int32: 1 where the row
    holds what its length needs, 0 where there were too few free pages or places. A call
    that takes pages takes 23 us longer for every 100 000 taken ones below them."""
    gpu, R, width = _pool(table, held, refs, lens)
    if granted is None:
        granted = torch.empty_like(held)
    else:
        _need(granted, "granted", torch.int32, (R,), gpu)
    _launch(gpu, "dspark_resize_pages", (
        table.data_ptr(), held.data_ptr(), lens.data_ptr(), R, width, int(page_size),
        refs.data_ptr(), refs.numel(), granted.data_ptr(), _raw_stream(gpu)))
    return granted


def dspark_fork_pages(table, held, refs, src, dst, lens, page_size, out=None):
    """Row dst[i] becomes a copy of row src[i] up to position lens[src[i]]: full pages
    are shared, and where the positions end inside a page the row gets one of its own.
    Returns (copy_src, copy_dst, copy_slots, granted) [n] int32; the first three are
    what dspark_copy_pages takes to fill those pages. Rows that cannot be served have
    granted 0 and stay as they were."""
    gpu, R, width = _pool(table, held, refs, lens)
    n = src.numel()
    _need(src, "src", torch.int32, (n,), gpu)
    _need(dst, "dst", torch.int32, (n,), gpu)
    if out is None:
        out = src.new_empty((4, n)).unbind(0)
    else:
        for t, name in zip(out, ("copy_src", "copy_dst", "copy_slots", "granted")):
            _need(t, name, torch.int32, (n,), gpu)
    _launch(gpu, "dspark_fork_pages", (
        table.data_ptr(), held.data_ptr(), lens.data_ptr(), R, width, int(page_size),
        refs.data_ptr(), refs.numel(), src.data_ptr(), dst.data_ptr(), n,
        *[t.data_ptr() for t in out], _raw_stream(gpu)))
    return out


def dspark_copy_pages(k_cache, v_cache, src, dst, slots=None):
    """Copies the first slots[i] slots (None: all) of page src[i] to page dst[i], keys
    and values, in the caches of all layers or of one; entries outside the pool copy
    nothing."""
    gpu, pool = _layered(k_cache, v_cache)
    n = src.numel()
    _need(src, "src", torch.int32, (n,), gpu)
    _need(dst, "dst", torch.int32, (n,), gpu)
    if slots is not None:
        _need(slots, "slots", torch.int32, (n,), gpu)
    _launch(gpu, "dspark_copy_pages", (
        *pool, src.data_ptr(), dst.data_ptr(), None if slots is None else slots.data_ptr(), n,
        _raw_stream(gpu)))


__all__ = ["DsparkError", "lib", "LIB_PATH", "dspark_status_string", "dspark_confidence", "dspark_schedule",
           "dspark_compact", "dspark_accept", "dspark_step", "dspark_cap_accept",
           "dspark_gather_rows", "dspark_tier_select", "dspark_cost_cutoff",
           "dspark_step_ex", "dspark_step_status", "dspark_step_noalloc", "BoundStep", "bind_step",
           "dspark_append_kv", "dspark_verify_attention", "dspark_sample_accept",
           "dspark_tree_masks", "dspark_append_tree_kv", "dspark_tree_attention",
           "dspark_tree_accept", "dspark_move_kv", "dspark_resize_pages", "dspark_fork_pages",
           "dspark_copy_pages", "page_pool",
           "dspark_attention_workspace_bytes", "attention_workspace", "dspark_workspace_bytes",
           "dspark_workspace_init", "workspace", "alloc_step_outputs", "STEP_OUTPUTS",
           "DSPARK_CUT_THRESHOLD", "DSPARK_CUT_BUDGET", "DSPARK_CUT_STATIC",
           "DSPARK_CUT_COMBINED"]
