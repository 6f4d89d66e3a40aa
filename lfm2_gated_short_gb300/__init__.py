"""LFM2 gated short convolution (ShortConv) on GB300 (sm_103a).

A thin ctypes binding over ``libshortconv.so`` (see ``include/shortconv.h``).
Every function here only checks and marshals arguments: torch CUDA tensors
become device pointers plus sizes, the current torch stream becomes the
``cudaStream_t``, and all the work runs in the library's CUDA kernels. There
is no CPU or PyTorch fallback: if the library is not built, or a call fails,
an exception is raised.

Layouts (row-major, contiguous, one dtype per call: torch.bfloat16 or
torch.float32): ``bcx [T, 3H]`` (B | C | x), ``w [H, K]``, state pool
``[n_slots, H, K]`` (tap K-1 newest), ``y [T, H]``; index arrays are int32.
Every forward and backward call takes an optional conv ``bias [H]`` (the data
dtype; None for none), added to the conv output before the C gate.
"""
from __future__ import annotations

import ctypes
import functools
import os
import threading

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
# SHORTCONV_LIBRARY selects another build of this library (the tests use it to
# load the bounds-checked build, _build/bounds/libshortconv.so).
LIB_PATH = os.environ.get("SHORTCONV_LIBRARY") or os.path.join(_HERE, "_build", "libshortconv.so")
DEV_OUT_OF_BOUNDS = 0x20

SC_OK, SC_EINVAL, SC_EUNSUPPORTED, SC_ECUDA, SC_EDEVICE = 0, 1, 2, 3, 4
SC_F32, SC_BF16 = 0, 1
DEV_BAD_SLOT, DEV_BAD_SEQLENS, DEV_BAD_ACCEPTED, DEV_TIMEOUT, DEV_NO_SLOT = 0x1, 0x2, 0x4, 0x8, 0x10

DEV_NO_PAGE, DEV_BAD_PAGE, DEV_BAD_LENGTH, DEV_BAD_TOKEN, DEV_BAD_PROBS = (
    0x40, 0x80, 0x100, 0x200, 0x400)

_lock = threading.Lock()
_lib = None


class ShortConvError(RuntimeError):
    """A library call returned a status other than SC_OK."""

    def __init__(self, fn: str, status: int, message: str):
        super().__init__(f"{fn}: {message} (status {status})")
        self.status = status


def lib() -> ctypes.CDLL:
    """The loaded C library (argument types declared). Raises if it is not built."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise RuntimeError(
                    f"{LIB_PATH} is missing: build it with "
                    "`python -m lfm2_gated_short_gb300.build` (nvcc, sm_103a)")
            L = ctypes.CDLL(LIB_PATH)
            p, i32, i64 = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64
            L.shortconv_prefill.argtypes = [i32, i32, i32, p, i64, p, p, p, i32, p, p, i32, p, p]
            L.shortconv_prefill_tiled.argtypes = [i32, i32, i32, p, i64, p, p, p, i32, p, p,
                                                  i32, p, i32, p]
            L.shortconv_decode.argtypes = [i32, i32, i32, p, i32, p, p, p, p, i32, p, p]
            L.shortconv_verify.argtypes = [i32, i32, i32, p, i32, i32, p, p, p, p, i32, p, p,
                                           p]
            L.shortconv_rollback.argtypes = [i32, i32, i32, i32, i32, p, p, p, p, i32, p]
            L.shortconv_rollback_layers.argtypes = [i32, i32, i32, i32, i32, i32, p, p, p, p,
                                                    i32, p]
            L.shortconv_backward_workspace_bytes.argtypes = [i32, i32, i64]
            L.shortconv_backward_workspace_bytes.restype = ctypes.c_size_t
            L.shortconv_backward.argtypes = [i32, i32, i32, p, i64, p, p, p, p, p, p, p,
                                             ctypes.c_size_t, p]
            L.shortconv_backward_varlen.argtypes = [i32, i32, i32, p, i64, p, p, p, i32, p, p,
                                                    p, p, p, p, p, p, ctypes.c_size_t, p]
            L.shortconv_in_proj_workspace_bytes.argtypes = [i32, i32, i32]
            L.shortconv_in_proj_workspace_bytes.restype = ctypes.c_size_t
            L.shortconv_in_proj_prefill.argtypes = [i32, i32, i32, i32, p, i64, p, p, p, p, i32,
                                                    p, p, i32, p, p, ctypes.c_size_t, p]
            L.shortconv_out_proj.argtypes = [i32, i32, i32, p, i64, p, p, p]
            L.shortconv_in_proj_decode.argtypes = [i32, i32, i32, i32, p, i32, p, p, p, p, p,
                                                   i32, p, p]
            L.shortconv_slots_claim.argtypes = [p, i32, i32, p, i32, i32, i32, p, p]
            L.shortconv_slots_release.argtypes = [p, i32, p, i32, p]
            L.shortconv_pool_copy.argtypes = [i32, i32, i32, p, i32, p, p, i32, p]
            sz = ctypes.c_size_t
            L.shortconv_pages_workspace_bytes.argtypes = [i32, i32]
            L.shortconv_pages_workspace_bytes.restype = sz
            L.shortconv_pages_resize.argtypes = [p, i32, p, p, i32, i32, i32, p, p, i32, i32, i64,
                                                 p, p, p, sz, p]
            L.shortconv_pages_fork.argtypes = L.shortconv_pages_resize.argtypes
            L.shortconv_pages_compact.argtypes = [p, i32, p, p, i32, i32, i32, i32, i64, p, p, p,
                                                  p, sz, p]
            L.shortconv_pages_append.argtypes = [p, i64, p, i64, i32, i32, i64, p, p, i32, i32, p,
                                                 p, i32, i32, p, p]
            L.shortconv_prefix_attention_workspace_bytes.argtypes = [i32] * 6
            L.shortconv_prefix_attention_workspace_bytes.restype = sz
            L.shortconv_prefix_attention.argtypes = [i32, i32, i32, i32, p, i64, i32, i32, p, p,
                                                     i32, i32, p, p, i32, i32, p, i32,
                                                     ctypes.c_float, p, p, sz, p]
            L.shortconv_draft_accept.argtypes = [i32, i32, i32, i32, p, i64, p, i64, p, p, p, p, p,
                                                 p]
            L.shortconv_get_error.argtypes = [p, ctypes.POINTER(ctypes.c_int)]
            L.shortconv_check_wait_limit.argtypes = [p]
            L.shortconv_bounds_checked.argtypes = []
            L.shortconv_bounds_checked.restype = i32
            L.shortconv_bounds_trim_next.argtypes = [i32, ctypes.c_uint64]
            L.shortconv_bounds_take_first_bad.argtypes = [p, ctypes.POINTER(ctypes.c_uint64)]
            L.shortconv_status_string.argtypes = [i32]
            L.shortconv_status_string.restype = ctypes.c_char_p
            for f in ("prefill", "prefill_tiled", "decode", "verify", "rollback",
                      "rollback_layers", "backward",
                      "backward_varlen", "in_proj_prefill", "in_proj_decode", "out_proj",
                      "slots_claim",
                      "slots_release", "pool_copy", "pages_resize", "pages_fork",
                      "pages_compact", "pages_append", "prefix_attention", "draft_accept",
                      "get_error", "check_wait_limit",
                      "bounds_trim_next", "bounds_take_first_bad"):
                getattr(L, "shortconv_" + f).restype = i32
            _lib = L
    return _lib


def _raise_on(fn: str, status: int) -> None:
    if status != SC_OK:
        msg = lib().shortconv_status_string(status).decode()
        raise ShortConvError(fn, status, msg)


def _dcode(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return SC_BF16
    if t.dtype == torch.float32:
        return SC_F32
    raise TypeError(f"unsupported dtype {t.dtype}: use torch.bfloat16 or torch.float32")


def _dev(t: torch.Tensor, name: str, dtype=None, shape=None) -> int:
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor, got {t.device}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if shape is not None and t.shape != shape:  # torch.Size compares as a tuple
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    return t.data_ptr()


# The current stream's handle without building a torch.cuda.Stream object.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream, device) -> int:
    if stream is not None:
        return stream.cuda_stream
    if _raw_stream is not None and device.index is not None:
        return _raw_stream(device.index)
    return torch.cuda.current_stream(device).cuda_stream


def _bias(bias, dt, H):
    return None if bias is None else _dev(bias, "bias", dt, (H,))


def prefill(bcx, w, cu_seqlens, slot_ids, pool, y=None, rows_per_thread=0, stream=None,
            bias=None):
    """Packed varlen prefill; updates ``pool`` in place and returns ``y [T, H]``."""
    dt = bcx.dtype
    T, H3 = bcx.shape
    H, K = w.shape
    if H3 != 3 * H:
        raise ValueError("bcx must be [T, 3H] for w [H, K]")
    N = slot_ids.shape[0]
    if y is None:
        y = torch.empty((T, H), dtype=dt, device=bcx.device)
    args = (_dcode(bcx), H, K, _dev(bcx, "bcx", dt), T, _dev(w, "w", dt), _bias(bias, dt, H),
            _dev(cu_seqlens, "cu_seqlens", torch.int32, (N + 1,)), N,
            _dev(slot_ids, "slot_ids", torch.int32, (N,)),
            _dev(pool, "pool", dt, (pool.shape[0], H, K)), pool.shape[0],
            _dev(y, "y", dt, (T, H)))
    st = _stream(stream, bcx.device)
    if rows_per_thread:
        _raise_on("shortconv_prefill_tiled",
                  lib().shortconv_prefill_tiled(*args, rows_per_thread, st))
    else:
        _raise_on("shortconv_prefill", lib().shortconv_prefill(*args, st))
    return y


def decode(bcx, w, slot_ids, pool, y=None, stream=None, bias=None):
    """One token per sequence; updates ``pool`` in place and returns ``y [N, H]``."""
    dt = bcx.dtype
    N, H3 = bcx.shape
    H, K = w.shape
    if H3 != 3 * H:
        raise ValueError("bcx must be [N, 3H] for w [H, K]")
    if y is None:
        y = torch.empty((N, H), dtype=dt, device=bcx.device)
    _raise_on("shortconv_decode", lib().shortconv_decode(
        _dcode(bcx), H, K, _dev(bcx, "bcx", dt), N, _dev(w, "w", dt), _bias(bias, dt, H),
        _dev(slot_ids, "slot_ids", torch.int32, (N,)),
        _dev(pool, "pool", dt, (pool.shape[0], H, K)), pool.shape[0],
        _dev(y, "y", dt, (N, H)), _stream(stream, bcx.device)))
    return y


def verify(bcx, w, slot_ids, pool, D, win=None, y=None, stream=None, bias=None):
    """Speculative verify of ``D`` drafts per sequence; returns ``(win, y)``. Pool is read only."""
    dt = bcx.dtype
    H, K = w.shape
    N = slot_ids.shape[0]
    if tuple(bcx.shape) != (N * D, 3 * H):
        raise ValueError(f"bcx must be [N*D, 3H] = {(N * D, 3 * H)}")
    if win is None:
        win = torch.empty((N, D, H, K), dtype=dt, device=bcx.device)
    if y is None:
        y = torch.empty((N * D, H), dtype=dt, device=bcx.device)
    _raise_on("shortconv_verify", lib().shortconv_verify(
        _dcode(bcx), H, K, _dev(bcx, "bcx", dt), N, D, _dev(w, "w", dt), _bias(bias, dt, H),
        _dev(slot_ids, "slot_ids", torch.int32, (N,)),
        _dev(pool, "pool", dt, (pool.shape[0], H, K)), pool.shape[0],
        _dev(win, "win", dt, (N, D, H, K)), _dev(y, "y", dt, (N * D, H)),
        _stream(stream, bcx.device)))
    return win, y


def rollback(win, accepted, slot_ids, pool, stream=None):
    """Commit each sequence's accepted prefix into its slot (in place on ``pool``)."""
    dt = win.dtype
    N, D, H, K = win.shape
    _raise_on("shortconv_rollback", lib().shortconv_rollback(
        _dcode(win), H, K, N, D, _dev(win, "win", dt),
        _dev(accepted, "accepted", torch.int32, (N,)),
        _dev(slot_ids, "slot_ids", torch.int32, (N,)),
        _dev(pool, "pool", dt, (pool.shape[0], H, K)), pool.shape[0],
        _stream(stream, win.device)))


def rollback_layers(win, accepted, slot_ids, pool, stream=None):
    """Roll back L layers at once: ``win [L, N, D, H, K]`` (stacked verify tapes),
    ``pool [L, n_slots, H, K]`` (stacked pools, in place)."""
    dt = win.dtype
    L, N, D, H, K = win.shape
    if pool.dim() != 4 or pool.shape[0] != L:
        raise ValueError("pool must be [L, n_slots, H, K] for win [L, N, D, H, K]")
    _raise_on("shortconv_rollback_layers", lib().shortconv_rollback_layers(
        _dcode(win), H, K, L, N, D, _dev(win, "win", dt),
        _dev(accepted, "accepted", torch.int32, (N,)),
        _dev(slot_ids, "slot_ids", torch.int32, (N,)),
        _dev(pool, "pool", dt, (L, pool.shape[1], H, K)), pool.shape[1],
        _stream(stream, win.device)))


def backward_workspace_bytes(H: int, K: int, T: int) -> int:
    return int(lib().shortconv_backward_workspace_bytes(H, K, T))


def backward(bcx, w, dy, dbcx=None, dw=None, workspace=None, stream=None, bias=None,
             with_dbias=False, dbias=None):
    """Backward from a zero state; returns ``(dbcx [T, 3H], dw [H, K] fp32)``,
    plus ``dbias [H] fp32`` when ``with_dbias``."""
    dt = bcx.dtype
    T, H3 = bcx.shape
    H, K = w.shape
    if H3 != 3 * H:
        raise ValueError("bcx must be [T, 3H] for w [H, K]")
    need = backward_workspace_bytes(H, K, T)
    if dbcx is None:
        dbcx = torch.empty_like(bcx)
    if dw is None:
        dw = torch.empty((H, K), dtype=torch.float32, device=bcx.device)
    if with_dbias and dbias is None:
        dbias = torch.empty((H,), dtype=torch.float32, device=bcx.device)
    if workspace is None:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=bcx.device)
    if workspace.dtype != torch.uint8 or workspace.numel() < need:
        raise ValueError(f"workspace must be a uint8 tensor of at least {need} bytes")
    db_p = _dev(dbias, "dbias", torch.float32, (H,)) if with_dbias else None
    _raise_on("shortconv_backward", lib().shortconv_backward(
        _dcode(bcx), H, K, _dev(bcx, "bcx", dt), T, _dev(w, "w", dt), _bias(bias, dt, H),
        _dev(dy, "dy", dt, (T, H)), _dev(dbcx, "dbcx", dt, (T, 3 * H)),
        _dev(dw, "dw", torch.float32, (H, K)), db_p, _dev(workspace, "workspace"),
        workspace.numel(), _stream(stream, bcx.device)))
    return (dbcx, dw, dbias) if with_dbias else (dbcx, dw)


def backward_varlen(bcx, w, cu_seqlens, dy, init_states=None, d_final=None, dbcx=None,
                    dw=None, d_init=None, workspace=None, want_d_init=True, stream=None,
                    bias=None, with_dbias=False, dbias=None):
    """Packed varlen backward with initial states; returns ``(dbcx, dw, d_init)``,
    plus ``dbias [H] fp32`` when ``with_dbias``.

    ``init_states`` is ``[N, H, K]`` (the data dtype; None: zeros);
    ``d_final`` is ``[N, H, K]`` float32 (None: zeros); ``d_init`` is
    ``[N, H, K]`` float32 (None when ``want_d_init`` is False).
    """
    dt = bcx.dtype
    T, H3 = bcx.shape
    H, K = w.shape
    if H3 != 3 * H:
        raise ValueError("bcx must be [T, 3H] for w [H, K]")
    N = cu_seqlens.shape[0] - 1
    need = backward_workspace_bytes(H, K, T)
    if dbcx is None:
        dbcx = torch.empty_like(bcx)
    if dw is None:
        dw = torch.empty((H, K), dtype=torch.float32, device=bcx.device)
    if want_d_init and d_init is None:
        d_init = torch.empty((N, H, K), dtype=torch.float32, device=bcx.device)
    if with_dbias and dbias is None:
        dbias = torch.empty((H,), dtype=torch.float32, device=bcx.device)
    if workspace is None:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=bcx.device)
    if workspace.dtype != torch.uint8 or workspace.numel() < need:
        raise ValueError(f"workspace must be a uint8 tensor of at least {need} bytes")
    init_p = _dev(init_states, "init_states", dt, (N, H, K)) if init_states is not None else None
    dfin_p = _dev(d_final, "d_final", torch.float32, (N, H, K)) if d_final is not None else None
    dini_p = _dev(d_init, "d_init", torch.float32, (N, H, K)) if d_init is not None else None
    db_p = _dev(dbias, "dbias", torch.float32, (H,)) if with_dbias else None
    _raise_on("shortconv_backward_varlen", lib().shortconv_backward_varlen(
        _dcode(bcx), H, K, _dev(bcx, "bcx", dt), T, _dev(w, "w", dt), _bias(bias, dt, H),
        _dev(cu_seqlens, "cu_seqlens", torch.int32, (N + 1,)), N, init_p,
        _dev(dy, "dy", dt, (T, H)), dfin_p, _dev(dbcx, "dbcx", dt, (T, 3 * H)),
        _dev(dw, "dw", torch.float32, (H, K)), db_p, dini_p, _dev(workspace, "workspace"),
        workspace.numel(), _stream(stream, bcx.device)))
    return (dbcx, dw, d_init, dbias) if with_dbias else (dbcx, dw, d_init)


def in_proj_workspace_bytes(H: int, K: int, N: int) -> int:
    return int(lib().shortconv_in_proj_workspace_bytes(H, K, N))


def in_proj_prefill(hidden, w_in, w, cu_seqlens, slot_ids, pool, y=None, bias=None,
                    workspace=None, stream=None):
    """in_proj fused with the packed varlen prefill (bf16); updates ``pool`` and
    returns ``y [T, H]``. ``hidden [T, D]``, ``w_in [3H, D]`` (rows b | c | xv)."""
    dt = torch.bfloat16
    T, D = hidden.shape
    H, K = w.shape
    N = slot_ids.shape[0]
    need = in_proj_workspace_bytes(H, K, N)
    if y is None:
        y = torch.empty((T, H), dtype=dt, device=hidden.device)
    if workspace is None:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=hidden.device)
    if workspace.dtype != torch.uint8 or workspace.numel() < need:
        raise ValueError(f"workspace must be a uint8 tensor of at least {need} bytes")
    _raise_on("shortconv_in_proj_prefill", lib().shortconv_in_proj_prefill(
        _dcode(hidden), D, H, K, _dev(hidden, "hidden", dt), T,
        _dev(w_in, "w_in", dt, (3 * H, D)), _dev(w, "w", dt), _bias(bias, dt, H),
        _dev(cu_seqlens, "cu_seqlens", torch.int32, (N + 1,)), N,
        _dev(slot_ids, "slot_ids", torch.int32, (N,)),
        _dev(pool, "pool", dt, (pool.shape[0], H, K)), pool.shape[0], _dev(y, "y", dt, (T, H)),
        _dev(workspace, "workspace"), workspace.numel(), _stream(stream, hidden.device)))
    return y


def in_proj_decode(hidden, w_in, w, slot_ids, pool, y=None, bias=None, stream=None):
    """in_proj fused with the decode of one token per sequence (bf16): row i of
    ``hidden [N, D]`` is sequence i; updates ``pool`` and returns ``y [N, H]``."""
    dt = torch.bfloat16
    N, D = hidden.shape
    H, K = w.shape
    if y is None:
        y = torch.empty((N, H), dtype=dt, device=hidden.device)
    _raise_on("shortconv_in_proj_decode", lib().shortconv_in_proj_decode(
        _dcode(hidden), D, H, K, _dev(hidden, "hidden", dt), N,
        _dev(w_in, "w_in", dt, (3 * H, D)), _dev(w, "w", dt), _bias(bias, dt, H),
        _dev(slot_ids, "slot_ids", torch.int32, (N,)),
        _dev(pool, "pool", dt, (pool.shape[0], H, K)), pool.shape[0], _dev(y, "y", dt, (N, H)),
        _stream(stream, hidden.device)))
    return y


def out_proj(y, w_out, out=None, stream=None):
    """out = y w_out^T (bf16, fp32 accumulation): ``y [T, H]``, ``w_out [D, H]``."""
    dt = torch.bfloat16
    T, H = y.shape
    D = w_out.shape[0]
    if out is None:
        out = torch.empty((T, D), dtype=dt, device=y.device)
    _raise_on("shortconv_out_proj", lib().shortconv_out_proj(
        _dcode(y), H, D, _dev(y, "y", dt), T, _dev(w_out, "w_out", dt, (D, H)),
        _dev(out, "out", dt, (T, D)), _stream(stream, y.device)))
    return out


def slot_bitmap(n_slots: int, device="cuda") -> torch.Tensor:
    """An all-free in-use bitmap for ``n_slots`` slots (int32 words, bit per slot)."""
    return torch.zeros(((n_slots + 31) // 32,), dtype=torch.int32, device=device)


def slots_claim(in_use, n_slots, n_claim, pool=None, slots_out=None, stream=None):
    """Claim ``n_claim`` free slots (lowest first, all-or-nothing); zero their
    states in ``pool`` if given. Returns the int32 slot ids (-1s if none)."""
    if slots_out is None:
        slots_out = torch.empty((n_claim,), dtype=torch.int32, device=in_use.device)
    dt, H, K, pp = SC_BF16, 8, 1, None
    if pool is not None:
        dt, H, K = _dcode(pool), pool.shape[1], pool.shape[2]
        pp = _dev(pool, "pool", pool.dtype, (n_slots, H, K))
    _raise_on("shortconv_slots_claim", lib().shortconv_slots_claim(
        _dev(in_use, "in_use", torch.int32, ((n_slots + 31) // 32,)), n_slots, n_claim,
        _dev(slots_out, "slots_out", torch.int32, (n_claim,)), dt, H, K, pp,
        _stream(stream, in_use.device)))
    return slots_out


def slots_release(in_use, n_slots, slot_ids, stream=None):
    """Mark ``slot_ids`` free."""
    n = slot_ids.shape[0]
    _raise_on("shortconv_slots_release", lib().shortconv_slots_release(
        _dev(in_use, "in_use", torch.int32, ((n_slots + 31) // 32,)), n_slots,
        _dev(slot_ids, "slot_ids", torch.int32, (n,)), n, _stream(stream, in_use.device)))


def pool_copy(pool, src_slots, dst_slots, stream=None):
    """``pool[dst[i]] = pool[src[i]]`` (destinations distinct, not among sources)."""
    n_slots, H, K = pool.shape
    n = src_slots.shape[0]
    _raise_on("shortconv_pool_copy", lib().shortconv_pool_copy(
        _dcode(pool), H, K, _dev(pool, "pool", pool.dtype, (n_slots, H, K)), n_slots,
        _dev(src_slots, "src_slots", torch.int32, (n,)),
        _dev(dst_slots, "dst_slots", torch.int32, (n,)), n, _stream(stream, pool.device)))


def _rows(t, name, dtype, shape):
    """Data pointer and row stride (elements) of a CUDA tensor whose rows (the
    dims after the first) are contiguous and may lie further apart."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor, got {t.device}")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    strides, width = t.stride(), 1
    for n, s in zip(shape[:0:-1], strides[:0:-1]):
        if n != 1 and s != width:
            raise ValueError(f"{name} must have contiguous rows")
        width *= n
    return t.data_ptr(), (strides[0] if shape[0] > 1 else width)


_I32, _BF16 = torch.int32, torch.bfloat16


def _ints(t, name, shape) -> int:
    """``_dev`` for an int32 array, with one test on the way that calls usually take."""
    if (type(t) is torch.Tensor and t.is_cuda and t.dtype is _I32 and t.is_contiguous()
            and t.shape == shape):
        return t.data_ptr()
    return _dev(t, name, _I32, shape)


def _cache(refs, table, lens):
    n_slots, max_pages = table.shape
    n_pages = refs.shape[0]
    return (_ints(refs, "refs", (n_pages,)), n_pages, _ints(table, "table", (n_slots, max_pages)),
            _ints(lens, "lens", (n_slots,)), n_slots, max_pages)


def _pools(k_pages, v_pages, n_pages):
    """(page_size, L, token_bytes, k, v) of [L, n_pages, page_size, Hkv, Dh] or
    [n_pages, page_size, Hkv, Dh] pools."""
    full = k_pages.shape
    shape = full if len(full) == 5 else (1,) + full
    if len(shape) != 5 or shape[1] != n_pages:
        raise ValueError("k_pages must be [L, n_pages, page_size, Hkv, Dh] or "
                         "[n_pages, page_size, Hkv, Dh]")
    _dcode(k_pages)
    return (shape[2], shape[0], shape[3] * shape[4] * k_pages.element_size(),
            _dev(k_pages, "k_pages"), _dev(v_pages, "v_pages", k_pages.dtype, full))


# Scratch straight from torch's caching allocator: no tensor object (3 us of host time a
# call), and the block belongs to the stream that the call runs on, so that it is safe
# to give back as soon as the call is enqueued.
_raw_alloc = getattr(torch._C, "_cuda_cudaCachingAllocator_raw_alloc", None)
_raw_delete = getattr(torch._C, "_cuda_cudaCachingAllocator_raw_delete", None)
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _call_with_workspace(name, fn, workspace, need, device, stream, *args):
    """``fn(*args, workspace, bytes, stream)``, with the caller's workspace or one of its own."""
    st = _stream(stream, device)
    if workspace is not None:
        if workspace.dtype != torch.uint8 or workspace.numel() < need:
            raise ValueError(f"workspace must be a uint8 tensor of at least {need} bytes")
        status = fn(*args, _dev(workspace, "workspace"), workspace.numel(), st)
    elif _raw_alloc is not None and _raw_delete is not None and device.index == _current_device():
        p = _raw_alloc(max(need, 16), st)
        try:
            status = fn(*args, p, need, st)
        finally:
            _raw_delete(p)
    else:
        with torch.cuda.stream(stream if stream is not None else torch.cuda.current_stream(device)):
            ws = torch.empty(max(need, 16), dtype=torch.uint8, device=device)
        status = fn(*args, ws.data_ptr(), need, st)
    if status:
        _raise_on(name, status)


def _output(shape, dtype, device, stream):
    """A new tensor that belongs to the stream the call runs on, for the same reason."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def page_cache(n_slots: int, max_pages: int, n_pages: int, device="cuda"):
    """``(refs [n_pages], table [n_slots, max_pages], lens [n_slots])`` of an empty cache."""
    i32 = dict(dtype=torch.int32, device=device)
    return (torch.zeros((n_pages,), **i32), torch.full((n_slots, max_pages), -1, **i32),
            torch.zeros((n_slots,), **i32))


@functools.lru_cache(maxsize=1024)
def pages_workspace_bytes(n_pages: int, n: int) -> int:
    return int(lib().shortconv_pages_workspace_bytes(n_pages, n))


def pages_resize(refs, table, lens, slot_ids, new_lens, k_pages, v_pages, workspace=None,
                 stream=None):
    """Give each listed sequence a new length: claims, truncates (a rollback) or frees
    (0) its pages; in place on ``refs``, ``table``, ``lens`` and, where a shared page
    has to be copied, on the pools."""
    n = slot_ids.shape[0]
    ps, L, token_bytes, kp, vp = _pools(k_pages, v_pages, refs.shape[0])
    _call_with_workspace(
        "shortconv_pages_resize", lib().shortconv_pages_resize, workspace,
        pages_workspace_bytes(refs.shape[0], n), refs.device, stream,
        *_cache(refs, table, lens), ps, _ints(slot_ids, "slot_ids", (n,)),
        _ints(new_lens, "new_lens", (n,)), n, L, token_bytes, kp, vp)


def pages_fork(refs, table, lens, src_slots, dst_slots, k_pages, v_pages, workspace=None,
               stream=None):
    """``dst_slots[i]`` becomes a branch of ``src_slots[i]``: full pages shared, a partly
    filled last page copied. In place."""
    n = src_slots.shape[0]
    ps, L, token_bytes, kp, vp = _pools(k_pages, v_pages, refs.shape[0])
    _call_with_workspace(
        "shortconv_pages_fork", lib().shortconv_pages_fork, workspace,
        pages_workspace_bytes(refs.shape[0], n), refs.device, stream,
        *_cache(refs, table, lens), ps, _ints(src_slots, "src_slots", (n,)),
        _ints(dst_slots, "dst_slots", (n,)), n, L, token_bytes, kp, vp)


def pages_compact(refs, table, lens, k_pages, v_pages, n_used=None, workspace=None, stream=None):
    """Move the used pages to the front of the pools (in place); returns the int32
    ``n_used [1]``: no page at or past it is in use."""
    ps, L, token_bytes, kp, vp = _pools(k_pages, v_pages, refs.shape[0])
    if n_used is None:
        n_used = _output((1,), _I32, refs.device, stream)
    _call_with_workspace(
        "shortconv_pages_compact", lib().shortconv_pages_compact, workspace,
        pages_workspace_bytes(refs.shape[0], 0), refs.device, stream,
        *_cache(refs, table, lens), ps, L, token_bytes, kp, vp,
        _ints(n_used, "n_used", (1,)))
    return n_used


def pages_append(k, v, k_pages, v_pages, table, lens, slot_ids, D, stream=None):
    """Write each listed sequence's ``D`` newest tokens, already counted in ``lens``:
    ``k``, ``v`` ``[N*D, Hkv, Dh]`` (rows may be strided) into one layer's pools."""
    N = slot_ids.shape[0]
    pool = k_pages.shape
    n_pages, ps, Hkv, Dh = pool
    n_slots, max_pages = table.shape
    dt = k_pages.dtype
    es = 2 if dt is _BF16 else 4 if _dcode(k_pages) == SC_F32 else 0
    k_p, k_s = _rows(k, "k", dt, (N * D, Hkv, Dh))
    v_p, v_s = _rows(v, "v", dt, (N * D, Hkv, Dh))
    status = lib().shortconv_pages_append(
        k_p, k_s * es, v_p, v_s * es, N, D, Hkv * Dh * es, _dev(k_pages, "k_pages"),
        _dev(v_pages, "v_pages", dt, pool), n_pages, ps,
        _ints(table, "table", (n_slots, max_pages)), _ints(lens, "lens", (n_slots,)), n_slots,
        max_pages, _ints(slot_ids, "slot_ids", (N,)), _stream(stream, k_pages.device))
    if status:
        _raise_on("shortconv_pages_append", status)


@functools.lru_cache(maxsize=1024)
def prefix_attention_workspace_bytes(Hq, Hkv, Dh, N, D, shared_pages=0) -> int:
    return int(lib().shortconv_prefix_attention_workspace_bytes(Hq, Hkv, Dh, N, D, shared_pages))


def prefix_attention(q, k_pages, v_pages, table, lens, slot_ids, D, shared_pages=0, scale=None,
                     out=None, workspace=None, stream=None):
    """Attention of a decode (``D`` = 1) or verify step over the paged cache (bf16):
    row ``i*D + j`` of ``q [N*D, Hq, Dh]`` (rows may be strided) is new token j of the
    sequence in ``slot_ids[i]``. The first ``shared_pages`` pages are the same for all
    listed sequences and read once. Returns ``out [N*D, Hq, Dh]``."""
    N = slot_ids.shape[0]
    pool = k_pages.shape
    n_pages, ps, Hkv, Dh = pool
    n_slots, max_pages = table.shape
    Hq = q.shape[1]
    rows = (N * D, Hq, Dh)
    device = q.device
    if scale is None:
        scale = Dh ** -0.5
    if out is None:
        out = _output(rows, _BF16, device, stream)
        out_p = out.data_ptr()
    else:
        out_p = _dev(out, "out", _BF16, rows)
    q_p, q_s = _rows(q, "q", _BF16, rows)
    _call_with_workspace(
        "shortconv_prefix_attention", lib().shortconv_prefix_attention, workspace,
        prefix_attention_workspace_bytes(Hq, Hkv, Dh, N, D, shared_pages), device, stream,
        SC_BF16, Hq, Hkv, Dh, q_p, q_s, N, D, _dev(k_pages, "k_pages", _BF16),
        _dev(v_pages, "v_pages", _BF16, pool), n_pages, ps,
        _ints(table, "table", (n_slots, max_pages)), _ints(lens, "lens", (n_slots,)), n_slots,
        max_pages, _ints(slot_ids, "slot_ids", (N,)), shared_pages, scale, out_p)
    return out


def draft_accept(target, draft, tokens, uniforms, n_drafts=None, accepted=None, out_tokens=None,
                 stream=None):
    """Verify drafts against the target: ``target [N, D+1, V]`` and ``draft [N, D, V]``
    (None: certain drafts) are probabilities (float32 or bfloat16; a last dim sliced
    from wider rows is fine, broadcast rows are refused), ``tokens [N, D]`` int32,
    ``uniforms [N, D+1]`` float32, ``n_drafts [N]`` int32 or None. Returns int32
    ``(accepted [N], out_tokens [N, D+1])``: the accepted drafts, the next token, then -1."""
    N, D1, V = target.shape
    D = D1 - 1
    dt = target.dtype
    code = SC_F32 if dt is torch.float32 else _dcode(target)
    device = target.device
    t_p, t_s = _prob_rows(target, "target", dt, (N, D1, V))
    d_p, d_s = (None, V) if draft is None else _prob_rows(draft, "draft", dt, (N, D, V))
    if accepted is None:
        accepted = _output((N,), _I32, device, stream)
    if out_tokens is None:
        out_tokens = _output((N, D1), _I32, device, stream)
    status = lib().shortconv_draft_accept(
        code, V, N, D, t_p, t_s, d_p, d_s, _ints(tokens, "tokens", (N, D)),
        None if n_drafts is None else _ints(n_drafts, "n_drafts", (N,)),
        _dev(uniforms, "uniforms", torch.float32, (N, D1)), _ints(accepted, "accepted", (N,)),
        _ints(out_tokens, "out_tokens", (N, D1)), _stream(stream, device))
    if status:
        _raise_on("shortconv_draft_accept", status)
    return accepted, out_tokens


def _prob_rows(t, name, dtype, shape):
    """Data pointer and row distance of ``[N, n, V]`` probabilities whose rows are
    contiguous and evenly spaced, at least V apart (broadcast rows are not)."""
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor, got {t.device}")
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    N, n, V = shape
    s0, s1, s2 = t.stride()
    step = V if N * n <= 1 else s1 if n > 1 else s0  # of a single row: any
    if (V > 1 and s2 != 1) or (n > 1 and N > 1 and s0 != n * s1) or step < V:
        raise ValueError(f"{name} must have contiguous, evenly spaced rows that do not overlap "
                         f"(broadcast ones: .contiguous()), got strides {t.stride()}")
    return t.data_ptr(), step


def check_wait_limit(stream=None, device=None) -> None:
    """Enqueue the device-side timeout check: a kernel whose bounded wait runs
    out (about 2 s) and sets DEV_TIMEOUT, which get_error() then returns."""
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else device
    _raise_on("shortconv_check_wait_limit", lib().shortconv_check_wait_limit(_stream(stream, dev)))


def get_error(stream=None, device=None) -> int:
    """Synchronize the stream, return and clear the device error word (SC_DEV_* bits)."""
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else device
    code = ctypes.c_int(0)
    st = lib().shortconv_get_error(_stream(stream, dev), ctypes.byref(code))
    if st not in (SC_OK, SC_EDEVICE):
        _raise_on("shortconv_get_error", st)
    return code.value


def bounds_checked() -> bool:
    """True when the loaded library is the bounds-checked build."""
    return bool(lib().shortconv_bounds_checked())


def bounds_trim_next(region: int, nbytes: int) -> None:
    """Bounds-checked build: shorten buffer ``region`` of the next call's record."""
    _raise_on("shortconv_bounds_trim_next", lib().shortconv_bounds_trim_next(region, nbytes))


def bounds_take_first_bad(stream=None, device=None) -> int:
    """Bounds-checked build: the first refused device address since the last take (0: none)."""
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else device
    addr = ctypes.c_uint64(0)
    _raise_on("shortconv_bounds_take_first_bad",
              lib().shortconv_bounds_take_first_bad(_stream(stream, dev), ctypes.byref(addr)))
    return addr.value
