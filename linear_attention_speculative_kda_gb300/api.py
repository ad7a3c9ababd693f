"""Thin ctypes binding of ``libkda.so`` (the C ABI of ``include/kda.h``).

Argument marshalling only: every function checks dtypes, devices and shapes
of the torch tensors it is given, fills a ``kda_config`` and passes raw
device pointers and the current CUDA stream to the entry point of the same
name.  Every step of the method runs in the library's CUDA kernels; there is
no fallback of any kind.  If the library has not been built, the first call
raises.
"""

from __future__ import annotations

import ctypes
import functools
import os
import struct
from typing import NamedTuple

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
_LIBRARY = os.path.join(_PKG, "libkda.so")

HEAD_DIM = 128
MAX_WINDOW = 8
RECORD_STRIDE = 392          # bf16 elements per token record (k, v, g, beta, pad)
CORRECTION_RECORD_BYTES = 1024  # fp32 delta, bf16 k, bf16 g_raw per token
RECORD_FORMATS = {"raw": 0, "correction": 1}

KDA_OK = 0
KDA_ERR_INVALID_ARG = 1
KDA_ERR_UNSUPPORTED = 2
KDA_ERR_CUDA = 3

ROW_BAD_LENGTH = 1
ROW_BAD_SLOT = 2
ROW_BAD_RECORD = 4
ROW_BAD_PENDING = 8
ERR_WAIT_TIMEOUT = 16
ROW_BAD_BLOCK = 32
ROW_BAD_TOKEN = 64

MAX_QUERY_ROWS = 128         # window * q_heads / kv_heads of kda_window_attention
MAX_TOP = 32                 # alternatives of kda_token_logprobs
DTYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}

EXPORTED = (
    "kda_records_bytes",
    "kda_correction_records_bytes",
    "kda_verify",
    "kda_commit",
    "kda_flush",
    "kda_conv_compact",
    "kda_commit_align",
    "kda_conv_compact_align",
    "kda_record_state_blocks",
    "kda_kv_append",
    "kda_attention_workspace_bytes",
    "kda_window_attention",
    "kda_token_logprobs",
    "kda_prefill",
    "kda_decode",
    "kda_kv_norm_append",
    "kda_kv_append_packed",
    "kda_kv_norm_append_packed",
    "kda_prefill_packed",
    "kda_decode_packed",
    "kda_window_attention_packed",
    "kda_token_logprobs_packed",
    "kda_status_string",
    "kda_abi_version",
)


class KDAError(RuntimeError):
    """A call into libkda returned a status other than KDA_OK."""

    def __init__(self, fn: str, status: int):
        super().__init__(f"{fn} failed: status {status} ({_status_name(status)})")
        self.status = status


class KdaConfig(ctypes.Structure):
    _fields_ = [
        ("num_heads", ctypes.c_int32),
        ("head_dim", ctypes.c_int32),
        ("window", ctypes.c_int32),
        ("num_slots", ctypes.c_int32),
        ("record_slots", ctypes.c_int32),
        ("use_lower_bound", ctypes.c_int32),
        ("lower_bound", ctypes.c_float),
        ("scale", ctypes.c_float),
        ("stride_q_t", ctypes.c_int64),
        ("stride_k_t", ctypes.c_int64),
        ("stride_v_t", ctypes.c_int64),
        ("stride_g_t", ctypes.c_int64),
        ("stride_beta_t", ctypes.c_int64),
        ("record_format", ctypes.c_int32),
        ("reserved", ctypes.c_int32),
    ]


class KdaConvConfig(ctypes.Structure):
    _fields_ = [
        ("num_slots", ctypes.c_int32),
        ("conv_dim", ctypes.c_int32),
        ("width", ctypes.c_int32),
        ("window", ctypes.c_int32),
        ("elem_bytes", ctypes.c_int32),
        ("reserved", ctypes.c_int32),
        ("stride_slot", ctypes.c_int64),
        ("stride_dim", ctypes.c_int64),
        ("stride_col", ctypes.c_int64),
    ]


MAX_CONV_HISTORY = 16


class KdaAlign(ctypes.Structure):
    _fields_ = [
        ("block_table", ctypes.c_void_p),
        ("block_table_stride", ctypes.c_int64),
        ("block_table_width", ctypes.c_int32),
        ("block_size", ctypes.c_int32),
        ("num_requests", ctypes.c_int32),
        ("reserved", ctypes.c_int32),
        ("num_computed", ctypes.c_void_p),
        ("request_indices", ctypes.c_void_p),
    ]


class KdaCacheConfig(ctypes.Structure):
    _fields_ = [
        ("q_heads", ctypes.c_int32),
        ("kv_heads", ctypes.c_int32),
        ("head_dim", ctypes.c_int32),
        ("dtype", ctypes.c_int32),
        ("num_blocks", ctypes.c_int32),
        ("window", ctypes.c_int32),
        ("left_window", ctypes.c_int32),
        ("rotary_dim", ctypes.c_int32),
        ("interleaved", ctypes.c_int32),
        ("scale", ctypes.c_float),
        ("stride_block", ctypes.c_int64),
        ("stride_token", ctypes.c_int64),
        ("stride_head", ctypes.c_int64),
        ("stride_q_t", ctypes.c_int64),
        ("stride_k_t", ctypes.c_int64),
        ("stride_v_t", ctypes.c_int64),
    ]


_quick = None        # the compiled part of the binding of the short calls
_quick_more = None   # the same, for those whose argument structures it records apart
_lib_handle = None


def library_path() -> str:
    return _LIBRARY


def load_library():
    """Load libkda.so (once).  Raises if it is missing: there is no fallback."""
    global _lib_handle
    if _lib_handle is not None:
        return _lib_handle
    if not os.path.exists(_LIBRARY):
        raise RuntimeError(
            f"libkda.so not found at {_LIBRARY}; build it first "
            "(python -c 'import __graft_entry__ as g; g.build()')")
    _lib_handle = bind_library(_LIBRARY)
    _load_quick()
    return _lib_handle


def _load_quick():
    """The compiled part of the binding of the short calls, where it was built
    for these argument structures and this PyTorch."""
    global _quick, _quick_more
    try:
        from . import _binding
    except ImportError:
        _binding = None
    fits = (getattr(_binding, "torch_version", None) == torch.__version__
            and _binding.argument_sizes == _ARGUMENT_SIZES)
    _quick = _binding if fits else None
    _quick_more = (_quick if getattr(_quick, "more_argument_sizes", None) == _MORE_ARGUMENT_SIZES
                   else None)


def bind_library(path: str):
    """A ctypes handle of a build of the library at ``path`` (libkda.so, or a
    test variant from build.build_variant) with every entry point's argument
    types declared."""
    lib = ctypes.CDLL(path)
    vp, i32 = ctypes.c_void_p, ctypes.c_int32
    cfgp = ctypes.POINTER(KdaConfig)
    lib.kda_records_bytes.restype = ctypes.c_size_t
    lib.kda_records_bytes.argtypes = [i32, i32, i32]
    lib.kda_correction_records_bytes.restype = ctypes.c_size_t
    lib.kda_correction_records_bytes.argtypes = [i32, i32, i32]
    lib.kda_verify.restype = ctypes.c_int
    lib.kda_verify.argtypes = [cfgp] + [vp] * 10 + [i32] + [vp] * 7
    lib.kda_commit.restype = ctypes.c_int
    lib.kda_commit.argtypes = [cfgp] + [vp] * 5 + [i32] + [vp] * 7
    lib.kda_flush.restype = ctypes.c_int
    lib.kda_flush.argtypes = [cfgp] + [vp] * 4 + [i32] + [vp] * 5
    lib.kda_conv_compact.restype = ctypes.c_int
    lib.kda_conv_compact.argtypes = [ctypes.POINTER(KdaConvConfig)] + [vp] * 3 + [i32] + [vp] * 3
    alp = ctypes.POINTER(KdaAlign)
    lib.kda_commit_align.restype = ctypes.c_int
    lib.kda_commit_align.argtypes = [cfgp] + [vp] * 5 + [i32] + [vp] * 3 + [alp, vp, vp, vp, vp]
    lib.kda_conv_compact_align.restype = ctypes.c_int
    lib.kda_conv_compact_align.argtypes = ([ctypes.POINTER(KdaConvConfig)] + [vp] * 3 + [i32] +
                                           [vp, alp, vp, vp])
    lib.kda_record_state_blocks.restype = ctypes.c_int
    lib.kda_record_state_blocks.argtypes = [alp, vp, vp, i32, vp, vp, i32, vp, vp]
    ccp = ctypes.POINTER(KdaCacheConfig)
    lib.kda_kv_append.restype = ctypes.c_int
    lib.kda_kv_append.argtypes = [ccp] + [vp] * 8 + [i32, i32, alp, vp, vp]
    lib.kda_attention_workspace_bytes.restype = ctypes.c_size_t
    lib.kda_attention_workspace_bytes.argtypes = [ccp, i32]
    lib.kda_window_attention.restype = ctypes.c_int
    lib.kda_window_attention.argtypes = ([ccp] + [vp] * 4 + [i32, i32, alp, vp, ctypes.c_size_t] +
                                         [vp] * 4)
    lib.kda_token_logprobs.restype = ctypes.c_int
    lib.kda_token_logprobs.argtypes = [vp, i32, ctypes.c_int64, i32, i32, vp, i32] + [vp] * 7
    delta = [cfgp] + [vp] * 8
    lib.kda_prefill.restype = ctypes.c_int
    lib.kda_prefill.argtypes = delta + [vp, vp, vp, i32, i32, vp, vp, vp]
    lib.kda_decode.restype = ctypes.c_int
    lib.kda_decode.argtypes = delta + [vp, vp, i32, vp, vp, vp]
    lib.kda_kv_norm_append.restype = ctypes.c_int
    lib.kda_kv_norm_append.argtypes = ([ccp] + [vp] * 5 + [i32, ctypes.c_float] + [vp] * 5 +
                                       [i32, i32, alp, vp, vp])
    for fn in (lib.kda_kv_append_packed, lib.kda_window_attention_packed,
               lib.kda_token_logprobs_packed, lib.kda_kv_norm_append_packed,
               lib.kda_prefill_packed, lib.kda_decode_packed):
        fn.restype = ctypes.c_int
        fn.argtypes = [ctypes.c_char_p]   # the bytes of the argument structure
    lib.kda_status_string.restype = ctypes.c_char_p
    lib.kda_status_string.argtypes = [ctypes.c_int]
    lib.kda_abi_version.restype = i32
    lib.kda_abi_version.argtypes = []
    # for the compiled part of the binding, which calls the library it is given
    (lib.append_address, lib.attend_address, lib.logprobs_address, lib.norm_append_address,
     lib.prefill_address, lib.decode_address) = (
        ctypes.cast(fn, vp).value for fn in (lib.kda_kv_append_packed,
                                             lib.kda_window_attention_packed,
                                             lib.kda_token_logprobs_packed,
                                             lib.kda_kv_norm_append_packed,
                                             lib.kda_prefill_packed, lib.kda_decode_packed))
    return lib


def _status_name(status: int) -> str:
    try:
        return load_library().kda_status_string(status).decode()
    except Exception:  # pragma: no cover - only for messages
        return "?"


def _check(fn: str, status: int) -> None:
    if status != KDA_OK:
        raise KDAError(fn, status)


def _ptr(t):
    # a plain int: ctypes converts it for c_void_p parameters (None is NULL)
    return None if t is None else t.data_ptr()


def _stream_ptr(device) -> int:
    return torch.cuda.current_stream(device).cuda_stream


def _on(index: int, fn, *args):
    """fn(*args) with the tensors' GPU as the current one: the library launches
    on the current device, and a stream handle may not say which it belongs to."""
    if index == torch.cuda.current_device():
        return fn(*args)
    with torch.cuda.device(index):
        return fn(*args)


def _token_stride(t: torch.Tensor) -> int:
    # [T, H, D] (or [1, T, H, D]) activation with heads and channels packed
    if t.dim() == 4:
        t = t[0]
    if t.dim() == 3:
        if t.stride(2) != 1 or t.stride(1) != t.shape[2]:
            raise ValueError("activations need contiguous [H, D] inside a token")
    elif t.dim() == 2:
        if t.stride(1) != 1:
            raise ValueError("beta needs contiguous heads inside a token")
    else:
        raise ValueError("unexpected activation rank")
    return t.stride(0) if t.shape[0] > 1 else max(t.stride(0), 1)


def _req(t, dtype, name, device):
    if t is None:
        raise ValueError(f"{name} is required")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.device != device:
        raise ValueError(f"{name} must be on {device}")
    return t


def _opt(t, dtype, name, device):
    return None if t is None else _req(t, dtype, name, device)


# Shape and size checks.  The C ABI takes bare pointers and cannot see how
# large a buffer is, so the binding checks every tensor the kernels index
# against the sizes the call implies, before anything is launched.

def _tokens(t, name, H, D):
    """Token count of a [T, H, D] (or [1, T, H, D]) activation, or of a
    [T, H] (or [1, T, H]) one when D is None."""
    lead = 4 if D is not None else 3
    if t.dim() == lead:
        if t.shape[0] != 1:
            raise ValueError(f"{name}: a leading batch dimension must be 1")
        t = t[0]
    want = (H, D) if D is not None else (H,)
    if t.dim() != len(want) + 1 or tuple(t.shape[1:]) != want:
        shape = "[T, H, D]" if D is not None else "[T, H]"
        raise ValueError(f"{name} must be {shape} with H={H}" +
                         (f", D={D}" if D is not None else "") + f", got {tuple(t.shape)}")
    return t.shape[0]


def _at_least(t, n, name):
    if t is not None and t.numel() < n:
        raise ValueError(f"{name} needs at least {n} elements, has {t.numel()}")


def _check_pool(state_pool):
    if (state_pool.dim() != 4 or not state_pool.is_contiguous()
            or state_pool.shape[2] != state_pool.shape[3]):
        raise ValueError("state_pool must be a contiguous [S, H, V, K] tensor with V == K")
    return state_pool.shape[0], state_pool.shape[1], state_pool.shape[3]


def _check_gate(A_log, g_bias, H, D):
    if not A_log.is_contiguous() or not g_bias.is_contiguous():
        raise ValueError("A_log and g_bias must be contiguous")
    _at_least(A_log, H, "A_log")
    _at_least(g_bias, H * D, "g_bias")


def _check_rows(B, record_slots, record_rows=None, pending=None, eager=None, error_word=None):
    for name, t in (("record_rows", record_rows), ("pending", pending), ("eager", eager),
                    ("error_word", error_word)):
        if t is not None and not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
    _at_least(record_rows, B, "record_rows")
    _at_least(pending, record_slots, "pending")
    _at_least(eager, B, "eager")
    _at_least(error_word, 1, "error_word")


def _format_code(record_format: str) -> int:
    try:
        return RECORD_FORMATS[record_format]
    except KeyError:
        raise ValueError(f"record_format must be one of {sorted(RECORD_FORMATS)}") from None


def make_config(num_heads, window, num_slots, record_slots, *, lower_bound=None,
                scale=None, strides=(1, 1, 1, 1, 1), head_dim=HEAD_DIM,
                record_format: str = "raw") -> KdaConfig:
    """A new ``kda_config`` (the entry points below share read-only cached
    ones, see ``_config``)."""
    cfg = KdaConfig()
    cfg.record_format = _format_code(record_format)
    cfg.reserved = 0
    cfg.num_heads = num_heads
    cfg.head_dim = head_dim
    cfg.window = window
    cfg.num_slots = num_slots
    cfg.record_slots = record_slots
    cfg.use_lower_bound = 0 if lower_bound is None else 1
    cfg.lower_bound = 0.0 if lower_bound is None else float(lower_bound)
    cfg.scale = head_dim ** -0.5 if scale is None else float(scale)
    (cfg.stride_q_t, cfg.stride_k_t, cfg.stride_v_t, cfg.stride_g_t,
     cfg.stride_beta_t) = [int(s) for s in strides]
    return cfg


@functools.lru_cache(maxsize=256)
def _config(num_heads, window, num_slots, record_slots, lower_bound, scale, strides, head_dim,
            record_format) -> KdaConfig:
    # the library only reads the config during the call, so one object per
    # distinct argument set serves every call
    return make_config(num_heads, window, num_slots, record_slots, lower_bound=lower_bound,
                       scale=scale, strides=strides, head_dim=head_dim,
                       record_format=record_format)


def kda_records_bytes(num_heads: int, window: int, record_slots: int) -> int:
    """Size in bytes of a raw-format records buffer (``kda_records_bytes``)."""
    return int(load_library().kda_records_bytes(num_heads, window, record_slots))


def kda_correction_records_bytes(num_heads: int, window: int, record_slots: int) -> int:
    """Size in bytes of a correction-format records buffer
    (``kda_correction_records_bytes``)."""
    return int(load_library().kda_correction_records_bytes(num_heads, window, record_slots))


@functools.lru_cache(maxsize=256)
def records_bytes(num_heads: int, window: int, record_slots: int, record_format: str) -> int:
    _format_code(record_format)
    fn = kda_records_bytes if record_format == "raw" else kda_correction_records_bytes
    return fn(num_heads, window, record_slots)


def allocate_records(num_heads: int, window: int, record_slots: int, device,
                     record_format: str = "raw") -> torch.Tensor:
    """A records buffer (raw or correction format) for ``record_slots``
    slots plus the scratch row, as a flat bf16 tensor."""
    nbytes = records_bytes(num_heads, window, record_slots, record_format)
    if nbytes == 0:
        raise ValueError("invalid record sizes")
    return torch.empty(nbytes // 2, dtype=torch.bfloat16, device=device)


def _check_records(records, H, window, record_slots, record_format):
    """The records buffer holds the format's size (sizes the library does
    not support are left for it to report)."""
    need = records_bytes(H, window, record_slots, record_format)
    if need > 0 and (records.numel() * records.element_size() < need
                     or not records.is_contiguous()):
        raise ValueError(f"records must be a contiguous buffer of at least {need} bytes "
                         f"for the {record_format} format")


def kda_verify(q, k, v, g_raw, beta_raw, A_log, g_bias, state_pool, cu_seqlens,
               state_indices, records, out, *, window: int, record_slots: int,
               lower_bound=None, scale=None, record_rows=None, pending=None,
               trajectory_out=None, error_word=None, record_format: str = "raw") -> torch.Tensor:
    """``kda_verify``: speculative verify from each row's checkpoint.

    q, k, v, g_raw: bf16 [T, H, 128] (token stride free, [H, D] packed);
    beta_raw: bf16 [T, H]; A_log fp32 [H]; g_bias fp32 [H*128];
    state_pool fp32 [S, H, 128, 128]; cu_seqlens int32 [B+1];
    state_indices int32 [B]; records: buffer from ``allocate_records``
    for the same ``record_format`` ("raw": k, v, g_raw and beta_raw per
    token; "correction": each token's fp32 delta with k and g_raw);
    out: bf16 [T, H, 128] contiguous.  Returns ``out``.
    """
    dev = state_pool.device
    bf, f32, i32 = torch.bfloat16, torch.float32, torch.int32
    for name, t in (("q", q), ("k", k), ("v", v), ("g_raw", g_raw), ("beta_raw", beta_raw),
                    ("records", records), ("out", out)):
        _req(t, bf, name, dev)
    for name, t in (("A_log", A_log), ("g_bias", g_bias), ("state_pool", state_pool)):
        _req(t, f32, name, dev)
    _req(cu_seqlens, i32, "cu_seqlens", dev)
    _req(state_indices, i32, "state_indices", dev)
    _opt(record_rows, i32, "record_rows", dev)
    _opt(pending, i32, "pending", dev)
    _opt(trajectory_out, f32, "trajectory_out", dev)
    _opt(error_word, i32, "error_word", dev)
    S, H, D = _check_pool(state_pool)
    _check_gate(A_log, g_bias, H, D)
    for t in (cu_seqlens, state_indices):
        if not t.is_contiguous():
            raise ValueError("metadata tensors must be contiguous")
    B = state_indices.shape[0]
    if cu_seqlens.shape[0] != B + 1:
        raise ValueError("cu_seqlens must have B + 1 entries")
    _check_rows(B, record_slots, record_rows, pending, None, error_word)
    T = _tokens(q, "q", H, D)
    for name, t in (("k", k), ("v", v), ("g_raw", g_raw), ("out", out)):
        if _tokens(t, name, H, D) != T:
            raise ValueError(f"{name} has a different token count from q")
    if _tokens(beta_raw, "beta_raw", H, None) != T:
        raise ValueError("beta_raw has a different token count from q")
    if not out.is_contiguous():
        raise ValueError("out must be contiguous")
    if trajectory_out is not None:
        if not trajectory_out.is_contiguous():
            raise ValueError("trajectory_out must be contiguous")
        _at_least(trajectory_out, T * H * D * D, "trajectory_out")
    strides = (_token_stride(q), _token_stride(k), _token_stride(v), _token_stride(g_raw),
               _token_stride(beta_raw))
    cfg = _config(H, window, S, record_slots, lower_bound, scale, strides, state_pool.shape[-1],
                  record_format)
    _check_records(records, H, window, record_slots, record_format)
    lib = load_library()
    st = _on(dev.index, lib.kda_verify, ctypes.byref(cfg), _ptr(q), _ptr(k), _ptr(v), _ptr(g_raw),
             _ptr(beta_raw), _ptr(A_log), _ptr(g_bias), _ptr(state_pool), _ptr(cu_seqlens),
             _ptr(state_indices), B, _ptr(record_rows), _ptr(pending), _ptr(records), _ptr(out),
             _ptr(trajectory_out), _ptr(error_word), _stream_ptr(dev))
    _check("kda_verify", st)
    return out


def kda_commit(A_log, g_bias, state_pool, cu_seqlens, state_indices, num_accepted, records,
               *, window: int, record_slots: int, lower_bound=None, record_rows=None,
               pending=None, eager=None, error_word=None, record_format: str = "raw") -> None:
    """``kda_commit``: fold each row's accepted tokens into its checkpoint
    (eager), or store them as pending replays (deferred, ``pending`` given).
    ``record_format`` must be the one the verify wrote ``records`` with."""
    dev = state_pool.device
    f32, i32 = torch.float32, torch.int32
    for name, t in (("A_log", A_log), ("g_bias", g_bias), ("state_pool", state_pool)):
        _req(t, f32, name, dev)
    _req(records, torch.bfloat16, "records", dev)
    _req(cu_seqlens, i32, "cu_seqlens", dev)
    _req(state_indices, i32, "state_indices", dev)
    _req(num_accepted, i32, "num_accepted", dev)
    _opt(record_rows, i32, "record_rows", dev)
    _opt(pending, i32, "pending", dev)
    _opt(eager, torch.uint8, "eager", dev)
    _opt(error_word, i32, "error_word", dev)
    S, H, D = _check_pool(state_pool)
    _check_gate(A_log, g_bias, H, D)
    B = state_indices.shape[0]
    for t in (cu_seqlens, state_indices, num_accepted):
        if not t.is_contiguous():
            raise ValueError("metadata tensors must be contiguous")
    if cu_seqlens.shape[0] != B + 1 or num_accepted.shape[0] < B:
        raise ValueError("metadata sizes do not match the batch")
    _check_rows(B, record_slots, record_rows, pending, eager, error_word)
    cfg = _config(H, window, S, record_slots, lower_bound, None, (1, 1, 1, 1, 1), D,
                  record_format)
    _check_records(records, H, window, record_slots, record_format)
    lib = load_library()
    st = _on(dev.index, lib.kda_commit, ctypes.byref(cfg), _ptr(A_log), _ptr(g_bias),
             _ptr(state_pool), _ptr(cu_seqlens), _ptr(state_indices), B, _ptr(num_accepted),
             _ptr(record_rows), _ptr(records), _ptr(pending), _ptr(eager), _ptr(error_word),
             _stream_ptr(dev))
    _check("kda_commit", st)


def kda_flush(A_log, g_bias, state_pool, state_indices, records, pending, *, window: int,
              record_slots: int, lower_bound=None, record_rows=None, error_word=None,
              record_format: str = "raw") -> None:
    """``kda_flush``: fold pending replays into the checkpoints in place
    (``record_format`` as for ``kda_commit``)."""
    dev = state_pool.device
    f32, i32 = torch.float32, torch.int32
    for name, t in (("A_log", A_log), ("g_bias", g_bias), ("state_pool", state_pool)):
        _req(t, f32, name, dev)
    _req(records, torch.bfloat16, "records", dev)
    _req(state_indices, i32, "state_indices", dev)
    _req(pending, i32, "pending", dev)
    _opt(record_rows, i32, "record_rows", dev)
    _opt(error_word, i32, "error_word", dev)
    S, H, D = _check_pool(state_pool)
    _check_gate(A_log, g_bias, H, D)
    B = state_indices.shape[0]
    if not state_indices.is_contiguous():
        raise ValueError("metadata tensors must be contiguous")
    _check_rows(B, record_slots, record_rows, pending, None, error_word)
    cfg = _config(H, window, S, record_slots, lower_bound, None, (1, 1, 1, 1, 1), D,
                  record_format)
    _check_records(records, H, window, record_slots, record_format)
    lib = load_library()
    st = _on(dev.index, lib.kda_flush, ctypes.byref(cfg), _ptr(A_log), _ptr(g_bias),
             _ptr(state_pool), _ptr(state_indices), B, _ptr(record_rows), _ptr(records),
             _ptr(pending), _ptr(error_word), _stream_ptr(dev))
    _check("kda_flush", st)


def make_conv_config(conv_state: torch.Tensor, window: int) -> KdaConvConfig:
    """``kda_conv_config`` of a conv-state pool viewed as [S, conv_dim, width]
    (any strides: a channel-major pool or a transposed view of a
    column-major one)."""
    if conv_state.dim() != 3:
        raise ValueError("conv_state must be viewed as [S, conv_dim, width]")
    cc = KdaConvConfig()
    cc.num_slots, cc.conv_dim, cc.width = (int(x) for x in conv_state.shape)
    cc.window = window
    cc.elem_bytes = conv_state.element_size()
    cc.reserved = 0
    cc.stride_slot, cc.stride_dim, cc.stride_col = (int(x) for x in conv_state.stride())
    return cc


def kda_conv_compact(conv_state, cu_seqlens, state_indices, num_accepted, *, window: int,
                     error_word=None) -> None:
    """``kda_conv_compact``: move each committed row's conv window (starting
    at column n - 1) to column 0, in place.  conv_state: [S, conv_dim, width]
    view of 2- or 4-byte elements."""
    dev = conv_state.device
    i32 = torch.int32
    if conv_state.element_size() not in (2, 4):
        raise TypeError("conv_state elements must be 2 or 4 bytes")
    _req(cu_seqlens, i32, "cu_seqlens", dev)
    _req(state_indices, i32, "state_indices", dev)
    _req(num_accepted, i32, "num_accepted", dev)
    _opt(error_word, i32, "error_word", dev)
    for t in (cu_seqlens, state_indices, num_accepted):
        if not t.is_contiguous():
            raise ValueError("metadata tensors must be contiguous")
    B = state_indices.shape[0]
    if cu_seqlens.shape[0] != B + 1 or num_accepted.shape[0] < B:
        raise ValueError("metadata sizes do not match the batch")
    cc = make_conv_config(conv_state, window)
    lib = load_library()
    st = _on(dev.index, lib.kda_conv_compact, ctypes.byref(cc), _ptr(conv_state), _ptr(cu_seqlens),
             _ptr(state_indices), B, _ptr(num_accepted), _ptr(error_word), _stream_ptr(dev))
    _check("kda_conv_compact", st)


def make_align(block_table, num_computed, block_size: int, request_indices=None) -> KdaAlign:
    """``kda_align`` of an int32 block table [num_requests, width] (row stride
    free, columns contiguous) and int32 num_computed [num_requests]."""
    if block_table.dim() != 2 or block_table.stride(1) != 1:
        raise ValueError("block_table must be [num_requests, width] with contiguous columns")
    al = KdaAlign()
    al.block_table = block_table.data_ptr()
    al.block_table_stride = block_table.stride(0)
    al.block_table_width = block_table.shape[1]
    al.block_size = block_size
    al.num_requests = block_table.shape[0]
    al.reserved = 0
    al.num_computed = num_computed.data_ptr()
    al.request_indices = None if request_indices is None else request_indices.data_ptr()
    return al


def _check_align(block_table, num_computed, request_indices, dev):
    i32 = torch.int32
    _req(block_table, i32, "block_table", dev)
    _req(num_computed, i32, "num_computed", dev)
    _opt(request_indices, i32, "request_indices", dev)
    if num_computed.shape[0] < block_table.shape[0] or not num_computed.is_contiguous():
        raise ValueError("num_computed must be contiguous with one entry per request")
    if request_indices is not None and not request_indices.is_contiguous():
        raise ValueError("request_indices must be contiguous")


def kda_commit_align(A_log, g_bias, state_pool, cu_seqlens, state_indices, num_accepted, records,
                     block_table, num_computed, *, block_size: int, window: int,
                     record_slots: int, lower_bound=None, record_rows=None,
                     request_indices=None, pending=None, eager=None, error_word=None,
                     record_format: str = "raw") -> None:
    """``kda_commit_align``: the commit writing the final and boundary blocks
    of a paged state cache.  num_accepted, num_computed and the block table
    rows are per request; ``record_format`` as for ``kda_commit``.  With
    ``pending`` (and optionally ``eager``), the deferred form: rows that stay
    in their own slot and owe no boundary block only record their pending
    replay."""
    dev = state_pool.device
    f32, i32 = torch.float32, torch.int32
    for name, t in (("A_log", A_log), ("g_bias", g_bias), ("state_pool", state_pool)):
        _req(t, f32, name, dev)
    _req(records, torch.bfloat16, "records", dev)
    _req(cu_seqlens, i32, "cu_seqlens", dev)
    _req(state_indices, i32, "state_indices", dev)
    _req(num_accepted, i32, "num_accepted", dev)
    _opt(record_rows, i32, "record_rows", dev)
    _opt(pending, i32, "pending", dev)
    _opt(eager, torch.uint8, "eager", dev)
    _opt(error_word, i32, "error_word", dev)
    _check_align(block_table, num_computed, request_indices, dev)
    S, H, D = _check_pool(state_pool)
    _check_gate(A_log, g_bias, H, D)
    B = state_indices.shape[0]
    for t in (cu_seqlens, state_indices, num_accepted):
        if not t.is_contiguous():
            raise ValueError("metadata tensors must be contiguous")
    if cu_seqlens.shape[0] != B + 1 or num_accepted.shape[0] < block_table.shape[0]:
        raise ValueError("metadata sizes do not match the batch")
    _check_rows(B, record_slots, record_rows, pending, eager, error_word)
    if request_indices is not None:
        _at_least(request_indices, B, "request_indices")
    cfg = _config(H, window, S, record_slots, lower_bound, None, (1, 1, 1, 1, 1), D,
                  record_format)
    _check_records(records, H, window, record_slots, record_format)
    al = make_align(block_table, num_computed, block_size, request_indices)
    lib = load_library()
    st = _on(dev.index, lib.kda_commit_align, ctypes.byref(cfg), _ptr(A_log), _ptr(g_bias),
             _ptr(state_pool), _ptr(cu_seqlens), _ptr(state_indices), B, _ptr(num_accepted),
             _ptr(record_rows), _ptr(records), ctypes.byref(al), _ptr(pending), _ptr(eager),
             _ptr(error_word), _stream_ptr(dev))
    _check("kda_commit_align", st)


def kda_conv_compact_align(conv_state, cu_seqlens, state_indices, num_accepted, block_table,
                           num_computed, *, block_size: int, window: int,
                           request_indices=None, error_word=None) -> None:
    """``kda_conv_compact_align``: the conv windows of each committed row go
    to its final and boundary blocks."""
    dev = conv_state.device
    i32 = torch.int32
    if conv_state.element_size() not in (2, 4):
        raise TypeError("conv_state elements must be 2 or 4 bytes")
    _req(cu_seqlens, i32, "cu_seqlens", dev)
    _req(state_indices, i32, "state_indices", dev)
    _req(num_accepted, i32, "num_accepted", dev)
    _opt(error_word, i32, "error_word", dev)
    _check_align(block_table, num_computed, request_indices, dev)
    B = state_indices.shape[0]
    if cu_seqlens.shape[0] != B + 1 or num_accepted.shape[0] < block_table.shape[0]:
        raise ValueError("metadata sizes do not match the batch")
    cc = make_conv_config(conv_state, window)
    al = make_align(block_table, num_computed, block_size, request_indices)
    lib = load_library()
    st = _on(dev.index, lib.kda_conv_compact_align, ctypes.byref(cc), _ptr(conv_state),
             _ptr(cu_seqlens), _ptr(state_indices), B, _ptr(num_accepted), ctypes.byref(al),
             _ptr(error_word), _stream_ptr(dev))
    _check("kda_conv_compact_align", st)


def kda_record_state_blocks(idx_mapping, num_sampled, num_computed, state_column, num_accepted,
                            *, block_size: int, block_table_width: int, num_rows=None,
                            request_indices=None, error_word=None) -> None:
    """``kda_record_state_blocks``: after an align-mode commit, point each
    committed request's running state column at the block of its last
    committed token and reset its accepted count to 1.  idx_mapping,
    num_sampled and num_computed are int32 per request; state_column and
    num_accepted int32 per running slot.  ``num_rows`` spec rows (default:
    request_indices' length, else one per request)."""
    dev = state_column.device
    i32 = torch.int32
    for name, t in (("idx_mapping", idx_mapping), ("num_sampled", num_sampled),
                    ("num_computed", num_computed), ("state_column", state_column),
                    ("num_accepted", num_accepted)):
        _req(t, i32, name, dev)
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
    _opt(request_indices, i32, "request_indices", dev)
    _opt(error_word, i32, "error_word", dev)
    num_requests = idx_mapping.shape[0]
    if num_sampled.shape[0] < num_requests or num_computed.shape[0] < num_requests:
        raise ValueError("num_sampled and num_computed need one entry per request")
    if num_accepted.shape[0] != state_column.shape[0]:
        raise ValueError("state_column and num_accepted must have the same length")
    if num_rows is None:
        num_rows = num_requests if request_indices is None else request_indices.shape[0]
    if request_indices is not None:
        if not request_indices.is_contiguous():
            raise ValueError("request_indices must be contiguous")
        _at_least(request_indices, num_rows, "request_indices")
    elif num_rows > num_requests:
        raise ValueError("more spec rows than requests without request_indices")
    al = KdaAlign()
    al.block_table = None  # not read by this call
    al.block_table_stride = 0
    al.block_table_width = block_table_width
    al.block_size = block_size
    al.num_requests = num_requests
    al.reserved = 0
    al.num_computed = num_computed.data_ptr()
    al.request_indices = None if request_indices is None else request_indices.data_ptr()
    lib = load_library()
    st = _on(dev.index, lib.kda_record_state_blocks, ctypes.byref(al), _ptr(idx_mapping),
             _ptr(num_sampled), num_rows, _ptr(state_column), _ptr(num_accepted),
             state_column.shape[0], _ptr(error_word), _stream_ptr(dev))
    _check("kda_record_state_blocks", st)


# ------------------------------------- full-attention layers and acceptance --
#
# These calls are short (a decode step's append takes 3 us on the device).  So
# the compiled part of the binding, _quick, checks and marshals what is plainly
# right; where it finds something else (None), or was not built, the functions
# here do.  Their checks too are written out inline, one comparison per fact,
# with the message worked out only once something is wrong, and their arguments
# go to the library as the bytes of one structure.

_CACHE_FORMAT = "9if6qQqiiiiQQ"     # kda_cache_config, kda_align
_FORMATS = [struct.Struct(f) for f in ("=" + _CACHE_FORMAT + "8Q2i2Q",
                                       "=" + _CACHE_FORMAT + "4Q2i6Q", "=Qq4i8Q")]
_APPEND_ARGS, _ATTENTION_ARGS, _LOGPROBS_ARGS = (f.pack for f in _FORMATS)
_ARGUMENT_SIZES = tuple(f.size for f in _FORMATS)
_MORE_FORMATS = [struct.Struct(f) for f in ("=2Qif", "=6i2f5q2i13Q2iQ")]
_NORM_ARGS, _DELTA_ARGS = (f.pack for f in _MORE_FORMATS)   # the norm's: behind the append's
_MORE_ARGUMENT_SIZES = (_FORMATS[0].size + _MORE_FORMATS[0].size, _MORE_FORMATS[1].size)


def _failed(fn: str, status: int):
    raise KDAError(fn, status)


def _raw_stream(device: int):
    # the handle torch.cuda.current_stream(device).cuda_stream holds, without
    # building the stream object; -1 is a host tensor's device, whose addresses
    # no kernel may be given
    if device < 0:
        raise ValueError("the tensors must be on a GPU")
    return torch._C._cuda_getCurrentRawStream(device)


def _address(t):
    return 0 if t is None else t.data_ptr()


def _mismatch(device, **tensors):
    """Raises for the first of name=(tensor, dtype) that is not on the device
    or of its type (the callers found that one is not)."""
    for name, (t, dtype) in tensors.items():
        if t is not None:
            _req(t, dtype, name, device)


def _check_cache(key_cache, value_cache):
    """Shape and strides of a paged cache viewed as [num_blocks, block_size,
    kv_heads, head_dim].  The stride of a dimension of one element says nothing
    and may be anything; a head's channels stand for it."""
    shape, strides, others = key_cache.shape, key_cache.stride(), value_cache.stride()
    if len(shape) != 4 or strides[3] != 1:
        raise ValueError("the caches must be [num_blocks, block_size, kv_heads, head_dim] views "
                         "with contiguous channels")
    if 1 in shape:
        strides = tuple(shape[3] if n == 1 else s for n, s in zip(shape, strides))
        others = tuple(shape[3] if n == 1 else s for n, s in zip(value_cache.shape, others))
    if others != strides or value_cache.shape != shape:
        raise ValueError("key_cache and value_cache must have the same shape and strides")
    return shape, strides


def _heads_tokens(t, name, dim):
    """Token count, heads and token stride of a [T, heads, dim] activation
    with heads and channels packed."""
    shape, stride = t.shape, t.stride()
    if len(shape) != 3 or shape[2] != dim:
        raise ValueError(f"{name} must be [T, H, {dim}], got {tuple(shape)}")
    tokens, heads, _ = shape
    if stride[2] != 1 or (stride[1] != dim and heads > 1):
        raise ValueError(f"{name} needs contiguous [H, D] inside a token")
    return tokens, heads, stride[0] if tokens > 1 else heads * dim


def _plan(cu_seqlens, block_table, num_computed, request_indices, error_word):
    """Row count, and the table's requests, width and row stride, of a call on
    a paged key/value cache."""
    B = cu_seqlens.numel() - 1
    requests, width = block_table.shape
    stride, one = block_table.stride()
    if B < 0 or not cu_seqlens.is_contiguous():
        raise ValueError("cu_seqlens must be contiguous with B + 1 entries")
    if one != 1 and width > 1:
        raise ValueError("block_table must be [num_requests, width] with contiguous columns")
    if num_computed.numel() < requests or not num_computed.is_contiguous():
        raise ValueError("num_computed must be contiguous with one entry per request")
    if request_indices is not None:
        if not request_indices.is_contiguous():
            raise ValueError("request_indices must be contiguous")
        _at_least(request_indices, B, "request_indices")
    elif B > requests:
        raise ValueError("more rows than requests without request_indices")
    if error_word is not None:
        _at_least(error_word, 1, "error_word")
    return B, requests, width, stride if requests > 1 else width


def kda_kv_append(q, k, v, key_cache, value_cache, cu_seqlens, block_table, num_computed, *,
                  inv_freq=None, interleaved: bool = False, q_out=None, request_indices=None,
                  error_word=None):
    """``kda_kv_append``: rotate the new tokens' queries and keys by position
    and write keys and values to the paged cache.

    q: [T, Hq, D] or None; k, v: [T, Hkv, D] (token stride free, [H, D]
    packed), bf16 or fp16; key_cache, value_cache: [num_blocks, block_size,
    Hkv, D] views of the same strides; cu_seqlens int32 [B + 1]; block_table
    int32 [num_requests, width] (entries <= 0: nothing is stored);
    num_computed int32 [num_requests].  inv_freq: fp64 [rotary_dim / 2],
    radians per position (None: no rotation).  Returns the rotated queries
    (``q_out``, which may be ``q`` when it is contiguous; allocated when
    None), or None without ``q``.
    """
    lib = load_library()
    if _quick is not None:
        done = _quick.append(lib.append_address, q, k, v, key_cache, value_cache, cu_seqlens,
                             block_table, num_computed, inv_freq, interleaved, q_out,
                             request_indices, error_word)
        if done is not None:
            return done[0] if done.__class__ is tuple else _failed("kda_kv_append", done)
    dev, q_out, args = _append_arguments(q, k, v, key_cache, value_cache, cu_seqlens, block_table,
                                         num_computed, inv_freq, interleaved, q_out,
                                         request_indices, error_word)
    status = _on(dev, lib.kda_kv_append_packed, args)
    if status:
        raise KDAError("kda_kv_append", status)
    return q_out


def kda_kv_norm_append(q, k, v, key_cache, value_cache, cu_seqlens, block_table, num_computed, *,
                       q_weight=None, k_weight=None, eps: float = 1e-6, inv_freq=None,
                       interleaved: bool = False, q_out=None, request_indices=None,
                       error_word=None):
    """``kda_kv_norm_append``: ``kda_kv_append`` of a layer that norms each
    head's queries and keys before their rotation, ``y = x * weight /
    sqrt(mean(x * x) + eps)`` in fp32.

    q_weight, k_weight: [D] of the cache's type, or both fp32 (None: ones);
    all else as for ``kda_kv_append``.
    """
    lib = load_library()
    if _quick_more is not None:
        done = _quick_more.norm_append(lib.norm_append_address, q, k, v, key_cache, value_cache,
                                       cu_seqlens, block_table, num_computed, inv_freq,
                                       interleaved, q_out, request_indices, error_word, q_weight,
                                       k_weight, eps)
        if done is not None:
            return done[0] if done.__class__ is tuple else _failed("kda_kv_norm_append", done)
    dtype, dim = key_cache.dtype, key_cache.shape[-1]
    weight_dtype = next((w.dtype for w in (q_weight, k_weight) if w is not None), torch.float32)
    if weight_dtype not in (dtype, torch.float32):
        raise TypeError(f"the weights must be {dtype} or float32, got {weight_dtype}")
    for name, w in (("q_weight", q_weight), ("k_weight", k_weight)):
        if w is not None:
            _req(w, weight_dtype, name, key_cache.device)
            if tuple(w.shape) != (dim,) or not w.is_contiguous():
                raise ValueError(f"{name} must be contiguous with {dim} entries")
    dev, q_out, args = _append_arguments(q, k, v, key_cache, value_cache, cu_seqlens, block_table,
                                         num_computed, inv_freq, interleaved, q_out,
                                         request_indices, error_word)
    status = _on(dev, lib.kda_kv_norm_append_packed, args + _NORM_ARGS(
        _address(q_weight), _address(k_weight), DTYPES[weight_dtype], eps))
    if status:
        raise KDAError("kda_kv_norm_append", status)
    return q_out


def _append_arguments(q, k, v, key_cache, value_cache, cu_seqlens, block_table, num_computed,
                      inv_freq, interleaved, q_out, request_indices, error_word):
    """The device, the output and the argument structure of an append, checked."""
    dev, dtype, i32 = key_cache.get_device(), key_cache.dtype, torch.int32
    code = DTYPES.get(dtype, 2)
    if code > 1:
        raise TypeError(f"key_cache must be bfloat16 or float16, got {dtype}")
    if (value_cache.dtype is not dtype or k.dtype is not dtype or v.dtype is not dtype
            or cu_seqlens.dtype is not i32 or block_table.dtype is not i32
            or num_computed.dtype is not i32 or value_cache.get_device() != dev
            or k.get_device() != dev or v.get_device() != dev or cu_seqlens.get_device() != dev
            or block_table.get_device() != dev or num_computed.get_device() != dev):
        _mismatch(key_cache.device, value_cache=(value_cache, dtype), k=(k, dtype), v=(v, dtype),
                  cu_seqlens=(cu_seqlens, i32), block_table=(block_table, i32),
                  num_computed=(num_computed, i32))
    if request_indices is not None or error_word is not None:
        _mismatch(key_cache.device, request_indices=(request_indices, i32),
                  error_word=(error_word, i32))
    (blocks, block_size, kv_heads, dim), strides = _check_cache(key_cache, value_cache)
    B, requests, width, table_stride = _plan(cu_seqlens, block_table, num_computed,
                                             request_indices, error_word)
    T, heads, stride_k = _heads_tokens(k, "k", dim)
    Tv, heads_v, stride_v = _heads_tokens(v, "v", dim)
    if heads != kv_heads or heads_v != kv_heads or Tv != T:
        raise ValueError(f"k and v must be [T, {kv_heads}, {dim}] with the same T")
    q_heads, stride_q, q_ptr, out_ptr = kv_heads, 8, 0, 0
    if q is not None:
        if q.dtype is not dtype or q.get_device() != dev:
            _mismatch(key_cache.device, q=(q, dtype))
        Tq, q_heads, stride_q = _heads_tokens(q, "q", dim)
        if Tq != T or q_heads < 1 or q_heads % kv_heads:
            raise ValueError("q must be [T, Hq, D] with k's T and Hq a multiple of the cache's "
                             "heads")
        if q_out is None:
            q_out = torch.empty_like(q, memory_format=torch.contiguous_format)
        else:
            _req(q_out, dtype, "q_out", key_cache.device)
            if q_out.shape != q.shape or not q_out.is_contiguous():
                raise ValueError("q_out must be contiguous and shaped like q")
        q_ptr, out_ptr = q.data_ptr(), q_out.data_ptr()
    elif q_out is not None:
        raise ValueError("q_out without q")
    rotary_dim = freq_ptr = 0
    if inv_freq is not None:
        if inv_freq.dtype is not torch.float64 or inv_freq.get_device() != dev:
            _mismatch(key_cache.device, inv_freq=(inv_freq, torch.float64))
        if inv_freq.dim() != 1 or not inv_freq.is_contiguous():
            raise ValueError("inv_freq must be contiguous with rotary_dim / 2 entries")
        rotary_dim, freq_ptr = 2 * inv_freq.numel(), inv_freq.data_ptr()
    return dev, q_out, _APPEND_ARGS(
        q_heads, kv_heads, dim, code, blocks, 1, 0, rotary_dim, 1 if interleaved else 0, 1.0,
        strides[0], strides[1], strides[2], stride_q, stride_k, stride_v, block_table.data_ptr(),
        table_stride, width, block_size, requests, 0, num_computed.data_ptr(),
        _address(request_indices), q_ptr, k.data_ptr(), v.data_ptr(), out_ptr,
        key_cache.data_ptr(), value_cache.data_ptr(), freq_ptr, cu_seqlens.data_ptr(), B, T,
        _address(error_word), _raw_stream(dev))


@functools.lru_cache(maxsize=256)
def kda_attention_workspace_bytes(num_rows: int, q_heads: int, kv_heads: int, head_dim: int,
                                  window: int = MAX_WINDOW) -> int:
    """Size in bytes of the workspace of ``kda_window_attention``
    (``kda_attention_workspace_bytes``); 0 for sizes it does not support."""
    cfg = KdaCacheConfig(q_heads, kv_heads, head_dim, 0, 1, window, 0, 0, 0, 1.0, 8, 8, 8, 8, 8, 8)
    return int(load_library().kda_attention_workspace_bytes(ctypes.byref(cfg), num_rows))


def _largest_window(q_heads: int, kv_heads: int) -> int:
    group = q_heads // max(kv_heads, 1)
    return min(MAX_WINDOW, max(1, MAX_QUERY_ROWS // max(group, 1)))


def allocate_attention_workspace(num_rows: int, q_heads: int, kv_heads: int, head_dim: int, device,
                                 window: int | None = None) -> torch.Tensor:
    """A workspace for ``kda_window_attention`` calls of up to ``num_rows``
    rows and ``window`` tokens each (None: the largest window the head counts
    allow).  It holds nothing between calls; calls that may overlap need one
    each."""
    if window is None:
        window = _largest_window(q_heads, kv_heads)
    nbytes = kda_attention_workspace_bytes(num_rows, q_heads, kv_heads, head_dim, window)
    if nbytes == 0:
        raise ValueError("invalid attention sizes")
    return torch.empty(nbytes, dtype=torch.uint8, device=device)


def kda_window_attention(q, key_cache, value_cache, cu_seqlens, block_table, num_computed,
                         workspace, *, window: int | None = None, scale=None, left_window: int = 0,
                         request_indices=None, out=None, lse=None, error_word=None):
    """``kda_window_attention``: softmax attention of each row's new tokens
    (at most ``window``; None: the largest window the head counts allow) over
    its paged keys and values, the new ones included (``kda_kv_append`` first).

    q: [T, Hq, D] (token stride free), bf16 or fp16; caches, block_table and
    num_computed as for ``kda_kv_append``; ``left_window``: keys a query sees,
    itself included (0: all); ``scale``: D ** -0.5 when None; workspace from
    ``allocate_attention_workspace``.  Returns ``(out, lse)``: out [T, Hq, D]
    and the scores' log sum of exponentials, fp32 [T, Hq].  Rows that are
    skipped leave theirs untouched."""
    lib = load_library()
    if _quick is not None:
        done = _quick.attend(lib.attend_address, q, key_cache, value_cache, cu_seqlens,
                             block_table, num_computed, workspace, window, scale, left_window,
                             request_indices, out, lse, error_word)
        if done is not None:
            return done if done.__class__ is tuple else _failed("kda_window_attention", done)
    dev, dtype, i32 = key_cache.get_device(), key_cache.dtype, torch.int32
    code = DTYPES.get(dtype, 2)
    if code > 1:
        raise TypeError(f"key_cache must be bfloat16 or float16, got {dtype}")
    if (value_cache.dtype is not dtype or q.dtype is not dtype
            or workspace.dtype is not torch.uint8 or cu_seqlens.dtype is not i32
            or block_table.dtype is not i32 or num_computed.dtype is not i32
            or value_cache.get_device() != dev or q.get_device() != dev
            or workspace.get_device() != dev or cu_seqlens.get_device() != dev
            or block_table.get_device() != dev or num_computed.get_device() != dev):
        _mismatch(key_cache.device, value_cache=(value_cache, dtype), q=(q, dtype),
                  workspace=(workspace, torch.uint8), cu_seqlens=(cu_seqlens, i32),
                  block_table=(block_table, i32), num_computed=(num_computed, i32))
    if request_indices is not None or error_word is not None:
        _mismatch(key_cache.device, request_indices=(request_indices, i32),
                  error_word=(error_word, i32))
    (blocks, block_size, kv_heads, dim), strides = _check_cache(key_cache, value_cache)
    B, requests, width, table_stride = _plan(cu_seqlens, block_table, num_computed,
                                             request_indices, error_word)
    T, q_heads, stride_q = _heads_tokens(q, "q", dim)
    if q_heads < 1 or q_heads % kv_heads:
        raise ValueError("q must be [T, Hq, D] with Hq a multiple of the cache's heads")
    if window is None:
        window = _largest_window(q_heads, kv_heads)
    if out is None:
        out = torch.empty_like(q, memory_format=torch.contiguous_format)
    else:
        _req(out, dtype, "out", key_cache.device)
        if out.shape != q.shape or not out.is_contiguous():
            raise ValueError("out must be contiguous and shaped like q")
    if lse is None:
        lse = torch.empty((T, q_heads), dtype=torch.float32, device=q.device)
    else:
        _req(lse, torch.float32, "lse", key_cache.device)
        if tuple(lse.shape) != (T, q_heads) or not lse.is_contiguous():
            raise ValueError("lse must be a contiguous [T, Hq] tensor")
    if not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    if T == 0:  # an empty tensor has no address to pass on
        return out, lse
    status = _on(dev, lib.kda_window_attention_packed, _ATTENTION_ARGS(
        q_heads, kv_heads, dim, code, blocks, window, left_window, 0, 0,
        dim ** -0.5 if scale is None else scale, strides[0], strides[1], strides[2], stride_q, 8,
        8, block_table.data_ptr(), table_stride, width, block_size, requests, 0,
        num_computed.data_ptr(), _address(request_indices), q.data_ptr(), key_cache.data_ptr(),
        value_cache.data_ptr(), cu_seqlens.data_ptr(), B, T, workspace.data_ptr(),
        workspace.numel(),
        out.data_ptr(), lse.data_ptr(), _address(error_word), _raw_stream(dev)))
    if status:
        raise KDAError("kda_window_attention", status)
    return out, lse


class TokenLogprobs(NamedTuple):
    """Outputs of ``kda_token_logprobs``: fp32 [rows] each, the alternatives
    fp32 and int32 [rows, num_top].  Those that a call allocates may lie in one
    allocation."""

    logprob: torch.Tensor
    entropy: torch.Tensor
    lse: torch.Tensor
    top_logprob: torch.Tensor
    top_index: torch.Tensor


def allocate_token_logprobs(rows: int, num_top: int, device) -> TokenLogprobs:
    """Output buffers of ``kda_token_logprobs``."""
    def one(*shape, dtype=torch.float32):
        return torch.empty(shape, dtype=dtype, device=device)
    return TokenLogprobs(one(rows), one(rows), one(rows), one(rows, num_top),
                         one(rows, num_top, dtype=torch.int32))


def kda_token_logprobs(logits, tokens, *, num_top: int = 0, out: TokenLogprobs | None = None,
                       error_word=None) -> TokenLogprobs:
    """``kda_token_logprobs``: log probability of ``tokens`` (int32 [rows];
    negative: none, 0), entropy, log sum of exponentials and the ``num_top``
    largest logits (ties: the lower index) of each row of ``logits`` [rows,
    vocab], bf16, fp16 or fp32 with any row stride."""
    lib = load_library()
    if _quick is not None and out is None:
        done = _quick.logprobs(lib.logprobs_address, logits, tokens, num_top, error_word)
        if done is not None:
            return (TokenLogprobs._make(done) if done.__class__ is tuple
                    else _failed("kda_token_logprobs", done))
    dev, i32, f32 = logits.get_device(), torch.int32, torch.float32
    code = DTYPES.get(logits.dtype)
    if code is None:
        raise TypeError(f"logits must be bfloat16, float16 or float32, got {logits.dtype}")
    if tokens.dtype is not i32 or tokens.get_device() != dev:
        _mismatch(logits.device, tokens=(tokens, i32))
    if error_word is not None:
        _req(error_word, i32, "error_word", logits.device)
        _at_least(error_word, 1, "error_word")
    shape, strides = logits.shape, logits.stride()
    if len(shape) != 2:
        raise ValueError("logits must be [rows, vocab]")
    rows, vocab = shape
    if strides[1] != 1 and vocab > 1:
        raise ValueError("logits must have contiguous columns")
    if tokens.dim() != 1 or tokens.numel() != rows or not tokens.is_contiguous():
        raise ValueError("tokens must be contiguous with one entry per row")
    if out is None:
        out = TokenLogprobs(torch.empty_like(tokens, dtype=f32),
                            torch.empty_like(tokens, dtype=f32),
                            torch.empty_like(tokens, dtype=f32),
                            torch.empty((rows, num_top), dtype=f32, device=tokens.device),
                            torch.empty((rows, num_top), dtype=i32, device=tokens.device))
    else:
        for name, t in zip(TokenLogprobs._fields, out):
            _req(t, i32 if name == "top_index" else f32, name, logits.device)
            want = (rows, num_top) if name.startswith("top_") else (rows,)
            if tuple(t.shape) != want or not t.is_contiguous():
                raise ValueError(f"{name} must be a contiguous {want} tensor")
    logprob, entropy, lse, top_logprob, top_index = out
    status = _on(dev, lib.kda_token_logprobs_packed, _LOGPROBS_ARGS(
        logits.data_ptr(), strides[0], code, rows, vocab, num_top, tokens.data_ptr(),
        logprob.data_ptr(), entropy.data_ptr(), lse.data_ptr(), top_logprob.data_ptr(),
        top_index.data_ptr(), _address(error_word), _raw_stream(dev)))
    if status:
        raise KDAError("kda_token_logprobs", status)
    return out


# ------------------------------------------ prompts and plain decoding of KDA --

def _delta_call(name, lib, q, k, v, g_raw, beta_raw, A_log, g_bias, state_pool, cu_seqlens,
                state_indices, lower_bound, scale, initial_indices, out, error_word):
    address = lib.prefill_address if cu_seqlens is not None else lib.decode_address
    if _quick_more is not None:
        done = _quick_more.delta(address, q, k, v, g_raw, beta_raw, A_log, g_bias, state_pool,
                                 cu_seqlens, state_indices, lower_bound, scale, initial_indices,
                                 out, error_word)
        if done is not None:
            return done[0] if done.__class__ is tuple else _failed(name, done)
    dev, bf, f32, i32 = state_pool.device, torch.bfloat16, torch.float32, torch.int32
    for label, t in (("q", q), ("k", k), ("v", v), ("g_raw", g_raw), ("beta_raw", beta_raw)):
        _req(t, bf, label, dev)
    for label, t in (("A_log", A_log), ("g_bias", g_bias), ("state_pool", state_pool)):
        _req(t, f32, label, dev)
    _req(state_indices, i32, "state_indices", dev)
    _opt(cu_seqlens, i32, "cu_seqlens", dev)
    _opt(initial_indices, i32, "initial_indices", dev)
    _opt(out, bf, "out", dev)
    _opt(error_word, i32, "error_word", dev)
    S, H, D = _check_pool(state_pool)
    _check_gate(A_log, g_bias, H, D)
    if state_indices.dim() != 1 or not state_indices.is_contiguous():
        raise ValueError("state_indices must be contiguous with one entry per row")
    B = state_indices.shape[0]
    if initial_indices is not None and (tuple(initial_indices.shape) != (B,)
                                        or not initial_indices.is_contiguous()):
        raise ValueError("initial_indices must be contiguous with one entry per row")
    if cu_seqlens is not None and (tuple(cu_seqlens.shape) != (B + 1,)
                                   or not cu_seqlens.is_contiguous()):
        raise ValueError("cu_seqlens must be contiguous with B + 1 entries")
    T, heads, _ = _heads_tokens(q, "q", D)
    if heads != H:
        raise ValueError(f"q must be [T, {H}, {D}], got {tuple(q.shape)}")
    strides = []
    for label, t in (("q", q), ("k", k), ("v", v), ("g_raw", g_raw)):
        tokens, heads, stride = _heads_tokens(t, label, D)
        if tokens != T or heads != H:
            raise ValueError(f"{label} must be shaped like q, got {tuple(t.shape)}")
        strides.append(stride)
    if tuple(beta_raw.shape) != (T, H) or (beta_raw.stride(1) != 1 and H > 1):
        raise ValueError("beta_raw must be [T, H] with contiguous heads inside a token")
    strides.append(beta_raw.stride(0) if T > 1 else H)
    if cu_seqlens is None and T != B:
        raise ValueError("q must have one token per row")
    if out is None:
        out = torch.empty_like(q, memory_format=torch.contiguous_format)
    elif out.shape != q.shape or not out.is_contiguous():
        raise ValueError("out must be contiguous and shaped like q")
    _at_least(error_word, 1, "error_word")
    if T == 0 or B == 0:  # an empty tensor has no address to pass on
        return out
    fn = lib.kda_prefill_packed if cu_seqlens is not None else lib.kda_decode_packed
    status = _on(dev.index, fn, _DELTA_ARGS(
        H, D, 1, S, 0, 0 if lower_bound is None else 1,
        0.0 if lower_bound is None else lower_bound, D ** -0.5 if scale is None else scale,
        *strides, 0, 0, q.data_ptr(), k.data_ptr(), v.data_ptr(), g_raw.data_ptr(),
        beta_raw.data_ptr(), A_log.data_ptr(), g_bias.data_ptr(), state_pool.data_ptr(),
        state_indices.data_ptr(), _address(initial_indices), out.data_ptr(), _address(error_word),
        _raw_stream(state_pool.get_device()), B, T, _address(cu_seqlens)))
    if status:
        raise KDAError(name, status)
    return out


def kda_prefill(q, k, v, g_raw, beta_raw, A_log, g_bias, state_pool, cu_seqlens, state_indices, *,
                lower_bound=None, scale=None, initial_indices=None, out=None, error_word=None):
    """``kda_prefill``: the gated delta rule over rows of any length, prompts
    or pieces of them, with ``kda_verify``'s norms, gates and recurrence.

    q, k, v, g_raw: bf16 [T, H, 128] (token stride free, [H, D] packed);
    beta_raw: bf16 [T, H]; A_log fp32 [H]; g_bias fp32 [H * 128]; state_pool
    fp32 [S, H, 128, 128]; cu_seqlens int32 [B + 1]; state_indices int32 [B]:
    the slot that takes the state behind the row's last token (<= 0: the row
    is skipped); initial_indices int32 [B]: the slot that the row starts from
    (<= 0: zeros; None: state_indices).  No row may write a slot that another
    reads or writes.  Returns ``out``, bf16 [T, H, 128], which overlaps no input;
    rows that are skipped leave theirs untouched, and rows without tokens write
    no state.

    Tokens are taken 16 at a time: what the decays take away within them is told
    from what stays to 2^-23 of a row of the state and to 2^-40 between tokens
    (include/kda.h has the limits, and where NaN and infinities go)."""
    if cu_seqlens is None:
        raise ValueError("cu_seqlens is required")
    return _delta_call("kda_prefill", load_library(), q, k, v, g_raw, beta_raw, A_log, g_bias,
                       state_pool, cu_seqlens, state_indices, lower_bound, scale, initial_indices,
                       out, error_word)


def kda_decode(q, k, v, g_raw, beta_raw, A_log, g_bias, state_pool, state_indices, *,
               lower_bound=None, scale=None, initial_indices=None, out=None, error_word=None):
    """``kda_decode``: one token of each row through the gated delta rule, the
    state read and written once.  q, k, v, g_raw: bf16 [B, H, 128]; all else as
    for ``kda_prefill``."""
    return _delta_call("kda_decode", load_library(), q, k, v, g_raw, beta_raw, A_log, g_bias,
                       state_pool, None, state_indices, lower_bound, scale, initial_indices, out,
                       error_word)
