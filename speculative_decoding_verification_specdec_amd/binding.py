"""ctypes binding of ``libspecdec.so`` (the C ABI in ``include/specdec.h``).

Argument marshalling only: torch device tensors are checked for device, dtype, contiguity and
shape, turned into raw pointers and handed to the library together with the current HIP
stream.  Every step of the verify computation runs in the library's HIP kernels; there is no
CPU or PyTorch fallback, and a missing library raises ``SpecdecError``.
"""
from __future__ import annotations

import contextlib
import ctypes
import os
import pathlib

import numpy as np
import torch

_LIB = None

SPECDEC_F32 = 0
SPECDEC_BF16 = 1
SPECDEC_F16 = 2
SPECDEC_MAX_K = 63


class SpecdecError(RuntimeError):
    pass


class _Options(ctypes.Structure):
    _fields_ = [("hot_event_begin", ctypes.c_void_p), ("hot_event_end", ctypes.c_void_p),
                ("path", ctypes.c_int32), ("spin_limit", ctypes.c_int32),
                ("draw_event_begin", ctypes.c_void_p), ("draw_event_end", ctypes.c_void_p)]


class _KvCache(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("dtype", ctypes.c_int32),
                ("num_pages", ctypes.c_int32), ("page_size", ctypes.c_int32),
                ("num_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("max_pages", ctypes.c_int32), ("page_stride", ctypes.c_int64),
                ("slot_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64),
                ("page_table", ctypes.c_void_p), ("weight", ctypes.c_void_p),
                ("position", ctypes.c_void_p)]


class _Rope(ctypes.Structure):
    _fields_ = [("inv_freq", ctypes.c_void_p), ("rotary_dim", ctypes.c_int32),
                ("interleaved", ctypes.c_int32), ("scale", ctypes.c_float)]


# Execution paths of specdec_verify (include/specdec.h).
SPECDEC_SMALL_V_MAX = 1024
SPECDEC_PATH_AUTO, SPECDEC_PATH_STREAMING, SPECDEC_PATH_SMALL_VOCAB = 0, 1, 2
SPECDEC_PATH_ONE_LAUNCH = 3
SPECDEC_PATH_QUAD = 4


def _event_pair(events):
    return (None, None) if events is None else tuple(
        e if isinstance(e, int) or e is None else e.cuda_event for e in events)


def _options(hot_events, path, spin_limit=0, draw_events=None):
    ev, dv = _event_pair(hot_events), _event_pair(draw_events)
    return _Options(ev[0], ev[1], int(path), int(spin_limit), dv[0], dv[1])


def library_path() -> pathlib.Path:
    env = os.environ.get("SPECDEC_LIBRARY")
    return pathlib.Path(env) if env else pathlib.Path(__file__).with_name("libspecdec.so")


def load_library():
    """Load the HIP library once; raise SpecdecError if it is not built."""
    global _LIB
    if _LIB is not None:
        return _LIB
    path = library_path()
    if not path.exists():
        raise SpecdecError(f"{path} is missing: build it with `python -c 'import __graft_entry__ as g; "
                           f"g.build()'` (hipcc, gfx950). There is no fallback path.")
    lib = ctypes.CDLL(str(path))
    vp, i32, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_size_t
    common = [vp, i32, vp, vp, vp, vp, vp, vp, i32, i32, i32, vp, vp, vp, vp, sz, vp]
    lib.specdec_verify.argtypes = common
    lib.specdec_verify.restype = i32
    lib.specdec_verify_ex.argtypes = common + [ctypes.POINTER(_Options)]
    lib.specdec_verify_ex.restype = i32
    lib.specdec_verify_greedy.argtypes = [vp, i32, vp, vp, i32, i32, i32, vp, vp, vp, vp, sz, vp]
    lib.specdec_verify_greedy.restype = i32
    lib.specdec_verify_match.argtypes = [vp, i32, vp, vp, vp, vp, i32, i32, i32, vp, vp, vp, vp,
                                         sz, vp]
    lib.specdec_verify_match.restype = i32
    lib.specdec_verify_noalloc.argtypes = [vp, i32, vp, vp, vp, vp, vp, vp, i32, i32, i32, vp, vp,
                                           vp, vp]
    lib.specdec_verify_noalloc.restype = i32
    lib.specdec_noalloc_scratch_bytes.argtypes = []
    lib.specdec_noalloc_scratch_bytes.restype = sz
    lib.specdec_workspace_size.argtypes = [i32, i32, i32]
    lib.specdec_workspace_size.restype = sz
    lib.specdec_ngram_workspace_size.argtypes = [i32, i32]
    lib.specdec_ngram_workspace_size.restype = sz
    lib.specdec_ngram_propose.argtypes = [vp, vp, i32, i32, i32, i32, i32, vp, vp, vp, sz, vp]
    lib.specdec_ngram_propose.restype = i32
    lib.specdec_commit.argtypes = [vp, vp, i32, i32, vp, i32, vp, vp, vp, vp, vp, vp]
    lib.specdec_commit.restype = i32
    lib.specdec_telemetry_update.argtypes = [vp, vp, vp, i32, i32, i32, vp, vp]
    lib.specdec_telemetry_update.restype = i32
    lib.specdec_apply_k.argtypes = [vp, vp, vp, i32, i32, vp]
    lib.specdec_apply_k.restype = i32
    f64 = ctypes.c_double
    lib.specdec_alpha_estimate.argtypes = [vp]
    lib.specdec_alpha_estimate.restype = f64
    lib.specdec_expected_tokens.argtypes = [f64, i32]
    lib.specdec_expected_tokens.restype = f64
    lib.specdec_speedup.argtypes = [f64, i32, f64]
    lib.specdec_speedup.restype = f64
    lib.specdec_choose_k.argtypes = [f64, f64, i32, i32]
    lib.specdec_choose_k.restype = i32
    lib.specdec_plan_k.argtypes = [vp, i32, f64, i32, i32, i32, vp]
    lib.specdec_plan_k.restype = i32
    i64, f32 = ctypes.c_int64, ctypes.c_float
    lib.specdec_rope_frequencies.argtypes = [i32, f64, i32, f64, f64, f64, f64, vp]
    lib.specdec_rope_frequencies.restype = i32
    lib.specdec_rope_append.argtypes = [vp, vp, vp, i64, i64, i64, i32, i32, i32, vp, vp, vp, vp,
                                        vp, vp, vp]
    lib.specdec_rope_append.restype = i32
    lib.specdec_paged_attention_workspace_size.argtypes = [i32, i32, i32, i32, i32]
    lib.specdec_paged_attention_workspace_size.restype = sz
    lib.specdec_paged_attention.argtypes = [vp, i64, i32, i32, i32, vp, vp, f32, vp, vp, vp, vp, sz,
                                            vp]
    lib.specdec_paged_attention.restype = i32
    lib.specdec_kv_weights.argtypes = [vp, i64, vp, i32, i32, i32, vp, vp, vp, f32, vp, vp]
    lib.specdec_kv_weights.restype = i32
    lib.specdec_kv_evict_workspace_size.argtypes = [i32, vp, i32]
    lib.specdec_kv_evict_workspace_size.restype = sz
    lib.specdec_kv_evict.argtypes = [vp, vp, i32, i32, i32, i32, vp, vp, sz, vp]
    lib.specdec_kv_evict.restype = i32
    lib.specdec_status_string.argtypes = [i32]
    lib.specdec_status_string.restype = ctypes.c_char_p
    lib.specdec_version.argtypes = []
    lib.specdec_version.restype = i32
    _LIB = lib
    return lib


def specdec_status_string(status: int) -> str:
    return load_library().specdec_status_string(int(status)).decode()


def specdec_workspace_size(B: int, K: int, V: int) -> int:
    return int(load_library().specdec_workspace_size(int(B), int(K), int(V)))


def _ptr(t: torch.Tensor | None) -> int | None:
    return None if t is None else t.data_ptr()


def _check(t: torch.Tensor | None, name: str, dtype, shape, device, optional=False):
    if t is None:
        if optional:
            return
        raise SpecdecError(f"{name} is required")
    if t.device != device:
        raise SpecdecError(f"{name} is on {t.device}, expected {device}")
    if t.dtype != dtype:
        raise SpecdecError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if t.shape != shape and tuple(t.shape) != tuple(shape):
        raise SpecdecError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if not t.is_contiguous():
        raise SpecdecError(f"{name} must be contiguous")


def _stream_handle(stream) -> int:
    if stream is None:
        stream = torch.cuda.current_stream()
    return int(stream.cuda_stream)


def _on(stream):
    """Allocation context for buffers a call creates itself: they belong to the stream the call
    is enqueued on, so torch's caching allocator does not hand them to other work on its current
    stream while the library's kernels still use them."""
    return torch.cuda.stream(stream) if stream is not None else contextlib.nullcontext()


def _outputs(B, K, device, out, want_probs, stream=None):
    if out is not None:
        return out
    with _on(stream):
        acc = torch.empty(B, dtype=torch.int32, device=device)
        tok = torch.empty((B, K + 1), dtype=torch.int32, device=device)
        prb = (torch.empty((B, K + 1), dtype=torch.float32, device=device) if want_probs
               else None)
    return acc, tok, prb


def new_workspace(B: int, K: int, V: int, device, stream=None) -> torch.Tensor:
    """A verify workspace for these sizes (uninitialised: the library needs none), allocated
    for ``stream``."""
    need = specdec_workspace_size(B, K, V)
    with _on(stream):
        return torch.empty(max(need, 16), dtype=torch.uint8, device=device)


def _workspace(B, K, V, device, workspace, stream=None):
    need = specdec_workspace_size(B, K, V)
    if workspace is None:
        workspace = new_workspace(B, K, V, device, stream)
    return workspace, need


def _raise(status: int, fn: str):
    if status != 0:
        raise SpecdecError(f"{fn}: {specdec_status_string(status)} (status {status})")


def specdec_verify(target_logits: torch.Tensor, draft_probs: torch.Tensor | None,
                   proposed: torch.Tensor | None, temperature: torch.Tensor,
                   uniforms: torch.Tensor, *, draft_onehot: torch.Tensor | None = None,
                   num_draft: torch.Tensor | None = None, out=None, workspace=None,
                   want_probs: bool = True, stream=None, hot_events=None,
                   path: int = SPECDEC_PATH_AUTO, spin_limit: int = 0, draw_events=None):
    """Batched verify.  Shapes: target_logits [B, K+1, V] (bf16 or fp32), draft_probs
    [B, K, V] fp32 or None, proposed [B, K] int32, temperature [B] fp32, uniforms [B, K+1]
    fp32, draft_onehot [B] uint8 or None, num_draft [B] int32 or None.  Returns
    (accept_len [B] int32, out_tokens [B, K+1] int32, out_probs [B, K+1] fp32 or None),
    enqueued on ``stream`` (default: torch's current stream) without synchronising.
    ``hot_events``: optional (begin, end) pair of hipEvent_t handles (ints) recorded around the
    kernel that reads every target row; ``draw_events`` the same around the kernels after it
    (streaming path only).  ``path``: SPECDEC_PATH_AUTO (the one-kernel small-vocabulary
    path when V <= SPECDEC_SMALL_V_MAX, else the streaming kernels), _STREAMING, _SMALL_VOCAB
    or _ONE_LAUNCH.
    ``workspace``: a uint8 tensor of at least specdec_workspace_size(B, K, V) bytes
    (``new_workspace``), reusable across calls; None allocates one for this call.
    ``spin_limit``: SPECDEC_PATH_ONE_LAUNCH only, polls of a bounded wait (0 = the default)."""
    lib = load_library()
    if target_logits.dim() != 3:
        raise SpecdecError("target_logits must be [B, K+1, V]")
    B, K1, V = (int(s) for s in target_logits.shape)
    K = K1 - 1
    dev = target_logits.device
    if target_logits.dtype == torch.bfloat16:
        dt = SPECDEC_BF16
    elif target_logits.dtype == torch.float32:
        dt = SPECDEC_F32
    else:
        raise SpecdecError(f"target_logits dtype {target_logits.dtype} is not bf16/fp32")
    if not target_logits.is_contiguous():
        raise SpecdecError("target_logits must be contiguous")
    _check(draft_probs, "draft_probs", torch.float32, (B, K, V), dev, optional=True)
    _check(proposed, "proposed", torch.int32, (B, K), dev, optional=(K == 0))
    _check(temperature, "temperature", torch.float32, (B,), dev)
    _check(uniforms, "uniforms", torch.float32, (B, K + 1), dev)
    _check(draft_onehot, "draft_onehot", torch.uint8, (B,), dev, optional=True)
    _check(num_draft, "num_draft", torch.int32, (B,), dev, optional=True)
    acc, tok, prb = _outputs(B, K, dev, out, want_probs, stream)
    ws, need = _workspace(B, K, V, dev, workspace, stream)
    args = (_ptr(target_logits), dt, _ptr(draft_probs), _ptr(draft_onehot), _ptr(proposed),
            _ptr(num_draft), _ptr(temperature), _ptr(uniforms), B, K, V, _ptr(acc), _ptr(tok),
            _ptr(prb), _ptr(ws), ws.numel(), _stream_handle(stream))
    if (hot_events is None and draw_events is None and path == SPECDEC_PATH_AUTO
            and spin_limit == 0):
        status = lib.specdec_verify(*args)
    else:
        opts = _options(hot_events, path, spin_limit, draw_events)
        status = lib.specdec_verify_ex(*args, ctypes.byref(opts))
    _raise(status, "specdec_verify")
    return acc, tok, prb


def specdec_verify_noalloc(target_logits: torch.Tensor, draft_probs: torch.Tensor | None,
                           proposed: torch.Tensor | None, temperature: torch.Tensor,
                           uniforms: torch.Tensor, *, draft_onehot: torch.Tensor | None = None,
                           num_draft: torch.Tensor | None = None, out, stream=None):
    """specdec_verify through the entry point that allocates nothing: its workspace is the
    library's built-in device scratch (``out`` = (accept_len, out_tokens, out_probs or None) is
    required, so that this call creates no tensor either).  Shapes as for specdec_verify."""
    lib = load_library()
    if target_logits.dim() != 3:
        raise SpecdecError("target_logits must be [B, K+1, V]")
    B, K1, V = (int(s) for s in target_logits.shape)
    K = K1 - 1
    dev = target_logits.device
    if target_logits.dtype == torch.bfloat16:
        dt = SPECDEC_BF16
    elif target_logits.dtype == torch.float32:
        dt = SPECDEC_F32
    else:
        raise SpecdecError(f"target_logits dtype {target_logits.dtype} is not bf16/fp32")
    if not target_logits.is_contiguous():
        raise SpecdecError("target_logits must be contiguous")
    _check(draft_probs, "draft_probs", torch.float32, (B, K, V), dev, optional=True)
    _check(proposed, "proposed", torch.int32, (B, K), dev, optional=(K == 0))
    _check(temperature, "temperature", torch.float32, (B,), dev)
    _check(uniforms, "uniforms", torch.float32, (B, K + 1), dev)
    _check(draft_onehot, "draft_onehot", torch.uint8, (B,), dev, optional=True)
    _check(num_draft, "num_draft", torch.int32, (B,), dev, optional=True)
    acc, tok, prb = out
    _check(acc, "accept_len", torch.int32, (B,), dev)
    _check(tok, "out_tokens", torch.int32, (B, K + 1), dev)
    _check(prb, "out_probs", torch.float32, (B, K + 1), dev, optional=True)
    status = lib.specdec_verify_noalloc(_ptr(target_logits), dt, _ptr(draft_probs),
                                        _ptr(draft_onehot), _ptr(proposed), _ptr(num_draft),
                                        _ptr(temperature), _ptr(uniforms), B, K, V, _ptr(acc),
                                        _ptr(tok), _ptr(prb), _stream_handle(stream))
    _raise(status, "specdec_verify_noalloc")
    return acc, tok, prb


def specdec_verify_greedy(target_logits: torch.Tensor, proposed: torch.Tensor | None, *,
                          num_draft: torch.Tensor | None = None, out=None, workspace=None,
                          want_probs: bool = True, stream=None):
    """Greedy-only verify (every row at temperature 0).  Returns (accept_len, out_tokens,
    out_probs or None)."""
    lib = load_library()
    if target_logits.dim() != 3:
        raise SpecdecError("target_logits must be [B, K+1, V]")
    B, K1, V = (int(s) for s in target_logits.shape)
    K = K1 - 1
    dev = target_logits.device
    if target_logits.dtype == torch.bfloat16:
        dt = SPECDEC_BF16
    elif target_logits.dtype == torch.float32:
        dt = SPECDEC_F32
    else:
        raise SpecdecError(f"target_logits dtype {target_logits.dtype} is not bf16/fp32")
    if not target_logits.is_contiguous():
        raise SpecdecError("target_logits must be contiguous")
    _check(proposed, "proposed", torch.int32, (B, K), dev, optional=(K == 0))
    _check(num_draft, "num_draft", torch.int32, (B,), dev, optional=True)
    acc, tok, prb = _outputs(B, K, dev, out, want_probs, stream)
    ws, need = _workspace(B, K, V, dev, workspace, stream)
    status = lib.specdec_verify_greedy(_ptr(target_logits), dt, _ptr(proposed), _ptr(num_draft),
                                       B, K, V, _ptr(acc), _ptr(tok), _ptr(prb), _ptr(ws),
                                       ws.numel(), _stream_handle(stream))
    _raise(status, "specdec_verify_greedy")
    return acc, tok, prb


def specdec_verify_match(target_logits: torch.Tensor, proposed: torch.Tensor | None,
                         temperature: torch.Tensor, uniforms: torch.Tensor, *,
                         num_draft: torch.Tensor | None = None, out=None, workspace=None,
                         want_probs: bool = True, stream=None):
    """Sample-and-match verify (no draft distribution).  Shapes as for specdec_verify.  Returns
    (accept_len, out_tokens, out_probs or None)."""
    lib = load_library()
    if target_logits.dim() != 3:
        raise SpecdecError("target_logits must be [B, K+1, V]")
    B, K1, V = (int(s) for s in target_logits.shape)
    K = K1 - 1
    dev = target_logits.device
    if target_logits.dtype == torch.bfloat16:
        dt = SPECDEC_BF16
    elif target_logits.dtype == torch.float32:
        dt = SPECDEC_F32
    else:
        raise SpecdecError(f"target_logits dtype {target_logits.dtype} is not bf16/fp32")
    if not target_logits.is_contiguous():
        raise SpecdecError("target_logits must be contiguous")
    _check(proposed, "proposed", torch.int32, (B, K), dev, optional=(K == 0))
    _check(temperature, "temperature", torch.float32, (B,), dev)
    _check(uniforms, "uniforms", torch.float32, (B, K + 1), dev)
    _check(num_draft, "num_draft", torch.int32, (B,), dev, optional=True)
    acc, tok, prb = _outputs(B, K, dev, out, want_probs, stream)
    ws, need = _workspace(B, K, V, dev, workspace, stream)
    status = lib.specdec_verify_match(_ptr(target_logits), dt, _ptr(proposed), _ptr(num_draft),
                                      _ptr(temperature), _ptr(uniforms), B, K, V, _ptr(acc),
                                      _ptr(tok), _ptr(prb), _ptr(ws), ws.numel(),
                                      _stream_handle(stream))
    _raise(status, "specdec_verify_match")
    return acc, tok, prb


def specdec_ngram_workspace_size(B: int, capacity: int) -> int:
    return int(load_library().specdec_ngram_workspace_size(int(B), int(capacity)))


def specdec_ngram_propose(tokens: torch.Tensor, lengths: torch.Tensor, K: int, *, n_min: int = 1,
                          n_max: int = 4, out=None, workspace=None, stream=None):
    """N-gram drafter.  tokens [B, capacity] int32 histories, lengths [B] int32.  Returns
    (proposed [B, K] int32, num_draft [B] int32), enqueued on ``stream`` without synchronising."""
    lib = load_library()
    if tokens.dim() != 2:
        raise SpecdecError("tokens must be [B, capacity]")
    B, cap = (int(s) for s in tokens.shape)
    dev = tokens.device
    _check(tokens, "tokens", torch.int32, (B, cap), dev)
    _check(lengths, "lengths", torch.int32, (B,), dev)
    if out is None:
        with _on(stream):
            out = (torch.empty((B, K), dtype=torch.int32, device=dev),
                   torch.empty(B, dtype=torch.int32, device=dev))
    proposed, num_draft = out
    _check(proposed, "proposed", torch.int32, (B, K), dev)
    _check(num_draft, "num_draft", torch.int32, (B,), dev)
    need = specdec_ngram_workspace_size(B, cap)
    if workspace is None:
        with _on(stream):
            workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=dev)
    status = lib.specdec_ngram_propose(_ptr(tokens), _ptr(lengths), B, cap, int(n_min), int(n_max),
                                       int(K), _ptr(proposed) if K > 0 else None, _ptr(num_draft),
                                       _ptr(workspace), workspace.numel(), _stream_handle(stream))
    _raise(status, "specdec_ngram_propose")
    return proposed, num_draft


def specdec_commit(accept_len: torch.Tensor, out_tokens: torch.Tensor, seq_len: torch.Tensor, *,
                   tokens: torch.Tensor | None = None, capacity: int | None = None,
                   target_kv_len: torch.Tensor | None = None,
                   draft_kv_len: torch.Tensor | None = None, packed: bool = True, out=None,
                   stream=None):
    """Commit a verified round in place: append the emitted tokens to ``tokens`` [B, capacity]
    (optional), advance ``seq_len`` [B], roll ``target_kv_len`` / ``draft_kv_len`` [B] back
    (optional), and with ``packed`` return (packed_tokens [B*(K+1)], packed_offsets [B+1]);
    otherwise return None.  ``capacity`` defaults to tokens.shape[1]."""
    lib = load_library()
    if out_tokens.dim() != 2:
        raise SpecdecError("out_tokens must be [B, K+1]")
    B, K1 = (int(s) for s in out_tokens.shape)
    dev = out_tokens.device
    _check(accept_len, "accept_len", torch.int32, (B,), dev)
    _check(out_tokens, "out_tokens", torch.int32, (B, K1), dev)
    _check(seq_len, "seq_len", torch.int32, (B,), dev)
    if tokens is not None:
        if tokens.dim() != 2:
            raise SpecdecError("tokens must be [B, capacity]")
        _check(tokens, "tokens", torch.int32, (B, int(tokens.shape[1])), dev)
        cap = int(tokens.shape[1])
        if capacity is not None and int(capacity) != cap:
            raise SpecdecError("capacity differs from tokens.shape[1]")
    elif capacity is None:
        raise SpecdecError("capacity is required when no history tensor is given")
    else:
        cap = int(capacity)
    _check(target_kv_len, "target_kv_len", torch.int32, (B,), dev, optional=True)
    _check(draft_kv_len, "draft_kv_len", torch.int32, (B,), dev, optional=True)
    pk = off = None
    if packed:
        if out is None:
            with _on(stream):
                out = (torch.empty(max(B * K1, 1), dtype=torch.int32, device=dev),
                       torch.empty(B + 1, dtype=torch.int32, device=dev))
        pk, off = out
    status = lib.specdec_commit(_ptr(accept_len), _ptr(out_tokens), B, K1 - 1, _ptr(tokens), cap,
                                _ptr(seq_len), _ptr(target_kv_len), _ptr(draft_kv_len), _ptr(pk),
                                _ptr(off), _stream_handle(stream))
    _raise(status, "specdec_commit")
    return (pk, off) if packed else None


TELEMETRY_ROW = 72
TELEMETRY_MAX_ROUTES = 64


def telemetry_counters(n_routes: int, device) -> torch.Tensor:
    """Zeroed device counters [n_routes, 72] int64 for specdec_telemetry_update."""
    return torch.zeros((n_routes, TELEMETRY_ROW), dtype=torch.int64, device=device)


def specdec_telemetry_update(counters: torch.Tensor, accept_len: torch.Tensor, *,
                             num_draft: torch.Tensor | None = None,
                             route: torch.Tensor | None = None, K: int, stream=None):
    """Add one verified batch to the device counters [n_routes, 72] int64 (in place)."""
    lib = load_library()
    B = int(accept_len.shape[0])
    dev = accept_len.device
    n_routes = int(counters.shape[0])
    _check(counters, "counters", torch.int64, (n_routes, TELEMETRY_ROW), dev)
    _check(accept_len, "accept_len", torch.int32, (B,), dev)
    _check(num_draft, "num_draft", torch.int32, (B,), dev, optional=True)
    _check(route, "route", torch.int32, (B,), dev, optional=True)
    status = lib.specdec_telemetry_update(_ptr(accept_len), _ptr(num_draft), _ptr(route), B,
                                          int(K), n_routes, _ptr(counters), _stream_handle(stream))
    _raise(status, "specdec_telemetry_update")
    return counters


def specdec_apply_k(num_draft: torch.Tensor, k_table: torch.Tensor, *,
                    route: torch.Tensor | None = None, stream=None):
    """Clamp num_draft [B] (in place) to k_table [n_routes] of each sequence's route."""
    lib = load_library()
    B = int(num_draft.shape[0])
    dev = num_draft.device
    _check(num_draft, "num_draft", torch.int32, (B,), dev)
    _check(k_table, "k_table", torch.int32, (int(k_table.shape[0]),), dev)
    _check(route, "route", torch.int32, (B,), dev, optional=True)
    status = lib.specdec_apply_k(_ptr(num_draft), _ptr(route), _ptr(k_table), B,
                                 int(k_table.shape[0]), _stream_handle(stream))
    _raise(status, "specdec_apply_k")
    return num_draft


def specdec_plan_k(counters_host, c: float, k_min: int, k_max: int, k_default: int):
    """Host planner: counters (host int64 [n_routes, 72], numpy or CPU tensor) -> k per route
    (numpy int32), through the library's host arithmetic."""
    import numpy as np
    cnt = np.ascontiguousarray(np.asarray(counters_host, dtype=np.int64))
    n_routes = cnt.shape[0]
    out = np.empty(n_routes, dtype=np.int32)
    status = load_library().specdec_plan_k(cnt.ctypes.data, n_routes, float(c), int(k_min),
                                           int(k_max), int(k_default), out.ctypes.data)
    _raise(status, "specdec_plan_k")
    return out


SPECDEC_MAX_HEAD_DIM = 256
_KV_DTYPES = {torch.float32: SPECDEC_F32, torch.bfloat16: SPECDEC_BF16, torch.float16: SPECDEC_F16}
_ROPE_SCALINGS = {"plain": 0, "linear": 1, "base": 2, "turns": 3}


class PagedKvCache:
    """A paged key-value cache as the entry points of include/specdec.h take it: the pools ``k`` and
    ``v`` [num_pages, page_size, kv_heads, head_dim] (bf16, fp16 or fp32; any strides with dense
    rows, the same for both, so a head-major pool is passed as ``pool.transpose(1, 2)``),
    ``page_table`` [B, max_pages] int32, and for caches that evict the slots' records ``weight``
    (fp32) and ``position`` (int32) [num_pages, kv_heads, page_size].  Holds the tensors; checked
    once here, so that a decode loop's calls pass it on as it is."""

    def __init__(self, k: torch.Tensor, v: torch.Tensor, page_table: torch.Tensor, *,
                 weight: torch.Tensor | None = None, position: torch.Tensor | None = None):
        if k.dim() != 4:
            raise SpecdecError("k must be [num_pages, page_size, kv_heads, head_dim]")
        if k.dtype not in _KV_DTYPES:
            raise SpecdecError(f"k dtype {k.dtype} is not bf16/fp16/fp32")
        if v.device != k.device or v.dtype != k.dtype or v.shape != k.shape:
            raise SpecdecError("v must have the device, dtype and shape of k")
        pages, page_size, heads, dim = (int(x) for x in k.shape)
        used = [n for n, size in enumerate(k.shape) if size > 1]
        if any(k.stride(n) != v.stride(n) for n in used):
            raise SpecdecError("v must have the strides of k")
        if dim > 1 and k.stride(3) != 1:
            raise SpecdecError("the rows (last dimension) of k and v must be contiguous")
        if page_table.dim() != 2:
            raise SpecdecError("page_table must be [B, max_pages]")
        self.B, max_pages = (int(x) for x in page_table.shape)
        _check(page_table, "page_table", torch.int32, (self.B, max_pages), k.device)
        _check(weight, "weight", torch.float32, (pages, heads, page_size), k.device, optional=True)
        _check(position, "position", torch.int32, (pages, heads, page_size), k.device, optional=True)
        self.k, self.v, self.page_table, self.weight, self.position = (k, v, page_table, weight,
                                                                       position)
        self.device, self.dtype = k.device, k.dtype
        self.num_pages, self.page_size, self.kv_heads, self.head_dim = pages, page_size, heads, dim
        self.max_pages = max_pages
        self._c = _KvCache(_ptr(k), _ptr(v), _KV_DTYPES[k.dtype], pages, page_size, heads, dim,
                           max_pages, k.stride(0), k.stride(1), k.stride(2), _ptr(page_table),
                           _ptr(weight), _ptr(position))
        self._ref = ctypes.addressof(self._c)


def _call(cache: PagedKvCache, stream, fn, name: str, *args):
    """fn(*args, stream) with the cache's device current (a launch goes to the current device)."""
    dev = cache.device
    if dev.type != "cuda":
        raise SpecdecError(f"the cache is on {dev}, expected a GPU")
    if stream is None:  # (the handle alone: a torch.cuda.Stream takes 1.8 us of a call's 9 to make)
        handle = torch._C._cuda_getCurrentRawStream(dev.index)
    elif stream.device != dev:
        raise SpecdecError(f"stream is on {stream.device}, expected {dev}")
    else:
        handle = stream.cuda_stream
    if torch.cuda.current_device() == dev.index:
        status = fn(*args, handle)
    else:
        with torch.cuda.device(dev):
            status = fn(*args, handle)
    if status != 0:
        _raise(status, name)


def _tokens(t: torch.Tensor, name: str, cache: PagedKvCache, B: int, T: int, heads: int) -> int:
    """Checks a [B, T, heads, head_dim] tensor of the cache's type with dense tokens evenly spaced;
    returns the spacing in elements."""
    if t.device != cache.device:
        raise SpecdecError(f"{name} is on {t.device}, expected {cache.device}")
    if t.dtype != cache.dtype:
        raise SpecdecError(f"{name} has dtype {t.dtype}, expected {cache.dtype}")
    if t.shape != (B, T, heads, cache.head_dim):
        raise SpecdecError(f"{name} has shape {tuple(t.shape)}, expected "
                           f"{(B, T, heads, cache.head_dim)}")
    s0, s1, s2, s3 = t.stride()
    if s3 != 1 or (heads > 1 and s2 != cache.head_dim):
        raise SpecdecError(f"the heads and rows of {name} must be contiguous")
    if B > 1 and T > 1 and s0 != T * s1:
        raise SpecdecError(f"the tokens of {name} must be evenly spaced")
    return s1 if T > 1 else s0


def _round_shape(q: torch.Tensor, cache: PagedKvCache):
    if q.dim() != 4:
        raise SpecdecError("q must be [B, K+1, heads, head_dim]")
    B, T, heads, _ = q.shape
    if B != cache.B:
        raise SpecdecError(f"q has {B} sequences, the cache's page table {cache.B}")
    if T < 1:
        raise SpecdecError("q must hold K+1 >= 1 tokens a sequence")
    return B, T, heads


def _scale_of(scale, cache: PagedKvCache) -> float:
    return cache.head_dim ** -0.5 if scale is None else float(scale)


def specdec_rope_frequencies(rotary_dim: int, base: float = 10000.0, *, scaling: str = "plain",
                             factor: float = 1.0, original_len: float = 0.0,
                             turns_low: float = 1.0, turns_high: float = 32.0) -> np.ndarray:
    """Angular frequencies of the rotary pairs (host float64 [rotary_dim / 2]); ``scaling``: "plain",
    "linear" (positions divided by ``factor``), "base" (a larger base) or "turns" (by each pair's
    number of turns over ``original_len``).  Copy them to the device for specdec_rope_append."""
    if scaling not in _ROPE_SCALINGS:
        raise SpecdecError(f"scaling {scaling!r} is not one of {sorted(_ROPE_SCALINGS)}")
    out = np.empty(max(int(rotary_dim) // 2, 1), dtype=np.float64)
    status = load_library().specdec_rope_frequencies(
        int(rotary_dim), float(base), _ROPE_SCALINGS[scaling], float(factor), float(original_len),
        float(turns_low), float(turns_high), out.ctypes.data)
    _raise(status, "specdec_rope_frequencies")
    return out


def specdec_rope_append(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, cache: PagedKvCache,
                        kv_len: torch.Tensor, inv_freq: torch.Tensor | None, *,
                        interleaved: bool = False, rope_scale: float = 1.0,
                        num_draft: torch.Tensor | None = None,
                        first_pos: torch.Tensor | None = None, out: torch.Tensor | None = None,
                        stream=None) -> torch.Tensor:
    """Rotate a round's new tokens and append them to the cache.  q [B, K+1, heads, head_dim], k and v
    [B, K+1, kv_heads, head_dim] in the cache's type (slices of a fused projection included), kv_len
    [B] int32 slots in use, inv_freq [rotary_dim / 2] float64 on the device (None: nothing is
    rotated), num_draft / first_pos [B] int32 or None (K; kv_len).  Returns the rotated q (``out``,
    which may be q itself), enqueued on ``stream`` without synchronising."""
    lib = load_library()
    B, T, heads = _round_shape(q, cache)
    dev = cache.device
    qs = _tokens(q, "q", cache, B, T, heads)
    ks = _tokens(k, "k", cache, B, T, cache.kv_heads)
    vs = _tokens(v, "v", cache, B, T, cache.kv_heads)
    _check(kv_len, "kv_len", torch.int32, (B,), dev)
    _check(num_draft, "num_draft", torch.int32, (B,), dev, optional=True)
    _check(first_pos, "first_pos", torch.int32, (B,), dev, optional=True)
    half = 0
    if inv_freq is not None:
        half = int(inv_freq.numel())
        _check(inv_freq, "inv_freq", torch.float64, (half,), dev)
    if out is None:
        with _on(stream):
            out = torch.empty((B, T, heads, cache.head_dim), dtype=cache.dtype, device=dev)
    else:
        _check(out, "out", cache.dtype, (B, T, heads, cache.head_dim), dev)
    rope = _Rope(_ptr(inv_freq), 2 * half, 1 if interleaved else 0, rope_scale)
    _call(cache, stream, lib.specdec_rope_append, "specdec_rope_append", q.data_ptr(), k.data_ptr(),
          v.data_ptr(), qs, ks, vs, B, T - 1, heads, _ptr(num_draft), kv_len.data_ptr(),
          _ptr(first_pos), ctypes.addressof(rope), cache._ref, out.data_ptr())
    return out


def specdec_paged_attention_workspace_size(B: int, K: int, heads: int, kv_heads: int,
                                           head_dim: int) -> int:
    return int(load_library().specdec_paged_attention_workspace_size(
        int(B), int(K), int(heads), int(kv_heads), int(head_dim)))


def new_paged_attention_workspace(cache: PagedKvCache, K: int, heads: int, stream=None) -> torch.Tensor:
    """A workspace for specdec_paged_attention calls of up to K drafts (uninitialised: the library
    needs none), allocated for ``stream``."""
    need = specdec_paged_attention_workspace_size(cache.B, K, heads, cache.kv_heads, cache.head_dim)
    with _on(stream):
        return torch.empty(max(need, 16), dtype=torch.uint8, device=cache.device)


def specdec_paged_attention(q: torch.Tensor, cache: PagedKvCache, kv_len: torch.Tensor, *,
                            num_draft: torch.Tensor | None = None, scale: float | None = None,
                            out: torch.Tensor | None = None, lse: torch.Tensor | None = None,
                            want_lse: bool = False, workspace: torch.Tensor | None = None,
                            stream=None):
    """Attention of a round's tokens (already appended) over the cache.  q [B, K+1, heads, head_dim],
    kv_len [B] int32 slots before the round, num_draft [B] int32 or None, scale (default
    head_dim^-0.5).  Returns (out [B, K+1, heads, head_dim], lse [B, K+1, heads] fp32 or None; lse
    when ``want_lse`` or a tensor for it is given), enqueued on ``stream`` without synchronising.
    ``workspace``: new_paged_attention_workspace, reusable across calls; None allocates one."""
    lib = load_library()
    B, T, heads = _round_shape(q, cache)
    dev = cache.device
    qs = _tokens(q, "q", cache, B, T, heads)
    _check(kv_len, "kv_len", torch.int32, (B,), dev)
    _check(num_draft, "num_draft", torch.int32, (B,), dev, optional=True)
    if out is None:
        with _on(stream):
            out = torch.empty((B, T, heads, cache.head_dim), dtype=cache.dtype, device=dev)
    else:
        _check(out, "out", cache.dtype, (B, T, heads, cache.head_dim), dev)
    if lse is not None:
        _check(lse, "lse", torch.float32, (B, T, heads), dev)
    elif want_lse:
        with _on(stream):
            lse = torch.empty((B, T, heads), dtype=torch.float32, device=dev)
    if workspace is None:
        workspace = new_paged_attention_workspace(cache, T - 1, heads, stream)
    else:
        _check_workspace(workspace, dev)
    _call(cache, stream, lib.specdec_paged_attention, "specdec_paged_attention", q.data_ptr(), qs, B,
          T - 1, heads, _ptr(num_draft), kv_len.data_ptr(), _scale_of(scale, cache), cache._ref,
          out.data_ptr(), _ptr(lse), workspace.data_ptr(), workspace.numel())
    return out, lse


def _check_workspace(workspace: torch.Tensor, dev):
    if workspace.device != dev or workspace.dtype != torch.uint8 or not workspace.is_contiguous():
        raise SpecdecError(f"workspace must be a contiguous uint8 tensor on {dev}")


def specdec_kv_weights(q: torch.Tensor, lse: torch.Tensor, cache: PagedKvCache,
                       kv_len: torch.Tensor, *, num_draft: torch.Tensor | None = None,
                       accept_len: torch.Tensor | None = None, scale: float | None = None,
                       stream=None) -> torch.Tensor:
    """Add to ``cache.weight`` (in place; returned) the attention weights that the accepted rows of a
    round gave each slot: q, lse, kv_len, num_draft and scale of the attention call, accept_len [B]
    int32 of the verify step (None: every row)."""
    lib = load_library()
    B, T, heads = _round_shape(q, cache)
    dev = cache.device
    if cache.weight is None:
        raise SpecdecError("the cache has no weight records")
    qs = _tokens(q, "q", cache, B, T, heads)
    _check(lse, "lse", torch.float32, (B, T, heads), dev)
    _check(kv_len, "kv_len", torch.int32, (B,), dev)
    _check(num_draft, "num_draft", torch.int32, (B,), dev, optional=True)
    _check(accept_len, "accept_len", torch.int32, (B,), dev, optional=True)
    _call(cache, stream, lib.specdec_kv_weights, "specdec_kv_weights", q.data_ptr(), qs,
          lse.data_ptr(), B, T - 1, heads, _ptr(num_draft), _ptr(accept_len), kv_len.data_ptr(),
          _scale_of(scale, cache), cache._ref)
    return cache.weight


def new_kv_evict_workspace(cache: PagedKvCache, budget: int, stream=None) -> torch.Tensor:
    """A workspace for specdec_kv_evict calls with this budget (uninitialised), allocated for
    ``stream``."""
    need = int(load_library().specdec_kv_evict_workspace_size(cache.B, cache._ref, int(budget)))
    with _on(stream):
        return torch.empty(max(need, 16), dtype=torch.uint8, device=cache.device)


def specdec_kv_evict(cache: PagedKvCache, kv_len: torch.Tensor, budget: int, *, keep_first: int = 0,
                     keep_last: int = 0, new_len: torch.Tensor | None = None,
                     workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Evict the lightest slots of every sequence longer than ``budget``, in place in the cache's k,
    v, weight and position.  Returns new_len [B] int32 (``new_len`` may be kv_len itself; None
    allocates it): min(kv_len, budget), or -1 for an invalid sequence."""
    lib = load_library()
    dev = cache.device
    if cache.weight is None or cache.position is None:
        raise SpecdecError("the cache has no weight and position records")
    _check(kv_len, "kv_len", torch.int32, (cache.B,), dev)
    if new_len is None:
        with _on(stream):
            new_len = torch.empty(cache.B, dtype=torch.int32, device=dev)
    else:
        _check(new_len, "new_len", torch.int32, (cache.B,), dev)
    if workspace is None:
        workspace = new_kv_evict_workspace(cache, budget, stream)
    else:
        _check_workspace(workspace, dev)
    _call(cache, stream, lib.specdec_kv_evict, "specdec_kv_evict", cache._ref, kv_len.data_ptr(),
          cache.B, int(budget), int(keep_first), int(keep_last), new_len.data_ptr(),
          workspace.data_ptr(), workspace.numel())
    return new_len


def inputs_to_device(inp, device) -> dict:
    """Copy a host ``VerifyInputs`` batch to device tensors (bf16 bit patterns become bf16)."""
    def dev(a, dtype=None):
        if a is None:
            return None
        if not a.flags.writeable:  # e.g. a broadcast view: torch wants a writable buffer
            a = np.array(a)
        t = torch.from_numpy(a)
        if dtype is not None:
            t = t.view(dtype)
        return t.to(device).contiguous()
    if inp.logits_dtype == "bf16":
        logits = dev(inp.logits.view("int16"), torch.bfloat16)
    elif inp.logits_dtype == "f32":
        logits = dev(inp.logits)
    else:
        raise SpecdecError(f"logits dtype {inp.logits_dtype!r} has no device form")
    return dict(logits=logits, draft_probs=dev(inp.draft_probs), draft_onehot=dev(inp.draft_onehot),
                proposed=dev(inp.proposed), num_draft=dev(inp.num_draft),
                temperature=dev(inp.temperature), uniforms=dev(inp.uniforms))


class PreparedVerify:
    """A specdec_verify call with its arguments marshalled once (for tight loops and HIP-graph
    capture).  ``__call__(stream=None, hot_events=None, draw_events=None)`` enqueues it on ``stream`` (default:
    torch's current stream) and raises on a non-zero status."""

    def __init__(self, target_logits, draft_probs, proposed, temperature, uniforms, *,
                 draft_onehot=None, num_draft=None, out=None, workspace=None,
                 path=SPECDEC_PATH_AUTO):
        # Validate once through the checked entry point's rules.
        B, K1, V = (int(s) for s in target_logits.shape)
        dev = target_logits.device
        self.lib = load_library()
        self.keep = (target_logits, draft_probs, proposed, temperature, uniforms, draft_onehot,
                     num_draft)
        dt = SPECDEC_BF16 if target_logits.dtype == torch.bfloat16 else SPECDEC_F32
        _check(draft_probs, "draft_probs", torch.float32, (B, K1 - 1, V), dev, optional=True)
        _check(proposed, "proposed", torch.int32, (B, K1 - 1), dev, optional=(K1 == 1))
        _check(temperature, "temperature", torch.float32, (B,), dev)
        _check(uniforms, "uniforms", torch.float32, (B, K1), dev)
        _check(draft_onehot, "draft_onehot", torch.uint8, (B,), dev, optional=True)
        _check(num_draft, "num_draft", torch.int32, (B,), dev, optional=True)
        self.out = _outputs(B, K1 - 1, dev, out, True)
        self.ws, _ = _workspace(B, K1 - 1, V, dev, workspace)
        acc, tok, prb = self.out
        self.path = int(path)
        self.args = (_ptr(target_logits), dt, _ptr(draft_probs), _ptr(draft_onehot),
                     _ptr(proposed), _ptr(num_draft), _ptr(temperature), _ptr(uniforms), B,
                     K1 - 1, V, _ptr(acc), _ptr(tok), _ptr(prb), _ptr(self.ws), self.ws.numel())

    def __call__(self, stream=None, hot_events=None, draw_events=None):
        s = _stream_handle(stream)
        if hot_events is None and draw_events is None and self.path == SPECDEC_PATH_AUTO:
            status = self.lib.specdec_verify(*self.args, s)
        else:
            opts = _options(hot_events, self.path, 0, draw_events)
            status = self.lib.specdec_verify_ex(*self.args, s, ctypes.byref(opts))
        if status != 0:
            _raise(status, "specdec_verify")
        return self.out
