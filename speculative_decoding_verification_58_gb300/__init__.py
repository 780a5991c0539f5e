"""GB300-native batched speculative-decoding verification.

A thin Python binding over the C ABI of ``libspecverify.so`` (declared in
``include/spec_verify.h``).  Every step of verification runs in the
library's CUDA kernels; this module only checks tensor shapes, passes raw
device pointers and the current CUDA stream, and turns status codes into
exceptions.  There is no CPU fallback: if the library has not been built,
every call raises.

The functions keep the C names:

``spec_verify(...)``                 batched verification (asynchronous)
``spec_verify_packed(...)``          the same over a packed (ragged) batch of rows
``Verifier(...)``                    spec_verify bound to fixed buffers (one C call per round)
``spec_verify_workspace_bytes(...)`` workspace size for (B, k, V)
``spec_verify_report(ws)``           what the device recorded for the last call
``spec_verify_device_status(ws)``    just the recorded status
``spec_row_stats(...)``              the row sweep alone: max, logsumexp, argmax
``spec_opd_stats(...)``              OPD supervision statistics (hard label, reverse KL, clipped)
``spec_verify_opd(...)``             verification and OPD statistics in one pass over the rows
``spec_d3d_select(...)``             D3D branch selection: reuse a prepared successor block
``spec_linear_ce(...)``              cross entropy of a linear vocabulary head, without the logits
``spec_linear_ce_grad(...)``         its gradients (hidden states and weight)
``LinearCe(...)``                    both bound to fixed buffers
``spec_opd_grad(...)``               gradient of the OPD mixture loss (draft logits)
``spec_grad_norm(...)``              global norm of many gradient tensors
``spec_clip_grad_norm(...)``         the same, and the tensors scaled to a largest norm
``GradClipper(...)``                 the clip bound to fixed tensors
``spec_sample(...)``                 tokens drawn under temperature, top-k, top-p and min-p
``spec_truncate(...)``               the same truncation, written as logits
``Sampler(...)``                     both bound to fixed buffers
``spec_kv_append(...)``              new tokens' keys and values into a paged cache
``spec_paged_attention(...)``        attention of the new tokens over their pages
``PagedCache(...)``                  both bound to fixed buffers
``spec_status_string(code)``
``spec_debug_build()``, ``spec_debug_checks()``, ``spec_debug_inject()``
                                     the range-checking build (SPEC_VERIFY_DEBUG=1)
"""

from __future__ import annotations

import contextlib
import ctypes
import os
from dataclasses import dataclass

_HERE = os.path.dirname(os.path.abspath(__file__))
# SPEC_VERIFY_DEBUG=1 in the environment loads the range-checking build
# (same entry points; see spec_debug_checks) instead of the release one.
DEBUG_BUILD = os.environ.get("SPEC_VERIFY_DEBUG", "") not in ("", "0")
LIB_PATH = os.path.join(_HERE, "libspecverify_debug.so" if DEBUG_BUILD else "libspecverify.so")

SPEC_OK = 0
SPEC_ERR_INVALID_ARG = 1
SPEC_ERR_UNSUPPORTED = 2
SPEC_ERR_WORKSPACE = 3
SPEC_ERR_CUDA = 4
SPEC_ERR_BAD_INPUT = 5
SPEC_ERR_TIMEOUT = 6
SPEC_ERR_INTERNAL = 7
SPEC_F32 = 0
SPEC_BF16 = 1
SPEC_TIMEOUT_NAN = 0x7fc10557
SPEC_FLAG_FULL_SWEEP = 1
SPEC_FLAG_TEST_LATE_SLICES = 2

# Every entry point include/spec_verify.h declares.
EXPORTS = ("spec_verify_workspace_bytes", "spec_verify", "spec_verify_ex", "spec_verify_timed",
           "spec_verify_packed", "spec_verify_report",
           "spec_verify_device_status", "spec_row_stats_workspace_bytes", "spec_row_stats",
           "spec_status_string", "spec_abi_version", "spec_verify_static", "spec_opd_stats",
           "spec_verify_opd", "spec_d3d_select", "spec_linear_ce_workspace_bytes",
           "spec_linear_ce", "spec_linear_ce_grad_workspace_bytes", "spec_linear_ce_grad",
           "spec_opd_grad", "spec_grad_norm_workspace_bytes", "spec_grad_norm",
           "spec_clip_grad_norm", "spec_sample", "spec_truncate", "spec_kv_append",
           "spec_paged_attention_workspace_bytes", "spec_paged_attention",
           "spec_debug_build", "spec_debug_checks", "spec_debug_inject")
SPEC_STATIC_SCRATCH_BYTES = 8 << 20


class SpecVerifyError(RuntimeError):
    def __init__(self, code: int, where: str):
        self.code = code
        super().__init__(f"{where}: {status_string(code)} (status {code})")


class _Report(ctypes.Structure):
    _fields_ = [("status", ctypes.c_int32), ("bad_requests", ctypes.c_int32),
                ("first_bad_request", ctypes.c_int32), ("rows_planned", ctypes.c_int32),
                ("chunks_swept", ctypes.c_int64), ("chunks_per_row", ctypes.c_int32),
                ("chunk_elems", ctypes.c_int32), ("final_rows", ctypes.c_int64),
                ("residual_zero", ctypes.c_int32), ("reserved", ctypes.c_int32),
                ("sweep_bytes", ctypes.c_int64), ("final_bytes", ctypes.c_int64)]


class _PagedCache(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_void_p) for n in ("k_cache", "v_cache")]
                + [(n, ctypes.c_longlong) for n in ("k_page", "k_slot", "k_head", "v_page",
                                                    "v_slot", "v_head")]
                + [(n, ctypes.c_int) for n in ("num_pages", "page_size", "kv_heads", "width")]
                + [("page_table", ctypes.c_void_p), ("max_pages", ctypes.c_int),
                   ("new_start", ctypes.c_void_p), ("kv_len", ctypes.c_void_p),
                   ("B", ctypes.c_int)])


@dataclass
class Report:
    status: int
    bad_requests: int
    first_bad_request: int
    rows_planned: int
    chunks_swept: int
    chunks_per_row: int
    chunk_elems: int
    final_rows: int
    residual_zero: int
    sweep_bytes: int
    final_bytes: int


_lib = None


def lib() -> ctypes.CDLL:
    """The loaded ``libspecverify.so``; raises if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"{LIB_PATH} is missing: build it first "
                           "(python -c 'import __graft_entry__ as g; g.build()')")
    L = ctypes.CDLL(LIB_PATH)
    vp, i32p, f32p = ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p
    ci, csz = ctypes.c_int, ctypes.c_size_t
    L.spec_verify_workspace_bytes.argtypes = [ci, ci, ci]
    L.spec_verify_workspace_bytes.restype = csz
    L.spec_verify.argtypes = [vp, vp, ci, i32p, i32p, f32p, f32p, ci, ci, ci, i32p, i32p, vp, csz, vp]
    L.spec_verify.restype = ci
    L.spec_verify_ex.argtypes = L.spec_verify.argtypes + [ctypes.c_uint]
    L.spec_verify_ex.restype = ci
    L.spec_verify_timed.argtypes = L.spec_verify_ex.argtypes + [vp, vp, vp, vp]
    L.spec_verify_timed.restype = ci
    L.spec_verify_packed.argtypes = [vp, ctypes.c_longlong, vp, ctypes.c_longlong, ci, i32p, i32p,
                                     i32p, i32p, f32p, f32p, ci, ci, ci, i32p, i32p, vp, csz, vp,
                                     ctypes.c_uint]
    L.spec_verify_packed.restype = ci
    L.spec_verify_static.argtypes = [vp, vp, ci, i32p, i32p, f32p, f32p, ci, ci, ci, i32p, i32p, vp]
    L.spec_verify_static.restype = ci
    L.spec_verify_report.argtypes = [vp, vp, ctypes.POINTER(_Report)]
    L.spec_verify_report.restype = ci
    L.spec_verify_device_status.argtypes = [vp, vp]
    L.spec_verify_device_status.restype = ci
    L.spec_row_stats_workspace_bytes.argtypes = [ci, ci]
    L.spec_row_stats_workspace_bytes.restype = csz
    L.spec_row_stats.argtypes = [vp, ci, ci, ci, f32p, f32p, f32p, i32p, vp, csz, vp]
    L.spec_row_stats.restype = ci
    L.spec_opd_stats.argtypes = [vp, vp, ci, i32p, ci, ci, ci, ctypes.c_float, ctypes.c_float,
                                 i32p, f32p, f32p, f32p, f32p, vp]
    L.spec_opd_stats.restype = ci
    L.spec_verify_opd.argtypes = [vp, vp, ci, i32p, i32p, f32p, f32p, ci, ci, ci, ctypes.c_float,
                                  ctypes.c_float, i32p, i32p, i32p, f32p, f32p, f32p, f32p, vp, csz,
                                  vp]
    L.spec_verify_opd.restype = ci
    L.spec_d3d_select.argtypes = [i32p, i32p, i32p, i32p, i32p, ci, ci, ci, ci, i32p, i32p, i32p,
                                  vp]
    L.spec_d3d_select.restype = ci
    for name in ("spec_linear_ce_workspace_bytes", "spec_linear_ce_grad_workspace_bytes"):
        getattr(L, name).argtypes = [ci, ci, ci]
        getattr(L, name).restype = csz
    L.spec_linear_ce.argtypes = [vp, vp, ci, i32p, ci, ci, ci, f32p, f32p, vp, csz, vp]
    L.spec_linear_ce.restype = ci
    L.spec_linear_ce_grad.argtypes = [vp, vp, ci, i32p, f32p, f32p, f32p, ci, ci, ci, vp, vp, vp,
                                      csz, vp]
    L.spec_linear_ce_grad.restype = ci
    L.spec_opd_grad.argtypes = [vp, vp, ci, i32p, f32p, ci, ci, ci, ctypes.c_float, ctypes.c_float,
                                vp, vp]
    L.spec_opd_grad.restype = ci
    L.spec_grad_norm_workspace_bytes.argtypes = [ci]
    L.spec_grad_norm_workspace_bytes.restype = csz
    L.spec_grad_norm.argtypes = [vp, vp, vp, ci, f32p, vp, csz, vp]
    L.spec_grad_norm.restype = ci
    L.spec_clip_grad_norm.argtypes = [vp, vp, vp, vp, ci, ctypes.c_float, f32p, vp, csz, vp]
    L.spec_clip_grad_norm.restype = ci
    L.spec_sample.argtypes = [vp, ci, ci, ci, ci, f32p, i32p, f32p, f32p, f32p, i32p, vp, vp]
    L.spec_sample.restype = ci
    L.spec_truncate.argtypes = [vp, ci, ci, ci, ci, f32p, i32p, f32p, f32p, vp, vp]
    L.spec_truncate.restype = ci
    cll = ctypes.c_longlong
    L.spec_kv_append.argtypes = [vp, ci, vp, vp, ci, cll, cll, vp]
    L.spec_kv_append.restype = ci
    L.spec_paged_attention_workspace_bytes.argtypes = [ci, ci, ci, ci]
    L.spec_paged_attention_workspace_bytes.restype = csz
    L.spec_paged_attention.argtypes = [vp, ci, vp, ci, ci, cll, ci, ci, ctypes.c_float, vp, f32p, vp,
                                       csz, vp]
    L.spec_paged_attention.restype = ci
    L.spec_status_string.argtypes = [ci]
    L.spec_status_string.restype = ctypes.c_char_p
    L.spec_abi_version.argtypes = []
    L.spec_abi_version.restype = ci
    L.spec_debug_build.argtypes = []
    L.spec_debug_build.restype = ci
    L.spec_debug_checks.argtypes = [vp, vp, ci, vp]
    L.spec_debug_checks.restype = ci
    L.spec_debug_inject.argtypes = [ci, vp]
    L.spec_debug_inject.restype = ci
    _lib = L
    return L


def build(force: bool = False) -> str:
    """Compile the library and its range-checking build in-tree with nvcc
    for sm_103a; return the path of the one this process loads."""
    global _lib
    from . import make_lib
    make_lib.build_all(force=force)
    _lib = None
    return LIB_PATH


def spec_debug_build() -> bool:
    """Whether the loaded library is the range-checking build."""
    return bool(lib().spec_debug_build())


def spec_debug_checks(reset: bool = False, stream=None) -> tuple[int, int]:
    """(failed range checks on the current device since the last reset, site
    of the first); both 0 in a release build."""
    import torch
    f, site = ctypes.c_int32(0), ctypes.c_int32(0)
    st = torch.cuda.current_stream() if stream is None else stream
    code = lib().spec_debug_checks(ctypes.addressof(f), ctypes.addressof(site), int(reset),
                                   ctypes.c_void_p(st.cuda_stream))
    if code != SPEC_OK:
        raise SpecVerifyError(code, "spec_debug_checks")
    return f.value, site.value


def spec_debug_inject(status: int, stream=None) -> None:
    """Range-checking build: linear cross entropy and paged attention record ``status`` (SPEC_ERR_TIMEOUT, or
    SPEC_OK to end it) as if a wait had run out; a release build refuses."""
    _check(lib().spec_debug_inject(status, _stream_ptr(stream)), "spec_debug_inject")


def status_string(code: int) -> str:
    try:
        return lib().spec_status_string(code).decode()
    except RuntimeError:
        return f"status {code}"


spec_status_string = status_string


def _check(code: int, where: str) -> None:
    if code != SPEC_OK:
        raise SpecVerifyError(code, where)


def _torch():
    import torch
    return torch


def _stream_ptr(stream) -> int:
    torch = _torch()
    if stream is None:
        stream = torch.cuda.current_stream()
    return int(stream.cuda_stream) if hasattr(stream, "cuda_stream") else int(stream)


def _dtype_code(t) -> int:
    torch = _torch()
    if t.dtype == torch.float32:
        return SPEC_F32
    if t.dtype == torch.bfloat16:
        return SPEC_BF16
    raise TypeError(f"logits must be float32 or bfloat16, got {t.dtype}")


def _need(t, name, dtype, shape, device):
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _need_logits(t, name, dtype, shape, device):
    """Logits on ``device``, or in pinned host memory, which the kernels then
    read themselves over the CPU-GPU link (no copy; early exit also spares
    the link the rows it skips)."""
    if t.device.type == "cpu":
        if not t.is_pinned():
            raise ValueError(f"{name} is in pageable host memory: pin it (pin_memory()) or move it "
                             f"to {device}")
        _need(t, name, dtype, shape, t.device)
    else:
        _need(t, name, dtype, shape, device)


def spec_verify_workspace_bytes(B: int, k: int, V: int) -> int:
    return int(lib().spec_verify_workspace_bytes(B, k, V))


def alloc_workspace(B: int, k: int, V: int, device=None):
    """A device workspace (torch uint8 tensor, 256-byte aligned by the caching allocator)."""
    torch = _torch()
    n = spec_verify_workspace_bytes(B, k, V)
    if n == 0:
        raise SpecVerifyError(SPEC_ERR_UNSUPPORTED, "spec_verify_workspace_bytes")
    return torch.empty(n, dtype=torch.uint8, device=device or "cuda")


def spec_verify(target_logits, draft_logits, draft_tokens, lengths, uniforms, temperature, *,
                workspace=None, out_tokens=None, num_accepted=None, stream=None,
                full_sweep: bool = False, events=None, flags: int = 0):
    """Batched verification on the current (or given) CUDA stream.

    Shapes: target [B, k+1, V], draft [B, k, V] (float32 or bfloat16, same),
    draft_tokens int32 [B, k], lengths int32 [B], uniforms float32 [B, k+1],
    temperature float32 [B].  Returns (out_tokens int32 [B, k+1],
    num_accepted int32 [B]); results are ready when the stream reaches them.

    ``events``: optional four recorded ``torch.cuda.Event`` objects (or None
    entries) marking plan / sweep / final / end, for per-kernel timing
    (measurement only: it disables the kernels' launch overlap).
    ``flags``: further SPEC_FLAG_* bits passed through unchanged.
    """
    torch = _torch()
    B, k1, V = target_logits.shape
    k = k1 - 1
    dev = draft_tokens.device
    dt = _dtype_code(target_logits)
    _need_logits(target_logits, "target_logits", target_logits.dtype, (B, k + 1, V), dev)
    _need_logits(draft_logits, "draft_logits", target_logits.dtype, (B, k, V), dev)
    _need(draft_tokens, "draft_tokens", torch.int32, (B, k), dev)
    _need(lengths, "lengths", torch.int32, (B,), dev)
    _need(uniforms, "uniforms", torch.float32, (B, k + 1), dev)
    _need(temperature, "temperature", torch.float32, (B,), dev)
    if workspace is None:
        workspace = alloc_workspace(B, k, V, dev)
    if out_tokens is None:
        out_tokens = torch.empty((B, k + 1), dtype=torch.int32, device=dev)
    if num_accepted is None:
        num_accepted = torch.empty((B,), dtype=torch.int32, device=dev)
    _need(out_tokens, "out_tokens", torch.int32, (B, k + 1), dev)
    _need(num_accepted, "num_accepted", torch.int32, (B,), dev)
    flags = int(flags) | (SPEC_FLAG_FULL_SWEEP if full_sweep else 0)
    args = (target_logits.data_ptr(), draft_logits.data_ptr(), dt, draft_tokens.data_ptr(),
            lengths.data_ptr(), uniforms.data_ptr(), temperature.data_ptr(), B, k, V,
            out_tokens.data_ptr(), num_accepted.data_ptr(), workspace.data_ptr(),
            workspace.numel() * workspace.element_size(), _stream_ptr(stream), flags)
    if events is None:
        code = lib().spec_verify_ex(*args)
    else:
        handles = [None if e is None else (e.cuda_event or None) for e in events]
        code = lib().spec_verify_timed(*args, *handles)
    _check(code, "spec_verify")
    return out_tokens, num_accepted


def spec_verify_packed(target_rows, draft_rows, target_row_start, draft_row_start, draft_tokens,
                       lengths, uniforms, temperature, *, workspace=None, out_tokens=None,
                       num_accepted=None, stream=None, full_sweep: bool = False):
    """Verification over a packed batch (AdaFlash Section 3.3: total length sum_b k_b).

    ``target_rows`` [rows_t, V] and ``draft_rows`` [rows_d, V] (float32 or
    bfloat16, same); request b reads target rows ``target_row_start[b] + 0..L_b``
    and draft rows ``draft_row_start[b] + 0..L_b-1`` (int32 [B] each).
    ``draft_tokens`` int32 [B, k] fixes k.  Other arguments and the results are
    those of ``spec_verify``.
    """
    torch = _torch()
    rows_t, V = target_rows.shape
    B, k = draft_tokens.shape
    dev = draft_tokens.device
    dt = _dtype_code(target_rows)
    rows_d = draft_rows.shape[0]
    _need_logits(target_rows, "target_rows", target_rows.dtype, (rows_t, V), dev)
    _need_logits(draft_rows, "draft_rows", target_rows.dtype, (rows_d, V), dev)
    _need(target_row_start, "target_row_start", torch.int32, (B,), dev)
    _need(draft_row_start, "draft_row_start", torch.int32, (B,), dev)
    _need(draft_tokens, "draft_tokens", torch.int32, (B, k), dev)
    _need(lengths, "lengths", torch.int32, (B,), dev)
    _need(uniforms, "uniforms", torch.float32, (B, k + 1), dev)
    _need(temperature, "temperature", torch.float32, (B,), dev)
    if workspace is None:
        workspace = alloc_workspace(B, k, V, dev)
    if out_tokens is None:
        out_tokens = torch.empty((B, k + 1), dtype=torch.int32, device=dev)
    if num_accepted is None:
        num_accepted = torch.empty((B,), dtype=torch.int32, device=dev)
    _need(out_tokens, "out_tokens", torch.int32, (B, k + 1), dev)
    _need(num_accepted, "num_accepted", torch.int32, (B,), dev)
    code = lib().spec_verify_packed(
        target_rows.data_ptr(), rows_t, draft_rows.data_ptr() if rows_d else None, rows_d, dt,
        target_row_start.data_ptr(), draft_row_start.data_ptr(), draft_tokens.data_ptr(),
        lengths.data_ptr(), uniforms.data_ptr(), temperature.data_ptr(), B, k, V,
        out_tokens.data_ptr(), num_accepted.data_ptr(), workspace.data_ptr(),
        workspace.numel() * workspace.element_size(), _stream_ptr(stream),
        SPEC_FLAG_FULL_SWEEP if full_sweep else 0)
    _check(code, "spec_verify_packed")
    return out_tokens, num_accepted


class Verifier:
    """``spec_verify`` bound to one fixed set of device buffers.

    A serving loop verifies into the same buffers every round; this object
    checks their shapes, dtypes and devices once, at construction, and keeps
    the C call's argument tuple, so that each round costs the host one ctypes
    call (the Python checks of ``spec_verify`` cost more than a short round
    on the GPU).  The buffers' contents may change between calls; the
    tensors themselves must stay alive and keep their storage.
    """

    def __init__(self, target_logits, draft_logits, draft_tokens, lengths, uniforms, temperature,
                 *, workspace=None, out_tokens=None, num_accepted=None, stream=None,
                 full_sweep: bool = False):
        torch = _torch()
        B, k1, V = target_logits.shape
        k = k1 - 1
        dev = draft_tokens.device
        dt = _dtype_code(target_logits)
        _need_logits(target_logits, "target_logits", target_logits.dtype, (B, k + 1, V), dev)
        _need_logits(draft_logits, "draft_logits", target_logits.dtype, (B, k, V), dev)
        _need(draft_tokens, "draft_tokens", torch.int32, (B, k), dev)
        _need(lengths, "lengths", torch.int32, (B,), dev)
        _need(uniforms, "uniforms", torch.float32, (B, k + 1), dev)
        _need(temperature, "temperature", torch.float32, (B,), dev)
        if workspace is None:
            workspace = alloc_workspace(B, k, V, dev)
        if out_tokens is None:
            out_tokens = torch.empty((B, k + 1), dtype=torch.int32, device=dev)
        if num_accepted is None:
            num_accepted = torch.empty((B,), dtype=torch.int32, device=dev)
        _need(out_tokens, "out_tokens", torch.int32, (B, k + 1), dev)
        _need(num_accepted, "num_accepted", torch.int32, (B,), dev)
        # Keep every buffer referenced for as long as the bound call exists.
        self._keep = (target_logits, draft_logits, draft_tokens, lengths, uniforms, temperature,
                      workspace)
        self.workspace, self.out_tokens, self.num_accepted = workspace, out_tokens, num_accepted
        self._fn = lib().spec_verify_ex
        self._args = (target_logits.data_ptr(), draft_logits.data_ptr(), dt,
                      draft_tokens.data_ptr(), lengths.data_ptr(), uniforms.data_ptr(),
                      temperature.data_ptr(), B, k, V, out_tokens.data_ptr(),
                      num_accepted.data_ptr(), workspace.data_ptr(),
                      workspace.numel() * workspace.element_size(), _stream_ptr(stream),
                      SPEC_FLAG_FULL_SWEEP if full_sweep else 0)

    def __call__(self):
        """Enqueue one round on the bound stream; returns (out_tokens, num_accepted)."""
        code = self._fn(*self._args)
        if code != SPEC_OK:
            raise SpecVerifyError(code, "spec_verify")
        return self.out_tokens, self.num_accepted


def spec_verify_static(target_logits, draft_logits, draft_tokens, lengths, uniforms, temperature,
                       *, out_tokens=None, num_accepted=None, stream=None):
    """spec_verify for callers that cannot allocate: no workspace argument.

    The library uses its own fixed scratch array (SPEC_STATIC_SCRATCH_BYTES
    per GPU, held until exit) instead.  Calls that overlap on the GPU share it
    and race.  If ``out_tokens`` / ``num_accepted`` are given, this wrapper
    allocates nothing either.
    """
    torch = _torch()
    B, k1, V = target_logits.shape
    k = k1 - 1
    dev = draft_tokens.device
    dt = _dtype_code(target_logits)
    _need_logits(target_logits, "target_logits", target_logits.dtype, (B, k + 1, V), dev)
    _need_logits(draft_logits, "draft_logits", target_logits.dtype, (B, k, V), dev)
    _need(draft_tokens, "draft_tokens", torch.int32, (B, k), dev)
    _need(lengths, "lengths", torch.int32, (B,), dev)
    _need(uniforms, "uniforms", torch.float32, (B, k + 1), dev)
    _need(temperature, "temperature", torch.float32, (B,), dev)
    if out_tokens is None:
        out_tokens = torch.empty((B, k + 1), dtype=torch.int32, device=dev)
    if num_accepted is None:
        num_accepted = torch.empty((B,), dtype=torch.int32, device=dev)
    _need(out_tokens, "out_tokens", torch.int32, (B, k + 1), dev)
    _need(num_accepted, "num_accepted", torch.int32, (B,), dev)
    code = lib().spec_verify_static(
        target_logits.data_ptr(), draft_logits.data_ptr(), dt, draft_tokens.data_ptr(),
        lengths.data_ptr(), uniforms.data_ptr(), temperature.data_ptr(), B, k, V,
        out_tokens.data_ptr(), num_accepted.data_ptr(), _stream_ptr(stream))
    _check(code, "spec_verify_static")
    return out_tokens, num_accepted


def spec_verify_report(workspace, stream=None) -> Report:
    """Synchronise the stream and read what the last call on ``workspace`` recorded."""
    r = _Report()
    _check(lib().spec_verify_report(workspace.data_ptr(), _stream_ptr(stream), ctypes.byref(r)),
           "spec_verify_report")
    return Report(r.status, r.bad_requests, r.first_bad_request, r.rows_planned, r.chunks_swept,
                  r.chunks_per_row, r.chunk_elems, r.final_rows, r.residual_zero, r.sweep_bytes,
                  r.final_bytes)


def spec_verify_device_status(workspace, stream=None) -> int:
    return int(lib().spec_verify_device_status(workspace.data_ptr(), _stream_ptr(stream)))


def spec_row_stats(logits, temperature, *, stream=None):
    """Row sweep alone over [rows, V] logits: (max, natural-log logsumexp of z/T, argmax).

    ``lse`` is NaN for T == 0 rows; ``argmax`` is -1 for T > 0 rows.
    """
    torch = _torch()
    rows, V = logits.shape
    dev = temperature.device
    dt = _dtype_code(logits)
    _need_logits(logits, "logits", logits.dtype, (rows, V), dev)
    _need(temperature, "temperature", torch.float32, (rows,), dev)
    n = int(lib().spec_row_stats_workspace_bytes(rows, V))
    if n == 0:
        raise SpecVerifyError(SPEC_ERR_UNSUPPORTED, "spec_row_stats_workspace_bytes")
    ws = torch.empty(n, dtype=torch.uint8, device=dev)
    mx = torch.empty(rows, dtype=torch.float32, device=dev)
    lse = torch.empty(rows, dtype=torch.float32, device=dev)
    arg = torch.empty(rows, dtype=torch.int32, device=dev)
    _check(lib().spec_row_stats(logits.data_ptr(), dt, rows, V, temperature.data_ptr(),
                                mx.data_ptr(), lse.data_ptr(), arg.data_ptr(), ws.data_ptr(), n,
                                _stream_ptr(stream)), "spec_row_stats")
    return mx, lse, arg


def _logits_to_device(a, device):
    torch = _torch()
    import numpy as np
    if a.dtype == np.uint16:
        return torch.from_numpy(a.view(np.int16)).view(torch.bfloat16).to(device)
    return torch.from_numpy(a).to(device)


def to_device_packed(packed, device="cuda"):
    """Copy a ``synth.PackedRows`` layout to the device (the packed entry's row buffers)."""
    torch = _torch()
    return dict(target_rows=_logits_to_device(packed.target_rows, device),
                draft_rows=_logits_to_device(packed.draft_rows, device),
                target_row_start=torch.from_numpy(packed.target_row_start).to(device),
                draft_row_start=torch.from_numpy(packed.draft_row_start).to(device))


@dataclass
class OpdStats:
    x_star: object    # int32 [B, k]
    hard: object      # float32 [B, k]
    rkl: object       # float32 [B, k]
    rkl_clip: object  # float32 [B, k]
    loss: object      # float32 [B]


def spec_opd_stats(target_logits, draft_logits, lengths, *, delta: float = 0.01,
                   alpha: float = 0.8, out=None, stream=None) -> OpdStats:
    """OPD supervision statistics (AdaFlash Section 3.1) on the verification buffers.

    target [B, k+1, V], draft [B, k, V] (float32 or bfloat16), lengths int32 [B].
    Per verified position: target argmax, -log q(argmax), reverse KL and its
    entry-wise clipped form; per request the alpha mixture loss.  ``out`` may
    be an ``OpdStats`` of preallocated tensors.
    """
    torch = _torch()
    B, k1, V = target_logits.shape
    k = k1 - 1
    dev = lengths.device
    dt = _dtype_code(target_logits)
    # Host-resident logits reach the library, which refuses them.
    _need_logits(target_logits, "target_logits", target_logits.dtype, (B, k + 1, V), dev)
    _need_logits(draft_logits, "draft_logits", target_logits.dtype, (B, k, V), dev)
    _need(lengths, "lengths", torch.int32, (B,), dev)
    if out is None:
        f = dict(dtype=torch.float32, device=dev)
        out = OpdStats(torch.empty((B, k), dtype=torch.int32, device=dev), torch.empty((B, k), **f),
                       torch.empty((B, k), **f), torch.empty((B, k), **f), torch.empty(B, **f))
    _need(out.x_star, "x_star", torch.int32, (B, k), dev)
    for name in ("hard", "rkl", "rkl_clip"):
        _need(getattr(out, name), name, torch.float32, (B, k), dev)
    _need(out.loss, "loss", torch.float32, (B,), dev)
    _check(lib().spec_opd_stats(target_logits.data_ptr(), draft_logits.data_ptr(), dt,
                                lengths.data_ptr(), B, k, V, float(delta), float(alpha),
                                out.x_star.data_ptr(), out.hard.data_ptr(), out.rkl.data_ptr(),
                                out.rkl_clip.data_ptr(), out.loss.data_ptr(), _stream_ptr(stream)),
           "spec_opd_stats")
    return out


def spec_verify_opd(target_logits, draft_logits, draft_tokens, lengths, uniforms, temperature, *,
                    delta: float = 0.01, alpha: float = 0.8, workspace=None, out_tokens=None,
                    num_accepted=None, out=None, stream=None):
    """Verification and OPD statistics in one pass over the rows.

    Arguments as ``spec_verify`` plus ``delta`` and ``alpha`` as
    ``spec_opd_stats``; ``out`` may be an ``OpdStats`` of preallocated
    tensors.  Returns (out_tokens, num_accepted, OpdStats).
    """
    torch = _torch()
    B, k1, V = target_logits.shape
    k = k1 - 1
    dev = target_logits.device
    dt = _dtype_code(target_logits)
    _need(target_logits, "target_logits", target_logits.dtype, (B, k + 1, V), dev)
    _need(draft_logits, "draft_logits", target_logits.dtype, (B, k, V), dev)
    _need(draft_tokens, "draft_tokens", torch.int32, (B, k), dev)
    _need(lengths, "lengths", torch.int32, (B,), dev)
    _need(uniforms, "uniforms", torch.float32, (B, k + 1), dev)
    _need(temperature, "temperature", torch.float32, (B,), dev)
    if workspace is None:
        workspace = alloc_workspace(B, k, V, dev)
    if out_tokens is None:
        out_tokens = torch.empty((B, k + 1), dtype=torch.int32, device=dev)
    if num_accepted is None:
        num_accepted = torch.empty((B,), dtype=torch.int32, device=dev)
    _need(out_tokens, "out_tokens", torch.int32, (B, k + 1), dev)
    _need(num_accepted, "num_accepted", torch.int32, (B,), dev)
    if out is None:
        f = dict(dtype=torch.float32, device=dev)
        out = OpdStats(torch.empty((B, k), dtype=torch.int32, device=dev), torch.empty((B, k), **f),
                       torch.empty((B, k), **f), torch.empty((B, k), **f), torch.empty(B, **f))
    _need(out.x_star, "x_star", torch.int32, (B, k), dev)
    for name in ("hard", "rkl", "rkl_clip"):
        _need(getattr(out, name), name, torch.float32, (B, k), dev)
    _need(out.loss, "loss", torch.float32, (B,), dev)
    _check(lib().spec_verify_opd(
        target_logits.data_ptr(), draft_logits.data_ptr(), dt, draft_tokens.data_ptr(),
        lengths.data_ptr(), uniforms.data_ptr(), temperature.data_ptr(), B, k, V, float(delta),
        float(alpha), out_tokens.data_ptr(), num_accepted.data_ptr(), out.x_star.data_ptr(),
        out.hard.data_ptr(), out.rkl.data_ptr(), out.rkl_clip.data_ptr(), out.loss.data_ptr(),
        workspace.data_ptr(), workspace.numel() * workspace.element_size(), _stream_ptr(stream)),
        "spec_verify_opd")
    return out_tokens, num_accepted, out


def spec_d3d_select(num_accepted, out_tokens, branch_pos, branch_tok, branch_block, *,
                    hit=None, next_block=None, hits=None, stream=None):
    """D3D branch selection (D3D paper, Methodology, asynchronous inference).

    num_accepted int32 [B], out_tokens int32 [B, k+1] (spec_verify's outputs);
    branch_pos, branch_tok int32 [B, NB]; branch_block int32 [B, NB, blk].
    Returns (hit [B], next_block [B, blk], hits [1]) device tensors.
    """
    torch = _torch()
    B, k1 = out_tokens.shape
    NB, blk = branch_block.shape[1], branch_block.shape[2]
    dev = out_tokens.device
    i32 = torch.int32
    _need(num_accepted, "num_accepted", i32, (B,), dev)
    _need(out_tokens, "out_tokens", i32, (B, k1), dev)
    _need(branch_pos, "branch_pos", i32, (B, NB), dev)
    _need(branch_tok, "branch_tok", i32, (B, NB), dev)
    _need(branch_block, "branch_block", i32, (B, NB, blk), dev)
    if hit is None:
        hit = torch.empty(B, dtype=i32, device=dev)
    if next_block is None:
        next_block = torch.empty((B, blk), dtype=i32, device=dev)
    if hits is None:
        hits = torch.empty(1, dtype=i32, device=dev)
    _need(hit, "hit", i32, (B,), dev)
    _need(next_block, "next_block", i32, (B, blk), dev)
    _need(hits, "hits", i32, (1,), dev)
    _check(lib().spec_d3d_select(num_accepted.data_ptr(), out_tokens.data_ptr(),
                                 branch_pos.data_ptr(), branch_tok.data_ptr(),
                                 branch_block.data_ptr(), B, k1 - 1, NB, blk, hit.data_ptr(),
                                 next_block.data_ptr(), hits.data_ptr(), _stream_ptr(stream)),
           "spec_d3d_select")
    return hit, next_block, hits


def _stream_on(stream, device) -> int:
    """The given stream, or the current one of the tensors' own device."""
    if stream is None:
        # The handle alone: making a torch.cuda.Stream costs as much as the C call.
        return _torch()._C._cuda_getCurrentRawStream(device.index)
    return _stream_ptr(stream)


def _alloc_on(stream, device):
    """Context in which a call's own tensors are allocated: on the stream that uses them.

    The caching allocator hands a freed tensor's memory out again in the order of the
    stream it was allocated on; a workspace of the current stream's, freed when the call
    returns, could be in other hands while another stream still works in it.
    """
    if stream is None:
        return contextlib.nullcontext()
    cuda = _torch().cuda
    if not hasattr(stream, "cuda_stream"):
        # (An external stream of handle 0 would be a new one.)
        stream = cuda.ExternalStream(int(stream), device=device) if int(stream) else \
            cuda.default_stream(device)
    return cuda.stream(stream)


def _need_cuda(t, name):
    if t.device.type != "cuda":
        raise ValueError(f"{name} is on {t.device}, expected a CUDA device")


def _need_workspace(ws, name, nbytes, device, stream):
    torch = _torch()
    if ws is None:
        with _alloc_on(stream, device):
            return torch.empty(nbytes, dtype=torch.uint8, device=device)
    if ws.device != device:
        raise ValueError(f"{name} is on {ws.device}, expected {device}")
    if not ws.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return ws


class LinearCe:
    """Cross entropy of a linear vocabulary head and its gradients, bound to fixed buffers.

    ``hidden`` [N, D] and ``weight`` [V, D] bfloat16, ``labels`` int32 [N]
    (negative: no label), ``grad_nll`` float32 [N] (the loss's derivative by
    each token's nll; needed for ``grad``).  Like ``Verifier``, the object
    checks its buffers once and keeps the C calls' arguments; the buffers'
    contents may change between calls, the tensors must stay alive.

    ``loss()`` fills and returns (nll, lse), ``grad()`` (d_hidden, d_weight)
    from the nll and lse of the last ``loss()``, or from those that the caller
    gave with both buffers; without either it is refused.  ``need_hidden`` / ``need_weight``
    False leaves that gradient out (None).  Both calls share one workspace:
    enqueue them on one stream.
    """

    def __init__(self, hidden, weight, labels, grad_nll=None, *, nll=None, lse=None, d_hidden=None,
                 d_weight=None, need_hidden: bool = True, need_weight: bool = True, workspace=None,
                 stream=None):
        torch = _torch()
        N, D = hidden.shape
        V = weight.shape[0]
        dev = hidden.device
        _need_cuda(hidden, "hidden")
        dt = _dtype_code(hidden)
        _need(hidden, "hidden", hidden.dtype, (N, D), dev)
        _need(weight, "weight", hidden.dtype, (V, D), dev)
        _need(labels, "labels", torch.int32, (N,), dev)
        # Whether grad() has a loss to start from: another call's, or loss() sets it.
        self._filled = nll is not None and lse is not None
        with _alloc_on(stream, dev):
            if nll is None:
                nll = torch.empty(N, dtype=torch.float32, device=dev)
            if lse is None:
                lse = torch.empty(N, dtype=torch.float32, device=dev)
        _need(nll, "nll", torch.float32, (N,), dev)
        _need(lse, "lse", torch.float32, (N,), dev)
        n = int(lib().spec_linear_ce_workspace_bytes(N, V, D))
        if grad_nll is not None:
            _need(grad_nll, "grad_nll", torch.float32, (N,), dev)
            n = max(n, int(lib().spec_linear_ce_grad_workspace_bytes(N, V, D)))
            if not (need_hidden or need_weight):
                raise ValueError("grad_nll is given, but neither gradient is wanted")
            with _alloc_on(stream, dev):
                if need_hidden and d_hidden is None:
                    d_hidden = torch.empty_like(hidden)
                if need_weight and d_weight is None:
                    d_weight = torch.empty_like(weight)
            if need_hidden:
                _need(d_hidden, "d_hidden", hidden.dtype, (N, D), dev)
            if need_weight:
                _need(d_weight, "d_weight", hidden.dtype, (V, D), dev)
        # Unsupported sizes (n == 0) reach the library, which says so.
        ws = _need_workspace(workspace, "workspace", max(n, 256), dev, stream)
        self._keep = (hidden, weight, labels, grad_nll, ws)
        self.workspace, self.nll, self.lse = ws, nll, lse
        self.d_hidden = d_hidden if grad_nll is not None and need_hidden else None
        self.d_weight = d_weight if grad_nll is not None and need_weight else None
        st = _stream_on(stream, dev)
        wsb = ws.numel() * ws.element_size()
        self._loss = lib().spec_linear_ce
        self._loss_args = (hidden.data_ptr(), weight.data_ptr(), dt, labels.data_ptr(), N, V, D,
                           nll.data_ptr(), lse.data_ptr(), ws.data_ptr(), wsb, st)
        self._grad = lib().spec_linear_ce_grad
        self._grad_args = None if grad_nll is None else (
            hidden.data_ptr(), weight.data_ptr(), dt, labels.data_ptr(), nll.data_ptr(),
            lse.data_ptr(), grad_nll.data_ptr(), N, V, D,
            None if self.d_hidden is None else d_hidden.data_ptr(),
            None if self.d_weight is None else d_weight.data_ptr(), ws.data_ptr(), wsb, st)

    def loss(self):
        """Enqueue the loss; returns (nll, lse)."""
        _check(self._loss(*self._loss_args), "spec_linear_ce")
        self._filled = True
        return self.nll, self.lse

    def grad(self):
        """Enqueue the gradients; returns (d_hidden, d_weight)."""
        if self._grad_args is None:
            raise ValueError("LinearCe was made without grad_nll")
        if not self._filled:
            raise ValueError("grad() needs nll and lse: call loss() first, or give both buffers")
        _check(self._grad(*self._grad_args), "spec_linear_ce_grad")
        return self.d_hidden, self.d_weight


def spec_linear_ce(hidden, weight, labels, *, nll=None, lse=None, workspace=None, stream=None):
    """Token losses of a linear vocabulary head, without keeping the logits.

    hidden [N, D], weight [V, D] bfloat16 (D a multiple of 8), labels int32
    [N] (negative: no label, nll 0).  Returns (nll, lse), float32 [N]:
    lse_i = logsumexp_v(hidden_i . weight_v), nll_i = lse_i - hidden_i .
    weight_{labels_i}.
    """
    return LinearCe(hidden, weight, labels, nll=nll, lse=lse, workspace=workspace,
                    stream=stream).loss()


def spec_linear_ce_grad(hidden, weight, labels, nll, lse, grad_nll, *, d_hidden=None, d_weight=None,
                        need_hidden: bool = True, need_weight: bool = True, workspace=None,
                        stream=None):
    """Gradients of sum_i grad_nll_i nll_i: (d_hidden [N, D], d_weight [V, D]), bfloat16.

    ``nll`` and ``lse`` are ``spec_linear_ce``'s on the same inputs; ``grad_nll`` float32 [N].
    ``need_hidden`` / ``need_weight`` False leaves that gradient out (None).
    """
    if nll is None or lse is None:
        raise ValueError("spec_linear_ce_grad needs spec_linear_ce's nll and lse")
    return LinearCe(hidden, weight, labels, grad_nll, nll=nll, lse=lse, d_hidden=d_hidden,
                    d_weight=d_weight, need_hidden=need_hidden, need_weight=need_weight,
                    workspace=workspace, stream=stream).grad()


def spec_opd_grad(target_logits, draft_logits, lengths, grad_loss, *, delta: float = 0.01,
                  alpha: float = 0.8, d_draft=None, stream=None):
    """Gradient of sum_b grad_loss_b loss_b with respect to the draft logits.

    loss is ``spec_opd_stats``'s mixture loss; target [B, k+1, V], draft [B, k, V]
    (float32 or bfloat16), lengths int32 [B], grad_loss float32 [B].  Returns
    ``d_draft`` [B, k, V] of the logits' dtype, 0 past each request's length.
    """
    torch = _torch()
    B, k1, V = target_logits.shape
    k = k1 - 1
    dev = lengths.device
    dt = _dtype_code(target_logits)
    # Host-resident logits reach the library, which refuses them.
    _need_logits(target_logits, "target_logits", target_logits.dtype, (B, k + 1, V), dev)
    _need_logits(draft_logits, "draft_logits", target_logits.dtype, (B, k, V), dev)
    _need_cuda(lengths, "lengths")
    _need(lengths, "lengths", torch.int32, (B,), dev)
    _need(grad_loss, "grad_loss", torch.float32, (B,), dev)
    if d_draft is None:
        with _alloc_on(stream, dev):
            d_draft = torch.empty((B, k, V), dtype=target_logits.dtype, device=dev)
    _need(d_draft, "d_draft", target_logits.dtype, (B, k, V), dev)
    _check(lib().spec_opd_grad(target_logits.data_ptr(), draft_logits.data_ptr(), dt,
                               lengths.data_ptr(), grad_loss.data_ptr(), B, k, V, float(delta),
                               float(alpha), d_draft.data_ptr(), _stream_on(stream, dev)),
           "spec_opd_grad")
    return d_draft


class GradClipper:
    """``spec_clip_grad_norm`` bound to one fixed set of gradient tensors.

    ``grads``: contiguous float32 / bfloat16 tensors of one device, any shapes;
    ``out``: tensors of the same shapes and types for the results, or None to
    scale in place; ``max_norm`` None only takes the norm.  Calling the object
    enqueues the clip and returns ``norm`` (float32 [1], on the device).
    """

    def __init__(self, grads, max_norm, *, out=None, norm=None, workspace=None, stream=None):
        torch = _torch()
        grads = list(grads)
        if not grads:
            raise ValueError("grads is empty")
        out = None if out is None else list(out)
        if out is not None and (max_norm is None or len(out) != len(grads)):
            raise ValueError("out has one tensor for each of grads, and needs a max_norm")
        dev = grads[0].device
        _need_cuda(grads[0], "grads[0]")
        for i, g in enumerate(grads):
            _need(g, f"grads[{i}]", g.dtype, g.shape, dev)
            if out is not None:
                _need(out[i], f"out[{i}]", g.dtype, g.shape, dev)
        if norm is None:
            with _alloc_on(stream, dev):
                norm = torch.empty(1, dtype=torch.float32, device=dev)
        _need(norm, "norm", torch.float32, (1,), dev)
        m = len(grads)
        n = int(lib().spec_grad_norm_workspace_bytes(m))
        ws = _need_workspace(workspace, "workspace", max(n, 256), dev, stream)
        self._keep = (grads, out, ws)
        self.norm, self.workspace = norm, ws
        ptrs = (ctypes.c_void_p * m)(*[g.data_ptr() or None for g in grads])
        outs = None if out is None else (ctypes.c_void_p * m)(*[t.data_ptr() or None for t in out])
        sizes = (ctypes.c_longlong * m)(*[g.numel() for g in grads])
        codes = (ctypes.c_int * m)(*[_dtype_code(g) for g in grads])
        tail = (norm.data_ptr(), ws.data_ptr(), ws.numel() * ws.element_size(),
                _stream_on(stream, dev))
        if max_norm is None:
            self._fn, self._name = lib().spec_grad_norm, "spec_grad_norm"
            self._args = (ptrs, sizes, codes, m) + tail
        else:
            self._fn, self._name = lib().spec_clip_grad_norm, "spec_clip_grad_norm"
            self._args = (ptrs, outs, sizes, codes, m, float(max_norm)) + tail

    def __call__(self):
        """Enqueue on the bound stream; returns the norm before clipping."""
        _check(self._fn(*self._args), self._name)
        return self.norm


def spec_grad_norm(grads, *, norm=None, workspace=None, stream=None):
    """Global norm sqrt(sum x^2) over all entries of ``grads`` (float32 [1], on the device)."""
    return GradClipper(grads, None, norm=norm, workspace=workspace, stream=stream)()


def spec_clip_grad_norm(grads, max_norm, *, out=None, norm=None, workspace=None, stream=None):
    """Scale ``grads`` by min(1, max_norm / norm), in place or into ``out``; returns the norm.

    A norm that is infinite or NaN (because an entry is) leaves every value as it is.
    """
    return GradClipper(grads, max_norm, out=out, norm=norm, workspace=workspace,
                       stream=stream)()


class Sampler:
    """Truncated sampling bound to fixed buffers.

    ``logits`` [B, n, V] or [B, V] (float32 or bfloat16), one set of settings per request:
    ``temperature`` float32 [B] (0: greedy), ``top_k`` int32 [B] (0: off), ``top_p`` float32
    [B] (1: off), ``min_p`` float32 [B] (0: off); None leaves a setting off.  ``uniforms``
    float32 [B, n] or [B].  Like ``Verifier``, the object checks its buffers once; their
    contents may change between calls, the tensors must stay alive.

    ``sample()`` fills and returns ``tokens`` (int32, the shape of ``uniforms``); where
    ``kept`` was given it writes the truncated logits as well.  ``truncate()`` only writes
    and returns them (``kept``; made on the first call if None, ``logits`` itself truncates
    in place).
    """

    def __init__(self, logits, temperature, uniforms=None, *, top_k=None, top_p=None, min_p=None,
                 tokens=None, kept=None, stream=None):
        torch = _torch()
        if logits.dim() not in (2, 3):
            raise ValueError(f"logits must have shape [B, n, V] or [B, V], got {tuple(logits.shape)}")
        shape, V = tuple(logits.shape[:-1]), logits.shape[-1]
        B, n = shape[0], shape[1] if len(shape) == 2 else 1
        dev = logits.device
        _need_cuda(logits, "logits")
        dt = _dtype_code(logits)
        _need(logits, "logits", logits.dtype, shape + (V,), dev)
        _need(temperature, "temperature", torch.float32, (B,), dev)
        for name, t, dtype in (("top_k", top_k, torch.int32), ("top_p", top_p, torch.float32),
                               ("min_p", min_p, torch.float32)):
            if t is not None:
                _need(t, name, dtype, (B,), dev)
        if uniforms is not None:
            _need(uniforms, "uniforms", torch.float32, shape, dev)
            if tokens is None:
                with _alloc_on(stream, dev):
                    tokens = torch.empty(shape, dtype=torch.int32, device=dev)
            _need(tokens, "tokens", torch.int32, shape, dev)
        if kept is not None:
            _need(kept, "kept", logits.dtype, shape + (V,), dev)
        self._keep = (logits, temperature, uniforms, top_k, top_p, min_p)
        self.tokens, self.kept = tokens if uniforms is not None else None, kept
        self._head = (logits.data_ptr(), dt, B * n, V, n, temperature.data_ptr(),
                      *(None if t is None else t.data_ptr() for t in (top_k, top_p, min_p)))
        self._st = _stream_on(stream, dev)
        self._sample, self._truncate = lib().spec_sample, lib().spec_truncate
        self._bind()

    def _bind(self):
        kept = None if self.kept is None else self.kept.data_ptr()
        uniforms = self._keep[2]
        self._sample_args = None if uniforms is None else self._head + (
            uniforms.data_ptr(), self.tokens.data_ptr(), kept, self._st)
        self._truncate_args = None if kept is None else self._head + (kept, self._st)

    def sample(self):
        """Enqueue the draw; returns the tokens, or (tokens, kept) where ``kept`` was given."""
        if self._sample_args is None:
            raise ValueError("Sampler was made without uniforms")
        _check(self._sample(*self._sample_args), "spec_sample")
        return self.tokens if self._sample_args[-2] is None else (self.tokens, self.kept)

    def truncate(self):
        """Enqueue the truncation; returns the truncated logits."""
        if self._truncate_args is None:
            logits = self._keep[0]
            # (On the stream that the object is bound to, whichever is current by now.)
            with _alloc_on(self._st, logits.device):
                self.kept = _torch().empty_like(logits)
            self._truncate_args = self._head + (self.kept.data_ptr(), self._st)
        _check(self._truncate(*self._truncate_args), "spec_truncate")
        return self.kept


def spec_sample(logits, temperature, uniforms, *, top_k=None, top_p=None, min_p=None, tokens=None,
                kept=None, stream=None):
    """Tokens drawn by inverse CDF under temperature, top-k, top-p and min-p.

    Arguments as ``Sampler``.  Returns int32 tokens of ``uniforms``' shape (-1 where a
    request's settings or a row are invalid), with ``kept`` also the truncated logits.
    """
    if uniforms is None:
        raise ValueError("spec_sample needs uniforms (spec_truncate does not)")
    return Sampler(logits, temperature, uniforms, top_k=top_k, top_p=top_p, min_p=min_p,
                   tokens=tokens, kept=kept, stream=stream).sample()


def spec_truncate(logits, temperature, *, top_k=None, top_p=None, min_p=None, kept=None,
                  stream=None):
    """The logits that truncated sampling may draw, -inf elsewhere (NaN rows: invalid).

    Target and draft rows truncated with their requests' settings make ``spec_verify``
    lossless for truncated sampling.  ``kept`` may be ``logits`` itself (in place).
    """
    return Sampler(logits, temperature, top_k=top_k, top_p=top_p, min_p=min_p, kept=kept,
                   stream=stream).truncate()


def _need_rows(t, name, dtype, shape, device):
    """Rows of heads, contiguous within a row; rows may lie apart (a slice of a fused
    projection, say)."""
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if t.stride(2) != 1 or (shape[1] > 1 and t.stride(1) != shape[2]):
        raise ValueError(f"{name} must be contiguous within a row")


class PagedCache:
    """A paged key-value cache, a batch's new tokens, and the calls on them, bound to fixed buffers.

    ``k_cache``, ``v_cache`` [pages, page_size, kv_heads, width] bfloat16, any strides with
    contiguous heads (a permuted [pages, kv_heads, page_size, width] too); ``page_table``
    int32 [B, max_pages]; ``new_start`` int32 [B + 1], request b's new tokens being rows
    new_start[b] .. new_start[b + 1] - 1 of the batch; ``kv_len`` int32 [B], its entries
    with the new ones, which are the last.

    ``append()`` writes ``k_new``, ``v_new`` [rows, kv_heads, width] into the pages and
    returns the caches.  ``attend()`` is the attention of ``q`` [rows, heads, width] over
    them; returns ``out`` (bfloat16, as ``q``), with ``need_lse`` (out, lse float32
    [rows, heads]).  ``causal`` False lets a request's new tokens see each other;
    ``window`` > 0 is the number of entries a token sees; ``scale`` None is
    1 / sqrt(width).  Like ``Verifier``, the object checks its buffers once; their contents
    may change between calls, the tensors must stay alive.
    """

    def __init__(self, k_cache, v_cache, page_table, new_start, kv_len, *, k_new=None, v_new=None,
                 q=None, causal: bool = True, window: int = 0, scale=None, out=None, lse=None,
                 need_lse: bool = False, workspace=None, stream=None):
        torch = _torch()
        if k_cache.dim() != 4:
            raise ValueError("k_cache must have shape [pages, page_size, kv_heads, width], got "
                             f"{tuple(k_cache.shape)}")
        pages, P, Hk, D = k_cache.shape
        dev = k_cache.device
        _need_cuda(k_cache, "k_cache")
        dt = _dtype_code(k_cache)
        for name, t in (("k_cache", k_cache), ("v_cache", v_cache)):
            if t.dtype != k_cache.dtype:
                raise TypeError(f"{name} must be {k_cache.dtype}, got {t.dtype}")
            if t.shape != k_cache.shape:
                raise ValueError(f"{name} must have shape {tuple(k_cache.shape)}, got "
                                 f"{tuple(t.shape)}")
            if t.device != dev:
                raise ValueError(f"{name} is on {t.device}, expected {dev}")
            if t.stride(3) != 1:
                raise ValueError(f"{name} must be contiguous within a head")
        B, i32 = kv_len.shape[0], torch.int32
        _need(kv_len, "kv_len", i32, (B,), dev)
        _need(new_start, "new_start", i32, (B + 1,), dev)
        _need(page_table, "page_table", i32, (B, page_table.shape[-1]), dev)
        self._keep = (k_cache, v_cache, page_table, new_start, kv_len, k_new, v_new, q)
        self.k_cache, self.v_cache = k_cache, v_cache
        self._c = _PagedCache(k_cache.data_ptr(), v_cache.data_ptr(), *k_cache.stride()[:3],
                              *v_cache.stride()[:3], pages, P, Hk, D, page_table.data_ptr(),
                              page_table.shape[1], new_start.data_ptr(), kv_len.data_ptr(), B)
        c = ctypes.addressof(self._c)
        st = _stream_on(stream, dev)
        self._append_args = self._attend_args = None
        if (k_new is None) != (v_new is None):
            raise ValueError("k_new and v_new are given together")
        if k_new is not None:
            rows = k_new.shape[0]
            _need_rows(k_new, "k_new", k_cache.dtype, (rows, Hk, D), dev)
            _need_rows(v_new, "v_new", k_cache.dtype, (rows, Hk, D), dev)
            self._append = lib().spec_kv_append
            self._append_args = (c, dt, k_new.data_ptr(), v_new.data_ptr(), rows, k_new.stride(0),
                                 v_new.stride(0), st)
        self.out = self.lse = self.workspace = None
        if q is not None:
            rows, H = q.shape[:2]
            _need_rows(q, "q", k_cache.dtype, (rows, H, D), dev)
            with _alloc_on(stream, dev):
                if out is None:
                    out = torch.empty((rows, H, D), dtype=q.dtype, device=dev)
                if lse is None and need_lse:
                    lse = torch.empty((rows, H), dtype=torch.float32, device=dev)
            _need(out, "out", q.dtype, (rows, H, D), dev)
            if lse is not None:
                _need(lse, "lse", torch.float32, (rows, H), dev)
            n = int(lib().spec_paged_attention_workspace_bytes(rows, H, Hk, D))
            # Unsupported sizes (n == 0) reach the library, which says so.
            ws = _need_workspace(workspace, "workspace", max(n, 256), dev, stream)
            self.out, self.lse, self.workspace = out, lse, ws
            self._attend = lib().spec_paged_attention
            # (A C int: of a larger number it would get the lower bits.)
            window = max(-1, min(int(window), 2 ** 31 - 1))
            self._attend_args = (c, dt, q.data_ptr(), rows, H, q.stride(0), int(causal), window,
                                 D ** -0.5 if scale is None else float(scale), out.data_ptr(),
                                 None if lse is None else lse.data_ptr(), ws.data_ptr(),
                                 ws.numel() * ws.element_size(), st)

    def append(self):
        """Enqueue the writes of the new keys and values; returns (k_cache, v_cache)."""
        if self._append_args is None:
            raise ValueError("PagedCache was made without k_new and v_new")
        _check(self._append(*self._append_args), "spec_kv_append")
        return self.k_cache, self.v_cache

    def attend(self):
        """Enqueue the attention; returns out, or (out, lse) where lse is wanted."""
        if self._attend_args is None:
            raise ValueError("PagedCache was made without q")
        _check(self._attend(*self._attend_args), "spec_paged_attention")
        return self.out if self.lse is None else (self.out, self.lse)


def spec_kv_append(k_new, v_new, k_cache, v_cache, page_table, new_start, kv_len, *, stream=None):
    """Write new tokens' keys and values into their pages; returns (k_cache, v_cache).

    Arguments as ``PagedCache``.
    """
    if k_new is None or v_new is None:
        raise ValueError("spec_kv_append needs k_new and v_new")
    return PagedCache(k_cache, v_cache, page_table, new_start, kv_len, k_new=k_new, v_new=v_new,
                      stream=stream).append()


def spec_paged_attention(q, k_cache, v_cache, page_table, new_start, kv_len, *,
                         causal: bool = True, window: int = 0, scale=None, out=None, lse=None,
                         need_lse: bool = False, workspace=None, stream=None):
    """Attention of new tokens over a paged cache that holds their own entries already.

    Arguments as ``PagedCache``.  Returns out, or (out, lse) with ``need_lse`` or ``lse``.
    """
    if q is None:
        raise ValueError("spec_paged_attention needs q")
    return PagedCache(k_cache, v_cache, page_table, new_start, kv_len, q=q, causal=causal,
                      window=window, scale=scale, out=out, lse=lse, need_lse=need_lse,
                      workspace=workspace, stream=stream).attend()


def to_device(inputs, device="cuda"):
    """Copy a ``synth.SpecInputs`` batch to the device as the C-ABI's buffers."""
    torch = _torch()
    import numpy as np
    if inputs.dtype == "bf16":
        t = torch.from_numpy(inputs.target.view(np.int16)).view(torch.bfloat16)
        d = torch.from_numpy(inputs.draft.view(np.int16)).view(torch.bfloat16)
    else:
        t = torch.from_numpy(inputs.target)
        d = torch.from_numpy(inputs.draft)
    return dict(
        target_logits=t.to(device), draft_logits=d.to(device),
        draft_tokens=torch.from_numpy(inputs.tokens).to(device),
        lengths=torch.from_numpy(inputs.lengths).to(device),
        uniforms=torch.from_numpy(inputs.uniforms).to(device),
        temperature=torch.from_numpy(inputs.temperature).to(device))
