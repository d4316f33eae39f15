"""ctypes binding of libmsa (include/msa.h), with the same names.

Argument marshalling only: every step of the MSA hot path runs in the CUDA
kernels of ``libmsa.so``.  Tensor arguments may be torch tensors (their
device pointer is passed; shapes are checked against the sizes given) or raw
integer device addresses.  ``stream`` defaults to torch's current stream on
the current device.  A non-zero status raises ``MsaError``; the library must
have been built (``python -m latent_memory_routing_b200.build``) -- there is
no fallback.

With ``MSA_DEBUG=1`` in the environment the binding loads
``libmsa_debug.so`` (``python -m latent_memory_routing_b200.build --debug``)
instead: the same kernels, with every call first checking the device-side
index arrays it is given and then waiting for its own work, so that a
device-detected error is raised by the call that caused it.
"""

from __future__ import annotations

import ctypes
import os
import re

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "libmsa_debug.so" if os.environ.get("MSA_DEBUG") == "1"
                         else "libmsa.so")
HEADER = os.path.join(os.path.dirname(PKG), "include", "msa.h")

MSA_F32 = 0
MSA_BF16 = 1

_STATUS = {0: "MSA_OK", -1: "MSA_ERR_INVALID_ARG", -2: "MSA_ERR_UNSUPPORTED",
           -3: "MSA_ERR_CAPACITY", -4: "MSA_ERR_CUDA", -5: "MSA_ERR_TIMEOUT",
           -6: "MSA_ERR_WORKSPACE"}


class MsaError(RuntimeError):
    def __init__(self, fn: str, status: int, detail: str = ""):
        self.status = status
        super().__init__(f"{fn} -> {_STATUS.get(status, status)}"
                         + (f" ({detail})" if detail else ""))


_lib = None

c_i = ctypes.c_int
c_i64 = ctypes.c_int64
c_f = ctypes.c_float
c_sz = ctypes.c_size_t
c_p = ctypes.c_void_p

_SIGS = {
    "msa_status_string": (ctypes.c_char_p, [c_i]),
    "msa_last_cuda_error": (c_i, []),
    "msa_version": (ctypes.c_char_p, []),
    "msa_device_status": (c_i, [c_p, c_i, c_p]),
    "msa_check_bounded_wait": (c_i, [c_i64, c_i, c_p]),
    "msa_chunk_offsets": (c_i, [c_i, c_p, c_i, c_p, c_p]),
    "msa_encode_pool": (c_i, [c_i, c_i, c_i64, c_i, c_i, c_i, c_p, c_p, c_p, c_p, c_p,
                              c_i64, c_f, c_i, c_p, c_p, c_p, c_p]),
    "msa_encode_pool_prepared": (c_i, [c_i, c_i, c_i64, c_i, c_i, c_i, c_p, c_p, c_p, c_p, c_p,
                                       c_i64, c_f, c_i, c_p, c_p, c_p, c_p, c_p]),
    "msa_route_workspace_size": (c_sz, [c_i, c_i, c_i, c_i, c_i]),
    "msa_route_scores": (c_i, [c_i, c_i, c_i, c_i, c_i, c_p, c_p, c_i64, c_p, c_i, c_p, c_p,
                               c_p, c_sz, c_p]),
    "msa_route_prepare_bank": (c_i, [c_i, c_i64, c_i, c_i, c_p, c_p, c_p]),
    "msa_route_scores_prepared": (c_i, [c_i, c_i, c_i, c_i, c_i, c_p, c_p, c_i64, c_p, c_i, c_p,
                                        c_p, c_p, c_sz, c_p]),
    "msa_route_noalloc_scratch_bytes": (c_sz, []),
    "msa_route_scores_noalloc": (c_i, [c_i, c_i, c_i, c_i, c_i, c_p, c_p, c_i64, c_p, c_i, c_p,
                                       c_p, c_p]),
    "msa_topk_workspace_size": (c_sz, [c_i, c_i, c_i]),
    "msa_topk_docs": (c_i, [c_i, c_i, c_i, c_p, c_p, c_p, c_p, c_sz, c_p]),
    "msa_topk_merge_shards": (c_i, [c_i, c_i, c_i, c_p, c_p, c_p, c_p, c_p, c_p]),
    "msa_gather_kv": (c_i, [c_i, c_i, c_i, c_i, c_i, c_p, c_p, c_i, c_p, c_p, c_i, c_p, c_p,
                            c_p, c_p]),
    "msa_sparse_attn_workspace_size": (c_sz, [c_i, c_i, c_i, c_i, c_i, c_i, c_i, c_i]),
    "msa_sparse_attn_fused_workspace_size": (c_sz, [c_i] * 9),
    "msa_route_backward_workspace_size": (c_sz, [c_i, c_i, c_i, c_i, c_i, c_i64, c_i]),
    "msa_route_backward": (c_i, [c_i, c_i, c_i, c_i, c_i, c_p, c_p, c_i64, c_p, c_i, c_p, c_p,
                                 c_p, c_p, c_sz, c_p]),
    "msa_encode_pool_backward": (c_i, [c_i, c_i64, c_i, c_i, c_i, c_p, c_p, c_p, c_p, c_p,
                                       c_i64, c_f, c_p, c_p, c_p, c_p]),
    "msa_sparse_attn_fused": (c_i, [c_i, c_i, c_i, c_i, c_i, c_i, c_i, c_p, c_p, c_i, c_p, c_i,
                                    c_p, c_p, c_i64, c_i, c_p, c_p, c_i, c_f, c_f, c_p, c_p,
                                    c_p, c_sz, c_p]),
    "msa_sparse_attn": (c_i, [c_i, c_i, c_i, c_i, c_i, c_i, c_i, c_p, c_p, c_p, c_p, c_i, c_p,
                              c_p, c_i, c_f, c_f, c_p, c_p, c_sz, c_p]),
    "msa_qk_norm_rope": (c_i, [c_i, c_i64, c_i, c_i, c_i, c_p, c_i64, c_p, c_i64, c_p, c_p, c_p,
                               c_f, c_f, c_p, c_p, c_p]),
    "msa_qk_norm_rope_backward_workspace_size": (c_sz, [c_i64, c_i]),
    "msa_qk_norm_rope_backward": (c_i, [c_i, c_i, c_i64, c_i, c_i, c_i, c_p, c_i64, c_p, c_i64,
                                        c_p, c_p, c_p, c_f, c_f, c_p, c_p, c_p, c_i64, c_p, c_i64,
                                        c_p, c_p, c_p, c_sz, c_p]),
    "msa_paged_append": (c_i, [c_i, c_i, c_i64, c_i, c_i, c_i, c_p, c_i64, c_p, c_i64, c_p, c_i64,
                               c_p, c_p, c_p, c_p, c_f, c_f, c_p, c_i, c_p, c_i, c_i, c_p, c_p,
                               c_p, c_p]),
    "msa_tree_attn_workspace_size": (c_sz, [c_i] * 9),
    "msa_tree_attn": (c_i, [c_i, c_i, c_i64, c_i, c_i, c_i, c_i, c_p, c_p, c_p, c_p, c_p, c_p, c_i,
                            c_p, c_p, c_i, c_i, c_p, c_i, c_p, c_f, c_p, c_p, c_sz, c_p]),
}


def header_symbols(path: str = HEADER) -> list[str]:
    """Function names declared in include/msa.h."""
    with open(path, encoding="utf-8") as f:
        text = re.sub(r"/\*.*?\*/", "", f.read(), flags=re.S)
    return sorted(set(re.findall(r"\b(msa_[a-z0-9_]+)\s*\(", text)))


def lib(path: str = LIB_PATH) -> ctypes.CDLL:
    """Loads libmsa.so (once) and declares every signature."""
    global _lib
    if _lib is None:
        if not os.path.exists(path):
            raise ImportError(f"{path} is missing: build it with "
                              "`python -m latent_memory_routing_b200.build`")
        handle = ctypes.CDLL(path)
        for name, (res, args) in _SIGS.items():
            fn = getattr(handle, name)
            fn.restype = res
            fn.argtypes = args
        _lib = handle
    return _lib


def _ptr(x) -> int | None:
    if x is None:
        return None
    if isinstance(x, int):
        return x
    return x.data_ptr()


_torch = None


def _th():
    """torch, imported with the first call that needs it (the checks below run
    several times a call, and a small call's time is theirs)."""
    global _torch
    if _torch is None:
        import torch
        _torch = torch
    return _torch


def _device() -> int:
    """The current CUDA device, without torch's checks for an uninitialised
    CUDA (-2, no tensor's device, where there is none)."""
    try:
        return _th()._C._cuda_getDevice()
    except (AttributeError, RuntimeError):
        return -2


def _stream(stream) -> int | None:
    if stream is None:
        torch = _th()
        raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        if raw is None:
            return torch.cuda.current_stream().cuda_stream
        return raw(torch._C._cuda_getDevice())  # the same handle, 3 us sooner
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def dtype_code(t) -> int:
    torch = _th()
    if t == torch.float32:
        return MSA_F32
    if t == torch.bfloat16:
        return MSA_BF16
    raise ValueError(f"unsupported dtype {t}")


def _check(name: str, rc: int):
    if rc != 0:
        detail = ""
        if rc == -4:
            detail = f"cudaError {lib().msa_last_cuda_error()}"
        raise MsaError(name, rc, detail)


# Element type of each tensor argument: the call's `dt` for floating-point
# tensors, and these fixed types for the rest.
F32, I32, I64 = "f32", "i32", "i64"


_DTYPES: dict = {}


def _torch_dtype(kind):
    if not _DTYPES:
        torch = _th()
        _DTYPES.update({MSA_F32: torch.float32, MSA_BF16: torch.bfloat16, F32: torch.float32,
                        I32: torch.int32, I64: torch.int64})
    return _DTYPES.get(kind)


def _es(dt):
    """The element type of a `dt`-typed tensor (None for an unknown dt, which
    the library itself rejects)."""
    return dt if dt in (MSA_F32, MSA_BF16) else None


def _device_ok(t, host_ok: bool) -> bool:
    """A tensor the kernels may read: on the current CUDA device, or (where
    the call reads a tiered bank over the host link) in pinned host memory."""
    if t.is_cuda:  # CUDA is up then: its current device without the checks for that
        return t.get_device() == _device()
    return host_ok and t.is_pinned()


def _numel_ok(t, n, what, kind=None, host_ok=False):
    """Checks a tensor argument before its address goes to the library:
    contiguous, of exactly the element type the call reads (`kind`: a dt code
    or F32/I32/I64), holding at least n elements, and on the current device
    (pinned host memory only where ``host_ok``).  Raw integer addresses are
    the caller's responsibility and pass unchecked."""
    if t is None or isinstance(t, int):
        return
    if not t.is_contiguous():
        raise ValueError(f"{what} must be contiguous")
    want = _torch_dtype(kind)
    if want is not None and t.dtype != want:
        raise ValueError(f"{what} is {t.dtype}, the call reads {want}")
    if t.numel() < n:
        raise ValueError(f"{what} holds {t.numel()} elements, needs {n}")
    if not _device_ok(t, host_ok):
        where = "the current CUDA device or pinned host memory" if host_ok else \
            "the current CUDA device"
        raise ValueError(f"{what} is on {t.device}{' (pageable)' if not t.is_cuda else ''}; "
                         f"the kernels read it from {where}")


def _arg(t, n, what, kind, dev):
    """The address of a tensor argument that passes _numel_ok; dev is
    _device()."""
    if t is None or isinstance(t, int):
        return t
    if (t.get_device() != dev or t.dtype is not _torch_dtype(kind) or t.numel() < n
            or not t.is_contiguous()):
        _numel_ok(t, n, what, kind)  # says what is wrong with it
    return t.data_ptr()


def _rows(t, n, heads, D, what, kind, dev):
    """The address of an operand of n tokens of [heads][D] and the elements
    from token to token: the tokens may lie apart (a slice of a fused
    projection's output), each token's heads contiguous and the tokens a
    16-byte multiple apart.  (Raw addresses, None and empty tensors are
    dense.)"""
    stride = heads * D
    if t is None or isinstance(t, int):
        return t, stride
    want = _torch_dtype(kind)
    if want is not None and t.dtype is not want:
        raise ValueError(f"{what} is {t.dtype}, the call reads {want}")
    shape = t.shape
    if len(shape) != 3 or shape[0] < n or shape[1] != heads or shape[2] != D:
        raise ValueError(f"{what} has shape {tuple(shape)}, needs [>= {n}, {heads}, {D}]")
    if shape[0] > 0 and heads > 0:
        s0, s1, s2 = t.stride()
        if s2 != 1 or (heads > 1 and s1 != D):
            raise ValueError(f"{what}: a token's heads must be contiguous")
        if shape[0] > 1:
            if s0 < stride or s0 * t.element_size() % 16:
                raise ValueError(f"{what}: tokens must be a multiple of 16 bytes apart, and not "
                                 f"overlap (stride {s0} elements)")
            stride = s0
    if t.get_device() != dev and not _device_ok(t, False):
        raise ValueError(f"{what} is on {t.device}; it must be on the current CUDA device")
    return t.data_ptr(), stride


def _ws_ok(ws, ws_bytes):
    """A workspace tensor must lie on the current device and hold at least
    the ws_bytes the library is told it may use."""
    if ws is None or isinstance(ws, int):
        return
    if not ws.is_contiguous():
        raise ValueError("ws must be contiguous")
    if ws.numel() * ws.element_size() < ws_bytes:
        raise ValueError(f"ws holds {ws.numel() * ws.element_size()} bytes, "
                         f"ws_bytes says {ws_bytes}")
    if not _device_ok(ws, False):
        raise ValueError(f"ws is on {ws.device}; it must be on the current CUDA device")


# ---------------------------------------------------------------- entry points

def msa_status_string(status: int) -> str:
    return lib().msa_status_string(status).decode()


def msa_version() -> str:
    return lib().msa_version().decode()


def msa_last_cuda_error() -> int:
    return lib().msa_last_cuda_error()


def msa_device_status(clear: bool = True, stream=None) -> int:
    out = ctypes.c_int32(0)
    _check("msa_device_status",
           lib().msa_device_status(ctypes.addressof(out), int(clear), _stream(stream)))
    return out.value


def msa_check_bounded_wait(limit_ns: int, arrive: bool, stream=None):
    _check("msa_check_bounded_wait",
           lib().msa_check_bounded_wait(int(limit_ns), int(arrive), _stream(stream)))


def msa_chunk_offsets(n_docs, tok_offsets, chunk, chunk_offsets, stream=None):
    _numel_ok(tok_offsets, n_docs + 1, "tok_offsets", I64)
    _numel_ok(chunk_offsets, n_docs + 1, "chunk_offsets", I64)
    _check("msa_chunk_offsets", lib().msa_chunk_offsets(
        n_docs, _ptr(tok_offsets), chunk, _ptr(chunk_offsets), _stream(stream)))


def msa_encode_pool(dt, L, n_tok, n_docs, H, D, k_tok, v_tok, kr_tok, tok_offsets,
                    chunk_offsets, n_chunks, rope_base, chunk, k_bar, v_bar, kr_bar,
                    stream=None):
    for t, what in ((k_tok, "k_tok"), (v_tok, "v_tok"), (kr_tok, "kr_tok")):
        _numel_ok(t, L * n_tok * H * D, what, _es(dt))
    for t, what in ((k_bar, "k_bar"), (v_bar, "v_bar"), (kr_bar, "kr_bar")):
        _numel_ok(t, L * n_chunks * H * D, what, _es(dt))
    _numel_ok(tok_offsets, n_docs + 1, "tok_offsets", I64)
    _numel_ok(chunk_offsets, n_docs + 1, "chunk_offsets", I64)
    _check("msa_encode_pool", lib().msa_encode_pool(
        dt, L, n_tok, n_docs, H, D, _ptr(k_tok), _ptr(v_tok), _ptr(kr_tok),
        _ptr(tok_offsets), _ptr(chunk_offsets), n_chunks, rope_base, chunk,
        _ptr(k_bar), _ptr(v_bar), _ptr(kr_bar), _stream(stream)))


def msa_encode_pool_prepared(dt, L, n_tok, n_docs, H, D, k_tok, v_tok, kr_tok, tok_offsets,
                             chunk_offsets, n_chunks, rope_base, chunk, k_bar, v_bar, kr_bar,
                             kr_hat, stream=None):
    for t, what in ((k_tok, "k_tok"), (v_tok, "v_tok"), (kr_tok, "kr_tok")):
        _numel_ok(t, L * n_tok * H * D, what, _es(dt))
    for t, what in ((k_bar, "k_bar"), (v_bar, "v_bar"), (kr_bar, "kr_bar"), (kr_hat, "kr_hat")):
        _numel_ok(t, L * n_chunks * H * D, what, _es(dt))
    _numel_ok(tok_offsets, n_docs + 1, "tok_offsets", I64)
    _numel_ok(chunk_offsets, n_docs + 1, "chunk_offsets", I64)
    _check("msa_encode_pool_prepared", lib().msa_encode_pool_prepared(
        dt, L, n_tok, n_docs, H, D, _ptr(k_tok), _ptr(v_tok), _ptr(kr_tok),
        _ptr(tok_offsets), _ptr(chunk_offsets), n_chunks, rope_base, chunk,
        _ptr(k_bar), _ptr(v_bar), _ptr(kr_bar), _ptr(kr_hat), _stream(stream)))


def msa_route_workspace_size(dt, B, T, H, D) -> int:
    return lib().msa_route_workspace_size(dt, B, T, H, D)


def msa_route_scores(dt, B, T, H, D, q_r, kr_bar, n_chunks, chunk_offsets, n_docs,
                     doc_scores, chunk_scores, ws, ws_bytes, stream=None):
    _numel_ok(q_r, B * T * H * D, "q_r", _es(dt))
    _numel_ok(kr_bar, n_chunks * H * D, "kr_bar", _es(dt))
    _numel_ok(chunk_offsets, n_docs + 1, "chunk_offsets", I64)
    _numel_ok(doc_scores, B * n_docs, "doc_scores", F32)
    _numel_ok(chunk_scores, B * n_chunks, "chunk_scores", F32)
    _ws_ok(ws, ws_bytes)
    _check("msa_route_scores", lib().msa_route_scores(
        dt, B, T, H, D, _ptr(q_r), _ptr(kr_bar), n_chunks, _ptr(chunk_offsets), n_docs,
        _ptr(doc_scores), _ptr(chunk_scores), _ptr(ws), ws_bytes, _stream(stream)))


def msa_route_prepare_bank(dt, n_chunks, H, D, kr_bar, kr_hat, stream=None):
    _numel_ok(kr_bar, n_chunks * H * D, "kr_bar", _es(dt))
    _numel_ok(kr_hat, n_chunks * H * D, "kr_hat", _es(dt))
    _check("msa_route_prepare_bank", lib().msa_route_prepare_bank(
        dt, n_chunks, H, D, _ptr(kr_bar), _ptr(kr_hat), _stream(stream)))


def msa_route_scores_prepared(dt, B, T, H, D, q_r, kr_hat, n_chunks, chunk_offsets, n_docs,
                              doc_scores, chunk_scores, ws, ws_bytes, stream=None):
    _numel_ok(q_r, B * T * H * D, "q_r", _es(dt))
    _numel_ok(kr_hat, n_chunks * H * D, "kr_hat", _es(dt))
    _numel_ok(chunk_offsets, n_docs + 1, "chunk_offsets", I64)
    _numel_ok(doc_scores, B * n_docs, "doc_scores", F32)
    _numel_ok(chunk_scores, B * n_chunks, "chunk_scores", F32)
    _ws_ok(ws, ws_bytes)
    _check("msa_route_scores_prepared", lib().msa_route_scores_prepared(
        dt, B, T, H, D, _ptr(q_r), _ptr(kr_hat), n_chunks, _ptr(chunk_offsets), n_docs,
        _ptr(doc_scores), _ptr(chunk_scores), _ptr(ws), ws_bytes, _stream(stream)))


def msa_route_noalloc_scratch_bytes() -> int:
    return lib().msa_route_noalloc_scratch_bytes()


def msa_route_scores_noalloc(dt, B, T, H, D, q_r, kr_bar, n_chunks, chunk_offsets, n_docs,
                             doc_scores, chunk_scores, stream=None):
    """msa_route_scores with the library's fixed scratch array instead of a
    caller workspace (for callers that cannot allocate device memory)."""
    _numel_ok(q_r, B * T * H * D, "q_r", _es(dt))
    _numel_ok(kr_bar, n_chunks * H * D, "kr_bar", _es(dt))
    _numel_ok(chunk_offsets, n_docs + 1, "chunk_offsets", I64)
    _numel_ok(doc_scores, B * n_docs, "doc_scores", F32)
    _numel_ok(chunk_scores, B * n_chunks, "chunk_scores", F32)
    _check("msa_route_scores_noalloc", lib().msa_route_scores_noalloc(
        dt, B, T, H, D, _ptr(q_r), _ptr(kr_bar), n_chunks, _ptr(chunk_offsets), n_docs,
        _ptr(doc_scores), _ptr(chunk_scores), _stream(stream)))


def msa_topk_workspace_size(B, n_docs, k) -> int:
    return lib().msa_topk_workspace_size(B, n_docs, k)


def msa_topk_merge_shards(B, world, k, cand_scores, cand_idx, doc_base, idx, top_scores,
                          stream=None):
    _numel_ok(cand_scores, world * B * k, "cand_scores", F32)
    _numel_ok(cand_idx, world * B * k, "cand_idx", I32)
    _numel_ok(doc_base, world, "doc_base", I32)
    _numel_ok(idx, B * k, "idx", I32)
    _numel_ok(top_scores, B * k, "top_scores", F32)
    _check("msa_topk_merge_shards", lib().msa_topk_merge_shards(
        B, world, k, _ptr(cand_scores), _ptr(cand_idx), _ptr(doc_base), _ptr(idx),
        _ptr(top_scores), _stream(stream)))


def msa_topk_docs(B, n_docs, k, scores, idx, top_scores, ws, ws_bytes, stream=None):
    _numel_ok(scores, B * n_docs, "scores", F32)
    _numel_ok(idx, B * k, "idx", I32)
    _numel_ok(top_scores, B * k, "top_scores", F32)
    _ws_ok(ws, ws_bytes)
    _check("msa_topk_docs", lib().msa_topk_docs(
        B, n_docs, k, _ptr(scores), _ptr(idx), _ptr(top_scores), _ptr(ws), ws_bytes,
        _stream(stream)))


def msa_gather_kv(dt, B, k, H, D, idx, chunk_offsets, n_docs, k_bar, v_bar, m_cap, k_mem,
                  v_mem, mem_len, stream=None):
    _numel_ok(idx, B * k, "idx", I32)
    _numel_ok(chunk_offsets, n_docs + 1, "chunk_offsets", I64)
    # the bank's row count sits on the device (chunk_offsets[n_docs]); its
    # type and placement are checked here: device or pinned host tier
    for t, what in ((k_bar, "k_bar"), (v_bar, "v_bar")):
        _numel_ok(t, 0, what, _es(dt), host_ok=True)
    _numel_ok(k_mem, B * m_cap * H * D, "k_mem", _es(dt))
    _numel_ok(v_mem, B * m_cap * H * D, "v_mem", _es(dt))
    _numel_ok(mem_len, B, "mem_len", I32)
    _check("msa_gather_kv", lib().msa_gather_kv(
        dt, B, k, H, D, _ptr(idx), _ptr(chunk_offsets), n_docs, _ptr(k_bar), _ptr(v_bar),
        m_cap, _ptr(k_mem), _ptr(v_mem), _ptr(mem_len), _stream(stream)))


def msa_sparse_attn_workspace_size(dt, B, T, T_loc, Hq, H, D, m_cap) -> int:
    return lib().msa_sparse_attn_workspace_size(dt, B, T, T_loc, Hq, H, D, m_cap)


def msa_sparse_attn(dt, B, T, T_loc, Hq, H, D, q, k_mem, v_mem, mem_len, m_cap, k_loc, v_loc,
                    pos0, rope_base, scale, out, ws, ws_bytes, stream=None):
    _numel_ok(q, B * T * Hq * D, "q", _es(dt))
    _numel_ok(k_mem, B * m_cap * H * D, "k_mem", _es(dt))
    _numel_ok(v_mem, B * m_cap * H * D, "v_mem", _es(dt))
    _numel_ok(mem_len, B, "mem_len", I32)
    _numel_ok(k_loc, B * T_loc * H * D, "k_loc", _es(dt))
    _numel_ok(v_loc, B * T_loc * H * D, "v_loc", _es(dt))
    _numel_ok(out, B * T * Hq * D, "out", _es(dt))
    _ws_ok(ws, ws_bytes)
    _check("msa_sparse_attn", lib().msa_sparse_attn(
        dt, B, T, T_loc, Hq, H, D, _ptr(q), _ptr(k_mem), _ptr(v_mem), _ptr(mem_len), m_cap,
        _ptr(k_loc), _ptr(v_loc), pos0, rope_base, scale, _ptr(out), _ptr(ws), ws_bytes,
        _stream(stream)))


def msa_sparse_attn_fused_workspace_size(dt, B, T, T_loc, Hq, H, D, k, m_cap) -> int:
    return lib().msa_sparse_attn_fused_workspace_size(dt, B, T, T_loc, Hq, H, D, k, m_cap)


def msa_sparse_attn_fused(dt, B, T, T_loc, Hq, H, D, q, idx, k, chunk_offsets, n_docs, k_bar,
                          v_bar, n_chunks, m_cap, k_loc, v_loc, pos0, rope_base, scale, out,
                          mem_len, ws, ws_bytes, stream=None):
    _numel_ok(q, B * T * Hq * D, "q", _es(dt))
    _numel_ok(idx, B * k, "idx", I32)
    _numel_ok(chunk_offsets, n_docs + 1, "chunk_offsets", I64)
    _numel_ok(k_bar, n_chunks * H * D, "k_bar", _es(dt), host_ok=True)
    _numel_ok(v_bar, n_chunks * H * D, "v_bar", _es(dt), host_ok=True)
    _numel_ok(k_loc, B * T_loc * H * D, "k_loc", _es(dt))
    _numel_ok(v_loc, B * T_loc * H * D, "v_loc", _es(dt))
    _numel_ok(out, B * T * Hq * D, "out", _es(dt))
    _numel_ok(mem_len, B, "mem_len", I32)
    _ws_ok(ws, ws_bytes)
    _check("msa_sparse_attn_fused", lib().msa_sparse_attn_fused(
        dt, B, T, T_loc, Hq, H, D, _ptr(q), _ptr(idx), k, _ptr(chunk_offsets), n_docs,
        _ptr(k_bar), _ptr(v_bar), n_chunks, m_cap, _ptr(k_loc), _ptr(v_loc), pos0, rope_base,
        scale, _ptr(out), _ptr(mem_len), _ptr(ws), ws_bytes, _stream(stream)))


def msa_route_backward_workspace_size(dt, B, T, H, D, n_chunks, n_docs) -> int:
    return lib().msa_route_backward_workspace_size(dt, B, T, H, D, n_chunks, n_docs)


def msa_route_backward(dt, B, T, H, D, q_r, kr_bar, n_chunks, chunk_offsets, n_docs, d_doc,
                       dq_r, dkr_bar, ws=None, ws_bytes=0, stream=None):
    _numel_ok(q_r, B * T * H * D, "q_r", _es(dt))
    _numel_ok(kr_bar, n_chunks * H * D, "kr_bar", _es(dt))
    _numel_ok(chunk_offsets, n_docs + 1, "chunk_offsets", I64)
    _numel_ok(d_doc, B * n_docs, "d_doc", F32)
    _numel_ok(dq_r, B * T * H * D, "dq_r", F32)
    _numel_ok(dkr_bar, n_chunks * H * D, "dkr_bar", F32)
    _ws_ok(ws, ws_bytes)
    _check("msa_route_backward", lib().msa_route_backward(
        dt, B, T, H, D, _ptr(q_r), _ptr(kr_bar), n_chunks, _ptr(chunk_offsets), n_docs,
        _ptr(d_doc), _ptr(dq_r), _ptr(dkr_bar), _ptr(ws), ws_bytes, _stream(stream)))


def msa_encode_pool_backward(L, n_tok, n_docs, H, D, dk_bar, dv_bar, dkr_bar, tok_offsets,
                             chunk_offsets, n_chunks, rope_base, dk_tok, dv_tok, dkr_tok,
                             stream=None):
    for t, nm in ((dk_bar, "dk_bar"), (dv_bar, "dv_bar"), (dkr_bar, "dkr_bar")):
        _numel_ok(t, L * n_chunks * H * D, nm, F32)
    for t, nm in ((dk_tok, "dk_tok"), (dv_tok, "dv_tok"), (dkr_tok, "dkr_tok")):
        _numel_ok(t, L * n_tok * H * D, nm, F32)
    _numel_ok(tok_offsets, n_docs + 1, "tok_offsets", I64)
    _numel_ok(chunk_offsets, n_docs + 1, "chunk_offsets", I64)
    _check("msa_encode_pool_backward", lib().msa_encode_pool_backward(
        L, n_tok, n_docs, H, D, _ptr(dk_bar), _ptr(dv_bar), _ptr(dkr_bar), _ptr(tok_offsets),
        _ptr(chunk_offsets), n_chunks, rope_base, _ptr(dk_tok), _ptr(dv_tok), _ptr(dkr_tok),
        _stream(stream)))


# The native marshalling of the calls below (csrc/marshal.cpp): it does what
# the Python path of each does where every check passes, and returns None,
# without having called the library, where one does not.
_bound: list = [None, None]  # the library handle it was bound to, the module


def _native():
    handle = lib()
    if handle is not _bound[0]:
        module = None
        if isinstance(handle, ctypes.CDLL):
            try:
                from . import _marshal as module
            except ImportError:  # not built: the Python path alone
                module = None
        if module is not None:
            torch = _th()
            raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
            dev = getattr(torch._C, "_cuda_getDevice", None)
            if raw is None or dev is None:
                module = None
            else:
                module.bind(
                    tuple(ctypes.cast(getattr(handle, name), ctypes.c_void_p).value for name in
                          ("msa_qk_norm_rope", "msa_qk_norm_rope_backward", "msa_paged_append",
                           "msa_tree_attn")),
                    (torch.float32, torch.bfloat16, torch.int32, torch.int64, torch.uint8), dev,
                    raw)
        _bound[:] = [handle, module]
    return _bound[1]


def msa_qk_norm_rope(dt, n_tok, Hq, H, D, q, k, q_weight, k_weight, positions, eps, rope_base,
                     q_out, k_out, stream=None):
    """q and k: [n_tok][heads][D] tensors, the token strides taken from them
    (raw addresses are dense)."""
    native = _native()
    if native is not None:
        rc = native.msa_qk_norm_rope(
            dt, n_tok, Hq, H, D, q, k, q_weight, k_weight, positions, eps, rope_base, q_out, k_out,
            stream)
        if rc is not None:
            return _check("msa_qk_norm_rope", rc)
    es, dev = _es(dt), _device()
    qp, qs = _rows(q, n_tok, Hq, D, "q", es, dev)
    kp, ks = _rows(k, n_tok, H, D, "k", es, dev)
    _check("msa_qk_norm_rope", lib().msa_qk_norm_rope(
        dt, n_tok, Hq, H, D, qp, qs, kp, ks, _arg(q_weight, D, "q_weight", es, dev),
        _arg(k_weight, D, "k_weight", es, dev), _arg(positions, n_tok, "positions", I32, dev), eps,
        rope_base, _arg(q_out, n_tok * Hq * D, "q_out", es, dev),
        _arg(k_out, n_tok * H * D, "k_out", es, dev), _stream(stream)))


def msa_qk_norm_rope_backward_workspace_size(n_tok, D) -> int:
    return lib().msa_qk_norm_rope_backward_workspace_size(n_tok, D)


def msa_qk_norm_rope_backward(dt, grad_dt, n_tok, Hq, H, D, q, k, q_weight, k_weight, positions,
                              eps, rope_base, dq_out, dk_out, dq, dk, dq_weight, dk_weight, ws,
                              ws_bytes, stream=None):
    """q, k, dq and dk: [n_tok][heads][D] tensors, the token strides taken
    from them (raw addresses are dense)."""
    native = _native()
    if native is not None:
        rc = native.msa_qk_norm_rope_backward(
            dt, grad_dt, n_tok, Hq, H, D, q, k, q_weight, k_weight, positions, eps, rope_base,
            dq_out, dk_out, dq, dk, dq_weight, dk_weight, ws, ws_bytes, stream)
        if rc is not None:
            return _check("msa_qk_norm_rope_backward", rc)
    es, gs, dev = _es(dt), _es(grad_dt), _device()
    qp, qs = _rows(q, n_tok, Hq, D, "q", es, dev)
    kp, ks = _rows(k, n_tok, H, D, "k", es, dev)
    dqp, dqs = _rows(dq, n_tok, Hq, D, "dq", gs, dev)
    dkp, dks = _rows(dk, n_tok, H, D, "dk", gs, dev)
    _ws_ok(ws, ws_bytes)
    _check("msa_qk_norm_rope_backward", lib().msa_qk_norm_rope_backward(
        dt, grad_dt, n_tok, Hq, H, D, qp, qs, kp, ks,
        _arg(q_weight, D, "q_weight", es, dev), _arg(k_weight, D, "k_weight", es, dev),
        _arg(positions, n_tok, "positions", I32, dev), eps, rope_base,
        _arg(dq_out, n_tok * Hq * D, "dq_out", gs, dev),
        _arg(dk_out, n_tok * H * D, "dk_out", gs, dev), dqp, dqs, dkp, dks,
        _arg(dq_weight, D, "dq_weight", F32, dev),
        _arg(dk_weight, D, "dk_weight", F32, dev), _ptr(ws), ws_bytes, _stream(stream)))


def msa_paged_append(dt, B, n_tok, Hq, H, D, q, k, v, q_weight, k_weight, tok_offsets, positions,
                     eps, rope_base, block_table, max_pages, cache_len, page_size, n_pages,
                     k_pages, v_pages, q_out, stream=None):
    """q, k and v: [n_tok][heads][D] tensors, the token strides taken from
    them (raw addresses are dense)."""
    native = _native()
    if native is not None:
        rc = native.msa_paged_append(
            dt, B, n_tok, Hq, H, D, q, k, v, q_weight, k_weight, tok_offsets, positions, eps,
            rope_base, block_table, max_pages, cache_len, page_size, n_pages, k_pages, v_pages,
            q_out, stream)
        if rc is not None:
            return _check("msa_paged_append", rc)
    es, dev = _es(dt), _device()
    qp, qs = _rows(q, n_tok, Hq, D, "q", es, dev)
    kp, ks = _rows(k, n_tok, H, D, "k", es, dev)
    vp, vs = _rows(v, n_tok, H, D, "v", es, dev)
    pool = n_pages * H * page_size * D
    _check("msa_paged_append", lib().msa_paged_append(
        dt, B, n_tok, Hq, H, D, qp, qs, kp, ks, vp, vs,
        _arg(q_weight, D, "q_weight", es, dev), _arg(k_weight, D, "k_weight", es, dev),
        _arg(tok_offsets, B + 1, "tok_offsets", I64, dev),
        _arg(positions, n_tok, "positions", I32, dev),
        eps, rope_base, _arg(block_table, B * max_pages, "block_table", I32, dev), max_pages,
        _arg(cache_len, B, "cache_len", I32, dev), page_size, n_pages,
        _arg(k_pages, pool, "k_pages", es, dev), _arg(v_pages, pool, "v_pages", es, dev),
        _arg(q_out, n_tok * Hq * D, "q_out", es, dev), _stream(stream)))


def msa_tree_attn_workspace_size(dt, B, n_max, Hq, H, D, m_cap, max_pages, page_size) -> int:
    return lib().msa_tree_attn_workspace_size(dt, B, n_max, Hq, H, D, m_cap, max_pages, page_size)


def msa_tree_attn(dt, B, n_tok, n_max, Hq, H, D, q, tok_offsets, parents, k_mem, v_mem, mem_len,
                  m_cap, k_pages, v_pages, n_pages, page_size, block_table, max_pages, cache_len,
                  scale, out, ws, ws_bytes, stream=None):
    native = _native()
    if native is not None:
        rc = native.msa_tree_attn(
            dt, B, n_tok, n_max, Hq, H, D, q, tok_offsets, parents, k_mem, v_mem, mem_len, m_cap,
            k_pages, v_pages, n_pages, page_size, block_table, max_pages, cache_len, scale, out, ws,
            ws_bytes, stream)
        if rc is not None:
            return _check("msa_tree_attn", rc)
    es, dev = _es(dt), _device()
    rows, mem, pool = n_tok * Hq * D, B * m_cap * H * D, n_pages * H * page_size * D
    _ws_ok(ws, ws_bytes)
    _check("msa_tree_attn", lib().msa_tree_attn(
        dt, B, n_tok, n_max, Hq, H, D, _arg(q, rows, "q", es, dev),
        _arg(tok_offsets, B + 1, "tok_offsets", I64, dev),
        _arg(parents, n_tok, "parents", I32, dev),
        _arg(k_mem, mem, "k_mem", es, dev), _arg(v_mem, mem, "v_mem", es, dev),
        _arg(mem_len, B if m_cap else 0, "mem_len", I32, dev), m_cap,
        _arg(k_pages, pool, "k_pages", es, dev), _arg(v_pages, pool, "v_pages", es, dev), n_pages,
        page_size, _arg(block_table, B * max_pages, "block_table", I32, dev), max_pages,
        _arg(cache_len, B, "cache_len", I32, dev), scale, _arg(out, rows, "out", es, dev), _ptr(ws),
        ws_bytes, _stream(stream)))
