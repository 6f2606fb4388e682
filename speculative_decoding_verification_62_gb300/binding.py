"""Thin ctypes binding of the C ABI in include/spec_verify.h.

Argument marshalling only: every step of the verify path runs in the CUDA
library.  Functions keep the C names.  Tensors must be CUDA, contiguous and
of the documented dtype and shape; the call is issued on the current torch
stream unless `stream` is given.  There is no CPU fallback: if the library
cannot be loaded or built, the first call raises.
"""
from __future__ import annotations

import ctypes
import functools
import threading

import torch

from . import build as _build

SV_F32, SV_BF16, SV_F16, SV_E4M3 = 0, 1, 2, 3
SV_MAX_GAMMA = 31
SV_MAX_HEAD_DIM = 128
SV_MAX_VOCAB = 1 << 24
SV_MAX_BLOCK = 128
STATUS_BITS = {1: "BAD_GAMMA", 2: "BAD_TOKEN", 4: "BAD_UNIFORM", 8: "BAD_TEMPERATURE",
               16: "NONFINITE_ROW", 32: "INTERNAL", 64: "TIMEOUT", 128: "BAD_PROB",
               256: "BAD_PAGE", 512: "BAD_LENGTH", 1024: "BAD_SCALE", 2048: "BAD_ROW", 4096: "NO_PAGES"}
SV_NOALLOC_SCRATCH_BYTES = 4 << 20
EXPORTS = ("spec_verify_workspace_size", "spec_verify_sample", "spec_verify_greedy",
           "spec_verify_sample_packed", "spec_verify_greedy_packed", "spec_verify_draw",
           "spec_verify_sample_noalloc", "spec_verify_status", "spec_verify_strerror",
           "spec_verify_set_schedule", "spec_verify_route", "spec_verify_cluster_size",
           "spec_verify_set_wait_limit", "spec_verify_set_lazy", "spec_verify_sample_probs",
           "spec_verify_sample_probs_packed", "spec_verify_kv_append", "spec_verify_attention",
           "spec_verify_attention_workspace_size", "spec_verify_kv_append_e4m3",
           "spec_verify_attention_e4m3", "spec_verify_attention_e4m3_workspace_size",
           "spec_verify_pages_workspace_size", "spec_verify_pages_step", "spec_verify_pages_compact")
SCHEDULE_AUTO, SCHEDULE_PERSISTENT, SCHEDULE_STREAM = 0, 1, 2
ROUTE_PERSISTENT, ROUTE_CLUSTER, ROUTE_STREAM, ROUTE_CLAIMS, ROUTE_PIPELINE = 0, 1, 2, 3, 4

_lock = threading.Lock()
_lib = None


class _KvCache(ctypes.Structure):
    """sv_kv_cache of include/spec_verify.h."""
    _fields_ = [("k_pages", ctypes.c_void_p), ("v_pages", ctypes.c_void_p), ("dtype", ctypes.c_int),
                ("num_pages", ctypes.c_int), ("page_size", ctypes.c_int), ("kv_heads", ctypes.c_int),
                ("head_dim", ctypes.c_int), ("k_strides", ctypes.c_int64 * 3),
                ("v_strides", ctypes.c_int64 * 3), ("page_table", ctypes.c_void_p),
                ("max_pages", ctypes.c_int), ("batch", ctypes.c_int), ("kv_len", ctypes.c_void_p)]


class _KvScales(ctypes.Structure):
    """sv_kv_scales of include/spec_verify.h."""
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("block", ctypes.c_int)]


class _PagePool(ctypes.Structure):
    """sv_page_pool of include/spec_verify.h."""
    _fields_ = [("held", ctypes.c_void_p), ("ref", ctypes.c_void_p), ("free_pages", ctypes.c_void_p),
                ("free_count", ctypes.c_void_p)]


class SpecVerifyError(RuntimeError):
    def __init__(self, code: int):
        super().__init__(f"{spec_verify_strerror(code)} (code {code})")
        self.code = code


def load_library():
    """Load (building first if needed) libspec_verify.so and declare signatures."""
    global _lib
    with _lock:
        if _lib is not None:
            return _lib
        lib = ctypes.CDLL(_build.build())
        vp, ci, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
        lib.spec_verify_workspace_size.restype = sz
        lib.spec_verify_workspace_size.argtypes = [ci, ci, ci]
        lib.spec_verify_sample.restype = ci
        lib.spec_verify_sample.argtypes = [vp, vp, ci, ci, ci, ci, vp, vp, vp, vp, vp, vp, vp,
                                           vp, vp, sz, vp]
        lib.spec_verify_greedy.restype = ci
        lib.spec_verify_greedy.argtypes = [vp, ci, ci, ci, ci, vp, vp, vp, vp, vp, sz, vp]
        lib.spec_verify_sample_packed.restype = ci
        lib.spec_verify_sample_packed.argtypes = [vp, vp, ci, ci, ci, ci, vp, ci, vp, vp, vp,
                                                  vp, vp, vp, vp, vp, sz, vp]
        lib.spec_verify_greedy_packed.restype = ci
        lib.spec_verify_greedy_packed.argtypes = [vp, ci, ci, ci, ci, vp, ci, vp, vp, vp, vp,
                                                  sz, vp]
        lib.spec_verify_draw.restype = ci
        lib.spec_verify_draw.argtypes = [vp, ci, ci, ci, vp, vp, vp, vp, sz, vp]
        lib.spec_verify_sample_noalloc.restype = ci
        lib.spec_verify_sample_noalloc.argtypes = [vp, vp, ci, ci, ci, ci, vp, vp, vp, vp, vp,
                                                   vp, vp, vp, vp]
        lib.spec_verify_status.restype = ci
        lib.spec_verify_status.argtypes = [vp, vp, ctypes.POINTER(ctypes.c_uint32)]
        lib.spec_verify_strerror.restype = ctypes.c_char_p
        lib.spec_verify_strerror.argtypes = [ci]
        lib.spec_verify_set_schedule.restype = ci
        lib.spec_verify_set_schedule.argtypes = [ci]
        lib.spec_verify_route.restype = ci
        lib.spec_verify_route.argtypes = [ci, ci, ci, ci, ci, ctypes.POINTER(ci)]
        lib.spec_verify_cluster_size.restype = ci
        lib.spec_verify_cluster_size.argtypes = [ci, ci, ci, ci, ci]
        lib.spec_verify_set_wait_limit.restype = ctypes.c_ulonglong
        lib.spec_verify_set_wait_limit.argtypes = [ctypes.c_ulonglong]
        lib.spec_verify_set_lazy.restype = ci
        lib.spec_verify_set_lazy.argtypes = [ci]
        i64p, cf = ctypes.POINTER(ctypes.c_int64), ctypes.c_float
        lib.spec_verify_sample_probs.restype = ci
        lib.spec_verify_sample_probs.argtypes = [vp, vp, ci, ci, ci, ci, vp, vp, vp, vp, vp, vp,
                                                 sz, vp]
        lib.spec_verify_sample_probs_packed.restype = ci
        lib.spec_verify_sample_probs_packed.argtypes = [vp, vp, ci, ci, ci, ci, vp, ci, vp, vp,
                                                        vp, vp, vp, sz, vp]
        cache = ctypes.POINTER(_KvCache)
        lib.spec_verify_kv_append.restype = ci
        lib.spec_verify_kv_append.argtypes = [vp, i64p, ci, vp, i64p, vp, i64p, vp, i64p, cache, vp,
                                              ci, ci, vp, ci, ci, cf, vp, ci, vp, sz, vp]
        lib.spec_verify_attention_workspace_size.restype = sz
        lib.spec_verify_attention_workspace_size.argtypes = [ci, ci, ci]
        lib.spec_verify_attention.restype = ci
        lib.spec_verify_attention.argtypes = [vp, i64p, ci, cache, vp, ci, vp, ci, ci, cf, vp, vp,
                                              vp, vp, sz, vp]
        scales, pool = ctypes.POINTER(_KvScales), ctypes.POINTER(_PagePool)
        lib.spec_verify_kv_append_e4m3.restype = ci
        lib.spec_verify_kv_append_e4m3.argtypes = [vp, i64p, ci, vp, i64p, vp, i64p, ci, vp, i64p, cache,
                                                   scales, vp, ci, ci, vp, ci, ci, cf, vp, ci, vp, sz, vp]
        lib.spec_verify_attention_e4m3_workspace_size.restype = sz
        lib.spec_verify_attention_e4m3_workspace_size.argtypes = [ci, ci, ci]
        lib.spec_verify_attention_e4m3.restype = ci
        lib.spec_verify_attention_e4m3.argtypes = [vp, i64p, ci, ci, cache, scales, vp, ci, vp, ci, ci, cf,
                                                   vp, vp, vp, vp, sz, vp]
        lib.spec_verify_pages_workspace_size.restype = sz
        lib.spec_verify_pages_workspace_size.argtypes = [ci, ci, ci]
        lib.spec_verify_pages_step.restype = ci
        lib.spec_verify_pages_step.argtypes = [cache, scales, pool, vp, vp, vp, sz, vp]
        lib.spec_verify_pages_compact.restype = ci
        lib.spec_verify_pages_compact.argtypes = [cache, scales, pool, vp, vp, sz, vp]
        _lib = lib
        return lib


def spec_verify_strerror(code: int) -> str:
    return load_library().spec_verify_strerror(int(code)).decode()


def spec_verify_set_schedule(schedule: int) -> int:
    """SCHEDULE_AUTO, SCHEDULE_PERSISTENT or SCHEDULE_STREAM for the calls that follow;
    returns the previous policy."""
    rc = load_library().spec_verify_set_schedule(int(schedule))
    if rc < 0:
        raise SpecVerifyError(rc)
    return rc


def spec_verify_set_lazy(on: bool) -> bool:
    """Position-by-position reading on the request-claims schedule for the calls
    that follow (the default); returns the previous setting."""
    rc = load_library().spec_verify_set_lazy(1 if on else 0)
    if rc < 0:
        raise SpecVerifyError(rc)
    return bool(rc)


def spec_verify_set_wait_limit(ns: int) -> int:
    """Limit (ns) of every bounded wait in later calls (0: the 2 s default);
    returns the previous limit."""
    return int(load_library().spec_verify_set_wait_limit(int(ns)))


def spec_verify_route(dtype: torch.dtype, B: int, G: int, V: int, greedy: bool = False):
    """(ROUTE_*, CTAs per request) of the kernel a call of this shape would use."""
    code = SV_BF16 if dtype == torch.bfloat16 else SV_F32
    C = ctypes.c_int(0)
    rc = load_library().spec_verify_route(code, int(B), int(G), int(V), int(bool(greedy)),
                                          ctypes.byref(C))
    if rc < 0:
        raise SpecVerifyError(rc)
    return rc, C.value


def spec_verify_cluster_size(dtype: torch.dtype, B: int, G: int, V: int, greedy: bool = False) -> int:
    """CTAs per request of the cluster schedule (resident, streaming; 1 for request claims)
    for this shape, 0 for the persistent grid."""
    code = SV_BF16 if dtype == torch.bfloat16 else SV_F32
    rc = load_library().spec_verify_cluster_size(code, int(B), int(G), int(V), int(bool(greedy)))
    if rc < 0:
        raise SpecVerifyError(rc)
    return rc


def spec_verify_workspace_size(B: int, G: int, V: int) -> int:
    return int(load_library().spec_verify_workspace_size(int(B), int(G), int(V)))


def make_workspace(B: int, G: int, V: int, device="cuda") -> torch.Tensor:
    """Zero-filled device workspace (256-byte aligned by the caching allocator)."""
    n = spec_verify_workspace_size(B, G, V)
    if n == 0:
        raise ValueError(f"invalid sizes B={B} G={G} V={V}")
    return torch.zeros(n, dtype=torch.uint8, device=device)


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return SV_BF16
    if t.dtype == torch.float32:
        return SV_F32
    raise TypeError(f"logits must be bfloat16 or float32, got {t.dtype}")


def _dev(t, name, dtype=None, shape=None):
    if t is None:
        return None
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    return ctypes.c_void_p(t.data_ptr()) if t.numel() else ctypes.c_void_p(0)


def _stream(stream):
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def spec_verify_sample(target_logits, draft_logits, draft_tokens, gamma, uniforms, temperature,
                       out_tokens, num_accepted, workspace, p_tok=None, q_tok=None,
                       stream=None) -> None:
    """Sampling verify step; see include/spec_verify.h for the contract."""
    B, G1, V = target_logits.shape
    G = G1 - 1
    code = _dtype_code(target_logits)
    args = (
        _dev(target_logits, "target_logits"),
        _dev(draft_logits, "draft_logits", target_logits.dtype, (B, G, V)),
        code, B, G, V,
        _dev(draft_tokens, "draft_tokens", torch.int32, (B, G)),
        _dev(gamma, "gamma", torch.int32, (B,)),
        _dev(uniforms, "uniforms", torch.float32, (B, G + 1)),
        _dev(temperature, "temperature", torch.float32, (B,)),
        _dev(out_tokens, "out_tokens", torch.int32, (B, G + 1)),
        _dev(num_accepted, "num_accepted", torch.int32, (B,)),
        _dev(p_tok, "p_tok", torch.float64, (B, G)),
        _dev(q_tok, "q_tok", torch.float64, (B, G)),
        _dev(workspace, "workspace", torch.uint8), workspace.numel(), _stream(stream))
    rc = load_library().spec_verify_sample(*args)
    if rc != 0:
        raise SpecVerifyError(rc)


def spec_verify_sample_packed(target_logits, draft_logits, cu_draft, draft_tokens, uniforms,
                              temperature, out_tokens, num_accepted, workspace, p_tok=None,
                              q_tok=None, stream=None) -> None:
    """Sampling verify step on the packed layout; see include/spec_verify.h."""
    B = cu_draft.numel() - 1
    total = draft_tokens.numel()
    V = target_logits.shape[1]
    G = out_tokens.shape[1] - 1
    if target_logits.shape[0] != total + B:
        raise ValueError("target_logits must have total_drafts + B rows")
    code = _dtype_code(target_logits)
    args = (
        _dev(target_logits, "target_logits"),
        _dev(draft_logits, "draft_logits", target_logits.dtype, (total, V)),
        code, B, G, V,
        _dev(cu_draft, "cu_draft", torch.int32, (B + 1,)), total,
        _dev(draft_tokens, "draft_tokens", torch.int32, (total,)),
        _dev(uniforms, "uniforms", torch.float32, (total + B,)),
        _dev(temperature, "temperature", torch.float32, (B,)),
        _dev(out_tokens, "out_tokens", torch.int32, (B, G + 1)),
        _dev(num_accepted, "num_accepted", torch.int32, (B,)),
        _dev(p_tok, "p_tok", torch.float64, (total,)),
        _dev(q_tok, "q_tok", torch.float64, (total,)),
        _dev(workspace, "workspace", torch.uint8), workspace.numel(), _stream(stream))
    rc = load_library().spec_verify_sample_packed(*args)
    if rc != 0:
        raise SpecVerifyError(rc)


def spec_verify_greedy_packed(target_logits, cu_draft, draft_tokens, out_tokens, num_accepted,
                              workspace, stream=None) -> None:
    """Greedy verify step on the packed layout; see include/spec_verify.h."""
    B = cu_draft.numel() - 1
    total = draft_tokens.numel()
    V = target_logits.shape[1]
    G = out_tokens.shape[1] - 1
    if target_logits.shape[0] != total + B:
        raise ValueError("target_logits must have total_drafts + B rows")
    args = (
        _dev(target_logits, "target_logits"), _dtype_code(target_logits), B, G, V,
        _dev(cu_draft, "cu_draft", torch.int32, (B + 1,)), total,
        _dev(draft_tokens, "draft_tokens", torch.int32, (total,)),
        _dev(out_tokens, "out_tokens", torch.int32, (B, G + 1)),
        _dev(num_accepted, "num_accepted", torch.int32, (B,)),
        _dev(workspace, "workspace", torch.uint8), workspace.numel(), _stream(stream))
    rc = load_library().spec_verify_greedy_packed(*args)
    if rc != 0:
        raise SpecVerifyError(rc)


def spec_verify_draw(logits, uniforms, temperature, tokens, workspace, stream=None) -> None:
    """One token per row from softmax(logits / T) by inverse CDF (argmax at T = 0)."""
    B, V = logits.shape
    args = (
        _dev(logits, "logits"), _dtype_code(logits), B, V,
        _dev(uniforms, "uniforms", torch.float32, (B,)),
        _dev(temperature, "temperature", torch.float32, (B,)),
        _dev(tokens, "tokens", torch.int32, (B,)),
        _dev(workspace, "workspace", torch.uint8), workspace.numel(), _stream(stream))
    rc = load_library().spec_verify_draw(*args)
    if rc != 0:
        raise SpecVerifyError(rc)


def spec_verify_sample_noalloc(target_logits, draft_logits, draft_tokens, gamma, uniforms,
                               temperature, out_tokens, num_accepted, p_tok=None, q_tok=None,
                               stream=None) -> None:
    """Sampling verify step on the library's built-in scratch array (no workspace)."""
    B, G1, V = target_logits.shape
    G = G1 - 1
    code = _dtype_code(target_logits)
    args = (
        _dev(target_logits, "target_logits"),
        _dev(draft_logits, "draft_logits", target_logits.dtype, (B, G, V)),
        code, B, G, V,
        _dev(draft_tokens, "draft_tokens", torch.int32, (B, G)),
        _dev(gamma, "gamma", torch.int32, (B,)),
        _dev(uniforms, "uniforms", torch.float32, (B, G + 1)),
        _dev(temperature, "temperature", torch.float32, (B,)),
        _dev(out_tokens, "out_tokens", torch.int32, (B, G + 1)),
        _dev(num_accepted, "num_accepted", torch.int32, (B,)),
        _dev(p_tok, "p_tok", torch.float64, (B, G)),
        _dev(q_tok, "q_tok", torch.float64, (B, G)),
        _stream(stream))
    rc = load_library().spec_verify_sample_noalloc(*args)
    if rc != 0:
        raise SpecVerifyError(rc)


def spec_verify_greedy(target_logits, draft_tokens, gamma, out_tokens, num_accepted, workspace,
                       stream=None) -> None:
    """Greedy (argmax-match) verify step; see include/spec_verify.h."""
    B, G1, V = target_logits.shape
    G = G1 - 1
    args = (
        _dev(target_logits, "target_logits"), _dtype_code(target_logits), B, G, V,
        _dev(draft_tokens, "draft_tokens", torch.int32, (B, G)),
        _dev(gamma, "gamma", torch.int32, (B,)),
        _dev(out_tokens, "out_tokens", torch.int32, (B, G + 1)),
        _dev(num_accepted, "num_accepted", torch.int32, (B,)),
        _dev(workspace, "workspace", torch.uint8), workspace.numel(), _stream(stream))
    rc = load_library().spec_verify_greedy(*args)
    if rc != 0:
        raise SpecVerifyError(rc)


# The calls below check their tensors in one expression: a small batch's kernel takes 4 to
# 10 us, less than a careless wrapper.  What does not pass goes through _arg, tensor by
# tensor, which says what is wrong.
def _arg(t, name, dtype, shape, index):
    """Address of a contiguous tensor of that dtype and shape (None: any) on CUDA device `index`."""
    if isinstance(t, torch.Tensor):
        if (t.dtype is dtype and t.get_device() == index and t.is_contiguous()
                and (shape is None or t.shape == shape)):
            return t.data_ptr()
        _dev(t, name, dtype, shape)  # raises what it finds wrong
        raise ValueError(f"{name} is on {t.device}, other arguments on cuda:{index}")
    raise TypeError(f"{name} must be a CUDA tensor")


def _index(t, name):
    """CUDA device index of the tensor that the others go by."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    return t.get_device()


# (the public ways take 1 us more)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)
_current = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _launch(call, index, stream, *args):
    """The C call on the tensors' device, on `stream` or that device's current one."""
    stream = _raw_stream(index) if stream is None else stream.cuda_stream
    if _current() == index:
        rc = call(*args, stream)
    else:
        with torch.cuda.device(index):
            rc = call(*args, stream)
    if rc != 0:
        raise SpecVerifyError(rc)


@functools.lru_cache(maxsize=256)
def _two(a, b):
    return (ctypes.c_int64 * 2)(a, b)


def _probs(target, draft, d_shape, first, f_name, f_shape, tokens, k_shape, uniforms,
           u_shape, out, o_shape, accepted, B, workspace, index):
    """Checks the tensors of the two calls below; the addresses of rows, and the type code."""
    i32, dtype = torch.int32, target.dtype
    try:
        fine = (tokens.dtype is i32 and first.dtype is i32 and out.dtype is i32
                and accepted.dtype is i32 and uniforms.dtype is torch.float32
                and workspace.dtype is torch.uint8 and tokens.shape == k_shape
                and first.shape == f_shape and out.shape == o_shape and accepted.shape == (B,)
                and uniforms.shape == u_shape and target.is_contiguous() and tokens.is_contiguous()
                and first.is_contiguous() and out.is_contiguous() and accepted.is_contiguous()
                and uniforms.is_contiguous() and workspace.is_contiguous()
                and tokens.get_device() == index and first.get_device() == index
                and out.get_device() == index and accepted.get_device() == index
                and uniforms.get_device() == index and workspace.get_device() == index)
    except AttributeError:
        fine = False
    if not fine:
        _arg(target, "target_probs", dtype, None, index)
        _arg(first, f_name, i32, f_shape, index)
        _arg(tokens, "draft_tokens", i32, k_shape, index)
        _arg(uniforms, "uniforms", torch.float32, u_shape, index)
        _arg(out, "out_tokens", i32, o_shape, index)
        _arg(accepted, "num_accepted", i32, (B,), index)
        _arg(workspace, "workspace", torch.uint8, None, index)
    return (target.data_ptr(), None if draft is None else _arg(draft, "draft_probs", dtype, d_shape, index),
            SV_F32 if dtype is torch.float32 else _dtype_code(target))


def spec_verify_sample_probs(target_probs, draft_probs, draft_tokens, gamma, uniforms, out_tokens,
                             num_accepted, workspace, stream=None) -> None:
    """Sampling verify step on probabilities instead of logits; draft_probs None: the
    drafts were certain (looked up).  See include/spec_verify.h."""
    index = _index(target_probs, "target_probs")
    B, G1, V = target_probs.shape
    G = G1 - 1
    rows = (B, G1)
    tp, dp, code = _probs(target_probs, draft_probs, (B, G, V), gamma, "gamma", (B,),
                          draft_tokens, (B, G), uniforms, rows, out_tokens, rows, num_accepted, B,
                          workspace, index)
    _launch((_lib or load_library()).spec_verify_sample_probs, index, stream, tp, dp, code, B, G, V,
            draft_tokens.data_ptr(), gamma.data_ptr(), uniforms.data_ptr(), out_tokens.data_ptr(),
            num_accepted.data_ptr(), workspace.data_ptr(), workspace.numel())


def spec_verify_sample_probs_packed(target_probs, draft_probs, cu_draft, draft_tokens, uniforms,
                                    out_tokens, num_accepted, workspace, stream=None) -> None:
    """spec_verify_sample_probs on the packed layout; see include/spec_verify.h."""
    index = _index(target_probs, "target_probs")
    B = cu_draft.numel() - 1
    total = draft_tokens.numel()
    rows, V = target_probs.shape
    G = out_tokens.shape[1] - 1
    if rows != total + B:
        raise ValueError("target_probs must have total_drafts + B rows")
    tp, dp, code = _probs(target_probs, draft_probs, (total, V), cu_draft, "cu_draft", (B + 1,),
                          draft_tokens, (total,), uniforms, (rows,), out_tokens, (B, G + 1),
                          num_accepted, B, workspace, index)
    _launch((_lib or load_library()).spec_verify_sample_probs_packed, index, stream, tp, dp, code, B,
            G, V, cu_draft.data_ptr(), total, draft_tokens.data_ptr(), uniforms.data_ptr(),
            out_tokens.data_ptr(), num_accepted.data_ptr(), workspace.data_ptr(), workspace.numel())


class PagedCache:
    """The target's KV cache of a batch: page pools, page table and lengths.

    k_pages, v_pages [num_pages, page_size, kv_heads, head_dim] (bfloat16 or float16, the
    last dimension contiguous, the others of any stride that is a multiple of 8: a pool
    stored [page, head, token, value] is passed as its transpose(1, 2)), page_table
    [batch, max_pages] int32 and kv_len [batch] int32.  The tensors stay the caller's: they
    are used in place (their contents may change between calls, the attributes may not be
    assigned), and kv_len is advanced by commit() alone.  Pages or rows of the pools may
    not overlap one another.

    A cache in 8 bits: pools of float8_e4m3fn (head_dim and strides multiples of 16) with
    k_scales, v_scales [num_pages, page_size / block, kv_heads] float32, whose shape says
    how many tokens share a scale.
    """
    k_pages = property(lambda self: self._tensors[0])
    v_pages = property(lambda self: self._tensors[1])
    page_table = property(lambda self: self._tensors[2])
    kv_len = property(lambda self: self._tensors[3])
    k_scales = property(lambda self: self._tensors[4])
    v_scales = property(lambda self: self._tensors[5])

    def __init__(self, k_pages, v_pages, page_table, kv_len, k_scales=None, v_scales=None):
        self.index = _index(k_pages, "k_pages")
        for name, t in (("v_pages", v_pages), ("page_table", page_table), ("kv_len", kv_len)):
            if _index(t, name) != self.index:
                raise ValueError(f"{name} is on {t.device}, k_pages on {k_pages.device}")
        e4m3 = k_scales is not None or v_scales is not None
        if e4m3 and k_pages.dtype != torch.float8_e4m3fn:
            raise TypeError(f"k_pages with scales must be float8_e4m3fn, got {k_pages.dtype}")
        if not e4m3 and k_pages.dtype == torch.float8_e4m3fn:
            raise ValueError("k_pages of float8_e4m3fn need k_scales and v_scales")
        if not e4m3 and k_pages.dtype not in (torch.bfloat16, torch.float16):
            raise TypeError(f"k_pages must be bfloat16 or float16, got {k_pages.dtype}")
        if v_pages.dtype != k_pages.dtype:
            raise TypeError(f"v_pages must be {k_pages.dtype}, got {v_pages.dtype}")
        if k_pages.dim() != 4 or v_pages.shape != k_pages.shape:
            raise ValueError("k_pages and v_pages must have one shape [num_pages, page_size, "
                             "kv_heads, head_dim]")
        n, page, heads, dim = k_pages.shape
        if n < 1 or heads < 1:
            raise ValueError("a pool needs a page and a head")
        if page < 16 or page > 4096 or page & (page - 1):
            raise ValueError(f"page_size must be a power of two from 16 to 4096, got {page}")
        unit = 16 if e4m3 else 8
        if dim < unit or dim > SV_MAX_HEAD_DIM or dim % unit:
            raise ValueError(f"head_dim must be a multiple of {unit} up to {SV_MAX_HEAD_DIM}, got {dim}")
        for name, t in (("k_pages", k_pages), ("v_pages", v_pages)):
            if t.stride(3) != 1 or any(s <= 0 or s % unit for s in t.stride()[:3]) or t.data_ptr() % 16:
                raise ValueError(f"{name} must be 16-byte aligned with contiguous heads and "
                                 f"strides that are multiples of {unit}")
            order = sorted(range(4), key=lambda i: t.stride(i))
            reach = 0
            for i in order:
                if t.shape[i] > 1:
                    if t.stride(i) <= reach:
                        raise ValueError(f"{name} overlaps itself")
                    reach += (t.shape[i] - 1) * t.stride(i)
        if page_table.dim() != 2 or page_table.dtype != torch.int32 or not page_table.is_contiguous():
            raise ValueError("page_table must be a contiguous int32 [batch, max_pages]")
        B, width = page_table.shape
        _dev(kv_len, "kv_len", torch.int32, (B,))
        self.block, self.scales_ref = 0, None
        if e4m3:
            per = k_scales.shape[1] if isinstance(k_scales, torch.Tensor) and k_scales.dim() == 3 else 0
            self.block = page // per if per and page % per == 0 else 0
            if not 0 < self.block <= SV_MAX_BLOCK:  # (page and so block are powers of two)
                raise ValueError("k_scales must be [num_pages, page_size / block, kv_heads] with a block of at "
                                 f"most {SV_MAX_BLOCK} tokens")
            self._scales = _KvScales(_arg(k_scales, "k_scales", torch.float32, (n, per, heads), self.index),
                                     _arg(v_scales, "v_scales", torch.float32, (n, per, heads), self.index), self.block)
            self.scales_ref = ctypes.byref(self._scales)
        self._tensors = (k_pages, v_pages, page_table, kv_len, k_scales, v_scales)
        self.cu_shape = (B + 1,)
        self.sizes = (self.index, n, B, width)  # device, pages, rows, pages of a row
        self.batch, self.kv_heads, self.head_dim, self.dtype = B, heads, dim, k_pages.dtype
        self.page_size, self.scale = page, dim ** -0.5
        ptr = lambda t: t.data_ptr() if t.numel() else None  # noqa: E731
        self.struct = _KvCache(
            k_pages.data_ptr(), v_pages.data_ptr(),
            SV_E4M3 if e4m3 else SV_BF16 if k_pages.dtype == torch.bfloat16 else SV_F16, n, page, heads, dim,
            (ctypes.c_int64 * 3)(*k_pages.stride()[:3]), (ctypes.c_int64 * 3)(*v_pages.stride()[:3]),
            ptr(page_table), width, B, ptr(kv_len))
        self.ref = ctypes.byref(self.struct)

    def commit(self, num_accepted) -> None:
        """After a verification: every request keeps its last token and its accepted
        drafts (kv_len += num_accepted + 1); the rejected drafts' entries lie behind the
        new length and are overwritten by the next append.  On the current stream."""
        self.kv_len.add_(num_accepted).add_(1)


def make_attention_workspace(total_rows: int, q_heads: int, head_dim: int,
                             device="cuda") -> torch.Tensor:
    """Workspace of spec_verify_attention for steps of up to total_rows rows."""
    n = int(load_library().spec_verify_attention_workspace_size(int(total_rows), int(q_heads),
                                                                int(head_dim)))
    if n == 0:
        raise ValueError(f"invalid sizes rows={total_rows} q_heads={q_heads} head_dim={head_dim}")
    ws = torch.empty(n, dtype=torch.uint8, device=device)
    ws[:256].zero_()
    return ws


def make_attention_e4m3_workspace(total_rows: int, q_heads: int, head_dim: int,
                                  device="cuda") -> torch.Tensor:
    """Workspace of spec_verify_attention_e4m3 for steps of up to total_rows rows."""
    n = int(load_library().spec_verify_attention_e4m3_workspace_size(int(total_rows), int(q_heads),
                                                                     int(head_dim)))
    if n == 0:
        raise ValueError(f"invalid sizes rows={total_rows} q_heads={q_heads} head_dim={head_dim}")
    ws = torch.empty(n, dtype=torch.uint8, device=device)
    ws[:256].zero_()
    return ws


def _heads(t, name, cache, shape, dtype=None):
    """Address and (row, head) strides of a [rows, heads, head_dim] view of that shape, of the
    cache's type or of `dtype`."""
    dtype = dtype or cache.dtype
    if (isinstance(t, torch.Tensor) and t.dtype is dtype and t.get_device() == cache.index
            and t.shape == shape):
        row, head, one = t.stride()
        if one == 1:
            return t.data_ptr(), _two(row, head)
    if _index(t, name) != cache.index:
        raise ValueError(f"{name} is on {t.device}, the cache on cuda:{cache.index}")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if tuple(t.shape) != shape:
        raise ValueError(f"{name} must have shape {shape}, got {tuple(t.shape)}")
    raise ValueError(f"{name} must have contiguous heads")


def _cu_rows(cu_draft, cache, rows):
    if rows < cache.batch:
        raise ValueError(f"a step of {cache.batch} requests has at least as many rows, got {rows}")
    return _arg(cu_draft, "cu_draft", torch.int32, cache.cu_shape, cache.index)


def _rows16(t, name):
    """The type of rows beside a cache in 8 bits, and its code."""
    dtype = getattr(t, "dtype", None)
    if dtype is torch.bfloat16:
        return dtype, SV_BF16
    if dtype is torch.float16:
        return dtype, SV_F16
    raise TypeError(f"{name} must be bfloat16 or float16, got {dtype or type(t).__name__}")


def _in_8_bits(cache):
    if cache.scales_ref is None:
        raise TypeError("the cache must hold float8_e4m3fn with scales")


def spec_verify_kv_append(q, k, v, cache, cu_draft, max_drafts, freq, q_out, workspace,
                          interleaved=False, rope_scale=1.0, positions=None, position_offset=0,
                          stream=None) -> None:
    """Append a step's keys and values to the paged cache and rotate its queries and keys;
    q and q_out may be None, freq (rope.fixed_point) None for no rotation.  q_out is q
    itself or overlaps none of q, k and v.  To a cache in 8 bits q, k, v and q_out are
    bfloat16 or float16 (spec_verify_kv_append_e4m3).  See include/spec_verify.h."""
    index, dtype, dim, scales = cache.index, cache.dtype, cache.head_dim, cache.scales_ref
    if scales is not None:
        dtype, code = _rows16(k, "k")
    if (q is None) != (q_out is None):
        raise ValueError("q and q_out go together")
    _index(k, "k")
    rows = k.shape[0]
    cu = _cu_rows(cu_draft, cache, rows)
    shape = (rows, cache.kv_heads, dim)
    ks, vs = k.stride(), v.stride()
    if not (k.shape == shape and v.shape == shape and k.dtype is dtype and v.dtype is dtype
            and k.get_device() == index and v.get_device() == index and ks[2] == 1 and vs[2] == 1):
        _heads(k, "k", cache, shape, dtype)
        _heads(v, "v", cache, shape, dtype)
    heads, qp, qs, op, os_ = 0, None, None, None, None
    if q is not None:
        heads = q.shape[1]
        shape = (rows, heads, dim)
        qs, os_ = q.stride(), q_out.stride()
        if not (q.shape == shape and q_out.shape == shape and q.dtype is dtype and q_out.dtype is dtype
                and q.get_device() == index and q_out.get_device() == index and qs[2] == 1
                and os_[2] == 1):
            _heads(q, "q", cache, shape, dtype)
            _heads(q_out, "q_out", cache, shape, dtype)
        row, head = os_[0], os_[1]
        if ((rows > 1 and row < dim) or (heads > 1 and head < dim)
                or (rows > 1 and heads > 1 and row < (heads - 1) * head + dim
                    and head < (rows - 1) * row + dim)):
            raise ValueError("q_out overlaps itself")
        qp, qs, op, os_ = q.data_ptr(), _two(qs[0], qs[1]), q_out.data_ptr(), _two(os_[0], os_[1])
    rot, fp = 0, None
    if freq is not None:
        half = freq.numel()
        rot, fp = 2 * half, _arg(freq, "freq", torch.int64, (half,), index)
    if scales is not None:
        _launch((_lib or load_library()).spec_verify_kv_append_e4m3, index, stream,
                qp, qs, heads, k.data_ptr(), _two(ks[0], ks[1]), v.data_ptr(), _two(vs[0], vs[1]), code, op, os_,
                cache.ref, scales, cu, rows - cache.batch, max_drafts, fp, rot, 1 if interleaved else 0, rope_scale,
                None if positions is None else _arg(positions, "positions", torch.int32, (rows,), index),
                position_offset, _arg(workspace, "workspace", torch.uint8, None, index), workspace.numel())
        return
    _launch((_lib or load_library()).spec_verify_kv_append, index, stream,
            qp, qs, heads, k.data_ptr(), _two(ks[0], ks[1]), v.data_ptr(), _two(vs[0], vs[1]), op, os_,
            cache.ref, cu, rows - cache.batch, max_drafts, fp, rot, 1 if interleaved else 0, rope_scale,
            None if positions is None else _arg(positions, "positions", torch.int32, (rows,), index),
            position_offset, _arg(workspace, "workspace", torch.uint8, None, index), workspace.numel())


def spec_verify_kv_append_e4m3(q, k, v, cache, cu_draft, max_drafts, freq, q_out, workspace, **more) -> None:
    """spec_verify_kv_append to a cache in 8 bits, and to no other: keys and values are stored as
    codes with a scale for each block of tokens and head.  See include/spec_verify.h."""
    _in_8_bits(cache)
    spec_verify_kv_append(q, k, v, cache, cu_draft, max_drafts, freq, q_out, workspace, **more)


def spec_verify_attention(q, cache, cu_draft, max_drafts, out, workspace, prefix_table=None,
                          prefix_len=0, scale=None, draft_mask=None, lse=None, stream=None) -> None:
    """Attention of a step's rows over the paged cache (and a prefix that the batch shares);
    scale None: head_dim ** -0.5; out may not lie within q.  Over a cache in 8 bits q and out
    are bfloat16 or float16, the workspace is make_attention_e4m3_workspace's
    (spec_verify_attention_e4m3).  See include/spec_verify.h."""
    index, dtype, scales = cache.index, cache.dtype, cache.scales_ref
    _index(q, "q")
    if scales is not None:
        dtype, code = _rows16(q, "q")
    rows, heads = q.shape[0], q.shape[1]
    cu = _cu_rows(cu_draft, cache, rows)
    shape = (rows, heads, cache.head_dim)
    qp, qs = _heads(q, "q", cache, shape, dtype)
    pt = mask = None
    if prefix_len > 0:
        if not isinstance(prefix_table, torch.Tensor) or prefix_table.numel() * cache.page_size < prefix_len:
            raise ValueError(f"prefix_table must hold {-(-prefix_len // cache.page_size)} pages")
        pt = _arg(prefix_table, "prefix_table", torch.int32, None, index)
    if draft_mask is not None:
        if getattr(draft_mask, "dtype", None) not in (torch.int32, torch.uint32):
            raise TypeError("draft_mask must be int32 or uint32 words")
        mask = _arg(draft_mask, "draft_mask", draft_mask.dtype, (rows,), index)
    if scales is not None:
        _launch((_lib or load_library()).spec_verify_attention_e4m3, index, stream,
                qp, qs, heads, code, cache.ref, scales, pt, prefix_len, cu, rows - cache.batch, max_drafts,
                cache.scale if scale is None else scale, mask, _arg(out, "out", dtype, shape, index),
                None if lse is None else _arg(lse, "lse", torch.float32, (rows, heads), index),
                _arg(workspace, "workspace", torch.uint8, None, index), workspace.numel())
        return
    _launch((_lib or load_library()).spec_verify_attention, index, stream,
            qp, qs, heads, cache.ref, pt, prefix_len, cu, rows - cache.batch, max_drafts,
            cache.scale if scale is None else scale, mask,
            _arg(out, "out", dtype, shape, index),
            None if lse is None else _arg(lse, "lse", torch.float32, (rows, heads), index),
            _arg(workspace, "workspace", torch.uint8, None, index), workspace.numel())


def spec_verify_attention_e4m3(q, cache, cu_draft, max_drafts, out, workspace, **more) -> None:
    """spec_verify_attention over a cache in 8 bits, and over no other.  See
    include/spec_verify.h."""
    _in_8_bits(cache)
    spec_verify_attention(q, cache, cu_draft, max_drafts, out, workspace, **more)


class PagePool:
    """Who holds which pages of a cache's pool, on the device: held [batch] (pages of each row of
    the page table, its first ones), ref [num_pages] (rows that hold a page), free_pages
    [num_pages] (the free pages, in its first entries) and free_count [1], all int32.

    PagePool(cache) starts with every page free and rows that hold none;
    PagePool.of_table(cache, held) takes up a page table that is filled already.  The tensors
    may also be the caller's own, all four (used in place; the attributes may not be assigned).
    A pool serves caches of the device, pages, rows and table width that it was made for.
    """
    held = property(lambda self: self._tensors[0])
    ref = property(lambda self: self._tensors[1])
    free_pages = property(lambda self: self._tensors[2])
    free_count = property(lambda self: self._tensors[3])

    def __init__(self, cache, held=None, ref=None, free_pages=None, free_count=None):
        self.sizes = index, n, B, width = cache.sizes
        given = [t is not None for t in (held, ref, free_pages, free_count)]
        if any(given) and not all(given):  # (they describe one state)
            raise ValueError("held, ref, free_pages and free_count go together")
        dev, i32 = torch.device("cuda", index), torch.int32
        if held is None:
            held = torch.zeros((B,), dtype=i32, device=dev)
            ref = torch.zeros((n,), dtype=i32, device=dev)
            free_pages = torch.arange(n - 1, -1, -1, dtype=i32, device=dev)  # page 0 is taken first
            free_count = torch.full((1,), n, dtype=i32, device=dev)
        ptrs = (_arg(held, "held", i32, (B,), index) or None, _arg(ref, "ref", i32, (n,), index),
                _arg(free_pages, "free_pages", i32, (n,), index), _arg(free_count, "free_count", i32, (1,), index))
        self.struct = _PagePool(*ptrs)
        self.ref_struct = ctypes.byref(self.struct)
        self._tensors = (held, ref, free_pages, free_count)
        size = int(load_library().spec_verify_pages_workspace_size(n, B, width))
        if size == 0:
            raise ValueError(f"no page pool for {B} rows of {width} pages")
        self.workspace = torch.zeros(size, dtype=torch.uint8, device=dev)

    @classmethod
    def of_table(cls, cache, held, prefix_table=None):
        """The pool of a page table whose rows hold their first held[b] entries already;
        a prefix that the batch shares counts as a row of its own.  (Synchronises.)"""
        n = cache.struct.num_pages
        held = held.to(torch.int32)
        table = cache.page_table
        mine = torch.arange(table.shape[1], device=table.device)[None, :] < held[:, None]
        pages = table[mine].long()
        if prefix_table is not None:
            pages = torch.cat([pages, prefix_table.long().flatten()])
        if pages.numel() and (int(pages.min()) < 0 or int(pages.max()) >= n):
            raise ValueError("the rows hold pages outside the pool")
        ref = torch.bincount(pages, minlength=n).int()
        free = (ref == 0).nonzero()[:, 0].flip(0).int()
        room = torch.full((n,), -1, dtype=torch.int32, device=table.device)
        room[:free.numel()] = free
        count = torch.full((1,), free.numel(), dtype=torch.int32, device=table.device)
        return cls(cache, held.contiguous(), ref, room, count)


def _of_one_size(cache, pool):
    if pool.sizes != cache.sizes:
        raise ValueError("the pool was made for another cache: device, pages, rows and table width are "
                         f"{pool.sizes}, the cache's {cache.sizes}")


def spec_verify_pages_step(cache, pool, tokens, parents=None, stream=None) -> None:
    """The page table of the next step: row b continues row parents[b] (-1: it ends; None: every
    row itself), gives back what lies behind its tokens and holds pages for tokens[b] more, with
    a copy of a partly filled page that others hold.  The status word is in pool.workspace.
    See include/spec_verify.h."""
    _of_one_size(cache, pool)
    index, i32, shape = cache.index, torch.int32, (cache.batch,)
    _launch((_lib or load_library()).spec_verify_pages_step, index, stream, cache.ref,
            cache.scales_ref, pool.ref_struct,
            None if parents is None else _arg(parents, "parents", i32, shape, index),
            _arg(tokens, "tokens", i32, shape, index), pool.workspace.data_ptr(), pool.workspace.numel())


def spec_verify_pages_compact(cache, pool, remap, stream=None) -> None:
    """The pages in use move to the front of the pool; remap [num_pages] int32 receives each
    page's new place (-1: it was free).  See include/spec_verify.h."""
    _of_one_size(cache, pool)
    _launch((_lib or load_library()).spec_verify_pages_compact, cache.index, stream, cache.ref,
            cache.scales_ref, pool.ref_struct,
            _arg(remap, "remap", torch.int32, (cache.struct.num_pages,), cache.index), pool.workspace.data_ptr(),
            pool.workspace.numel())


def spec_verify_status(workspace, stream=None) -> int:
    """Read and clear the workspace status word (synchronises the stream)."""
    out = ctypes.c_uint32(0)
    rc = load_library().spec_verify_status(_dev(workspace, "workspace", torch.uint8),
                                           _stream(stream), ctypes.byref(out))
    if rc != 0:
        raise SpecVerifyError(rc)
    return int(out.value)


def status_names(bits: int) -> list[str]:
    return [n for b, n in STATUS_BITS.items() if bits & b]


class Verifier:
    """Owns output buffers and a workspace for one (B, G, V) shape on one device."""

    def __init__(self, B: int, G: int, V: int, device="cuda"):
        self.B, self.G, self.V = B, G, V
        self.workspace = make_workspace(B, G, V, device)
        self.out_tokens = torch.empty((B, G + 1), dtype=torch.int32, device=device)
        self.num_accepted = torch.empty((B,), dtype=torch.int32, device=device)

    def sample(self, target, draft, draft_tokens, gamma, uniforms, temperature, p_tok=None,
               q_tok=None, stream=None):
        spec_verify_sample(target, draft, draft_tokens, gamma, uniforms, temperature,
                           self.out_tokens, self.num_accepted, self.workspace, p_tok, q_tok,
                           stream)
        return self.out_tokens, self.num_accepted

    def greedy(self, target, draft_tokens, gamma, stream=None):
        spec_verify_greedy(target, draft_tokens, gamma, self.out_tokens, self.num_accepted,
                           self.workspace, stream)
        return self.out_tokens, self.num_accepted

    def sample_packed(self, target, draft, cu_draft, draft_tokens, uniforms, temperature,
                      p_tok=None, q_tok=None, stream=None):
        spec_verify_sample_packed(target, draft, cu_draft, draft_tokens, uniforms, temperature,
                                  self.out_tokens, self.num_accepted, self.workspace, p_tok,
                                  q_tok, stream)
        return self.out_tokens, self.num_accepted

    def greedy_packed(self, target, cu_draft, draft_tokens, stream=None):
        spec_verify_greedy_packed(target, cu_draft, draft_tokens, self.out_tokens,
                                  self.num_accepted, self.workspace, stream)
        return self.out_tokens, self.num_accepted

    def sample_probs(self, target_probs, draft_probs, draft_tokens, gamma, uniforms, stream=None):
        spec_verify_sample_probs(target_probs, draft_probs, draft_tokens, gamma, uniforms,
                                 self.out_tokens, self.num_accepted, self.workspace, stream)
        return self.out_tokens, self.num_accepted

    def sample_probs_packed(self, target_probs, draft_probs, cu_draft, draft_tokens, uniforms,
                            stream=None):
        spec_verify_sample_probs_packed(target_probs, draft_probs, cu_draft, draft_tokens,
                                        uniforms, self.out_tokens, self.num_accepted,
                                        self.workspace, stream)
        return self.out_tokens, self.num_accepted
