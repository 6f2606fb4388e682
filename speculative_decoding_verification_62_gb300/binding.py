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

SV_F32, SV_BF16, SV_F16 = 0, 1, 2
SV_MAX_GAMMA = 31
SV_MAX_HEAD_DIM = 128
SV_MAX_VOCAB = 1 << 24
STATUS_BITS = {1: "BAD_GAMMA", 2: "BAD_TOKEN", 4: "BAD_UNIFORM", 8: "BAD_TEMPERATURE",
               16: "NONFINITE_ROW", 32: "INTERNAL", 64: "TIMEOUT", 128: "BAD_PROB",
               256: "BAD_PAGE", 512: "BAD_LENGTH"}
SV_NOALLOC_SCRATCH_BYTES = 4 << 20
EXPORTS = ("spec_verify_workspace_size", "spec_verify_sample", "spec_verify_greedy",
           "spec_verify_sample_packed", "spec_verify_greedy_packed", "spec_verify_draw",
           "spec_verify_sample_noalloc", "spec_verify_status", "spec_verify_strerror",
           "spec_verify_set_schedule", "spec_verify_route", "spec_verify_cluster_size",
           "spec_verify_set_wait_limit", "spec_verify_set_lazy", "spec_verify_sample_probs",
           "spec_verify_sample_probs_packed", "spec_verify_kv_append", "spec_verify_attention",
           "spec_verify_attention_workspace_size")
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
    """
    k_pages = property(lambda self: self._tensors[0])
    v_pages = property(lambda self: self._tensors[1])
    page_table = property(lambda self: self._tensors[2])
    kv_len = property(lambda self: self._tensors[3])

    def __init__(self, k_pages, v_pages, page_table, kv_len):
        self.index = _index(k_pages, "k_pages")
        for name, t in (("v_pages", v_pages), ("page_table", page_table), ("kv_len", kv_len)):
            if _index(t, name) != self.index:
                raise ValueError(f"{name} is on {t.device}, k_pages on {k_pages.device}")
        if k_pages.dtype not in (torch.bfloat16, torch.float16):
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
        if dim < 8 or dim > SV_MAX_HEAD_DIM or dim % 8:
            raise ValueError(f"head_dim must be a multiple of 8 up to {SV_MAX_HEAD_DIM}, got {dim}")
        for name, t in (("k_pages", k_pages), ("v_pages", v_pages)):
            if t.stride(3) != 1 or any(s <= 0 or s % 8 for s in t.stride()[:3]) or t.data_ptr() % 16:
                raise ValueError(f"{name} must be 16-byte aligned with contiguous heads and "
                                 "strides that are multiples of 8")
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
        self._tensors = (k_pages, v_pages, page_table, kv_len)
        self.cu_shape = (B + 1,)
        self.batch, self.kv_heads, self.head_dim, self.dtype = B, heads, dim, k_pages.dtype
        self.page_size, self.scale = page, dim ** -0.5
        ptr = lambda t: t.data_ptr() if t.numel() else None  # noqa: E731
        self.struct = _KvCache(
            k_pages.data_ptr(), v_pages.data_ptr(),
            SV_BF16 if k_pages.dtype == torch.bfloat16 else SV_F16, n, page, heads, dim,
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


def _heads(t, name, cache, shape):
    """Address and (row, head) strides of a [rows, heads, head_dim] view of that shape."""
    if (isinstance(t, torch.Tensor) and t.dtype is cache.dtype and t.get_device() == cache.index
            and t.shape == shape):
        row, head, one = t.stride()
        if one == 1:
            return t.data_ptr(), _two(row, head)
    if _index(t, name) != cache.index:
        raise ValueError(f"{name} is on {t.device}, the cache on cuda:{cache.index}")
    if t.dtype != cache.dtype:
        raise TypeError(f"{name} must be {cache.dtype}, got {t.dtype}")
    if tuple(t.shape) != shape:
        raise ValueError(f"{name} must have shape {shape}, got {tuple(t.shape)}")
    raise ValueError(f"{name} must have contiguous heads")


def _cu_rows(cu_draft, cache, rows):
    if rows < cache.batch:
        raise ValueError(f"a step of {cache.batch} requests has at least as many rows, got {rows}")
    return _arg(cu_draft, "cu_draft", torch.int32, cache.cu_shape, cache.index)


def spec_verify_kv_append(q, k, v, cache, cu_draft, max_drafts, freq, q_out, workspace,
                          interleaved=False, rope_scale=1.0, positions=None, position_offset=0,
                          stream=None) -> None:
    """Append a step's keys and values to the paged cache and rotate its queries and keys;
    q and q_out may be None, freq (rope.fixed_point) None for no rotation.  q_out is q
    itself or overlaps none of q, k and v.  See include/spec_verify.h."""
    index, dtype, dim = cache.index, cache.dtype, cache.head_dim
    if (q is None) != (q_out is None):
        raise ValueError("q and q_out go together")
    _index(k, "k")
    rows = k.shape[0]
    cu = _cu_rows(cu_draft, cache, rows)
    shape = (rows, cache.kv_heads, dim)
    ks, vs = k.stride(), v.stride()
    if not (k.shape == shape and v.shape == shape and k.dtype is dtype and v.dtype is dtype
            and k.get_device() == index and v.get_device() == index and ks[2] == 1 and vs[2] == 1):
        _heads(k, "k", cache, shape)
        _heads(v, "v", cache, shape)
    heads, qp, qs, op, os_ = 0, None, None, None, None
    if q is not None:
        heads = q.shape[1]
        shape = (rows, heads, dim)
        qs, os_ = q.stride(), q_out.stride()
        if not (q.shape == shape and q_out.shape == shape and q.dtype is dtype and q_out.dtype is dtype
                and q.get_device() == index and q_out.get_device() == index and qs[2] == 1
                and os_[2] == 1):
            _heads(q, "q", cache, shape)
            _heads(q_out, "q_out", cache, shape)
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
    _launch((_lib or load_library()).spec_verify_kv_append, index, stream,
            qp, qs, heads, k.data_ptr(), _two(ks[0], ks[1]), v.data_ptr(), _two(vs[0], vs[1]), op, os_,
            cache.ref, cu, rows - cache.batch, max_drafts, fp, rot, 1 if interleaved else 0, rope_scale,
            None if positions is None else _arg(positions, "positions", torch.int32, (rows,), index),
            position_offset, _arg(workspace, "workspace", torch.uint8, None, index), workspace.numel())


def spec_verify_attention(q, cache, cu_draft, max_drafts, out, workspace, prefix_table=None,
                          prefix_len=0, scale=None, draft_mask=None, lse=None, stream=None) -> None:
    """Attention of a step's rows over the paged cache (and a prefix that the batch shares);
    scale None: head_dim ** -0.5; out may not lie within q.  See include/spec_verify.h."""
    index = cache.index
    _index(q, "q")
    rows, heads = q.shape[0], q.shape[1]
    cu = _cu_rows(cu_draft, cache, rows)
    shape = (rows, heads, cache.head_dim)
    qp, qs = _heads(q, "q", cache, shape)
    pt = mask = None
    if prefix_len > 0:
        if not isinstance(prefix_table, torch.Tensor) or prefix_table.numel() * cache.page_size < prefix_len:
            raise ValueError(f"prefix_table must hold {-(-prefix_len // cache.page_size)} pages")
        pt = _arg(prefix_table, "prefix_table", torch.int32, None, index)
    if draft_mask is not None:
        if getattr(draft_mask, "dtype", None) not in (torch.int32, torch.uint32):
            raise TypeError("draft_mask must be int32 or uint32 words")
        mask = _arg(draft_mask, "draft_mask", draft_mask.dtype, (rows,), index)
    _launch((_lib or load_library()).spec_verify_attention, index, stream,
            qp, qs, heads, cache.ref, pt, prefix_len, cu, rows - cache.batch, max_drafts,
            cache.scale if scale is None else scale, mask,
            _arg(out, "out", cache.dtype, shape, index),
            None if lse is None else _arg(lse, "lse", torch.float32, (rows, heads), index),
            _arg(workspace, "workspace", torch.uint8, None, index), workspace.numel())


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
