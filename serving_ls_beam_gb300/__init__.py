"""Python binding of the ls_beam CUDA library (``libls_beam.so``).

Argument marshalling only: every function passes device pointers, sizes and the
stream handle to the C entry point of the same name (declared in
``include/ls_beam.h``) and returns its status code.  All computation happens in
the library's sm_103a kernels; there is no Python or CPU fallback, and a missing
library raises ``LsBeamError``.

PyTorch is used only for device memory and streams.
"""
from __future__ import annotations

import ctypes
import os
import threading

__all__ = [
    "LS_OK", "LS_ERR_INVALID_ARG", "LS_ERR_UNSUPPORTED", "LS_ERR_CUDA", "LS_ERR_TIMEOUT", "LS_ERR_INTERNAL",
    "LS_DTYPE_F32", "LS_DTYPE_F16", "LS_DTYPE_BF16", "LS_MAX_K", "LsBeamError", "library_path", "load_library",
    "check", "ls_beam_step_workspace_size", "ls_workspace_init", "ls_beam_step", "ls_cache_reorder",
    "ls_read_status", "ls_status_string", "ls_read_row_stats", "ls_beam_step_noalloc", "ls_beam_step_noalloc_status",
    "ls_backtrack",
    "ls_sample_workspace_size", "ls_sample", "ls_cache_refresh_inplace", "ls_logits_beam_step",
    "ls_beam_step_refresh_inplace", "LS_MAX_NODES", "ls_cross_attention_workspace_size", "ls_cross_attention",
    "ls_tree_attention_workspace_size", "ls_tree_attention", "ls_tree_commit", "LS_DTYPE_E4M3", "LS_DTYPE_I8", "LsPages",
    "ls_pages", "ls_paged_write", "ls_paged_read", "ls_paged_attention_workspace_size", "ls_paged_attention",
    "ls_sample_filtered",
]

LS_OK, LS_ERR_INVALID_ARG, LS_ERR_UNSUPPORTED, LS_ERR_CUDA, LS_ERR_TIMEOUT, LS_ERR_INTERNAL = range(6)
LS_DTYPE_F32, LS_DTYPE_F16, LS_DTYPE_BF16 = 0, 1, 2
LS_DTYPE_E4M3, LS_DTYPE_I8 = 3, 4  # a paged cache's
LS_MAX_K = 64
LS_MAX_NODES = 64

_HERE = os.path.dirname(os.path.abspath(__file__))
_lock = threading.Lock()
_lib = None


class LsBeamError(RuntimeError):
    pass


class _View(ctypes.Structure):
    """ls_view: a device pointer and the element strides of [layer, row, pos, head, head_dim]."""
    _fields_ = [("data", ctypes.c_void_p), ("layer", ctypes.c_int64), ("row", ctypes.c_int64), ("pos", ctypes.c_int64),
                ("head", ctypes.c_int64)]


class _Pages(ctypes.Structure):
    """ls_pages: the views of a paged cache, its table and sizes."""
    _fields_ = [("key", _View), ("value", _View), ("key_scale", _View), ("value_scale", _View),
                ("table", ctypes.c_void_p), ("table_row", ctypes.c_int64), ("dtype", ctypes.c_int),
                ("num_pages", ctypes.c_int), ("page_size", ctypes.c_int), ("max_pages", ctypes.c_int),
                ("kv_heads", ctypes.c_int), ("head_dim", ctypes.c_int)]


def library_path() -> str:
    return os.path.join(_HERE, "libls_beam.so")


def load_library():
    """Load libls_beam.so (built by ``__graft_entry__.build()``); raise if it is missing."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is not None:
            return _lib
        path = library_path()
        if not os.path.exists(path):
            raise LsBeamError(f"CUDA library not built: {path} is missing (run __graft_entry__.build())")
        lib = ctypes.CDLL(path)
        vp, ip, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
        lib.ls_beam_step_workspace_size.argtypes = [ip, ip, ip]
        lib.ls_beam_step_workspace_size.restype = sz
        lib.ls_workspace_init.argtypes = [vp, sz, vp]
        lib.ls_workspace_init.restype = ip
        lib.ls_beam_step.argtypes = [vp, ip, vp, vp, vp, ip, ip, ip, ip, vp, vp, vp, vp, vp, sz, vp]
        lib.ls_beam_step.restype = ip
        lib.ls_cache_reorder.argtypes = [vp, vp, ip, vp, ip, ip, ip, ip, ip, ip, ip, vp, vp]
        lib.ls_cache_reorder.restype = ip
        lib.ls_read_status.argtypes = [vp, vp]
        lib.ls_read_status.restype = ip
        lib.ls_status_string.argtypes = [ip]
        lib.ls_status_string.restype = ctypes.c_char_p
        lib.ls_read_row_stats.argtypes = [vp, ip, ip, ip, vp, vp, vp, vp, vp]
        lib.ls_read_row_stats.restype = ip
        lib.ls_beam_step_noalloc.argtypes = [vp, ip, vp, vp, vp, ip, ip, ip, ip, vp, vp, vp, vp, vp]
        lib.ls_beam_step_noalloc.restype = ip
        lib.ls_beam_step_noalloc_status.argtypes = [vp]
        lib.ls_beam_step_noalloc_status.restype = ip
        lib.ls_backtrack.argtypes = [vp, vp, ip, ip, ip, ip, vp, vp, vp, vp]
        lib.ls_backtrack.restype = ip
        lib.ls_sample_workspace_size.argtypes = [ip, ip, ip]
        lib.ls_sample_workspace_size.restype = sz
        lib.ls_sample.argtypes = [vp, ip, vp, vp, ip, ip, ip, ctypes.c_float, vp, vp, vp, sz, vp]
        lib.ls_sample.restype = ip
        lib.ls_cache_refresh_inplace.argtypes = [vp, ip, vp, ip, ip, ip, ip, ip, ip, ip, vp, vp]
        lib.ls_cache_refresh_inplace.restype = ip
        lib.ls_logits_beam_step.argtypes = [vp, vp, ip, ip, vp, vp, vp, ip, ip, ip, ip, vp, vp, vp, vp, vp, sz, vp]
        lib.ls_logits_beam_step.restype = ip
        lib.ls_beam_step_refresh_inplace.argtypes = [vp, ip, vp, vp, vp, ip, ip, ip, ip, vp, vp, vp, vp, vp, ip, ip,
                                                     ip, ip, ip, ip, vp, sz, vp]
        lib.ls_beam_step_refresh_inplace.restype = ip
        view, fl = ctypes.POINTER(_View), ctypes.c_float
        lib.ls_cross_attention_workspace_size.argtypes = [ip] * 7
        lib.ls_cross_attention_workspace_size.restype = sz
        lib.ls_cross_attention.argtypes = [view, view, view, ip, vp, fl, ip, ip, ip, ip, ip, ip, ip, view, vp, sz, vp]
        lib.ls_cross_attention.restype = ip
        lib.ls_tree_attention_workspace_size.argtypes = [ip] * 6
        lib.ls_tree_attention_workspace_size.restype = sz
        lib.ls_tree_attention.argtypes = [view, view, view, vp, view, view, vp, ip, fl, ip, ip, ip, ip, ip, ip, view,
                                          vp, sz, vp]
        lib.ls_tree_attention.restype = ip
        lib.ls_tree_commit.argtypes = [vp, vp, vp, view, view, ip, vp, vp, vp, vp, ip, ip, ip, ip, ip, ip, ip, vp, vp,
                                       vp, vp, vp, vp, vp]
        lib.ls_tree_commit.restype = ip
        pages = ctypes.POINTER(_Pages)
        lib.ls_paged_write.argtypes = [view, view, ip, vp, vp, pages, ip, ip, vp, vp]
        lib.ls_paged_write.restype = ip
        lib.ls_paged_read.argtypes = [pages, vp, vp, view, view, ip, ip, ip, vp, vp]
        lib.ls_paged_read.restype = ip
        lib.ls_paged_attention_workspace_size.argtypes = [ip] * 4
        lib.ls_paged_attention_workspace_size.restype = sz
        lib.ls_paged_attention.argtypes = [view, pages, vp, ip, fl, ip, ip, view, vp, sz, vp]
        lib.ls_paged_attention.restype = ip
        lib.ls_sample_filtered.argtypes = [vp, ip, ctypes.c_int64, vp, vp, vp, vp, vp, vp, ip, ip, vp, vp, vp, vp]
        lib.ls_sample_filtered.restype = ip
        _lib = lib
        return lib


_codes: dict = {}


def _dtype_code(t) -> int:
    if not _codes:
        import torch

        _codes.update({torch.float32: LS_DTYPE_F32, torch.float16: LS_DTYPE_F16, torch.bfloat16: LS_DTYPE_BF16})
    code = _codes.get(t.dtype)
    if code is None:
        raise TypeError(f"unsupported dtype {t.dtype}")
    return code


def _ptr(t) -> int | None:
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _stream(stream) -> int | None:
    if stream is None:
        import torch

        # the handle alone, a tenth of the cost of torch.cuda.current_stream()'s object
        raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        if raw is not None and torch.cuda.is_initialized():
            return raw(torch._C._cuda_getDevice())
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def check(status: int, what: str = "ls_beam") -> None:
    if status != LS_OK:
        raise LsBeamError(f"{what}: {ls_status_string(status)} ({status})")


def ls_status_string(status: int) -> str:
    return load_library().ls_status_string(int(status)).decode()


def ls_beam_step_workspace_size(batch: int, k: int, vocab: int) -> int:
    return int(load_library().ls_beam_step_workspace_size(batch, k, vocab))


def ls_workspace_init(workspace, stream=None) -> int:
    return load_library().ls_workspace_init(_ptr(workspace), workspace.numel() * workspace.element_size(),
                                            _stream(stream))


def ls_beam_step(logits, bias, beam_scores, finished, eos_id: int, out_token, out_parent, out_score,
                 out_finished, workspace, stream=None) -> int:
    """logits [batch, k, vocab] (f32/f16/bf16), bias [vocab] f32 or None, beam_scores [batch, k] f32,
    finished [batch, k] uint8 or None, outputs [batch, k] (int32, int32, f32, uint8 or None),
    workspace a uint8 device tensor of ls_beam_step_workspace_size() bytes."""
    batch, k, vocab = logits.shape
    return load_library().ls_beam_step(
        _ptr(logits), _dtype_code(logits), _ptr(bias), _ptr(beam_scores), _ptr(finished), batch, k, vocab,
        int(eos_id), _ptr(out_token), _ptr(out_parent), _ptr(out_score), _ptr(out_finished), _ptr(workspace),
        workspace.numel() * workspace.element_size(), _stream(stream))


def ls_beam_step_refresh_inplace(logits, bias, beam_scores, finished, eos_id: int, out_token, out_parent, out_score,
                                 out_finished, cache, length: int, workspace, stream=None) -> int:
    """ls_beam_step, then the in-place refresh of cache [layers, batch*k, heads, max_len, head_dim] by
    out_parent over positions [0, length); one kernel where the step runs a batch per CTA."""
    batch, k, vocab = logits.shape
    layers, rows, heads, max_len, head_dim = cache.shape
    if rows != batch * k:
        raise ValueError("cache rows do not match batch * k")
    return load_library().ls_beam_step_refresh_inplace(
        _ptr(logits), _dtype_code(logits), _ptr(bias), _ptr(beam_scores), _ptr(finished), batch, k, vocab,
        int(eos_id), _ptr(out_token), _ptr(out_parent), _ptr(out_score), _ptr(out_finished), _ptr(cache),
        _dtype_code(cache), layers, heads, max_len, int(length), head_dim, _ptr(workspace),
        workspace.numel() * workspace.element_size(), _stream(stream))


def ls_logits_beam_step(hidden, weight, bias, beam_scores, finished, eos_id: int, out_token, out_parent, out_score,
                        out_finished, workspace, stream=None) -> int:
    """The beam step fused into the output projection: hidden [batch, k, dim] and weight [vocab, dim]
    (both f16 or both bf16, logits = hidden . weight^T, never stored); everything else as ls_beam_step.
    The workspace is the one of ls_beam_step_workspace_size(batch, k, vocab)."""
    batch, k, dim = hidden.shape
    vocab, dim_w = weight.shape
    if dim_w != dim or weight.dtype != hidden.dtype:
        raise ValueError("weight must be [vocab, dim] of the hidden states' dtype")
    return load_library().ls_logits_beam_step(
        _ptr(hidden), _ptr(weight), _dtype_code(hidden), dim, _ptr(bias), _ptr(beam_scores), _ptr(finished), batch, k,
        vocab, int(eos_id), _ptr(out_token), _ptr(out_parent), _ptr(out_score), _ptr(out_finished), _ptr(workspace),
        workspace.numel() * workspace.element_size(), _stream(stream))


def ls_beam_step_noalloc(logits, bias, beam_scores, finished, eos_id: int, out_token, out_parent, out_score,
                         out_finished, stream=None) -> int:
    """ls_beam_step for callers that cannot allocate: no workspace argument, the library's
    fixed device scratch is used instead (shapes needing more than 64 MiB are rejected)."""
    batch, k, vocab = logits.shape
    return load_library().ls_beam_step_noalloc(
        _ptr(logits), _dtype_code(logits), _ptr(bias), _ptr(beam_scores), _ptr(finished), batch, k, vocab,
        int(eos_id), _ptr(out_token), _ptr(out_parent), _ptr(out_score), _ptr(out_finished), _stream(stream))


def ls_beam_step_noalloc_status(stream=None) -> int:
    """Device-detected status of the last ls_beam_step_noalloc on the current device (read and
    cleared; synchronises the stream)."""
    return load_library().ls_beam_step_noalloc_status(_stream(stream))


def ls_cache_reorder(src, dst, parent, length: int, workspace=None, stream=None) -> int:
    """src, dst [layers, batch*k, heads, max_len, head_dim]; parent [batch, k] int32."""
    layers, rows, heads, max_len, head_dim = src.shape
    batch, k = parent.shape
    if batch * k != rows:
        raise ValueError("parent shape does not match cache rows")
    return load_library().ls_cache_reorder(
        _ptr(src), _ptr(dst), _dtype_code(src), _ptr(parent), layers, batch, k, heads, max_len, int(length),
        head_dim, _ptr(workspace), _stream(stream))


def ls_backtrack(token_hist, parent_hist, eos_id: int, out_seq, out_len, workspace=None, stream=None) -> int:
    """token_hist, parent_hist [steps, batch, k] int32; out_seq [batch, k, steps] int32; out_len [batch, k] int32."""
    steps, batch, k = token_hist.shape
    return load_library().ls_backtrack(_ptr(token_hist), _ptr(parent_hist), steps, batch, k, int(eos_id),
                                       _ptr(out_seq), _ptr(out_len), _ptr(workspace), _stream(stream))


def ls_sample_workspace_size(rows: int, top_k: int, vocab: int) -> int:
    return int(load_library().ls_sample_workspace_size(rows, top_k, vocab))


def ls_sample(logits, bias, u, top_k: int, top_p: float, out_token, out_logprob, workspace, stream=None) -> int:
    """logits [rows, vocab] (f32/f16/bf16), bias [vocab] f32 or None, u [rows] f32, out_token [rows] int32,
    out_logprob [rows] f32 or None, workspace a uint8 device tensor of ls_sample_workspace_size() bytes."""
    rows, vocab = logits.shape
    return load_library().ls_sample(_ptr(logits), _dtype_code(logits), _ptr(bias), _ptr(u), rows, vocab, int(top_k),
                                    float(top_p), _ptr(out_token), _ptr(out_logprob), _ptr(workspace),
                                    workspace.numel() * workspace.element_size(), _stream(stream))


def ls_cache_refresh_inplace(cache, parent, length: int, workspace=None, stream=None) -> int:
    """cache [layers, batch*k, heads, max_len, head_dim] (refreshed in place); parent [batch, k] int32."""
    layers, rows, heads, max_len, head_dim = cache.shape
    batch, k = parent.shape
    if batch * k != rows:
        raise ValueError("parent shape does not match cache rows")
    return load_library().ls_cache_refresh_inplace(
        _ptr(cache), _dtype_code(cache), _ptr(parent), layers, batch, k, heads, max_len, int(length), head_dim,
        _ptr(workspace), _stream(stream))


# The wrappers of the operators below run once per layer and token, where a small call's time is
# the host's: each checks its shapes in one expression and asks every tensor for its strides once.
def _index(t, shape, dtype) -> bool:
    """A device-side index array: of `shape` and `dtype`, contiguous."""
    return t.shape == shape and t.dtype is dtype and t.is_contiguous()


def _refuse(what: str, *tensors) -> None:
    raise ValueError(f"{what}: shapes, dtypes or layouts do not fit: "
                     + ", ".join(f"{tuple(t.shape)} {t.dtype} strides {t.stride()}" for t in tensors if t is not None))


def ls_cross_attention_workspace_size(batch: int, k: int, q_len: int, heads: int, kv_heads: int, max_src: int,
                                      head_dim: int) -> int:
    return int(load_library().ls_cross_attention_workspace_size(batch, k, q_len, heads, kv_heads, max_src, head_dim))


def ls_cross_attention(q, key, value, src_len, out, workspace, scale: float | None = None, stream=None) -> int:
    """Attention of the beams' queries q [batch, k, q_len, heads, head_dim] over their sentence's keys and values
    [batch, kv_heads, max_src, head_dim] (positions < src_len [batch] int32), into out of q's shape.  The tensors may
    be strided views (last dimension contiguous; q's and out's batch and k as one dimension).  scale: 1/sqrt(head_dim)
    by default.  workspace: ls_cross_attention_workspace_size() bytes."""
    import torch

    shape, dt = q.shape, q.dtype
    batch, k, q_len, heads, dim = shape
    _, kv_heads, max_src, _ = key.shape
    sq, sk, sv, so = q.stride(), key.stride(), value.stride(), out.stride()
    flat = batch == 1 or k == 1
    if not (key.shape == (batch, kv_heads, max_src, dim) and value.shape == key.shape and out.shape == shape
            and key.dtype is dt and value.dtype is dt and out.dtype is dt and _index(src_len, (batch,), torch.int32)
            and (dim == 1 or sq[4] == sk[3] == sv[3] == so[4] == 1)
            and (flat or (sq[0] == k * sq[1] and so[0] == k * so[1]))):
        _refuse("ls_cross_attention", q, key, value, src_len, out)
    r = 1 if k > 1 else 0
    return load_library().ls_cross_attention(
        _View(q.data_ptr(), 0, sq[r], sq[2], sq[3]), _View(key.data_ptr(), 0, sk[0], sk[2], sk[1]),
        _View(value.data_ptr(), 0, sv[0], sv[2], sv[1]), _dtype_code(q), src_len.data_ptr(),
        dim ** -0.5 if scale is None else scale, batch, k, q_len, heads, kv_heads, max_src, dim,
        _View(out.data_ptr(), 0, so[r], so[2], so[3]), workspace.data_ptr(),
        workspace.numel() * workspace.element_size(), _stream(stream))


def ls_tree_attention_workspace_size(rows: int, nodes: int, heads: int, kv_heads: int, max_len: int,
                                     head_dim: int) -> int:
    return int(load_library().ls_tree_attention_workspace_size(rows, nodes, heads, kv_heads, max_len, head_dim))


def ls_tree_attention(q, cache_key, cache_value, cache_len, draft_key, draft_value, parent, out, workspace,
                      scale: float | None = None, stream=None) -> int:
    """Attention of a tree of drafted tokens: q, out [rows, nodes, heads, head_dim] over one layer of the cache
    [rows, kv_heads, max_len, head_dim] (positions < cache_len [rows] int32) and over the drafted keys and values
    [rows, nodes, kv_heads, head_dim] of each node's own branch (parent [rows, nodes] int32: -1 follows the cache,
    below -1 an empty place).  nodes = 1 is the single-token step.  The tensors may be strided views (last dimension
    contiguous).  scale: 1/sqrt(head_dim) by default.  workspace: ls_tree_attention_workspace_size() bytes."""
    import torch

    shape, dt, i32 = q.shape, q.dtype, torch.int32
    rows, nodes, heads, dim = shape
    _, kv_heads, max_len, _ = cache_key.shape
    draft = (rows, nodes, kv_heads, dim)
    sq, sk, sv, so = q.stride(), cache_key.stride(), cache_value.stride(), out.stride()
    dk, dv = draft_key.stride(), draft_value.stride()
    if not (cache_key.shape == (rows, kv_heads, max_len, dim) and cache_value.shape == cache_key.shape
            and draft_key.shape == draft and draft_value.shape == draft and out.shape == shape
            and cache_key.dtype is dt and cache_value.dtype is dt and draft_key.dtype is dt and draft_value.dtype is dt
            and out.dtype is dt and _index(cache_len, (rows,), i32) and _index(parent, (rows, nodes), i32)
            and (dim == 1 or sq[3] == sk[3] == sv[3] == so[3] == dk[3] == dv[3] == 1)):
        _refuse("ls_tree_attention", q, cache_key, cache_value, cache_len, draft_key, draft_value, parent, out)
    return load_library().ls_tree_attention(
        _View(q.data_ptr(), 0, sq[0], sq[1], sq[2]), _View(cache_key.data_ptr(), 0, sk[0], sk[2], sk[1]),
        _View(cache_value.data_ptr(), 0, sv[0], sv[2], sv[1]), cache_len.data_ptr(),
        _View(draft_key.data_ptr(), 0, dk[0], dk[1], dk[2]), _View(draft_value.data_ptr(), 0, dv[0], dv[1], dv[2]),
        parent.data_ptr(), _dtype_code(q), dim ** -0.5 if scale is None else scale, rows, nodes, heads, kv_heads, max_len,
        dim, _View(out.data_ptr(), 0, so[0], so[1], so[2]), workspace.data_ptr(),
        workspace.numel() * workspace.element_size(), _stream(stream))


def ls_tree_commit(cache_key, cache_value, cache_len, draft_key, draft_value, parent, token, target, finished,
                   eos_id: int, out_len, out_path, out_count, out_token, out_finished=None, workspace=None,
                   stream=None) -> int:
    """Finds the branch of each row's tree that `target` confirms (parent, token, target [rows, nodes] int32) and
    appends its keys and values (draft_* [layers, rows, nodes, heads, head_dim], strided views) at position cache_len
    of the contiguous caches [layers, rows, heads, max_len, head_dim].  Outputs: out_len, out_count, out_token [rows]
    int32, out_path [rows, nodes] int32, out_finished [rows] uint8 or None; finished [rows] uint8 or None."""
    import torch

    dt, i32, u8 = cache_key.dtype, torch.int32, torch.uint8
    layers, rows, heads, max_len, dim = cache_key.shape
    tree = parent.shape
    nodes = tree[1]
    draft, row = (layers, rows, nodes, heads, dim), (rows,)
    dk, dv = draft_key.stride(), draft_value.stride()
    if not (cache_value.shape == cache_key.shape and cache_key.is_contiguous() and cache_value.is_contiguous()
            and draft_key.shape == draft and draft_value.shape == draft and (dim == 1 or dk[4] == dv[4] == 1)
            and cache_value.dtype is dt and draft_key.dtype is dt and draft_value.dtype is dt and tree[0] == rows
            and _index(parent, tree, i32) and _index(token, tree, i32) and _index(target, tree, i32)
            and _index(out_path, tree, i32) and _index(cache_len, row, i32) and _index(out_len, row, i32)
            and _index(out_count, row, i32) and _index(out_token, row, i32)
            and (finished is None or _index(finished, row, u8))
            and (out_finished is None or _index(out_finished, row, u8))):
        _refuse("ls_tree_commit", cache_key, cache_value, cache_len, draft_key, draft_value, parent, token, target,
                finished, out_len, out_path, out_count, out_token, out_finished)
    return load_library().ls_tree_commit(
        cache_key.data_ptr(), cache_value.data_ptr(), cache_len.data_ptr(),
        _View(draft_key.data_ptr(), dk[0], dk[1], dk[2], dk[3]), _View(draft_value.data_ptr(), dv[0], dv[1], dv[2], dv[3]),
        _dtype_code(cache_key), parent.data_ptr(), token.data_ptr(), target.data_ptr(), _ptr(finished), eos_id, layers,
        rows, nodes, heads, max_len, dim, out_len.data_ptr(), out_path.data_ptr(), out_count.data_ptr(),
        out_token.data_ptr(), _ptr(out_finished), _ptr(workspace), _stream(stream))


class LsPages:
    """One layer's cache in pages, as the calls below take it: the C structure, made once, and the tensors that it points
    to.  Holds no state of its own: what the tensors hold may change between calls, their memory may not."""

    __slots__ = ("c", "ref", "tensors", "rows", "row", "kv_heads", "head_dim", "dtype", "coded", "int32")

    def __init__(self, key, value, table, key_scale=None, value_scale=None):
        import torch

        codes = {torch.float32: LS_DTYPE_F32, torch.float16: LS_DTYPE_F16, torch.bfloat16: LS_DTYPE_BF16,
                 torch.float8_e4m3fn: LS_DTYPE_E4M3, torch.int8: LS_DTYPE_I8}
        if key.dtype not in codes:
            raise TypeError(f"unsupported dtype {key.dtype}")
        code = codes[key.dtype]
        self.coded = code in (LS_DTYPE_E4M3, LS_DTYPE_I8)
        ok = (key.dim() == 4 and value.shape == key.shape and value.dtype is key.dtype and table.dim() == 2
              and table.dtype is torch.int32 and (table.shape[1] <= 1 or table.stride(1) == 1)
              and (key.shape[3] == 1 or key.stride(3) == value.stride(3) == 1)
              and (key_scale is not None) == (value_scale is not None) == self.coded)
        if ok and self.coded:
            ok = (key_scale.shape == key.shape[:3] and value_scale.shape == key.shape[:3]
                  and key_scale.dtype is torch.float32 and value_scale.dtype is torch.float32)
        if not ok:
            _refuse("ls_pages", key, value, table, key_scale, value_scale)

        def view(t):
            return _View() if t is None else _View(t.data_ptr(), 0, t.stride(0), t.stride(2), t.stride(1))

        pages, heads, size, dim = key.shape
        self.rows, self.kv_heads, self.head_dim, self.dtype = table.shape[0], heads, dim, key.dtype
        self.tensors = (key, value, table, key_scale, value_scale)
        self.c = _Pages(view(key), view(value), view(key_scale), view(value_scale), table.data_ptr(), table.stride(0), code,
                        pages, size, table.shape[1], heads, dim)
        self.ref, self.row, self.int32 = ctypes.byref(self.c), (self.rows,), torch.int32


def ls_pages(key, value, table, key_scale=None, value_scale=None) -> LsPages:
    """A cache's pages key, value [num_pages, kv_heads, page_size, head_dim] (f32, f16, bf16, float8_e4m3fn or int8; strided
    views with the last dimension contiguous, so a [num_pages, page_size, kv_heads, head_dim] tensor goes in as its
    transpose(1, 2)), for the 8-bit types with the scales [num_pages, kv_heads, page_size] f32 (strided views too), and the
    table [rows, max_pages] int32 of each row's pages."""
    return LsPages(key, value, table, key_scale, value_scale)


def ls_paged_write(key, value, start, count, pages: LsPages, workspace=None, stream=None) -> int:
    """New tokens key, value [rows, tokens, kv_heads, head_dim] (f32, f16 or bf16 strided views; the pages' own type where
    that is not an 8-bit one) to the positions start [rows] int32 and on of their rows' pages, the first count [rows] int32
    of each row (None: all), quantised where the pages have 8 bits."""
    shape, dt, i32, row = key.shape, key.dtype, pages.int32, pages.row
    rows, tokens, heads, dim = shape
    sk, sv = key.stride(), value.stride()
    if not (rows == pages.rows and heads == pages.kv_heads and dim == pages.head_dim and value.shape == shape
            and value.dtype is dt and (pages.coded or dt is pages.dtype) and (dim == 1 or sk[3] == sv[3] == 1)
            and _index(start, row, i32) and (count is None or _index(count, row, i32))):
        _refuse("ls_paged_write", key, value, start, count)
    return load_library().ls_paged_write(
        _View(key.data_ptr(), 0, sk[0], sk[1], sk[2]), _View(value.data_ptr(), 0, sv[0], sv[1], sv[2]), _dtype_code(key),
        start.data_ptr(), _ptr(count), pages.ref, rows, tokens, _ptr(workspace), _stream(stream))


def ls_paged_read(pages: LsPages, start, count, key, value, workspace=None, stream=None) -> int:
    """Positions start (None: 0) and on of every row, count [rows] int32 (None: all) of them, into key, value [rows, tokens,
    kv_heads, head_dim] (f32, f16 or bf16 strided views); what lies behind a row's count stays as it is."""
    shape, dt, i32, row = key.shape, key.dtype, pages.int32, pages.row
    rows, tokens, heads, dim = shape
    sk, sv = key.stride(), value.stride()
    if not (rows == pages.rows and heads == pages.kv_heads and dim == pages.head_dim and value.shape == shape
            and value.dtype is dt and (pages.coded or dt is pages.dtype) and (dim == 1 or sk[3] == sv[3] == 1)
            and (start is None or _index(start, row, i32)) and (count is None or _index(count, row, i32))):
        _refuse("ls_paged_read", key, value, start, count)
    return load_library().ls_paged_read(
        pages.ref, _ptr(start), _ptr(count), _View(key.data_ptr(), 0, sk[0], sk[1], sk[2]),
        _View(value.data_ptr(), 0, sv[0], sv[1], sv[2]), _dtype_code(key), rows, tokens, _ptr(workspace), _stream(stream))


def ls_paged_attention_workspace_size(rows: int, heads: int, kv_heads: int, head_dim: int) -> int:
    return int(load_library().ls_paged_attention_workspace_size(rows, heads, kv_heads, head_dim))


def ls_paged_attention(q, pages: LsPages, length, out, workspace, scale: float | None = None, stream=None) -> int:
    """Attention of one new token per row: q, out [rows, heads, head_dim] (strided views, last dimension contiguous) over the
    positions < length [rows] int32 of the rows' pages.  scale: 1/sqrt(head_dim) by default.  workspace:
    ls_paged_attention_workspace_size() bytes."""
    shape, dt = q.shape, q.dtype
    rows, heads, dim = shape
    sq, so = q.stride(), out.stride()
    if not (rows == pages.rows and dim == pages.head_dim and heads % pages.kv_heads == 0 and out.shape == shape
            and out.dtype is dt and (pages.coded or pages.dtype is dt) and _index(length, pages.row, pages.int32)
            and (dim == 1 or sq[2] == so[2] == 1)):
        _refuse("ls_paged_attention", q, length, out)
    return load_library().ls_paged_attention(
        _View(q.data_ptr(), 0, sq[0], 0, sq[1]), pages.ref, length.data_ptr(), _dtype_code(q),
        dim ** -0.5 if scale is None else scale, rows, heads, _View(out.data_ptr(), 0, so[0], 0, so[1]),
        workspace.data_ptr(), workspace.numel() * workspace.element_size(), _stream(stream))


def ls_sample_filtered(logits, bias, u, temperature, top_k, top_p, min_p, out_token, out_logprob=None, workspace=None,
                       stream=None) -> int:
    """One token per row of logits [rows, vocab] (f32/f16/bf16; rows may be strided) with a temperature, top_k (0: off), top_p
    and min_p of its own: each [rows] (top_k int32, the others f32) or None for off, drawn at u [rows] f32.  bias [vocab]
    f32 or None, out_token [rows] int32, out_logprob [rows] f32 or None: of the probability that it was drawn with."""
    import torch

    rows, vocab = logits.shape
    f32, i32, row = torch.float32, torch.int32, (rows,)
    if not ((vocab <= 1 or logits.stride(1) == 1) and (bias is None or _index(bias, (vocab,), f32)) and _index(u, row, f32)
            and (temperature is None or _index(temperature, row, f32)) and (top_k is None or _index(top_k, row, i32))
            and (top_p is None or _index(top_p, row, f32)) and (min_p is None or _index(min_p, row, f32))
            and _index(out_token, row, i32) and (out_logprob is None or _index(out_logprob, row, f32))):
        _refuse("ls_sample_filtered", logits, bias, u, temperature, top_k, top_p, min_p, out_token, out_logprob)
    return load_library().ls_sample_filtered(
        _ptr(logits), _dtype_code(logits), logits.stride(0) if rows > 1 else vocab, _ptr(bias), _ptr(u), _ptr(temperature),
        _ptr(top_k), _ptr(top_p), _ptr(min_p), rows, vocab, _ptr(out_token), _ptr(out_logprob), _ptr(workspace),
        _stream(stream))


def ls_read_status(workspace, stream=None) -> int:
    return load_library().ls_read_status(_ptr(workspace), _stream(stream))


def ls_read_row_stats(workspace, batch: int, k: int, vocab: int, stream=None):
    """Host numpy arrays (lse, rtopk, ncand, path) of the last step run on `workspace`."""
    import numpy as np

    lse = np.empty(batch * k, np.float32)
    rt = np.empty(batch * k, np.float32)
    nc = np.empty(batch * k, np.int32)
    path = np.empty(batch, np.int32)
    st = load_library().ls_read_row_stats(_ptr(workspace), batch, k, vocab, lse.ctypes.data, rt.ctypes.data,
                                          nc.ctypes.data, path.ctypes.data, _stream(stream))
    check(st, "ls_read_row_stats")
    return lse.reshape(batch, k), rt.reshape(batch, k), nc.reshape(batch, k), path
