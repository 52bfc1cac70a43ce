"""ctypes binding of libtreeverify.so (argument marshalling only).

Every function here forwards torch tensors' device pointers and the current CUDA stream to the
C entry point of the same name declared in ``include/treeverify.h``; all arithmetic runs in the
library's CUDA kernels.  A missing or unloadable library raises ``RuntimeError``: there is no
fallback implementation.
"""

import ctypes
import os
import threading

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
# TV_LIB_CHECKED=1 loads the bounds-checked debug build of the same library instead
LIB_PATH = os.path.join(_PKG, "libtreeverify_checked.so" if os.environ.get("TV_LIB_CHECKED") == "1"
                        else "libtreeverify.so")

TV_OK = 0
TV_ERR = {
    -1: "TV_ERR_ARG", -2: "TV_ERR_SHAPE", -3: "TV_ERR_BAD_TREE", -4: "TV_ERR_CAPACITY",
    -5: "TV_ERR_DTYPE", -6: "TV_ERR_CUDA", -7: "TV_ERR_WORKSPACE", -8: "TV_ERR_TIMEOUT",
    -9: "TV_ERR_SELECTION", -10: "TV_ERR_BOUNDS", -11: "TV_ERR_VALUE",
}
TV_TAIL_WINDOW, TV_TAIL_REMAINDER = 0, 1
TV_COMP_C4, TV_COMP_C128 = 1, 2
TV_F32, TV_BF16 = 0, 1
TV_ATTN_AUTO, TV_ATTN_SIMT, TV_ATTN_TCGEN05 = 0, 1, 2
TV_ROPE_HALVES, TV_ROPE_PAIRS = 0, 1
_LOGIT_TYPES = {torch.float32: TV_F32, torch.bfloat16: TV_BF16}

EXPORTS = (
    "tv_version", "tv_status_string", "tv_last_error_string", "tv_workspace_size",
    "tv_attn_kernel_for",
    "tv_build_ancestor_mask", "tv_prefill_compress", "tv_branch_compress",
    "tv_tree_verify_attn", "tv_accept_walk", "tv_refresh_commit", "tv_tree_verify_attn_noalloc",
    "tv_indexer_workspace_size", "tv_indexer_topk", "tv_debug_attn_timeout", "tv_noalloc_prepare",
    "tv_token_logprobs", "tv_pages_workspace_size", "tv_pages_fork", "tv_pages_reserve",
    "tv_pages_compact", "tv_chunk_append", "tv_chunk_workspace_size", "tv_chunk_attn",
    "tv_beam_workspace_size", "tv_beam_select",
)


class tv_shape(ctypes.Structure):
    _fields_ = [
        ("B", ctypes.c_int32), ("D", ctypes.c_int32), ("H", ctypes.c_int32),
        ("d", ctypes.c_int32), ("W", ctypes.c_int32), ("tail_mode", ctypes.c_int32),
        ("comp_mask", ctypes.c_int32), ("dtype", ctypes.c_int32), ("n_sel", ctypes.c_int32),
        ("attn_kernel", ctypes.c_int32), ("raw_cap", ctypes.c_int64), ("c4_cap", ctypes.c_int64),
        ("c128_cap", ctypes.c_int64), ("page_tokens", ctypes.c_int32),
        ("max_pages", ctypes.c_int32), ("n_pool_pages", ctypes.c_int32),
        ("stage_chain", ctypes.c_int32), ("page_table", ctypes.c_void_p),
    ]


class TreeVerifyError(RuntimeError):
    def __init__(self, fn, code, message):
        super().__init__(f"{fn}: {TV_ERR.get(code, code)}: {message}")
        self.code = code


_lock = threading.Lock()
_lib = None

_P = ctypes.c_void_p
_SHAPE = ctypes.POINTER(tv_shape)
_SIGS = {
    "tv_version": ([], ctypes.c_char_p),
    "tv_status_string": ([ctypes.c_int], ctypes.c_char_p),
    "tv_last_error_string": ([], ctypes.c_char_p),
    "tv_workspace_size": ([_SHAPE], ctypes.c_size_t),
    "tv_attn_kernel_for": ([_SHAPE], ctypes.c_int),
    "tv_build_ancestor_mask": ([_SHAPE] + [_P] * 8 + [_P], ctypes.c_int),
    "tv_prefill_compress": ([_SHAPE] + [_P] * 10 + [_P], ctypes.c_int),
    "tv_branch_compress": ([_SHAPE] + [_P] * 15 + [_P], ctypes.c_int),
    "tv_tree_verify_attn": ([_SHAPE] + [_P] * 19 + [ctypes.c_float, _P, _P, _P, ctypes.c_size_t,
                                                    _P, _P], ctypes.c_int),
    "tv_tree_verify_attn_noalloc": ([_SHAPE] + [_P] * 19 + [ctypes.c_float, _P, _P, _P, _P],
                                    ctypes.c_int),
    "tv_accept_walk": ([_SHAPE] + [_P] * 7 + [_P], ctypes.c_int),
    "tv_refresh_commit": ([_SHAPE] + [_P] * 18 + [_P], ctypes.c_int),
    "tv_indexer_workspace_size": ([_SHAPE], ctypes.c_size_t),
    "tv_indexer_topk": ([_SHAPE, ctypes.c_int] + [_P] * 5 + [ctypes.c_size_t, _P, _P],
                        ctypes.c_int),
    "tv_noalloc_prepare": ([], ctypes.c_int),
    "tv_debug_attn_timeout": ([ctypes.c_int64, ctypes.c_int32], ctypes.c_int),
    "tv_token_logprobs": ([_SHAPE, ctypes.c_int32, ctypes.c_int64, ctypes.c_int32, _P,
                           ctypes.c_int32, _P, _P, ctypes.c_float, ctypes.c_int32] + [_P] * 8,
                          ctypes.c_int),
    "tv_pages_workspace_size": ([_SHAPE], ctypes.c_size_t),
    "tv_pages_fork": ([_SHAPE] + [_P] * 11 + [ctypes.c_int32, _P, ctypes.c_size_t, _P, _P],
                      ctypes.c_int),
    "tv_pages_reserve": ([_SHAPE] + [_P] * 4 + [ctypes.c_size_t, _P, _P], ctypes.c_int),
    "tv_pages_compact": ([_SHAPE] + [_P] * 11 + [ctypes.c_size_t, _P, _P], ctypes.c_int),
    "tv_chunk_append": ([_SHAPE, ctypes.c_int32] + [_P] * 3 + [ctypes.c_int64, _P, ctypes.c_int32,
                                                               ctypes.c_int32] + [_P] * 13,
                        ctypes.c_int),
    "tv_chunk_workspace_size": ([_SHAPE, ctypes.c_int32], ctypes.c_size_t),
    "tv_chunk_attn": ([_SHAPE, ctypes.c_int32] + [_P] * 9 + [ctypes.c_float, _P, _P, _P,
                                                             ctypes.c_size_t, _P, _P], ctypes.c_int),
    "tv_beam_workspace_size": ([_SHAPE, ctypes.c_int32], ctypes.c_size_t),
    "tv_beam_select": ([_SHAPE, ctypes.c_int32, ctypes.c_int32, ctypes.c_int64, ctypes.c_int32]
                       + [_P] * 3 + [ctypes.c_int32, ctypes.c_float] + [_P] * 6
                       + [ctypes.c_size_t, _P, _P], ctypes.c_int),
}


def load():
    """Load (once) and return the library; raise if it is missing."""
    global _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise RuntimeError(
                    f"libtreeverify.so not found at {LIB_PATH}: build it first "
                    "(python -c 'import __graft_entry__ as g; g.build()')")
            lib = ctypes.CDLL(LIB_PATH)
            for name, (args, res) in _SIGS.items():
                fn = getattr(lib, name)
                fn.argtypes = args
                fn.restype = res
            _lib = lib
        return _lib


def version():
    return load().tv_version().decode()


def make_shape(*, B, D, H, d, W=0, tail_mode=TV_TAIL_WINDOW, comp_mask=TV_COMP_C4 | TV_COMP_C128,
               dtype=TV_BF16, n_sel=0, attn_kernel=TV_ATTN_AUTO, raw_cap=0, c4_cap=0, c128_cap=0,
               page_tokens=0, max_pages=0, n_pool_pages=0, page_table=None, stage_chain=0):
    """``page_table``: a CUDA int32 tensor [B][max_pages] (paged pools only); the shape keeps its
    device address, so the tensor must outlive the shape's use.  ``stage_chain``: 1 stages the
    cached chain's raw rows and C4 entries in tv_branch_compress and skips them in
    tv_refresh_commit."""
    pt = None if page_table is None else _p(page_table).value
    return tv_shape(B, D, H, d, W, tail_mode, comp_mask, dtype, n_sel, attn_kernel, raw_cap,
                    c4_cap, c128_cap, page_tokens, max_pages, n_pool_pages, stage_chain, pt)


def _p(t):
    if t is None:
        return None
    if not isinstance(t, torch.Tensor):
        raise TypeError("expected a torch.Tensor or None")
    if not t.is_cuda:
        raise ValueError("tensor arguments must live on the CUDA device")
    if not t.is_contiguous():
        raise ValueError("tensor arguments must be contiguous")
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _check(fn, rc):
    if rc != TV_OK:
        msg = load().tv_last_error_string().decode()
        raise TreeVerifyError(fn, rc, msg)


def tv_workspace_size(shape):
    return int(load().tv_workspace_size(ctypes.byref(shape)))


def tv_attn_kernel_for(shape):
    rc = int(load().tv_attn_kernel_for(ctypes.byref(shape)))
    if rc < 0:
        _check("tv_attn_kernel_for", rc)
    return rc


def tv_build_ancestor_mask(shape, parents, L, anc, depth, raw_lo, scr_vis4, scr_vis128, status,
                           stream=None):
    rc = load().tv_build_ancestor_mask(ctypes.byref(shape), _p(parents), _p(L), _p(anc), _p(depth),
                                       _p(raw_lo), _p(scr_vis4), _p(scr_vis128), _p(status),
                                       _stream(stream))
    _check("tv_build_ancestor_mask", rc)


def tv_prefill_compress(shape, rawK, rawV, L, g4, g128, c4K, c4V, c128K, c128V, status,
                        stream=None):
    rc = load().tv_prefill_compress(ctypes.byref(shape), _p(rawK), _p(rawV), _p(L), _p(g4),
                                    _p(g128), _p(c4K), _p(c4V), _p(c128K), _p(c128V), _p(status),
                                    _stream(stream))
    _check("tv_prefill_compress", rc)


def tv_branch_compress(shape, rawK, rawV, c4K, c4V, L, treeK, treeV, parents, g4, g128, scrK4,
                       scrV4, scrK128, scrV128, status, stream=None):
    rc = load().tv_branch_compress(ctypes.byref(shape), _p(rawK), _p(rawV), _p(c4K), _p(c4V),
                                   _p(L), _p(treeK), _p(treeV), _p(parents), _p(g4), _p(g128),
                                   _p(scrK4), _p(scrV4), _p(scrK128), _p(scrV128), _p(status),
                                   _stream(stream))
    _check("tv_branch_compress", rc)


def tv_tree_verify_attn(shape, Q, c4K, c4V, sel, c128K, c128V, rawK, rawV, L, treeK, treeV, anc,
                        raw_lo, scr_vis4, scr_vis128, scrK4, scrV4, scrK128, scrV128, scale, O,
                        lse, workspace, status, stream=None):
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    rc = load().tv_tree_verify_attn(ctypes.byref(shape), _p(Q), _p(c4K), _p(c4V), _p(sel),
                                    _p(c128K), _p(c128V), _p(rawK), _p(rawV), _p(L), _p(treeK),
                                    _p(treeV), _p(anc), _p(raw_lo), _p(scr_vis4), _p(scr_vis128),
                                    _p(scrK4), _p(scrV4), _p(scrK128), _p(scrV128),
                                    ctypes.c_float(scale), _p(O), _p(lse), _p(workspace),
                                    ctypes.c_size_t(ws_bytes), _p(status), _stream(stream))
    _check("tv_tree_verify_attn", rc)


def tv_tree_verify_attn_noalloc(shape, Q, c4K, c4V, sel, c128K, c128V, rawK, rawV, L, treeK,
                                treeV, anc, raw_lo, scr_vis4, scr_vis128, scrK4, scrV4, scrK128,
                                scrV128, scale, O, lse, status, stream=None):
    """tv_tree_verify_attn for callers that cannot allocate: no workspace argument; the library's
    built-in scratch holds the split-KV partials (see include/treeverify.h)."""
    rc = load().tv_tree_verify_attn_noalloc(
        ctypes.byref(shape), _p(Q), _p(c4K), _p(c4V), _p(sel), _p(c128K), _p(c128V), _p(rawK),
        _p(rawV), _p(L), _p(treeK), _p(treeV), _p(anc), _p(raw_lo), _p(scr_vis4), _p(scr_vis128),
        _p(scrK4), _p(scrV4), _p(scrK128), _p(scrV128), ctypes.c_float(scale), _p(O), _p(lse),
        _p(status), _stream(stream))
    _check("tv_tree_verify_attn_noalloc", rc)


def tv_accept_walk(shape, parents, draft, target, accept_len, path, bonus, status, stream=None):
    rc = load().tv_accept_walk(ctypes.byref(shape), _p(parents), _p(draft), _p(target),
                               _p(accept_len), _p(path), _p(bonus), _p(status), _stream(stream))
    _check("tv_accept_walk", rc)


def tv_refresh_commit(shape, parents, accept_len, path, treeK, treeV, scrK4, scrV4, scrK128,
                      scrV128, rawK, rawV, c4K, c4V, c128K, c128V, L, committed_pos, status,
                      stream=None):
    rc = load().tv_refresh_commit(ctypes.byref(shape), _p(parents), _p(accept_len), _p(path),
                                  _p(treeK), _p(treeV), _p(scrK4), _p(scrV4), _p(scrK128),
                                  _p(scrV128), _p(rawK), _p(rawV), _p(c4K), _p(c4V), _p(c128K),
                                  _p(c128V), _p(L), _p(committed_pos), _p(status), _stream(stream))
    _check("tv_refresh_commit", rc)


def tv_noalloc_prepare():
    """Load the library's device code (with the 32 MiB built-in scratch) on the current device."""
    _check("tv_noalloc_prepare", load().tv_noalloc_prepare())


def tv_indexer_workspace_size(shape):
    return int(load().tv_indexer_workspace_size(ctypes.byref(shape)))


def tv_indexer_topk(shape, d_idx, q_idx, k_idx, L, sel, workspace, status, stream=None):
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    rc = load().tv_indexer_topk(ctypes.byref(shape), ctypes.c_int(d_idx), _p(q_idx), _p(k_idx),
                                _p(L), _p(sel), _p(workspace), ctypes.c_size_t(ws_bytes),
                                _p(status), _stream(stream))
    _check("tv_indexer_topk", rc)


# The calls below check their tensors' types, sizes and device, and pass plain integers: their kernels
# are short, so the binding's own time counts (a tensor takes 0.3 us, the current stream's handle
# 0.1 us against 2.9 us through a torch.cuda.Stream).
def _here():
    """The current device's index (None without a CUDA device: every tensor is then refused)."""
    try:
        return torch.cuda.current_device()
    except (RuntimeError, AssertionError):
        return None


def _refuse(t, dtype, numel, name, dev):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a torch.Tensor or None")
    if not t.is_cuda:
        raise ValueError(f"{name}: tensor arguments must live on the CUDA device")
    if t.get_device() != dev:
        raise ValueError(f"{name}: the tensor lives on another device than the current one")
    if t.dtype != dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name}: tensor arguments must be contiguous")
    raise ValueError(f"{name}: {t.numel()} elements, {numel} needed")


def _a(t, dtype, numel, name, dev):
    """Device address of a contiguous tensor of the given type with at least numel elements on
    device dev (None: a null pointer)."""
    if t is None:
        return None
    try:
        if (t.get_device() == dev and t.dtype is dtype and t.is_contiguous()
                and t.numel() >= numel):
            return t.data_ptr()
    except AttributeError:
        pass
    _refuse(t, dtype, numel, name, dev)


def _s(stream, dev):
    return torch._C._cuda_getCurrentRawStream(dev) if stream is None else stream.cuda_stream


def tv_token_logprobs(shape, logits, tokens, nodes, scale, lse, entropy, logprobs, top_ids,
                      top_logprobs, target, status, stream=None):
    """``logits``: [B][D][vocab] fp32 or bf16 with unit last stride; the rows may lie further apart
    than the vocabulary (a slice of a padded buffer).  ``tokens``, ``nodes`` and ``logprobs``: [B][n_tok]
    or None; ``top_ids`` and ``top_logprobs``: [B][D][n_top] or None."""
    lib, dev, B, D = _lib or load(), _here(), shape.B, shape.D
    size = logits.shape
    if len(size) != 3 or size[0] != B or size[1] != D:
        raise ValueError(f"logits: expected [{B}][{D}][vocab], got {tuple(size)}")
    if logits.get_device() != dev:
        raise ValueError("logits: the tensor must live on the current CUDA device")
    dtype = _LOGIT_TYPES.get(logits.dtype)
    if dtype is None:
        raise TypeError(f"logits: expected float32 or bfloat16, got {logits.dtype}")
    vocab, (sB, ld, unit) = size[2], logits.stride()
    if D == 1:
        ld = sB if B > 1 else vocab
    if (unit != 1 and vocab > 1) or ld < vocab or (B > 1 and sB != D * ld):
        raise ValueError(f"logits: rows must be contiguous and evenly spaced, strides {logits.stride()}")
    n_tok = 0 if tokens is None else tokens.shape[-1]
    n_top = 0 if top_ids is None else top_ids.shape[-1]
    rows, given, i32, f32 = B * D, B * n_tok, torch.int32, torch.float32
    rc = lib.tv_token_logprobs(
        ctypes.byref(shape), vocab, ld, dtype, logits.data_ptr(), n_tok,
        _a(tokens, i32, given, "tokens", dev), _a(nodes, i32, given, "nodes", dev), scale, n_top,
        _a(lse, f32, rows, "lse", dev), _a(entropy, f32, rows, "entropy", dev),
        _a(logprobs, f32, given, "logprobs", dev), _a(top_ids, i32, rows * n_top, "top_ids", dev),
        _a(top_logprobs, f32, rows * n_top, "top_logprobs", dev), _a(target, i32, rows, "target", dev),
        _a(status, i32, 1, "status", dev), _s(stream, dev))
    if rc:
        _check("tv_token_logprobs", rc)


def tv_pages_workspace_size(shape):
    return int(load().tv_pages_workspace_size(ctypes.byref(shape)))


def _pools(shape, rawK, rawV, c4K, c4V, c128K, c128V, dev):
    dt = torch.bfloat16 if shape.dtype == TV_BF16 else torch.float32
    mask, n = shape.comp_mask, shape.n_pool_pages * shape.page_tokens * shape.d
    n4, n128 = n // 4 if mask & TV_COMP_C4 else 0, n // 128 if mask & TV_COMP_C128 else 0
    return (_a(rawK, dt, n, "rawK", dev), _a(rawV, dt, n, "rawV", dev), _a(c4K, dt, n4, "c4K", dev),
            _a(c4V, dt, n4, "c4V", dev), _a(c128K, dt, n128, "c128K", dev),
            _a(c128V, dt, n128, "c128V", dev))


def _pages(shape, L, page_refs, workspace, dev):
    """Addresses of what all tv_pages_* calls take, and the workspace's size."""
    i32 = torch.int32
    ws = None if workspace is None else _a(workspace, workspace.dtype, 0, "workspace", dev)
    ws_bytes = 0 if ws is None else workspace.numel() * workspace.element_size()
    return (_a(L, i32, shape.B, "L", dev), _a(page_refs, i32, shape.n_pool_pages, "page_refs", dev),
            ws, ws_bytes)


def tv_pages_fork(shape, source, keep, L, page_refs, rawK, rawV, c4K, c4V, c128K, c128V, k_idx,
                  workspace, status, stream=None):
    """``k_idx``: [B][c4_cap][d_idx] bf16 indexer keys, or None."""
    lib, dev, B, i32 = _lib or load(), _here(), shape.B, torch.int32
    d_idx = 0 if k_idx is None else k_idx.shape[-1]
    L, page_refs, ws, ws_bytes = _pages(shape, L, page_refs, workspace, dev)
    rc = lib.tv_pages_fork(
        ctypes.byref(shape), _a(source, i32, B, "source", dev), _a(keep, i32, B, "keep", dev), L,
        page_refs, *_pools(shape, rawK, rawV, c4K, c4V, c128K, c128V, dev),
        _a(k_idx, torch.bfloat16, B * shape.c4_cap * d_idx, "k_idx", dev), d_idx, ws, ws_bytes,
        _a(status, i32, 1, "status", dev), _s(stream, dev))
    if rc:
        _check("tv_pages_fork", rc)


def tv_pages_reserve(shape, need, L, page_refs, workspace, status, stream=None):
    lib, dev, i32 = _lib or load(), _here(), torch.int32
    L, page_refs, ws, ws_bytes = _pages(shape, L, page_refs, workspace, dev)
    rc = lib.tv_pages_reserve(
        ctypes.byref(shape), _a(need, i32, shape.B, "need", dev), L, page_refs, ws, ws_bytes,
        _a(status, i32, 1, "status", dev), _s(stream, dev))
    if rc:
        _check("tv_pages_reserve", rc)


def tv_pages_compact(shape, L, page_refs, rawK, rawV, c4K, c4V, c128K, c128V, remap, n_live,
                     workspace, status, stream=None):
    lib, dev, i32 = _lib or load(), _here(), torch.int32
    L, page_refs, ws, ws_bytes = _pages(shape, L, page_refs, workspace, dev)
    rc = lib.tv_pages_compact(
        ctypes.byref(shape), L, page_refs, *_pools(shape, rawK, rawV, c4K, c4V, c128K, c128V, dev),
        _a(remap, i32, shape.n_pool_pages, "remap", dev), _a(n_live, i32, 1, "n_live", dev), ws,
        ws_bytes, _a(status, i32, 1, "status", dev), _s(stream, dev))
    if rc:
        _check("tv_pages_compact", rc)


def _layers(shape, rawK, rawV, c4K, c4V, c128K, c128V, dev):
    """Addresses of the cache's layers, contiguous [B][cap][d] or pools."""
    if shape.page_tokens:
        return _pools(shape, rawK, rawV, c4K, c4V, c128K, c128V, dev)
    dt = torch.bfloat16 if shape.dtype == TV_BF16 else torch.float32
    mask, row = shape.comp_mask, shape.B * shape.d
    n = shape.raw_cap * row
    n4 = shape.c4_cap * row if mask & TV_COMP_C4 else 0
    n128 = shape.c128_cap * row if mask & TV_COMP_C128 else 0
    return (_a(rawK, dt, n, "rawK", dev), _a(rawV, dt, n, "rawV", dev), _a(c4K, dt, n4, "c4K", dev),
            _a(c4V, dt, n4, "c4V", dev), _a(c128K, dt, n128, "c128K", dev),
            _a(c128V, dt, n128, "c128V", dev))


def tv_chunk_append(shape, starts, K, V, Q, rope_dim, rope_pairs, inv_freq, g4, g128, Qr, rawK, rawV,
                    c4K, c4V, c128K, c128V, L, status, stream=None):
    """``K``, ``V``: [n_new][d] with unit last stride, both with the same row stride (slices of a wider
    projection's output, say); ``Q``, ``Qr``: [n_new][H][d] or None; ``inv_freq``: [rope_dim / 2]
    fp32 or None."""
    lib, dev, B, d = _lib or load(), _here(), shape.B, shape.d
    dt = torch.bfloat16 if shape.dtype == TV_BF16 else torch.float32
    f32, i32, size = torch.float32, torch.int32, K.shape
    if len(size) != 2 or size[1] != d or V.shape != size:
        raise ValueError(f"K, V: expected [n_new][{d}], got {tuple(size)} and {tuple(V.shape)}")
    n, ld = size[0], d
    if K.is_contiguous() and V.is_contiguous():
        k, v = _a(K, dt, 0, "K", dev), _a(V, dt, 0, "V", dev)
    else:
        ld = K.stride(0) if n > 1 else d
        for t, name in ((K, "K"), (V, "V")):
            if t.get_device() != dev:
                raise ValueError(f"{name}: the tensor must live on the current CUDA device")
            if t.dtype != dt:
                raise TypeError(f"{name}: expected {dt}, got {t.dtype}")
            if t.stride(1) != 1 or (n > 1 and t.stride(0) != ld):
                raise ValueError(f"{name}: rows must be contiguous and as far apart as K's")
        k, v = K.data_ptr(), V.data_ptr()
    rows = n * shape.H * d
    rc = lib.tv_chunk_append(
        ctypes.byref(shape), n, _a(starts, i32, B + 1, "starts", dev), k, v, ld,
        _a(Q, dt, rows, "Q", dev), rope_dim, rope_pairs, _a(inv_freq, f32, rope_dim // 2, "inv_freq", dev),
        _a(g4, f32, d, "g4", dev), _a(g128, f32, d, "g128", dev), _a(Qr, dt, rows, "Qr", dev),
        *_layers(shape, rawK, rawV, c4K, c4V, c128K, c128V, dev), _a(L, i32, B, "L", dev),
        _a(status, i32, 1, "status", dev), _s(stream, dev))
    if rc:
        _check("tv_chunk_append", rc)


def tv_chunk_workspace_size(shape, n_new):
    return int(load().tv_chunk_workspace_size(ctypes.byref(shape), n_new))


def tv_chunk_attn(shape, starts, Q, c4K, c4V, c128K, c128V, rawK, rawV, L, scale, O, lse, workspace,
                  status, stream=None):
    """``Q``, ``O``: [n_new][H][d]; ``lse``: [n_new][H]."""
    lib, dev, i32 = _lib or load(), _here(), torch.int32
    dt = torch.bfloat16 if shape.dtype == TV_BF16 else torch.float32
    if Q.dim() != 3 or Q.shape[1] != shape.H or Q.shape[2] != shape.d:
        raise ValueError(f"Q: expected [n_new][{shape.H}][{shape.d}], got {tuple(Q.shape)}")
    n = Q.shape[0]
    ws = None if workspace is None else _a(workspace, workspace.dtype, 0, "workspace", dev)
    ws_bytes = 0 if ws is None else workspace.numel() * workspace.element_size()
    rawK, rawV, c4K, c4V, c128K, c128V = _layers(shape, rawK, rawV, c4K, c4V, c128K, c128V, dev)
    rc = lib.tv_chunk_attn(
        ctypes.byref(shape), n, _a(starts, i32, shape.B + 1, "starts", dev),
        _a(Q, dt, n * shape.H * shape.d, "Q", dev), c4K, c4V, c128K, c128V, rawK, rawV,
        _a(L, i32, shape.B, "L", dev), scale, _a(O, dt, n * shape.H * shape.d, "O", dev),
        _a(lse, torch.float32, n * shape.H, "lse", dev), ws, ws_bytes,
        _a(status, i32, 1, "status", dev), _s(stream, dev))
    if rc:
        _check("tv_chunk_attn", rc)


def tv_beam_workspace_size(shape, width):
    return int(load().tv_beam_workspace_size(ctypes.byref(shape), width))


def tv_beam_select(shape, width, logits, scores, done, eos, scale, source, token, new_scores, new_done,
                   rank, workspace, status, stream=None):
    """``logits``: [B][vocab] fp32 or bf16 with unit last stride, the rows at least the vocabulary
    apart; ``done``, ``new_done`` and ``rank`` may be None."""
    lib, dev, B, i32, f32 = _lib or load(), _here(), shape.B, torch.int32, torch.float32
    size = logits.shape
    if len(size) != 2 or size[0] != B:
        raise ValueError(f"logits: expected [{B}][vocab], got {tuple(size)}")
    if logits.get_device() != dev:
        raise ValueError("logits: the tensor must live on the current CUDA device")
    dtype = _LOGIT_TYPES.get(logits.dtype)
    if dtype is None:
        raise TypeError(f"logits: expected float32 or bfloat16, got {logits.dtype}")
    vocab, (ld, unit) = size[1], logits.stride()
    if B <= 1:
        ld = vocab
    if (unit != 1 and vocab > 1) or ld < vocab:
        raise ValueError(f"logits: rows must be contiguous, strides {logits.stride()}")
    ws = None if workspace is None else _a(workspace, workspace.dtype, 0, "workspace", dev)
    ws_bytes = 0 if ws is None else workspace.numel() * workspace.element_size()
    rc = lib.tv_beam_select(
        ctypes.byref(shape), width, vocab, ld, dtype, logits.data_ptr(),
        _a(scores, f32, B, "scores", dev), _a(done, i32, B, "done", dev), eos, scale,
        _a(source, i32, B, "source", dev), _a(token, i32, B, "token", dev),
        _a(new_scores, f32, B, "new_scores", dev), _a(new_done, i32, B, "new_done", dev),
        _a(rank, i32, B, "rank", dev), ws, ws_bytes, _a(status, i32, 1, "status", dev),
        _s(stream, dev))
    if rc:
        _check("tv_beam_select", rc)


def tv_debug_attn_timeout(timeout_ns, withhold_tile):
    """Testing aid: the wait bound and a withheld KV tile of later tensor-core attention calls."""
    _check("tv_debug_attn_timeout", load().tv_debug_attn_timeout(int(timeout_ns), int(withhold_tile)))
