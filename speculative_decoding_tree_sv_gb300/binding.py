"""ctypes binding of ``libsv.so`` (argument marshalling only).

The functions carry the names of the C entry points declared in
``include/sv.h``.  Tensor arguments may be torch tensors (their
``data_ptr()`` is passed) or raw integer device addresses; ``stream``
defaults to torch's current CUDA stream.  Every step of the computation
runs in the library's CUDA kernels: if the library is not built, loading
fails with an error instead of falling back to anything else.
"""

from __future__ import annotations

import ctypes
import importlib.util
import os
from ctypes import c_float, c_int, c_longlong, c_size_t, c_void_p
from typing import Optional

from . import build as _build

SV_OK = 0
STATUS_NAMES = {0: "SV_OK", 1: "SV_ERR_INVALID_ARG", 2: "SV_ERR_UNSUPPORTED", 3: "SV_ERR_CUDA",
                4: "SV_ERR_WORKSPACE", 5: "SV_ERR_DEVICE", 6: "SV_ERR_TIMEOUT"}
# device error codes (sv_deverr in include/sv.h)
SV_DEVERR_NONE, SV_DEVERR_TIMEOUT, SV_DEVERR_BAD_PARENT, SV_DEVERR_BAD_PAGE = 0, 1, 2, 3
SV_DEVERR_BAD_PATH, SV_DEVERR_DEPTH, SV_DEVERR_BAD_TREE = 4, 5, 6
SV_DEVERR_BAD_LENGTH, SV_DEVERR_NO_PAGES, SV_DEVERR_BAD_ROW = 7, 8, 9
SV_BF16, SV_FP16 = 0, 1
SV_ATTN_EARLY_CONTEXT = 1
SV_ATTN_KERNEL_PAIRED = 2
SV_ATTN_KERNEL_WIDE = 4
SV_ATTN_KERNEL_DEALT = 8
DEVICE_ERRORS = {0: "none", 1: "timeout", 2: "bad parent", 3: "bad page", 4: "bad path", 5: "depth",
                 6: "bad tree", 7: "bad length", 8: "no pages", 9: "bad row"}


class SvError(RuntimeError):
    def __init__(self, status: int, where: str):
        super().__init__(f"{where}: {STATUS_NAMES.get(status, status)}")
        self.status = status


class sv_attn_params(ctypes.Structure):
    _fields_ = [
        ("batch", c_int), ("num_q_heads", c_int), ("num_kv_heads", c_int), ("head_dim", c_int),
        ("page_size", c_int), ("num_pages", c_int), ("total_nodes", c_int), ("max_nodes", c_int),
        ("max_pages_per_seq", c_int), ("max_kv_pages", c_int), ("num_splits", c_int),
        ("split_reduce", c_int), ("sm_scale", c_float), ("flags", c_int),
        ("q", c_void_p), ("tree_k", c_void_p), ("tree_v", c_void_p), ("k_cache", c_void_p),
        ("v_cache", c_void_p), ("block_table", c_void_p), ("ctx_lens", c_void_p),
        ("cu_nodes", c_void_p), ("parents", c_void_p), ("kv_pages", c_void_p),
        ("cu_kv_pages", c_void_p), ("out", c_void_p), ("lse", c_void_p), ("workspace", c_void_p),
        ("workspace_bytes", c_size_t),
    ]


class sv_retrieve_params(ctypes.Structure):
    _fields_ = [
        ("batch", c_int), ("num_q_heads", c_int), ("num_kv_heads", c_int), ("head_dim", c_int),
        ("page_size", c_int), ("num_pages", c_int), ("total_nodes", c_int), ("max_pages_per_seq", c_int),
        ("max_ctx_pages", c_int), ("sink_tokens", c_int), ("window_tokens", c_int), ("topk", c_int),
        ("reduce", c_int),
        ("q", c_void_p), ("summaries", c_void_p), ("block_table", c_void_p), ("ctx_lens", c_void_p),
        ("cu_nodes", c_void_p), ("kv_pages", c_void_p), ("cu_kv_pages", c_void_p), ("scores", c_void_p),
        ("kv_pages_capacity", c_size_t), ("workspace", c_void_p), ("workspace_bytes", c_size_t),
    ]


class sv_chunk_params(ctypes.Structure):
    _fields_ = [
        ("batch", c_int), ("num_q_heads", c_int), ("num_kv_heads", c_int), ("head_dim", c_int),
        ("page_size", c_int), ("num_pages", c_int), ("total_tokens", c_int), ("max_tokens", c_int),
        ("max_pages_per_seq", c_int), ("dtype", c_int), ("window_tokens", c_int), ("sink_tokens", c_int),
        ("sm_scale", c_float), ("flags", c_int), ("q_stride", c_longlong), ("out_stride", c_longlong),
        ("q", c_void_p), ("k_cache", c_void_p), ("v_cache", c_void_p), ("block_table", c_void_p),
        ("ctx_lens", c_void_p), ("cu_tokens", c_void_p), ("out", c_void_p), ("lse", c_void_p),
        ("workspace", c_void_p), ("workspace_bytes", c_size_t),
    ]


SV_REDUCE_MEAN, SV_REDUCE_MAX, SV_REDUCE_LAST = 0, 1, 2
SV_VERIFY_PARTIAL, SV_VERIFY_FULL = 0, 1


class sv_specpv_seq(ctypes.Structure):
    _fields_ = [("has_partial_cache", c_int), ("refresh_ctx_len", c_int), ("buffer_tokens", c_int)]

_LIB = None


def load(path: Optional[str] = None):
    """Load the built library (raises if it is missing)."""
    global _LIB
    if _LIB is not None and path is None:
        return _LIB
    path = path or _build.library_path()
    if not os.path.exists(path):
        raise RuntimeError(f"libsv.so is not built ({path}); run __graft_entry__.build() or "
                           "python -m speculative_decoding_tree_sv_gb300.build")
    lib = ctypes.CDLL(path)
    P = ctypes.POINTER
    lib.sv_abi_version.restype = c_int
    lib.sv_abi_version.argtypes = []
    lib.sv_status_string.restype = ctypes.c_char_p
    lib.sv_status_string.argtypes = [c_int]
    lib.sv_tree_attention_workspace_size.restype = c_int
    lib.sv_tree_attention_workspace_size.argtypes = [P(sv_attn_params), P(c_size_t)]
    lib.sv_tree_attention_plan.restype = c_int
    lib.sv_tree_attention_plan.argtypes = [P(sv_attn_params), P(c_int), P(c_int), P(c_int)]
    lib.sv_tree_attention.restype = c_int
    lib.sv_tree_attention.argtypes = [P(sv_attn_params), c_void_p]
    lib.sv_greedy_accept_workspace_size.restype = c_int
    lib.sv_greedy_accept_workspace_size.argtypes = [c_int, c_int, P(c_size_t)]
    lib.sv_greedy_accept.restype = c_int
    lib.sv_greedy_accept.argtypes = [c_void_p, c_int, c_void_p, c_void_p, c_void_p, c_int, c_int, c_int, c_int,
                                     c_void_p, c_void_p, c_void_p, c_void_p, c_void_p, c_size_t, c_void_p]
    lib.sv_greedy_accept_noalloc.restype = c_int
    lib.sv_greedy_accept_noalloc.argtypes = [c_void_p, c_int, c_void_p, c_void_p, c_void_p, c_int, c_int, c_int,
                                             c_int, c_void_p, c_void_p, c_void_p, c_void_p, c_void_p, c_void_p]
    lib.sv_sample_accept_workspace_size.restype = c_int
    lib.sv_sample_accept_workspace_size.argtypes = [c_int, c_int, P(c_size_t)]
    lib.sv_sample_accept.restype = c_int
    lib.sv_sample_accept.argtypes = [c_void_p, c_void_p, c_int, ctypes.c_float, c_void_p, c_void_p, c_void_p,
                                     c_int, c_int, c_int, c_int, c_void_p, c_void_p, c_void_p, c_void_p,
                                     c_void_p, c_void_p, c_void_p, c_size_t, c_void_p]
    lib.sv_selftest_bounded_wait.restype = c_int
    lib.sv_selftest_bounded_wait.argtypes = [c_void_p, c_longlong, c_void_p]
    lib.sv_kv_commit.restype = c_int
    lib.sv_kv_commit.argtypes = [c_void_p, c_void_p, c_longlong, c_void_p, c_void_p, c_longlong, c_int, c_int,
                                 c_void_p, c_int, c_void_p, c_void_p, c_void_p, c_void_p, c_int, c_int, c_int,
                                 c_int, c_int, c_void_p, c_void_p, c_size_t, c_void_p]
    lib.sv_kv_page_summaries.restype = c_int
    lib.sv_kv_page_summaries.argtypes = [c_void_p, c_int, c_int, c_int, c_int, c_void_p, c_int, c_void_p, c_void_p,
                                         c_int, c_int, c_void_p, c_void_p, c_size_t, c_void_p]
    lib.sv_retrieve_pages_workspace_size.restype = c_int
    lib.sv_retrieve_pages_workspace_size.argtypes = [c_int, c_int, c_int, c_int, P(c_size_t)]
    lib.sv_retrieve_pages.restype = c_int
    lib.sv_retrieve_pages.argtypes = [P(sv_retrieve_params), c_void_p]
    lib.sv_partial_list_extend.restype = c_int
    lib.sv_partial_list_extend.argtypes = [c_void_p, c_void_p, c_void_p, c_void_p, c_int, c_void_p, c_void_p,
                                           c_void_p, c_size_t, c_void_p]
    lib.sv_specpv_full_trees.restype = c_int
    lib.sv_specpv_full_trees.argtypes = [c_void_p, c_void_p, c_void_p, c_void_p, c_void_p, c_int, c_void_p,
                                         c_void_p, c_void_p, c_void_p, c_size_t, c_void_p]
    lib.sv_specpv_next.restype = c_int
    lib.sv_specpv_next.argtypes = [P(sv_specpv_seq), c_int, c_int]
    lib.sv_specpv_after.restype = c_int
    lib.sv_specpv_after.argtypes = [P(sv_specpv_seq), c_int, c_int]
    V, I, L, Z = c_void_p, c_int, c_longlong, c_size_t
    for name, args in (
            ("sv_kv_append", [V, V, L, L, V, V, L, I, I, V, I, V, V, I, I, I, I, I, V, V, Z, V]),
            ("sv_chunk_attention_workspace_size", [P(sv_chunk_params), P(Z)]),
            ("sv_chunk_attention", [P(sv_chunk_params), V]),
            ("sv_pages_workspace_size", [I, I, P(Z)]),
            ("sv_pages_release", [V, I, V, I, V, V, I, I, V, Z, V]),
            ("sv_pages_fork", [V, V, I, V, I, I, V, V, V, I, I, V, Z, V]),
            ("sv_pages_reserve", [V, V, I, V, I, V, V, I, I, V, V, V, V, Z, V]),
            ("sv_pages_compact", [V, V, I, I, V, I, V, V, V, V, V, V, V, Z, V]),
            ("sv_pages_copy", [V, V, L, I, I, I, V, V, V, I, V, Z, V])):
        getattr(lib, name).restype = c_int
        getattr(lib, name).argtypes = args
    lib.sv_set_trace_buffer.restype = c_int
    lib.sv_set_trace_buffer.argtypes = [c_void_p, c_size_t]
    lib.sv_get_device_error.restype = c_int
    lib.sv_get_device_error.argtypes = [c_void_p, P(c_int), c_void_p]
    if path == _build.library_path():
        _LIB = lib
    return lib


_MARSHAL = None


def _marshal():
    """The module that checks and passes the cache operators' tensors."""
    global _MARSHAL
    if _MARSHAL is None:
        load()
        import torch  # noqa: F401  (its libraries must be in the process)
        path = _build.marshal_path()
        if not os.path.exists(path):
            raise RuntimeError(f"the tensor module of this torch is not built ({path}); run __graft_entry__.build() or "
                               "python -m speculative_decoding_tree_sv_gb300.build")
        spec = importlib.util.spec_from_file_location("_marshal", path)
        module = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(module)
        _MARSHAL = module
    return _MARSHAL


def _ptr(x) -> Optional[int]:
    """Address of a device buffer: None, a raw device address, or a CUDA
    tensor.  A tensor in host memory is refused here, before the library
    could hand its address to a kernel."""
    if x is None:
        return None
    if isinstance(x, int):
        return x
    if getattr(x, "is_cuda", True) is False:
        raise ValueError(f"the library takes device memory; got a tensor on {x.device}")
    return int(x.data_ptr())


def _stream(stream) -> Optional[int]:
    if stream is None:
        # the handle alone: building torch's Stream object costs 3 us a call,
        # as much as the launch
        import torch
        return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())
    if isinstance(stream, int):
        return stream
    return int(stream.cuda_stream)


def _where(stream):
    """The current device (-1 before CUDA is initialised) and the stream's handle."""
    import torch
    if not torch.cuda.is_initialized():
        return -1, (_stream(stream) or 0) if stream is not None else 0
    device = torch.cuda.current_device()
    if stream is None:
        return device, torch._C._cuda_getCurrentRawStream(device)
    return device, _stream(stream) or 0


def _check(status: int, where: str):
    if status != SV_OK:
        raise SvError(status, where)


def sv_abi_version() -> int:
    return load().sv_abi_version()


def sv_status_string(status: int) -> str:
    return load().sv_status_string(status).decode()


def make_attn_params(*, q, tree_k, tree_v, k_cache, v_cache, block_table, ctx_lens, cu_nodes, parents,
                     out, total_nodes: int, max_nodes: int, workspace=None, workspace_bytes: int = 0,
                     kv_pages=None, cu_kv_pages=None, max_kv_pages: int = 0, lse=None,
                     sm_scale: float = 0.0, num_splits: int = 0, split_reduce: int = 0, flags: int = 0,
                     page_size: int = 16, batch=None,
                     num_q_heads=None, num_kv_heads=None, head_dim=None, num_pages=None,
                     max_pages_per_seq=None) -> sv_attn_params:
    """Fill an ``sv_attn_params``; shapes come from torch tensors unless given."""
    p = sv_attn_params()
    p.batch = batch if batch is not None else int(block_table.shape[0])
    p.num_q_heads = num_q_heads if num_q_heads is not None else int(q.shape[1])
    p.num_kv_heads = num_kv_heads if num_kv_heads is not None else int(tree_k.shape[1])
    p.head_dim = head_dim if head_dim is not None else int(q.shape[2])
    p.page_size = page_size
    p.num_pages = num_pages if num_pages is not None else int(k_cache.shape[0])
    p.total_nodes = int(total_nodes)
    p.max_nodes = int(max_nodes)
    p.max_pages_per_seq = max_pages_per_seq if max_pages_per_seq is not None else int(block_table.shape[1])
    p.max_kv_pages = int(max_kv_pages)
    p.num_splits = int(num_splits)
    p.split_reduce = int(split_reduce)
    p.sm_scale = float(sm_scale)
    p.flags = int(flags)
    p.q, p.tree_k, p.tree_v = _ptr(q), _ptr(tree_k), _ptr(tree_v)
    p.k_cache, p.v_cache = _ptr(k_cache), _ptr(v_cache)
    p.block_table, p.ctx_lens, p.cu_nodes, p.parents = _ptr(block_table), _ptr(ctx_lens), _ptr(cu_nodes), _ptr(parents)
    p.kv_pages, p.cu_kv_pages = _ptr(kv_pages), _ptr(cu_kv_pages)
    p.out, p.lse = _ptr(out), _ptr(lse)
    p.workspace = _ptr(workspace)
    p.workspace_bytes = int(workspace_bytes if workspace_bytes else
                            (workspace.numel() * workspace.element_size() if hasattr(workspace, "numel") else 0))
    return p


def sv_tree_attention_workspace_size(params: sv_attn_params) -> int:
    n = c_size_t(0)
    _check(load().sv_tree_attention_workspace_size(ctypes.byref(params), ctypes.byref(n)),
           "sv_tree_attention_workspace_size")
    return int(n.value)


def sv_tree_attention_plan(params: sv_attn_params, with_kernel: bool = False):
    """(num_splits, split_reduce) the library would launch with, plus the
    kernel (0 = paired, 1 = wide, 2 = dealt) when with_kernel is set."""
    s, m, k = c_int(0), c_int(0), c_int(0)
    _check(load().sv_tree_attention_plan(ctypes.byref(params), ctypes.byref(s), ctypes.byref(m), ctypes.byref(k)),
           "sv_tree_attention_plan")
    if with_kernel:
        return int(s.value), int(m.value), int(k.value)
    return int(s.value), int(m.value)


def sv_tree_attention(params: sv_attn_params, stream=None) -> None:
    _check(load().sv_tree_attention(ctypes.byref(params), _stream(stream)), "sv_tree_attention")


def sv_greedy_accept_workspace_size(batch: int, total_nodes: int) -> int:
    n = c_size_t(0)
    _check(load().sv_greedy_accept_workspace_size(batch, total_nodes, ctypes.byref(n)),
           "sv_greedy_accept_workspace_size")
    return int(n.value)


def sv_greedy_accept(logits, vocab: int, tokens, parents, cu_nodes, batch: int, total_nodes: int,
                     max_nodes: int, max_depth: int, argmax_out, accept_len, accepted_nodes, bonus_token,
                     workspace, workspace_bytes: Optional[int] = None, stream=None) -> None:
    if workspace_bytes is None:
        workspace_bytes = workspace.numel() * workspace.element_size()
    _check(load().sv_greedy_accept(_ptr(logits), vocab, _ptr(tokens), _ptr(parents), _ptr(cu_nodes), batch,
                                   total_nodes, max_nodes, max_depth, _ptr(argmax_out), _ptr(accept_len),
                                   _ptr(accepted_nodes), _ptr(bonus_token), _ptr(workspace), workspace_bytes,
                                   _stream(stream)), "sv_greedy_accept")


def sv_greedy_accept_noalloc(logits, vocab: int, tokens, parents, cu_nodes, batch: int, total_nodes: int,
                             max_nodes: int, max_depth: int, argmax_out, accept_len, accepted_nodes, bonus_token,
                             device_error=None, stream=None) -> None:
    """Greedy acceptance without a workspace, for callers that cannot
    allocate device memory; its scratch is a fixed array in the library (see
    include/sv.h for its limits and for why overlapping calls race)."""
    _check(load().sv_greedy_accept_noalloc(_ptr(logits), vocab, _ptr(tokens), _ptr(parents), _ptr(cu_nodes),
                                           batch, total_nodes, max_nodes, max_depth, _ptr(argmax_out),
                                           _ptr(accept_len), _ptr(accepted_nodes), _ptr(bonus_token),
                                           _ptr(device_error), _stream(stream)), "sv_greedy_accept_noalloc")


def sv_selftest_bounded_wait(workspace, abort_after_ns: int = 0, stream=None) -> None:
    """Launches a kernel whose bounded mbarrier wait must give up (see
    include/sv.h); read the outcome with sv_get_device_error."""
    _check(load().sv_selftest_bounded_wait(_ptr(workspace), int(abort_after_ns), _stream(stream)),
           "sv_selftest_bounded_wait")


def sv_sample_accept_workspace_size(batch: int, total_nodes: int) -> int:
    n = c_size_t(0)
    _check(load().sv_sample_accept_workspace_size(batch, total_nodes, ctypes.byref(n)),
           "sv_sample_accept_workspace_size")
    return int(n.value)


def sv_sample_accept(logits, draft_probs, vocab: int, temperature: float, tokens, parents, cu_nodes, batch: int,
                     total_nodes: int, max_nodes: int, max_depth: int, u_accept, u_bonus, accepted_child,
                     accept_len, accepted_nodes, bonus_token, workspace, workspace_bytes: Optional[int] = None,
                     stream=None) -> None:
    """Stochastic (temperature > 0) acceptance: speculative sampling node by
    node over the tree (see include/sv.h for the rule and the layouts)."""
    if workspace_bytes is None:
        workspace_bytes = workspace.numel() * workspace.element_size()
    _check(load().sv_sample_accept(_ptr(logits), _ptr(draft_probs), vocab, float(temperature), _ptr(tokens),
                                   _ptr(parents), _ptr(cu_nodes), batch, total_nodes, max_nodes, max_depth,
                                   _ptr(u_accept), _ptr(u_bonus), _ptr(accepted_child), _ptr(accept_len),
                                   _ptr(accepted_nodes), _ptr(bonus_token), _ptr(workspace), workspace_bytes,
                                   _stream(stream)), "sv_sample_accept")


def sv_kv_commit(tree_k, tree_v, tree_layer_stride: int, k_cache, v_cache, cache_layer_stride: int,
                 num_layers: int, num_pages: int, block_table, max_pages_per_seq: int, ctx_lens, cu_nodes,
                 accepted_nodes, accept_len, batch: int, max_depth: int, num_kv_heads: int, head_dim: int,
                 page_size: int = 16, new_ctx_lens=None, workspace=None, workspace_bytes: int = 0,
                 stream=None) -> None:
    if workspace is not None and not workspace_bytes:
        workspace_bytes = workspace.numel() * workspace.element_size()
    _check(load().sv_kv_commit(_ptr(tree_k), _ptr(tree_v), tree_layer_stride, _ptr(k_cache), _ptr(v_cache),
                               cache_layer_stride, num_layers, num_pages, _ptr(block_table), max_pages_per_seq,
                               _ptr(ctx_lens), _ptr(cu_nodes), _ptr(accepted_nodes), _ptr(accept_len), batch,
                               max_depth, num_kv_heads, head_dim, page_size, _ptr(new_ctx_lens),
                               _ptr(workspace), workspace_bytes, _stream(stream)), "sv_kv_commit")


def sv_kv_page_summaries(k_cache, num_pages: int, num_kv_heads: int, head_dim: int, block_table,
                         max_pages_per_seq: int, ctx_lens, first_page, batch: int, max_ctx_pages: int, summaries,
                         workspace=None, workspace_bytes: int = 0, page_size: int = 16, stream=None) -> None:
    if workspace is not None and not workspace_bytes:
        workspace_bytes = workspace.numel() * workspace.element_size()
    _check(load().sv_kv_page_summaries(_ptr(k_cache), num_pages, num_kv_heads, head_dim, page_size,
                                       _ptr(block_table), max_pages_per_seq, _ptr(ctx_lens), _ptr(first_page),
                                       batch, max_ctx_pages, _ptr(summaries), _ptr(workspace), workspace_bytes,
                                       _stream(stream)), "sv_kv_page_summaries")


def retrieve_list_bound(sink_tokens: int, window_tokens: int, topk: int, page_size: int = 16) -> int:
    """Longest partial list sv_retrieve_pages writes for one sequence."""
    return -(-sink_tokens // page_size) + topk + -(-window_tokens // page_size) + 1


def sv_retrieve_pages_workspace_size(batch: int, num_kv_heads: int, head_dim: int, max_ctx_pages: int) -> int:
    n = c_size_t(0)
    _check(load().sv_retrieve_pages_workspace_size(batch, num_kv_heads, head_dim, max_ctx_pages, ctypes.byref(n)),
           "sv_retrieve_pages_workspace_size")
    return int(n.value)


def make_retrieve_params(*, q, summaries, block_table, ctx_lens, cu_nodes, kv_pages, cu_kv_pages, batch: int,
                         num_q_heads: int, num_kv_heads: int, head_dim: int, num_pages: int, total_nodes: int,
                         max_pages_per_seq: int, max_ctx_pages: int, sink_tokens: int, window_tokens: int,
                         topk: int, reduce: int = SV_REDUCE_MEAN, scores=None, kv_pages_capacity=None,
                         workspace=None, workspace_bytes: int = 0, page_size: int = 16) -> sv_retrieve_params:
    r = sv_retrieve_params()
    r.batch, r.num_q_heads, r.num_kv_heads, r.head_dim = batch, num_q_heads, num_kv_heads, head_dim
    r.page_size, r.num_pages, r.total_nodes, r.max_pages_per_seq = page_size, num_pages, total_nodes, max_pages_per_seq
    r.max_ctx_pages, r.sink_tokens, r.window_tokens, r.topk, r.reduce = (max_ctx_pages, sink_tokens, window_tokens,
                                                                         topk, reduce)
    r.q, r.summaries, r.block_table, r.ctx_lens, r.cu_nodes = (_ptr(q), _ptr(summaries), _ptr(block_table),
                                                              _ptr(ctx_lens), _ptr(cu_nodes))
    r.kv_pages, r.cu_kv_pages, r.scores = _ptr(kv_pages), _ptr(cu_kv_pages), _ptr(scores)
    if kv_pages_capacity is None:
        kv_pages_capacity = kv_pages.numel() if hasattr(kv_pages, "numel") else 0
    r.kv_pages_capacity = int(kv_pages_capacity)
    r.workspace = _ptr(workspace)
    r.workspace_bytes = int(workspace_bytes if workspace_bytes else
                            (workspace.numel() * workspace.element_size() if hasattr(workspace, "numel") else 0))
    return r


def sv_retrieve_pages(params: sv_retrieve_params, stream=None) -> None:
    _check(load().sv_retrieve_pages(ctypes.byref(params), _stream(stream)), "sv_retrieve_pages")


def sv_partial_list_extend(ref_pages, ref_cu, ref_ctx_lens, ctx_lens, batch: int, kv_pages, cu_kv_pages,
                           workspace=None, workspace_bytes: int = 0, stream=None) -> None:
    if workspace is not None and not workspace_bytes:
        workspace_bytes = workspace.numel() * workspace.element_size()
    _check(load().sv_partial_list_extend(_ptr(ref_pages), _ptr(ref_cu), _ptr(ref_ctx_lens), _ptr(ctx_lens), batch,
                                         _ptr(kv_pages), _ptr(cu_kv_pages), _ptr(workspace), workspace_bytes,
                                         _stream(stream)), "sv_partial_list_extend")


def sv_specpv_full_trees(cand_parents, cand_tokens, cand_cu, buffer_tokens, buffer_cu, batch: int, parents,
                         tokens, cu_nodes, workspace=None, workspace_bytes: int = 0, stream=None) -> None:
    if workspace is not None and not workspace_bytes:
        workspace_bytes = workspace.numel() * workspace.element_size()
    _check(load().sv_specpv_full_trees(_ptr(cand_parents), _ptr(cand_tokens), _ptr(cand_cu), _ptr(buffer_tokens),
                                       _ptr(buffer_cu), batch, _ptr(parents), _ptr(tokens), _ptr(cu_nodes),
                                       _ptr(workspace), workspace_bytes, _stream(stream)), "sv_specpv_full_trees")


def sv_specpv_next(seq: sv_specpv_seq, step_tokens: int, buffer_limit: int) -> int:
    return int(load().sv_specpv_next(ctypes.byref(seq), step_tokens, buffer_limit))


def sv_specpv_after(seq: sv_specpv_seq, kind: int, ctx_len_after: int) -> None:
    _check(load().sv_specpv_after(ctypes.byref(seq), kind, ctx_len_after), "sv_specpv_after")


def _on_device(*tensors) -> None:
    """Every tensor (None is left out) lies on the current CUDA device, where
    the launch goes."""
    import torch
    current = torch.cuda.current_device() if torch.cuda.is_initialized() else None
    for t in tensors:
        if t is not None and t.get_device() != current:
            if not t.is_cuda:
                raise ValueError(f"the library takes device memory; got a tensor on {t.device}")
            raise ValueError(f"got a tensor on {t.device}, the current device is cuda:{current}")


def _ints(name: str, t, count: Optional[int] = None) -> None:
    """int32, contiguous, of `count` elements."""
    import torch
    if t.dtype is torch.int32 and t.is_contiguous() and (count is None or t.numel() == count):
        return
    if t.dtype is not torch.int32 or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous int32 tensor")
    raise ValueError(f"{name} must have {count} elements, got {t.numel()}")


def _space(workspace):
    """(address, bytes) of an optional workspace tensor."""
    if workspace is None:
        return None, 0
    return workspace.data_ptr(), workspace.nbytes


def _pool(k_cache, v_cache):
    """Layers, pages, heads, page size, head dim and layer stride of a cache
    [layers, pages, Hkv, page, D] (or one layer of it, without the first)."""
    shape, stride = k_cache.shape, k_cache.stride()
    if len(shape) not in (4, 5) or k_cache.itemsize != 2:
        raise ValueError("a cache is [layers, pages, Hkv, page_size, D] or [pages, Hkv, page_size, D] of 16-bit elements")
    if not k_cache.is_contiguous() and not (len(shape) == 5 and k_cache[0].is_contiguous()):
        raise ValueError("a layer of the cache must be contiguous")
    if v_cache is not None and (v_cache.stride() != stride or v_cache.shape != shape or
                                v_cache.dtype is not k_cache.dtype):
        raise ValueError("k_cache and v_cache must have the same shape, type and strides")
    if len(shape) == 4:
        return (1, *shape, 0)
    return (*shape, stride[0] if shape[0] > 1 else 0)


def make_chunk_params(*, q, k_cache, v_cache, block_table, ctx_lens, cu_tokens, out, max_tokens: int, lse=None,
                      workspace=None, window_tokens: int = 0, sink_tokens: int = 0,
                      sm_scale: float = 0.0) -> sv_chunk_params:
    """Fill an ``sv_chunk_params`` from torch tensors: q/out [T, Hq, D] (heads
    contiguous, Hq * D elements or more from a token to the next), caches
    [pages, Hkv, 16, D], all bf16 or all fp16; lse fp32 [T, Hq] if wanted.  The
    result keeps the tensors alive."""
    import torch
    if q.dim() != 3 or out.shape != q.shape:
        raise ValueError("q and out must both be [tokens, heads, head_dim]")
    if q.dtype not in (torch.bfloat16, torch.float16):
        raise ValueError(f"q must be bfloat16 or float16, got {q.dtype}")
    for name, t in (("k_cache", k_cache), ("v_cache", v_cache), ("out", out)):
        if t.dtype != q.dtype:
            raise ValueError(f"{name} is {t.dtype}, q is {q.dtype}")
    T, Hq, D = q.shape
    layers, pages, Hkv, page, Dk, _ = _pool(k_cache, v_cache)
    if layers != 1 or k_cache.dim() != 4 or Dk != D:
        raise ValueError("the caches must be one layer, [pages, Hkv, page_size, head_dim], of q's head_dim")
    for name, t in (("q", q), ("out", out)):
        if D > 1 and t.stride(2) != 1 or Hq > 1 and t.stride(1) != D:
            raise ValueError(f"the heads of {name} must be contiguous")
        if T > 1 and t.stride(0) < Hq * D:  # (0 is the parameters' word for dense)
            raise ValueError(f"the rows of {name} overlap: {t.stride(0)} elements from a token to the next")
    if block_table.dim() != 2:
        raise ValueError("block_table must be [batch, max_pages]")
    B, width = block_table.shape
    _ints("block_table", block_table)
    _ints("ctx_lens", ctx_lens, B)
    _ints("cu_tokens", cu_tokens, B + 1)
    if lse is not None and (lse.dtype != torch.float32 or tuple(lse.shape) != (T, Hq) or not lse.is_contiguous()):
        raise ValueError(f"lse must be a contiguous float32 tensor of shape {(T, Hq)}")
    for name, n in (("max_tokens", max_tokens), ("window_tokens", window_tokens), ("sink_tokens", sink_tokens)):
        if not -1 << 31 <= int(n) < 1 << 31:  # (a field would keep the low 32 bits)
            raise ValueError(f"{name} does not fit 32 bits: {n}")
    _on_device(q, k_cache, v_cache, block_table, ctx_lens, cu_tokens, out, lse, workspace)
    p = sv_chunk_params()
    p.batch, p.num_q_heads, p.num_kv_heads, p.head_dim = B, Hq, Hkv, D
    p.page_size, p.num_pages, p.total_tokens, p.max_tokens = page, pages, T, int(max_tokens)
    p.max_pages_per_seq = width
    p.dtype = SV_BF16 if q.dtype == torch.bfloat16 else SV_FP16
    p.window_tokens, p.sink_tokens, p.sm_scale, p.flags = int(window_tokens), int(sink_tokens), float(sm_scale), 0
    p.q_stride = q.stride(0) if T > 1 else 0
    p.out_stride = out.stride(0) if T > 1 else 0
    p.q, p.k_cache, p.v_cache, p.out = q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), out.data_ptr()
    p.block_table, p.ctx_lens, p.cu_tokens = block_table.data_ptr(), ctx_lens.data_ptr(), cu_tokens.data_ptr()
    p.lse = None if lse is None else lse.data_ptr()
    p.workspace, p.workspace_bytes = _space(workspace)
    p.tensors = (q, k_cache, v_cache, block_table, ctx_lens, cu_tokens, out, lse, workspace)
    return p


def sv_chunk_attention_workspace_size(params: sv_chunk_params) -> int:
    n = c_size_t(0)
    _check(load().sv_chunk_attention_workspace_size(ctypes.byref(params), ctypes.byref(n)),
           "sv_chunk_attention_workspace_size")
    return int(n.value)


def sv_chunk_attention(params: sv_chunk_params, stream=None) -> None:
    """Causal attention of every sequence's new tokens over its paged cache,
    which already holds their K/V (see include/sv.h)."""
    device, handle = _where(stream)
    held = getattr(params, "tensors", None)
    if held is not None and held[0].get_device() != device:
        _on_device(held[0])
    _check(load().sv_chunk_attention(ctypes.byref(params), handle), "sv_chunk_attention")


def sv_kv_append(k, v, k_cache, v_cache, block_table, ctx_lens, cu_tokens, new_ctx_lens=None, workspace=None,
                 stream=None) -> None:
    """Copies a chunk's K/V to its cache slots.  k/v: [layers, T, Hkv, D], or
    [T, Hkv, D] with caches of one layer [pages, Hkv, page_size, D]; heads
    contiguous, any token and layer stride."""
    device, handle = _where(stream)
    status = _marshal().kv_append(k, v, k_cache, v_cache, block_table, ctx_lens, cu_tokens, new_ctx_lens, workspace,
                                  device, handle)
    if status != SV_OK:
        raise SvError(status, "sv_kv_append")


def sv_pages_workspace_size(rows: int, num_pages: int) -> int:
    n = c_size_t(0)
    _check(load().sv_pages_workspace_size(rows, num_pages, ctypes.byref(n)), "sv_pages_workspace_size")
    return int(n.value)


def sv_pages_release(keep_lens, block_table, held_pages, page_refs, page_size: int = 16, workspace=None,
                     stream=None) -> None:
    """Gives back the pages behind keep_lens[b] tokens of every row."""
    device, handle = _where(stream)
    status = _marshal().pages_release(keep_lens, block_table, held_pages, page_refs, page_size, workspace, device, handle)
    if status != SV_OK:
        raise SvError(status, "sv_pages_release")


def sv_pages_fork(parents, children, block_table, ctx_lens, held_pages, page_refs, page_size: int = 16,
                  workspace=None, stream=None) -> None:
    """Row children[i] becomes a copy of row parents[i] that shares its pages."""
    device, handle = _where(stream)
    status = _marshal().pages_fork(parents, children, block_table, ctx_lens, held_pages, page_refs, page_size, workspace,
                                   device, handle)
    if status != SV_OK:
        raise SvError(status, "sv_pages_fork")


def sv_pages_reserve(ctx_lens, new_lens, block_table, held_pages, page_refs, copy_src, copy_dst, copy_count,
                     page_size: int = 16, workspace=None, stream=None) -> None:
    """Makes the slots ctx_lens[b] .. new_lens[b] - 1 of every row writable and
    lists the pages to copy (sv_pages_copy) for those it had to replace."""
    device, handle = _where(stream)
    status = _marshal().pages_reserve(ctx_lens, new_lens, block_table, held_pages, page_refs, copy_src, copy_dst,
                                      copy_count, page_size, workspace, device, handle)
    if status != SV_OK:
        raise SvError(status, "sv_pages_reserve")


def sv_pages_compact(block_table, held_pages, page_refs, block_table_out, page_refs_out, copy_src, copy_dst,
                     copy_count, num_live, workspace=None, stream=None) -> None:
    """Moves the used pages to the front of the pool: lists the copies and
    writes the tables and references after them (the outputs may be the
    inputs themselves)."""
    device, handle = _where(stream)
    status = _marshal().pages_compact(block_table, held_pages, page_refs, block_table_out, page_refs_out, copy_src,
                                      copy_dst, copy_count, num_live, workspace, device, handle)
    if status != SV_OK:
        raise SvError(status, "sv_pages_compact")


def sv_pages_copy(k_cache, v_cache, copy_src, copy_dst, copy_count, workspace=None, stream=None) -> None:
    """Copies the listed pages in every layer.  Caches [layers, pages, ...] of
    five dimensions, or one layer [pages, ...] of four; v_cache may be None.
    Page summaries [pages, Hkv, 2, D] are such a pool too."""
    device, handle = _where(stream)
    status = _marshal().pages_copy(k_cache, v_cache, copy_src, copy_dst, copy_count, workspace, device, handle)
    if status != SV_OK:
        raise SvError(status, "sv_pages_copy")


TRACE_SLOTS = 16
TRACE_EVENTS = ["start_ns", "prologue", "inputs", "first_ids", "first_mma", "first_s", "loop_end", "o_ready",
                "epilogue", "merge_ready", "merge_done", "exit", "tree_mask"]


def sv_set_trace_buffer(buffer, nbytes: int = 0) -> None:
    """Install (or with None remove) the per-CTA phase trace buffer."""
    if buffer is not None and not nbytes:
        nbytes = buffer.numel() * buffer.element_size()
    _check(load().sv_set_trace_buffer(_ptr(buffer), nbytes), "sv_set_trace_buffer")


def sv_get_device_error(workspace, stream=None) -> int:
    """Returns the workspace's device error code (0 = none) and clears it."""
    code = c_int(0)
    st = load().sv_get_device_error(_ptr(workspace), ctypes.byref(code), _stream(stream))
    if st not in (SV_OK, 5, 6):
        _check(st, "sv_get_device_error")
    return int(code.value)
