"""Python binding of ``libtsd.so``, the GB300 tree-speculative-decoding verify step.

Argument marshalling only: every function takes torch CUDA tensors, checks
their element types and shapes, passes their device pointers to the C ABI
declared in ``include/tsd.h`` (same names), and raises :class:`TsdError` on a
non-OK status.  All arithmetic runs in the library's CUDA kernels; there is no
CPU fallback.  The library is loaded on first use (``lib``), so importing the
package, or its input generators in ``workloads``, maps nothing; the first
call fails with ImportError if the compiled library is missing.

Typical step on one stream::

    ws = workspace(...)                      # caller-owned scratch
    tsd_tree_build(probs, root, D, tree..., ws_build, err)
    tsd_tree_verify_attn(desc, q, kcache, vcache, prefix_len, ktree, vtree,
                         tree.mask, out, lse, ws_verify, err)
    tsd_accept_walk(logits, S, tree..., walk..., ws_walk, err)
    tsd_commit_path(desc, S, ktree, vtree, walk.accept_rows, walk.accept_len,
                    kcache, vcache, prefix_len, err)

or the last two as one call, ``tsd_accept_commit`` (the walk's kernel commits
the path it finds).
"""

from __future__ import annotations

import ctypes
import math
import os

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libtsd.so")

TSD_OK = 0
TSD_ERR_INVALID_ARG = 1
TSD_ERR_UNSUPPORTED = 2
TSD_ERR_CUDA = 3
TSD_ERR_DEVICE = 4
TSD_ERR_DEVICE_TIMEOUT = 5
TSD_DEV_ERR_CAPACITY = 0x01000000
TSD_DEV_ERR_BAD_TREE = 0x02000000
TSD_DEV_ERR_BAD_PAGE = 0x04000000
TSD_DEV_ERR_BAD_PROBS = 0x05000000
TSD_DEV_ERR_TIMEOUT = 0x03000000
TSD_DEV_ERR_MASK = 0x7F000000
TSD_F32 = 0
TSD_BF16 = 1
TSD_Q8_BLOCK = 64
TSD_Q4_GROUP = 32
VERIFY_PATHS = {"auto": 0, "generic": 1, "mma": 2, "tc": 3}   # TSD_PATH_* of tsd.h

# every symbol the header declares
EXPORTED = ("tsd_status_string", "tsd_version", "tsd_tree_build_workspace_size",
            "tsd_tree_build", "tsd_tree_build_adaptive", "tsd_tree_build_conditioned",
            "tsd_verify_workspace_size",
            "tsd_tree_verify_attn", "tsd_tree_verify_attn_paged", "tsd_commit_path_paged",
            "tsd_accept_walk_workspace_size", "tsd_accept_walk", "tsd_accept_walk_static",
            "tsd_commit_path", "tsd_accept_commit", "tsd_target_argmax", "tsd_walk_commit",
            "tsd_set_verify_path", "tsd_set_wait_budget",
            "tsd_cache_write_q8", "tsd_commit_path_q8", "tsd_verify_q8_workspace_size",
            "tsd_tree_verify_attn_q8", "tsd_cache_weights", "tsd_cache_weights_q8",
            "tsd_cache_evict_workspace_size", "tsd_cache_evict", "tsd_cache_evict_q8",
            "tsd_cache_write_q4", "tsd_commit_path_q4", "tsd_cache_read_q4",
            "tsd_verify_q4_workspace_size", "tsd_tree_verify_attn_q4", "tsd_qk_norm_rope")


class TsdError(RuntimeError):
    def __init__(self, func, status):
        self.status = status
        super().__init__(f"{func}: {tsd_status_string(status)} (status {status})")


class tsd_attn_desc(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int), ("R", ctypes.c_int), ("Hq", ctypes.c_int),
                ("Hkv", ctypes.c_int), ("dk", ctypes.c_int), ("dv", ctypes.c_int),
                ("cap", ctypes.c_int), ("dtype", ctypes.c_int), ("v_aliases_k", ctypes.c_int),
                ("scale", ctypes.c_float)]


class tsd_rope_desc(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int), ("T", ctypes.c_int), ("Hq", ctypes.c_int),
                ("Hkv", ctypes.c_int), ("d", ctypes.c_int), ("dtype", ctypes.c_int),
                ("rot", ctypes.c_int), ("neighbours", ctypes.c_int), ("axes", ctypes.c_int),
                ("norm", ctypes.c_int), ("eps", ctypes.c_float), ("amplitude", ctypes.c_float)]


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"libtsd.so not built ({LIB_PATH}); run __graft_entry__.build()")
    lib = ctypes.CDLL(LIB_PATH)
    P, I, Z = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
    lib.tsd_status_string.argtypes = [I]
    lib.tsd_status_string.restype = ctypes.c_char_p
    lib.tsd_version.restype = I
    lib.tsd_tree_build_workspace_size.argtypes = [I, I, I, I]
    lib.tsd_tree_build_workspace_size.restype = Z
    lib.tsd_tree_build.argtypes = [P, I, I, I, I, I, P, P, P, P, P, P, P, P, Z, P, P]
    lib.tsd_tree_build.restype = I
    lib.tsd_tree_build_adaptive.argtypes = [P, I, I, I, I, I, P, P, P, P, P, P, P, P, P, P, P, Z,
                                            P, P]
    lib.tsd_tree_build_adaptive.restype = I
    lib.tsd_tree_build_conditioned.argtypes = [P, P, P, I, I, I, P, P, P, P, P, P, P, P, P]
    lib.tsd_tree_build_conditioned.restype = I
    lib.tsd_verify_workspace_size.argtypes = [ctypes.POINTER(tsd_attn_desc)]
    lib.tsd_verify_workspace_size.restype = Z
    lib.tsd_tree_verify_attn.argtypes = [ctypes.POINTER(tsd_attn_desc), P, P, P, P, P, P, P, P,
                                         P, P, Z, P, P]
    lib.tsd_tree_verify_attn.restype = I
    lib.tsd_accept_walk_workspace_size.argtypes = [I, I, I]
    lib.tsd_accept_walk_workspace_size.restype = Z
    lib.tsd_accept_walk.argtypes = [P, I, I, I, I, P, P, P, P, P, P, P, P, P, P, Z, P, P]
    lib.tsd_accept_walk.restype = I
    lib.tsd_accept_walk_static.argtypes = [P, I, I, I, I, P, P, P, P, P, P, P, P, P, P, P]
    lib.tsd_accept_walk_static.restype = I
    lib.tsd_commit_path.argtypes = [ctypes.POINTER(tsd_attn_desc), I, P, P, P, P, P, P, P, P, P]
    lib.tsd_commit_path.restype = I
    lib.tsd_tree_verify_attn_paged.argtypes = [ctypes.POINTER(tsd_attn_desc), P, P, P, P, I, I, I,
                                               P, P, P, P, P, P, P, Z, P, P]
    lib.tsd_tree_verify_attn_paged.restype = I
    lib.tsd_commit_path_paged.argtypes = [ctypes.POINTER(tsd_attn_desc), I, P, P, P, P, P, P, P, I,
                                          I, I, P, P, P]
    lib.tsd_commit_path_paged.restype = I
    lib.tsd_accept_commit.argtypes = [P, I, I, I, I, P, P, P, P, P, P, P, P, P,
                                      ctypes.POINTER(tsd_attn_desc), P, P, P, P, P, I, I, I, P,
                                      P, Z, P, P]
    lib.tsd_accept_commit.restype = I
    lib.tsd_target_argmax.argtypes = [P, I, I, I, P, Z, P]
    lib.tsd_target_argmax.restype = I
    lib.tsd_walk_commit.argtypes = [I, I, I, I, P, P, P, P, P, P, P, P, P,
                                    ctypes.POINTER(tsd_attn_desc), P, P, P, P, P, I, I, I, P, P,
                                    Z, P, P]
    lib.tsd_walk_commit.restype = I
    D, F = ctypes.POINTER(tsd_attn_desc), ctypes.c_float
    paging = [P, I, I, I]
    lib.tsd_cache_write_q8.argtypes = [D, I, P, P, P, P, P, P, P, *paging, P, P, P]
    lib.tsd_cache_write_q8.restype = I
    lib.tsd_commit_path_q8.argtypes = [D, I, P, P, P, P, P, P, P, P, *paging, P, P, P]
    lib.tsd_commit_path_q8.restype = I
    lib.tsd_verify_q8_workspace_size.argtypes = [D]
    lib.tsd_verify_q8_workspace_size.restype = Z
    lib.tsd_tree_verify_attn_q8.argtypes = [D, P, P, P, P, P, *paging, P, P, P, P, P, P, P, Z, P, P]
    lib.tsd_tree_verify_attn_q8.restype = I
    lib.tsd_cache_weights.argtypes = [D, I, P, P, *paging, P, P, P, P, P, F, P, P, P, P, P]
    lib.tsd_cache_weights.restype = I
    lib.tsd_cache_weights_q8.argtypes = [D, I, P, P, P, *paging, P, P, P, P, P, F, P, P, P, P, P]
    lib.tsd_cache_weights_q8.restype = I
    lib.tsd_cache_evict_workspace_size.argtypes = [D]
    lib.tsd_cache_evict_workspace_size.restype = Z
    lib.tsd_cache_evict.argtypes = [D, I, I, I, P, P, P, P, P, *paging, P, P, Z, P, P]
    lib.tsd_cache_evict.restype = I
    lib.tsd_cache_evict_q8.argtypes = [D, I, I, I, P, P, P, P, P, P, P, *paging, P, P, Z, P, P]
    lib.tsd_cache_evict_q8.restype = I
    lib.tsd_cache_write_q4.argtypes = [D, I, P, P, P, P, P, P, P, *paging, P, P, P]
    lib.tsd_cache_write_q4.restype = I
    lib.tsd_commit_path_q4.argtypes = [D, I, P, P, P, P, P, P, P, P, *paging, P, P, P]
    lib.tsd_commit_path_q4.restype = I
    lib.tsd_cache_read_q4.argtypes = [D, I, P, P, P, P, *paging, P, P, P, P, P, P, P]
    lib.tsd_cache_read_q4.restype = I
    lib.tsd_verify_q4_workspace_size.argtypes = [D]
    lib.tsd_verify_q4_workspace_size.restype = Z
    lib.tsd_tree_verify_attn_q4.argtypes = [D, P, P, P, P, P, *paging, P, P, P, P, P, P, P, Z, P, P]
    lib.tsd_tree_verify_attn_q4.restype = I
    L = ctypes.c_int64
    lib.tsd_qk_norm_rope.argtypes = [ctypes.POINTER(tsd_rope_desc), P, L, P, L, P, L, P, P, P, P, P,
                                     I, P, P, P, P, P]
    lib.tsd_qk_norm_rope.restype = I
    lib.tsd_set_verify_path.argtypes = [I]
    lib.tsd_set_verify_path.restype = I
    lib.tsd_set_wait_budget.argtypes = [ctypes.c_longlong]
    lib.tsd_set_wait_budget.restype = ctypes.c_longlong
    return lib


_lib = None


def _L():
    """The loaded library (loaded on first use; ImportError if it is not built)."""
    global _lib
    if _lib is None:
        _lib = _load()
    return _lib


def __getattr__(name):
    if name == "lib":
        return _L()
    raise AttributeError(f"module {__name__!r} has no attribute {name!r}")


def tsd_set_verify_path(path) -> int:
    """Force an attention path ("auto", "generic", "mma", "tc" or a TSD_PATH_*
    value) for the verify calls that follow; returns the previous value."""
    code = VERIFY_PATHS[path] if isinstance(path, str) else int(path)
    prev = _L().tsd_set_verify_path(code)
    if prev < 0:
        raise ValueError(f"unknown verify path {path!r}")
    return prev


class verify_path:
    """Context manager: the verify calls inside use the given path."""

    def __init__(self, path):
        self.path = path

    def __enter__(self):
        self.prev = tsd_set_verify_path(self.path)
        return self

    def __exit__(self, *exc):
        tsd_set_verify_path(self.prev)
        return False


def tsd_set_wait_budget(cycles: int) -> int:
    """Budget (SM clock cycles) of the pipeline waits of the tcgen05 verify, 8-bit
    attention and weights kernels for the calls that follow; 0 restores the
    default.  Returns the previous setting."""
    if int(cycles) < 0:
        raise ValueError("wait budget must be >= 0")
    return int(_L().tsd_set_wait_budget(int(cycles)))


class wait_budget:
    """Context manager: the calls inside use the given wait budget."""

    def __init__(self, cycles):
        self.cycles = cycles

    def __enter__(self):
        self.prev = tsd_set_wait_budget(self.cycles)
        return self

    def __exit__(self, *exc):
        tsd_set_wait_budget(self.prev)
        return False


def tsd_status_string(status: int) -> str:
    return _L().tsd_status_string(int(status)).decode()


def tsd_version() -> int:
    return _L().tsd_version()


def _ptr(t):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("tensor must live on a CUDA device")
    if not t.is_contiguous():
        raise ValueError("tensor must be contiguous")
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def _check(func, status):
    if status != TSD_OK:
        raise TsdError(func, status)


def _nbytes(ws):
    return 0 if ws is None else ws.numel() * ws.element_size()


def make_desc(B, R, Hq, Hkv, dk, dv, cap, dtype, v_aliases_k, scale) -> tsd_attn_desc:
    if isinstance(dtype, torch.dtype):
        dtype = TSD_BF16 if dtype == torch.bfloat16 else TSD_F32
    return tsd_attn_desc(B, R, Hq, Hkv, dk, dv, cap, dtype, 1 if v_aliases_k else 0, scale)


def workspace(nbytes: int, device=None) -> torch.Tensor:
    """Caller-owned device scratch of at least nbytes (16-byte aligned)."""
    return torch.empty(max(int(nbytes), 16), dtype=torch.uint8, device=device or "cuda")


# ------------------------------------------------------------------ calls --

_I32, _F32, _U8 = torch.int32, torch.float32, torch.uint8
_MASK = (torch.int64,) + ((torch.uint64,) if hasattr(torch, "uint64") else ())


def _t(t, name, dtypes, shape=None):
    """Device pointer of ``t`` after checking its element type and shape
    (None passes through as a NULL pointer)."""
    if t is None:
        return None
    if not isinstance(dtypes, tuple):
        dtypes = (dtypes,)
    if t.dtype not in dtypes:
        raise TypeError(f"{name}: element type {t.dtype}, expected "
                        f"{' or '.join(str(d) for d in dtypes)}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")
    return _ptr(t)


def _err(err):
    return _t(err, "err", _I32)


def _tree(B, R, token, parent, depth, score, mask, is_leaf):
    return (_t(token, "token", _I32, (B, R)), _t(parent, "parent", _I32, (B, R)),
            _t(depth, "depth", _I32, (B, R)), _t(score, "score", _F32, (B, R)),
            _t(mask, "mask", _MASK, (B, R)), _t(is_leaf, "is_leaf", _U8, (B, R)))


def _attn_dtype(desc):
    return torch.bfloat16 if desc.dtype == TSD_BF16 else torch.float32


def tsd_tree_build_workspace_size(B, S, V, k) -> int:
    return _L().tsd_tree_build_workspace_size(B, S, V, k)


def tsd_tree_build(probs, k, D, root_tok, token, parent, depth, score, mask, is_leaf, ws,
                   err=None, stream=None):
    B, S, V = probs.shape
    _check("tsd_tree_build", _L().tsd_tree_build(
        _t(probs, "probs", _F32), B, S, V, k, D, _t(root_tok, "root_tok", _I32, (B,)),
        *_tree(B, D + 1, token, parent, depth, score, mask, is_leaf), _ptr(ws), _nbytes(ws),
        _err(err), _stream(stream)))


def tsd_tree_build_adaptive(probs, k, D_max, root_tok, cost_d, cost_v, token, parent, depth,
                            score, mask, is_leaf, n_nodes, ws, err=None, stream=None):
    B, S, V = probs.shape
    _check("tsd_tree_build_adaptive", _L().tsd_tree_build_adaptive(
        _t(probs, "probs", _F32), B, S, V, k, D_max, _t(root_tok, "root_tok", _I32, (B,)),
        _t(cost_d, "cost_d", _F32, (B,)), _t(cost_v, "cost_v", _F32, (B, D_max + 1)),
        *_tree(B, D_max + 1, token, parent, depth, score, mask, is_leaf),
        _t(n_nodes, "n_nodes", _I32, (B,)), _ptr(ws), _nbytes(ws), _err(err), _stream(stream)))


def tsd_tree_build_conditioned(cand_p, cand_tok, cand_parent, D, root_tok, token, parent, depth,
                               score, mask, is_leaf, err=None, stream=None):
    B, C = cand_p.shape
    _check("tsd_tree_build_conditioned", _L().tsd_tree_build_conditioned(
        _t(cand_p, "cand_p", _F32), _t(cand_tok, "cand_tok", _I32, (B, C)),
        _t(cand_parent, "cand_parent", _I32, (B, C)), B, C, D,
        _t(root_tok, "root_tok", _I32, (B,)),
        *_tree(B, D + 1, token, parent, depth, score, mask, is_leaf), _err(err),
        _stream(stream)))


def tsd_verify_workspace_size(desc: tsd_attn_desc) -> int:
    return _L().tsd_verify_workspace_size(ctypes.byref(desc))


def _verify_common(desc, q, prefix_len, ktree, vtree, mask, out, lse):
    d = desc
    dt = _attn_dtype(d)
    alias = bool(d.v_aliases_k)
    return (_t(q, "q", dt, (d.B, d.R, d.Hq, d.dk)), _t(prefix_len, "prefix_len", _I32, (d.B,)),
            _t(ktree, "ktree", dt, (d.B, d.R, d.Hkv, d.dk)),
            None if alias else _t(vtree, "vtree", dt, (d.B, d.R, d.Hkv, d.dv)),
            _t(mask, "mask", _MASK, (d.B, d.R)), _t(out, "out", dt, (d.B, d.R, d.Hq, d.dv)),
            _t(lse, "lse", _F32, (d.B, d.R, d.Hq)))


def tsd_tree_verify_attn(desc, q, kcache, vcache, prefix_len, ktree, vtree, mask, out, lse, ws,
                         err=None, stream=None):
    d = desc
    dt = _attn_dtype(d)
    pq, pl, pkt, pvt, pm, po, pls = _verify_common(d, q, prefix_len, ktree, vtree, mask, out, lse)
    pkc = _t(kcache, "kcache", dt, (d.B, d.Hkv, d.cap, d.dk))
    pvc = None if d.v_aliases_k else _t(vcache, "vcache", dt, (d.B, d.Hkv, d.cap, d.dv))
    _check("tsd_tree_verify_attn", _L().tsd_tree_verify_attn(
        ctypes.byref(d), pq, pkc, pvc, pl, pkt, pvt, pm, po, pls, _ptr(ws), _nbytes(ws),
        _err(err), _stream(stream)))


def tsd_accept_walk_workspace_size(B, D, V) -> int:
    return _L().tsd_accept_walk_workspace_size(B, D, V)


def _walk_args(logits, S, token, parent, mask, is_leaf, tgt, accept_len, accept_rows, bonus,
               chain_id):
    B, R, V = logits.shape
    return (_t(logits, "logits", _F32), B, R - 1, S, V, _t(token, "token", _I32, (B, R)),
            _t(parent, "parent", _I32, (B, R)), _t(mask, "mask", _MASK, (B, R)),
            _t(is_leaf, "is_leaf", _U8, (B, R)), _t(tgt, "tgt", _I32, (B, R)),
            _t(accept_len, "accept_len", _I32, (B,)),
            _t(accept_rows, "accept_rows", _I32, (B, S + 1)), _t(bonus, "bonus", _I32, (B,)),
            _t(chain_id, "chain_id", _I32, (B,)))


def tsd_accept_walk(logits, S, token, parent, mask, is_leaf, tgt, accept_len, accept_rows, bonus,
                    chain_id, ws, err=None, stream=None):
    _check("tsd_accept_walk", _L().tsd_accept_walk(
        *_walk_args(logits, S, token, parent, mask, is_leaf, tgt, accept_len, accept_rows, bonus,
                    chain_id), _ptr(ws), _nbytes(ws), _err(err), _stream(stream)))


def tsd_accept_walk_static(logits, S, token, parent, mask, is_leaf, tgt, accept_len, accept_rows,
                           bonus, chain_id, err=None, stream=None):
    """tsd_accept_walk without a workspace (fixed in-library scratch; see tsd.h)."""
    _check("tsd_accept_walk_static", _L().tsd_accept_walk_static(
        *_walk_args(logits, S, token, parent, mask, is_leaf, tgt, accept_len, accept_rows, bonus,
                    chain_id), _err(err), _stream(stream)))


def tsd_tree_verify_attn_paged(desc, q, kpool, vpool, page_table, page_size, prefix_len, ktree,
                               vtree, mask, out, lse, ws, err=None, stream=None):
    """page_table [B][max_pages] int32; pools [num_pages][Hkv][page_size][d]."""
    d = desc
    dt = _attn_dtype(d)
    pq, pl, pkt, pvt, pm, po, pls = _verify_common(d, q, prefix_len, ktree, vtree, mask, out, lse)
    npg, mp = kpool.shape[0], page_table.shape[1]
    pkp = _t(kpool, "kpool", dt, (npg, d.Hkv, page_size, d.dk))
    pvp = None if d.v_aliases_k else _t(vpool, "vpool", dt, (npg, d.Hkv, page_size, d.dv))
    _check("tsd_tree_verify_attn_paged", _L().tsd_tree_verify_attn_paged(
        ctypes.byref(d), pq, pkp, pvp, _t(page_table, "page_table", _I32, (d.B, mp)), mp,
        page_size, npg, pl, pkt, pvt, pm, po, pls, _ptr(ws), _nbytes(ws), _err(err),
        _stream(stream)))


def _commit_common(desc, S, ktree, vtree, accept_rows, accept_len, prefix_len):
    d = desc
    dt = _attn_dtype(d)
    return (_t(ktree, "ktree", dt, (d.B, d.R, d.Hkv, d.dk)),
            None if d.v_aliases_k else _t(vtree, "vtree", dt, (d.B, d.R, d.Hkv, d.dv)),
            _t(accept_rows, "accept_rows", _I32, (d.B, S + 1)),
            _t(accept_len, "accept_len", _I32, (d.B,)),
            _t(prefix_len, "prefix_len", _I32, (d.B,)))


def tsd_commit_path_paged(desc, S, ktree, vtree, accept_rows, accept_len, kpool, vpool,
                          page_table, page_size, prefix_len, err=None, stream=None):
    d = desc
    dt = _attn_dtype(d)
    pkt, pvt, par, pal, ppl = _commit_common(d, S, ktree, vtree, accept_rows, accept_len,
                                             prefix_len)
    npg, mp = kpool.shape[0], page_table.shape[1]
    pkp = _t(kpool, "kpool", dt, (npg, d.Hkv, page_size, d.dk))
    pvp = None if d.v_aliases_k else _t(vpool, "vpool", dt, (npg, d.Hkv, page_size, d.dv))
    _check("tsd_commit_path_paged", _L().tsd_commit_path_paged(
        ctypes.byref(d), S, pkt, pvt, par, pal, pkp, pvp,
        _t(page_table, "page_table", _I32, (d.B, mp)), mp, page_size, npg, ppl, _err(err),
        _stream(stream)))


def tsd_commit_path(desc, S, ktree, vtree, accept_rows, accept_len, kcache, vcache, prefix_len,
                    err=None, stream=None):
    d = desc
    dt = _attn_dtype(d)
    pkt, pvt, par, pal, ppl = _commit_common(d, S, ktree, vtree, accept_rows, accept_len,
                                             prefix_len)
    pkc = _t(kcache, "kcache", dt, (d.B, d.Hkv, d.cap, d.dk))
    pvc = None if d.v_aliases_k else _t(vcache, "vcache", dt, (d.B, d.Hkv, d.cap, d.dv))
    _check("tsd_commit_path", _L().tsd_commit_path(
        ctypes.byref(d), S, pkt, pvt, par, pal, pkc, pvc, ppl, _err(err), _stream(stream)))


def _commit_targets(d, kcache, vcache, page_table, page_size):
    dt = _attn_dtype(d)
    if page_table is None:
        pkc = _t(kcache, "kcache", dt, (d.B, d.Hkv, d.cap, d.dk))
        pvc = None if d.v_aliases_k else _t(vcache, "vcache", dt, (d.B, d.Hkv, d.cap, d.dv))
        return pkc, pvc, (None, 0, 0, 0)
    npg, mp = kcache.shape[0], page_table.shape[1]
    pkc = _t(kcache, "kpool", dt, (npg, d.Hkv, page_size, d.dk))
    pvc = None if d.v_aliases_k else _t(vcache, "vpool", dt, (npg, d.Hkv, page_size, d.dv))
    return pkc, pvc, (_t(page_table, "page_table", _I32, (d.B, mp)), mp, page_size, npg)


def tsd_target_argmax(logits, ws, stream=None):
    """The argmax part of tsd_accept_commit: per-chunk candidates of every row into ws."""
    B, R, V = logits.shape
    _check("tsd_target_argmax", _L().tsd_target_argmax(
        _t(logits, "logits", _F32), B, R - 1, V, _ptr(ws), _nbytes(ws), _stream(stream)))


def tsd_walk_commit(V, S, token, parent, mask, is_leaf, tgt, accept_len, accept_rows, bonus,
                    chain_id, desc, ktree, vtree, kcache, vcache, prefix_len, ws, err=None,
                    stream=None, page_table=None, page_size=0):
    """The rest of tsd_accept_commit, from the candidates tsd_target_argmax left in ws."""
    d = desc
    B, R = token.shape
    if B != d.B or R != d.R:
        raise ValueError("tsd_walk_commit: tree batch / rows do not match desc (B, R)")
    pkt, pvt, _, _, ppl = _commit_common(d, S, ktree, vtree, accept_rows, accept_len, prefix_len)
    pkc, pvc, paging = _commit_targets(d, kcache, vcache, page_table, page_size)
    _check("tsd_walk_commit", _L().tsd_walk_commit(
        B, R - 1, S, V, _t(token, "token", _I32, (B, R)), _t(parent, "parent", _I32, (B, R)),
        _t(mask, "mask", _MASK, (B, R)), _t(is_leaf, "is_leaf", _U8, (B, R)),
        _t(tgt, "tgt", _I32, (B, R)), _t(accept_len, "accept_len", _I32, (B,)),
        _t(accept_rows, "accept_rows", _I32, (B, S + 1)), _t(bonus, "bonus", _I32, (B,)),
        _t(chain_id, "chain_id", _I32, (B,)), ctypes.byref(d), pkt, pvt, pkc, pvc, *paging, ppl,
        _ptr(ws), _nbytes(ws), _err(err), _stream(stream)))


def tsd_accept_commit(logits, S, token, parent, mask, is_leaf, tgt, accept_len, accept_rows,
                      bonus, chain_id, desc, ktree, vtree, kcache, vcache, prefix_len, ws,
                      err=None, stream=None, page_table=None, page_size=0):
    """tsd_accept_walk, then the commit of the accepted paths, in one call.

    kcache/vcache are the contiguous cache, or with ``page_table`` [B][max_pages]
    the page pools [num_pages][Hkv][page_size][d] of tsd_commit_path_paged.
    """
    d = desc
    walk = _walk_args(logits, S, token, parent, mask, is_leaf, tgt, accept_len, accept_rows,
                      bonus, chain_id)
    if walk[1] != d.B or walk[2] + 1 != d.R:
        raise ValueError("tsd_accept_commit: logits batch / rows do not match desc (B, R)")
    pkt, pvt, _, _, ppl = _commit_common(d, S, ktree, vtree, accept_rows, accept_len, prefix_len)
    pkc, pvc, paging = _commit_targets(d, kcache, vcache, page_table, page_size)
    _check("tsd_accept_commit", _L().tsd_accept_commit(
        *walk, ctypes.byref(d), pkt, pvt, pkc, pvc, *paging, ppl, _ptr(ws), _nbytes(ws),
        _err(err), _stream(stream)))


# ------------------------------------- the 8-bit cache, and eviction --

_CODES = (torch.uint8, torch.float8_e4m3fn)
_EXPS = (torch.uint8,) + ((torch.float8_e8m0fnu,) if hasattr(torch, "float8_e8m0fnu") else ())


def _p(t, name, dtypes, shape, dev):
    """Address of ``t`` after checking its element type, shape, density and device (the
    current one, ``dev``, where the call launches).  None passes through as NULL."""
    if t is None:
        return None
    if t.dtype not in dtypes:
        raise TypeError(f"{name}: element type {t.dtype}, expected "
                        f"{' or '.join(str(d) for d in dtypes)}")
    if t.shape != shape:
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.get_device() != dev:
        raise ValueError(f"{name}: tensor on {t.device}, but the current device is cuda:{dev}")
    if not t.is_contiguous():
        raise ValueError(f"{name}: tensor must be contiguous")
    return t.data_ptr()


_I32T, _F32T = (_I32,), (_F32,)


def _scratch(ws, err, dev):
    """(workspace address, its bytes), error word address."""
    if ws is not None and (ws.get_device() != dev or not ws.is_contiguous()):
        raise ValueError(f"ws: a contiguous tensor on cuda:{dev} is needed")
    return ((None, 0) if ws is None else (ws.data_ptr(), _nbytes(ws)),
            None if err is None else _p(err, "err", _I32T, err.shape, dev))


# The current stream's handle, without a stream object made for it (1.1 us a call).
_current_handle = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _raw_stream(stream, dev):
    if stream is None:
        if _current_handle is not None:
            return _current_handle(dev)
        stream = torch.cuda.current_stream(dev)
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def q8_blocks(cap) -> int:
    """Exponent bytes per head of a contiguous 8-bit cache of ``cap`` positions."""
    return -(-int(cap) // TSD_Q8_BLOCK)


class _Dims:
    """A descriptor's fields, read once, with the current device."""

    __slots__ = ("B", "R", "Hq", "Hkv", "dk", "dv", "cap", "alias", "dt", "dev", "ref")

    def __init__(self, desc):
        self.B, self.R, self.Hq, self.Hkv = desc.B, desc.R, desc.Hq, desc.Hkv
        self.dk, self.dv, self.cap = desc.dk, desc.dv, desc.cap
        self.alias = bool(desc.v_aliases_k)
        self.dt = (_attn_dtype(desc),)
        self.dev = torch.cuda.current_device()
        self.ref = ctypes.byref(desc)


def _cache_shapes(d, kcache, page_table, page_size):
    """Leading dims and rows of a contiguous or paged cache, and its page arguments."""
    if page_table is None:
        if page_size:
            raise ValueError("page_size without a page_table")
        return (d.B, d.Hkv, d.cap), (None, 0, 0, 0)
    npg, mp = kcache.shape[0], page_table.shape[1]
    return (npg, d.Hkv, page_size), (_p(page_table, "page_table", _I32T, (d.B, mp), d.dev), mp,
                                     page_size, npg)


def _q8_cache(d, kq, vq, kexp, vexp, page_table, page_size):
    lead, paging = _cache_shapes(d, kq, page_table, page_size)
    dev, exps = d.dev, (lead[0], lead[1], q8_blocks(lead[2]))
    pk = _p(kq, "kq", _CODES, (*lead, d.dk), dev)
    pke = _p(kexp, "kexp", _EXPS, exps, dev)
    if d.alias:
        return (pk, None, pke, None), paging
    if vq is None or vexp is None:
        raise ValueError("vq, vexp: needed unless V aliases K")
    return (pk, _p(vq, "vq", _CODES, (*lead, d.dv), dev), pke,
            _p(vexp, "vexp", _EXPS, exps, dev)), paging


def _rows(d, k, v, names, n):
    """Addresses of new rows [B][n][Hkv][dk | dv]."""
    return (_p(k, names[0], d.dt, (d.B, n, d.Hkv, d.dk), d.dev),
            None if d.alias else _p(v, names[1], d.dt, (d.B, n, d.Hkv, d.dv), d.dev))


def tsd_cache_write_q8(desc, knew, vnew, new_len, kq, vq, kexp, vexp, prefix_len, err=None,
                       stream=None, page_table=None, page_size=0):
    """Append rows knew/vnew [B][T][Hkv][d], new_len[b] of them, to the 8-bit cache."""
    d = _Dims(desc)
    T, one = knew.shape[1], (d.B,)
    cache, paging = _q8_cache(d, kq, vq, kexp, vexp, page_table, page_size)
    _check("tsd_cache_write_q8", _L().tsd_cache_write_q8(
        d.ref, T, *_rows(d, knew, vnew, ("knew", "vnew"), T), _p(new_len, "new_len", _I32T, one, d.dev),
        *cache, *paging, _p(prefix_len, "prefix_len", _I32T, one, d.dev),
        _scratch(None, err, d.dev)[1], _raw_stream(stream, d.dev)))


def tsd_commit_path_q8(desc, S, ktree, vtree, accept_rows, accept_len, kq, vq, kexp, vexp,
                       prefix_len, err=None, stream=None, page_table=None, page_size=0):
    """tsd_commit_path into the 8-bit cache."""
    d = _Dims(desc)
    one = (d.B,)
    cache, paging = _q8_cache(d, kq, vq, kexp, vexp, page_table, page_size)
    _check("tsd_commit_path_q8", _L().tsd_commit_path_q8(
        d.ref, S, *_rows(d, ktree, vtree, ("ktree", "vtree"), d.R),
        _p(accept_rows, "accept_rows", _I32T, (d.B, S + 1), d.dev),
        _p(accept_len, "accept_len", _I32T, one, d.dev), *cache, *paging,
        _p(prefix_len, "prefix_len", _I32T, one, d.dev), _scratch(None, err, d.dev)[1],
        _raw_stream(stream, d.dev)))


def tsd_verify_q8_workspace_size(desc: tsd_attn_desc) -> int:
    return _L().tsd_verify_q8_workspace_size(ctypes.byref(desc))


def tsd_tree_verify_attn_q8(desc, q, kq, vq, kexp, vexp, prefix_len, ktree, vtree, mask, out, lse,
                            ws, err=None, stream=None, page_table=None, page_size=0):
    """tsd_tree_verify_attn over the 8-bit cache (contiguous, or pages with ``page_table``)."""
    d = _Dims(desc)
    B, R, Hq, dev = d.B, d.R, d.Hq, d.dev
    cache, paging = _q8_cache(d, kq, vq, kexp, vexp, page_table, page_size)
    (pws, nws), perr = _scratch(ws, err, dev)
    _check("tsd_tree_verify_attn_q8", _L().tsd_tree_verify_attn_q8(
        d.ref, _p(q, "q", d.dt, (B, R, Hq, d.dk), dev), *cache, *paging,
        _p(prefix_len, "prefix_len", _I32T, (B,), dev), *_rows(d, ktree, vtree, ("ktree", "vtree"), R),
        _p(mask, "mask", _MASK, (B, R), dev), _p(out, "out", d.dt, (B, R, Hq, d.dv), dev),
        _p(lse, "lse", _F32T, (B, R, Hq), dev), pws, nws, perr, _raw_stream(stream, dev)))


def _weight_args(d, S, prefix_len, ktree, accept_rows, accept_len, lse, decay, acc, pos, seen):
    dev = d.dev
    return (_p(prefix_len, "prefix_len", _I32T, (d.B,), dev),
            _p(ktree, "ktree", d.dt, (d.B, d.R, d.Hkv, d.dk), dev),
            _p(accept_rows, "accept_rows", _I32T, (d.B, S + 1), dev),
            _p(accept_len, "accept_len", _I32T, (d.B,), dev),
            _p(lse, "lse", _F32T, (d.B, d.R, d.Hq), dev), float(decay),
            *_evict_state(d, acc, pos, seen))


def _evict_state(d, acc, pos, seen):
    rows = (d.B, d.Hkv, d.cap)
    return (_p(acc, "acc", _F32T, rows, d.dev), _p(pos, "pos", _I32T, rows, d.dev),
            _p(seen, "seen", _I32T, (d.B, d.Hkv), d.dev))


def tsd_cache_weights(desc, S, q, kcache, prefix_len, ktree, accept_rows, accept_len, lse, decay,
                      acc, pos, seen, err=None, stream=None, page_table=None, page_size=0):
    """Add the attention weight that the accepted rows gave each cached row to ``acc``."""
    d = _Dims(desc)
    lead, paging = _cache_shapes(d, kcache, page_table, page_size)
    _check("tsd_cache_weights", _L().tsd_cache_weights(
        d.ref, S, _p(q, "q", d.dt, (d.B, d.R, d.Hq, d.dk), d.dev),
        _p(kcache, "kcache", d.dt, (*lead, d.dk), d.dev), *paging,
        *_weight_args(d, S, prefix_len, ktree, accept_rows, accept_len, lse, decay, acc, pos, seen),
        _scratch(None, err, d.dev)[1], _raw_stream(stream, d.dev)))


def tsd_cache_weights_q8(desc, S, q, kq, kexp, prefix_len, ktree, accept_rows, accept_len, lse,
                         decay, acc, pos, seen, err=None, stream=None, page_table=None,
                         page_size=0):
    """tsd_cache_weights for the 8-bit cache."""
    d = _Dims(desc)
    lead, paging = _cache_shapes(d, kq, page_table, page_size)
    _check("tsd_cache_weights_q8", _L().tsd_cache_weights_q8(
        d.ref, S, _p(q, "q", d.dt, (d.B, d.R, d.Hq, d.dk), d.dev),
        _p(kq, "kq", _CODES, (*lead, d.dk), d.dev),
        _p(kexp, "kexp", _EXPS, (lead[0], lead[1], q8_blocks(lead[2])), d.dev), *paging,
        *_weight_args(d, S, prefix_len, ktree, accept_rows, accept_len, lse, decay, acc, pos, seen),
        _scratch(None, err, d.dev)[1], _raw_stream(stream, d.dev)))


def tsd_cache_evict_workspace_size(desc: tsd_attn_desc) -> int:
    return _L().tsd_cache_evict_workspace_size(ctypes.byref(desc))


def tsd_cache_evict(desc, keep, sink, recent, acc, pos, seen, kcache, vcache, prefix_len, ws,
                    err=None, stream=None, page_table=None, page_size=0):
    """Cut every request of more than ``keep`` cached rows to the ``keep`` heaviest ones."""
    d = _Dims(desc)
    lead, paging = _cache_shapes(d, kcache, page_table, page_size)
    (pws, nws), perr = _scratch(ws, err, d.dev)
    _check("tsd_cache_evict", _L().tsd_cache_evict(
        d.ref, keep, sink, recent, *_evict_state(d, acc, pos, seen),
        _p(kcache, "kcache", d.dt, (*lead, d.dk), d.dev),
        None if d.alias else _p(vcache, "vcache", d.dt, (*lead, d.dv), d.dev), *paging,
        _p(prefix_len, "prefix_len", _I32T, (d.B,), d.dev), pws, nws, perr,
        _raw_stream(stream, d.dev)))


def tsd_cache_evict_q8(desc, keep, sink, recent, acc, pos, seen, kq, vq, kexp, vexp, prefix_len,
                       ws, err=None, stream=None, page_table=None, page_size=0):
    """tsd_cache_evict for the 8-bit cache."""
    d = _Dims(desc)
    cache, paging = _q8_cache(d, kq, vq, kexp, vexp, page_table, page_size)
    (pws, nws), perr = _scratch(ws, err, d.dev)
    _check("tsd_cache_evict_q8", _L().tsd_cache_evict_q8(
        d.ref, keep, sink, recent, *_evict_state(d, acc, pos, seen), *cache, *paging,
        _p(prefix_len, "prefix_len", _I32T, (d.B,), d.dev), pws, nws, perr,
        _raw_stream(stream, d.dev)))


# ------------------------------------------- the 4-bit cache, and rotation --

_BF16 = (torch.bfloat16,)


def _q4_cache(d, kq, vq, kscale, vscale, page_table, page_size):
    lead, paging = _cache_shapes(d, kq, page_table, page_size)
    codes, scales, dev = (*lead, d.dk // 2), (*lead, d.dk // TSD_Q4_GROUP), d.dev
    return (_p(kq, "kq", (_U8,), codes, dev), _p(vq, "vq", (_U8,), codes, dev),
            _p(kscale, "kscale", _BF16, scales, dev),
            _p(vscale, "vscale", _BF16, scales, dev)), paging


def tsd_cache_write_q4(desc, knew, vnew, new_len, kq, vq, kscale, vscale, prefix_len, err=None,
                       stream=None, page_table=None, page_size=0):
    """Append rows knew/vnew [B][T][Hkv][d], new_len[b] of them, to the 4-bit cache."""
    d = _Dims(desc)
    T, one = knew.shape[1], (d.B,)
    cache, paging = _q4_cache(d, kq, vq, kscale, vscale, page_table, page_size)
    _check("tsd_cache_write_q4", _L().tsd_cache_write_q4(
        d.ref, T, *_rows(d, knew, vnew, ("knew", "vnew"), T), _p(new_len, "new_len", _I32T, one, d.dev),
        *cache, *paging, _p(prefix_len, "prefix_len", _I32T, one, d.dev),
        _scratch(None, err, d.dev)[1], _raw_stream(stream, d.dev)))


def tsd_commit_path_q4(desc, S, ktree, vtree, accept_rows, accept_len, kq, vq, kscale, vscale,
                       prefix_len, err=None, stream=None, page_table=None, page_size=0):
    """tsd_commit_path into the 4-bit cache."""
    d = _Dims(desc)
    one = (d.B,)
    cache, paging = _q4_cache(d, kq, vq, kscale, vscale, page_table, page_size)
    _check("tsd_commit_path_q4", _L().tsd_commit_path_q4(
        d.ref, S, *_rows(d, ktree, vtree, ("ktree", "vtree"), d.R),
        _p(accept_rows, "accept_rows", _I32T, (d.B, S + 1), d.dev),
        _p(accept_len, "accept_len", _I32T, one, d.dev), *cache, *paging,
        _p(prefix_len, "prefix_len", _I32T, one, d.dev), _scratch(None, err, d.dev)[1],
        _raw_stream(stream, d.dev)))


def tsd_cache_read_q4(desc, kq, vq, kscale, vscale, prefix_len, first, count, kout, vout, err=None,
                      stream=None, page_table=None, page_size=0):
    """Rows first[b] .. first[b] + count[b] - 1 of the 4-bit cache to kout/vout [B][T][Hkv][d]."""
    d = _Dims(desc)
    T, one = kout.shape[1], (d.B,)
    cache, paging = _q4_cache(d, kq, vq, kscale, vscale, page_table, page_size)
    _check("tsd_cache_read_q4", _L().tsd_cache_read_q4(
        d.ref, T, *cache, *paging, _p(prefix_len, "prefix_len", _I32T, one, d.dev),
        _p(first, "first", _I32T, one, d.dev), _p(count, "count", _I32T, one, d.dev),
        *_rows(d, kout, vout, ("kout", "vout"), T), _scratch(None, err, d.dev)[1],
        _raw_stream(stream, d.dev)))


def tsd_verify_q4_workspace_size(desc: tsd_attn_desc) -> int:
    return _L().tsd_verify_q4_workspace_size(ctypes.byref(desc))


def tsd_tree_verify_attn_q4(desc, q, kq, vq, kscale, vscale, prefix_len, ktree, vtree, mask, out,
                            lse, ws, err=None, stream=None, page_table=None, page_size=0):
    """tsd_tree_verify_attn over the 4-bit cache (contiguous, or pages with ``page_table``)."""
    d = _Dims(desc)
    B, R, Hq, dev = d.B, d.R, d.Hq, d.dev
    cache, paging = _q4_cache(d, kq, vq, kscale, vscale, page_table, page_size)
    (pws, nws), perr = _scratch(ws, err, dev)
    _check("tsd_tree_verify_attn_q4", _L().tsd_tree_verify_attn_q4(
        d.ref, _p(q, "q", d.dt, (B, R, Hq, d.dk), dev), *cache, *paging,
        _p(prefix_len, "prefix_len", _I32T, (B,), dev), *_rows(d, ktree, vtree, ("ktree", "vtree"), R),
        _p(mask, "mask", _MASK, (B, R), dev), _p(out, "out", d.dt, (B, R, Hq, d.dv), dev),
        _p(lse, "lse", _F32T, (B, R, Hq), dev), pws, nws, perr, _raw_stream(stream, dev)))


def make_rope_desc(B, T, Hq, Hkv, d, dtype, rot=None, axes=1, neighbours=False, norm=True, eps=1e-6,
                   amplitude=1.0) -> tsd_rope_desc:
    """``rot`` dims of a head are rotated (all of them by default)."""
    return tsd_rope_desc(B, T, Hq, Hkv, d, TSD_BF16 if dtype == torch.bfloat16 else TSD_F32,
                         d if rot is None else rot, int(neighbours), axes, int(norm), eps, amplitude)


# 2^192 / (2 pi), to the nearest whole number
_PER_RADIAN = 999031769477504631556283515717616693813654938713089696784


def rope_turns(freq, device=None):
    """``turns`` of tsd_qk_norm_rope from radians per position, [rot / 2] or [axes][rot / 2]
    (float64, below 2^20 in magnitude): int64 with the bits of the fraction of a turn times 2^64.
    A host computation in whole numbers; ``device`` is that of freq by default."""
    freq = torch.as_tensor(freq, dtype=torch.float64)
    device = freq.device if device is None else device
    bits = []
    for x in freq.flatten().tolist():
        if not abs(x) < 1 << 20:
            raise ValueError(f"freq: {x} radians per position, expected less than 2^20")
        m, e = math.frexp(x)                       # x = m 2^53 2^(e - 53)
        shift = 128 + 53 - e
        b = ((int(m * (1 << 53)) * _PER_RADIAN >> shift - 1) + 1 >> 1) & (1 << 64) - 1
        bits.append(b - (1 << 64) if b >> 63 else b)
    return torch.tensor(bits, dtype=torch.int64).view(-1, freq.shape[-1]).to(device)


_TURNS = _MASK


def _strided_rows(t, name, dt, shape, dev):
    """(address, elements between two tokens) of rows [B][T][H][d] that may be a view of a
    wider array; (None, 0) for None."""
    if t is None:
        return None, 0
    if t.dtype not in dt:
        raise TypeError(f"{name}: element type {t.dtype}, expected {dt[0]}")
    if t.shape != shape:
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.get_device() != dev:
        raise ValueError(f"{name}: tensor on {t.device}, but the current device is cuda:{dev}")
    B, T, H, d = shape
    sb, st, sh, sd = t.stride()
    if T == 1:
        st = sb if B > 1 else H * d
    if sd != 1 or (H > 1 and sh != d) or (B > 1 and sb != T * st):
        raise ValueError(f"{name}: strides {t.stride()}; tokens have to lie at one distance and a "
                         f"token's heads side by side")
    return t.data_ptr(), st


def tsd_qk_norm_rope(desc, q, k, v, turns, q_out, k_out, v_out, q_weight=None, k_weight=None,
                     start=None, offset=None, count=None, stream=None):
    """RMS norm of every head's query and key and the position rotation; v is copied (v and
    v_out may be None).  q, k, v [B][T][H][d] may be views of a fused projection; offset is
    [axes][B][T], or [1][B][T] for all axes."""
    B, T, Hq, Hkv, d, axes = desc.B, desc.T, desc.Hq, desc.Hkv, desc.d, desc.axes
    dt, dev = (_attn_dtype(desc),), torch.cuda.current_device()
    rows_q, rows_k, one = (B, T, Hq, d), (B, T, Hkv, d), (B,)
    own_axes = axes if offset is None or offset.shape[0] != 1 else 1
    _check("tsd_qk_norm_rope", _L().tsd_qk_norm_rope(
        ctypes.byref(desc), *_strided_rows(q, "q", dt, rows_q, dev),
        *_strided_rows(k, "k", dt, rows_k, dev), *_strided_rows(v, "v", dt, rows_k, dev),
        _p(q_weight, "q_weight", dt, (d,), dev), _p(k_weight, "k_weight", dt, (d,), dev),
        _p(turns, "turns", _TURNS, (axes, desc.rot // 2), dev), _p(start, "start", _I32T, one, dev),
        _p(offset, "offset", _I32T, (own_axes, B, T), dev), own_axes, _p(count, "count", _I32T, one, dev),
        _p(q_out, "q_out", dt, rows_q, dev), _p(k_out, "k_out", dt, rows_k, dev),
        _p(v_out, "v_out", dt, rows_k, dev), _raw_stream(stream, dev)))
