"""Python binding of libsparstar (C ABI in include/sparstar.h).

Argument marshalling only: every function reads device pointers, shapes and
the current CUDA stream from torch tensors, allocates missing outputs with
torch, and calls the entry point of the same name.  Every step of the path
runs in the library's kernels; there is no Python or CPU path.  Importing
this module fails when the library has not been built.
"""
import ctypes
import math
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libsparstar.so")
BLOCK = 128

OK, EINVAL, EDTYPE, ECUDA, ESIZE, ENODEV = range(6)
STATUS_BAD_INDEX = 0x1
STATUS_TIMEOUT = 0x2
STATUS_NO_PAGES = 0x4
STATUS_CLAMPED = 0x8
STATUS_SHARED = 0x10
KV4_WORK_ZEROS = 1024

_DTYPE = {torch.bfloat16: 0, torch.float32: 1}


class _Kv4Struct(ctypes.Structure):
    _fields_ = [(name, ctypes.c_void_p) for name in ("pages", "refs", "table", "lens", "work")] + \
               [(name, ctypes.c_int64) for name in ("n_pages", "n_seqs", "max_pages", "Hkv", "D")]


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError("libsparstar.so is not built (run block_sparse_attention_18_b200/build.py "
                          "or __graft_entry__.build()); there is no fallback path")
    L = ctypes.CDLL(LIB_PATH)
    i64, i32, f32, f64, vp = (ctypes.c_int64, ctypes.c_int, ctypes.c_float, ctypes.c_double,
                              ctypes.c_void_p)
    L.sparstar_block_pool.argtypes = [vp, i32, i64, i64, i64, i64, vp, vp]
    L.sparstar_block_score.argtypes = [vp, vp, i64, i64, i64, i64, i64, f32, vp, vp]
    L.sparstar_forced_blocks.argtypes = [i64, i64]
    L.sparstar_forced_blocks.restype = i64
    L.sparstar_select_count.argtypes = [i64, i64, f64]
    L.sparstar_select_count.restype = i64
    L.sparstar_select.argtypes = [vp, i64, i64, i64, i64, i64, f64, vp, vp, i64, vp]
    L.sparstar_attn_fwd.argtypes = [vp, vp, vp, i32, i64, i64, i64, i64, i64, f32, vp, vp, i64,
                                    vp, vp, vp, vp]
    L.sparstar_forward.argtypes = [vp, vp, vp, i32, i64, i64, i64, i64, i64, i64, i64, f64, vp,
                                   vp, vp, vp, vp, i64, vp, vp, vp, vp]
    L.sparstar_forward_static.argtypes = [vp, vp, vp, i32, i64, i64, i64, i64, i64, i64, i64, f64,
                                          vp, vp, vp, vp]
    L.sparstar_forward_static.restype = i32
    L.sparstar_block_pool_qk.argtypes = [vp, vp, i32, i64, i64, i64, i64, i64, vp, vp, vp]
    L.sparstar_score_select.argtypes = [vp, vp, i64, i64, i64, i64, i64, f32, i64, f64, vp, vp,
                                        i64, vp, vp]
    L.sparstar_score_select_max_nkb.argtypes = [i64]
    L.sparstar_score_select_max_nkb.restype = i64
    L.sparstar_forward_fused.argtypes = [vp, vp, vp, i32, i64, i64, i64, i64, i64, i64, i64, f64,
                                         vp, vp, vp, vp, i64, vp, vp, vp, vp]
    L.sparstar_retained_mass.argtypes = [vp, vp, i32, i64, i64, i64, i64, i64, f32, i64, vp, vp,
                                         i64, vp, i64, vp, vp, vp, vp, vp, vp]
    L.sparstar_transfer_lists.argtypes = [vp, vp, i64, i64, i64, vp, vp, vp, vp, i64, vp]
    L.sparstar_transfer_max_sel.argtypes = [vp, vp, i64]
    L.sparstar_transfer_max_sel.restype = i64
    L.sparstar_test_attn_timeout.argtypes = [vp, vp, vp, i64, i64, i64, i64, vp, vp, i64, vp, vp,
                                             vp]
    L.sparstar_test_attn_timeout.restype = i32
    L.sparstar_strerror.argtypes = [i32]
    L.sparstar_strerror.restype = ctypes.c_char_p
    L.sparstar_version.restype = i32
    kv4 = ctypes.POINTER(_Kv4Struct)
    L.sparstar_kv4_page_bytes.argtypes = [i64]
    L.sparstar_kv4_page_bytes.restype = i64
    L.sparstar_kv4_work_ints.argtypes = [i64, i64]
    L.sparstar_kv4_work_ints.restype = i64
    L.sparstar_kv4_resize.argtypes = [kv4, vp, vp, i64, vp, vp]
    L.sparstar_kv4_fork.argtypes = [kv4, vp, vp, vp, i64, i32, vp, vp]
    L.sparstar_kv4_compact.argtypes = [kv4, vp, vp]
    L.sparstar_test_kv4_compact_timeout.argtypes = [kv4, vp, vp]
    L.sparstar_test_kv4_compact_timeout.restype = i32
    L.sparstar_test_kv4_attn_timeout.argtypes = [kv4, vp, i32, i64, i64, i64, f32, vp, vp, i64, vp,
                                                 vp]
    L.sparstar_test_kv4_attn_timeout.restype = i32
    L.sparstar_kv4_write.argtypes = [kv4, vp, vp, i32, i64, i64, vp, vp, vp, vp, vp]
    L.sparstar_kv4_read.argtypes = [kv4, vp, vp, i32, i64, i64, vp, vp, vp, vp, vp]
    L.sparstar_kv4_attn.argtypes = [kv4, vp, i32, i64, i64, i64, vp, f32, i32, vp, vp, i64, vp,
                                    vp, vp, i64, vp, vp]
    L.sparstar_kv4_attn_work_bytes.argtypes = [i64, i64, i64, i64, i64, i32, i64, i64]
    L.sparstar_kv4_attn_work_bytes.restype = i64
    for name in ("sparstar_kv4_resize", "sparstar_kv4_fork", "sparstar_kv4_compact",
                 "sparstar_kv4_write", "sparstar_kv4_read", "sparstar_kv4_attn"):
        getattr(L, name).restype = i32
    for name in ("sparstar_block_pool", "sparstar_block_score", "sparstar_select",
                 "sparstar_attn_fwd", "sparstar_forward", "sparstar_block_pool_qk",
                 "sparstar_score_select", "sparstar_forward_fused", "sparstar_retained_mass",
                 "sparstar_transfer_lists"):
        getattr(L, name).restype = i32
    return L


lib = _load()


class SparstarError(RuntimeError):
    def __init__(self, code: int, where: str):
        self.code = code
        super().__init__("%s: %s (%d)" % (where, lib.sparstar_strerror(code).decode(), code))


def _check(code: int, where: str):
    if code != OK:
        raise SparstarError(code, where)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _dev(t: torch.Tensor, name: str, dtype=None):
    if not t.is_cuda:
        raise ValueError("%s must be a CUDA tensor" % name)
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    if dtype is not None and t.dtype != dtype:
        raise ValueError("%s must be %s, got %s" % (name, dtype, t.dtype))
    return t


def nblocks(L: int) -> int:
    return (L + BLOCK - 1) // BLOCK


def default_tau(D: int) -> float:
    return float(torch.tensor(1.0 / math.sqrt(D), dtype=torch.float32))


_TAU = {D: default_tau(D) for D in (64, 128)}


def sparstar_forced_blocks(text_len: int, image_ref_len: int) -> int:
    return lib.sparstar_forced_blocks(text_len, image_ref_len)


def sparstar_select_count(nKB: int, n_forced_blocks: int, density: float) -> int:
    return lib.sparstar_select_count(nKB, n_forced_blocks, density)


def sparstar_block_pool(x: torch.Tensor, xbar: torch.Tensor = None, stream=None) -> torch.Tensor:
    _dev(x, "x")
    B, H, L, D = x.shape
    if xbar is None:
        xbar = torch.empty(B, H, nblocks(L), D, device=x.device, dtype=torch.float32)
    _dev(xbar, "xbar", torch.float32)
    _check(lib.sparstar_block_pool(_ptr(x), _DTYPE.get(x.dtype, -1), B, H, L, D, _ptr(xbar),
                                   _stream(stream)), "sparstar_block_pool")
    return xbar


def sparstar_block_score(qbar: torch.Tensor, kbar: torch.Tensor, tau: float = None,
                         S: torch.Tensor = None, stream=None) -> torch.Tensor:
    _dev(qbar, "qbar", torch.float32)
    _dev(kbar, "kbar", torch.float32)
    B, H, nQB, D = qbar.shape
    nKB = kbar.shape[2]
    if tau is None:
        tau = default_tau(D)
    if S is None:
        S = torch.empty(B, H, nQB, nKB, device=qbar.device, dtype=torch.float32)
    _dev(S, "S", torch.float32)
    _check(lib.sparstar_block_score(_ptr(qbar), _ptr(kbar), B, H, nQB, nKB, D, tau, _ptr(S),
                                    _stream(stream)), "sparstar_block_score")
    return S


def sparstar_select(S: torch.Tensor, n_forced_blocks: int, density: float, max_sel: int = None,
                    kv_idx: torch.Tensor = None, kv_cnt: torch.Tensor = None, stream=None):
    _dev(S, "S", torch.float32)
    B, H, nQB, nKB = S.shape
    if max_sel is None:
        max_sel = kv_idx.shape[-1] if kv_idx is not None else \
            sparstar_select_count(nKB, n_forced_blocks, density)
        if max_sel < 0:
            raise SparstarError(EINVAL, "sparstar_select")
    if kv_idx is None:
        kv_idx = torch.empty(B, H, nQB, max_sel, device=S.device, dtype=torch.int32)
    if kv_cnt is None:
        kv_cnt = torch.empty(B, H, nQB, device=S.device, dtype=torch.int32)
    _dev(kv_idx, "kv_idx", torch.int32)
    _dev(kv_cnt, "kv_cnt", torch.int32)
    _check(lib.sparstar_select(_ptr(S), B, H, nQB, nKB, n_forced_blocks, density, _ptr(kv_idx),
                               _ptr(kv_cnt), max_sel, _stream(stream)), "sparstar_select")
    return kv_idx, kv_cnt


def sparstar_attn_fwd(q, k, v, kv_idx, kv_cnt, tau: float = None, out=None, lse=None,
                      status=None, want_lse: bool = True, stream=None):
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        _dev(t, n)
    _dev(kv_idx, "kv_idx", torch.int32)
    _dev(kv_cnt, "kv_cnt", torch.int32)
    B, H, Lq, D = q.shape
    Lk = k.shape[2]
    if tau is None:
        tau = default_tau(D)
    if out is None:
        out = torch.empty_like(q)
    if lse is None and want_lse:
        lse = torch.empty(B, H, Lq, device=q.device, dtype=torch.float32)
    _check(lib.sparstar_attn_fwd(_ptr(q), _ptr(k), _ptr(v), _DTYPE.get(q.dtype, -1), B, H, Lq,
                                 Lk, D, tau, _ptr(kv_idx), _ptr(kv_cnt), kv_idx.shape[-1],
                                 _ptr(out), _ptr(lse), _ptr(status), _stream(stream)),
           "sparstar_attn_fwd")
    return out, lse


class Workspace:
    """Caller-owned device buffers for one scale of ``sparstar_forward``."""

    def __init__(self, B, H, D, text_len, image_ref_len, ref_len, cur_len, density, device,
                 scores: bool = True):
        Lk = text_len + image_ref_len + ref_len + cur_len
        self.nQB, self.nKB = nblocks(cur_len), nblocks(Lk)
        self.n_forced = sparstar_forced_blocks(text_len, image_ref_len)
        self.max_sel = sparstar_select_count(self.nKB, self.n_forced, density)
        if self.max_sel < 0:
            raise SparstarError(EINVAL, "Workspace")
        f32, i32 = torch.float32, torch.int32
        self.qbar = torch.empty(B, H, self.nQB, D, device=device, dtype=f32)
        self.kbar = torch.empty(B, H, self.nKB, D, device=device, dtype=f32)
        # The fused front-end keeps the scores on chip and needs no S.
        self.S = torch.empty(B, H, self.nQB, self.nKB, device=device, dtype=f32) \
            if scores else None
        self.kv_idx = torch.empty(B, H, self.nQB, self.max_sel, device=device, dtype=i32)
        self.kv_cnt = torch.empty(B, H, self.nQB, device=device, dtype=i32)


def sparstar_forward(q, k, v, text_len, image_ref_len, ref_len, cur_len, density,
                     workspace: Workspace = None, out=None, lse=None, status=None,
                     want_lse: bool = True, stream=None):
    """All four steps for one scale on one stream; returns (out, lse, workspace)."""
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        _dev(t, n)
    B, H, Lq, D = q.shape
    ws = workspace or Workspace(B, H, D, text_len, image_ref_len, ref_len, cur_len, density,
                                q.device)
    if out is None:
        out = torch.empty_like(q)
    if lse is None and want_lse:
        lse = torch.empty(B, H, Lq, device=q.device, dtype=torch.float32)
    _check(lib.sparstar_forward(_ptr(q), _ptr(k), _ptr(v), _DTYPE.get(q.dtype, -1), B, H, D,
                                text_len, image_ref_len, ref_len, cur_len, density, _ptr(ws.qbar),
                                _ptr(ws.kbar), _ptr(ws.S), _ptr(ws.kv_idx), _ptr(ws.kv_cnt),
                                ws.max_sel, _ptr(out), _ptr(lse), _ptr(status), _stream(stream)),
           "sparstar_forward")
    return out, lse, ws


def sparstar_block_pool_qk(q: torch.Tensor, k: torch.Tensor, qbar: torch.Tensor = None,
                           kbar: torch.Tensor = None, stream=None):
    """Block means of q and k in one launch; returns (qbar, kbar)."""
    _dev(q, "q")
    _dev(k, "k")
    B, H, Lq, D = q.shape
    Lk = k.shape[2]
    if qbar is None:
        qbar = torch.empty(B, H, nblocks(Lq), D, device=q.device, dtype=torch.float32)
    if kbar is None:
        kbar = torch.empty(B, H, nblocks(Lk), D, device=q.device, dtype=torch.float32)
    _dev(qbar, "qbar", torch.float32)
    _dev(kbar, "kbar", torch.float32)
    dt = _DTYPE.get(q.dtype, -1) if k.dtype == q.dtype else -1
    _check(lib.sparstar_block_pool_qk(_ptr(q), _ptr(k), dt, B, H, Lq, Lk, D, _ptr(qbar),
                                      _ptr(kbar), _stream(stream)), "sparstar_block_pool_qk")
    return qbar, kbar


def sparstar_score_select_max_nkb(D: int) -> int:
    return lib.sparstar_score_select_max_nkb(D)


def sparstar_score_select(qbar: torch.Tensor, kbar: torch.Tensor, n_forced_blocks: int,
                          density: float, tau: float = None, max_sel: int = None,
                          kv_idx: torch.Tensor = None, kv_cnt: torch.Tensor = None, status=None,
                          stream=None):
    """Block scores and block Top-K in one launch (no S buffer); returns
    (kv_idx, kv_cnt)."""
    _dev(qbar, "qbar", torch.float32)
    _dev(kbar, "kbar", torch.float32)
    B, H, nQB, D = qbar.shape
    nKB = kbar.shape[2]
    if tau is None:
        tau = default_tau(D)
    if max_sel is None:
        max_sel = kv_idx.shape[-1] if kv_idx is not None else \
            sparstar_select_count(nKB, n_forced_blocks, density)
        if max_sel < 0:
            raise SparstarError(EINVAL, "sparstar_score_select")
    if kv_idx is None:
        kv_idx = torch.empty(B, H, nQB, max_sel, device=qbar.device, dtype=torch.int32)
    if kv_cnt is None:
        kv_cnt = torch.empty(B, H, nQB, device=qbar.device, dtype=torch.int32)
    _dev(kv_idx, "kv_idx", torch.int32)
    _dev(kv_cnt, "kv_cnt", torch.int32)
    _check(lib.sparstar_score_select(_ptr(qbar), _ptr(kbar), B, H, nQB, nKB, D, tau,
                                     n_forced_blocks, density, _ptr(kv_idx), _ptr(kv_cnt),
                                     max_sel, _ptr(status), _stream(stream)),
           "sparstar_score_select")
    return kv_idx, kv_cnt


def sparstar_forward_fused(q, k, v, text_len, image_ref_len, ref_len, cur_len, density,
                           workspace: Workspace = None, out=None, lse=None, status=None,
                           want_lse: bool = True, stream=None):
    """The three-launch chain (pool q and k, score + select, attention) for one
    scale on one stream; returns (out, lse, workspace).  The workspace needs
    no S buffer."""
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        _dev(t, n)
    B, H, Lq, D = q.shape
    ws = workspace or Workspace(B, H, D, text_len, image_ref_len, ref_len, cur_len, density,
                                q.device, scores=False)
    if out is None:
        out = torch.empty_like(q)
    if lse is None and want_lse:
        lse = torch.empty(B, H, Lq, device=q.device, dtype=torch.float32)
    _check(lib.sparstar_forward_fused(_ptr(q), _ptr(k), _ptr(v), _DTYPE.get(q.dtype, -1), B, H,
                                      D, text_len, image_ref_len, ref_len, cur_len, density,
                                      _ptr(ws.qbar), _ptr(ws.kbar), _ptr(ws.kv_idx),
                                      _ptr(ws.kv_cnt), ws.max_sel, _ptr(out), _ptr(lse),
                                      _ptr(status), _stream(stream)), "sparstar_forward_fused")
    return out, lse, ws


def sparstar_forward_static(q, k, v, text_len, image_ref_len, ref_len, cur_len, density,
                            out=None, lse=None, status=None, want_lse: bool = True, stream=None):
    """The four steps for one scale with the intermediates in the library's
    own device arena (no workspace); returns (out, lse).  For callers that
    cannot allocate device memory; calls that overlap on the GPU race on the
    shared arena."""
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        _dev(t, n)
    B, H, Lq, D = q.shape
    if out is None:
        out = torch.empty_like(q)
    if lse is None and want_lse:
        lse = torch.empty(B, H, Lq, device=q.device, dtype=torch.float32)
    _check(lib.sparstar_forward_static(_ptr(q), _ptr(k), _ptr(v), _DTYPE.get(q.dtype, -1), B, H,
                                       D, text_len, image_ref_len, ref_len, cur_len, density,
                                       _ptr(out), _ptr(lse), _ptr(status), _stream(stream)),
           "sparstar_forward_static")
    return out, lse


def sparstar_retained_mass(q, k, kv_idx, kv_cnt, n_forced_blocks: int, rows, tau: float = None,
                           scratch=None, stream=None):
    """Diagnostic: dense LSE, retained attention mass of the block lists, the
    forced-block mass and the token-wise bound at the same candidate budget,
    for the flat query rows given (int64 device tensor).  Returns a dict of
    fp64 device tensors."""
    _dev(q, "q")
    _dev(k, "k")
    _dev(kv_idx, "kv_idx", torch.int32)
    _dev(kv_cnt, "kv_cnt", torch.int32)
    _dev(rows, "rows", torch.int64)
    B, H, Lq, D = q.shape
    Lk = k.shape[2]
    n = rows.numel()
    if tau is None:
        tau = default_tau(D)
    if scratch is None:
        scratch = torch.empty(n, Lk, device=q.device, dtype=torch.float32)
    _dev(scratch, "scratch", torch.float32)
    out = {name: torch.empty(n, device=q.device, dtype=torch.float64)
           for name in ("lse_dense", "mass_block", "mass_tok", "mass_forced")}
    dt = _DTYPE.get(q.dtype, -1) if k.dtype == q.dtype else -1
    _check(lib.sparstar_retained_mass(_ptr(q), _ptr(k), dt, B, H, Lq, Lk, D, tau,
                                      n_forced_blocks, _ptr(kv_idx), _ptr(kv_cnt),
                                      kv_idx.shape[-1], _ptr(rows), n, _ptr(scratch),
                                      _ptr(out["lse_dense"]), _ptr(out["mass_block"]),
                                      _ptr(out["mass_tok"]), _ptr(out["mass_forced"]),
                                      _stream(stream)), "sparstar_retained_mass")
    return out


def _segs(src_len, dst_len):
    return ((ctypes.c_int64 * 4)(*[int(x) for x in src_len]),
            (ctypes.c_int64 * 4)(*[int(x) for x in dst_len]))


def sparstar_transfer_max_sel(src_len, dst_len, src_max_sel: int) -> int:
    """Longest row sparstar_transfer_lists can write for these layouts."""
    ls, lt = _segs(src_len, dst_len)
    return lib.sparstar_transfer_max_sel(ls, lt, src_max_sel)


def sparstar_transfer_lists(kv_idx, kv_cnt, src_len, dst_len, dst_idx=None, dst_cnt=None,
                            stream=None):
    """Diagnostic: block lists of a source scale carried by token position to
    a target scale (mask reuse).  src_len / dst_len: the four segment lengths
    (text, image_ref, ref, cur) at each scale.  Returns (dst_idx, dst_cnt);
    dst_idx's row stride is sparstar_transfer_max_sel(...) unless given."""
    _dev(kv_idx, "kv_idx", torch.int32)
    _dev(kv_cnt, "kv_cnt", torch.int32)
    B, H = kv_idx.shape[0], kv_idx.shape[1]
    ls, lt = _segs(src_len, dst_len)
    nQB_t = (int(dst_len[3]) + BLOCK - 1) // BLOCK
    if dst_idx is None:
        stride = lib.sparstar_transfer_max_sel(ls, lt, kv_idx.shape[-1])
        if stride < 0:
            raise SparstarError(EINVAL, "sparstar_transfer_lists")
        dst_idx = torch.empty(B, H, nQB_t, stride, device=kv_idx.device, dtype=torch.int32)
    if dst_cnt is None:
        dst_cnt = torch.empty(B, H, nQB_t, device=kv_idx.device, dtype=torch.int32)
    _dev(dst_idx, "dst_idx", torch.int32)
    _dev(dst_cnt, "dst_cnt", torch.int32)
    _check(lib.sparstar_transfer_lists(_ptr(kv_idx), _ptr(kv_cnt), kv_idx.shape[-1], B, H, ls, lt,
                                       _ptr(dst_idx), _ptr(dst_cnt), dst_idx.shape[-1],
                                       _stream(stream)), "sparstar_transfer_lists")
    return dst_idx, dst_cnt


def sparstar_kv4_page_bytes(D: int) -> int:
    return lib.sparstar_kv4_page_bytes(D)


class Kv4Cache:
    """Caller-owned device buffers of a paged 4-bit key/value cache.

    ``Kv4Cache.empty(...)`` allocates an empty one; the constructor takes
    buffers that the caller has: pages [n_pages, Hkv, page_bytes(D)] uint8,
    refs [n_pages], table [n_seqs, max_pages] and lens [n_seqs] int32, and
    the scratch ``work`` of the page calls (allocated when not given).
    """

    def __init__(self, pages, refs, table, lens, D: int, work=None):
        _dev(pages, "pages", torch.uint8)
        for t, name in ((refs, "refs"), (table, "table"), (lens, "lens")):
            _dev(t, name, torch.int32)
            if t.device != pages.device:
                raise ValueError("%s must be on %s, got %s" % (name, pages.device, t.device))
        n_pages, n_seqs = refs.numel(), lens.numel()
        if pages.dim() != 3 or pages.shape[0] != n_pages \
                or pages.shape[2] != sparstar_kv4_page_bytes(D):
            raise ValueError("pages must be [n_pages, Hkv, page_bytes(D)], got %s"
                             % (tuple(pages.shape),))
        if refs.dim() != 1 or lens.dim() != 1 or table.dim() != 2 or table.shape[0] != n_seqs:
            raise ValueError("refs must be [n_pages], lens [n_seqs] and table [n_seqs, max_pages]")
        ints = lib.sparstar_kv4_work_ints(n_pages, n_seqs)
        if ints < 0:
            raise SparstarError(EINVAL, "Kv4Cache")
        if work is None:
            work = torch.empty(ints, device=pages.device, dtype=torch.int32)
        _dev(work, "work", torch.int32)
        if work.numel() < ints or work.device != pages.device:
            raise ValueError("work must hold %d int32 on %s" % (ints, pages.device))
        self.pages, self.refs, self.table, self.lens, self.work = pages, refs, table, lens, work
        self.n_pages, self.n_seqs, self.max_pages = n_pages, n_seqs, table.shape[1]
        self.Hkv, self.D, self.device = pages.shape[1], D, pages.device
        self.index = pages.get_device()
        self._work_of = {}  # stream handle -> scratch of its attention calls
        self._need = {}     # sizes of an attention call -> bytes of its scratch, a like of its lse
        self._struct = _Kv4Struct(pages.data_ptr(), refs.data_ptr(), table.data_ptr(),
                                  lens.data_ptr(), work.data_ptr(), n_pages, n_seqs,
                                  table.shape[1], pages.shape[1], D)

    def _attn_work(self, need: int, stream: int):
        """Scratch for attention calls on this stream, the current one."""
        if torch._C._cuda_isCurrentStreamCapturing():
            return self._new_work(need)
        work = self._work_of.get(stream)
        if work is None or work.numel() < need:
            work = self._work_of[stream] = self._new_work(need)
        return work

    def _new_work(self, need: int):
        work = torch.empty(need, dtype=torch.uint8, device=self.device)
        work[:KV4_WORK_ZEROS].zero_()
        return work

    def drop_work(self):
        """Gives up the scratch of attention calls: the next calls take fresh
        one, as they have to after a call that set STATUS_TIMEOUT."""
        self._work_of.clear()

    @classmethod
    def empty(cls, n_pages: int, n_seqs: int, max_pages: int, Hkv: int, D: int, device="cuda"):
        i32 = dict(device=device, dtype=torch.int32)
        per_head = sparstar_kv4_page_bytes(D)
        if per_head < 0 or min(n_pages, n_seqs, max_pages, Hkv) < 1:
            raise SparstarError(EINVAL, "Kv4Cache.empty")
        return cls(torch.empty(n_pages, Hkv, per_head, device=device, dtype=torch.uint8),
                   torch.zeros(n_pages, **i32), torch.full((n_seqs, max_pages), -1, **i32),
                   torch.zeros(n_seqs, **i32), D)


def _kv4_ints(cache, t, name, n):
    """A device list of n int32 (or None): its pointer."""
    if t is None:
        return None
    if t.dtype is not torch.int32 or t.dim() != 1 or t.shape[0] != n \
            or t.get_device() != cache.index or not t.is_contiguous():
        raise ValueError("%s must be contiguous int32 [%d] on %s" % (name, n, cache.device))
    return t.data_ptr()


def _kv4_tensor(cache, t, name, dtype, shape):
    if t.dtype is not dtype or t.shape != shape or t.get_device() != cache.index \
            or not t.is_contiguous():
        raise ValueError("%s must be contiguous %s %s on %s, got %s %s on %s"
                         % (name, dtype, tuple(shape), cache.device, t.dtype, tuple(t.shape),
                            t.device))
    return t.data_ptr()


def _kv4_status(cache, status):
    return None if status is None else _kv4_tensor(cache, status, "status", torch.int32, (1,))


def _kv4_elsewhere(cache, stream):
    """Whether a call has to switch to the cache's device or another stream."""
    if stream is not None and stream.device_index != cache.index:
        raise ValueError("stream must be one of %s" % (cache.device,))
    return stream is not None or torch._C._cuda_getDevice() != cache.index


class _Kv4There:
    """The cache's device and the stream given as the current ones."""

    def __init__(self, cache, stream):
        self.device, self.stream = torch.cuda.device(cache.index), torch.cuda.stream(stream)

    def __enter__(self):
        self.device.__enter__()
        self.stream.__enter__()

    def __exit__(self, *exc):
        self.stream.__exit__(*exc)
        self.device.__exit__(*exc)
        return False


def _kv4_raw_stream(cache):
    return torch._C._cuda_getCurrentRawStream(cache.index)


def sparstar_kv4_resize(cache: Kv4Cache, new_lens, seqs=None, status=None, stream=None):
    """Sets the lengths of n sequences (0 frees one); takes and gives pages."""
    if _kv4_elsewhere(cache, stream):
        with _Kv4There(cache, stream):
            return sparstar_kv4_resize(cache, new_lens, seqs, status)
    n = new_lens.numel()
    _check(lib.sparstar_kv4_resize(cache._struct, _kv4_ints(cache, seqs, "seqs", n),
                                   _kv4_ints(cache, new_lens, "new_lens", n), n,
                                   _kv4_status(cache, status), _kv4_raw_stream(cache)),
           "sparstar_kv4_resize")


def sparstar_kv4_fork(cache: Kv4Cache, src, dst, lens=None, deep: bool = False, status=None,
                      stream=None):
    """Empty sequences dst take the tokens of src: shared pages, or (deep) copies."""
    if _kv4_elsewhere(cache, stream):
        with _Kv4There(cache, stream):
            return sparstar_kv4_fork(cache, src, dst, lens, deep, status)
    n = src.numel()
    _check(lib.sparstar_kv4_fork(cache._struct, _kv4_ints(cache, src, "src", n),
                                 _kv4_ints(cache, dst, "dst", n),
                                 _kv4_ints(cache, lens, "lens", n), n, int(bool(deep)),
                                 _kv4_status(cache, status), _kv4_raw_stream(cache)),
           "sparstar_kv4_fork")


def sparstar_kv4_compact(cache: Kv4Cache, n_live=None, stream=None):
    """Moves the live pages to the lowest places; returns their number (device),
    or -1 there when the copy of a page gave up: fill the cache anew."""
    if _kv4_elsewhere(cache, stream):
        with _Kv4There(cache, stream):
            return sparstar_kv4_compact(cache, n_live)
    if n_live is None:
        n_live = torch.empty(1, dtype=torch.int32, device=cache.device)
    _check(lib.sparstar_kv4_compact(cache._struct,
                                    _kv4_tensor(cache, n_live, "n_live", torch.int32, (1,)),
                                    _kv4_raw_stream(cache)), "sparstar_kv4_compact")
    return n_live


def sparstar_kv4_write(cache: Kv4Cache, k, v, seqs=None, starts=None, counts=None, status=None,
                       stream=None):
    """Stores k, v [n, Hkv, T, D] at positions starts (default: the last T)."""
    if _kv4_elsewhere(cache, stream):
        with _Kv4There(cache, stream):
            return sparstar_kv4_write(cache, k, v, seqs, starts, counts, status)
    if k.dim() != 4:
        raise ValueError("k must be [n, Hkv, T, D]")
    n, _, T, _ = k.shape
    shape = (n, cache.Hkv, T, cache.D)
    _check(lib.sparstar_kv4_write(cache._struct, _kv4_tensor(cache, k, "k", k.dtype, shape),
                                  _kv4_tensor(cache, v, "v", k.dtype, shape),
                                  _DTYPE.get(k.dtype, -1), n, T,
                                  _kv4_ints(cache, seqs, "seqs", n),
                                  _kv4_ints(cache, starts, "starts", n),
                                  _kv4_ints(cache, counts, "counts", n),
                                  _kv4_status(cache, status), _kv4_raw_stream(cache)),
           "sparstar_kv4_write")


def sparstar_kv4_read(cache: Kv4Cache, T: int, n: int = None, dtype=torch.bfloat16, seqs=None,
                      starts=None, counts=None, k=None, v=None, status=None, stream=None):
    """The values of T tokens of each of n sequences; returns (k, v)
    [n, Hkv, T, D].  Rows beyond counts are not written (buffers that the
    call allocates hold zeros there), nor are those of entries that are left
    out (status; undefined in such buffers where counts is not given).  n,
    unless given, follows from seqs, starts, counts, k or v, and is every
    sequence without them."""
    if _kv4_elsewhere(cache, stream):
        with _Kv4There(cache, stream):
            return sparstar_kv4_read(cache, T, n, dtype, seqs, starts, counts, k, v, status)
    if n is None:
        sizes = [t.shape[0] for t in (seqs, starts, counts, k, v) if t is not None]
        n = sizes[0] if sizes else cache.n_seqs
    shape = (n, cache.Hkv, T, cache.D)
    if k is not None or v is not None:
        dtype = (k if k is not None else v).dtype
    elif _DTYPE.get(dtype, -1) < 0:
        raise SparstarError(EDTYPE, "sparstar_kv4_read")
    else:
        new = torch.empty if counts is None else torch.zeros
        k, v = (new(shape, dtype=dtype, device=cache.device) for _ in range(2))
    kp = None if k is None else _kv4_tensor(cache, k, "k", dtype, shape)
    vp = None if v is None else _kv4_tensor(cache, v, "v", dtype, shape)
    _check(lib.sparstar_kv4_read(cache._struct, kp, vp, _DTYPE.get(dtype, -1), n, T,
                                 _kv4_ints(cache, seqs, "seqs", n),
                                 _kv4_ints(cache, starts, "starts", n),
                                 _kv4_ints(cache, counts, "counts", n),
                                 _kv4_status(cache, status), _kv4_raw_stream(cache)),
           "sparstar_kv4_read")
    return k, v


def sparstar_kv4_attn_work_bytes(n: int, Hq: int, Hkv: int, Lq: int, D: int, max_pages: int,
                                 dtype=torch.bfloat16, max_sel: int = -1) -> int:
    """Bytes of scratch; max_sel: row stride of the block lists, -1 without."""
    return lib.sparstar_kv4_attn_work_bytes(n, Hq, Hkv, Lq, D, _DTYPE.get(dtype, -1), max_pages,
                                            max_sel)


def sparstar_kv4_attn(cache: Kv4Cache, q, seqs=None, tau: float = None, causal: bool = False,
                      kv_idx=None, kv_cnt=None, out=None, lse=None, want_lse: bool = True,
                      work=None, status=None, stream=None):
    """Attention of q [n, Hq, Lq, D] over the cached tokens of n sequences;
    returns (out, lse).  ``work`` (uint8, its first KV4_WORK_ZEROS bytes zero
    before its first use): when not given, the cache keeps one a stream (see
    ``drop_work``), and a call that is captured into a graph gets one of its
    own."""
    if _kv4_elsewhere(cache, stream):
        with _Kv4There(cache, stream):
            return sparstar_kv4_attn(cache, q, seqs, tau, causal, kv_idx, kv_cnt, out, lse,
                                     want_lse, work, status)
    if q.dim() != 4:
        raise ValueError("q must be [n, Hq, Lq, D]")
    shape = q.shape
    n, Hq, Lq, D = shape
    dtype = q.dtype
    dt = _DTYPE.get(dtype, -1)
    if D != cache.D:
        raise ValueError("q has head dim %d, the cache %d" % (D, cache.D))
    if tau is None:
        tau = _TAU[D]
    qp = _kv4_tensor(cache, q, "q", dtype, shape)
    if (kv_idx is None) != (kv_cnt is None):
        raise ValueError("kv_idx and kv_cnt go together")
    max_sel, ip, cp = -1, None, None
    if kv_idx is not None:
        rows = (n, Hq, nblocks(Lq))
        max_sel = kv_idx.shape[-1]
        ip = _kv4_tensor(cache, kv_idx, "kv_idx", torch.int32, rows + (max_sel,))
        cp = _kv4_tensor(cache, kv_cnt, "kv_cnt", torch.int32, rows)
    key = (n, Hq, Lq, dt, max_sel)
    need = cache._need.get(key)
    if need is None:
        need = lib.sparstar_kv4_attn_work_bytes(n, Hq, cache.Hkv, Lq, D, dt, cache.max_pages,
                                                max_sel)
        if need < 0:
            raise SparstarError(EDTYPE if dt < 0 else EINVAL, "sparstar_kv4_attn")
        # Making a tensor like another one costs half of making it from sizes.
        need = need, cache.lens[:1].view(torch.float32).expand(shape[:3])
        if len(cache._need) < 4096:
            cache._need[key] = need
    s = _kv4_raw_stream(cache)
    if out is None:
        out = torch.empty_like(q)
        op = out.data_ptr()
    else:
        op = _kv4_tensor(cache, out, "out", dtype, shape)
    if lse is not None:
        lp = _kv4_tensor(cache, lse, "lse", torch.float32, shape[:3])
    elif want_lse:
        lse = torch.empty_like(need[1], memory_format=torch.contiguous_format)
        lp = lse.data_ptr()
    else:
        lp = None
    if work is None:
        work = cache._attn_work(need[0], s)
    elif work.dtype is not torch.uint8 or work.get_device() != cache.index \
            or not work.is_contiguous():
        raise ValueError("work must be contiguous uint8 on %s" % cache.device)
    _check(lib.sparstar_kv4_attn(
        cache._struct, qp, dt, n, Hq, Lq,
        None if seqs is None else _kv4_ints(cache, seqs, "seqs", n), tau, 1 if causal else 0, ip,
        cp, max_sel if max_sel > 0 else 0, op, lp, work.data_ptr(), work.numel(),
        None if status is None else _kv4_status(cache, status), s), "sparstar_kv4_attn")
    return out, lse


def sparstar_test_attn_timeout(q, k, v, kv_idx, kv_cnt, out, status, stream=None):
    """Test hook: the attention kernel with its K/V copies withheld, so that
    its first ring wait runs out and SPARSTAR_STATUS_TIMEOUT is set in
    `status` (an int32 device tensor)."""
    for t, n in ((q, "q"), (k, "k"), (v, "v"), (out, "out")):
        _dev(t, n)
    _dev(kv_idx, "kv_idx", torch.int32)
    _dev(kv_cnt, "kv_cnt", torch.int32)
    _dev(status, "status", torch.int32)
    B, H, Lq, D = q.shape
    _check(lib.sparstar_test_attn_timeout(_ptr(q), _ptr(k), _ptr(v), B, H, Lq, k.shape[2],
                                          _ptr(kv_idx), _ptr(kv_cnt), kv_idx.shape[-1],
                                          _ptr(out), _ptr(status), _stream(stream)),
           "sparstar_test_attn_timeout")


def sparstar_test_kv4_compact_timeout(cache: Kv4Cache, n_live):
    """Test hook: a compaction with its copies withheld, so that they give up
    and n_live (an int32 device tensor) becomes -1."""
    _check(lib.sparstar_test_kv4_compact_timeout(
        cache._struct, _kv4_tensor(cache, n_live, "n_live", torch.int32, (1,)),
        _kv4_raw_stream(cache)), "sparstar_test_kv4_compact_timeout")


def sparstar_test_kv4_attn_timeout(cache: Kv4Cache, q, out, work, status):
    """Test hook: attention of sequences 0..n-1 with its copies withheld, so
    that its waits give up and STATUS_TIMEOUT is set in `status`.  ``work`` is
    not to be used again."""
    n, Hq, Lq, D = q.shape
    _check(lib.sparstar_test_kv4_attn_timeout(
        cache._struct, _kv4_tensor(cache, q, "q", q.dtype, q.shape), _DTYPE.get(q.dtype, -1), n,
        Hq, Lq, _TAU[D], _kv4_tensor(cache, out, "out", q.dtype, q.shape), work.data_ptr(),
        work.numel(), _kv4_status(cache, status), _kv4_raw_stream(cache)),
        "sparstar_test_kv4_attn_timeout")
