"""ctypes marshalling of the history-cache entry points (see ``include/rocs_ikbo.h`` for the contract)."""
from __future__ import annotations

import ctypes
from typing import NamedTuple

import torch

from . import _binding as _b
from ._binding import NORMS, ROCS_BF16, ROCS_F32, RocsError, _check, _f32, _i32, _i64, _offsets, _on_tensor_device, _stream, _sz, _vp, _workspace

_DTYPES = {torch.float32: ROCS_F32, torch.bfloat16: ROCS_BF16}


class NormRopeSide(ctypes.Structure):
    _fields_ = [("x", _vp), ("out", _vp), ("pos", _vp), ("gamma", _vp), ("beta", _vp), ("n", _i64), ("heads", _i64),
                ("ld_x", _i64), ("ld_out", _i64)]


class NormRopeArgs(ctypes.Structure):
    _fields_ = [("q", NormRopeSide), ("k", NormRopeSide), ("dh", _i64), ("dtype", _i32), ("norm", _i32), ("eps", _f32),
                ("rope", _vp), ("max_pos", _i64), ("rot", _i64), ("interleaved", _i32), ("workspace", _vp),
                ("workspace_bytes", _sz)]


class CacheQ4Args(ctypes.Structure):
    _fields_ = [("k_codes", _vp), ("v_codes", _vp), ("k_scale", _vp), ("v_scale", _vp), ("pages", _i64), ("page", _i64),
                ("heads", _i64), ("dh", _i64)]


class CacheMoveArgs(ctypes.Structure):
    _fields_ = [("cache", CacheQ4Args), ("R", _i64), ("max_pages", _i64), ("tok_off_dev", _vp), ("tok_off_host", _vp),
                ("base", _vp), ("page_table", _vp), ("k", _vp), ("v", _vp), ("k_ld", _i64), ("v_ld", _i64),
                ("dtype", _i32), ("rope", _vp), ("max_pos", _i64), ("rot", _i64), ("interleaved", _i32), ("pos", _vp),
                ("workspace", _vp), ("workspace_bytes", _sz)]


class DcaCacheArgs(ctypes.Structure):
    _fields_ = [("cache", CacheQ4Args), ("R", _i64), ("q", _i64), ("H", _i64), ("max_pages", _i64), ("scale", _f32),
                ("cand_off_dev", _vp), ("cand_off_host", _vp), ("seq_len", _vp), ("page_table", _vp), ("key_limit", _vp),
                ("q_ptr", _vp), ("q_ld", _i64), ("o_ptr", _vp), ("lse_ptr", _vp), ("workspace", _vp),
                ("workspace_bytes", _sz)]


_ready = None


def _lib():
    global _ready
    if _ready is None or _ready is not _b._lib:
        lib = _b.load_library()
        P = ctypes.POINTER
        for name, argt in [("rocs_qk_norm_rope_workspace_size", [P(NormRopeArgs)]),
                           ("rocs_cache_workspace_size", [P(CacheMoveArgs)]),
                           ("rocs_dca_cache_workspace_size", [P(DcaCacheArgs)])]:
            getattr(lib, name).restype = _sz
            getattr(lib, name).argtypes = argt
        for name, argt in [("rocs_qk_norm_rope_forward", [P(NormRopeArgs), _vp]),
                           ("rocs_rope_table", [_vp, _i64, _i64, ctypes.c_double, _vp]),
                           ("rocs_cache_append", [P(CacheMoveArgs), _vp]), ("rocs_cache_read", [P(CacheMoveArgs), _vp]),
                           ("rocs_dca_cache_forward", [P(DcaCacheArgs), _vp])]:
            getattr(lib, name).restype = ctypes.c_int
            getattr(lib, name).argtypes = argt
        _ready = lib
    return _ready


class CacheQ4(NamedTuple):
    """Paged 4-bit cache: codes ``[pages, heads, page, dh/2]`` uint8 and scale ``[pages, heads, page, 2]`` bf16 (step,
    minimum) of keys and of values.  Token ``j`` of request ``r`` is in page ``page_table[r, j // page]``."""
    k_codes: torch.Tensor
    v_codes: torch.Tensor
    k_scale: torch.Tensor
    v_scale: torch.Tensor

    @classmethod
    def empty(cls, pages, page, heads, dh, device="cuda"):
        def codes():
            return torch.empty((pages, heads, page, dh // 2), dtype=torch.uint8, device=device)

        def scale():
            return torch.empty((pages, heads, page, 2), dtype=torch.bfloat16, device=device)
        return cls(codes(), codes(), scale(), scale())


def _hold(stream, *tensors):
    """Tensors made on the current stream and used on another: their memory is not handed out again before that stream
    has passed this point."""
    if stream is not None:
        for t in tensors:
            if t is not None and t.is_cuda:
                t.record_stream(stream)


def _cuda(t, dtype, what, dev, dims=None, contiguous=True):
    if not (isinstance(t, torch.Tensor) and t.is_cuda and t.dtype == dtype and (dims is None or t.dim() == dims)):
        raise RocsError(1, f"{what} must be a {'' if dims is None else f'{dims}-dimensional '}CUDA tensor of {dtype}")
    if contiguous and not t.is_contiguous():
        raise RocsError(1, f"{what} must be contiguous")
    if t.device != dev:
        raise RocsError(1, f"{what} is on {t.device}, the call's tensors are on {dev}")
    return t.data_ptr()


def _rows(t, dtype, what, dev, heads=None, dh=None):
    """``t`` [n, heads, dh] whose tokens may lie apart: ``(pointer or None, row stride in elements)``."""
    _cuda(t, dtype, what, dev, 3, contiguous=False)
    if (heads is not None and t.shape[1] != heads) or (dh is not None and t.shape[2] != dh):
        raise RocsError(1, f"{what} has heads and channels {tuple(t.shape[1:])}, expected {(heads, dh)}")
    if t.numel() == 0:
        return None, 0
    if t.stride(2) != 1 or (t.shape[1] > 1 and t.stride(1) != t.shape[2]):
        raise RocsError(1, f"{what}: the heads of a token must be dense (only tokens may lie apart)")
    row = t.shape[1] * t.shape[2]
    ld = t.stride(0) if t.shape[0] > 1 else row
    if ld < row:
        raise RocsError(1, f"{what}: tokens overlap (stride {ld}, {row} values a token)")
    return t.data_ptr(), ld


def _rope(rope, dev):
    """(pointer, positions, rotated channels) of a rope table, or of none."""
    if rope is None:
        return None, 0, 0
    return _cuda(rope, torch.float32, "rope", dev, 2), rope.shape[0], rope.shape[1]


@_on_tensor_device
def _fill_rope(table, base, stream):
    _check(_lib().rocs_rope_table(table.data_ptr() if table.numel() else None, table.shape[0], table.shape[1], float(base),
                                  _stream(stream)), "rocs_rope_table")


def rocs_rope_table(max_pos, rot, base=10000.0, device="cuda", stream=None):
    """``[max_pos, rot]`` fp32: ``rot/2`` cosines, then ``rot/2`` sines of the angles ``p * base^(-2i/rot)`` of every
    position ``p`` (angles in 64 bits)."""
    if max_pos < 0 or rot <= 0:
        raise RocsError(1, "rocs_rope_table: max_pos >= 0 and rot > 0")
    table = torch.empty((int(max_pos), int(rot)), dtype=torch.float32, device=device)
    _fill_rope(table, base, stream)
    return table


def _side(x, out, pos, gamma, beta, rope, what, dev, dtype, dh):
    if x is None:
        return NormRopeSide(), None
    x_ptr, ld_x = _rows(x, dtype, what, dev, None, dh)
    if out is None:
        out = torch.empty(x.shape, dtype=dtype, device=dev)
    elif tuple(out.shape) != tuple(x.shape):
        raise RocsError(1, f"{what}_out has shape {tuple(out.shape)}, expected {tuple(x.shape)}")
    out_ptr, ld_out = _rows(out, dtype, what + "_out", dev)
    n = x.shape[0] if x.numel() else 0
    if rope is not None:
        if pos is None:
            raise RocsError(1, f"pos_{what} must be given with a rope table")
        if pos.dim() != 1 or pos.shape[0] != x.shape[0]:
            raise RocsError(1, f"pos_{what} must have one position for each token")
    for name, t in (("gamma", gamma), ("beta", beta)):
        if t is not None and tuple(t.shape) != (dh,):
            raise RocsError(1, f"{name}_{what} must have {dh} values")
    return NormRopeSide(x=x_ptr, out=out_ptr, pos=None if rope is None else _cuda(pos, torch.int32, "pos_" + what, dev),
                        gamma=None if gamma is None else _cuda(gamma, torch.float32, "gamma_" + what, dev),
                        beta=None if beta is None else _cuda(beta, torch.float32, "beta_" + what, dev),
                        n=n, heads=x.shape[1] if n else 0, ld_x=ld_x, ld_out=ld_out), out


@_on_tensor_device
def rocs_qk_norm_rope_forward(q, k=None, pos_q=None, pos_k=None, rope=None, norm="rmsnorm", gamma_q=None, gamma_k=None,
                              beta_q=None, beta_k=None, eps=1e-6, interleaved=False, q_out=None, k_out=None,
                              workspace=None, stream=None):
    """Per-head norm of ``q`` [nq, H, dh] and ``k`` [nk, Hk, dh] (bf16 or fp32; either may be None) and the rotation by
    the tokens' positions in one pass.  ``rope``: the table of :func:`rocs_rope_table`, or None for no rotation.
    ``norm``: "none", "layernorm" or "rmsnorm".  Tokens may lie apart (rows of a wider projection output); an output
    may be its own input.  Returns ``(q_out, k_out)``."""
    lib = _lib()
    x = q if q is not None else k
    if x is None:
        raise RocsError(1, "rocs_qk_norm_rope_forward: q or k must be given")
    if x.dtype not in _DTYPES or x.dim() != 3:
        raise RocsError(1, "q and k must be [tokens, heads, dh] of bf16 or fp32")
    dev, dtype, dh = x.device, x.dtype, x.shape[2]
    sq, q_out = _side(q, q_out, pos_q, gamma_q, beta_q, rope, "q", dev, dtype, dh)
    sk, k_out = _side(k, k_out, pos_k, gamma_k, beta_k, rope, "k", dev, dtype, dh)
    rp, max_pos, rot = _rope(rope, dev)
    ws = _workspace(256, dev, workspace)
    a = NormRopeArgs(q=sq, k=sk, dh=dh, dtype=_DTYPES[dtype], norm=NORMS[norm] if isinstance(norm, str) else int(norm),
                     eps=float(eps), rope=rp, max_pos=max_pos, rot=rot, interleaved=int(bool(interleaved)),
                     workspace=ws.data_ptr(), workspace_bytes=ws.numel() * ws.element_size())
    _check(lib.rocs_qk_norm_rope_forward(ctypes.byref(a), _stream(stream)), "rocs_qk_norm_rope_forward")
    _hold(stream, ws, q_out, k_out)
    rocs_qk_norm_rope_forward.last_workspace = ws
    return q_out, k_out


def _cache(cache, dev):
    kc = cache.k_codes
    _cuda(kc, torch.uint8, "cache.k_codes", dev, 4)
    pages, heads, page, half = kc.shape
    for name, t, dtype, shape in (("v_codes", cache.v_codes, torch.uint8, (pages, heads, page, half)),
                                  ("k_scale", cache.k_scale, torch.bfloat16, (pages, heads, page, 2)),
                                  ("v_scale", cache.v_scale, torch.bfloat16, (pages, heads, page, 2))):
        _cuda(t, dtype, "cache." + name, dev)
        if tuple(t.shape) != shape:
            raise RocsError(1, f"cache.{name} has shape {tuple(t.shape)}, expected {shape}")
    return CacheQ4Args(k_codes=kc.data_ptr(), v_codes=cache.v_codes.data_ptr(), k_scale=cache.k_scale.data_ptr(),
                       v_scale=cache.v_scale.data_ptr(), pages=pages, page=page, heads=heads, dh=2 * half)


def _table(page_table, R, dev):
    ptr = _cuda(page_table, torch.int32, "page_table", dev, 2)
    if page_table.shape[0] != R:
        raise RocsError(1, f"page_table has {page_table.shape[0]} rows for {R} requests")
    return ptr if page_table.numel() else None


def _per_request(t, R, what, dev):
    ptr = _cuda(t, torch.int32, what, dev, 1)
    if t.shape[0] != R:
        raise RocsError(1, f"{what} has {t.shape[0]} entries for {R} requests")
    return ptr if R else None


def _move(cache, k, v, tok_off, base, page_table, dtype, dev, workspace):
    off_d, off_h = _offsets(tok_off, dev)
    R, T = len(off_h) - 1, int(off_h[-1])
    _cuda(off_d, torch.int32, "tok_off", dev, 1)
    c = _cache(cache, dev)
    for t, n in ((k, "k"), (v, "v")):
        if t.shape[0] != T:
            raise RocsError(1, f"{n} has {t.shape[0]} tokens, tok_off counts {T}")
    k_ptr, k_ld = _rows(k, dtype, "k", dev, c.heads, c.dh)
    v_ptr, v_ld = _rows(v, dtype, "v", dev, c.heads, c.dh)
    ws = _workspace(256, dev, workspace)
    return CacheMoveArgs(cache=c, R=R, max_pages=page_table.shape[1], tok_off_dev=off_d.data_ptr(),
                         tok_off_host=off_h.ctypes.data, base=_per_request(base, R, "base", dev),
                         page_table=_table(page_table, R, dev), k=k_ptr, v=v_ptr, k_ld=k_ld, v_ld=v_ld,
                         dtype=_DTYPES[dtype], workspace=ws.data_ptr(),
                         workspace_bytes=ws.numel() * ws.element_size()), (off_d, off_h), ws


def rocs_cache_append(cache, k, v, tok_off, base, page_table, rope=None, pos=None, interleaved=False, workspace=None,
                      stream=None):
    """Append ``k``, ``v`` [T, heads, dh] (bf16 or fp32) to the histories of a :class:`CacheQ4`: token ``i`` of request
    ``r`` (row ``tok_off[r] + i``) goes to slot ``base[r] + i``, keys rotated by ``pos`` (default: the slot) on the way.
    ``base`` [R] int32 is not changed.  Returns ``cache``."""
    return _append(k, cache, v, tok_off, base, page_table, rope, pos, interleaved, workspace, stream)


@_on_tensor_device
def _append(k, cache, v, tok_off, base, page_table, rope, pos, interleaved, workspace, stream):
    lib = _lib()
    if k.dtype not in _DTYPES:
        raise RocsError(1, "k and v must be bf16 or fp32")
    dev = k.device
    a, keep, ws = _move(cache, k, v, tok_off, base, page_table, k.dtype, dev, workspace)
    a.rope, a.max_pos, a.rot = _rope(rope, dev)
    a.interleaved = int(bool(interleaved))
    if pos is not None:
        if pos.dim() != 1 or pos.shape[0] != k.shape[0]:
            raise RocsError(1, "pos must have one position for each token")
        a.pos = _cuda(pos, torch.int32, "pos", dev) if pos.numel() else None
    _check(lib.rocs_cache_append(ctypes.byref(a), _stream(stream)), "rocs_cache_append")
    _hold(stream, ws, keep[0])
    rocs_cache_append.last_workspace = ws
    return cache


def rocs_cache_read(cache, tok_off, base, page_table, k=None, v=None, workspace=None, stream=None):
    """Slots ``base[r] ... base[r] + tok_off[r+1] - tok_off[r] - 1`` of every request's history as bf16 values, dense:
    ``(k, v)`` [T, heads, dh], what :func:`rocs_dca_forward` reads."""
    return _read(cache.k_codes, cache, tok_off, base, page_table, k, v, workspace, stream)


@_on_tensor_device
def _read(k_codes, cache, tok_off, base, page_table, k, v, workspace, stream):
    lib = _lib()
    dev = k_codes.device
    off = _offsets(tok_off, dev)
    shape = (int(off[1][-1]), k_codes.shape[1], 2 * k_codes.shape[3])
    k = torch.empty(shape, dtype=torch.bfloat16, device=dev) if k is None else k
    v = torch.empty(shape, dtype=torch.bfloat16, device=dev) if v is None else v
    a, keep, ws = _move(cache, k, v, off, base, page_table, torch.bfloat16, dev, workspace)
    _check(lib.rocs_cache_read(ctypes.byref(a), _stream(stream)), "rocs_cache_read")
    _hold(stream, ws, keep[0], k, v)
    rocs_cache_read.last_workspace = ws
    return k, v


@_on_tensor_device
def rocs_dca_cache_forward(q_t, cache, page_table, seq_len, cand_off, q_tokens, scale, key_limit=None, o=None, lse=True,
                           workspace=None, stream=None):
    """IKBO-DCA over a :class:`CacheQ4`: ``q_t`` [C*q, H, dh] bf16 (tokens may lie apart, H a multiple of the cache's
    heads), ``seq_len`` [R] int32 keys of each history, ``key_limit`` [C] int32 (optional) keys that a candidate sees.
    Returns ``(o [C*q, H, dh], lse [C*q, H] or None)``."""
    lib = _lib()
    dev = q_t.device
    off_d, off_h = _offsets(cand_off, dev)
    R, C = len(off_h) - 1, int(off_h[-1])
    _cuda(off_d, torch.int32, "cand_off", dev, 1)
    c = _cache(cache, dev)
    q_ptr, q_ld = _rows(q_t, torch.bfloat16, "q", dev, None, c.dh)
    if q_t.shape[0] != C * q_tokens:
        raise RocsError(1, f"q has {q_t.shape[0]} tokens, cand_off counts {C} candidates of {q_tokens}")
    shape = tuple(q_t.shape)
    if o is None:
        o = torch.empty(shape, dtype=torch.bfloat16, device=dev)
    _cuda(o, torch.bfloat16, "o", dev)
    if lse is True:
        lse = torch.empty(shape[:2], dtype=torch.float32, device=dev)
    elif lse is False:
        lse = None
    for t, want, what in ((o, shape, "o"), (lse, shape[:2], "lse")):
        if t is not None and tuple(t.shape) != want:
            raise RocsError(1, f"{what} has shape {tuple(t.shape)}, expected {want}")
    if key_limit is not None and tuple(key_limit.shape) != (C,):
        raise RocsError(1, f"key_limit must have one entry for each of {C} candidates")
    a = DcaCacheArgs(cache=c, R=R, q=int(q_tokens), H=shape[1], max_pages=page_table.shape[1], scale=float(scale),
                     cand_off_dev=off_d.data_ptr(), cand_off_host=off_h.ctypes.data,
                     seq_len=_per_request(seq_len, R, "seq_len", dev), page_table=_table(page_table, R, dev),
                     key_limit=None if key_limit is None or C == 0 else _cuda(key_limit, torch.int32, "key_limit", dev),
                     q_ptr=q_ptr, q_ld=q_ld, o_ptr=o.data_ptr() if C else None,
                     lse_ptr=_cuda(lse, torch.float32, "lse", dev) if lse is not None and C else None)
    nbytes = lib.rocs_dca_cache_workspace_size(ctypes.byref(a))
    if nbytes == 0:
        _check(lib.rocs_dca_cache_forward(ctypes.byref(a), _stream(stream)), "rocs_dca_cache_forward")
    ws = _workspace(nbytes, dev, workspace)
    a.workspace, a.workspace_bytes = ws.data_ptr(), ws.numel() * ws.element_size()
    _check(lib.rocs_dca_cache_forward(ctypes.byref(a), _stream(stream)), "rocs_dca_cache_forward")
    _hold(stream, ws, off_d, o, lse)
    rocs_dca_cache_forward.last_workspace = ws
    return o, lse
