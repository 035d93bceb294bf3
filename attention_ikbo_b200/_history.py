"""ctypes marshalling of the history-cache entry points (see ``include/rocs_ikbo.h`` for the contract).

With ``stream`` a call runs there instead of on the current stream.  The tensors that it is given must be ready on that
stream (the caller orders the two); what it makes itself comes from that stream's memory and may be used on both.
"""
from __future__ import annotations

import ctypes
import struct
from typing import NamedTuple

import torch

from . import _binding as _b
from ._binding import NORMS, ROCS_BF16, ROCS_F32, RocsError, _f32, _i32, _i64, _offsets, _sz, _vp, _workspace

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


# The structures as packed bytes (native alignment): a call of a few microseconds on the device is not to wait for
# ctypes to fill fields one by one.
_SIDE = "PPPPPqqqq"
_CACHE = "PPPPqqqq"
_PACK_NORM = struct.Struct("@" + _SIDE + _SIDE + "qiifPqqiPN")
_PACK_MOVE = struct.Struct("@" + _CACHE + "qqPPPPPPqqiPqqiPPN")
_PACK_DCA = struct.Struct("@" + _CACHE + "qqqqfPPPPPPqPPPN")
_NO_SIDE = (0,) * 9

_ready = None


def _lib():
    global _ready
    if _ready is None or _ready is not _b._lib:
        lib = _b.load_library()
        # argument structures are passed by address: a byref() of a Structure or packed bytes
        for name in ("rocs_qk_norm_rope_workspace_size", "rocs_cache_workspace_size", "rocs_dca_cache_workspace_size"):
            getattr(lib, name).restype = _sz
            getattr(lib, name).argtypes = [_vp]
        for name, argt in [("rocs_qk_norm_rope_forward", [_vp, _vp]), ("rocs_rope_table", [_vp, _i64, _i64, ctypes.c_double, _vp]),
                           ("rocs_cache_append", [_vp, _vp]), ("rocs_cache_read", [_vp, _vp]),
                           ("rocs_dca_cache_forward", [_vp, _vp])]:
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
    """Tensors that the current stream and the call's may both use: their memory is not handed out again before both have
    passed this point."""
    if stream is not None:
        here = torch.cuda.current_stream(stream.device)
        for t in tensors:
            if t is not None and t.is_cuda:
                t.record_stream(stream)
                t.record_stream(here)


def _refuse(t, dtype, what, idx, dims, contiguous=True):
    if not (isinstance(t, torch.Tensor) and t.is_cuda and t.dtype == dtype and (dims is None or t.dim() == dims)):
        raise RocsError(1, f"{what} must be a {'' if dims is None else f'{dims}-dimensional '}CUDA tensor of {dtype}")
    if contiguous and not t.is_contiguous():
        raise RocsError(1, f"{what} must be contiguous")
    raise RocsError(1, f"{what} is on {t.device}, the call's tensors are on cuda:{idx}")


def _ptr(t, dtype, what, idx, dims):
    """Address of a contiguous tensor of device ``idx``."""
    if not isinstance(t, torch.Tensor) or t.get_device() != idx or t.dtype is not dtype or t.dim() != dims or not t.is_contiguous():
        _refuse(t, dtype, what, idx, dims)
    return t.data_ptr()


def _rows(t, dtype, what, idx, heads=None, dh=None):
    """``t`` [n, heads, dh] whose tokens may lie apart: ``(address or 0, row stride in elements)``."""
    if not isinstance(t, torch.Tensor) or t.get_device() != idx or t.dtype is not dtype or t.dim() != 3:
        _refuse(t, dtype, what, idx, 3, False)
    n, h, d = t.shape
    if (heads is not None and h != heads) or (dh is not None and d != dh):
        raise RocsError(1, f"{what} has heads and channels {(h, d)}, expected {(heads, dh)}")
    row = h * d
    if n * row == 0:
        return 0, 0
    if t.is_contiguous():
        return t.data_ptr(), row
    st = t.stride()
    if st[2] != 1 or (h > 1 and st[1] != d):
        raise RocsError(1, f"{what}: the heads of a token must be dense (only tokens may lie apart)")
    ld = st[0] if n > 1 else row
    if ld < row:
        raise RocsError(1, f"{what}: tokens overlap (stride {ld}, {row} values a token)")
    return t.data_ptr(), ld


def _rope(rope, idx):
    """(address, positions, rotated channels) of a rope table, or of none."""
    if rope is None:
        return 0, 0, 0
    return (_ptr(rope, torch.float32, "rope", idx, 2), *rope.shape)


def _csr(off, dev, idx, what):
    """(device tensor, host array, device address, host address, R, total) of CSR offsets."""
    d, h = _offsets(off, dev)
    R = len(h) - 1
    if R < 0 or h.dtype != "int32" or not h.flags.c_contiguous:
        raise RocsError(1, f"{what}: host offsets must be a dense int32 array of R + 1 entries")
    ptr = _ptr(d, torch.int32, what, idx, 1)
    if d.shape[0] != R + 1:
        raise RocsError(1, f"{what}: {d.shape[0]} offsets on the device, {R + 1} on the host")
    return d, h, ptr, h.__array_interface__["data"][0], R, int(h[R])


def _ws(nbytes, dev, idx, given, stream):
    if given is None:
        return _empty(stream, max(int(nbytes), 256), torch.uint8, dev)
    if given.get_device() != idx or not given.is_contiguous():
        raise RocsError(6, "workspace: a contiguous tensor on the call's device")
    return _workspace(nbytes, dev, given)


def _on(t, what, fn, args):
    """``fn(index of t's device, *args)`` with that device current."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise RocsError(1, f"{what} must be a CUDA tensor")
    idx = t.get_device()
    if idx == torch.cuda.current_device():
        return fn(idx, *args)
    with torch.cuda.device(idx):
        return fn(idx, *args)


def _empty(stream, shape, dtype, device):
    """Memory for a call on ``stream``: from that stream's pool, since the current stream may still use what its own pool
    hands out."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _run(fn, packed, stream, idx, what):
    rc = fn(packed, torch._C._cuda_getCurrentRawStream(idx) if stream is None else stream.cuda_stream)
    if rc != 0:
        raise RocsError(rc, what)


def _fill_rope(idx, table, base, stream):
    rc = _lib().rocs_rope_table(table.data_ptr() if table.numel() else None, table.shape[0], table.shape[1], float(base),
                                torch._C._cuda_getCurrentRawStream(idx) if stream is None else stream.cuda_stream)
    if rc != 0:
        raise RocsError(rc, "rocs_rope_table")


def rocs_rope_table(max_pos, rot, base=10000.0, device="cuda", stream=None):
    """``[max_pos, rot]`` fp32: ``rot/2`` cosines, then ``rot/2`` sines of the angles ``p * base^(-2i/rot)`` of every
    position ``p`` (angles in 64 bits)."""
    if max_pos < 0 or rot <= 0:
        raise RocsError(1, "rocs_rope_table: max_pos >= 0 and rot > 0")
    table = _empty(stream, (int(max_pos), int(rot)), torch.float32, device)
    _on(table, "device", _fill_rope, (table, base, stream))
    _hold(stream, table)
    return table


def _side(x, out, pos, gamma, beta, rope, what, idx, dtype, dh, stream):
    if x is None:
        return _NO_SIDE, None
    x_ptr, ld_x = _rows(x, dtype, what, idx, None, dh)
    if out is None:
        out = torch.empty_like(x) if stream is None and x.is_contiguous() else _empty(stream, x.shape, dtype, x.device)
    elif out.shape != x.shape:
        raise RocsError(1, f"{what}_out has shape {tuple(out.shape)}, expected {tuple(x.shape)}")
    out_ptr, ld_out = _rows(out, dtype, what + "_out", idx)
    n, heads, _ = x.shape
    p_ptr = g_ptr = b_ptr = 0
    if rope is not None:
        if pos is None:
            raise RocsError(1, f"pos_{what} must be given with a rope table")
        p_ptr = _ptr(pos, torch.int32, "pos_" + what, idx, 1)
        if pos.shape[0] != n:
            raise RocsError(1, f"pos_{what} must have one position for each token")
    if gamma is not None:
        g_ptr = _ptr(gamma, torch.float32, "gamma_" + what, idx, 1)
        if gamma.shape[0] != dh:
            raise RocsError(1, f"gamma_{what} must have {dh} values")
    if beta is not None:
        b_ptr = _ptr(beta, torch.float32, "beta_" + what, idx, 1)
        if beta.shape[0] != dh:
            raise RocsError(1, f"beta_{what} must have {dh} values")
    if x_ptr == 0:
        return _NO_SIDE, out
    return (x_ptr, out_ptr, p_ptr, g_ptr, b_ptr, n, heads, ld_x, ld_out), out


def rocs_qk_norm_rope_forward(q, k=None, pos_q=None, pos_k=None, rope=None, norm="rmsnorm", gamma_q=None, gamma_k=None,
                              beta_q=None, beta_k=None, eps=1e-6, interleaved=False, q_out=None, k_out=None,
                              workspace=None, stream=None):
    """Per-head norm of ``q`` [nq, H, dh] and ``k`` [nk, Hk, dh] (bf16 or fp32; either may be None) and the rotation by
    the tokens' positions in one pass.  ``rope``: the table of :func:`rocs_rope_table`, or None for no rotation.
    ``norm``: "none", "layernorm" or "rmsnorm".  Tokens may lie apart (rows of a wider projection output); an output
    may be its own input.  Returns ``(q_out, k_out)``."""
    x = q if q is not None else k
    if x is None:
        raise RocsError(1, "rocs_qk_norm_rope_forward: q or k must be given")
    return _on(x, "q" if q is not None else "k", _norm_rope,
               (x, q, k, pos_q, pos_k, rope, norm, gamma_q, gamma_k, beta_q, beta_k, eps, interleaved, q_out, k_out, workspace, stream))


def _norm_rope(idx, x, q, k, pos_q, pos_k, rope, norm, gamma_q, gamma_k, beta_q, beta_k, eps, interleaved, q_out, k_out, workspace,
               stream):
    dtype = x.dtype
    if dtype not in _DTYPES or x.dim() != 3:
        raise RocsError(1, "q and k must be [tokens, heads, dh] of bf16 or fp32")
    dh = x.shape[2]
    sq, q_out = _side(q, q_out, pos_q, gamma_q, beta_q, rope, "q", idx, dtype, dh, stream)
    sk, k_out = _side(k, k_out, pos_k, gamma_k, beta_k, rope, "k", idx, dtype, dh, stream)
    ws = _ws(256, x.device, idx, workspace, stream)
    _run(_lib().rocs_qk_norm_rope_forward,
         _PACK_NORM.pack(*sq, *sk, dh, _DTYPES[dtype], NORMS[norm] if isinstance(norm, str) else int(norm), eps, *_rope(rope, idx),
                         1 if interleaved else 0, ws.data_ptr(), ws.nbytes), stream, idx, "rocs_qk_norm_rope_forward")
    _hold(stream, ws, q_out, k_out)
    rocs_qk_norm_rope_forward.last_workspace = ws
    return q_out, k_out


def _cache(cache, idx):
    kc, vc, ks, vs = cache.k_codes, cache.v_codes, cache.k_scale, cache.v_scale
    ptrs = (_ptr(kc, torch.uint8, "cache.k_codes", idx, 4), _ptr(vc, torch.uint8, "cache.v_codes", idx, 4),
            _ptr(ks, torch.bfloat16, "cache.k_scale", idx, 4), _ptr(vs, torch.bfloat16, "cache.v_scale", idx, 4))
    pages, heads, page, half = kc.shape
    if vc.shape != kc.shape or ks.shape != vs.shape or ks.shape != (pages, heads, page, 2):
        raise RocsError(1, f"cache: codes {tuple(kc.shape)}, {tuple(vc.shape)}, scale {tuple(ks.shape)}, {tuple(vs.shape)} do not belong "
                           "together")
    return ptrs + (pages, page, heads, 2 * half)


def _table(page_table, R, idx):
    """(address, pages of a row)"""
    ptr = _ptr(page_table, torch.int32, "page_table", idx, 2)
    rows, cols = page_table.shape
    if rows != R:
        raise RocsError(1, f"page_table has {rows} rows for {R} requests")
    return ptr, cols


def _per_request(t, R, what, idx):
    ptr = _ptr(t, torch.int32, what, idx, 1)
    if t.shape[0] != R:
        raise RocsError(1, f"{what} has {t.shape[0]} entries for {R} requests")
    return ptr


def _move(fn, what, idx, c, csr, k, v, base, page_table, rope, pos, interleaved, dtype, ws, stream):
    _, _, off_d, off_h, R, T = csr
    k_ptr, k_ld = _rows(k, dtype, "k", idx, c[6], c[7])
    v_ptr, v_ld = _rows(v, dtype, "v", idx, c[6], c[7])
    if k.shape[0] != T or v.shape[0] != T:
        raise RocsError(1, f"k and v have {k.shape[0]} and {v.shape[0]} tokens, tok_off counts {T}")
    table, cols = _table(page_table, R, idx)
    p_ptr = 0
    if pos is not None:
        p_ptr = _ptr(pos, torch.int32, "pos", idx, 1)
        if pos.shape[0] != T:
            raise RocsError(1, "pos must have one position for each token")
    _run(fn, _PACK_MOVE.pack(*c, R, cols, off_d, off_h, _per_request(base, R, "base", idx), table, k_ptr, v_ptr, k_ld, v_ld,
                             _DTYPES[dtype], *_rope(rope, idx), 1 if interleaved else 0, p_ptr, ws.data_ptr(), ws.nbytes),
         stream, idx, what)


def rocs_cache_append(cache, k, v, tok_off, base, page_table, rope=None, pos=None, interleaved=False, workspace=None,
                      stream=None):
    """Append ``k``, ``v`` [T, heads, dh] (bf16 or fp32) to the histories of a :class:`CacheQ4`: token ``i`` of request
    ``r`` (row ``tok_off[r] + i``) goes to slot ``base[r] + i``, keys rotated by ``pos`` (default: the slot) on the way.
    ``base`` [R] int32 is not changed.  Tokens may lie apart: the halves of a stacked K/V projection
    (:func:`rocs_proj_forward` of a request's sequence) go in as they are.  Returns ``cache``."""
    return _on(k, "k", _append, (cache, k, v, tok_off, base, page_table, rope, pos, interleaved, workspace, stream))


def _append(idx, cache, k, v, tok_off, base, page_table, rope, pos, interleaved, workspace, stream):
    if k.dtype not in _DTYPES:
        raise RocsError(1, "k and v must be bf16 or fp32")
    csr = _csr(tok_off, k.device, idx, "tok_off")
    ws = _ws(256, k.device, idx, workspace, stream)
    _move(_lib().rocs_cache_append, "rocs_cache_append", idx, _cache(cache, idx), csr, k, v, base, page_table, rope, pos, interleaved,
          k.dtype, ws, stream)
    _hold(stream, ws, csr[0])
    rocs_cache_append.last_workspace = ws
    return cache


def rocs_cache_read(cache, tok_off, base, page_table, k=None, v=None, workspace=None, stream=None):
    """Slots ``base[r] ... base[r] + tok_off[r+1] - tok_off[r] - 1`` of every request's history as bf16 values, dense:
    ``(k, v)`` [T, heads, dh], what :func:`rocs_dca_forward` reads."""
    return _on(cache.k_codes, "cache.k_codes", _read, (cache, tok_off, base, page_table, k, v, workspace, stream))


def _read(idx, cache, tok_off, base, page_table, k, v, workspace, stream):
    dev = cache.k_codes.device
    csr = _csr(tok_off, dev, idx, "tok_off")
    c = _cache(cache, idx)
    if k is None:
        k = _empty(stream, (csr[5], c[6], c[7]), torch.bfloat16, dev)
    if v is None:
        v = torch.empty_like(k) if stream is None and k.is_contiguous() else _empty(stream, k.shape, torch.bfloat16, dev)
    ws = _ws(256, dev, idx, workspace, stream)
    _move(_lib().rocs_cache_read, "rocs_cache_read", idx, c, csr, k, v, base, page_table, None, None, False, torch.bfloat16, ws, stream)
    _hold(stream, ws, csr[0], k, v)
    rocs_cache_read.last_workspace = ws
    return k, v


def rocs_dca_cache_forward(q_t, cache, page_table, seq_len, cand_off, q_tokens, scale, key_limit=None, o=None, lse=True,
                           workspace=None, stream=None):
    """IKBO-DCA over a :class:`CacheQ4`: ``q_t`` [C*q, H, dh] bf16 (tokens may lie apart, H a multiple of the cache's
    heads), ``seq_len`` [R] int32 keys of each history, ``key_limit`` [C] int32 (optional) keys that a candidate sees.
    Returns ``(o [C*q, H, dh], lse [C*q, H] or None)``."""
    return _on(q_t, "q", _dca_cache, (q_t, cache, page_table, seq_len, cand_off, q_tokens, scale, key_limit, o, lse, workspace, stream))


def _dca_cache(idx, q_t, cache, page_table, seq_len, cand_off, q_tokens, scale, key_limit, o, lse, workspace, stream):
    lib = _lib()
    off_dev, _, off_d, off_h, R, C = _csr(cand_off, q_t.device, idx, "cand_off")
    c = _cache(cache, idx)
    q_ptr, q_ld = _rows(q_t, torch.bfloat16, "q", idx, None, c[7])
    n, H, dh = q_t.shape
    if n != C * q_tokens:
        raise RocsError(1, f"q has {n} tokens, cand_off counts {C} candidates of {q_tokens}")
    if o is None:
        o = torch.empty_like(q_t) if stream is None and q_t.is_contiguous() else _empty(stream, (n, H, dh), torch.bfloat16, q_t.device)
    elif o.shape != q_t.shape:
        raise RocsError(1, f"o has shape {tuple(o.shape)}, expected {(n, H, dh)}")
    if lse is True:
        lse = _empty(stream, (n, H), torch.float32, q_t.device)
    elif lse is False:
        lse = None
    lse_ptr = lim_ptr = 0
    if lse is not None:
        lse_ptr = _ptr(lse, torch.float32, "lse", idx, 2)
        if lse.shape != (n, H):
            raise RocsError(1, f"lse has shape {tuple(lse.shape)}, expected {(n, H)}")
    if key_limit is not None:
        lim_ptr = _ptr(key_limit, torch.int32, "key_limit", idx, 1)
        if key_limit.shape[0] != C:
            raise RocsError(1, f"key_limit must have one entry for each of {C} candidates")
    table, cols = _table(page_table, R, idx)
    a = (*c, R, int(q_tokens), H, cols, scale, off_d, off_h, _per_request(seq_len, R, "seq_len", idx), table, lim_ptr, q_ptr, q_ld,
         _ptr(o, torch.bfloat16, "o", idx, 3), lse_ptr)
    nbytes = lib.rocs_dca_cache_workspace_size(_PACK_DCA.pack(*a, 0, 0))
    ws = _ws(nbytes, q_t.device, idx, workspace, stream)  # 0: refused arguments, the call below says which
    _run(lib.rocs_dca_cache_forward, _PACK_DCA.pack(*a, ws.data_ptr(), ws.nbytes), stream, idx, "rocs_dca_cache_forward")
    _hold(stream, ws, off_dev, o, lse)
    rocs_dca_cache_forward.last_workspace = ws
    return o, lse
