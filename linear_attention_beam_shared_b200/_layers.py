"""Binding of the operators around a GDN layer in ``include/onela.h``: paged
attention, cache write and eviction, block norms.

As in ``_lib``: argument checks and marshalling only.  A decode loop calls
these once per layer and step, so the sizes of a call (its configuration
struct and scratch size, plain numbers) are remembered by their values.
Nothing else is kept between calls.

They take no part in autograd: their outputs carry no gradient.

``stream``: None for the current stream of the tensors' device, a
``torch.cuda.Stream`` or a raw stream number.  What a call allocates (outputs
not given, scratch) is allocated on that stream.
"""
from __future__ import annotations

import ctypes
import math

import torch

from ._lib import ONELA_KERNEL_AUTO, ONELA_KERNEL_SIMT, _check, lib

ONELA_STATUS_PAGE, ONELA_STATUS_LENGTH, ONELA_STATUS_TIMEOUT = 1, 2, 4
ONELA_ACT_NONE, ONELA_ACT_SIGMOID, ONELA_ACT_SILU = 0, 1, 2

_i32, _i64, _f32, _vp = ctypes.c_int32, ctypes.c_int64, ctypes.c_float, ctypes.c_void_p


class onela_attention_config(ctypes.Structure):
    _fields_ = [(n, _i32) for n in (
        "R", "W", "H_q", "H_kv", "d", "dtype", "kernel", "page", "pages", "row_pages", "beam_page", "beam_pages",
        "beam_row_pages", "device")] + [("q_stride", _i64), ("scale", _f32)]


class onela_cache_write_config(ctypes.Structure):
    _fields_ = [(n, _i32) for n in ("B", "n", "H_kv", "d", "dtype", "page", "pages", "row_pages", "device")] + [
        ("k_stride", _i64), ("v_stride", _i64)]


class onela_cache_evict_config(ctypes.Structure):
    _fields_ = [(n, _i32) for n in (
        "R", "H_kv", "d", "dtype", "page", "pages", "row_pages", "dst_pages", "dst_row_pages", "keep", "recent",
        "device")]


class onela_block_norm_config(ctypes.Structure):
    _fields_ = [("N", _i64), ("y_stride", _i64), ("gate_stride", _i64), ("x_stride", _i64)] + [
        (n, _i32) for n in ("D", "group", "y_dtype", "dtype", "act", "device")] + [("alpha", _f32), ("eps", _f32)]


def _declare() -> None:
    sig = {
        "onela_paged_attention_scratch_bytes": ([_vp, _i32], ctypes.c_size_t),
        "onela_paged_attention": ([_vp] * 15 + [ctypes.c_size_t, _vp, _vp], ctypes.c_int),
        "onela_set_attention_wait_policy": ([ctypes.c_uint64, _i32], ctypes.c_int),
        "onela_cache_write": ([_vp] * 10, ctypes.c_int),
        "onela_cache_evict_scratch_bytes": ([_vp], ctypes.c_size_t),
        "onela_cache_evict": ([_vp] * 13 + [ctypes.c_size_t, _vp, _vp], ctypes.c_int),
        "onela_block_norm": ([_vp] * 10, ctypes.c_int),
    }
    for name, (args, res) in sig.items():
        fn = getattr(lib, name)
        fn.argtypes, fn.restype = args, res


_declare()
_attention, _attention_scratch = lib.onela_paged_attention, lib.onela_paged_attention_scratch_bytes
_write, _evict, _evict_scratch = lib.onela_cache_write, lib.onela_cache_evict, lib.onela_cache_evict_scratch_bytes
_norm = lib.onela_block_norm
_current_stream = torch._C._cuda_getCurrentRawStream

_CODE = {torch.float32: 0, torch.bfloat16: 1}
_CODE_OF = {**_CODE, "f32": 0, "bf16": 1}
_ACT = {"none": ONELA_ACT_NONE, "sigmoid": ONELA_ACT_SIGMOID, "silu": ONELA_ACT_SILU}
_TORCH = {0: torch.float32, 1: torch.bfloat16}
_I32, _F32 = torch.int32, torch.float32


def _arg(t, name, dtype, shape, index):
    """The pointer of a dense tensor on device `index` after its checks."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype is not dtype or t.shape != shape or t.get_device() != index or not t.is_contiguous():
        if t.get_device() != index:
            raise ValueError(f"{name} is on {t.device}, expected cuda:{index}")
        if t.dtype != dtype:
            raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
        if t.shape != shape:
            raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _floats(t, name, dim):
    """dtype code, device index and shape of a leading argument, a CUDA fp32 or
    bf16 tensor of `dim` dimensions."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    code = _CODE.get(t.dtype)
    if code is None:
        raise ValueError(f"{name} must be float32 or bfloat16, got {t.dtype}")
    shape = t.shape
    if len(shape) != dim:
        raise ValueError(f"{name} must have {dim} dimensions, got {len(shape)}")
    return code, t.get_device(), shape


def _pool(t, name, H, d):
    """Shape of a pool [pages][H_kv][page][d] that goes with H and d (None: any)."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    shape = t.shape
    if len(shape) != 4 or (H is not None and shape[1] != H) or shape[3] != d:
        raise ValueError(f"{name} must be [pages][H_kv][page][d] with matching H_kv and d, got {tuple(shape)}")
    return shape


def _last(t, name, dim):
    """Entries of a table's rows."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    shape = t.shape
    if len(shape) != dim:
        raise ValueError(f"{name} must have {dim} dimensions, got {len(shape)}")
    return shape[dim - 1]


def _token_stride(t, name, shape):
    """Elements between tokens of [A][B][H][d]: heads dense, tokens evenly spaced."""
    A, B, H, d = shape
    if t.is_contiguous():
        if A * B * H * d == 0:
            raise ValueError(f"{name} must not be empty")
        return H * d
    s = t.stride()
    if (d > 1 and s[3] != 1) or (H > 1 and s[2] != d):
        raise ValueError(f"{name} must be dense within a token")
    step = s[1] if B > 1 else (s[0] if A > 1 else H * d)
    if step < H * d or (A > 1 and B > 1 and s[0] != B * step):
        raise ValueError(f"{name} must have evenly spaced tokens")
    return step


def _row_stride(t, name, N, D):
    if t.is_contiguous():
        return D
    step = t.stride(0) if N > 1 else D
    if step < D or (D > 1 and t.stride(1) != 1):
        raise ValueError(f"{name} must be dense within a row, rows not overlapping")
    return step


def _raw_stream(stream, index):
    if stream is None:
        return _current_stream(index)
    return stream.cuda_stream if isinstance(stream, torch.cuda.Stream) else int(stream)


def _empty(shape, dtype, index, stream, like=None):
    """A new tensor that belongs to the call's stream.  like: a dense tensor of
    the same shape and type, if there is one (the quicker allocation)."""
    if stream is None:
        if like is not None:
            return torch.empty_like(like)
        return torch.empty(shape, dtype=dtype, device=torch.device("cuda", index))
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(int(stream), device=index) if stream else torch.cuda.default_stream(index)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=torch.device("cuda", index))


def _filled(struct, sizes):
    """The struct with these fields; ctypes would cut what does not fit one."""
    c = struct(*sizes)
    for (name, kind), x in zip(struct._fields_, sizes):
        if kind is not _f32 and getattr(c, name) != x:
            raise ValueError(f"{name} = {x} is out of range")
    return c


_sizes = {}


def _config(key, struct, sizes, scratch):
    """(struct, its address, scratch bytes) of a call's sizes."""
    hit = _sizes.get(key)
    if hit is None:
        if len(_sizes) >= 1024:
            _sizes.clear()
        c = _filled(struct, sizes)
        at = ctypes.addressof(c)
        hit = _sizes[key] = (c, at, scratch(at) if scratch else 0)
    return hit


def onela_paged_attention(q, k_pool, v_pool, table, lengths, beam=None, scale=None, mass=None, mass_out=None,
                          out=None, lse=None, scratch=None, status=None, kernel=ONELA_KERNEL_AUTO, stream=None):
    """Attention of new tokens over a paged cache (see onela.h).

    q [R][W][H_q][d] (its tokens may be spaced apart, as in a slice of a wider
    projection); k_pool, v_pool [pages][H_kv][page][d]; table int32
    [R][row_pages]; lengths int32 [R].  beam = (k_pool, v_pool, table int32
    [R][W][row_pages], lengths int32 [R][W]): the beams' own tokens.  mass (in)
    and mass_out fp32 [R][H_kv][row_pages * page]; lse fp32 [R][W][H_q].
    Returns o [R][W][H_q][d]."""
    code, dev, (R, W, H_q, d) = _floats(q, "q", 4)
    dt = q.dtype
    stride = _token_stride(q, "q", (R, W, H_q, d))
    pool = _pool(k_pool, "k_pool", None, d)
    pages, H_kv, page, _ = pool
    if H_kv < 1 or H_q % H_kv:
        raise ValueError(f"q's {H_q} heads are no multiple of the cache's {H_kv}")
    row_pages = _last(table, "table", 2)
    pk = _arg(k_pool, "k_pool", dt, pool, dev)
    pv = _arg(v_pool, "v_pool", dt, pool, dev)
    pt = _arg(table, "table", _I32, (R, row_pages), dev)
    pl = _arg(lengths, "lengths", _I32, (R,), dev)
    bk = bv = bt = bl = None
    bpage = bpages = brow = 0
    if beam is not None:
        tk, tv, tt, tl = beam
        bpool = _pool(tk, "beam k_pool", H_kv, d)
        bpages, _, bpage, _ = bpool
        brow = _last(tt, "beam table", 3)
        bk = _arg(tk, "beam k_pool", dt, bpool, dev)
        bv = _arg(tv, "beam v_pool", dt, bpool, dev)
        bt = _arg(tt, "beam table", _I32, (R, W, brow), dev)
        bl = _arg(tl, "beam lengths", _I32, (R, W), dev)
        if brow < 1 or bpages < 1 or bpage < 1:
            raise ValueError("the beams' pool and table must not be empty")
    pm = pmo = None
    if mass_out is not None:
        cells = (R, H_kv, row_pages * page)
        pm = None if mass is None else _arg(mass, "mass", _F32, cells, dev)
        pmo = _arg(mass_out, "mass_out", _F32, cells, dev)
    elif mass is not None:
        raise ValueError("mass needs mass_out")
    pq = q.data_ptr()
    if out is None:
        o = _empty((R, W, H_q, d), dt, dev, stream, q if stride == H_q * d and q.is_contiguous() else None)
        po = o.data_ptr()
    else:
        o, po = out, _arg(out, "out", dt, (R, W, H_q, d), dev)
    if kernel == ONELA_KERNEL_AUTO and ((pq | pk | pv) & 15 or po & 3):
        kernel = ONELA_KERNEL_SIMT  # what the call would take, and the scratch that goes with it
    scale = 1.0 / math.sqrt(d) if scale is None else float(scale)
    sizes = (R, W, H_q, H_kv, d, code, kernel, page, pages, row_pages, bpage, bpages, brow, dev, stride, scale)
    cfg, at, need = _config(("attention", pmo is None, sizes), onela_attention_config, sizes,
                            lambda a: _attention_scratch(a, pmo is not None))
    px, nbytes = None, 0
    if scratch is not None:
        px, nbytes = _arg(scratch, "scratch", torch.uint8, scratch.shape, dev), scratch.numel()
    elif need:
        scratch = _empty((need,), torch.uint8, dev, stream)
        px, nbytes = scratch.data_ptr(), need
    rc = _attention(at, pq, pk, pv, pt, pl, bk, bv, bt, bl, pm, pmo, po,
                    None if lse is None else _arg(lse, "lse", _F32, (R, W, H_q), dev), px, nbytes,
                    None if status is None else _arg(status, "status", _I32, (1,), dev), _raw_stream(stream, dev))
    if rc:
        _check(rc, "onela_paged_attention")
    return o


def onela_paged_attention_scratch_bytes(R, W, H_q, H_kv, d, dtype, page, pages, row_pages, beam_page=0, beam_pages=0,
                                        beam_row_pages=0, want_mass=False, kernel=ONELA_KERNEL_AUTO, device=0,
                                        q_stride=None):
    """Bytes of scratch a call of these sizes needs (to keep one buffer for all
    of a decode's calls); 0 for sizes no call takes.  q_stride: elements between
    q's tokens (default: dense; of no account for a single one).  The kernels
    need different sizes: a bf16 call whose q_stride is no multiple of 8, whose q
    or pools start off a 16-byte boundary or whose o starts off a 4-byte one
    takes the general kernel.  The stride is looked at here; for such addresses
    ask with kernel=ONELA_KERNEL_SIMT, and for both with the larger of the two."""
    if q_stride is None or R * W == 1:  # a single token is dense
        q_stride = H_q * d
    c = _filled(onela_attention_config, (R, W, H_q, H_kv, d, _CODE_OF[dtype], kernel, page, pages, row_pages, beam_page,
                                         beam_pages, beam_row_pages, device, q_stride, 1.0))
    return _attention_scratch(ctypes.addressof(c), 1 if want_mass else 0)


def onela_set_attention_wait_policy(limit_ns: int, stall: int = 0) -> None:
    """Bound of the waits inside the attention's tensor-core kernels, for the
    whole process (see onela.h); stall is a testing aid."""
    _check(lib.onela_set_attention_wait_policy(int(limit_ns), int(stall)), "onela_set_attention_wait_policy")


def onela_cache_write(k, v, k_pool, v_pool, table, start, counts=None, status=None, stream=None):
    """Write tokens to the cache (see onela.h): k, v [B][n][H_kv][d] (tokens may
    be spaced apart) to positions start[b] + i of table row b; pools
    [pages][H_kv][page][d]; table int32 [B][row_pages]; start, counts int32 [B]."""
    code, dev, (B, n, H_kv, d) = _floats(k, "k", 4)
    dt = k.dtype
    if not isinstance(v, torch.Tensor) or v.shape != (B, n, H_kv, d) or v.dtype is not dt or v.get_device() != dev:
        raise ValueError("v must match k")
    pool = _pool(k_pool, "k_pool", H_kv, d)
    row_pages = _last(table, "table", 2)
    sizes = (B, n, H_kv, d, code, pool[2], pool[0], row_pages, dev, _token_stride(k, "k", (B, n, H_kv, d)),
             _token_stride(v, "v", (B, n, H_kv, d)))
    cfg, at, _ = _config(("write", sizes), onela_cache_write_config, sizes, None)
    rc = _write(at, k.data_ptr(), v.data_ptr(), _arg(k_pool, "k_pool", dt, pool, dev),
                _arg(v_pool, "v_pool", dt, pool, dev), _arg(table, "table", _I32, (B, row_pages), dev),
                _arg(start, "start", _I32, (B,), dev),
                None if counts is None else _arg(counts, "counts", _I32, (B,), dev),
                None if status is None else _arg(status, "status", _I32, (1,), dev), _raw_stream(stream, dev))
    if rc:
        _check(rc, "onela_cache_write")


def onela_cache_evict(k_pool, v_pool, table, lengths, mass, keep, recent, dst_k, dst_v, dst_table, dst_lengths,
                      dst_mass, kept=None, scratch=None, status=None, stream=None):
    """Keep, per (request, key-value head), the last `recent` positions and the
    heaviest others, `keep` in all, copied in order to the pages of dst_table
    (see onela.h).  mass fp32 [R][H_kv][row_pages * page]; dst_mass fp32
    [R][H_kv][dst_row_pages * page]; kept int32 [R][H_kv][keep] or None."""
    code, dev, pool = _floats(k_pool, "k_pool", 4)
    dt = k_pool.dtype
    pages, H_kv, page, d = pool
    to = _pool(dst_k, "dst_k", H_kv, d)
    if to[2] != page:
        raise ValueError("dst_k must have pages of k_pool's size")
    row_pages, dst_row = _last(table, "table", 2), _last(dst_table, "dst_table", 2)
    R = table.shape[0]
    keep, recent = int(keep), int(recent)
    sizes = (R, H_kv, d, code, page, pages, row_pages, to[0], dst_row, keep, recent, dev)
    cfg, at, need = _config(("evict", sizes), onela_cache_evict_config, sizes, _evict_scratch)
    pkept = None if kept is None else _arg(kept, "kept", _I32, (R, H_kv, keep), dev)
    px, nbytes = None, 0
    if scratch is not None:
        px, nbytes = _arg(scratch, "scratch", torch.uint8, scratch.shape, dev), scratch.numel()
    elif pkept is None and need:
        scratch = _empty((need,), torch.uint8, dev, stream)
        px, nbytes = scratch.data_ptr(), need
    rc = _evict(
        at, _arg(k_pool, "k_pool", dt, pool, dev), _arg(v_pool, "v_pool", dt, pool, dev),
        _arg(table, "table", _I32, (R, row_pages), dev), _arg(lengths, "lengths", _I32, (R,), dev),
        _arg(mass, "mass", _F32, (R, H_kv, row_pages * page), dev), _arg(dst_k, "dst_k", dt, to, dev),
        _arg(dst_v, "dst_v", dt, to, dev), _arg(dst_table, "dst_table", _I32, (R, dst_row), dev),
        _arg(dst_lengths, "dst_lengths", _I32, (R,), dev),
        _arg(dst_mass, "dst_mass", _F32, (R, H_kv, dst_row * page), dev), pkept, px, nbytes,
        None if status is None else _arg(status, "status", _I32, (1,), dev), _raw_stream(stream, dev))
    if rc:
        _check(rc, "onela_cache_evict")


def onela_block_norm(y=None, x=None, gate=None, gate_act="none", w_post=None, scale=None, alpha=1.0, w_pre=None,
                     eps=1e-6, dtype=None, x_out=None, n_out=None, want_x=True, stream=None):
    """The norms around a block with its gate and residual scale (see onela.h).

    y [N][D] (fp32 or bf16), gate and x [N][D] in `dtype` (default: theirs, or
    y's); w_post fp32 [group], scale and w_pre fp32 [D].  gate_act "none",
    "sigmoid" or "silu".  Returns (x_out, n_out): x' (None with want_x=False)
    and, with w_pre, its norm (else None)."""
    lead = y if y is not None else x
    if lead is None:
        raise ValueError("give y, x or both")
    ycode, dev, (N, D) = _floats(lead, "y" if y is not None else "x", 2)
    if dtype is None:
        dtype = x.dtype if x is not None else gate.dtype if gate is not None else lead.dtype
    code = _CODE_OF.get(dtype)
    if code is None:
        raise ValueError("dtype must be f32 or bf16")
    dt = _TORCH[code]
    act = _ACT.get(gate_act)
    if act is None:
        raise ValueError(f"gate_act must be one of {sorted(_ACT)}")
    if (gate is None) != (act == ONELA_ACT_NONE):
        raise ValueError("gate and gate_act go together")
    py = pg = px = None
    sy = sg = sx = D
    like = None  # a dense tensor of the outputs' shape and type
    if y is not None:
        py, sy = y.data_ptr(), _row_stride(y, "y", N, D)
        if ycode == code and y.is_contiguous():
            like = y
    if gate is not None:
        pg, sg = _plane(gate, "gate", dt, N, D, dev), _row_stride(gate, "gate", N, D)
        if gate.is_contiguous():
            like = gate
    if x is not None:
        px, sx = _plane(x, "x", dt, N, D, dev), _row_stride(x, "x", N, D)
        if x.is_contiguous():
            like = x
    group, pw = D, None
    if w_post is not None:
        group = _last(w_post, "w_post", 1)
        if group < 1 or D % group:
            raise ValueError("w_post must be a vector whose length divides D")
        pw = _arg(w_post, "w_post", _F32, (group,), dev)
    sizes = (N, sy, sg, sx, D, group, ycode if y is not None else code, code, act, dev, float(alpha), float(eps))
    cfg, at, _ = _config(("norm", sizes), onela_block_norm_config, sizes, None)
    pxo = pno = None
    if x_out is not None:
        pxo = _arg(x_out, "x_out", dt, (N, D), dev)
    elif want_x:
        x_out = _empty((N, D), dt, dev, stream, like)
        pxo = x_out.data_ptr()
    if n_out is not None:
        pno = _arg(n_out, "n_out", dt, (N, D), dev)
    elif w_pre is not None:
        n_out = _empty((N, D), dt, dev, stream, like)
        pno = n_out.data_ptr()
    rc = _norm(at, py, pg, px, pw, None if scale is None else _arg(scale, "scale", _F32, (D,), dev),
               None if w_pre is None else _arg(w_pre, "w_pre", _F32, (D,), dev), pxo, pno, _raw_stream(stream, dev))
    if rc:
        _check(rc, "onela_block_norm")
    return x_out, n_out


def _plane(t, name, dt, N, D, index):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.get_device() != index or t.dtype is not dt or t.shape != (N, D):
        raise ValueError(f"{name} must be {dt} {(N, D)} on cuda:{index}")
    return t.data_ptr()
