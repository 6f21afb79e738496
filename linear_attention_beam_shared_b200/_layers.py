"""Binding of the operators around a GDN layer in ``include/onela.h``: paged
attention, cache write and eviction, block norms.

As in ``_lib``: argument checks and marshalling only.  A decode loop calls
these once per layer and step, so the sizes of a call (its configuration
struct and scratch size, plain numbers) are remembered by their values.
Nothing else is kept between calls.

``stream``: None for the current stream of the tensors' device, a
``torch.cuda.Stream`` or a raw stream number.  What a call allocates (outputs
not given, scratch) is allocated on that stream.
"""
from __future__ import annotations

import contextlib
import ctypes
import math

import torch

from ._lib import ONELA_KERNEL_AUTO, _check, lib

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
        "onela_cache_write": ([_vp] * 10, ctypes.c_int),
        "onela_cache_evict_scratch_bytes": ([_vp], ctypes.c_size_t),
        "onela_cache_evict": ([_vp] * 13 + [ctypes.c_size_t, _vp, _vp], ctypes.c_int),
        "onela_block_norm": ([_vp] * 10, ctypes.c_int),
    }
    for name, (args, res) in sig.items():
        fn = getattr(lib, name)
        fn.argtypes, fn.restype = args, res


_declare()

_CODE = {torch.float32: 0, torch.bfloat16: 1}
_CODE_OF = {**_CODE, "f32": 0, "bf16": 1}
_ACT = {"none": ONELA_ACT_NONE, "sigmoid": ONELA_ACT_SIGMOID, "silu": ONELA_ACT_SILU}
_TORCH = {0: torch.float32, 1: torch.bfloat16}


def _arg(t, name, dtype, shape, device, optional=False):
    """The pointer of a dense tensor after its checks (None: NULL)."""
    if t is None:
        if optional:
            return None
        raise TypeError(f"{name} must be a torch.Tensor")
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _floats(t, name, dim):
    """dtype code and device of a leading argument, a CUDA fp32 or bf16 tensor of `dim` dimensions."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    code = _CODE.get(t.dtype)
    if code is None:
        raise ValueError(f"{name} must be float32 or bfloat16, got {t.dtype}")
    if t.dim() != dim:
        raise ValueError(f"{name} must have {dim} dimensions, got {t.dim()}")
    return code, t.device


def _token_stride(t, name):
    """Elements between tokens of [A][B][H][d]: heads dense, tokens evenly spaced."""
    A, B, H, d = t.shape
    if t.numel() == 0:
        raise ValueError(f"{name} must not be empty")
    s = t.stride()
    if (d > 1 and s[3] != 1) or (H > 1 and s[2] != d):
        raise ValueError(f"{name} must be dense within a token")
    step = s[1] if B > 1 else (s[0] if A > 1 else H * d)
    if step < H * d or (A > 1 and B > 1 and s[0] != B * step):
        raise ValueError(f"{name} must have evenly spaced tokens")
    return step


def _row_stride(t, name):
    N, D = t.shape
    if D > 1 and t.stride(1) != 1:
        raise ValueError(f"{name} must be dense within a row")
    step = t.stride(0) if N > 1 else D
    if step < D:
        raise ValueError(f"{name} must not have overlapping rows")
    return step


def _raw_stream(stream, device):
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(device.index)
    return stream.cuda_stream if isinstance(stream, torch.cuda.Stream) else int(stream)


def _on(stream, device):
    """The context to allocate in, so that what is allocated belongs to the call's stream."""
    if stream is None:
        return contextlib.nullcontext()
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(int(stream), device=device)
    return torch.cuda.stream(stream)


def _empty(shape, dtype, device, stream):
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with _on(stream, device):
        return torch.empty(shape, dtype=dtype, device=device)


_sizes = {}


def _config(key, make, scratch):
    """(struct, its address, scratch bytes) of a call's sizes."""
    hit = _sizes.get(key)
    if hit is None:
        if len(_sizes) >= 1024:
            _sizes.clear()
        c = make()
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
    code, dev = _floats(q, "q", 4)
    dt = q.dtype
    R, W, H_q, d = q.shape
    stride = _token_stride(q, "q")
    if not isinstance(k_pool, torch.Tensor) or k_pool.dim() != 4:
        raise ValueError("k_pool must be a 4-D tensor [pages][H_kv][page][d]")
    pool = k_pool.shape
    pages, H_kv, page, _ = pool
    if pool[3] != d or H_kv < 1 or H_q % H_kv:
        raise ValueError(f"k_pool {tuple(pool)} does not fit q {tuple(q.shape)}")
    if not isinstance(table, torch.Tensor) or table.dim() != 2:
        raise ValueError("table must be a 2-D int32 tensor [R][row_pages]")
    row_pages = table.shape[1]
    pk = _arg(k_pool, "k_pool", dt, pool, dev)
    pv = _arg(v_pool, "v_pool", dt, pool, dev)
    pt = _arg(table, "table", torch.int32, (R, row_pages), dev)
    pl = _arg(lengths, "lengths", torch.int32, (R,), dev)
    bk = bv = bt = bl = None
    bpage = bpages = brow = 0
    if beam is not None:
        tk, tv, tt, tl = beam
        if not isinstance(tk, torch.Tensor) or tk.dim() != 4 or tk.shape[1] != H_kv or tk.shape[3] != d:
            raise ValueError("the beams' k_pool must be [pages][H_kv][page][d] with the prompt's H_kv and d")
        bpages, _, bpage, _ = tk.shape
        if not isinstance(tt, torch.Tensor) or tt.dim() != 3:
            raise ValueError("the beams' table must be a 3-D int32 tensor [R][W][row_pages]")
        brow = tt.shape[2]
        bk = _arg(tk, "beam k_pool", dt, tk.shape, dev)
        bv = _arg(tv, "beam v_pool", dt, tk.shape, dev)
        bt = _arg(tt, "beam table", torch.int32, (R, W, brow), dev)
        bl = _arg(tl, "beam lengths", torch.int32, (R, W), dev)
        if brow < 1 or bpages < 1 or bpage < 1:
            raise ValueError("the beams' pool and table must not be empty")
    if mass is not None and mass_out is None:
        raise ValueError("mass needs mass_out")
    pm = _arg(mass, "mass", torch.float32, (R, H_kv, row_pages * page), dev, True)
    pmo = _arg(mass_out, "mass_out", torch.float32, (R, H_kv, row_pages * page), dev, True)
    ps = _arg(lse, "lse", torch.float32, (R, W, H_q), dev, True)
    scale = 1.0 / math.sqrt(d) if scale is None else float(scale)
    sizes = (R, W, H_q, H_kv, d, code, kernel, page, pages, row_pages, bpage, bpages, brow, dev.index, stride, scale)
    want = pmo is not None
    cfg, at, need = _config(("attention", want, sizes), lambda: onela_attention_config(*sizes),
                            lambda a: lib.onela_paged_attention_scratch_bytes(a, want))
    o = _empty((R, W, H_q, d), dt, dev, stream) if out is None else out
    po = _arg(o, "out", dt, (R, W, H_q, d), dev)
    if scratch is None:
        scratch = _empty((max(need, 16),), torch.uint8, dev, stream)
    px = _arg(scratch, "scratch", torch.uint8, scratch.shape, dev)
    _check(lib.onela_paged_attention(at, q.data_ptr(), pk, pv, pt, pl, bk, bv, bt, bl, pm, pmo, po, ps, px,
                                     scratch.numel(), _arg(status, "status", torch.int32, (1,), dev, True),
                                     _raw_stream(stream, dev)), "onela_paged_attention")
    return o


def onela_paged_attention_scratch_bytes(R, W, H_q, H_kv, d, dtype, page, pages, row_pages, beam_page=0, beam_pages=0,
                                        beam_row_pages=0, want_mass=False, kernel=ONELA_KERNEL_AUTO, device=0):
    """Bytes of scratch a call of these sizes needs (to keep one buffer for all of a decode's calls)."""
    c = onela_attention_config(R, W, H_q, H_kv, d, _CODE_OF[dtype], kernel, page, pages, row_pages, beam_page,
                               beam_pages, beam_row_pages, device, H_q * d, 1.0)
    return lib.onela_paged_attention_scratch_bytes(ctypes.addressof(c), 1 if want_mass else 0)


def onela_cache_write(k, v, k_pool, v_pool, table, start, counts=None, status=None, stream=None):
    """Write tokens to the cache (see onela.h): k, v [B][n][H_kv][d] (tokens may
    be spaced apart) to positions start[b] + i of table row b; pools
    [pages][H_kv][page][d]; table int32 [B][row_pages]; start, counts int32 [B]."""
    code, dev = _floats(k, "k", 4)
    B, n, H_kv, d = k.shape
    if not isinstance(v, torch.Tensor) or v.shape != k.shape or v.dtype != k.dtype or v.device != dev:
        raise ValueError("v must match k")
    ks, vs = _token_stride(k, "k"), _token_stride(v, "v")
    if not isinstance(k_pool, torch.Tensor) or k_pool.dim() != 4 or k_pool.shape[1] != H_kv or k_pool.shape[3] != d:
        raise ValueError("k_pool must be [pages][H_kv][page][d] with k's H_kv and d")
    pool = k_pool.shape
    if not isinstance(table, torch.Tensor) or table.dim() != 2:
        raise ValueError("table must be a 2-D int32 tensor [B][row_pages]")
    row_pages = table.shape[1]
    sizes = (B, n, H_kv, d, code, pool[2], pool[0], row_pages, dev.index, ks, vs)
    cfg, at, _ = _config(("write", sizes), lambda: onela_cache_write_config(*sizes), None)
    _check(lib.onela_cache_write(
        at, k.data_ptr(), v.data_ptr(), _arg(k_pool, "k_pool", k.dtype, pool, dev),
        _arg(v_pool, "v_pool", k.dtype, pool, dev), _arg(table, "table", torch.int32, (B, row_pages), dev),
        _arg(start, "start", torch.int32, (B,), dev), _arg(counts, "counts", torch.int32, (B,), dev, True),
        _arg(status, "status", torch.int32, (1,), dev, True), _raw_stream(stream, dev)), "onela_cache_write")


def onela_cache_evict(k_pool, v_pool, table, lengths, mass, keep, recent, dst_k, dst_v, dst_table, dst_lengths,
                      dst_mass, kept=None, scratch=None, status=None, stream=None):
    """Keep, per (request, key-value head), the last `recent` positions and the
    heaviest others, `keep` in all, copied in order to the pages of dst_table
    (see onela.h).  mass fp32 [R][H_kv][row_pages * page]; dst_mass fp32
    [R][H_kv][dst_row_pages * page]; kept int32 [R][H_kv][keep] or None."""
    code, dev = _floats(k_pool, "k_pool", 4)
    pool = k_pool.shape
    pages, H_kv, page, d = pool
    if not isinstance(dst_k, torch.Tensor) or dst_k.dim() != 4 or dst_k.shape[1:] != pool[1:]:
        raise ValueError("dst_k must be a pool with k_pool's H_kv, page and d")
    for t, name in ((table, "table"), (dst_table, "dst_table")):
        if not isinstance(t, torch.Tensor) or t.dim() != 2:
            raise ValueError(f"{name} must be a 2-D int32 tensor [R][row_pages]")
    R, row_pages = table.shape
    dst_row = dst_table.shape[1]
    keep, recent = int(keep), int(recent)
    sizes = (R, H_kv, d, code, page, pages, row_pages, dst_k.shape[0], dst_row, keep, recent, dev.index)
    cfg, at, need = _config(("evict", sizes), lambda: onela_cache_evict_config(*sizes),
                            lib.onela_cache_evict_scratch_bytes)
    dt, i32, f32 = k_pool.dtype, torch.int32, torch.float32
    if scratch is None:
        scratch = _empty((max(need, 16),), torch.uint8, dev, stream)
    _check(lib.onela_cache_evict(
        at, _arg(k_pool, "k_pool", dt, pool, dev), _arg(v_pool, "v_pool", dt, pool, dev),
        _arg(table, "table", i32, (R, row_pages), dev), _arg(lengths, "lengths", i32, (R,), dev),
        _arg(mass, "mass", f32, (R, H_kv, row_pages * page), dev), _arg(dst_k, "dst_k", dt, dst_k.shape, dev),
        _arg(dst_v, "dst_v", dt, dst_k.shape, dev), _arg(dst_table, "dst_table", i32, (R, dst_row), dev),
        _arg(dst_lengths, "dst_lengths", i32, (R,), dev),
        _arg(dst_mass, "dst_mass", f32, (R, H_kv, dst_row * page), dev),
        _arg(kept, "kept", i32, (R, H_kv, keep), dev, True),
        _arg(scratch, "scratch", torch.uint8, scratch.shape, dev), scratch.numel(),
        _arg(status, "status", i32, (1,), dev, True), _raw_stream(stream, dev)), "onela_cache_evict")


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
    ycode, dev = _floats(lead, "y" if y is not None else "x", 2)
    N, D = lead.shape
    for t in (x, gate):
        if t is not None and dtype is None:
            dtype = t.dtype
    code = _CODE_OF.get(dtype if dtype is not None else lead.dtype)
    if code is None:
        raise ValueError("dtype must be f32 or bf16")
    dt = _TORCH[code]
    if gate_act not in _ACT:
        raise ValueError(f"gate_act must be one of {sorted(_ACT)}")
    act = _ACT[gate_act]
    if (gate is None) != (act == ONELA_ACT_NONE):
        raise ValueError("gate and gate_act go together")
    strides, ptrs = [], []
    for t, name, want in ((y, "y", None), (gate, "gate", dt), (x, "x", dt)):
        if t is None:
            strides.append(D)
            ptrs.append(None)
            continue
        if t.device != dev or t.shape != lead.shape or (want is not None and t.dtype != want):
            raise ValueError(f"{name} must be {want or 'float32 or bfloat16'} {tuple(lead.shape)} on {dev}")
        strides.append(_row_stride(t, name))
        ptrs.append(t.data_ptr())
    f32 = torch.float32
    group = D
    if w_post is not None:
        if not isinstance(w_post, torch.Tensor) or w_post.dim() != 1 or not w_post.numel() or D % w_post.numel():
            raise ValueError("w_post must be a vector whose length divides D")
        group = w_post.numel()
    sizes = (N, *strides, D, group, ycode if y is not None else code, code, act, dev.index, float(alpha), float(eps))
    cfg, at, _ = _config(("norm", sizes), lambda: onela_block_norm_config(*sizes), None)
    if x_out is None and want_x:
        x_out = _empty((N, D), dt, dev, stream)
    if n_out is None and w_pre is not None:
        n_out = _empty((N, D), dt, dev, stream)
    _check(lib.onela_block_norm(
        at, *ptrs, _arg(w_post, "w_post", f32, (group,), dev, True), _arg(scale, "scale", f32, (D,), dev, True),
        _arg(w_pre, "w_pre", f32, (D,), dev, True), _arg(x_out, "x_out", dt, (N, D), dev, True),
        _arg(n_out, "n_out", dt, (N, D), dev, True), _raw_stream(stream, dev)), "onela_block_norm")
    return x_out, n_out
