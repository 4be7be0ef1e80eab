"""ctypes binding of libpkv (include/pkv.h): argument marshalling only.

Every function here has the name of the C entry point it calls and passes
plain pointers (ints, or anything with ``data_ptr()`` such as a torch tensor)
and sizes through. All compute runs in the library's CUDA kernels; there is no
fallback: ``lib()`` raises if libpkv.so is missing or does not load.
"""
from __future__ import annotations

import contextlib
import ctypes
import os
from typing import Optional

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libpkv.so")

PKV_OK, PKV_ERR_INVALID, PKV_ERR_OOM, PKV_ERR_CUDA = 0, 1, 2, 3
PKV_ERR_TIMEOUT, PKV_ERR_DEVICE_FAULT, PKV_ERR_UNSUPPORTED = 4, 5, 6
STATUS_NAMES = {0: "PKV_OK", 1: "PKV_ERR_INVALID", 2: "PKV_ERR_OOM", 3: "PKV_ERR_CUDA",
                4: "PKV_ERR_TIMEOUT", 5: "PKV_ERR_DEVICE_FAULT", 6: "PKV_ERR_UNSUPPORTED"}
PKV_BF16, PKV_F32 = 0, 1
PKV_RES_DEVICE, PKV_RES_PINNED_HOST, PKV_RES_META = 0, 1, 2
PKV_FLAG_SIMT_ONLY = 1
PKV_FLAG_LIN_ONE_TERM = 2
PKV_STAGE_KV, PKV_STAGE_GRADS = 1, 2


class PkvError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(f"{STATUS_NAMES.get(status, status)}: {msg}")
        self.status = status


class pkv_pool_desc(ctypes.Structure):
    _fields_ = [("page_size", ctypes.c_int32), ("n_kv_heads", ctypes.c_int32),
                ("n_q_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("dtype", ctypes.c_int32), ("residency", ctypes.c_int32),
                ("num_phys_pages", ctypes.c_int64), ("n_device_slots", ctypes.c_int64),
                ("flags", ctypes.c_uint32), ("reserved", ctypes.c_int32)]


class pkv_sel(ctypes.Structure):
    _fields_ = [("pages", ctypes.c_void_p), ("kmax", ctypes.c_int32),
                ("reserved", ctypes.c_int32), ("n_qp", ctypes.c_int64)]


class pkv_rope(ctypes.Structure):
    _fields_ = [("inv_freq", ctypes.c_void_p), ("positions", ctypes.c_void_p),
                ("pos0", ctypes.c_int64), ("rotary_dim", ctypes.c_int32),
                ("interleaved", ctypes.c_int32)]


class pkv_score_mod(ctypes.Structure):
    _fields_ = [("softcap", ctypes.c_float), ("reserved", ctypes.c_int32),
                ("slopes", ctypes.c_void_p), ("k_begin", ctypes.c_void_p),
                ("k_end", ctypes.c_void_p)]


class pkv_lin_desc(ctypes.Structure):
    _fields_ = [("n_kv_heads", ctypes.c_int32), ("n_q_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("residency", ctypes.c_int32), ("grads", ctypes.c_int32),
                ("n_slots", ctypes.c_int64), ("flags", ctypes.c_uint32),
                ("reserved", ctypes.c_int32)]


class pkv_lin_batch(ctypes.Structure):
    _fields_ = [("cu", ctypes.c_void_p), ("slot_in", ctypes.c_void_p),
                ("slot_out", ctypes.c_void_p), ("n_seq", ctypes.c_int64)]


class pkv_norm(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int32), ("w_dtype", ctypes.c_int32),
                ("groups", ctypes.c_int32), ("eps", ctypes.c_float),
                ("width", ctypes.c_int64), ("weight", ctypes.c_void_p),
                ("bias", ctypes.c_void_p)]


_P = ctypes.c_void_p
_I64 = ctypes.c_int64
_I32 = ctypes.c_int32
_ST = ctypes.c_int
# name -> (restype, argtypes)
_SIGS = {
    "pkv_last_error": (ctypes.c_char_p, []),
    "pkv_check": (_ST, [_P]),
    "pkv_pool_create": (_ST, [ctypes.POINTER(pkv_pool_desc), ctypes.POINTER(_P)]),
    "pkv_pool_destroy": (None, [_P]),
    "pkv_pool_free_pages": (_ST, [_P, ctypes.POINTER(_I64)]),
    "pkv_pool_arrays": (_ST, [_P] + [ctypes.POINTER(_P)] * 5),
    "pkv_seq_create": (_ST, [_P, ctypes.POINTER(_P)]),
    "pkv_seq_free": (None, [_P]),
    "pkv_seq_reset": (_ST, [_P]),
    "pkv_seq_length": (_ST, [_P, ctypes.POINTER(_I64)]),
    "pkv_seq_reserve": (_ST, [_P, _I64]),
    "pkv_get_block_table": (_ST, [_P, _P, _I64, ctypes.POINTER(_I64)]),
    "pkv_set_block_table": (_ST, [_P, _P, _I64]),
    "pkv_append": (_ST, [_P, _P, _P, _I64, _P]),
    "pkv_append_rope": (_ST, [_P, _P, _I64, _P, _P, _I64, _P, _I64, _I64,
                              ctypes.POINTER(pkv_rope), _P]),
    "pkv_rope_rows": (_ST, [_P, _P, _I64, _P, _I64, _I64, _I32, ctypes.POINTER(pkv_rope), _I32, _P]),
    "pkv_rope_grad": (_ST, [_P, _I64, _I64, ctypes.POINTER(pkv_rope), _P, _I64, _P, _I64, _P, _I64,
                            _P, _I64, _P]),
    "pkv_chunk_attn_fwd": (_ST, [_P, _P, _I64, _I64, _P, _P, ctypes.POINTER(pkv_sel), _P]),
    "pkv_chunk_attn_bwd": (_ST, [_P, _P, _P, _P, _P, _I64, _I64, _P, ctypes.POINTER(pkv_sel), _P]),
    "pkv_chunk_attn_mod_fwd": (_ST, [_P, _P, _I64, _I64, _P, _P, ctypes.POINTER(pkv_score_mod),
                                     ctypes.POINTER(pkv_sel), _P]),
    "pkv_chunk_attn_mod_bwd": (_ST, [_P, _P, _P, _P, _P, _I64, _I64, _P,
                                     ctypes.POINTER(pkv_score_mod), ctypes.POINTER(pkv_sel), _P]),
    "pkv_chunk_attn_bwd_noalloc": (_ST, [_P, _P, _P, _P, _P, _I64, _I64, _P,
                                         ctypes.POINTER(pkv_sel), _P]),
    "pkv_grad_zero": (_ST, [_P, _P]),
    "pkv_gather": (_ST, [_P, _P, _P, _P, _P, _P, _P]),
    "pkv_gather_rows": (_ST, [_P, _I64, _I64, _P, _P, _P, _P, _P]),
    "pkv_grad_accumulate": (_ST, [_P, _I64, _I64, _P, _P, _P]),
    "pkv_page_local": (_ST, [_P, _I64, _I64, _I32, _I32, _P, _P, _P]),
    "pkv_page_topk": (_ST, [_P, _P, _I64, _I64, _I32, _I32, _I32, _P, _P, _P]),
    "pkv_prefetch": (_ST, [_P, _P, _I64, _I32, _P]),
    "pkv_writeback_grads": (_ST, [_P, _P]),
    "pkv_release_slots": (_ST, [_P, _P]),
    "pkv_stage_stats": (_ST, [_P, ctypes.POINTER(_I64), ctypes.POINTER(_I64), ctypes.POINTER(_I64)]),
    "pkv_wait": (_ST, [_P, _P, _I64]),
    "pkv_selftest_umma": (_ST, [_I32, _P, _P, _P, _I32, _I32]),
    "pkv_lin_create": (_ST, [ctypes.POINTER(pkv_lin_desc), ctypes.POINTER(_P)]),
    "pkv_lin_destroy": (None, [_P]),
    "pkv_lin_arrays": (_ST, [_P] + [ctypes.POINTER(_P)] * 2),
    "pkv_lin_check": (_ST, [_P]),
    "pkv_lin_attn_fwd": (_ST, [_P] + [_P, _I64] * 4 + [_I64, _P, ctypes.POINTER(pkv_lin_batch), _P]),
    "pkv_lin_attn_bwd": (_ST, [_P] + [_P, _I64] * 7 + [_I64, _P, ctypes.POINTER(pkv_lin_batch), _P]),
    "pkv_lin_attn_step": (_ST, [_P] + [_P, _I64] * 4 + [_I64, _P, _P, _P]),
    "pkv_layer_norm_fwd": (_ST, [_P, _I64, _P, _I64, _P, _P, _I64, ctypes.POINTER(pkv_norm), _P]),
    "pkv_layer_norm_scratch": (_ST, [ctypes.POINTER(pkv_norm), _I64, ctypes.POINTER(_I64)]),
    "pkv_layer_norm_bwd": (_ST, [_P, _I64, _P, _I64, _P, _P, _P, _I64, _P, _P, _I32, _P, _I64,
                                 ctypes.POINTER(pkv_norm), _P]),
    "pkv_profile_enable": (_ST, [_I32]),
    "pkv_profile_collect": (_ST, [_I32, _P, _P, _P, ctypes.POINTER(_I32)]),
}
EXPORTED = tuple(_SIGS)

_lib: Optional[ctypes.CDLL] = None


def lib() -> ctypes.CDLL:
    """Loads libpkv.so (built by ``paged_kv_chunk_chunked_gb300.build.build()``)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"{LIB_PATH} is missing: run __graft_entry__.build() first "
                              "(the CUDA library is required; there is no CPU path)")
        l = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in _SIGS.items():
            f = getattr(l, name)
            f.restype = res
            f.argtypes = args
        _lib = l
    return _lib


def ptr(x) -> Optional[int]:
    """Address of a tensor-like (``data_ptr()``), an int, or None. Every array
    the library reads or writes is dense in the layout its header states, so a
    strided view is refused here instead of being read as if it were dense."""
    if x is None:
        return None
    if isinstance(x, int):
        return x
    if hasattr(x, "is_contiguous") and not x.is_contiguous():
        raise ValueError(f"tensor of shape {tuple(x.shape)} with strides {x.stride()} is not "
                         "contiguous; pass .contiguous()")
    return x.data_ptr()


# What a handle's tensors must be, for the calls that check them: pool or sequence
# handle -> (torch dtype, Hq, Hkv, d). Entered at creation.
_KIND: dict = {}
_ANY = (None, None, None, None)


def _torch_dtype(dtype):
    try:
        import torch
    except ImportError:                       # raw addresses only
        return None
    return torch.bfloat16 if dtype == PKV_BF16 else torch.float32


_HERE = contextlib.nullcontext()
_DTYPES = {}                                  # by name


def _device(stream):
    """The stream's device, which a call's tensors must be on; None: the current one."""
    return getattr(stream, "device_index", None)


def _current(dev):
    """The stream's device as the current one, for calls without a handle (whose
    kernels run on the current device); None leaves it as it is."""
    if dev is None:
        return _HERE
    import torch
    return _HERE if torch.cuda.current_device() == dev else torch.cuda.device(dev)


def _on_device(x, dev) -> None:
    at = x.get_device()                       # -1: host memory
    if dev is None and at >= 0:
        import torch
        want = torch.cuda.current_device()
    else:
        want = dev
    if at < 0 or at != want:
        raise ValueError(f"expected a CUDA tensor on {'the current device' if dev is None else f'cuda:{dev}'}, "
                         f"got one on {x.device}")


def rows_ptr(x, n: int, heads=None, d=None, dtype=None):
    """(address, row stride in elements) of a tensor [n, heads, d] whose rows are
    dense and may lie apart, such as a slice of a wider projection's output; an
    int address is taken as dense (stride 0)."""
    if x is None or isinstance(x, int):
        return x, 0
    shape, stride = x.shape, x.stride()
    if len(shape) != 3 or shape[0] != n or (heads and shape[1] != heads) or (d and shape[2] != d):
        raise ValueError(f"expected a tensor [{n}, {heads or 'heads'}, {d or 'd'}], got shape {tuple(shape)}")
    if dtype is not None and x.dtype != dtype:
        raise ValueError(f"expected {dtype} like the pool's pages, got {x.dtype}")
    _, h, w = shape
    if stride != (h * w, w, 1) and n * h * w and (stride[2] != 1 or (h > 1 and stride[1] != w) or
                                                  (n > 1 and stride[0] < h * w)):
        raise ValueError(f"tensor of shape {tuple(shape)} with strides {stride}: every row "
                         "must be dense [heads, d] memory of its own")
    return x.data_ptr(), (stride[0] if n > 1 else 0)


def _rows(x, n, heads, d, dtype, dev, dense=False):
    """rows_ptr of a call's operand, on its device; dense: without gaps."""
    if x is None or isinstance(x, int):
        return x, 0
    p = rows_ptr(x, n, heads, d, dtype)
    if x.get_device() != dev:
        _on_device(x, dev)
    if dense and p[1] and p[1] != x.shape[1] * x.shape[2]:
        raise ValueError(f"tensor of shape {tuple(x.shape)} with strides {x.stride()} is not "
                         "contiguous; pass .contiguous()")
    return p


def _typed(x, name: str, dtype: str, n=None):
    """Address of a tensor that must have this dtype (and number of elements), an int, or None."""
    if x is None or isinstance(x, int):
        return x
    if str(x.dtype) != "torch." + dtype:
        raise ValueError(f"{name} must be {dtype}, got {x.dtype}")
    if n is not None and x.numel() != n:
        raise ValueError(f"{name} must have {n} elements, got {x.numel()}")
    return ptr(x)


def rope(inv_freq, pos0: int = 0, positions=None, interleaved: bool = False, rotary_dim: Optional[int] = None) -> pkv_rope:
    """The rotation of a call: inv_freq float32 [rotary_dim / 2], positions int64
    [n] (one per row) or None for pos0 + row. Keeps the tensors alive. inv_freq may
    be an address, with rotary_dim given."""
    p = _typed(inv_freq, "inv_freq", "float32")
    n = None if inv_freq is None or isinstance(inv_freq, int) else 2 * inv_freq.numel()
    if n is None and rotary_dim is None:
        raise ValueError("inv_freq is not a tensor: rotary_dim is needed")
    if n is not None and rotary_dim not in (None, n):
        raise ValueError(f"inv_freq must have rotary_dim / 2 = {rotary_dim // 2} elements, got {n // 2}")
    r = pkv_rope(p, _typed(positions, "positions", "int64"), int(pos0), n if n is not None else int(rotary_dim),
                 1 if interleaved else 0)
    r.tensors = (inv_freq, positions)
    return r


def _rope(r: Optional[pkv_rope], n: int, dev=None):
    if r is None:
        return None
    inv_freq, pos = getattr(r, "tensors", (None, None))
    if inv_freq is not None and not isinstance(inv_freq, int):
        _on_device(inv_freq, dev)
    if pos is not None and not isinstance(pos, int):
        _on_device(pos, dev)
        if pos.numel() != n:
            raise ValueError(f"positions must have one entry per row ({n}), got {pos.numel()}")
    return ctypes.byref(r)


def score_mod(softcap: float = 0.0, slopes=None, k_begin=None, k_end=None) -> pkv_score_mod:
    """The score modification of a call: softcap (0: none), slopes float32 [Hq],
    k_begin / k_end int64 [n_q] (first visible key of each query, one past its
    last). Keeps the tensors alive."""
    m = pkv_score_mod(float(softcap), 0, _typed(slopes, "slopes", "float32"),
                      _typed(k_begin, "k_begin", "int64"), _typed(k_end, "k_end", "int64"))
    m.tensors = (slopes, k_begin, k_end)
    return m


def _mod(m: Optional[pkv_score_mod], n_q: int, heads, dev):
    if m is None:
        return None
    for x, n, what in zip(getattr(m, "tensors", (None, None, None)), (heads, n_q, n_q),
                          ("slopes: one entry per query head", "k_begin: one entry per query",
                           "k_end: one entry per query")):
        if x is None or isinstance(x, int):
            continue
        if n is not None and x.numel() != n:
            raise ValueError(f"{what} ({n}), got {x.numel()}")
        _on_device(x, dev)
    return ctypes.byref(m)


def _lse_ptr(x, heads, n_q, dev):
    if x is None or isinstance(x, int):
        return x
    if x.element_size() != 4 or not x.is_floating_point() or (heads and x.shape != (heads, n_q)):
        raise ValueError(f"lse must be float32 [{heads or 'heads'}, {n_q}], got {x.dtype} {tuple(x.shape)}")
    _on_device(x, dev)
    return ptr(x)


def stream_ptr(stream) -> Optional[int]:
    if stream is None:
        return None
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _check(status: int):
    if status != PKV_OK:
        raise PkvError(status, lib().pkv_last_error().decode())


def _sel(sel) -> Optional[pkv_sel]:
    """(pages tensor [n_qp, Hkv, kmax]) -> pkv_sel by reference, or None for dense."""
    if sel is None:
        return None
    s = pkv_sel()
    s.pages = ptr(sel)
    s.kmax = int(sel.shape[-1])
    s.n_qp = int(sel.shape[0])
    return ctypes.byref(s)


def _mod_sel(sel, heads, dev) -> Optional[pkv_sel]:
    """_sel of a call that checks its tensors: int32 [n_qp, Hkv, kmax], on its device."""
    if sel is None:
        return None
    if str(sel.dtype) != "torch.int32" or sel.dim() != 3 or (heads and sel.shape[1] != heads):
        raise ValueError(f"sel must be int32 [query pages, {heads or 'Hkv'}, kmax], got {sel.dtype} {tuple(sel.shape)}")
    _on_device(sel, dev)
    return _sel(sel)


# ---------------------------------------------------------------- one function per entry point

def pkv_last_error() -> str:
    return lib().pkv_last_error().decode()


def pkv_check(pool) -> None:
    _check(lib().pkv_check(pool))


def pkv_pool_create(page_size, n_kv_heads, n_q_heads, head_dim, dtype=PKV_BF16,
                    num_phys_pages=1, residency=PKV_RES_DEVICE, n_device_slots=0, flags=0) -> int:
    d = pkv_pool_desc(page_size, n_kv_heads, n_q_heads, head_dim, dtype, residency,
                      num_phys_pages, n_device_slots, flags, 0)
    out = _P()
    _check(lib().pkv_pool_create(ctypes.byref(d), ctypes.byref(out)))
    # (a tuple of the pool's own: its sequences' entries are the same object)
    _KIND[out.value] = (_torch_dtype(dtype), n_q_heads, n_kv_heads, head_dim)
    return out.value


def pkv_pool_destroy(pool) -> None:
    kind = _KIND.pop(pool, None)
    for seq in [h for h, x in _KIND.items() if x is kind]:    # freed with the pool
        del _KIND[seq]
    lib().pkv_pool_destroy(pool)


def pkv_pool_free_pages(pool) -> int:
    n = _I64()
    _check(lib().pkv_pool_free_pages(pool, ctypes.byref(n)))
    return n.value


def pkv_pool_arrays(pool) -> dict:
    vals = [_P() for _ in range(5)]
    _check(lib().pkv_pool_arrays(pool, *[ctypes.byref(v) for v in vals]))
    return dict(zip(("k", "v", "dk", "dv", "rep"), (v.value for v in vals)))


def pkv_seq_create(pool) -> int:
    out = _P()
    _check(lib().pkv_seq_create(pool, ctypes.byref(out)))
    _KIND[out.value] = _KIND.get(pool, _ANY)
    return out.value


def pkv_seq_free(seq) -> None:
    _KIND.pop(seq, None)
    lib().pkv_seq_free(seq)


def pkv_seq_reset(seq) -> None:
    _check(lib().pkv_seq_reset(seq))


def pkv_seq_length(seq) -> int:
    n = _I64()
    _check(lib().pkv_seq_length(seq, ctypes.byref(n)))
    return n.value


def pkv_seq_reserve(seq, n_tok) -> None:
    _check(lib().pkv_seq_reserve(seq, n_tok))


def pkv_get_block_table(seq) -> list:
    n = _I64()
    _check(lib().pkv_get_block_table(seq, None, 0, ctypes.byref(n)))
    buf = (ctypes.c_int32 * max(1, n.value))()
    _check(lib().pkv_get_block_table(seq, ctypes.cast(buf, _P), n.value, ctypes.byref(n)))
    return list(buf[: n.value])


def pkv_set_block_table(seq, bt) -> None:
    arr = (ctypes.c_int32 * max(1, len(bt)))(*[int(x) for x in bt])
    _check(lib().pkv_set_block_table(seq, ctypes.cast(arr, _P), len(bt)))


def pkv_append(seq, k, v, n_tok, stream=None) -> None:
    _check(lib().pkv_append(seq, ptr(k), ptr(v), n_tok, stream_ptr(stream)))


def pkv_append_rope(seq, q, q_out, k, v, n_tok, rope, stream=None) -> None:
    """q, k, v: tensors [n_tok, heads, d] whose rows may lie apart (slices of one
    projection's output); q and q_out (dense) may be None."""
    (dt, hq, hkv, d), dev = _KIND.get(seq, _ANY), _device(stream)
    qp, qs = _rows(q, n_tok, hq, d, dt, dev)
    op, _ = _rows(q_out, n_tok, hq, d, dt, dev, dense=True)
    kp, ks = _rows(k, n_tok, hkv, d, dt, dev)
    vp, vs = _rows(v, n_tok, hkv, d, dt, dev)
    _check(lib().pkv_append_rope(seq, qp, qs, op, kp, ks, vp, vs, n_tok, _rope(rope, n_tok, dev),
                                 stream_ptr(stream)))


def pkv_rope_rows(pool, x, out, n, n_heads, rope, inverse=False, stream=None) -> None:
    (dt, _, _, d), dev = _KIND.get(pool, _ANY), _device(stream)
    xp, xs = _rows(x, n, n_heads, d, dt, dev)
    op, os_ = _rows(out, n, n_heads, d, dt, dev)
    _check(lib().pkv_rope_rows(pool, xp, xs, op, os_, n, n_heads, _rope(rope, n, dev),
                               1 if inverse else 0, stream_ptr(stream)))


def pkv_rope_grad(seq, row0, n_rows, rope, dq=None, dq_out=None, dk_out=None, dv_out=None,
                  stream=None) -> None:
    """dq and the outputs: tensors [n_rows, heads, d] whose rows may lie apart."""
    (dt, hq, hkv, d), dev = _KIND.get(seq, _ANY), _device(stream)
    qp, qs = _rows(dq, n_rows, hq, d, dt, dev)
    op, os_ = _rows(dq_out, n_rows, hq, d, dt, dev)
    kp, ks = _rows(dk_out, n_rows, hkv, d, dt, dev)
    vp, vs = _rows(dv_out, n_rows, hkv, d, dt, dev)
    _check(lib().pkv_rope_grad(seq, row0, n_rows, _rope(rope, n_rows, dev), qp, qs, op, os_, kp, ks, vp, vs,
                               stream_ptr(stream)))


def pkv_chunk_attn_fwd(seq, q, q_start, n_q, o, lse, sel=None, stream=None) -> None:
    _check(lib().pkv_chunk_attn_fwd(seq, ptr(q), q_start, n_q, ptr(o), ptr(lse), _sel(sel),
                                    stream_ptr(stream)))


def pkv_chunk_attn_bwd(seq, q, o, dout, lse, q_start, n_q, dq, sel=None, stream=None) -> None:
    _check(lib().pkv_chunk_attn_bwd(seq, ptr(q), ptr(o), ptr(dout), ptr(lse), q_start, n_q,
                                    ptr(dq), _sel(sel), stream_ptr(stream)))


def pkv_chunk_attn_mod_fwd(seq, q, q_start, n_q, o, lse, mod, sel=None, stream=None) -> None:
    (dt, hq, hkv, d), dev = _KIND.get(seq, _ANY), _device(stream)
    (qp, _), (op, _) = (_rows(x, n_q, hq, d, dt, dev, dense=True) for x in (q, o))
    _check(lib().pkv_chunk_attn_mod_fwd(seq, qp, q_start, n_q, op, _lse_ptr(lse, hq, n_q, dev),
                                        _mod(mod, n_q, hq, dev), _mod_sel(sel, hkv, dev), stream_ptr(stream)))


def pkv_chunk_attn_mod_bwd(seq, q, o, dout, lse, q_start, n_q, dq, mod, sel=None, stream=None) -> None:
    (dt, hq, hkv, d), dev = _KIND.get(seq, _ANY), _device(stream)
    (qp, _), (op, _), (gp, _), (dp, _) = (_rows(x, n_q, hq, d, dt, dev, dense=True)
                                          for x in (q, o, dout, dq))
    _check(lib().pkv_chunk_attn_mod_bwd(seq, qp, op, gp, _lse_ptr(lse, hq, n_q, dev), q_start, n_q, dp,
                                        _mod(mod, n_q, hq, dev), _mod_sel(sel, hkv, dev), stream_ptr(stream)))


def pkv_chunk_attn_bwd_noalloc(seq, q, o, dout, lse, q_start, n_q, dq, sel=None,
                               stream=None) -> None:
    """Same as pkv_chunk_attn_bwd, with the library's fixed device scratch instead
    of an allocation (for callers that cannot allocate at call time)."""
    _check(lib().pkv_chunk_attn_bwd_noalloc(seq, ptr(q), ptr(o), ptr(dout), ptr(lse), q_start,
                                            n_q, ptr(dq), _sel(sel), stream_ptr(stream)))


def pkv_grad_zero(seq, stream=None) -> None:
    _check(lib().pkv_grad_zero(seq, stream_ptr(stream)))


def pkv_grad_accumulate(seq, row0, n_rows, dk=None, dv=None, stream=None) -> None:
    _check(lib().pkv_grad_accumulate(seq, row0, n_rows, ptr(dk), ptr(dv), stream_ptr(stream)))


def pkv_gather(seq, k=None, v=None, dk=None, dv=None, rep=None, stream=None) -> None:
    _check(lib().pkv_gather(seq, ptr(k), ptr(v), ptr(dk), ptr(dv), ptr(rep), stream_ptr(stream)))


def pkv_gather_rows(seq, row0, n_rows, k=None, v=None, dk=None, dv=None, stream=None) -> None:
    _check(lib().pkv_gather_rows(seq, row0, n_rows, ptr(k), ptr(v), ptr(dk), ptr(dv),
                                 stream_ptr(stream)))


def pkv_page_topk(seq, q, q_start, n_q, k, n_sink, n_local, pages_out, counts_out=None,
                  stream=None) -> None:
    _check(lib().pkv_page_topk(seq, ptr(q), q_start, n_q, k, n_sink, n_local, ptr(pages_out),
                               ptr(counts_out), stream_ptr(stream)))


def pkv_page_local(seq, q_start, n_q, n_sink, n_local, pages_out, counts_out=None,
                   stream=None) -> None:
    _check(lib().pkv_page_local(seq, q_start, n_q, n_sink, n_local, ptr(pages_out),
                                ptr(counts_out), stream_ptr(stream)))


def pkv_prefetch(seq, logical_pages=None, n=0, what=3, side=None) -> None:
    """what: PKV_STAGE_KV (1) | PKV_STAGE_GRADS (2)."""
    _check(lib().pkv_prefetch(seq, ptr(logical_pages), n, what, stream_ptr(side)))


def pkv_writeback_grads(seq, side=None) -> None:
    _check(lib().pkv_writeback_grads(seq, stream_ptr(side)))


def pkv_release_slots(seq, side=None) -> None:
    _check(lib().pkv_release_slots(seq, stream_ptr(side)))


def pkv_stage_stats(seq) -> dict:
    """Page-heads moved by the sequence's staging so far."""
    kv, gi, go = ctypes.c_int64(), ctypes.c_int64(), ctypes.c_int64()
    _check(lib().pkv_stage_stats(seq, ctypes.byref(kv), ctypes.byref(gi), ctypes.byref(go)))
    return {"kv_in": kv.value, "grads_in": gi.value, "grads_out": go.value}


def pkv_wait(seq, main=None, timeout_us=10_000_000) -> None:
    _check(lib().pkv_wait(seq, stream_ptr(main), timeout_us))


def pkv_lin_create(n_kv_heads, n_q_heads, head_dim, dtype=PKV_BF16, n_slots=1, grads=False,
                   residency=PKV_RES_DEVICE, flags=0) -> int:
    d = pkv_lin_desc(n_kv_heads, n_q_heads, head_dim, dtype, residency, 1 if grads else 0, n_slots, flags, 0)
    out = _P()
    _check(lib().pkv_lin_create(ctypes.byref(d), ctypes.byref(out)))
    _KIND[out.value] = (_torch_dtype(dtype), n_q_heads, n_kv_heads, head_dim)
    return out.value


def pkv_lin_destroy(lin) -> None:
    _KIND.pop(lin, None)
    lib().pkv_lin_destroy(lin)


def pkv_lin_arrays(lin) -> dict:
    """Addresses of the float32 [n_slots, Hkv, d, d] states and of their gradients (None without)."""
    s, g = _P(), _P()
    _check(lib().pkv_lin_arrays(lin, ctypes.byref(s), ctypes.byref(g)))
    return {"state": s.value, "dstate": g.value}


def pkv_lin_check(lin) -> None:
    _check(lib().pkv_lin_check(lin))


def lin_batch(n_seq: int = 1, cu=None, slot_in=None, slot_out=None) -> pkv_lin_batch:
    """The sequences of a call: cu int64 [n_seq + 1] (None: one sequence of all
    rows), slot_in and slot_out int32 [n_seq] or None. Keeps the tensors alive."""
    b = pkv_lin_batch(_typed(cu, "cu", "int64", n_seq + 1), _typed(slot_in, "slot_in", "int32", n_seq),
                      _typed(slot_out, "slot_out", "int32", n_seq), int(n_seq))
    b.tensors = (cu, slot_in, slot_out)
    return b


def _array(x, name: str, dtype: str, n, dev):
    """_typed of a call's array, on its device. Usual ones pass by the first comparison."""
    if x is None or x.__class__ is int:
        return x
    if x.get_device() == dev and x.dtype is _dtypes()[dtype] and x.numel() == n and x.is_contiguous():
        return x.data_ptr()
    if x.get_device() != dev:
        _on_device(x, dev)
    return _typed(x, name, dtype, n)


def _dtypes():
    if not _DTYPES:
        import torch
        _DTYPES.update(float32=torch.float32, int32=torch.int32, int64=torch.int64)
    return _DTYPES


def _lin_operands(lin, n, operands, dev):
    """Addresses and row strides of tensors [n, heads, d], (tensor, of the query heads)
    each. Usual ones pass by one comparison of their shape and strides each (these calls
    are short: a microsecond of checks a tensor shows); _rows looks at the others."""
    dt, hq, hkv, d = _KIND.get(lin, _ANY)
    at = []
    for x, of_q in operands:
        h = hq if of_q else hkv
        if x.__class__ is not int and x is not None and d and x.shape == (n, h, d) and x.dtype is dt and x.get_device() == dev:
            s0, s1, s2 = x.stride()
            if s2 == 1 and s1 == d and s0 >= h * d:
                at.append(x.data_ptr())
                at.append(s0 if n > 1 else 0)
                continue
        at.extend(_rows(x, n, h, d, dt, dev))
    return at


def _lin_batch_ref(batch, dev):
    for x in getattr(batch, "tensors", ()):
        if x is not None and x.__class__ is not int and x.get_device() != dev:
            _on_device(x, dev)
    return ctypes.byref(batch)


def _lin_heads(lin):
    return _KIND.get(lin, _ANY)[2]


def pkv_lin_attn_fwd(lin, q, k, v, o, n, log_decay, batch, stream=None) -> None:
    """q, k, v, o: tensors [n, heads, d] whose rows may lie apart."""
    dev = _device(stream)
    at = _lin_operands(lin, n, ((q, True), (k, False), (v, False), (o, True)), dev)
    _check(lib().pkv_lin_attn_fwd(lin, *at, n, _array(log_decay, "log_decay", "float32", _lin_heads(lin), dev),
                                  _lin_batch_ref(batch, dev), stream_ptr(stream)))


def pkv_lin_attn_bwd(lin, q, k, v, dout, dq, dk, dv, n, log_decay, batch, stream=None) -> None:
    """All seven: tensors [n, heads, d] whose rows may lie apart."""
    dev = _device(stream)
    at = _lin_operands(lin, n, ((q, True), (k, False), (v, False), (dout, True), (dq, True), (dk, False), (dv, False)), dev)
    _check(lib().pkv_lin_attn_bwd(lin, *at, n, _array(log_decay, "log_decay", "float32", _lin_heads(lin), dev),
                                  _lin_batch_ref(batch, dev), stream_ptr(stream)))


def pkv_lin_attn_step(lin, q, k, v, o, n, log_decay, slots, stream=None) -> None:
    """q, k, v, o: tensors [n, heads, d] whose rows may lie apart; slots int32 [n]."""
    dev = _device(stream)
    at = _lin_operands(lin, n, ((q, True), (k, False), (v, False), (o, True)), dev)
    _check(lib().pkv_lin_attn_step(lin, *at, n, _array(log_decay, "log_decay", "float32", _lin_heads(lin), dev),
                                   _array(slots, "slots", "int32", n, dev), stream_ptr(stream)))


def norm(width, groups: int = 1, eps: float = 1e-5, weight=None, bias=None, dtype=PKV_BF16, w_dtype=None) -> pkv_norm:
    """The normalisation of a call: rows of groups * width columns in `dtype`; weight
    and bias [groups * width], both bfloat16 or both float32 (w_dtype, where they are
    addresses), or None. Keeps the tensors alive."""
    kinds = {"torch.bfloat16": PKV_BF16, "torch.float32": PKV_F32}
    for name, x in (("weight", weight), ("bias", bias)):
        if x is None or isinstance(x, int):
            continue
        if str(x.dtype) not in kinds or w_dtype not in (None, kinds[str(x.dtype)]):
            raise ValueError(f"weight and bias must both be bfloat16 or both float32, got {x.dtype} for {name}")
        w_dtype = kinds[str(x.dtype)]
        if x.numel() != groups * width:
            raise ValueError(f"{name} must have groups * width = {groups * width} elements, got {x.numel()}")
    m = pkv_norm(int(dtype), dtype if w_dtype is None else w_dtype, int(groups), float(eps), int(width), ptr(weight), ptr(bias))
    m.tensors = (weight, bias)
    m.torch_dtype = _torch_dtype(dtype)
    return m


def _norm_rows(x, n: int, m: pkv_norm, dev, name: str):
    """(address, row stride) of a tensor [n, columns] (any shape that has these
    columns in its trailing dimensions), an int, or None."""
    if x is None or isinstance(x, int):
        return x, 0
    cols = m.groups * m.width
    if x.dtype != m.torch_dtype:
        raise ValueError(f"{name} must be {m.torch_dtype}, got {x.dtype}")
    if x.shape == (n, cols) and x.get_device() == dev:        # the usual ones
        s0, s1 = x.stride()
        if s1 == 1 and s0 >= cols:
            return x.data_ptr(), (s0 if n > 1 else 0)
    if x.dim() < 1 or x.shape[0] != n or x.numel() != n * cols:
        raise ValueError(f"{name} must have {n} rows of {cols} columns, got shape {tuple(x.shape)}")
    dense = 1                                 # every row dense memory of its own
    for size, stride in zip(reversed(x.shape[1:]), reversed(x.stride()[1:])):
        if size > 1 and stride != dense and n:
            raise ValueError(f"{name} of shape {tuple(x.shape)} with strides {x.stride()}: rows must be dense")
        dense *= size
    if n > 1 and x.stride(0) < cols:
        raise ValueError(f"{name} of shape {tuple(x.shape)} with strides {x.stride()}: rows overlap")
    _on_device(x, dev)
    return x.data_ptr(), (x.stride(0) if n > 1 else 0)


def _norm_ref(m: pkv_norm, dev):
    for x in getattr(m, "tensors", ()):
        if x is not None and x.__class__ is not int and x.get_device() != dev:
            _on_device(x, dev)
    return ctypes.byref(m)


def pkv_layer_norm_fwd(x, y, mean, rstd, n, norm, stream=None) -> None:
    """x, y: tensors of n rows that may lie apart; mean, rstd float32 [n, groups] or None."""
    dev = _device(stream)
    (xp, xs), (yp, ys) = _norm_rows(x, n, norm, dev, "x"), _norm_rows(y, n, norm, dev, "y")
    m, r = _array(mean, "mean", "float32", n * norm.groups, dev), _array(rstd, "rstd", "float32", n * norm.groups, dev)
    with _current(dev):
        _check(lib().pkv_layer_norm_fwd(xp, xs, yp, ys, m, r, n, _norm_ref(norm, dev), stream_ptr(stream)))


def pkv_layer_norm_scratch(norm, n) -> int:
    """Floats of scratch that pkv_layer_norm_bwd needs for n rows."""
    f = _I64()
    _check(lib().pkv_layer_norm_scratch(ctypes.byref(norm), n, ctypes.byref(f)))
    return f.value


def pkv_layer_norm_bwd(dy, x, mean, rstd, dx, dw, db, n, norm, scratch, accumulate=False, stream=None) -> None:
    """dy, x, dx: tensors of n rows that may lie apart; mean, rstd the forward's;
    dw, db float32 [groups * width], each or dx may be None."""
    dev = _device(stream)
    at = [y for t, w in ((dy, "dy"), (x, "x"), (dx, "dx")) for y in _norm_rows(t, n, norm, dev, w)]
    m, r = _array(mean, "mean", "float32", n * norm.groups, dev), _array(rstd, "rstd", "float32", n * norm.groups, dev)
    gw, gb = (_array(t, w, "float32", norm.groups * norm.width, dev) for t, w in ((dw, "dw"), (db, "db")))
    if scratch is not None and not isinstance(scratch, int):
        need = pkv_layer_norm_scratch(norm, n) if gw or gb else 0
        if scratch.numel() < need:
            raise ValueError(f"scratch must have {need} floats, got {scratch.numel()}")
        scratch = _array(scratch, "scratch", "float32", None, dev)
    with _current(dev):
        _check(lib().pkv_layer_norm_bwd(*at[:4], m, r, *at[4:], gw, gb, 1 if accumulate else 0, scratch, n,
                                        _norm_ref(norm, dev), stream_ptr(stream)))


def pkv_profile_enable(on: bool) -> None:
    _check(lib().pkv_profile_enable(1 if on else 0))


def pkv_profile_collect(max_kernels: int = 64) -> dict:
    """{kernel name: (launches, total device ms)} since profiling was enabled."""
    names = ctypes.create_string_buffer(64 * max_kernels)
    ms = (ctypes.c_double * max_kernels)()
    cnt = (ctypes.c_int64 * max_kernels)()
    n = _I32()
    _check(lib().pkv_profile_collect(max_kernels, ctypes.cast(names, _P), ctypes.cast(ms, _P),
                                     ctypes.cast(cnt, _P), ctypes.byref(n)))
    out = {}
    for k in range(min(n.value, max_kernels)):
        name = names.raw[64 * k: 64 * k + 64].split(b"\0", 1)[0].decode()
        out[name] = (int(cnt[k]), float(ms[k]))
    return out


def pkv_selftest_umma(mode, a, b, d, lbo=0, sbo=0) -> None:
    _check(lib().pkv_selftest_umma(mode, ptr(a), ptr(b), ptr(d), lbo, sbo))
