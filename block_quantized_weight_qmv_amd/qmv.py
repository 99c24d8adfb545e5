"""Python binding of libqmv.so: the C ABI of include/qmv.h, one function per entry point.

Argument marshalling only.  Device buffers are torch tensors (or raw integer
device pointers); every computation runs in the library's HIP kernels.  If the
library is not built, the first call raises: there is no fallback path.

torch is imported before the library is loaded so that libqmv.so binds to the
HIP runtime torch already mapped (both use the soname libamdhip64.so.7), which
makes torch's hipStream_t values valid inside the library.
"""
from __future__ import annotations

import ctypes
import os

import numpy as np

PKG_DIR = os.path.dirname(os.path.abspath(__file__))
# QMV_LIBRARY names another build of the same library (the sanitizer build of
# the CPU test suite); by default the in-tree libqmv.so.
LIB_PATH = os.environ.get("QMV_LIBRARY") or os.path.join(PKG_DIR, "libqmv.so")

FMT = {"q8_0": 1, "q4_k": 2, "q6_k": 3, "int4_g128": 4, "q5_k": 5}
DTYPE = {"f32": 0, "f16": 1, "bf16": 2}
LAYOUT = {"blocks": 0, "planes": 1}

QMV_OK = 0
STATUS = {0: "QMV_OK", -1: "QMV_ERR_NULL", -2: "QMV_ERR_FORMAT", -3: "QMV_ERR_SHAPE",
          -4: "QMV_ERR_ALIGN", -5: "QMV_ERR_SIZE", -6: "QMV_ERR_UNSUPPORTED",
          -7: "QMV_ERR_RANGE", -8: "QMV_ERR_HIP"}


class QmvError(RuntimeError):
    def __init__(self, status: int, detail: str):
        self.status = status
        super().__init__(f"{STATUS.get(status, status)}: {detail}")


class QmvWeights(ctypes.Structure):
    """Mirror of struct qmv_weights."""
    _fields_ = [("fmt", ctypes.c_int32), ("layout", ctypes.c_int32),
                ("rows", ctypes.c_int64), ("cols", ctypes.c_int64),
                ("data", ctypes.c_void_p), ("nbytes", ctypes.c_uint64),
                ("scales_offset", ctypes.c_uint64)]


class QmvGemvItem(ctypes.Structure):
    """Mirror of struct qmv_gemv_item."""
    _fields_ = [("W", ctypes.POINTER(QmvWeights)), ("x", ctypes.c_void_p), ("y", ctypes.c_void_p)]


class QmvAttnArgs(ctypes.Structure):
    """Mirror of struct qmv_attn_args."""
    _fields_ = [(n, ctypes.c_int32) for n in ("dtype", "head_dim", "heads", "kv_heads", "nseq", "max_rows",
                                              "page_size")] + \
               [("scale", ctypes.c_float)] + \
               [(n, ctypes.c_int64) for n in ("rows", "prefix_len", "max_suffix", "num_pages", "table_stride",
                                              "q_row", "q_head", "out_row", "out_head", "prefix_row", "prefix_head",
                                              "page_stride", "page_row", "page_head")] + \
               [(n, ctypes.c_void_p) for n in ("q", "k_prefix", "v_prefix", "prefix_pages", "k_pages", "v_pages",
                                               "block_table", "row_start", "suffix_len", "tree_mask", "out", "lse")]


class QmvVerifyArgs(ctypes.Structure):
    """Mirror of struct qmv_verify_args."""
    _fields_ = [(n, ctypes.c_int32) for n in ("logits_dtype", "nseq", "max_rows", "reserved")] + \
               [(n, ctypes.c_int64) for n in ("rows", "vocab", "logits_row", "draft_row")] + \
               [(n, ctypes.c_void_p) for n in ("logits", "draft_probs", "tokens", "row_start", "temperature",
                                               "u_accept", "u_sample", "out_tokens", "accepted")]


_lib = None

_i32, _i64, _u64, _p = ctypes.c_int32, ctypes.c_int64, ctypes.c_uint64, ctypes.c_void_p
_SIGS = {
    "qmv_block_size": (_i32, [_i32]),
    "qmv_packed_size": (_u64, [_i32, _i64, _i64]),
    "qmv_pack_q8_0": (_i32, [_p, _p, _i64, _i64, _p, _u64]),
    "qmv_pack_q4_k": (_i32, [_p, _p, _p, _p, _p, _i64, _i64, _p, _u64]),
    "qmv_pack_q5_k": (_i32, [_p, _p, _p, _p, _p, _i64, _i64, _p, _u64]),
    "qmv_pack_q6_k": (_i32, [_p, _p, _p, _i64, _i64, _p, _u64]),
    "qmv_pack_int4_g128": (_i32, [_p, _p, _i64, _i64, _p, _u64]),
    "qmv_create_weights": (_i32, [_i32, _i64, _i64, _p, _u64, ctypes.POINTER(QmvWeights)]),
    "qmv_planes_size": (_u64, [_i32, _i64, _i64]),
    "qmv_create_weights_planes": (_i32, [_i32, _i64, _i64, _p, _u64, ctypes.POINTER(QmvWeights)]),
    "qmv_repack_planes": (_i32, [ctypes.POINTER(QmvWeights), _p, _u64, ctypes.POINTER(QmvWeights), _p]),
    "qmv_gemv": (_i32, [_i32, ctypes.POINTER(QmvWeights), _p, _i32, _p, _i64, _i64, _i64, _p]),
    "qmv_gemv_noalloc": (_i32, [_i32, ctypes.POINTER(QmvWeights), _p, _i32, _p, _i64, _i64, _i64, _p]),
    "qmv_gemv_multi": (_i32, [_i32, _i32, _i64, ctypes.POINTER(QmvGemvItem), _i32, _p]),
    "qmv_workspace_size": (_i32, [_i32, _i32, _i64, ctypes.POINTER(QmvGemvItem), _i32,
                                  ctypes.POINTER(_u64)]),
    "qmv_gemv_multi_ws": (_i32, [_i32, _i32, _i64, ctypes.POINTER(QmvGemvItem), _i32, _p, _u64, _p]),
    "qmv_gemv_swiglu": (_i32, [_i32, ctypes.POINTER(QmvWeights), ctypes.POINTER(QmvWeights), _p, _i32, _p,
                               _i64, _i64, _i64, _p]),
    "qmv_dequant": (_i32, [ctypes.POINTER(QmvWeights), _p, _i32, _p]),
    "qmv_embed": (_i32, [ctypes.POINTER(QmvWeights), _p, _i64, ctypes.c_float, _p, _i32, _p]),
    "qmv_attn_workspace_size": (_i32, [ctypes.POINTER(QmvAttnArgs), ctypes.POINTER(_u64)]),
    "qmv_attn": (_i32, [ctypes.POINTER(QmvAttnArgs), _p, _u64, _p]),
    "qmv_verify_workspace_size": (_i32, [ctypes.POINTER(QmvVerifyArgs), ctypes.POINTER(_u64)]),
    "qmv_verify": (_i32, [ctypes.POINTER(QmvVerifyArgs), _p, _u64, _p]),
    "qmv_probe_read_outputs": (_i64, [_u64]),
    "qmv_probe_read": (_i32, [_p, _u64, _p, _p]),
    "qmv_probe_copy": (_i32, [_p, _p, _u64, _p]),
    "qmv_status_string": (ctypes.c_char_p, [_i32]),
    "qmv_last_error": (ctypes.c_char_p, []),
}
EXPORTED = tuple(_SIGS)


def lib() -> ctypes.CDLL:
    """Load libqmv.so (once).  Raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                               "`python -m block_quantized_weight_qmv_amd.build`")
        try:
            import torch  # noqa: F401  (maps torch's HIP runtime first)
        except ImportError:
            pass
        handle = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in _SIGS.items():
            fn = getattr(handle, name)
            fn.restype = res
            fn.argtypes = args
        _lib = handle
    return _lib


def _check(status: int) -> None:
    if status != QMV_OK:
        raise QmvError(status, (lib().qmv_last_error() or b"").decode())


def _ptr(a):
    """Device or host address of a torch tensor, numpy array, int or None."""
    if a is None:
        return None
    if isinstance(a, int):
        return a
    if isinstance(a, np.ndarray):
        return a.ctypes.data
    return a.data_ptr()


_raw_stream = None


def _current_stream(t) -> int:
    """The current stream of a tensor's device as an address (torch's raw lookup where it has one: 0.2 us against 1.8)."""
    global _raw_stream
    if _raw_stream is None:
        import torch
        _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
            (lambda i: torch.cuda.current_stream(i).cuda_stream)
    return _raw_stream(t.get_device())


def _stream(stream, *tensors):
    if stream is not None:
        return stream if isinstance(stream, int) else stream.cuda_stream
    for t in tensors:
        if getattr(t, "is_cuda", False):
            return _current_stream(t)
    return None


_names = {}


def _dtype_name(t) -> str:
    d = t.dtype
    name = _names.get(d)
    if name is None:
        name = _names[d] = str(d).replace("torch.", "")
    return name


# Tensor dtypes accepted for each activation / output dtype code (bf16 may
# also arrive as its 16-bit patterns).
_TORCH_OK = {0: ("float32",), 1: ("float16",), 2: ("bfloat16", "int16", "uint16")}
_ELEM = {0: 4, 1: 2, 2: 2}


def _check_dev(t, what: str, dtype_code: int | None, min_elems: int) -> None:
    """Refuse a device buffer the kernels could not use safely.

    The C ABI sees raw pointers only, so this is the one layer that can check
    a torch tensor before the kernels read or write through it: it must live
    on the GPU, be contiguous, have the element type of ``dtype_code`` (None:
    any) and hold at least ``min_elems`` elements of that type.  Integer
    addresses are passed through unchecked (the caller vouches for them)."""
    if t is None or isinstance(t, int):
        return
    if isinstance(t, np.ndarray):
        raise QmvError(-6, f"{what}: a host numpy array; device memory (a GPU tensor) is required")
    if not getattr(t, "is_cuda", False):
        raise QmvError(-6, f"{what}: tensor is not on a GPU")
    if not t.is_contiguous():
        raise QmvError(-6, f"{what}: tensor is not contiguous")
    if dtype_code is not None:
        name = _dtype_name(t)
        if name not in _TORCH_OK[dtype_code]:
            raise QmvError(-2, f"{what}: tensor dtype {name}, expected one of {_TORCH_OK[dtype_code]}")
        have = t.numel() * t.element_size() // _ELEM[dtype_code]
    else:
        have = t.numel() * t.element_size()
    if have < min_elems:
        raise QmvError(-5, f"{what}: holds {have} elements, needs {min_elems}")


def _fmt(fmt) -> int:
    return FMT[fmt] if isinstance(fmt, str) else int(fmt)


def _dtype(dt) -> int:
    if isinstance(dt, str):
        return DTYPE[dt]
    if isinstance(dt, int):
        return dt
    import torch
    return {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2}[dt]


# -- entry points -------------------------------------------------------------
def qmv_block_size(fmt) -> int:
    return lib().qmv_block_size(_fmt(fmt))


def qmv_packed_size(fmt, rows: int, cols: int) -> int:
    return lib().qmv_packed_size(_fmt(fmt), rows, cols)


def _pack_out(fmt, rows, cols):
    n = qmv_packed_size(fmt, rows, cols)
    if n == 0:
        raise QmvError(-3, f"bad shape {rows}x{cols} for {fmt}")
    return np.empty(n, np.uint8)


def _c(a, dtype):
    return np.ascontiguousarray(a, dtype=dtype)


def qmv_pack_q8_0(d_bits, q, rows: int, cols: int) -> np.ndarray:
    d, qq, out = _c(d_bits, np.uint16), _c(q, np.int8), _pack_out("q8_0", rows, cols)
    _check(lib().qmv_pack_q8_0(_ptr(d), _ptr(qq), rows, cols, _ptr(out), out.size))
    return out


def qmv_pack_q4_k(d_bits, dmin_bits, sc6, m6, q4, rows: int, cols: int) -> np.ndarray:
    d, dm = _c(d_bits, np.uint16), _c(dmin_bits, np.uint16)
    sc, m, q = _c(sc6, np.uint8), _c(m6, np.uint8), _c(q4, np.uint8)
    out = _pack_out("q4_k", rows, cols)
    _check(lib().qmv_pack_q4_k(_ptr(d), _ptr(dm), _ptr(sc), _ptr(m), _ptr(q), rows, cols,
                               _ptr(out), out.size))
    return out


def qmv_pack_q5_k(d_bits, dmin_bits, sc6, m6, q5, rows: int, cols: int) -> np.ndarray:
    d, dm = _c(d_bits, np.uint16), _c(dmin_bits, np.uint16)
    sc, m, q = _c(sc6, np.uint8), _c(m6, np.uint8), _c(q5, np.uint8)
    out = _pack_out("q5_k", rows, cols)
    _check(lib().qmv_pack_q5_k(_ptr(d), _ptr(dm), _ptr(sc), _ptr(m), _ptr(q), rows, cols,
                               _ptr(out), out.size))
    return out


def qmv_pack_q6_k(d_bits, sc8, q6, rows: int, cols: int) -> np.ndarray:
    d, sc, q = _c(d_bits, np.uint16), _c(sc8, np.int8), _c(q6, np.uint8)
    out = _pack_out("q6_k", rows, cols)
    _check(lib().qmv_pack_q6_k(_ptr(d), _ptr(sc), _ptr(q), rows, cols, _ptr(out), out.size))
    return out


def qmv_pack_int4_g128(s_bits, q, rows: int, cols: int) -> np.ndarray:
    s, qq, out = _c(s_bits, np.uint16), _c(q, np.int8), _pack_out("int4_g128", rows, cols)
    _check(lib().qmv_pack_int4_g128(_ptr(s), _ptr(qq), rows, cols, _ptr(out), out.size))
    return out


def pack_fields(fmt: str, fields: dict, rows: int, cols: int) -> np.ndarray:
    """Call the packer of `fmt` with the field arrays named as in synth/."""
    if fmt == "q8_0":
        return qmv_pack_q8_0(fields["d_bits"], fields["q"], rows, cols)
    if fmt == "q4_k":
        return qmv_pack_q4_k(fields["d_bits"], fields["dmin_bits"], fields["sc"], fields["m"],
                             fields["u"], rows, cols)
    if fmt == "q5_k":
        return qmv_pack_q5_k(fields["d_bits"], fields["dmin_bits"], fields["sc"], fields["m"],
                             fields["u"], rows, cols)
    if fmt == "q6_k":
        return qmv_pack_q6_k(fields["d_bits"], fields["sc"], fields["q"], rows, cols)
    if fmt == "int4_g128":
        return qmv_pack_int4_g128(fields["s_bits"], fields["q"], rows, cols)
    raise ValueError(fmt)


def qmv_create_weights(fmt, rows: int, cols: int, dev_packed, nbytes: int | None = None) -> QmvWeights:
    """Descriptor for packed bytes already in device memory (a uint8 tensor or a pointer)."""
    if nbytes is None:
        nbytes = dev_packed.numel() * dev_packed.element_size()
    _check_dev(dev_packed, "packed weights", None, nbytes)
    w = QmvWeights()
    _check(lib().qmv_create_weights(_fmt(fmt), rows, cols, _ptr(dev_packed), nbytes, ctypes.byref(w)))
    # The descriptor holds a raw pointer: keep the tensor alive with it, or the
    # caching allocator may hand its memory back to the driver (empty_cache(),
    # which graph capture calls) while launches still read it.
    w.owner = None if isinstance(dev_packed, int) else dev_packed
    return w


def qmv_planes_size(fmt, rows: int, cols: int) -> int:
    return lib().qmv_planes_size(_fmt(fmt), rows, cols)


def qmv_create_weights_planes(fmt, rows: int, cols: int, dev_planes, nbytes: int | None = None) -> QmvWeights:
    """Descriptor for plane-layout bytes already in device memory (a uint8 tensor or a pointer)."""
    if nbytes is None:
        nbytes = dev_planes.numel() * dev_planes.element_size()
    _check_dev(dev_planes, "plane weights", None, nbytes)
    w = QmvWeights()
    _check(lib().qmv_create_weights_planes(_fmt(fmt), rows, cols, _ptr(dev_planes), nbytes, ctypes.byref(w)))
    w.owner = None if isinstance(dev_planes, int) else dev_planes
    return w


def qmv_repack_planes(src: QmvWeights, dst, dst_bytes: int | None = None, stream=None) -> QmvWeights:
    """Enqueue the repack of canonical Q4_K blocks into the plane layout at dst
    (a uint8 device tensor or a pointer); returns the planes descriptor."""
    if dst_bytes is None:
        dst_bytes = dst.numel() * dst.element_size()
    _check_dev(dst, "dst", None, dst_bytes)
    w = QmvWeights()
    _check(lib().qmv_repack_planes(ctypes.byref(src), _ptr(dst), dst_bytes, ctypes.byref(w),
                                   _stream(stream, dst)))
    w.owner = None if isinstance(dst, int) else dst
    return w


def qmv_gemv(fmt, W: QmvWeights, x, x_dtype, y, rows: int, cols: int, batch: int,
             stream=None) -> None:
    xd = _dtype(x_dtype)
    _check_dev(x, "x", xd, batch * cols)
    _check_dev(y, "y", 0, batch * rows)
    _check(lib().qmv_gemv(_fmt(fmt), ctypes.byref(W), _ptr(x), _dtype(x_dtype), _ptr(y),
                          rows, cols, batch, _stream(stream, x, y)))


def qmv_gemv_noalloc(fmt, W: QmvWeights, x, x_dtype, y, rows: int, cols: int, batch: int,
                     stream=None) -> None:
    xd = _dtype(x_dtype)
    _check_dev(x, "x", xd, batch * cols)
    _check_dev(y, "y", 0, batch * rows)
    _check(lib().qmv_gemv_noalloc(_fmt(fmt), ctypes.byref(W), _ptr(x), _dtype(x_dtype), _ptr(y),
                                  rows, cols, batch, _stream(stream, x, y)))


def _items(x_dtype, batch: int, items, check: bool = True):
    arr = (QmvGemvItem * max(1, len(items)))()
    xd = _dtype(x_dtype)
    for i, (W, x, y) in enumerate(items):
        if check:
            _check_dev(x, f"item {i} x", xd, batch * W.cols)
            _check_dev(y, f"item {i} y", 0, batch * W.rows)
        arr[i].W = ctypes.pointer(W)
        arr[i].x = _ptr(x)
        arr[i].y = _ptr(y)
    return arr


def qmv_gemv_multi(fmt, x_dtype, batch: int, items, stream=None) -> None:
    """items: sequence of (QmvWeights, x, y) triples; one launch for all of them."""
    arr = _items(x_dtype, batch, items)
    tensors = [t for _, x, y in items for t in (x, y)]
    _check(lib().qmv_gemv_multi(_fmt(fmt), _dtype(x_dtype), batch, arr, len(items),
                                _stream(stream, *tensors)))


def qmv_workspace_size(fmt, x_dtype, batch: int, items) -> int:
    """Bytes of workspace qmv_gemv_multi_ws needs for these items (0: none)."""
    arr = _items(x_dtype, batch, items, check=False)
    n = _u64(0)
    _check(lib().qmv_workspace_size(_fmt(fmt), _dtype(x_dtype), batch, arr, len(items),
                                    ctypes.byref(n)))
    return int(n.value)


def qmv_gemv_multi_ws(fmt, x_dtype, batch: int, items, workspace, workspace_bytes: int,
                      stream=None) -> None:
    """qmv_gemv_multi with a caller-owned device workspace (None: no workspace)."""
    arr = _items(x_dtype, batch, items)
    tensors = [t for _, x, y in items for t in (x, y)]
    if workspace is not None:
        _check_dev(workspace, "workspace", None, workspace_bytes)
        tensors.append(workspace)
    _check(lib().qmv_gemv_multi_ws(_fmt(fmt), _dtype(x_dtype), batch, arr, len(items),
                                   _ptr(workspace) if workspace is not None else None,
                                   workspace_bytes, _stream(stream, *tensors)))


def qmv_gemv_swiglu(fmt, Wg: QmvWeights, Wu: QmvWeights, x, x_dtype, h, rows: int, cols: int, batch: int,
                    stream=None) -> None:
    """h = silu(Wg x) * (Wu x) in one launch (h: [batch][rows] fp32)."""
    xd = _dtype(x_dtype)
    _check_dev(x, "x", xd, batch * cols)
    _check_dev(h, "h", 0, batch * rows)
    _check(lib().qmv_gemv_swiglu(_fmt(fmt), ctypes.byref(Wg), ctypes.byref(Wu), _ptr(x), xd, _ptr(h),
                                 rows, cols, batch, _stream(stream, x, h)))


def qmv_dequant(W: QmvWeights, out, out_dtype, stream=None) -> None:
    od = _dtype(out_dtype)
    _check_dev(out, "out", od, W.rows * W.cols)
    _check(lib().qmv_dequant(ctypes.byref(W), _ptr(out), _dtype(out_dtype), _stream(stream, out)))


# Element types of the index, mask and number tensors of the step's operators.
_I32, _I64, _F32 = ("int32",), ("int64", "uint64"), ("float32",)


def _check_vec(t, what: str, names, n: int) -> None:
    """A contiguous device tensor of one of the named element types with at least n elements."""
    if t is None:
        raise QmvError(-1, f"{what} is None")
    _check_dev(t, what, None, 0)
    if isinstance(t, int):
        return
    name = _dtype_name(t)
    if name not in names:
        raise QmvError(-2, f"{what}: tensor dtype {name}, expected one of {names}")
    if t.numel() < n:
        raise QmvError(-5, f"{what}: holds {t.numel()} elements, needs {n}")


def _check_view(t, what: str, name: str, ndim: int) -> None:
    """A device tensor of any strides whose last dimension is contiguous."""
    if t is None:
        raise QmvError(-1, f"{what} is None")
    if not getattr(t, "is_cuda", False):
        raise QmvError(-6, f"{what}: tensor is not on a GPU")
    if _dtype_name(t) != name:
        raise QmvError(-2, f"{what}: tensor dtype {t.dtype}, expected {name}")
    if t.dim() != ndim:
        raise QmvError(-3, f"{what}: {t.dim()} dimensions, expected {ndim}")
    if t.shape[-1] > 1 and t.stride(-1) != 1:
        raise QmvError(-6, f"{what}: the last dimension is not contiguous")


def _strides(t) -> list:
    """Strides with zero for dimensions of one element, whose stride says nothing."""
    return [t.stride(i) if t.shape[i] > 1 else 0 for i in range(t.dim() - 1)]


def _check_one_device(pairs) -> None:
    devices = {str(t.device) for _, t in pairs if t is not None and hasattr(t, "device")}
    if len(devices) > 1:
        raise QmvError(-6, f"{', '.join(n for n, t in pairs if t is not None)}: tensors on {sorted(devices)}")


def _check_with(what: str, t, name: str, u) -> None:
    """t on the device of u (integer addresses pass)."""
    if hasattr(t, "device") and hasattr(u, "device") and t.device != u.device:
        raise QmvError(-6, f"{what} on {t.device}, {name} on {u.device}")


def qmv_embed(W: QmvWeights, ids, n: int, out, out_dtype, scale: float = 1.0, stream=None) -> None:
    """out[i] = scale * W[ids[i]] for n int32 device ids; ids outside the table give rows of zeros."""
    od = _dtype(out_dtype)
    if n > 0:
        _check_vec(ids, "ids", _I32, n)
        _check_dev(out, "out", od, n * W.cols)
        _check_with("ids", ids, "out", out)
    _check(lib().qmv_embed(ctypes.byref(W), _ptr(ids), n, scale, _ptr(out), od, _stream(stream, out)))


def qmv_create_attn(q, out, row_start, max_rows: int, *, scale: float, k_prefix=None, v_prefix=None,
                    prefix_pages=None, prefix_len: int | None = None, k_pages=None, v_pages=None, block_table=None,
                    suffix_len=None, max_suffix: int = 0, tree_mask=None, lse=None) -> QmvAttnArgs:
    """Checked arguments of qmv_attn from device tensors, kept alive with them.

    q, out [rows, heads, D]; the prefix as k_prefix, v_prefix [tokens, kv_heads, D], or as prefix_pages (int32 page
    numbers) with prefix_len; k_pages, v_pages [pages, page_size, kv_heads, D]; block_table [nseq, entries] int32;
    row_start [nseq + 1], suffix_len [nseq] int32; tree_mask [rows] int64 bits; lse [rows, heads] float32.  Any
    strides with contiguous last dimensions (k and v of a pair alike)."""
    a = QmvAttnArgs()
    if getattr(q, "dtype", None) is None or str(q.dtype) not in ("torch.float16", "torch.bfloat16"):
        raise QmvError(-6, f"q: {getattr(q, 'dtype', type(q))}, expected a float16 or bfloat16 tensor")
    name = str(q.dtype).replace("torch.", "")
    _check_view(q, "q", name, 3)
    _check_view(out, "out", name, 3)
    rows, heads, d = (int(x) for x in q.shape)
    if tuple(out.shape) != (rows, heads, d):
        raise QmvError(-3, f"out: shape {tuple(out.shape)}, expected {(rows, heads, d)}")
    _check_vec(row_start, "row_start", _I32, 1)
    nseq = int(row_start.numel()) - 1
    a.dtype, a.rows, a.heads, a.head_dim = _dtype(q.dtype), rows, heads, d
    a.nseq, a.max_rows, a.max_suffix, a.scale = nseq, max_rows, max_suffix, scale
    (a.q_row, a.q_head), (a.out_row, a.out_head) = _strides(q), _strides(out)
    a.page_size, kv_heads = 1, None
    if prefix_pages is None:
        a.prefix_len = 0 if k_prefix is None else int(k_prefix.shape[0])
        if prefix_len is not None and prefix_len > a.prefix_len:
            raise QmvError(-5, f"k_prefix holds {a.prefix_len} tokens, prefix_len {prefix_len}")
        a.prefix_len = a.prefix_len if prefix_len is None else prefix_len
    else:
        if prefix_len is None:
            raise QmvError(-3, "prefix_pages without prefix_len")
        if k_prefix is not None or v_prefix is not None:
            raise QmvError(-3, "both prefix_pages and k_prefix or v_prefix")
        a.prefix_len = prefix_len
    pairs = [("k_prefix", "v_prefix", k_prefix, v_prefix, 3)] if k_prefix is not None or v_prefix is not None else []
    if k_pages is not None or v_pages is not None:
        pairs.append(("k_pages", "v_pages", k_pages, v_pages, 4))
    for kn, vn, k, v, nd in pairs:
        _check_view(k, kn, name, nd)
        _check_view(v, vn, name, nd)
        if k.shape != v.shape or _strides(k) != _strides(v):
            raise QmvError(-3, f"{kn} and {vn} differ in shape or strides")
        if k.shape[-1] != d:
            raise QmvError(-3, f"{kn}: head width {k.shape[-1]}, expected {d}")
        if kv_heads not in (None, int(k.shape[-2])):
            raise QmvError(-3, f"{kn}: {k.shape[-2]} heads, expected {kv_heads}")
        kv_heads = int(k.shape[-2])
    a.kv_heads = heads if kv_heads is None else kv_heads
    if k_prefix is not None:
        a.prefix_row, a.prefix_head = _strides(k_prefix)
    if k_pages is not None:
        a.num_pages, a.page_size = int(k_pages.shape[0]), int(k_pages.shape[1])
        a.page_stride, a.page_row, a.page_head = _strides(k_pages)
    elif prefix_pages is not None or max_suffix > 0:
        raise QmvError(-1, "k_pages is None")
    if prefix_pages is not None:
        _check_vec(prefix_pages, "prefix_pages", _I32, -(-prefix_len // max(1, a.page_size)))
    if max_suffix > 0:
        _check_view(block_table, "block_table", "int32", 2)
        if block_table.shape[0] < nseq:
            raise QmvError(-5, f"block_table: {block_table.shape[0]} rows, needs {nseq}")
        if block_table.shape[1] * a.page_size < max_suffix:
            raise QmvError(-5, f"block_table: {block_table.shape[1]} pages of {a.page_size} hold fewer than "
                               f"{max_suffix} tokens")
        # (one row of any stride; the library asks for a stride that covers max_suffix)
        a.table_stride = block_table.stride(0) if block_table.shape[0] > 1 else block_table.shape[1]
        _check_vec(suffix_len, "suffix_len", _I32, nseq)
    if tree_mask is not None:
        _check_vec(tree_mask, "tree_mask", _I64, rows)
    if lse is not None:
        _check_vec(lse, "lse", _F32, rows * heads)
    named = dict(q=q, k_prefix=k_prefix, v_prefix=v_prefix, prefix_pages=prefix_pages, k_pages=k_pages,
                 v_pages=v_pages, block_table=block_table, row_start=row_start, suffix_len=suffix_len,
                 tree_mask=tree_mask, out=out, lse=lse)
    _check_one_device(list(named.items()))
    for field, t in named.items():
        setattr(a, field, _ptr(t))
    a.owner = named
    _check(lib().qmv_attn_workspace_size(ctypes.byref(a), ctypes.byref(_u64(0))))
    return a


def qmv_attn_workspace_size(a: QmvAttnArgs) -> int:
    n = _u64(0)
    _check(lib().qmv_attn_workspace_size(ctypes.byref(a), ctypes.byref(n)))
    return int(n.value)


def qmv_attn(a: QmvAttnArgs, workspace, workspace_bytes: int, stream=None) -> None:
    """Attention of the step's rows (qmv_create_attn) over the shared prefix and their sequences' suffixes."""
    owner = getattr(a, "owner", None)
    q = owner["q"] if owner else None
    if workspace is not None:
        _check_dev(workspace, "workspace", None, workspace_bytes)
        _check_with("workspace", workspace, "q", q)
    _check(lib().qmv_attn(ctypes.byref(a), _ptr(workspace), workspace_bytes, _stream(stream, q, workspace)))


def qmv_create_verify(logits, tokens, row_start, max_rows: int, u_accept, u_sample, out_tokens, accepted, *,
                      draft_probs=None, temperature=None) -> QmvVerifyArgs:
    """Checked arguments of qmv_verify from device tensors, kept alive with them.

    logits [rows, vocab] float32, float16 or bfloat16, draft_probs [rows, vocab] float32 (rows of any stride);
    tokens, out_tokens [rows], row_start [nseq + 1], accepted [nseq] int32; u_accept [rows], u_sample and
    temperature [nseq] float32."""
    a = QmvVerifyArgs()
    name = str(getattr(logits, "dtype", "")).replace("torch.", "")
    if name not in ("float32", "float16", "bfloat16"):
        raise QmvError(-6, f"logits: {name or type(logits)}, expected a float32, float16 or bfloat16 tensor")
    _check_view(logits, "logits", name, 2)
    rows, vocab = (int(x) for x in logits.shape)
    _check_vec(row_start, "row_start", _I32, 1)
    nseq = int(row_start.numel()) - 1
    if draft_probs is not None:
        _check_view(draft_probs, "draft_probs", "float32", 2)
        if tuple(draft_probs.shape) != (rows, vocab):
            raise QmvError(-3, f"draft_probs: shape {tuple(draft_probs.shape)}, expected {(rows, vocab)}")
        a.draft_row = draft_probs.stride(0) if rows > 1 else vocab
    for what, t, kind, n in [("tokens", tokens, _I32, rows), ("u_accept", u_accept, _F32, rows),
                             ("u_sample", u_sample, _F32, nseq), ("out_tokens", out_tokens, _I32, rows),
                             ("accepted", accepted, _I32, nseq)]:
        _check_vec(t, what, kind, n)
    if temperature is not None:
        _check_vec(temperature, "temperature", _F32, nseq)
    a.logits_dtype, a.nseq, a.max_rows, a.rows, a.vocab = _dtype(logits.dtype), nseq, max_rows, rows, vocab
    a.logits_row = logits.stride(0) if rows > 1 else vocab
    named = dict(logits=logits, draft_probs=draft_probs, tokens=tokens, row_start=row_start, temperature=temperature,
                 u_accept=u_accept, u_sample=u_sample, out_tokens=out_tokens, accepted=accepted)
    _check_one_device(list(named.items()))
    for field, t in named.items():
        setattr(a, field, _ptr(t))
    a.owner = named
    _check(lib().qmv_verify_workspace_size(ctypes.byref(a), ctypes.byref(_u64(0))))
    return a


def qmv_verify_workspace_size(a: QmvVerifyArgs) -> int:
    n = _u64(0)
    _check(lib().qmv_verify_workspace_size(ctypes.byref(a), ctypes.byref(n)))
    return int(n.value)


def qmv_verify(a: QmvVerifyArgs, workspace, workspace_bytes: int, stream=None) -> None:
    """Drafted tokens checked against the target's probabilities (qmv_create_verify)."""
    owner = getattr(a, "owner", None)
    logits = owner["logits"] if owner else None
    if workspace is not None:
        _check_dev(workspace, "workspace", None, workspace_bytes)
        _check_with("workspace", workspace, "logits", logits)
    _check(lib().qmv_verify(ctypes.byref(a), _ptr(workspace), workspace_bytes, _stream(stream, logits, workspace)))


def qmv_probe_read_outputs(nbytes: int) -> int:
    return lib().qmv_probe_read_outputs(nbytes)


def qmv_probe_read(src, nbytes: int, out, stream=None) -> None:
    _check_dev(src, "src", None, nbytes)
    _check_dev(out, "out", 0, qmv_probe_read_outputs(nbytes))
    _check(lib().qmv_probe_read(_ptr(src), nbytes, _ptr(out), _stream(stream, src, out)))


def qmv_probe_copy(src, dst, nbytes: int, stream=None) -> None:
    _check_dev(src, "src", None, nbytes)
    _check_dev(dst, "dst", None, nbytes)
    _check(lib().qmv_probe_copy(_ptr(src), _ptr(dst), nbytes, _stream(stream, src, dst)))


def qmv_status_string(status: int) -> str:
    return lib().qmv_status_string(status).decode()


def qmv_last_error() -> str:
    return (lib().qmv_last_error() or b"").decode()
