"""Python binding of libqbd: argument marshalling only.

Each function takes torch tensors on one gfx950 device, checks dtypes,
shapes, contiguity and that all tensors share that device, allocates the
output with torch when none is given, and calls the C entry point of the
same name with that device current, on torch's current stream for it.  Every
step of the computation runs in the library's HIP kernels; there is no
fallback of any kind, and a missing library is an error.
"""

import ctypes
import functools
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libqbd.so")
HEADER_PATH = os.path.join(os.path.dirname(_HERE), "include", "qbd.h")

_P = ctypes.c_void_p
_I64 = ctypes.c_int64

# C signatures, mirrored from include/qbd.h
SIGNATURES = {
    "qbd_status_str": ([ctypes.c_int], ctypes.c_char_p),
    "qbd_abi_version": ([], ctypes.c_int),
    "qmv_q8_0_f32": ([_P, _P, _P, _P, _I64, _I64, _I64, _P], ctypes.c_int),
    "quantize_act_q8_0": ([_P, _P, _P, _I64, _I64, _P], ctypes.c_int),
    "qmm_q8_0_q8act": ([_P, _P, _P, _P, _P, _I64, _I64, _I64, _P], ctypes.c_int),
    "gate_up_swiglu_q4": ([_P, _P, _P, _P, _P, _P, _I64, _I64, _I64, _P], ctypes.c_int),
    "gate_up_swiglu_q8_0": ([_P, _P, _P, _P, _P, _P, _I64, _I64, _I64, _P], ctypes.c_int),
    "qmv_q4_0_f32": ([_P, _P, _P, _P, _I64, _I64, _I64, _P], ctypes.c_int),
    "qmm_q4_0_q8act": ([_P, _P, _P, _P, _P, _I64, _I64, _I64, _P], ctypes.c_int),
    "gate_up_swiglu_q4_q8act": ([_P, _P, _P, _P, _P, _P, _P, _I64, _I64, _I64, _P], ctypes.c_int),
    "qmm_q8_0_q8act_from_f32": ([_P, _P, _P, _P, _P, _P, _I64, _I64, _I64, _P], ctypes.c_int),
    "qmm_q4_0_q8act_from_f32": ([_P, _P, _P, _P, _P, _P, _I64, _I64, _I64, _P], ctypes.c_int),
    "gate_up_swiglu_q4_q8act_from_f32": ([_P, _P, _P, _P, _P, _P, _P, _P, _I64, _I64, _I64, _P], ctypes.c_int),
    "swiglu_f32": ([_P, _P, _P, _I64, _P], ctypes.c_int),
    "q8_0_split_blocks": ([_P, _P, _P, _I64, _I64], ctypes.c_int),
    "q4_0_split_blocks": ([_P, _P, _P, _I64, _I64], ctypes.c_int),
    "kv_cache_write": ([_P, _P, _P, ctypes.c_int, _I64, _I64, _I64, _I64, _P, _I64, _P], ctypes.c_int),
    "kv_cache_read": ([_P, _P, _I64, ctypes.c_int, _P, _P, _P], ctypes.c_int),
    "kv_attention_work_bytes": ([_P, _I64, _I64, _I64, _I64, _I64], _I64),
    "kv_attention": ([_P, _P, ctypes.c_int, _I64, _I64, _P, _I64, _P, _P, _I64, _I64, _I64, _I64, _I64,
                      ctypes.c_int, _I64, ctypes.c_float, _P, _P, _I64, _P], ctypes.c_int),
}


class KvCacheDesc(ctypes.Structure):
    """qbd_kv_cache of include/qbd.h."""
    _fields_ = [("kc", _P), ("kd", _P), ("vc", _P), ("vd", _P), ("pages", _I64), ("heads", _I64),
                ("page", _I64), ("dim", _I64), ("kbits", ctypes.c_int32), ("vbits", ctypes.c_int32)]

_lib = None


class QbdError(RuntimeError):
    """A libqbd entry point returned a non-zero status."""

    def __init__(self, name, status, text):
        super().__init__(f"{name}: {text} (status {status})")
        self.status = status


def lib():
    """Load libqbd.so once (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(
                f"{LIB_PATH} is missing: build it with `python -m block_quantized_decode_amd.build`")
        handle = ctypes.CDLL(LIB_PATH)
        for name, (args, res) in SIGNATURES.items():
            fn = getattr(handle, name)
            fn.argtypes = args
            fn.restype = res
        _lib = handle
    return _lib


def status_str(status):
    return lib().qbd_status_str(int(status)).decode()


def _call(name, *args):
    st = getattr(_lib or lib(), name)(*args)
    if st != 0:
        raise QbdError(name, st, status_str(st))


def _launch(name, tensors, *args):
    """Call entry point `name` with the tensors' device current (the library
    checks and launches on the current device); every tensor must be on it."""
    index = tensors[0].get_device()
    for t in tensors[1:]:
        if t.get_device() != index:
            raise ValueError(f"{name}: tensors on {tensors[0].device} and {t.device}")
    if index == torch.cuda.current_device():
        _call(name, *args, _stream(index))
        return
    with torch.cuda.device(index):
        _call(name, *args, _stream(index))


def _ptr(t):
    return t.data_ptr() if t is not None else 0  # ctypes makes it a void*


# the current stream's handle of a device index, without a Stream object where torch can tell it so
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(index):
    if _raw_stream is not None:
        return _raw_stream(index)
    return torch.cuda.current_stream(index).cuda_stream


def _need(t, name, dtypes, ndim):
    if type(t) is torch.Tensor and t.dtype in dtypes and t.ndim == ndim and t.is_cuda and t.is_contiguous():
        return
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype not in dtypes:
        raise TypeError(f"{name}: dtype {t.dtype}, expected one of {dtypes}")
    if t.dim() != ndim:
        raise ValueError(f"{name}: expected {ndim} dims, got shape {tuple(t.shape)}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be on a GPU device")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


_I8 = (torch.int8,)
_U8 = (torch.uint8,)
_F32 = (torch.float32,)
_SCALE = (torch.uint16, torch.int16)  # binary16 bit patterns


def _out(out, shape, dtype, like, name="out"):
    if out is None:
        return torch.empty(shape, dtype=dtype, device=like.device)
    _need(out, name, (dtype,), len(shape))
    if tuple(out.shape) != tuple(shape):
        raise ValueError(f"{name}: shape {tuple(out.shape)}, expected {tuple(shape)}")
    return out


def _weights(wq, wd, q4):
    _need(wq, "weight codes", _U8 if q4 else _I8, 2)
    _need(wd, "weight scales", _SCALE, 2)
    n = wq.shape[0]
    k = wq.shape[1] * (2 if q4 else 1)
    if tuple(wd.shape) != (n, k // 32) or k % 32:
        raise ValueError(f"weight planes {tuple(wq.shape)} / {tuple(wd.shape)} do not form [N][K]")
    return n, k


def qmv_q8_0_f32(wq, wd, x, out=None):
    """y[M][N] = x . W^T for Q8_0 weights (wq int8 [N][K], wd [N][K/32]) and fp32 x [M][K]."""
    n, k = _weights(wq, wd, False)
    _need(x, "x", _F32, 2)
    m = x.shape[0]
    if x.shape[1] != k:
        raise ValueError("x width differs from K")
    y = _out(out, (m, n), torch.float32, x)
    _launch("qmv_q8_0_f32", (x, wq, wd, y), _ptr(wq), _ptr(wd), _ptr(x), _ptr(y), m, n, k)
    return y


def qmv_q4_0_f32(wq4, wd, x, out=None):
    """y[M][N] = x . W^T for Q4 weights (wq4 uint8 [N][K/2], wd [N][K/32]) and fp32 x."""
    n, k = _weights(wq4, wd, True)
    _need(x, "x", _F32, 2)
    m = x.shape[0]
    if x.shape[1] != k:
        raise ValueError("x width differs from K")
    y = _out(out, (m, n), torch.float32, x)
    _launch("qmv_q4_0_f32", (x, wq4, wd, y), _ptr(wq4), _ptr(wd), _ptr(x), _ptr(y), m, n, k)
    return y


def gate_up_swiglu_q4(gq, gd, uq, ud, x, out=None):
    """out = silu(x . Wg^T) * (x . Wu^T), Q4 gate/up weights, fp32 x, one launch."""
    n, k = _weights(gq, gd, True)
    n2, k2 = _weights(uq, ud, True)
    if (n, k) != (n2, k2):
        raise ValueError("gate and up weights differ in shape")
    _need(x, "x", _F32, 2)
    m = x.shape[0]
    if x.shape[1] != k:
        raise ValueError("x width differs from K")
    o = _out(out, (m, n), torch.float32, x)
    _launch("gate_up_swiglu_q4", (x, gq, gd, uq, ud, o), _ptr(gq), _ptr(gd), _ptr(uq), _ptr(ud),
            _ptr(x), _ptr(o), m, n, k)
    return o


def gate_up_swiglu_q8_0(gq, gd, uq, ud, x, out=None):
    """out = silu(x . Wg^T) * (x . Wu^T), Q8_0 gate/up weights, fp32 x, one launch."""
    n, k = _weights(gq, gd, False)
    n2, k2 = _weights(uq, ud, False)
    if (n, k) != (n2, k2):
        raise ValueError("gate and up weights differ in shape")
    _need(x, "x", _F32, 2)
    m = x.shape[0]
    if x.shape[1] != k:
        raise ValueError("x width differs from K")
    o = _out(out, (m, n), torch.float32, x)
    _launch("gate_up_swiglu_q8_0", (x, gq, gd, uq, ud, o), _ptr(gq), _ptr(gd), _ptr(uq), _ptr(ud),
            _ptr(x), _ptr(o), m, n, k)
    return o


def quantize_act_q8_0(x, xq=None, xd=None):
    """Per-32-block Q8 quantization of fp32 x [M][K] -> (xq int8 [M][K], xd fp32 [M][K/32])."""
    _need(x, "x", _F32, 2)
    m, k = x.shape
    if k % 32:
        raise ValueError("K must be a multiple of 32")
    q = _out(xq, (m, k), torch.int8, x, "xq")
    d = _out(xd, (m, k // 32), torch.float32, x, "xd")
    _launch("quantize_act_q8_0", (x, q, d), _ptr(x), _ptr(q), _ptr(d), m, k)
    return q, d


def _act_q8(xq, xd, k):
    _need(xq, "xq", _I8, 2)
    _need(xd, "xd", _F32, 2)
    m = xq.shape[0]
    if xq.shape[1] != k or tuple(xd.shape) != (m, k // 32):
        raise ValueError("activation planes do not match K")
    return m


def qmm_q8_0_q8act(wq, wd, xq, xd, out=None):
    """y = sum_b d_w d_x dot_b for Q8_0 weights and Q8 activations (xq, xd)."""
    n, k = _weights(wq, wd, False)
    m = _act_q8(xq, xd, k)
    y = _out(out, (m, n), torch.float32, xq)
    _launch("qmm_q8_0_q8act", (xq, xd, wq, wd, y), _ptr(wq), _ptr(wd), _ptr(xq), _ptr(xd), _ptr(y),
            m, n, k)
    return y


def qmm_q4_0_q8act(wq4, wd, xq, xd, out=None):
    """y = sum_b d_w d_x dot_b for Q4 weights and Q8 activations (xq, xd)."""
    n, k = _weights(wq4, wd, True)
    m = _act_q8(xq, xd, k)
    y = _out(out, (m, n), torch.float32, xq)
    _launch("qmm_q4_0_q8act", (xq, xd, wq4, wd, y), _ptr(wq4), _ptr(wd), _ptr(xq), _ptr(xd), _ptr(y),
            m, n, k)
    return y


def gate_up_swiglu_q4_q8act(gq, gd, uq, ud, xq, xd, out=None):
    """out = silu(g) * u with g, u the Q4 x Q8-activation products, one launch."""
    n, k = _weights(gq, gd, True)
    n2, k2 = _weights(uq, ud, True)
    if (n, k) != (n2, k2):
        raise ValueError("gate and up weights differ in shape")
    m = _act_q8(xq, xd, k)
    o = _out(out, (m, n), torch.float32, xq)
    _launch("gate_up_swiglu_q4_q8act", (xq, xd, gq, gd, uq, ud, o), _ptr(gq), _ptr(gd), _ptr(uq),
            _ptr(ud), _ptr(xq), _ptr(xd), _ptr(o), m, n, k)
    return o


def _x_panel(x, k, xq, xd):
    _need(x, "x", _F32, 2)
    m = x.shape[0]
    if x.shape[1] != k:
        raise ValueError("x width differs from K")
    return m, _out(xq, (m, k), torch.int8, x, "xq"), _out(xd, (m, k // 32), torch.float32, x, "xd")


def qmm_q8_0_q8act_from_f32(wq, wd, x, xq=None, xd=None, out=None):
    """quantize_act_q8_0(x) then qmm_q8_0_q8act in one call -> (y, xq, xd)."""
    n, k = _weights(wq, wd, False)
    m, q, d = _x_panel(x, k, xq, xd)
    y = _out(out, (m, n), torch.float32, x)
    _launch("qmm_q8_0_q8act_from_f32", (x, q, d, wq, wd, y), _ptr(wq), _ptr(wd), _ptr(x), _ptr(q), _ptr(d),
            _ptr(y), m, n, k)
    return y, q, d


def qmm_q4_0_q8act_from_f32(wq4, wd, x, xq=None, xd=None, out=None):
    """quantize_act_q8_0(x) then qmm_q4_0_q8act in one call -> (y, xq, xd)."""
    n, k = _weights(wq4, wd, True)
    m, q, d = _x_panel(x, k, xq, xd)
    y = _out(out, (m, n), torch.float32, x)
    _launch("qmm_q4_0_q8act_from_f32", (x, q, d, wq4, wd, y), _ptr(wq4), _ptr(wd), _ptr(x), _ptr(q), _ptr(d),
            _ptr(y), m, n, k)
    return y, q, d


def gate_up_swiglu_q4_q8act_from_f32(gq, gd, uq, ud, x, xq=None, xd=None, out=None):
    """quantize_act_q8_0(x) then gate_up_swiglu_q4_q8act in one call -> (out, xq, xd)."""
    n, k = _weights(gq, gd, True)
    n2, k2 = _weights(uq, ud, True)
    if (n, k) != (n2, k2):
        raise ValueError("gate and up weights differ in shape")
    m, q, d = _x_panel(x, k, xq, xd)
    o = _out(out, (m, n), torch.float32, x)
    _launch("gate_up_swiglu_q4_q8act_from_f32", (x, q, d, gq, gd, uq, ud, o), _ptr(gq), _ptr(gd), _ptr(uq),
            _ptr(ud), _ptr(x), _ptr(q), _ptr(d), _ptr(o), m, n, k)
    return o, q, d


def swiglu_f32(g, u, out=None):
    """out = silu(g) * u elementwise (fp32, same shape)."""
    if not isinstance(g, torch.Tensor) or not isinstance(u, torch.Tensor):
        raise TypeError("g and u must be tensors")
    if g.shape != u.shape or g.dtype != torch.float32 or u.dtype != torch.float32:
        raise ValueError("g and u must be fp32 tensors of one shape")
    if not (g.is_cuda and u.is_cuda and g.is_contiguous() and u.is_contiguous()):
        raise ValueError("g and u must be contiguous GPU tensors")
    o = torch.empty_like(g) if out is None else out
    if o.shape != g.shape or o.dtype != torch.float32 or not o.is_contiguous():
        raise ValueError("out must be a contiguous fp32 tensor shaped like g")
    _launch("swiglu_f32", (g, u, o), _ptr(g), _ptr(u), _ptr(o), g.numel())
    return o


_ELEM = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}
_I32 = (torch.int32,)
_I64T = (torch.int64,)
_CODES = {torch.uint8: 4, torch.int8: 8}


def kv_cache_alloc(pages, heads, page, dim, kbits=4, vbits=4, device="cuda"):
    """Zeroed planes (kc, kd, vc, vd) of a quantized key/value cache: codes [pages][heads][page][dim/2] uint8
    for 4 bits or [..][dim] int8 for 8, scales [..][dim/32] uint16."""
    def codes(bits):
        if bits not in (4, 8):
            raise ValueError("kbits and vbits are 4 or 8")
        return torch.zeros((pages, heads, page, dim * bits // 8), dtype=torch.uint8 if bits == 4 else torch.int8,
                           device=device)

    def scales():
        return torch.zeros((pages, heads, page, dim // 32), dtype=torch.int16, device=device).view(torch.uint16)
    return codes(kbits), scales(), codes(vbits), scales()


def _kv(kc, kd, vc, vd):
    """The descriptor of a cache from its planes."""
    _need(kc, "kc", _CODES, 4)
    _need(kd, "kd", _SCALE, 4)
    _need(vc, "vc", _CODES, 4)
    _need(vd, "vd", _SCALE, 4)
    pages, heads, page, nb = kd.shape
    kbits, vbits = _CODES[kc.dtype], _CODES[vc.dtype]
    if vd.shape != kd.shape or kc.shape != (pages, heads, page, 4 * nb * kbits) or vc.shape != (pages, heads, page, 4 * nb * vbits):
        raise ValueError(f"cache planes {tuple(kc.shape)} / {tuple(kd.shape)} / {tuple(vc.shape)} / {tuple(vd.shape)} "
                         "do not form [pages][heads][page][dim]")
    return KvCacheDesc(kc.data_ptr(), kd.data_ptr(), vc.data_ptr(), vd.data_ptr(), pages, heads, page, 32 * nb,
                       kbits, vbits)


def _rows(t, name, heads, dim):
    """Strides of the rows [T][heads][dim]: the elements of a row contiguous.  A stride that no index uses may hold
    anything."""
    if type(t) is torch.Tensor and t.dtype in _ELEM and t.is_cuda and t.ndim == 3:
        tokens, h, d = t.shape
        token_stride, head_stride, step = t.stride()
        if h == heads and d == dim and step == 1:
            return (token_stride if tokens > 1 else 0), (head_stride if heads > 1 else 0)
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype not in _ELEM:
        raise TypeError(f"{name}: dtype {t.dtype}, expected one of {tuple(_ELEM)}")
    if t.dim() != 3 or t.shape[1] != heads or t.shape[2] != dim:
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected [T][{heads}][{dim}]")
    if not t.is_cuda:
        raise ValueError(f"{name} must be on a GPU device")
    if t.stride(2) != 1:
        raise ValueError(f"{name}: the elements of a row must be contiguous")
    return (t.stride(0) if t.shape[0] > 1 else 0), (t.stride(1) if heads > 1 else 0)  # a Tensor subclass


@functools.lru_cache(maxsize=4096)
def _work_bytes(heads, page, dim, kbits, vbits, batch, tokens, qheads, max_q, max_len):
    """kv_attention_work_bytes: a function of sizes alone."""
    c = KvCacheDesc(None, None, None, None, 0, heads, page, dim, kbits, vbits)
    return lib().kv_attention_work_bytes(ctypes.byref(c), batch, tokens, qheads, max_q, max_len)


def kv_cache_write(k, v, kc, kd, vc, vd, slots):
    """Quantize the rows k, v [T][heads][dim] (f32, bf16 or f16, strided) into the cache planes at slots int64 [T]
    (page number * page + offset; a slot outside the cache is skipped)."""
    c = _kv(kc, kd, vc, vd)
    ks, vs = _rows(k, "k", c.heads, c.dim), _rows(v, "v", c.heads, c.dim)
    _need(slots, "slots", _I64T, 1)
    if k.dtype != v.dtype or k.shape[0] != v.shape[0] or slots.shape[0] != k.shape[0]:
        raise ValueError("k, v and slots differ in dtype or length")
    _launch("kv_cache_write", (k, v, kc, kd, vc, vd, slots), ctypes.byref(c), _ptr(k), _ptr(v), _ELEM[k.dtype], *ks,
            *vs, _ptr(slots), k.shape[0])


def kv_cache_read(kc, kd, vc, vd, slots, dtype=torch.float32, k=None, v=None):
    """The rows (k, v) [T][heads][dim] that slots int64 [T] of the cache hold; zeros for a slot outside it."""
    c = _kv(kc, kd, vc, vd)
    _need(slots, "slots", _I64T, 1)
    if dtype not in _ELEM:
        raise TypeError(f"dtype {dtype}, expected one of {tuple(_ELEM)}")
    shape = (slots.shape[0], c.heads, c.dim)
    k, v = _out(k, shape, dtype, kc, "k"), _out(v, shape, dtype, kc, "v")
    _launch("kv_cache_read", (kc, kd, vc, vd, slots, k, v), ctypes.byref(c), _ptr(slots), slots.shape[0],
            _ELEM[dtype], _ptr(k), _ptr(v))
    return k, v


def kv_attention(q, kc, kd, vc, vd, table, lens, q_starts=None, max_q=None, max_len=None, causal=True, window=0,
                 scale=None, out=None, work=None):
    """Attention of the query rows q [T][qheads][dim] over the cached sequences: table int32 [batch][width] of page
    numbers, lens int32 [batch] (the new tokens among them), q_starts int32 [batch + 1] (None: T / batch rows each; rows
    that it gives to no sequence are not written: pass out where they are to hold something).
    max_q and max_len bound a sequence's rows and length, if known on the host: they shape the launch.  scale is
    1 / sqrt(dim) by default.  work: a uint8 scratch tensor (allocated when None)."""
    c = _kv(kc, kd, vc, vd)
    if not isinstance(q, torch.Tensor) or q.dim() != 3:
        raise ValueError("q must be a tensor [T][qheads][dim]")
    tokens, qheads = q.shape[0], q.shape[1]
    qs = _rows(q, "q", qheads, c.dim)
    if qheads == 0 or qheads % c.heads:
        raise ValueError(f"{qheads} query heads over {c.heads} cached heads")
    _need(table, "table", _I32, 2)
    _need(lens, "lens", _I32, 1)
    batch, width = table.shape
    if lens.shape[0] != batch:
        raise ValueError("table and lens differ in batch")
    used = (q, kc, kd, vc, vd, table, lens)
    if q_starts is not None:
        _need(q_starts, "q_starts", _I32, 1)
        if q_starts.shape[0] != batch + 1:
            raise ValueError("q_starts must have batch + 1 entries")
        used += (q_starts,)
    elif batch == 0 or tokens % batch:
        raise ValueError(f"{tokens} query rows over {batch} sequences: pass q_starts")
    o = _out(out, (tokens, qheads, c.dim), q.dtype, q)
    max_q, max_len = max_q or (0 if q_starts is not None else tokens // batch), max_len or 0
    if work is None:
        need = _work_bytes(c.heads, c.page, c.dim, c.kbits, c.vbits, batch, tokens, qheads, max_q, max_len)
        if need:
            work = torch.empty((need,), dtype=torch.uint8, device=q.device)
            used += (work,)
    else:
        _need(work, "work", _U8, 1)
        used += (work,)
    _launch("kv_attention", (*used, o), ctypes.byref(c), q.data_ptr(), _ELEM[q.dtype], *qs, table.data_ptr(), width,
            lens.data_ptr(), _ptr(q_starts), batch, tokens, qheads, max_q, max_len, 1 if causal else 0, window,
            c.dim ** -0.5 if scale is None else scale, o.data_ptr(), _ptr(work), 0 if work is None else work.shape[0])
    return o


def q8_0_split_blocks(blocks34, n, k):
    """Host helper: interleaved 34-byte Q8_0 blocks (bytes) -> (wq, wd) numpy planes."""
    import numpy as np
    src = np.ascontiguousarray(np.frombuffer(blocks34, dtype=np.uint8))
    wq = np.empty((n, k), dtype=np.int8)
    wd = np.empty((n, k // 32), dtype=np.uint16)
    if src.size != n * (k // 32) * 34:
        raise ValueError("blocks34 size does not match N, K")
    _call("q8_0_split_blocks", src.ctypes.data_as(_P), wq.ctypes.data_as(_P),
          wd.ctypes.data_as(_P), n, k)
    return wq, wd


def q4_0_split_blocks(blocks18, n, k):
    """Host helper: interleaved 18-byte Q4 blocks (bytes) -> (wq4, wd) numpy planes."""
    import numpy as np
    src = np.ascontiguousarray(np.frombuffer(blocks18, dtype=np.uint8))
    wq4 = np.empty((n, k // 2), dtype=np.uint8)
    wd = np.empty((n, k // 32), dtype=np.uint16)
    if src.size != n * (k // 32) * 18:
        raise ValueError("blocks18 size does not match N, K")
    _call("q4_0_split_blocks", src.ctypes.data_as(_P), wq4.ctypes.data_as(_P),
          wd.ctypes.data_as(_P), n, k)
    return wq4, wd
