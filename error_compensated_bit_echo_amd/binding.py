"""Thin Python binding of libecho (include/echo.h, include/echo_layer.h).

Argument marshalling only: every step of the pipeline runs in the HIP
kernels of libecho.so.  PyTorch provides device memory and streams: tensors
are passed by address, the stream defaults to torch's current stream.
Tensor arguments are checked on the host before the call (on the GPU,
contiguous, at least the bytes the call reads or writes); plain integer
addresses are passed through unchecked.

Functions keep the C names (echo_state_init, echo_encode, ...) and raise
EchoError on a non-zero status.  There is no fallback: if libecho.so is
missing the import fails loudly.
"""
from __future__ import annotations

import ctypes as C
import math
import os

import torch  # load torch's HIP runtime first: libecho binds to the same one

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libecho.so")

GROUP = 128
MAX_RANKS = 16


class EchoError(RuntimeError):
    def __init__(self, status: int, where: str):
        super().__init__(f"{where}: {status_string(status)} (status {status})")
        self.status = status


class EchoStateC(C.Structure):
    _fields_ = [("m_fast", C.c_void_p), ("m_slow", C.c_void_p), ("n", C.c_int64),
                ("nranks", C.c_int32), ("rank", C.c_int32), ("bits", C.c_int32),
                ("reserved", C.c_int32)]


class EchoConfigC(C.Structure):
    _fields_ = [("abi_version", C.c_int32), ("group", C.c_int32), ("qmax", C.c_int32),
                ("qmax8", C.c_int32), ("max_ranks", C.c_int32), ("w_fast", C.c_float), ("w_slow", C.c_float),
                ("beta_fast", C.c_float), ("alpha_fast", C.c_float), ("beta_slow", C.c_float),
                ("alpha_slow", C.c_float), ("max_elements", C.c_int64)]


class EchoNormDescC(C.Structure):
    _fields_ = [("tokens", C.c_int64), ("hidden", C.c_int64), ("ld_y", C.c_int64), ("ld_h", C.c_int64),
                ("gate_rows", C.c_int64), ("dtype", C.c_int32), ("stream_dtype", C.c_int32),
                ("post", C.c_int32), ("pre", C.c_int32), ("scale", C.c_float), ("eps", C.c_float)]


class EchoLinearDescC(C.Structure):
    _fields_ = [("m", C.c_int64), ("n", C.c_int64), ("k", C.c_int64), ("ld_x", C.c_int64),
                ("ld_w", C.c_int64), ("ld_out", C.c_int64), ("ld_r", C.c_int64), ("dtype", C.c_int32),
                ("act", C.c_int32), ("gated", C.c_int32), ("reserved", C.c_int32)]


_vp = C.c_void_p
_pp = C.POINTER(C.c_void_p)
_SIGNATURES = {
    "echo_state_init": [C.POINTER(EchoStateC), _vp, _vp, C.c_int64, C.c_int32, C.c_int32, _vp],
    "echo_encode": [C.POINTER(EchoStateC), _vp, _vp, _vp, _vp],
    "echo_reduce_shard": [C.c_int32, C.c_int64, C.c_int32, _pp, _pp, _vp, _vp, _vp, _vp, _vp],
    "echo_decode": [C.c_int64, C.c_int32, _vp, _vp, _vp, _vp],
    "echo_update": [C.POINTER(EchoStateC), _vp, _vp, _vp, _vp, _vp],
    "echo_correction": [C.POINTER(EchoStateC), _vp, _vp],
    "echo_encode_corr": [C.POINTER(EchoStateC), _vp, _vp, _vp, _vp, _vp],
    "echo_update_corr": [C.POINTER(EchoStateC), _vp, _vp, _vp, _vp, _vp, _vp],
    "echo_call_entry": [C.POINTER(EchoStateC), _vp, _vp, _vp, _vp],
    "echo_call_entry_range": [C.POINTER(EchoStateC), _vp, C.c_int32, C.c_int32, _vp, _vp, _vp],
    "echo_call_reduce": [C.POINTER(EchoStateC), _vp, _pp, _pp, _vp, _vp, _vp, _vp],
    "echo_call_exit": [C.POINTER(EchoStateC), _pp, _pp, _vp, _vp],
    "echo_call": [C.POINTER(EchoStateC), _vp, _pp, _pp, _pp, _pp, _vp, _vp, _vp, _vp, _vp, _vp],
    "echo_call_plain": [C.c_int32, C.c_int32, C.c_int64, C.c_int32, _vp, _pp, _pp, _pp, _pp, _vp,
                        _vp, _vp, _vp, _vp, _vp],
    "echo_reduce_shard_sum": [C.c_int32, C.c_int64, C.c_int32, _pp, _pp, _vp, _vp, _vp],
    "echo_rs_reduce": [C.POINTER(EchoStateC), _vp, _pp, _pp, _vp, _vp],
    "echo_rs_call": [C.POINTER(EchoStateC), _vp, _pp, _pp, _vp, _vp, _vp, _vp],
    "echo_stream_copy": [_vp, _vp, C.c_int64, _vp],
    "echo_get_config": [C.POINTER(EchoConfigC)],
    "echo_status_string": [C.c_int],
    "echo_version": [],
}
# include/echo_layer.h: the layer operators beside the all-reduce
_LAYER_SIGNATURES = {
    "echo_norm": [C.POINTER(EchoNormDescC)] + [_vp] * 11,
    "echo_norm_backward_workspace": [C.POINTER(EchoNormDescC)],
    "echo_norm_backward": [C.POINTER(EchoNormDescC)] + [_vp] * 17 + [C.c_int64, _vp],
    "echo_linear_workspace": [C.POINTER(EchoLinearDescC)],
    "echo_linear": [C.POINTER(EchoLinearDescC)] + [_vp] * 7 + [C.c_int64, _vp],
    "echo_linear_backward_workspace": [C.POINTER(EchoLinearDescC)],
    "echo_linear_backward": [C.POINTER(EchoLinearDescC)] + [_vp] * 8 + [C.c_int64, _vp],
}
_RETURNS = {"echo_status_string": C.c_char_p, "echo_norm_backward_workspace": C.c_int64,
            "echo_linear_workspace": C.c_int64, "echo_linear_backward_workspace": C.c_int64}
EXPORTED = tuple(_SIGNATURES)
EXPORTED_LAYER = tuple(_LAYER_SIGNATURES)


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"libecho.so not built at {LIB_PATH}; run __graft_entry__.build()")
    lib = C.CDLL(LIB_PATH)
    for name, args in {**_SIGNATURES, **_LAYER_SIGNATURES}.items():
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = _RETURNS.get(name, C.c_int)
    return lib


lib = _load()


def status_string(status: int) -> str:
    return lib.echo_status_string(int(status)).decode()


def _check(status: int, where: str) -> None:
    if status != 0:
        raise EchoError(status, where)


def _cb(n: int, bits: int) -> int:
    """bytes of the codes of n elements"""
    return n if bits == 8 else n // 2


def _sb(n: int) -> int:
    """bytes of the scales of n elements"""
    return (n // GROUP) * 4


def _ptr(t, nbytes: int = 0, what: str = "buffer"):
    """Device address of a tensor (None -> NULL; plain ints pass through
    unchecked).  A tensor must live on the GPU, be contiguous and hold at
    least nbytes: the library cannot see a host pointer or the end of a
    buffer, and a kernel given either would fault."""
    if t is None:
        return None
    if isinstance(t, int):
        return t
    if not t.is_cuda:
        raise ValueError(f"{what}: a GPU tensor is required (got one on {t.device})")
    if not t.is_contiguous():
        raise ValueError(f"{what}: the tensor must be contiguous")
    if t.nbytes < nbytes:
        raise ValueError(f"{what}: holds {t.nbytes} bytes, the call needs {nbytes}")
    return t.data_ptr()


_PTR16 = C.c_void_p * MAX_RANKS


def _ptrs(ts, nbytes: int = 0, what: str = "buffers"):
    """void*[>= MAX_RANKS] of device addresses: entries past the list are NULL,
    which the library rejects instead of reading past the array."""
    vals = [_ptr(t, nbytes, f"{what}[{i}]") for i, t in enumerate(ts)]
    if len(vals) <= MAX_RANKS:
        return _PTR16(*vals)
    return (C.c_void_p * len(vals))(*vals)


def _stream(stream):
    if stream is None:  # torch's current stream, without building a Stream object (2.7 us of a 12 us call)
        return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


class EchoState:
    """Compensator state of one call sequence: two float32 averages of n
    elements (caller-owned tensors), P ranks, this rank, and the code width of
    the next call's messages (`bits`, 4 or 8; may change from call to call)."""

    def __init__(self, m_fast: torch.Tensor, m_slow: torch.Tensor, n: int, nranks: int, rank: int,
                 bits: int = 4):
        self.m_fast, self.m_slow = m_fast, m_slow  # keep the buffers alive
        self.c = EchoStateC(_ptr(m_fast, 4 * int(n), "m_fast"), _ptr(m_slow, 4 * int(n), "m_slow"),
                            int(n), int(nranks), int(rank), int(bits), 0)

    @property
    def bits(self) -> int:
        return self.c.bits

    @bits.setter
    def bits(self, value: int) -> None:
        self.c.bits = int(value)

    @property
    def n(self) -> int:
        return self.c.n

    @property
    def nranks(self) -> int:
        return self.c.nranks

    @property
    def rank(self) -> int:
        return self.c.rank

    def sizes(self):
        """(n, chunk, bits) of this state's calls"""
        n, P = self.c.n, self.c.nranks
        return n, (n // P if P > 0 else 0), self.c.bits


def echo_state_init(m_fast, m_slow, n, nranks, rank, stream=None, bits: int = 4) -> EchoState:
    st = EchoState(m_fast, m_slow, n, nranks, rank)
    _check(lib.echo_state_init(C.byref(st.c), st.c.m_fast, st.c.m_slow, int(n), int(nranks),
                               int(rank), _stream(stream)), "echo_state_init")
    st.bits = bits
    return st


def echo_encode(st: EchoState, x, codes, scales, stream=None) -> None:
    n, _, bits = st.sizes()
    _check(lib.echo_encode(C.byref(st.c), _ptr(x, 2 * n, "x"), _ptr(codes, _cb(n, bits), "codes"),
                           _ptr(scales, _sb(n), "scales"), _stream(stream)), "echo_encode")


def echo_reduce_shard(shard_codes, shard_scales, out_codes, out_scales, out_y=None, out_e2=None,
                      chunk_n=None, stream=None, bits: int = 4) -> None:
    P = len(shard_codes)
    if chunk_n is None:
        chunk_n = out_codes.numel() * (1 if bits == 8 else 2)
    cn = int(chunk_n)
    _check(lib.echo_reduce_shard(P, cn, int(bits), _ptrs(shard_codes, _cb(cn, bits), "shard_codes"),
                                 _ptrs(shard_scales, _sb(cn), "shard_scales"),
                                 _ptr(out_codes, _cb(cn, bits), "out_codes"),
                                 _ptr(out_scales, _sb(cn), "out_scales"), _ptr(out_y, 2 * cn, "out_y"),
                                 _ptr(out_e2, 4 * cn, "out_e2"), _stream(stream)), "echo_reduce_shard")


def echo_decode(codes, scales, y, n=None, stream=None, bits: int = 4) -> None:
    if n is None:
        n = y.numel()
    n = int(n)
    _check(lib.echo_decode(n, int(bits), _ptr(codes, _cb(n, bits), "codes"), _ptr(scales, _sb(n), "scales"),
                           _ptr(y, 2 * n, "y"), _stream(stream)), "echo_decode")


def echo_stream_copy(src, dst, nbytes=None, stream=None) -> None:
    """Plain streaming copy (the bandwidth ceiling the kernels are measured
    against); nbytes defaults to dst's size in bytes."""
    if nbytes is None:
        nbytes = dst.numel() * dst.element_size()
    nb = int(nbytes)
    _check(lib.echo_stream_copy(_ptr(src, nb, "src"), _ptr(dst, nb, "dst"), nb, _stream(stream)),
           "echo_stream_copy")


def echo_update(st: EchoState, x, codes1, scales1, e2_own, stream=None) -> None:
    n, cn, bits = st.sizes()
    _check(lib.echo_update(C.byref(st.c), _ptr(x, 2 * n, "x"), _ptr(codes1, _cb(n, bits), "codes1"),
                           _ptr(scales1, _sb(n), "scales1"), _ptr(e2_own, 4 * cn, "e2_own"),
                           _stream(stream)), "echo_update")


def echo_correction(st: EchoState, corr, stream=None) -> None:
    n, _, _ = st.sizes()
    _check(lib.echo_correction(C.byref(st.c), _ptr(corr, 4 * n, "corr"), _stream(stream)),
           "echo_correction")


def echo_encode_corr(st: EchoState, x, corr, codes, scales, stream=None) -> None:
    n, _, bits = st.sizes()
    _check(lib.echo_encode_corr(C.byref(st.c), _ptr(x, 2 * n, "x"), _ptr(corr, 4 * n, "corr"),
                                _ptr(codes, _cb(n, bits), "codes"), _ptr(scales, _sb(n), "scales"),
                                _stream(stream)), "echo_encode_corr")


def echo_update_corr(st: EchoState, x, codes1, scales1, e2_own, corr, stream=None) -> None:
    n, cn, bits = st.sizes()
    _check(lib.echo_update_corr(C.byref(st.c), _ptr(x, 2 * n, "x"), _ptr(codes1, _cb(n, bits), "codes1"),
                                _ptr(scales1, _sb(n), "scales1"), _ptr(e2_own, 4 * cn, "e2_own"),
                                _ptr(corr, 4 * n, "corr"), _stream(stream)), "echo_update_corr")


def echo_call_entry(st: EchoState, x, send_codes, send_scales, stream=None) -> None:
    n, _, bits = st.sizes()
    _check(lib.echo_call_entry(C.byref(st.c), _ptr(x, 2 * n, "x"), _ptr(send_codes, _cb(n, bits), "send_codes"),
                               _ptr(send_scales, _sb(n), "send_scales"), _stream(stream)), "echo_call_entry")


def echo_call_entry_range(st: EchoState, x, chunk_begin, chunk_end, send_codes, send_scales,
                          stream=None) -> None:
    n, _, bits = st.sizes()
    _check(lib.echo_call_entry_range(C.byref(st.c), _ptr(x, 2 * n, "x"), int(chunk_begin), int(chunk_end),
                                     _ptr(send_codes, _cb(n, bits), "send_codes"),
                                     _ptr(send_scales, _sb(n), "send_scales"), _stream(stream)),
           "echo_call_entry_range")


def echo_call_reduce(st: EchoState, x, recv_codes, recv_scales, own_codes2, own_scales2, y,
                     stream=None) -> None:
    n, cn, bits = st.sizes()
    _check(lib.echo_call_reduce(C.byref(st.c), _ptr(x, 2 * n, "x"),
                                _ptrs(recv_codes, _cb(cn, bits), "recv_codes"),
                                _ptrs(recv_scales, _sb(cn), "recv_scales"),
                                _ptr(own_codes2, _cb(cn, bits), "own_codes2"),
                                _ptr(own_scales2, _sb(cn), "own_scales2"), _ptr(y, 2 * n, "y"),
                                _stream(stream)), "echo_call_reduce")


def echo_call_exit(st: EchoState, gath_codes, gath_scales, y, stream=None) -> None:
    n, cn, bits = st.sizes()
    _check(lib.echo_call_exit(C.byref(st.c), _ptrs(gath_codes, _cb(cn, bits), "gath_codes"),
                              _ptrs(gath_scales, _sb(cn), "gath_scales"), _ptr(y, 2 * n, "y"),
                              _stream(stream)), "echo_call_exit")


def _call_args(n, cn, bits, x, recv_codes, recv_scales, gath_codes, gath_scales, send_codes,
               send_scales, own_codes2, own_scales2, y):
    """checked addresses of one call's buffers (n elements, chunk cn, bits)"""
    return (_ptr(x, 2 * n, "x"), _ptrs(recv_codes, _cb(cn, bits), "recv_codes"),
            _ptrs(recv_scales, _sb(cn), "recv_scales"), _ptrs(gath_codes, _cb(cn, bits), "gath_codes"),
            _ptrs(gath_scales, _sb(cn), "gath_scales"), _ptr(send_codes, _cb(n, bits), "send_codes"),
            _ptr(send_scales, _sb(n), "send_scales"), _ptr(own_codes2, _cb(cn, bits), "own_codes2"),
            _ptr(own_scales2, _sb(cn), "own_scales2"), _ptr(y, 2 * n, "y"))


def echo_call(st: EchoState, x, recv_codes, recv_scales, gath_codes, gath_scales, send_codes,
              send_scales, own_codes2, own_scales2, y, stream=None) -> None:
    _check(lib.echo_call(C.byref(st.c), *_call_args(*st.sizes(), x, recv_codes, recv_scales, gath_codes,
                                                    gath_scales, send_codes, send_scales, own_codes2,
                                                    own_scales2, y), _stream(stream)), "echo_call")


def echo_call_plain(nranks, rank, x, recv_codes, recv_scales, gath_codes, gath_scales,
                    send_codes, send_scales, own_codes2, own_scales2, y, n=None,
                    stream=None, bits: int = 4) -> None:
    if n is None:
        n = x.numel()
    n, P = int(n), int(nranks)
    cn = n // P if P > 0 else 0
    _check(lib.echo_call_plain(P, int(rank), n, int(bits),
                               *_call_args(n, cn, int(bits), x, recv_codes, recv_scales, gath_codes,
                                           gath_scales, send_codes, send_scales, own_codes2,
                                           own_scales2, y), _stream(stream)), "echo_call_plain")


def echo_reduce_shard_sum(shard_codes, shard_scales, out_y, out_e2=None, chunk_n=None,
                          stream=None, bits: int = 4) -> None:
    if chunk_n is None:
        chunk_n = out_y.numel()
    cn = int(chunk_n)
    _check(lib.echo_reduce_shard_sum(len(shard_codes), cn, int(bits),
                                     _ptrs(shard_codes, _cb(cn, bits), "shard_codes"),
                                     _ptrs(shard_scales, _sb(cn), "shard_scales"),
                                     _ptr(out_y, 2 * cn, "out_y"), _ptr(out_e2, 4 * cn, "out_e2"),
                                     _stream(stream)), "echo_reduce_shard_sum")


def echo_rs_reduce(st: EchoState, x, recv_codes, recv_scales, y_own, stream=None) -> None:
    n, cn, bits = st.sizes()
    _check(lib.echo_rs_reduce(C.byref(st.c), _ptr(x, 2 * n, "x"),
                              _ptrs(recv_codes, _cb(cn, bits), "recv_codes"),
                              _ptrs(recv_scales, _sb(cn), "recv_scales"), _ptr(y_own, 2 * cn, "y_own"),
                              _stream(stream)), "echo_rs_reduce")


def echo_rs_call(st: EchoState, x, recv_codes, recv_scales, send_codes, send_scales, y_own,
                 stream=None) -> None:
    n, cn, bits = st.sizes()
    _check(lib.echo_rs_call(C.byref(st.c), _ptr(x, 2 * n, "x"),
                            _ptrs(recv_codes, _cb(cn, bits), "recv_codes"),
                            _ptrs(recv_scales, _sb(cn), "recv_scales"),
                            _ptr(send_codes, _cb(n, bits), "send_codes"),
                            _ptr(send_scales, _sb(n), "send_scales"), _ptr(y_own, 2 * cn, "y_own"),
                            _stream(stream)), "echo_rs_call")


class PreparedCall:
    """echo_call with every argument marshalled once: for loops that call the
    pipeline again and again on the same buffers (a serving loop's per-layer
    buffers).  Calling it enqueues the call on `stream` (default: torch's
    current stream).  The tensors are kept alive by this object; their
    contents may change between calls, their storage may not.

    The buffer sizes were checked for the state as it was when the call was
    prepared (its n, P, rank and code width).  The library is handed a copy
    of that state, and a call made after the EchoState changed (say, its
    `bits` set from 4 to 8) raises instead of launching: the buffers may be
    too small for the new width."""

    def __init__(self, st: EchoState, x, recv_codes, recv_scales, gath_codes, gath_scales,
                 send_codes, send_scales, own_codes2, own_scales2, y):
        self._keep = (st, x, recv_codes, recv_scales, gath_codes, gath_scales, send_codes,
                      send_scales, own_codes2, own_scales2, y)
        self._st = st
        self._snap = EchoStateC.from_buffer_copy(st.c)
        self._args = (C.byref(self._snap), *_call_args(*st.sizes(), x, recv_codes, recv_scales,
                                                       gath_codes, gath_scales, send_codes, send_scales,
                                                       own_codes2, own_scales2, y))
        self._fn = lib.echo_call

    def __call__(self, stream=None) -> None:
        if bytes(self._st.c) != bytes(self._snap):
            raise ValueError("echo_call: the state changed since the call was prepared "
                             f"(bits {self._snap.bits} -> {self._st.c.bits}); prepare it again")
        rc = self._fn(*self._args, _stream(stream))
        if rc != 0:
            raise EchoError(rc, "echo_call")


def echo_call_prepare(st: EchoState, x, recv_codes, recv_scales, gath_codes, gath_scales,
                      send_codes, send_scales, own_codes2, own_scales2, y) -> PreparedCall:
    """A reusable echo_call on fixed buffers (see PreparedCall)."""
    return PreparedCall(st, x, recv_codes, recv_scales, gath_codes, gath_scales, send_codes,
                        send_scales, own_codes2, own_scales2, y)


# ---- layer operators: norms and products beside the all-reduce -------------------

DTYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}
NORMS = {"none": 0, "rms": 1, "layer": 2}
ACTS = {"none": 0, "relu": 1, "gelu": 2, "gelu_tanh": 3, "silu": 4}


def _code(table, key, what):
    if key not in table:
        raise ValueError(f"{what}: {key!r} is not one of {', '.join(map(str, table))}")
    return table[key]


def _bad_tensor(t, shape, dtype, what):
    """what is wrong with a tensor that its call cannot take"""
    if not isinstance(t, torch.Tensor):
        return f"{what}: a tensor is required"
    if not t.is_cuda:
        return f"{what}: a GPU tensor is required (got one on {t.device})"
    if t.dtype != dtype:
        return f"{what}: {dtype} is required (got {t.dtype})"
    if t.dim() == 0 or t.shape[-1] != shape[-1] or t.numel() != math.prod(shape):
        return f"{what}: shape {tuple(t.shape)}, the call needs {tuple(shape)}"
    return None


def _matrix(t, rows, cols, dtype, what):
    """(address, row pitch in elements) of a [rows, cols] matrix with unit
    stride along its rows, or of a dense tensor of any shape whose last
    dimension is cols."""
    if isinstance(t, torch.Tensor) and t.is_cuda and t.dtype is dtype:
        shape = t.shape
        if shape and shape[-1] == cols and t.numel() == rows * cols:
            if t.is_contiguous():
                return t.data_ptr(), cols
            if len(shape) == 2:
                stride = t.stride()
                if (cols <= 1 or stride[1] == 1) and (rows <= 1 or stride[0] >= cols):
                    return t.data_ptr(), (stride[0] if rows > 1 else cols)
    bad = _bad_tensor(t, (rows, cols), dtype, what)
    raise ValueError(bad or f"{what}: rows of unit stride that do not overlap are required (strides {t.stride()})")


def _dense(t, shape, dtype, what):
    """address of a dense tensor of this shape, or of any whose last dimension
    and number of elements are the same (None -> NULL)"""
    if t is None:
        return None
    if isinstance(t, torch.Tensor) and t.is_cuda and t.dtype is dtype:
        have = t.shape
        if have == shape or (have and have[-1] == shape[-1] and t.numel() == math.prod(shape)):
            if t.is_contiguous():
                return t.data_ptr()
    bad = _bad_tensor(t, shape, dtype, what)
    raise ValueError(bad or f"{what}: the tensor must be contiguous")


def _workspace(t):
    """(address, bytes) of a workspace tensor (None -> NULL, 0)"""
    if t is None:
        return None, 0
    return _ptr(t, 0, "workspace"), t.nbytes


def _dtype_of(t, what):
    if not isinstance(t, torch.Tensor) or t.dtype not in DTYPES:
        raise ValueError(f"{what}: a bfloat16, float16 or float32 tensor is required")
    return t.dtype


def _rows_of(t, what):
    """(rows, columns) of a tensor whose last dimension is a row"""
    _dtype_of(t, what)
    shape = t.shape
    if not shape:
        raise ValueError(f"{what}: a tensor with rows is required")
    cols = shape[-1]
    return (t.numel() // cols if cols else math.prod(shape[:-1])), cols


def echo_norm(h, y, h_out, z, *, post="none", w_post=None, b_post=None, gate=None, scale=1.0,
              pre="rms", w_pre=None, b_pre=None, eps=1e-6, stats=None, stream=None) -> None:
    """h_out = h + scale * gate * N_post(y); z = N_pre(h_out), row by row.

    h and h_out [tokens, hidden] in the stream's type, y and z in y's type (or
    the stream's own); gate [rows, hidden] with tokens a multiple of its rows;
    weights and biases [hidden]; stats float32 [4, tokens] where a backward
    pass follows.  post and pre are "none", "rms" or "layer".  y, h_out and z
    may be None as include/echo_layer.h says; h_out may be h."""
    T, H = _rows_of(h, "h")
    dt, sdt = _dtype_of(h if y is None and z is None else z if y is None else y, "y, z"), h.dtype
    hp, ldh = _matrix(h, T, H, sdt, "h")
    yp, ldy = _matrix(y, T, H, dt, "y") if y is not None else (None, 0)
    op, ldo = _matrix(h_out, T, H, sdt, "h_out") if h_out is not None else (None, ldh)
    if ldo != ldh:
        raise ValueError(f"h, h_out: the same row pitch is required (got {ldh} and {ldo})")
    G = 0 if gate is None else _rows_of(gate, "gate")[0]
    d = EchoNormDescC(T, H, ldy, ldh, G, DTYPES[dt], DTYPES[sdt], NORMS.get(post, -1), NORMS.get(pre, -1), scale, eps)
    if d.post < 0 or d.pre < 0:
        _code(NORMS, post, "post"), _code(NORMS, pre, "pre")
    # (absent vectors are not worth a call each: the smallest norms cost their host time)
    rc = lib.echo_norm(C.byref(d), hp, yp, gate if gate is None else _dense(gate, (G, H), dt, "gate"),
                       w_post if w_post is None else _dense(w_post, (H,), dt, "w_post"),
                       b_post if b_post is None else _dense(b_post, (H,), dt, "b_post"),
                       w_pre if w_pre is None else _dense(w_pre, (H,), dt, "w_pre"),
                       b_pre if b_pre is None else _dense(b_pre, (H,), dt, "b_pre"), op,
                       z if z is None else _dense(z, (T, H), dt, "z"),
                       stats if stats is None else _dense(stats, (4, T), torch.float32, "stats"), _stream(stream))
    if rc:
        _check(rc, "echo_norm")


def echo_norm_backward_workspace(tokens, hidden, gate_rows=0) -> int:
    """bytes of workspace echo_norm_backward takes for this shape"""
    d = EchoNormDescC(int(tokens), int(hidden), 0, 0, int(gate_rows), 0, 0, 0, 0, 1.0, 0.0)
    n = lib.echo_norm_backward_workspace(C.byref(d))
    _check(min(n, 0), "echo_norm_backward_workspace")
    return n


def echo_norm_backward(dz, dh_out, h_out, y, stats, dh, dy, *, post="none", w_post=None, b_post=None,
                       gate=None, scale=1.0, pre="rms", w_pre=None, dw_post=None, db_post=None,
                       dgate=None, dw_pre=None, db_pre=None, workspace=None, stream=None) -> None:
    """Gradients of echo_norm: dh (may be dh_out), dy, and the parameters'
    gradients that are given, from dz and dh_out with the forward call's y,
    h_out and stats.  The parameters are those of the forward call; workspace
    is needed where a parameter's gradient is wanted."""
    T, H = _rows_of(dh, "dh")
    some = dz if dz is not None else dy if dy is not None else y if y is not None else dh
    dt, sdt = _dtype_of(some, "dz, dy, y"), dh.dtype
    hp, ldh = _matrix(h_out, T, H, sdt, "h_out") if h_out is not None else (None, 0)
    yp, ldy = _matrix(y, T, H, dt, "y") if y is not None else (None, 0)
    G = 0 if gate is None else _rows_of(gate, "gate")[0]
    d = EchoNormDescC(T, H, ldy, ldh, G, DTYPES[dt], DTYPES[sdt], _code(NORMS, post, "post"),
                      _code(NORMS, pre, "pre"), float(scale), 0.0)
    vec = lambda t, what: _dense(t, (H,), dt, what)  # noqa: E731
    wp, wn = _workspace(workspace)
    _check(lib.echo_norm_backward(
        C.byref(d), _dense(dz, (T, H), dt, "dz"), _dense(dh_out, (T, H), sdt, "dh_out"), hp, yp,
        _dense(stats, (4, T), torch.float32, "stats"), _dense(gate, (G, H), dt, "gate"),
        vec(w_post, "w_post"), vec(b_post, "b_post"), vec(w_pre, "w_pre"),
        _dense(dh, (T, H), sdt, "dh"), _dense(dy, (T, H), dt, "dy"), _dense(dgate, (G, H), dt, "dgate"),
        vec(dw_post, "dw_post"), vec(db_post, "db_post"), vec(dw_pre, "dw_pre"), vec(db_pre, "db_pre"),
        wp, wn, _stream(stream)), "echo_norm_backward")


def _linear_desc(m, n, k, act, gated, dtype=0, ld_x=0, ld_w=0, ld_out=0, ld_r=0):
    return EchoLinearDescC(int(m), int(n), int(k), ld_x, ld_w, ld_out, ld_r, dtype, _code(ACTS, act, "act"),
                           1 if gated else 0, 0)


def echo_linear_workspace(m, n, k, act="none", gated=False) -> int:
    """bytes of workspace echo_linear takes for m rows of x, n outputs, k inputs"""
    r = lib.echo_linear_workspace(C.byref(_linear_desc(m, n, k, act, gated)))
    _check(min(r, 0), "echo_linear_workspace")
    return r


def echo_linear_backward_workspace(m, n, k, act="none", gated=False) -> int:
    """bytes of workspace echo_linear_backward takes for this shape"""
    r = lib.echo_linear_backward_workspace(C.byref(_linear_desc(m, n, k, act, gated)))
    _check(min(r, 0), "echo_linear_backward_workspace")
    return r


def _linear_shape(x, w, gated):
    """(m, n, k, rows of w, type)"""
    m, k = _rows_of(x, "x")
    if x.dtype is torch.float32:
        raise ValueError("x: a bfloat16 or float16 tensor is required")
    if not isinstance(w, torch.Tensor) or w.dim() != 2 or (gated and w.shape[0] % 2):
        raise ValueError("w: a matrix is required, with an even number of rows if the product is gated")
    rows = w.shape[0]
    return m, (rows // 2 if gated else rows), k, rows, x.dtype


def echo_linear(x, w, out, *, bias=None, residual=None, act="none", gated=False, p=None, workspace=None,
                stream=None) -> None:
    """out = act(p) + residual for p = x w^T + bias; gated, w and bias hold the
    gate's rows and then the up rows, and out = act(p_gate) * p_up + residual.

    x [m, k], w [n, k] (gated [2n, k]), out and residual [m, n], bias and p
    (dense, kept for the backward call) as wide as w has rows; all bfloat16 or
    all float16.  act is "none", "relu", "gelu", "gelu_tanh" or "silu".  out may
    be residual."""
    m, n, k, rows, dt = _linear_shape(x, w, gated)
    xp, ldx = _matrix(x, m, k, dt, "x")
    wp, ldw = _matrix(w, rows, k, dt, "w")
    op, ldo = _matrix(out, m, n, dt, "out")
    rp, ldr = _matrix(residual, m, n, dt, "residual") if residual is not None else (None, 0)
    d = _linear_desc(m, n, k, act, gated, DTYPES[dt], ldx, ldw, ldo, ldr)
    sp, sn = _workspace(workspace)
    _check(lib.echo_linear(C.byref(d), xp, wp, _dense(bias, (rows,), dt, "bias"), rp, op,
                           _dense(p, (m, rows), dt, "p"), sp, sn, _stream(stream)), "echo_linear")


def echo_linear_backward(dout, x, w, p, dx, dw, *, dbias=None, act="none", gated=False, workspace=None,
                         stream=None) -> None:
    """Gradients of echo_linear: dx, dw and dbias, each None to skip it, from
    dout and the forward call's x, w and p (p may be None without an activation
    and a gate).  The residual's gradient is dout."""
    m, n, k, rows, dt = _linear_shape(x, w, gated)
    gp, ldo = _matrix(dout, m, n, dt, "dout")
    xp, ldx = _matrix(x, m, k, dt, "x")
    wp, ldw = _matrix(w, rows, k, dt, "w")
    d = _linear_desc(m, n, k, act, gated, DTYPES[dt], ldx, ldw, ldo, 0)
    sp, sn = _workspace(workspace)
    _check(lib.echo_linear_backward(C.byref(d), gp, xp, wp, _dense(p, (m, rows), dt, "p"),
                                    _dense(dx, (m, k), dt, "dx"), _dense(dw, (rows, k), dt, "dw"),
                                    _dense(dbias, (rows,), dt, "dbias"), sp, sn, _stream(stream)),
           "echo_linear_backward")


def echo_get_config() -> dict:
    cfg = EchoConfigC()
    _check(lib.echo_get_config(C.byref(cfg)), "echo_get_config")
    return {name: getattr(cfg, name) for name, _ in EchoConfigC._fields_}


def echo_version() -> int:
    return int(lib.echo_version())
