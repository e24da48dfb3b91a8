"""ctypes binding of include/ec.h (argument marshalling only).

Every operation runs in libec.so.  Device buffers are torch CUDA tensors (their
data_ptr()), host inputs are numpy arrays or CPU tensors.  If libec.so is missing
the import fails loudly: there is no CPU fallback.
"""
from __future__ import annotations

import ctypes
import os
import struct

import numpy as np

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libec.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(
        f"{LIB_PATH} is missing: build it with `python -m lossless_entropy_coded_gb300.build` "
        "(or __graft_entry__.build()); the library has no fallback path")

lib = ctypes.CDLL(LIB_PATH)

EC_OK = 0
EC_ERR_INVALID_ARG = -1
EC_ERR_SHAPE = -2
EC_ERR_OVERFLOW = -3
EC_ERR_UNSUPPORTED = -4
EC_ERR_CORRUPT = -5
EC_ERR_CUDA = -6
EC_ERR_OOM = -7
EC_MAX_BATCH = 64
EC_MAX_GROUP = 8
EC_KIND_HUFFMAN_BF16 = 1
EC_KIND_RANS_INT4 = 2
EC_KIND_E8 = 3
EC_KIND_RANS_FP8 = 4
EC_KIND_RANS_EXP = 5

EXPORTS = ["ec_encode_bf16", "ec_encode_rans", "ec_decode", "ec_decode_batch", "ec_gemv", "ec_gemv_group",
           "ec_bf16_gemv", "ec_stats", "ec_code_lengths", "ec_serialize", "ec_deserialize", "ec_status", "ec_free",
           "ec_strerror", "ec_gemv_static", "ec_gemv_path", "ec_encode_e8", "ec_decode_as", "ec_encode_fp8",
           "ec_gemm", "ec_gemm_work_bytes", "ec_bf16_gemm", "ec_encode_bf16_exp", "ec_gemm_group",
           "ec_gemm_group_work_bytes", "ec_kv_pool_bytes", "ec_kv_create", "ec_kv_free", "ec_kv_append", "ec_kv_read",
           "ec_kv_attend", "ec_kv_attend_work_bytes", "ec_kv_fork", "ec_kv_compact", "ec_kv_pages_work_bytes"]


class HuffParams(ctypes.Structure):
    _fields_ = [("max_code_len", ctypes.c_int32), ("tile_steps", ctypes.c_int32), ("hierarchical", ctypes.c_int32),
                ("reserved", ctypes.c_int32)]


class RansParams(ctypes.Structure):
    _fields_ = [("prob_bits", ctypes.c_int32), ("tile_syms", ctypes.c_int32), ("group", ctypes.c_int32),
                ("codes_per_symbol", ctypes.c_int32), ("values", ctypes.c_int32)]


_RANS_VALUES = {"int4": 0, "fp4": 1}  # EC_RANS_VALUES_INT4, EC_RANS_VALUES_FP4_E2M1


class E8Params(ctypes.Structure):
    _fields_ = [("prob_bits", ctypes.c_int32), ("tile_vectors", ctypes.c_int32), ("reserved", ctypes.c_int32 * 2)]


class Fp8Params(ctypes.Structure):
    _fields_ = [("prob_bits", ctypes.c_int32), ("tile_syms", ctypes.c_int32), ("top_t", ctypes.c_int32),
                ("reserved", ctypes.c_int32)]


class ExpParams(ctypes.Structure):
    _fields_ = [("prob_bits", ctypes.c_int32), ("tile_syms", ctypes.c_int32), ("top_t", ctypes.c_int32),
                ("single", ctypes.c_int32)]


class Stats(ctypes.Structure):
    _fields_ = [("kind", ctypes.c_int32), ("max_code_len", ctypes.c_int32), ("n_rows", ctypes.c_int64),
                ("k_cols", ctypes.c_int64), ("k_pad", ctypes.c_int64), ("n_tiles", ctypes.c_int64),
                ("payload_bits", ctypes.c_int64), ("raw_bytes", ctypes.c_int64), ("aux_bytes", ctypes.c_int64),
                ("table_bytes", ctypes.c_int64), ("device_bytes", ctypes.c_int64),
                ("bits_per_weight", ctypes.c_double), ("entropy_bits", ctypes.c_double),
                ("coded_bits_per_symbol", ctypes.c_double), ("n_records", ctypes.c_int64)]

    def as_dict(self):
        return {k: getattr(self, k) for k, _ in self._fields_}


class KvParams(ctypes.Structure):
    _fields_ = [("n_layers", ctypes.c_int32), ("n_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("page_tokens", ctypes.c_int32), ("n_pages", ctypes.c_int64)]


class KvAttn(ctypes.Structure):
    _fields_ = [("n_q_heads", ctypes.c_int32), ("window", ctypes.c_int32), ("sinks", ctypes.c_int32),
                ("scale", ctypes.c_float)]


_vp, _i64, _i32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int
_sig = {
    "ec_encode_bf16": ([_vp, _i64, _i64, ctypes.POINTER(HuffParams), _i32, ctypes.POINTER(_vp)], _i32),
    "ec_encode_rans": ([_vp, _vp, _i64, _i64, ctypes.POINTER(RansParams), _i32, ctypes.POINTER(_vp)], _i32),
    "ec_encode_e8": ([_vp, _vp, ctypes.c_float, _i64, _i64, ctypes.POINTER(E8Params), _i32, ctypes.POINTER(_vp)],
                     _i32),
    "ec_encode_fp8": ([_vp, _vp, _i64, _i64, ctypes.POINTER(Fp8Params), _i32, ctypes.POINTER(_vp)], _i32),
    "ec_encode_bf16_exp": ([_vp, _i64, _i64, ctypes.POINTER(ExpParams), _i32, ctypes.POINTER(_vp)], _i32),
    "ec_decode": ([_vp, _vp, _vp], _i32),
    "ec_decode_batch": ([_vp, _vp, _i32, _vp], _i32),
    "ec_decode_as": ([_vp, _vp, _i32, _vp], _i32),
    "ec_gemv": ([_vp, _vp, _vp, _i32, _vp], _i32),
    "ec_gemv_group": ([_vp, _i32, _vp, _vp, _i32, _vp], _i32),
    "ec_bf16_gemv": ([_vp, _i64, _i64, _vp, _vp, _i32, _vp], _i32),
    "ec_gemm": ([_vp, _vp, _vp, _i32, _vp, ctypes.c_size_t, _vp], _i32),
    "ec_gemm_work_bytes": ([_vp, _i32, ctypes.POINTER(ctypes.c_size_t)], _i32),
    "ec_gemm_group": ([_vp, _i32, _vp, _vp, _i32, _vp, ctypes.c_size_t, _vp], _i32),
    "ec_gemm_group_work_bytes": ([_vp, _i32, _i32, ctypes.POINTER(ctypes.c_size_t)], _i32),
    "ec_bf16_gemm": ([_vp, _i64, _i64, _vp, _vp, _i32, _vp, ctypes.c_size_t, _vp], _i32),
    "ec_gemv_static": ([_vp, _vp, _vp, _i32, _vp], _i32),
    "ec_gemv_path": ([_vp, _i32, _i32], _i32),
    "ec_kv_pool_bytes": ([_vp, _vp], _i32),
    "ec_kv_create": ([_vp, _vp, ctypes.c_size_t, _i32, _vp], _i32),
    "ec_kv_free": ([_vp], None),
    "ec_kv_append": ([_vp, _vp, _vp], _i32),
    "ec_kv_read": ([_vp, _vp, _vp], _i32),
    "ec_kv_attend": ([_vp, _vp, _vp], _i32),
    "ec_kv_attend_work_bytes": ([_vp, _i32, _i64, _i32, _i64, _vp, _vp], _i32),
    "ec_kv_fork": ([_vp, _vp, _vp], _i32),
    "ec_kv_compact": ([_vp, _vp, _vp], _i32),
    "ec_kv_pages_work_bytes": ([_vp, _i32, _i32, _vp], _i32),
    "ec_stats": ([_vp, ctypes.POINTER(Stats)], _i32),
    "ec_code_lengths": ([_vp, _vp], _i32),
    "ec_serialize": ([_vp, _vp, _i64, ctypes.POINTER(_i64)], _i32),
    "ec_deserialize": ([_vp, _i64, _i32, ctypes.POINTER(_vp)], _i32),
    "ec_status": ([_vp], _i32),
    "ec_free": ([_vp], None),
    "ec_strerror": ([_i32], ctypes.c_char_p),
}
for _n, (_a, _r) in _sig.items():
    _f = getattr(lib, _n)
    _f.argtypes = _a
    _f.restype = _r


class EcError(RuntimeError):
    def __init__(self, code: int, what: str = ""):
        self.code = code
        super().__init__(f"{what}: {lib.ec_strerror(code).decode()} ({code})")


def _check(rc: int, what: str) -> None:
    if rc != EC_OK:
        raise EcError(rc, what)


def strerror(code: int) -> str:
    return lib.ec_strerror(code).decode()


def _host_ptr(a):
    """(pointer, keepalive) for a C-contiguous host array (numpy or CPU tensor)."""
    if hasattr(a, "data_ptr"):
        assert not a.is_cuda and a.is_contiguous()
        return a.data_ptr(), a
    a = np.ascontiguousarray(a)
    return a.ctypes.data, a


def _stream_ptr(stream):
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    if hasattr(stream, "cuda_stream"):
        return stream.cuda_stream
    return int(stream)


def _work_buffer(nbytes: int, device, stream):
    """A work buffer for one call on `stream`, allocated there: on the current stream its bytes
    could still be in use by work queued before the call, or be handed to work queued after it
    while the call runs."""
    import torch
    if stream is None:
        return torch.empty(nbytes, dtype=torch.uint8, device=device)
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(_stream_ptr(stream), device=device)
    with torch.cuda.stream(stream):
        return torch.empty(nbytes, dtype=torch.uint8, device=device)


def _dev_ptr(t):
    return 0 if t is None else t.data_ptr()


class Matrix:
    """An encoded matrix resident on one GPU (owns its device blob)."""

    def __init__(self, handle: int, n_rows: int, k_cols: int, kind: int, device: int):
        self.handle = ctypes.c_void_p(handle)
        self.n_rows, self.k_cols, self.kind, self.device = n_rows, k_cols, kind, device

    @property
    def shape(self):
        return (self.n_rows, self.k_cols)

    def stats(self) -> dict:
        s = Stats()
        _check(lib.ec_stats(self.handle, ctypes.byref(s)), "ec_stats")
        return s.as_dict()

    def code_lengths(self) -> np.ndarray:
        out = np.zeros(256, np.uint8)
        _check(lib.ec_code_lengths(self.handle, out.ctypes.data), "ec_code_lengths")
        return out

    def serialize(self) -> bytes:
        """Metadata block + device blob (copied back to the host)."""
        n = ctypes.c_int64()
        _check(lib.ec_serialize(self.handle, None, 0, ctypes.byref(n)), "ec_serialize")
        buf = (ctypes.c_uint8 * n.value)()
        _check(lib.ec_serialize(self.handle, buf, n.value, ctypes.byref(n)), "ec_serialize")
        return bytes(buf)

    def free(self) -> None:
        if self.handle:
            lib.ec_free(self.handle)
            self.handle = ctypes.c_void_p(0)

    def __del__(self):
        try:
            self.free()
        except Exception:
            pass


def encode_bf16(w, max_code_len: int = 12, tile_steps: int = 0, device: int = 0, hierarchical: bool = False) -> Matrix:
    """Huffman-exponent encode a host BF16 matrix [N, K] (uint16 bit patterns);
    hierarchical=True decodes overflowing pairs through DFloat11's hierarchical tables
    instead of window records."""
    n, k = int(w.shape[0]), int(w.shape[1])
    p, keep = _host_ptr(w)
    prm = HuffParams(max_code_len, tile_steps, 1 if hierarchical else 0)
    h = ctypes.c_void_p()
    _check(lib.ec_encode_bf16(p, n, k, ctypes.byref(prm), device, ctypes.byref(h)), "ec_encode_bf16")
    del keep
    return Matrix(h.value, n, k, EC_KIND_HUFFMAN_BF16, device)


def encode_rans(codes, scales_f16, prob_bits: int = 12, tile_syms: int = 4096, group: int = 128,
                device: int = 0, codes_per_symbol: int = 1, values: str = "int4") -> Matrix:
    """rANS-encode host int8 codes [N, K] with FP16 scales [N, ceil(K/group)]: values
    "int4" takes signed codes in [-8, 7], "fp4" FP4 E2M1 patterns in [0, 15]
    (codes_per_symbol 2: one symbol per pair of a lane's consecutive codes)."""
    n, k = int(codes.shape[0]), int(codes.shape[1])
    pc, kc = _host_ptr(codes)
    ps, ks = _host_ptr(scales_f16)
    prm = RansParams(prob_bits, tile_syms, group, codes_per_symbol, _RANS_VALUES[values])
    h = ctypes.c_void_p()
    _check(lib.ec_encode_rans(pc, ps, n, k, ctypes.byref(prm), device, ctypes.byref(h)), "ec_encode_rans")
    return Matrix(h.value, n, k, EC_KIND_RANS_INT4, device)


def encode_e8(q2, row_scales, scale: float, prob_bits: int = 0, tile_vectors: int = 0,
              device: int = 0) -> Matrix:
    """Encode host int8 doubled E8 points q2 [N, K] (each run of 8 columns is 2 p with
    p in E8) with FP32 row scales [N] and the global scale s; decode gives
    bf16(q2 / 2 * s * r_i).  0 selects the defaults (2^11 slots, 1024 vectors a tile)."""
    n, k = int(q2.shape[0]), int(q2.shape[1])
    pq, kq = _host_ptr(q2)
    pr, kr = _host_ptr(row_scales)
    prm = E8Params(prob_bits, tile_vectors)
    h = ctypes.c_void_p()
    _check(lib.ec_encode_e8(pq, pr, float(scale), n, k, ctypes.byref(prm), device, ctypes.byref(h)), "ec_encode_e8")
    return Matrix(h.value, n, k, EC_KIND_E8, device)


def encode_fp8(codes, row_scales, top_t: int = 0, prob_bits: int = 0, tile_syms: int = 0,
               device: int = 0) -> Matrix:
    """Encode host FP8 E4M3 bytes [N, K] with FP32 row scales [N] under a top-t table
    (top_t 0: every code present; 0 for prob_bits / tile_syms: 12 and 4096)."""
    n, k = int(codes.shape[0]), int(codes.shape[1])
    pc, kc = _host_ptr(codes)
    pr, kr = _host_ptr(row_scales)
    prm = Fp8Params(prob_bits, tile_syms, top_t)
    h = ctypes.c_void_p()
    _check(lib.ec_encode_fp8(pc, pr, n, k, ctypes.byref(prm), device, ctypes.byref(h)), "ec_encode_fp8")
    return Matrix(h.value, n, k, EC_KIND_RANS_FP8, device)


def encode_bf16_exp(w, prob_bits: int = 0, tile_syms: int = 0, top_t: int = 0, single: bool = False,
                    device: int = 0) -> Matrix:
    """Encode a host BF16 matrix [N, K] (uint16 bit patterns) with its exponents as rANS
    symbols under a top-t table (pairs of a lane's consecutive exponents unless single),
    escaped exponents as records, sign and mantissa as plain bytes.  0 selects the
    defaults (2^12 slots, 4096-weight tiles, t chosen by the size bound)."""
    n, k = int(w.shape[0]), int(w.shape[1])
    p, keep = _host_ptr(w)
    prm = ExpParams(prob_bits, tile_syms, top_t, 1 if single else 0)
    h = ctypes.c_void_p()
    _check(lib.ec_encode_bf16_exp(p, n, k, ctypes.byref(prm), device, ctypes.byref(h)), "ec_encode_bf16_exp")
    del keep
    return Matrix(h.value, n, k, EC_KIND_RANS_EXP, device)


def deserialize(data: bytes, device: int = 0) -> Matrix:
    """Validate and load ec_serialize output (device < 0: host-only matrix)."""
    buf = (ctypes.c_uint8 * len(data)).from_buffer_copy(data)
    h = ctypes.c_void_p()
    _check(lib.ec_deserialize(buf, len(data), device, ctypes.byref(h)), "ec_deserialize")
    m = Matrix(h.value, 0, 0, 0, device)
    s = m.stats()
    m.n_rows, m.k_cols, m.kind = s["n_rows"], s["k_cols"], s["kind"]
    return m


def decode(W: Matrix, out, stream=None) -> None:
    _check(lib.ec_decode(W.handle, _dev_ptr(out), _stream_ptr(stream)), "ec_decode")


EC_DTYPE_BF16, EC_DTYPE_FP8_E4M3, EC_DTYPE_INT8 = 0, 1, 2
_DTYPES = {"bf16": EC_DTYPE_BF16, "e4m3": EC_DTYPE_FP8_E4M3, "int8": EC_DTYPE_INT8}


def decode_as(W: Matrix, out, dtype: str = "bf16", stream=None) -> None:
    """ec_decode_as: decode into `out` as "bf16" (2 bytes), "e4m3" or "int8" (1 byte)."""
    _check(lib.ec_decode_as(W.handle, _dev_ptr(out), _DTYPES[dtype], _stream_ptr(stream)), "ec_decode_as")


def decode_batch(Ws, outs, stream=None) -> None:
    n = len(Ws)
    hs = (ctypes.c_void_p * n)(*[W.handle.value for W in Ws])
    os_ = (ctypes.c_void_p * n)(*[_dev_ptr(o) for o in outs])
    _check(lib.ec_decode_batch(hs, os_, n, _stream_ptr(stream)), "ec_decode_batch")


def gemv(W: Matrix, x, y, batch: int = 1, stream=None) -> None:
    _check(lib.ec_gemv(W.handle, _dev_ptr(x), _dev_ptr(y), batch, _stream_ptr(stream)), "ec_gemv")


def gemv_static(W: Matrix, x, y, batch: int = 1, stream=None) -> None:
    """ec_gemv_static: the GEMV with no device or host allocation (fixed built-in
    scratch; serialise calls that could overlap on the GPU)."""
    _check(lib.ec_gemv_static(W.handle, _dev_ptr(x), _dev_ptr(y), batch, _stream_ptr(stream)), "ec_gemv_static")


EC_PATH_CUDA_CORES, EC_PATH_TENSOR_CORES = 1, 2


def gemv_path(Ws, batch: int = 1) -> str:
    """Which kernels gemv_group(Ws, ..., batch) uses: "cuda_cores" or "tensor_cores"."""
    if not isinstance(Ws, (list, tuple)):
        Ws = [Ws]
    hs = (ctypes.c_void_p * len(Ws))(*[W.handle.value for W in Ws])
    rc = lib.ec_gemv_path(hs, len(Ws), batch)
    _check(rc if rc < 0 else 0, "ec_gemv_path")
    return "tensor_cores" if rc == EC_PATH_TENSOR_CORES else "cuda_cores"


def gemv_group(Ws, x, ys, batch: int = 1, stream=None) -> None:
    n = len(Ws)
    hs = (ctypes.c_void_p * n)(*[W.handle.value for W in Ws])
    yp = (ctypes.c_void_p * n)(*[_dev_ptr(y) for y in ys])
    _check(lib.ec_gemv_group(hs, n, _dev_ptr(x), yp, batch, _stream_ptr(stream)), "ec_gemv_group")


def bf16_gemv(w, x, y, batch: int = 1, stream=None) -> None:
    n, k = int(w.shape[0]), int(w.shape[1])
    _check(lib.ec_bf16_gemv(_dev_ptr(w), n, k, _dev_ptr(x), _dev_ptr(y), batch, _stream_ptr(stream)),
           "ec_bf16_gemv")


def gemm_work_bytes(W: Matrix, batch: int) -> int:
    """ec_gemm_work_bytes: the work buffer ec_gemm uses with full-size chunks."""
    n = ctypes.c_size_t(0)
    _check(lib.ec_gemm_work_bytes(W.handle, batch, ctypes.byref(n)), "ec_gemm_work_bytes")
    return int(n.value)


def gemm(W: Matrix, x, y, batch: int, work=None, stream=None) -> None:
    """ec_gemm: y = x W^T for any batch (chunked decode + tensor-core GEMM).  work: a
    device tensor (its bytes are the buffer); None allocates one of gemm_work_bytes."""
    if work is None:
        work = _work_buffer(gemm_work_bytes(W, batch), x.device, stream)
    nbytes = work.numel() * work.element_size()
    _check(lib.ec_gemm(W.handle, _dev_ptr(x), _dev_ptr(y), batch, _dev_ptr(work), nbytes, _stream_ptr(stream)),
           "ec_gemm")


def gemm_group_work_bytes(Ws, batch: int) -> int:
    """ec_gemm_group_work_bytes: the work buffer that decodes every packable matrix in one launch."""
    hs = (ctypes.c_void_p * len(Ws))(*[W.handle.value for W in Ws])
    n = ctypes.c_size_t(0)
    _check(lib.ec_gemm_group_work_bytes(hs, len(Ws), batch, ctypes.byref(n)), "ec_gemm_group_work_bytes")
    return int(n.value)


def gemm_group(Ws, xs, ys, batch: int, work=None, stream=None) -> None:
    """ec_gemm_group: ys[m] = xs[m] W_m^T for several matrices, decoded together where
    the work buffer allows (None allocates gemm_group_work_bytes)."""
    n = len(Ws)
    if work is None:
        work = _work_buffer(gemm_group_work_bytes(Ws, batch), ys[0].device, stream)
    hs = (ctypes.c_void_p * n)(*[W.handle.value for W in Ws])
    xp = (ctypes.c_void_p * n)(*[_dev_ptr(x) for x in xs])
    yp = (ctypes.c_void_p * n)(*[_dev_ptr(y) for y in ys])
    nbytes = work.numel() * work.element_size()
    _check(lib.ec_gemm_group(hs, n, xp, yp, batch, _dev_ptr(work), nbytes, _stream_ptr(stream)), "ec_gemm_group")


def bf16_gemm(w, x, y, batch: int, work=None, stream=None) -> None:
    """ec_bf16_gemm: the same tensor-core GEMM on a dense BF16 matrix (work: partial sums, optional)."""
    n, k = int(w.shape[0]), int(w.shape[1])
    nbytes = 0 if work is None else work.numel() * work.element_size()
    _check(lib.ec_bf16_gemm(_dev_ptr(w), n, k, _dev_ptr(x), _dev_ptr(y), batch, _dev_ptr(work), nbytes,
                            _stream_ptr(stream)), "ec_bf16_gemm")


def status(stream=None) -> int:
    """Synchronise the stream and return (and clear) the device status word."""
    return int(lib.ec_status(_stream_ptr(stream)))


# ---------------------------------------------------------------- key/value cache
EC_DTYPE_FP16, EC_DTYPE_FP32 = 3, 4
EC_KV_MAX_SEQS = 1024
_KV_MAX_LEN = 0x7FFFFFF0  # tokens of a sequence; a table may hold more
_ROW_DTYPES = {}   # torch dtype -> EC_DTYPE_*, filled on first use (torch is imported when needed)
_I32 = [None]
_RAW_STREAM = [None]
# The argument structures of ec.h, field by field: ec_kv_seqs, ec_kv_rows, then the rest.
_SEQS, _ROWS = struct.Struct("=qqqi4x"), struct.Struct("=qqqi4x")
_TOKENS = struct.Struct("=32sqqii32s32s")
_ATTENTION = struct.Struct("=32sqqiiqiiif32s32sqqq")
_PAGES = struct.Struct("=32s32sqqqqqqq")
_NO_ROWS = bytes(_ROWS.size)


def _torch_types() -> None:
    import torch
    _I32[0] = torch.int32
    _RAW_STREAM[0] = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
        lambda device: torch.cuda.current_stream(device).cuda_stream)
    _ROW_DTYPES.update({torch.bfloat16: EC_DTYPE_BF16, torch.float16: EC_DTYPE_FP16, torch.float32: EC_DTYPE_FP32})


def _kv_stream(stream, cache) -> int:
    """The stream's handle (None: the current stream of the cache's device, without building a Stream object)."""
    if stream is not None:
        return _stream_ptr(stream)
    return _RAW_STREAM[0](cache.device) if cache.device >= 0 else 0


class KvCache:
    """A paged 4-bit key/value cache over a pool tensor (kept alive here)."""

    def __init__(self, handle: int, params: KvParams, pool, device: int):
        self.handle = ctypes.c_void_p(handle)
        self.params, self.pool, self.device = params, pool, device

    def free(self) -> None:
        if self.handle:
            lib.ec_kv_free(self.handle)
            self.handle = ctypes.c_void_p(0)

    def __del__(self):
        try:
            self.free()
        except Exception:
            pass


def _at(t, cache, what: str) -> int:
    """The address of a tensor on the cache's device, whose bytes lie together."""
    if t.get_device() != cache.device or not t.is_contiguous():
        raise EcError(EC_ERR_INVALID_ARG, what + ": contiguous tensors on the cache's device")
    return t.data_ptr()


class KvSeqs:
    """Sequences of a cache: int32 device tensors table [n, pages] and lens [n] (kept alive here)."""

    def __init__(self, table, lens):
        if _I32[0] is None:
            _torch_types()
        for t, dims in ((table, 2), (lens, 1)):
            if t.dtype != _I32[0] or t.dim() != dims or not t.is_contiguous():
                raise EcError(EC_ERR_INVALID_ARG, "kv_seqs: contiguous int32 tensors [n, pages] and [n]")
        if table.shape[0] != lens.shape[0]:
            raise EcError(EC_ERR_SHAPE, "kv_seqs")
        if not table.is_cuda or table.device != lens.device:
            raise EcError(EC_ERR_INVALID_ARG, "kv_seqs: tensors on one GPU")
        self.device = table.get_device()
        self.table, self.lens = table, lens
        self.n, self.pages = int(table.shape[0]), int(table.shape[1])
        self.packed = _SEQS.pack(table.data_ptr(), self.pages, lens.data_ptr(), self.n)


def kv_pool_bytes(n_layers: int, n_pages: int, n_kv_heads: int, head_dim: int, page_tokens: int = 64) -> int:
    """ec_kv_pool_bytes: the pool's size."""
    n = ctypes.c_size_t(0)
    p = KvParams(n_layers, n_kv_heads, head_dim, page_tokens, n_pages)
    _check(lib.ec_kv_pool_bytes(ctypes.byref(p), ctypes.byref(n)), "ec_kv_pool_bytes")
    return int(n.value)


def kv_cache(n_layers: int, n_pages: int, n_kv_heads: int, head_dim: int, page_tokens: int = 64, pool=None,
             device: int = 0) -> KvCache:
    """ec_kv_create over `pool` (a contiguous device tensor of at least kv_pool_bytes;
    None allocates one).  device < 0: no pool."""
    p = KvParams(n_layers, n_kv_heads, head_dim, page_tokens, n_pages)
    nbytes = kv_pool_bytes(n_layers, n_pages, n_kv_heads, head_dim, page_tokens)
    if device >= 0 and pool is None:
        import torch
        pool = torch.empty(nbytes, dtype=torch.uint8, device=f"cuda:{device}")
    if pool is not None:
        if not pool.is_contiguous():
            raise EcError(EC_ERR_INVALID_ARG, "kv_cache: a contiguous pool")
        nbytes = pool.numel() * pool.element_size()
        if device >= 0 and pool.get_device() != device:
            raise EcError(EC_ERR_INVALID_ARG, "kv_cache: a pool on the cache's device")
    h = ctypes.c_void_p()
    _check(lib.ec_kv_create(ctypes.byref(p), _dev_ptr(pool), nbytes, device, ctypes.byref(h)), "ec_kv_create")
    return KvCache(h.value, p, pool, device)


def kv_seqs(table, lens) -> KvSeqs:
    return KvSeqs(table, lens)


def _seqs(seqs, cache, what: str) -> bytes:
    if seqs.device != cache.device:
        raise EcError(EC_ERR_INVALID_ARG, what + ": sequences on the cache's device")
    return seqs.packed


def _kv_rows(t, cache, heads: int, what: str) -> bytes:
    """ec_kv_rows of [rows, heads, head_dim] with any strides between rows and heads."""
    if _I32[0] is None:
        _torch_types()
    dtype, shape, stride = _ROW_DTYPES.get(t.dtype), t.shape, t.stride()
    if dtype is None or len(shape) != 3 or stride[2] != 1 or t.get_device() != cache.device:
        raise EcError(EC_ERR_INVALID_ARG, what + ": bfloat16, float16 or float32 [rows, heads, head_dim], contiguous in "
                                                 "head_dim, on the cache's device")
    if shape[1] != heads or shape[2] != cache.params.head_dim:
        raise EcError(EC_ERR_SHAPE, what)
    return _ROWS.pack(t.data_ptr(), stride[0], stride[1], dtype)


def _int32_ptr(t, cache, n: int, what: str) -> int:
    if t is None:
        return 0
    if t.dtype != _I32[0] or not t.is_contiguous():
        raise EcError(EC_ERR_INVALID_ARG, what + ": contiguous int32 tensors")
    if t.numel() != n:
        raise EcError(EC_ERR_SHAPE, what)
    return _at(t, cache, what)


def kv_append(cache: KvCache, layer: int, seqs: KvSeqs, k, v, starts=None, max_new: int = 1, stream=None) -> None:
    """ec_kv_append: quantise the new tokens' k and v [rows, n_kv_heads, head_dim] into the cache."""
    heads = cache.params.n_kv_heads
    kr, vr = _kv_rows(k, cache, heads, "ec_kv_append"), _kv_rows(v, cache, heads, "ec_kv_append")
    n = k.shape[0]
    if n != v.shape[0]:
        raise EcError(EC_ERR_SHAPE, "ec_kv_append")
    args = _TOKENS.pack(_seqs(seqs, cache, "ec_kv_append"), _int32_ptr(starts, cache, seqs.n + 1, "ec_kv_append"), n, layer,
                        max_new, kr, vr)
    rc = lib.ec_kv_append(cache.handle, args, _kv_stream(stream, cache))
    if rc:
        raise EcError(rc, "ec_kv_append")


def kv_read(cache: KvCache, layer: int, seqs: KvSeqs, k=None, v=None, starts=None, max_new: int = 1,
            stream=None) -> None:
    """ec_kv_read: the cached values of the sequences' last tokens into k and / or v."""
    heads = cache.params.n_kv_heads
    kr = _NO_ROWS if k is None else _kv_rows(k, cache, heads, "ec_kv_read")
    vr = _NO_ROWS if v is None else _kv_rows(v, cache, heads, "ec_kv_read")
    if k is not None and v is not None and k.shape[0] != v.shape[0]:
        raise EcError(EC_ERR_SHAPE, "ec_kv_read")
    if _I32[0] is None:
        _torch_types()
    n = k.shape[0] if k is not None else v.shape[0] if v is not None else 0
    args = _TOKENS.pack(_seqs(seqs, cache, "ec_kv_read"), _int32_ptr(starts, cache, seqs.n + 1, "ec_kv_read"), n, layer,
                        max_new, kr, vr)
    rc = lib.ec_kv_read(cache.handle, args, _kv_stream(stream, cache))
    if rc:
        raise EcError(rc, "ec_kv_read")


def kv_attend_work_bytes(cache: KvCache, n_seqs: int, n_rows: int, n_q_heads: int, max_new: int = 1,
                         max_len: int = 0, window: int = 0, sinks: int = 0) -> int:
    """ec_kv_attend_work_bytes: the work buffer of kv_attend for calls of at most these sizes
    (max_len 0: of any length)."""
    n = ctypes.c_size_t(0)
    at = KvAttn(n_q_heads, window, sinks, 0.0)
    _check(lib.ec_kv_attend_work_bytes(cache.handle, n_seqs, n_rows, max_new, max_len, ctypes.byref(at),
                                       ctypes.byref(n)), "ec_kv_attend_work_bytes")
    return int(n.value)


def kv_attend(cache: KvCache, layer: int, seqs: KvSeqs, q, out, starts=None, max_new: int = 1, max_len: int = 0,
              scale: float = 0.0, window: int = 0, sinks: int = 0, lse=None, work=None, stream=None) -> None:
    """ec_kv_attend: out [rows, n_q_heads, head_dim] = attention of the new tokens' q over
    the cache; lse float32 [rows, n_q_heads] (optional).  max_len 0: what the table can
    hold.  work: a device tensor of kv_attend_work_bytes; None allocates one."""
    shape = q.shape
    heads = shape[1] if len(shape) == 3 else 0
    qr, orr = _kv_rows(q, cache, heads, "ec_kv_attend"), _kv_rows(out, cache, heads, "ec_kv_attend")
    n = shape[0]
    if out.shape[0] != n:
        raise EcError(EC_ERR_SHAPE, "ec_kv_attend")
    if lse is not None and (lse.dtype not in _ROW_DTYPES or _ROW_DTYPES[lse.dtype] != EC_DTYPE_FP32
                            or not lse.is_contiguous() or lse.numel() != n * heads):
        raise EcError(EC_ERR_INVALID_ARG, "ec_kv_attend: lse is a contiguous float32 tensor [rows, n_q_heads]")
    if work is None:
        most = max_len or min(seqs.pages * cache.params.page_tokens, _KV_MAX_LEN)
        work = _work_buffer(kv_attend_work_bytes(cache, seqs.n, n, heads, max_new, most, window, sinks), q.device, stream)
    args = _ATTENTION.pack(_seqs(seqs, cache, "ec_kv_attend"), _int32_ptr(starts, cache, seqs.n + 1, "ec_kv_attend"), n, layer,
                           max_new, max_len, heads, window, sinks, scale, qr, orr,
                           0 if lse is None else _at(lse, cache, "ec_kv_attend"), _at(work, cache, "ec_kv_attend"), work.nbytes)
    rc = lib.ec_kv_attend(cache.handle, args, _kv_stream(stream, cache))
    if rc:
        raise EcError(rc, "ec_kv_attend")


def kv_pages_work_bytes(cache: KvCache, n_from: int, n_to: int) -> int:
    """ec_kv_pages_work_bytes: the work buffer of kv_fork and kv_compact."""
    n = ctypes.c_size_t(0)
    _check(lib.ec_kv_pages_work_bytes(cache.handle, n_from, n_to, ctypes.byref(n)), "ec_kv_pages_work_bytes")
    return int(n.value)


def _pages_work(cache, a: KvSeqs, b: KvSeqs, work, stream):
    return work if work is not None else _work_buffer(kv_pages_work_bytes(cache, a.n, b.n), a.lens.device, stream)


def kv_fork(cache: KvCache, seqs: KvSeqs, refs, to: KvSeqs, refs_out, parents=None, grow=None, work=None,
            stream=None) -> None:
    """ec_kv_fork: sequences `to` continue seqs[parents] with room for `grow` more tokens."""
    n, what = cache.params.n_pages, "ec_kv_fork"
    work = _pages_work(cache, seqs, to, work, stream)
    args = _PAGES.pack(_seqs(seqs, cache, what), _seqs(to, cache, what), _int32_ptr(refs, cache, n, what),
                       _int32_ptr(refs_out, cache, n, what), _int32_ptr(parents, cache, to.n, what),
                       _int32_ptr(grow, cache, to.n, what), 0, _at(work, cache, what), work.nbytes)
    rc = lib.ec_kv_fork(cache.handle, args, _kv_stream(stream, cache))
    if rc:
        raise EcError(rc, what)


def kv_compact(cache: KvCache, seqs: KvSeqs, refs, to: KvSeqs, refs_out, page_map=None, work=None, stream=None) -> None:
    """ec_kv_compact: the pages in use move to the lowest numbers; page_map: old number -> new."""
    n, what = cache.params.n_pages, "ec_kv_compact"
    work = _pages_work(cache, seqs, to, work, stream)
    args = _PAGES.pack(_seqs(seqs, cache, what), _seqs(to, cache, what), _int32_ptr(refs, cache, n, what),
                       _int32_ptr(refs_out, cache, n, what), 0, 0, _int32_ptr(page_map, cache, n, what),
                       _at(work, cache, what), work.nbytes)
    rc = lib.ec_kv_compact(cache.handle, args, _kv_stream(stream, cache))
    if rc:
        raise EcError(rc, what)
