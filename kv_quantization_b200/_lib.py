"""ctypes binding of librq (include/rq.h), argument marshalling only.

Every function here has the name of the C entry point it calls and forwards
its arguments unchanged: device buffers are torch CUDA tensors (passed by
data pointer), ``centroids`` is a host float32 array, ``stream`` defaults to
torch's current CUDA stream.  All arithmetic runs in librq's kernels; a
missing or unloadable librq.so raises immediately -- there is no fallback.
"""
from __future__ import annotations

import ctypes as C
import functools
import os
import struct
import threading

import numpy as np

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "librq.so")

RQ_F16, RQ_BF16 = 0, 1
RQ_CODES_PACKED, RQ_CODES_INT8 = 0, 1
RQ_ROPE_HALF, RQ_ROPE_INTERLEAVED = 0, 1
RQ_ROPE_PLAIN, RQ_ROPE_LINEAR, RQ_ROPE_NTK, RQ_ROPE_YARN, RQ_ROPE_BANDED = range(5)

_lock = threading.Lock()
_lib = None


class Strides(C.Structure):
    """rq_strides: batch, token and head strides in elements."""
    _fields_ = [("batch", C.c_int64), ("token", C.c_int64), ("head", C.c_int64)]


class Rows(C.Structure):
    """rq_rows: one array of per-token records to move."""
    _fields_ = [("src", C.c_void_p), ("dst", C.c_void_p), ("row_bytes", C.c_int64)]


class RQError(RuntimeError):
    def __init__(self, fn: str, status: int):
        super().__init__(f"{fn} failed: {status_string(status)} ({status})")
        self.status = status


def lib() -> C.CDLL:
    global _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise RuntimeError(f"librq.so not built ({LIB_PATH}); run python -m kv_quantization_b200.build")
            L = C.CDLL(LIB_PATH)
            vp, i64, i32, u64, sz = C.c_void_p, C.c_int64, C.c_int, C.c_uint64, C.c_size_t
            fp = C.POINTER(C.c_float)
            sig = {
                "rq_status_string": (C.c_char_p, [i32]),
                "rq_code_bytes": (i64, [i64, i32, i32, i32]),
                "rq_device_error": (i32, [i32]),
                "rq_last_launch": (C.c_char_p, []),
                "rq_probe_bounded_wait": (i32, [C.c_uint32, vp]),
                "rq_lloyd_max": (i32, [i32, fp]),
                "rq_quantize": (i32, [vp, i32, i64, i32, i32, i32, i32, u64, fp, vp, vp, vp]),
                "rq_dequantize": (i32, [vp, vp, i64, i32, i32, i32, i32, u64, fp, vp, i32, vp]),
                "rq_quantize_qjl": (i32, [vp, i32, i64, i32, i32, i32, i32, u64, fp, i32, vp, vp, vp, vp, vp, vp]),
                "qjl_make_projection": (i32, [u64, i32, i32, i32, vp, vp]),
                "qjl_sketch": (i32, [vp, i32, i64, i32, i32, vp, vp, vp, vp]),
                "qjl_score_workspace_bytes": (sz, [i64, i32, i32, i32]),
                "qjl_score": (i32, [vp, i64, i32, i32, i32, vp, i32, vp, vp, i64, vp, vp, i32, i32, i32, u64,
                                    fp, vp, vp, sz, vp]),
                "qjl_attention_workspace_bytes": (sz, [i64, i32, i32, i32, i64]),
                "qjl_attention": (i32, [vp, i64, i32, i32, i32, vp, i32, vp, vp, i64, vp, vp, i32, i32, i32, u64,
                                        vp, vp, vp, i32, i32, i32, u64, vp, C.c_float, vp, vp, sz, vp]),
                "qjl_score_noalloc": (i32, [vp, i64, i32, i32, i32, vp, i32, vp, vp, i64, vp, vp, i32, i32, i32,
                                            u64, fp, vp, vp]),
                "qjl_sketch_outlier_workspace_bytes": (sz, [i64, i32]),
                "qjl_sketch_outlier": (i32, [vp, i64, i32, i32, vp, i32, i32, vp, vp, vp, vp, vp, vp, sz, vp]),
                "qjl_score_outlier": (i32, [vp, i64, i32, i32, i32, vp, vp, vp, i64, i32, i32, vp, vp, vp, vp, vp, sz,
                                            vp]),
                "rq_beta_lloyd_max": (i32, [i32, i32, fp]),
                "rq_make_rotation": (i32, [i32, u64, fp]),
                "rq_quantize_dense": (i32, [vp, i32, i64, i32, vp, i32, i32, fp, vp, vp, vp]),
                "rq_dequantize_dense": (i32, [vp, vp, i64, i32, vp, i32, i32, fp, vp, i32, vp]),
                "rq_rotary_frequencies": (i32, [i32, C.c_double, i32, C.c_double, C.c_double, C.c_double, C.c_double,
                                                vp, vp]),
                "rq_rotary": (i32, [vp, vp, vp, vp, i32, vp, vp, vp, vp, i32, i32, i64, i64, i32, i32, i32, vp, i64,
                                    vp, C.c_double, i32, vp]),
                "qjl_tree_attention_workspace_bytes": (sz, [i64, i32, i32, i32, i32, i32, i64]),
                "qjl_tree_attention": (i32, [vp, vp, vp, vp, vp, vp, i64, i32, i32, i32, i32, vp, i64, i32, vp, i32, vp,
                                             vp, i64, vp, vp, vp, i32, i32, i32, u64, vp, vp, vp, i32, i32, i32, u64,
                                             vp, C.c_float, vp, vp, vp, sz, vp]),
                "rq_evict_accumulate_workspace_bytes": (sz, [i64, i32, i64]),
                "rq_evict_accumulate": (i32, [vp, i64, i32, i64, vp, C.c_float, C.c_float, vp, vp, vp, sz, vp]),
                "rq_evict_select": (i32, [vp, i64, i64, vp, i32, i32, i32, vp, vp, vp]),
                "rq_evict_gather": (i32, [vp, vp, i64, i32, i64, i64, vp, i32, vp]),
            }
            for name, (res, args) in sig.items():
                fn = getattr(L, name)
                fn.restype = res
                fn.argtypes = args
            _lib = L
    return _lib


def exported_symbols():
    """Names this binding expects librq.so to export."""
    return ["rq_status_string", "rq_device_error", "rq_last_launch", "rq_probe_bounded_wait", "rq_code_bytes", "rq_lloyd_max", "rq_quantize", "rq_dequantize",
            "rq_quantize_qjl", "qjl_make_projection", "qjl_sketch", "qjl_score_workspace_bytes", "qjl_score",
            "qjl_score_noalloc", "qjl_attention_workspace_bytes", "qjl_attention", "rq_beta_lloyd_max",
            "rq_make_rotation", "rq_quantize_dense", "rq_dequantize_dense", "qjl_sketch_outlier_workspace_bytes",
            "qjl_sketch_outlier", "qjl_score_outlier", "rq_rotary_frequencies", "rq_rotary",
            "qjl_tree_attention_workspace_bytes", "qjl_tree_attention",
            "rq_evict_accumulate_workspace_bytes", "rq_evict_accumulate", "rq_evict_select", "rq_evict_gather"]


def status_string(status: int) -> str:
    return lib().rq_status_string(int(status)).decode()


def _check(fn, status):
    if status != 0:
        raise RQError(fn, status)


def _dev(t):
    return None if t is None else C.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        import torch
        stream = torch.cuda.current_stream()
    return C.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def _table(centroids):
    c = np.ascontiguousarray(np.asarray(centroids, dtype=np.float32))
    return c, c.ctypes.data_as(C.POINTER(C.c_float))


def _dtype_code(t):
    import torch
    if t.dtype == torch.bfloat16:
        return RQ_BF16
    if t.dtype == torch.float16:
        return RQ_F16
    raise TypeError(f"expected a bfloat16 or float16 tensor, got {t.dtype}")


# ------------------------------------------------------------------ entry points

def rq_code_bytes(n: int, d: int, bits: int, layout: int) -> int:
    return lib().rq_code_bytes(n, d, bits, layout)


def rq_device_error(clear: bool = True) -> int:
    """RQ_OK, or RQ_EDEVICE when a kernel gave up a bounded wait since the last clear."""
    return lib().rq_device_error(int(clear))


def rq_last_launch() -> str:
    """Kernels enqueued by this thread's last librq call, comma-separated."""
    return lib().rq_last_launch().decode()


def rq_probe_bounded_wait(polls: int, stream=None):
    _check("rq_probe_bounded_wait", lib().rq_probe_bounded_wait(int(polls), _stream(stream)))


def rq_lloyd_max(bits: int) -> np.ndarray:
    out = np.zeros(1 << bits, np.float32)
    _check("rq_lloyd_max", lib().rq_lloyd_max(bits, out.ctypes.data_as(C.POINTER(C.c_float))))
    return out


def rq_quantize(x, d, bits, layout, use_signs, sign_seed, centroids, codes, norms, stream=None, n=None):
    c, cp = _table(centroids)
    _check("rq_quantize", lib().rq_quantize(_dev(x), _dtype_code(x), x.numel() if n is None else n, d, bits, layout,
                                            int(use_signs), sign_seed, cp, _dev(codes), _dev(norms), _stream(stream)))


def rq_dequantize(codes, norms, n, d, bits, layout, use_signs, sign_seed, centroids, out, stream=None):
    c, cp = _table(centroids)
    _check("rq_dequantize", lib().rq_dequantize(_dev(codes), _dev(norms), n, d, bits, layout, int(use_signs),
                                                sign_seed, cp, _dev(out), _dtype_code(out), _stream(stream)))


def qjl_sketch_outlier_workspace_bytes(n_vec: int, d: int) -> int:
    return lib().qjl_sketch_outlier_workspace_bytes(n_vec, d)


def qjl_sketch_outlier(keys, d, m, proj, m_o, n_out, signs, norms, out_idx, out_signs, out_norms, workspace,
                       stream=None, n_vec=None):
    nv = keys.numel() // d if n_vec is None else n_vec
    _check("qjl_sketch_outlier", lib().qjl_sketch_outlier(
        _dev(keys), nv, d, m, _dev(proj), m_o, n_out, _dev(signs), _dev(norms), _dev(out_idx), _dev(out_signs),
        _dev(out_norms), _dev(workspace), workspace.numel() * workspace.element_size(), _stream(stream)))


def qjl_score_outlier(q, G, n_q, d, m, proj, signs, norms, T, m_o, n_out, out_idx, out_signs, out_norms, scores,
                      workspace, stream=None):
    _check("qjl_score_outlier", lib().qjl_score_outlier(
        _dev(q), G, n_q, d, m, _dev(proj), _dev(signs), _dev(norms), T, m_o, n_out, _dev(out_idx), _dev(out_signs),
        _dev(out_norms), _dev(scores), _dev(workspace), workspace.numel() * workspace.element_size(),
        _stream(stream)))


def rq_beta_lloyd_max(d: int, bits: int) -> np.ndarray:
    """Lloyd-Max centroids (fp32, ascending) of one coordinate of a uniform unit vector in R^d."""
    out = np.zeros(1 << bits, np.float32)
    _check("rq_beta_lloyd_max", lib().rq_beta_lloyd_max(d, bits, out.ctypes.data_as(C.POINTER(C.c_float))))
    return out


def rq_make_rotation(d: int, seed: int) -> np.ndarray:
    """The seeded random orthogonal matrix Pi (d x d, fp32, row-major)."""
    out = np.zeros((d, d), np.float32)
    _check("rq_make_rotation", lib().rq_make_rotation(d, seed, out.ctypes.data_as(C.POINTER(C.c_float))))
    return out


def rq_quantize_dense(x, d, pi, bits, layout, centroids, codes, norms, stream=None, n=None):
    c, cp = _table(centroids)
    _check("rq_quantize_dense", lib().rq_quantize_dense(_dev(x), _dtype_code(x), x.numel() if n is None else n, d,
                                                        _dev(pi), bits, layout, cp, _dev(codes), _dev(norms),
                                                        _stream(stream)))


def rq_dequantize_dense(codes, norms, n, d, pi, bits, layout, centroids, out, stream=None):
    c, cp = _table(centroids)
    _check("rq_dequantize_dense", lib().rq_dequantize_dense(_dev(codes), _dev(norms), n, d, _dev(pi), bits, layout,
                                                            cp, _dev(out), _dtype_code(out), _stream(stream)))


def rq_quantize_qjl(x, d, bits, layout, use_signs, sign_seed, centroids, m, proj, codes, norms, qjl_signs,
                    qjl_norms, stream=None, n=None):
    c, cp = _table(centroids)
    _check("rq_quantize_qjl", lib().rq_quantize_qjl(
        _dev(x), _dtype_code(x), x.numel() if n is None else n, d, bits, layout, int(use_signs), sign_seed, cp,
        m, _dev(proj), _dev(codes), _dev(norms), _dev(qjl_signs), _dev(qjl_norms), _stream(stream)))


def qjl_make_projection(seed, m, d, proj, stream=None):
    _check("qjl_make_projection", lib().qjl_make_projection(seed, m, d, _dtype_code(proj), _dev(proj),
                                                            _stream(stream)))


def qjl_sketch(x, d, m, proj, signs, norms, stream=None, n_vec=None):
    nv = x.numel() // d if n_vec is None else n_vec
    _check("qjl_sketch", lib().qjl_sketch(_dev(x), _dtype_code(x), nv, d, m, _dev(proj), _dev(signs), _dev(norms),
                                          _stream(stream)))


def qjl_score_workspace_bytes(G, n_q, d, m) -> int:
    return lib().qjl_score_workspace_bytes(G, n_q, d, m)


def qjl_score(q, G, n_q, d, m, proj, signs, sk_norms, T, scores, workspace, codes=None, norms=None, bits=0,
              layout=RQ_CODES_PACKED, use_signs=0, sign_seed=0, centroids=None, stream=None):
    if centroids is None:
        cp = None
    else:
        c, cp = _table(centroids)
    _check("qjl_score", lib().qjl_score(
        _dev(q), G, n_q, d, m, _dev(proj), _dtype_code(proj), _dev(signs), _dev(sk_norms), T, _dev(codes),
        _dev(norms), bits, layout, int(use_signs), sign_seed, cp, _dev(scores), _dev(workspace),
        workspace.numel() * workspace.element_size(), _stream(stream)))


def qjl_attention_workspace_bytes(G, n_q, d, m, T) -> int:
    return lib().qjl_attention_workspace_bytes(G, n_q, d, m, T)


def qjl_attention(q, G, n_q, d, m, proj, signs, sk_norms, T, v_codes, v_norms, v_bits, v_centroids, out, workspace,
                  softmax_scale, codes=None, norms=None, bits=0, layout=RQ_CODES_PACKED, use_signs=0, sign_seed=0,
                  centroids=None, v_layout=RQ_CODES_PACKED, v_use_signs=0, v_sign_seed=0, stream=None):
    """Softmax(softmax_scale * score) over the T compressed keys of each group,
    applied to the in-kernel reconstructions of the compressed values:
    out fp32 [G][n_q][d]."""
    cp = None
    if centroids is not None:
        c, cp = _table(centroids)
    vc, vcp = _table(v_centroids)
    _check("qjl_attention", lib().qjl_attention(
        _dev(q), G, n_q, d, m, _dev(proj), _dtype_code(proj), _dev(signs), _dev(sk_norms), T, _dev(codes),
        _dev(norms), bits, layout, int(use_signs), sign_seed, cp, _dev(v_codes), _dev(v_norms), v_bits, v_layout,
        int(v_use_signs), v_sign_seed, vcp, float(softmax_scale), _dev(out), _dev(workspace),
        workspace.numel() * workspace.element_size(), _stream(stream)))


def qjl_score_noalloc(q, G, n_q, d, m, proj, signs, sk_norms, T, scores, codes=None, norms=None, bits=0,
                      layout=RQ_CODES_PACKED, use_signs=0, sign_seed=0, centroids=None, stream=None):
    """qjl_score with the library's own fixed 8 MiB device scratch instead of a
    caller workspace, for callers that cannot allocate device memory."""
    if centroids is None:
        cp = None
    else:
        c, cp = _table(centroids)
    _check("qjl_score_noalloc", lib().qjl_score_noalloc(
        _dev(q), G, n_q, d, m, _dev(proj), _dtype_code(proj), _dev(signs), _dev(sk_norms), T, _dev(codes),
        _dev(norms), bits, layout, int(use_signs), sign_seed, cp, _dev(scores), _stream(stream)))


def _ptr(t):
    return None if t is None else t.data_ptr()


def _call(name, t, stream, args):
    """Call `name` with `args` on the device of tensor `t`, also when another device is current, and on `stream`: that
    device's current one, if none is given."""
    import torch
    fn = getattr(_lib or lib(), name)
    index = t.get_device()
    if stream is None:
        raw = torch._C._cuda_getCurrentRawStream(index)
    else:
        raw = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
    if index == torch._C._cuda_getDevice():
        status = fn(*args, raw)
    else:
        with torch.cuda.device(index):
            status = fn(*args, raw)
    if status != 0:
        raise RQError(name, status)


@functools.lru_cache(None)
def _types():
    """The dtypes of fp32 arrays, int32 arrays, fp16 norms (or their bits) and projection matrices."""
    import torch
    return (torch.float32,), (torch.int32,), (torch.float16, torch.int16, torch.uint16), (torch.bfloat16, torch.float16)


def _need(fn, index, *arrays):
    """Refuse arrays that a kernel would misread or leave.  Each (tensor, types, bytes, name), if it is given, has to be of
    one of the types (None: any), contiguous, of at least that many bytes, and on GPU `index`."""
    for t, types, size, _ in arrays:
        if t is not None and (t.nbytes < size or t.get_device() != index or not t.is_contiguous() or
                              (types is not None and t.dtype not in types)):
            break
    else:
        if index >= 0:
            return
    for t, types, size, name in arrays:
        if t is not None and types is not None and t.dtype not in types:
            raise TypeError(f"{fn}: {name}: expected {' or '.join(map(str, types))}, got {t.dtype}")
        if t is not None and (not t.is_contiguous() or t.nbytes < size):
            raise ValueError(f"{fn}: {name}: expected a contiguous tensor of at least {size} bytes")
    _other_device(fn)


def _other_device(fn):
    raise ValueError(f"{fn}: expected all tensors on one GPU")


_pack3 = struct.Struct("3q").pack


def _strides(t, what):
    """rq_strides (as bytes) of a [batch][token][head][d] tensor with contiguous heads."""
    s = t.stride()
    if len(s) != 4 or (s[3] != 1 and t.shape[3] != 1):
        raise ValueError(f"{what}: expected a [batch, token, head, d] tensor with contiguous heads")
    return _pack3(s[0], s[1], s[2])


def _host(a, dtype):
    """The bytes of a host array as dtype."""
    if type(a) is not np.ndarray or a.dtype != dtype:
        a = np.asarray(a, dtype=dtype)
    return a.tobytes()


def _levels(fn, centroids, bits):
    """The bytes of a host table of 2^bits centroids."""
    table = _host(centroids, np.float32)
    if 1 <= bits <= 8 and len(table) < 4 << bits:
        raise ValueError(f"{fn}: table of {1 << bits} centroids expected")
    return table


def rq_rotary_frequencies(rot_dim: int, theta: float = 10000.0, scaling: int = RQ_ROPE_PLAIN, factor: float = 1.0,
                          original_len: float = 1.0, p0: float = 0.0, p1: float = 0.0):
    """(freq float64 [rot_dim / 2], scale): angle per position step of every pair, and the factor on cos and sin."""
    out, scale = np.zeros(max(1, rot_dim // 2), np.float64), C.c_double(0.0)
    _check("rq_rotary_frequencies", lib().rq_rotary_frequencies(rot_dim, theta, scaling, factor, original_len, p0, p1,
                                                                out.ctypes.data, C.addressof(scale)))
    return out, scale.value


def rq_rotary(x, out, positions, freq, rot_dim, style, scale=1.0, inverse=False, x2=None, out2=None, stream=None):
    """Rotate the heads of x [B, n_tok, heads, d] (and of x2, in the same launch) into out (out2); positions int64
    [B, n_tok] (batch stride 0: shared).  out may be x."""
    import torch
    f = _host(freq, np.float64)
    shape = x.shape
    B, n, H, d = shape
    ps = positions.stride()
    if len(f) < rot_dim // 2 * 8 or out.shape != shape or positions.dtype != torch.int64 or positions.shape != (B, n) or \
            (n > 1 and ps[1] != 1):
        raise ValueError("rq_rotary: freq [rot_dim / 2], out of x's shape, positions int64 [B, n_tok] expected")
    H2, p2 = 0, (None, None, None, None)
    if x2 is not None:
        shape2 = x2.shape
        if out2 is None or out2.shape != shape2 or shape2[0] != B or shape2[1] != n or shape2[3] != d or \
                x2.dtype != x.dtype or out2.dtype != x.dtype:
            raise ValueError("rq_rotary: x2 and out2 of x's batch, tokens, d and dtype expected")
        H2, p2 = shape2[2], (x2.data_ptr(), _strides(x2, "x2"), out2.data_ptr(), _strides(out2, "out2"))
    if out.dtype != x.dtype:
        raise TypeError("rq_rotary: out has another dtype than x")
    dtype, xs, ost = _dtype_code(x), _strides(x, "x"), _strides(out, "out")
    index = x.get_device()
    if index < 0 or out.get_device() != index or positions.get_device() != index or \
            (x2 is not None and (x2.get_device() != index or out2.get_device() != index)):
        _other_device("rq_rotary")
    _call("rq_rotary", x, stream, (
        x.data_ptr(), xs, out.data_ptr(), ost, H, *p2, H2, dtype, B, n, d, rot_dim, style, positions.data_ptr(), ps[0], f,
        scale, 1 if inverse else 0))


def rq_evict_accumulate_workspace_bytes(G, n_q, T) -> int:
    return lib().rq_evict_accumulate_workspace_bytes(G, n_q, T)


def rq_evict_accumulate(scores, G, n_q, T, softmax_scale, decay, acc, out, workspace, row_len=None, stream=None):
    """out [G][T] = decay * acc + sum over queries of softmax(softmax_scale * scores [G][n_q][T]); all fp32, row_len
    int32 [G][n_q]."""
    float32, int32, _, _ = _types()
    _need("rq_evict_accumulate", out.get_device(), (out, float32, 4 * G * T, "out"), (scores, float32, 4 * G * n_q * T, "scores"),
          (acc if decay else None, float32, 4 * G * T, "acc"), (row_len, int32, 4 * G * n_q, "row_len"), (workspace, None, 0, "workspace"))
    _call("rq_evict_accumulate", out, stream, (
        _ptr(scores), G, n_q, T, _ptr(row_len), softmax_scale, decay, _ptr(acc), out.data_ptr(), _ptr(workspace),
        0 if workspace is None else workspace.numel() * workspace.element_size()))


def rq_evict_select(acc, G, T, keep, idx, count, length=None, n_sink=0, n_recent=0, stream=None):
    """idx int32 [G][keep]: the tokens to keep of each group by acc fp32 [G][T], ascending, then -1; count int32 [G];
    length int32 [G]."""
    float32, int32, _, _ = _types()
    _need("rq_evict_select", idx.get_device(), (idx, int32, 4 * G * keep, "idx"), (count, int32, 4 * G, "count"),
          (acc, float32, 4 * G * T, "acc"), (length, int32, 4 * G, "length"))
    _call("rq_evict_select", idx, stream, (_ptr(acc), G, T, _ptr(length), keep, n_sink, n_recent, idx.data_ptr(),
                                           count.data_ptr()))


def rq_evict_gather(idx, count, G, keep, T, arrays, T_dst=None, stream=None):
    """Move the records idx (int32 [G][keep]), count (int32 [G]) of every (src [G][T]..., dst [G][T_dst]...) pair of
    contiguous tensors."""
    int32 = _types()[1]
    T_dst = keep if T_dst is None else T_dst
    rows, index, here = [], idx.get_device(), True
    for src, dst in arrays:
        have, room, size = src.nbytes, dst.nbytes, 0
        if G * T:
            size = have // (G * T)
        elif G * T_dst:                                        # nothing to move
            size = room // (G * T_dst)
        if have != size * G * T or room != size * G * T_dst or not src.is_contiguous() or not dst.is_contiguous():
            raise ValueError("rq_evict_gather: expected contiguous src [G][T] and dst [G][T_dst] of records of one size")
        here = here and src.get_device() == index and dst.get_device() == index
        rows += (src.data_ptr(), dst.data_ptr(), size)
    _need("rq_evict_gather", index if here else -1, (idx, int32, 4 * G * keep, "idx"), (count, int32, 4 * G, "count"))
    _call("rq_evict_gather", idx, stream, (idx.data_ptr(), count.data_ptr(), G, keep, T, T_dst,
                                           struct.pack(f"{len(rows)}q", *rows), len(arrays)))


def qjl_tree_attention_workspace_bytes(B, n_kv_heads, n_rep, n_nodes, d, m, T) -> int:
    return lib().qjl_tree_attention_workspace_bytes(B, n_kv_heads, n_rep, n_nodes, d, m, T)


def qjl_tree_attention(q, k_new, v_new, tree_mask, m, proj, signs, sk_norms, T, kv_len, v_codes, v_norms, v_bits,
                       v_centroids, out, workspace, softmax_scale, codes=None, norms=None, bits=0,
                       layout=RQ_CODES_PACKED, use_signs=0, sign_seed=0, centroids=None, v_layout=RQ_CODES_PACKED,
                       v_use_signs=0, v_sign_seed=0, stream=None):
    """Attention of drafted tokens q [B, n_nodes, heads, d] over the compressed cache and over k_new, v_new
    [B, n_nodes, kv_heads, d]; tree_mask int64 [B or 1, n_nodes, words] (None: a chain); kv_len int32 [B * kv_heads];
    out bf16 of q's shape."""
    import torch
    fn = "qjl_tree_attention"
    shape, kshape = q.shape, k_new.shape
    B, n, H, d = shape
    kv = kshape[2]
    if kshape != (B, n, kv, d) or v_new.shape != kshape or out.shape != shape or kv < 1 or H % kv:
        raise ValueError("qjl_tree_attention: k_new, v_new [B, n_nodes, kv_heads, d] and out of q's shape expected")
    bf16 = torch.bfloat16
    if q.dtype != bf16 or k_new.dtype != bf16 or v_new.dtype != bf16 or out.dtype != bf16:
        raise TypeError("qjl_tree_attention: bfloat16 q, k_new, v_new and out expected")
    stride = 0
    if tree_mask is not None:
        ms = tree_mask.shape
        if len(ms) != 3 or ms[0] not in (1, B) or ms[1] != n or ms[2] != (n + 63) // 64 or \
                tree_mask.dtype not in (torch.int64, torch.uint64) or not tree_mask.is_contiguous():
            raise ValueError("qjl_tree_attention: contiguous 64-bit tree_mask [B or 1, n_nodes, ceil(n_nodes / 64)] expected")
        stride = n * ms[2] if ms[0] > 1 else 0
    strides = _strides(q, "q"), _strides(k_new, "k_new"), _strides(v_new, "v_new"), _strides(out, "out")
    _, int32, half, proj16 = _types()
    rows, kw, vw = B * kv * T, 8 if layout == RQ_CODES_INT8 else bits, 8 if v_layout == RQ_CODES_INT8 else v_bits
    index = q.get_device()
    here = k_new.get_device() == index and v_new.get_device() == index and out.get_device() == index and \
        (tree_mask is None or tree_mask.get_device() == index)
    _need(fn, index if here else -1, (proj, proj16, 2 * m * d, "proj"), (signs, None, rows * m // 8, "signs"),
          (sk_norms, half, 2 * rows, "sk_norms"), (kv_len, int32, 4 * B * kv, "kv_len"), (codes, None, rows * d * kw // 8, "codes"),
          (norms, half, 2 * rows, "norms"), (v_codes, None, rows * d * vw // 8, "v_codes"), (v_norms, half, 2 * rows, "v_norms"),
          (workspace, None, 0, "workspace"))
    c = None if centroids is None else _levels(fn, centroids, bits)
    vc = _levels(fn, v_centroids, v_bits)
    _call("qjl_tree_attention", q, stream, (
        q.data_ptr(), strides[0], k_new.data_ptr(), strides[1], v_new.data_ptr(), strides[2], B, kv, H // kv, n, d,
        _ptr(tree_mask), stride, m, proj.data_ptr(), _dtype_code(proj), _ptr(signs), _ptr(sk_norms), T, _ptr(kv_len),
        _ptr(codes), _ptr(norms), bits, layout, int(use_signs), sign_seed, c, _ptr(v_codes), _ptr(v_norms), v_bits, v_layout,
        int(v_use_signs), v_sign_seed, vc, softmax_scale, out.data_ptr(), strides[3],
        workspace.data_ptr(), workspace.numel() * workspace.element_size()))
