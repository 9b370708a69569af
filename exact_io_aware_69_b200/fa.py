"""ctypes binding of libfa.so (include/fa.h) and libfa_paged.so (include/fa_paged.h):
argument marshalling only.

Every step of the attention computation runs in the library's CUDA kernels; this
module turns torch tensors into device pointers and the current CUDA stream, and
turns status codes into exceptions. It never computes attention itself, and it
raises if the library is missing -- there is no fallback path.
"""

from __future__ import annotations

import ctypes
import functools
import math
import os
import struct

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libfa.so")
PAGED_LIB_PATH = os.path.join(_HERE, "libfa_paged.so")

FA_OK = 0
FA_ERR_INVALID = -1
FA_ERR_UNSUPPORTED = -2
FA_ERR_CUDA = -3
FA_ERR_TIMEOUT = -4
FA_BF16 = 0
FA_FP16 = 1
FA_LAYOUT_BHND = 0
FA_LAYOUT_BNHD = 1
FA_STAGE_PREPROCESS = 1
FA_STAGE_DKDV = 2
FA_STAGE_DQ = 4
FA_STAGE_ALL = 7
LAYOUTS = {"bhnd": FA_LAYOUT_BHND, "bnhd": FA_LAYOUT_BNHD}
STAGES = {"preprocess": FA_STAGE_PREPROCESS, "dkdv": FA_STAGE_DKDV, "dq_convert": FA_STAGE_DQ}

# Every symbol include/fa.h declares, with its ctypes signature.
_vp, _int, _f32, _sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
SIGNATURES = {
    "fa_fwd": (_int, [_vp, _vp, _vp, _vp, _vp, _vp, _int, _int, _int, _int, _int, _f32, _int,
                      _vp]),
    "fa_fwd_qk": (_int, [_vp, _vp, _vp, _vp, _vp, _vp, _int, _int, _int, _int, _int, _int, _f32,
                         _int, _vp]),
    "fa_bwd_workspace_size": (_sz, [_int, _int, _int, _int]),
    "fa_bwd": (_int, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _int, _int, _int, _int,
                      _int, _f32, _int, _vp, _sz, _vp]),
    "fa_bwd_qk": (_int, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _int, _int, _int,
                         _int, _int, _int, _f32, _int, _vp, _sz, _vp]),
    "fa_bwd_preprocess": (_int, [_vp, _vp, _vp, _vp, _int, _int, _int, _int, _int, _vp, _sz,
                                 _vp]),
    "fa_bwd_dkdv": (_int, [_vp, _vp, _vp, _vp, _vp, _vp, _int, _int, _int, _int, _int, _f32,
                           _int, _vp, _sz, _vp]),
    "fa_bwd_dq_convert": (_int, [_vp, _int, _int, _int, _int, _f32, _int, _vp, _sz, _vp]),
    "fa_bwd_noalloc": (_int, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _int, _int, _int,
                              _int, _int, _f32, _int, _vp]),
    "fa_fwd_ex": (_int, [_vp, _vp, _vp, _vp, _vp, _vp, _int, _int, _int, _int, _int, _int, _int,
                         _int, _f32, _int, _vp]),
    "fa_bwd_ex_workspace_size": (_sz, [_int, _int, _int, _int, _int, _int]),
    "fa_bwd_ex": (_int, [_vp] * 10 + [_int] * 9 + [_f32, _int, _vp, _sz, _vp]),
    "fa_bwd_ex_stage": (_int, [_int] + [_vp] * 10 + [_int] * 9 + [_f32, _int, _vp, _sz, _vp]),
    "fa_tile_range": (_int, [_int] * 6 + [ctypes.POINTER(_int)] * 2),
    "fa_decode_workspace_size": (_sz, [_int] * 7),
    "fa_decode": (_int, [_vp] * 5 + [_int] * 8 + [_f32, _int, _vp, _sz, _vp]),
    "fa_get_device_status": (_int, [_vp]),
    "fa_selftest_wait_timeout": (_int, [ctypes.c_longlong, _vp]),
    "fa_selftest_exp2": (_int, [_vp, _vp, _int, _vp]),
    "fa_status_string": (ctypes.c_char_p, [_int]),
    "fa_version": (_int, []),
}


# Every symbol include/fa_paged.h declares, with its ctypes signature.
PAGED_SIGNATURES = {
    "fa_rope": (_int, [ctypes.c_char_p, _vp]),
    "fa_paged_append": (_int, [ctypes.c_char_p, _vp]),
    "fa_paged_workspace_size": (_sz, [_int] * 5),
    "fa_paged_attention": (_int, [ctypes.c_char_p, _vp]),
    "fa_paged_device_status": (_int, [_vp]),
}
# Its argument structs as native struct formats: a call's arguments are packed into one
# (building ctypes structures costs a few microseconds a call, as much as a small launch).
_ROWS = "QQ6qi4x"                  # fa_rope_rows: x, y, xs, ys, heads
_CACHE = "QQ6qQQQ9i4x"             # fa_paged_cache
_ROPE_ARGS = struct.Struct("@" + 2 * _ROWS + "QqQ7if")
_APPEND_ARGS = struct.Struct("@" + _CACHE + "QQ6q" + _ROWS + "QQ2if4x")
_ATTENTION_ARGS = struct.Struct("@" + _CACHE + "QQQ6q4if4xQQ")
_NO_ROWS = (0,) * 9

_lib = None
_paged_lib = None
# set with _paged_lib: an import and lookups in every call cost a microsecond
_torch = _raw_stream = _codes = None


class FaError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {status_string(status)} ({status})")


def load():
    """Load libfa.so (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    _lib = _load(LIB_PATH, SIGNATURES)
    return _lib


def load_paged():
    """Load libfa_paged.so (raises if it has not been built)."""
    global _paged_lib, _torch, _raw_stream, _codes
    if _paged_lib is None:
        import torch
        _torch = torch
        _codes = {torch.bfloat16: FA_BF16, torch.float16: FA_FP16}
        # the current stream's handle without building a Stream object, where torch has it
        _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
            lambda device: torch.cuda.current_stream(device).cuda_stream)
        _paged_lib = _load(PAGED_LIB_PATH, PAGED_SIGNATURES)
    return _paged_lib


def _load(path, signatures):
    if not os.path.exists(path):
        raise ImportError(f"{path} is missing: build it with "
                          "`python -m exact_io_aware_69_b200.build`")
    lib = ctypes.CDLL(path)
    for name, (res, args) in signatures.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    return lib


def status_string(status: int) -> str:
    return load().fa_status_string(int(status)).decode()


def _dtype_code(t):
    import torch
    if t.dtype == torch.bfloat16:
        return FA_BF16
    if t.dtype == torch.float16:
        return FA_FP16
    raise FaError(FA_ERR_UNSUPPORTED, f"dtype {t.dtype}")


def _stream_handle(stream):
    import torch
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _check(t, name, like=None):
    if not t.is_cuda:
        raise FaError(FA_ERR_INVALID, f"{name} is not a CUDA tensor")
    if not t.is_contiguous():
        raise FaError(FA_ERR_INVALID, f"{name} is not contiguous")
    if like is not None and (t.shape != like.shape or t.dtype != like.dtype):
        raise FaError(FA_ERR_INVALID, f"{name} shape/dtype differs from q")


def _ptr_or_none(t):
    return None if t is None else t.data_ptr()


def _dims(t, layout):
    """(B, H, N, d) of a tensor in `layout` ("bhnd": [B, H, N, d], "bnhd": [B, N, H, d])."""
    if t.dim() != 4:
        raise FaError(FA_ERR_INVALID, "expected a 4-D tensor")
    if layout == "bhnd":
        return tuple(t.shape)
    if layout == "bnhd":
        B, N, H, d = t.shape
        return B, H, N, d
    raise FaError(FA_ERR_INVALID, f"layout {layout!r}")


def _check_kv(q, k, v, layout="bhnd"):
    """k and v: like q except for the sequence length."""
    _check(k, "k")
    _check(v, "v", k)
    Bq, Hq, _, dq = _dims(q, layout)
    Bk, Hk, _, dk = _dims(k, layout)
    if (Bq, Hq, dq) != (Bk, Hk, dk) or k.dtype != q.dtype:
        raise FaError(FA_ERR_INVALID, "k/v batch, heads, head dim or dtype differ from q")


def _window(causal, window):
    """(left, right) key window; `window` overrides `causal` ((-1, 0) when set)."""
    if window is not None:
        return int(window[0]), int(window[1])
    return (-1, 0) if causal else (-1, -1)


def forward(q, k, v, causal: bool = False, scale: float | None = None, out=None, lse=None,
            out_res=None, residual: bool = True, stream=None, window=None, layout="bhnd"):
    """(O, L, O_res) = attention(q, k, v) for bf16/fp16 CUDA tensors in `layout` ("bhnd":
    q [B, H, Nq, d], k and v [B, H, Nk, d]; "bnhd": [B, N, H, d]). Masks: `causal`, or
    a key window (left, right) around the bottom-right diagonal, negative = unbounded.

    O_res is the 16-bit rounding residual of O (None when residual=False); pass it to
    backward() so that D = rowsum(dO * O) is formed from O at near-fp32 precision."""
    import torch
    lib = load()
    _check(q, "q")
    _check_kv(q, k, v, layout)
    B, H, N, d = _dims(q, layout)
    Nk = _dims(k, layout)[2]
    wl, wr = _window(causal, window)
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if out is None:
        out = torch.empty_like(q)
    if lse is None:
        lse = torch.empty((B, H, N), device=q.device, dtype=torch.float32)
    if out_res is None and residual:
        out_res = torch.empty_like(q)
    rc = lib.fa_fwd_ex(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(),
                       _ptr_or_none(out_res), lse.data_ptr(), B, H, N, Nk, d, LAYOUTS[layout],
                       wl, wr, float(scale), _dtype_code(q), _stream_handle(stream))
    if rc != FA_OK:
        raise FaError(rc, "fa_fwd_ex")
    return out, lse, out_res


def workspace_size(B, H, N, d, Nk=None, deterministic=False) -> int:
    return int(load().fa_bwd_ex_workspace_size(B, H, N, N if Nk is None else Nk, d,
                                               int(bool(deterministic))))


def _bwd_call(stages, q, k, v, o, lse, do, dq, dk, dv, workspace, causal, scale, o_res,
              stream, window, layout, deterministic):
    lib = load()
    B, H, N, d = _dims(q, layout)
    Nk = _dims(k, layout)[2]
    wl, wr = _window(causal, window)

    def p(t):
        return None if t is None else t.data_ptr()
    rc = lib.fa_bwd_ex_stage(stages, p(q), p(k), p(v), p(o), p(o_res), p(do), p(lse), p(dq),
                             p(dk), p(dv), B, H, N, Nk, d, LAYOUTS[layout], wl, wr,
                             int(bool(deterministic)), float(scale), _dtype_code(q),
                             workspace.data_ptr(),
                             workspace.numel() * workspace.element_size(), _stream_handle(stream))
    if rc != FA_OK:
        raise FaError(rc, f"fa_bwd_ex_stage({stages})")


def backward(q, k, v, o, lse, do, causal: bool = False, scale: float | None = None,
             o_res=None, workspace=None, dq=None, dk=None, dv=None, stream=None, window=None,
             layout="bhnd", deterministic=False):
    """dQ, dK, dV of attention, recomputing P from q, k, v and the forward's lse
    (o_res: the forward's rounding residual of O, or None). Masks and layouts as in
    forward()."""
    import torch
    for t, n in ((q, "q"), (o, "o"), (do, "do")):
        _check(t, n, q)
    _check_kv(q, k, v, layout)
    _check(lse, "lse")
    B, H, N, d = _dims(q, layout)
    Nk = _dims(k, layout)[2]
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    need = workspace_size(B, H, N, d, Nk, deterministic)
    if workspace is None:
        workspace = torch.empty(max(need, 1), device=q.device, dtype=torch.uint8)
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(k) if dv is None else dv
    _bwd_call(FA_STAGE_ALL, q, k, v, o, lse, do, dq, dk, dv, workspace, causal, scale, o_res,
              stream, window, layout, deterministic)
    return dq, dk, dv


def backward_stage(stage: str, q, k, v, o, lse, do, dq, dk, dv, workspace, causal: bool,
                   scale: float, o_res=None, stream=None, window=None, layout="bhnd",
                   deterministic=False) -> None:
    """Run one stage of the backward ("preprocess", "dkdv" or "dq_convert") on buffers
    the caller already holds; the three in that order equal backward()."""
    if stage not in STAGES:
        raise ValueError(stage)
    _bwd_call(STAGES[stage], q, k, v, o, lse, do, dq, dk, dv, workspace, causal, scale, o_res,
              stream, window, layout, deterministic)


def tile_range(query_side: bool, tile: int, Nq: int, Nk: int, window) -> tuple[int, int]:
    """(first, count) of the tiles a query tile (query_side) or key tile visits."""
    first, count = ctypes.c_int(), ctypes.c_int()
    rc = load().fa_tile_range(int(bool(query_side)), tile, Nq, Nk, int(window[0]),
                              int(window[1]), ctypes.byref(first), ctypes.byref(count))
    if rc != FA_OK:
        raise FaError(rc, "fa_tile_range")
    return first.value, count.value


def decode(q, k, v, causal: bool = False, scale: float | None = None, out=None, lse=None,
           workspace=None, stream=None, window=None, layout="bhnd"):
    """(O, L) for a few query rows (1 <= Nq <= 16 per head) against a long key sequence:
    the split-KV decode path, forward only. Shapes, masks and layouts as in forward()."""
    import torch
    lib = load()
    _check(q, "q")
    _check_kv(q, k, v, layout)
    B, H, N, d = _dims(q, layout)
    Nk = _dims(k, layout)[2]
    wl, wr = _window(causal, window)
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if out is None:
        out = torch.empty_like(q)
    if lse is None:
        lse = torch.empty((B, H, N), device=q.device, dtype=torch.float32)
    need = int(lib.fa_decode_workspace_size(B, H, N, Nk, d, wl, wr))
    if workspace is None and need > 0:
        workspace = torch.empty(need, device=q.device, dtype=torch.uint8)
    ws = None if workspace is None else workspace.data_ptr()
    wsb = 0 if workspace is None else workspace.numel() * workspace.element_size()
    rc = lib.fa_decode(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), lse.data_ptr(),
                       B, H, N, Nk, d, LAYOUTS[layout], wl, wr, float(scale), _dtype_code(q), ws,
                       wsb, _stream_handle(stream))
    if rc != FA_OK:
        raise FaError(rc, "fa_decode")
    return out, lse


# ------------------------------------------------- rotary positions and the paged cache
def rope_frequencies(rot_dim: int, base: float = 10000.0, method: str = "none",
                     factor: float = 1.0, train_len: int | None = None, low: float = 1.0,
                     high: float = 4.0, device="cuda"):
    """Angle per position of each of the rot_dim / 2 column pairs: a float64 tensor for
    rope() and paged_append(). Pair i turns by base**(-2 i / rot_dim) per position; to
    stretch the context by `factor`, method

    * "linear" divides every angle by it,
    * "base" multiplies the base by factor**(rot_dim / (rot_dim - 2)), which leaves the
      fastest pair as it is and divides the slowest by the factor,
    * "ramp" leaves pairs that turn at least `high` times over `train_len` positions as
      they are, divides those that turn at most `low` times, and blends between.
    """
    import torch
    if rot_dim < 2 or rot_dim % 2 or base <= 0 or factor <= 0:
        raise FaError(FA_ERR_INVALID, "rope_frequencies: rot_dim, base or factor")
    if method == "base":
        if rot_dim == 2:
            raise FaError(FA_ERR_INVALID, "rope_frequencies: method 'base' needs rot_dim > 2")
        base = base * factor ** (rot_dim / (rot_dim - 2))
    freqs = [base ** (-2 * i / rot_dim) for i in range(rot_dim // 2)]
    if method == "linear":
        freqs = [f / factor for f in freqs]
    elif method == "ramp":
        if not train_len or high <= low:
            raise FaError(FA_ERR_INVALID, "rope_frequencies: method 'ramp' needs train_len and "
                                          "high > low")
        keep = [min(1.0, max(0.0, (train_len * f / (2 * math.pi) - low) / (high - low)))
                for f in freqs]
        freqs = [f * (k + (1 - k) / factor) for f, k in zip(freqs, keep)]
    elif method not in ("none", "base"):
        raise FaError(FA_ERR_INVALID, f"rope_frequencies: method {method!r}")
    return torch.tensor(freqs, dtype=torch.float64, device=device)


def _bad(message):
    return FaError(FA_ERR_INVALID, message)


def _pack(fields, *values):
    try:
        return fields.pack(*values)
    except (struct.error, OverflowError) as e:  # a number that its C type does not hold
        raise _bad(str(e)) from None


def _on_stream(stream, like, call, *args):
    """call(*args) with `stream` as the current one, so that what the call allocates belongs
    to it."""
    import torch
    if stream.device_index != like.get_device():
        raise _bad("the stream is not of the tensors' device")
    with torch.cuda.stream(stream):
        return call(*args)


def _place(t, name):
    """The device index of a CUDA tensor."""
    device = t.get_device()
    if device < 0:
        raise _bad(f"{name} is not a CUDA tensor")
    return device


def _strides3(t, b, h, n, name):
    """Element strides of dimensions b, h, n of t (-1: absent), whose last is dense."""
    st, shape = t.stride(), t.shape
    if st[-1] != 1 and shape[-1] != 1:
        raise _bad(f"{name}: the last dimension is not dense")
    # a dimension of one row is never stepped over
    return (st[b] if b >= 0 and shape[b] != 1 else 0, st[h] if shape[h] != 1 else 0,
            st[n] if shape[n] != 1 else 0)


def _rope_rows(x, y, name, device, dtype, b, h, n):
    """(y, the fields of fa_rope_rows) of rows rotated from x into y (None: allocated)."""
    if x.get_device() != device or x.dtype != dtype:
        raise _bad(f"{name}: not on the device or of the dtype of the others")
    xs = _strides3(x, b, h, n, name)
    if y is None:
        y = _torch.empty_like(x)
        ys = xs if y.stride() == x.stride() else _strides3(y, b, h, n, name)
    else:
        if y.get_device() != device or y.dtype != dtype or y.shape != x.shape:
            raise _bad(f"{name}_out: not of {name}'s device, dtype or shape")
        ys = _strides3(y, b, h, n, name + "_out")
        if 0 in ys and any(s == 0 and y.shape[i] > 1 for s, i in zip(ys, (b, h, n)) if i >= 0):
            raise _bad(f"{name}_out: rows share memory")
    return y, (x.data_ptr(), y.data_ptr(), *xs, *ys, x.shape[h])


def _check_freqs(freqs, device):
    if freqs.get_device() != device or freqs.dtype != _torch.float64 or freqs.dim() != 1 or \
            not freqs.is_contiguous():
        raise _bad("freqs is not a dense float64 vector on the device of the others")
    return 2 * freqs.shape[0]


def _rope(q, k, freqs, positions, magnitude, interleaved, layout, q_out, k_out, stream, inverse):
    if stream is not None:
        return _on_stream(stream, q, _rope, q, k, freqs, positions, magnitude, interleaved, layout,
                          q_out, k_out, None, inverse)
    lib = _paged_lib or load_paged()
    torch = _torch
    dtype = q.dtype
    code = _codes.get(dtype)
    if code is None:
        raise FaError(FA_ERR_UNSUPPORTED, f"dtype {dtype}")
    device = _place(q, "q")
    if device != torch.cuda.current_device():
        with torch.cuda.device(device):
            return _rope(q, k, freqs, positions, magnitude, interleaved, layout, q_out, k_out,
                         None, inverse)
    B, H, N, d = _dims(q, layout)
    h, n = (1, 2) if layout == "bhnd" else (2, 1)
    rot = _check_freqs(freqs, device)
    q_out, q_rows = _rope_rows(q, q_out, "q", device, dtype, 0, h, n)
    k_rows = _NO_ROWS
    if k is not None:
        if k.dim() != 4 or k.shape[0] != B or k.shape[n] != N or k.shape[3] != d:
            raise _bad("k batch, length or head dim differ from q")
        k_out, k_rows = _rope_rows(k, k_out, "k", device, dtype, 0, h, n)
    else:
        k_out = None
    where = pos_row = 0
    if positions is not None:
        where = positions.data_ptr()
        if positions.get_device() != device or positions.dtype != torch.int32:
            raise _bad("positions is not an int32 tensor on the device of the others")
        st = positions.stride()
        if positions.shape == (B, N) and (N <= 1 or st[1] == 1):
            pos_row = st[0] if B > 1 else 0
        elif positions.shape != (N,) or (N > 1 and st[0] != 1):
            raise _bad("positions is not a dense [N] or [B, N] tensor")
    rc = lib.fa_rope(_pack(_ROPE_ARGS, *q_rows, *k_rows, where, pos_row, freqs.data_ptr(), rot,
                           1 if interleaved else 0, inverse, B, N, d, code, magnitude),
                     _raw_stream(device))
    if rc != FA_OK:
        raise FaError(rc, "fa_rope")
    return q_out, k_out


def rope(q, k, freqs, positions=None, magnitude: float = 1.0, interleaved: bool = False,
         layout="bhnd", q_out=None, k_out=None, stream=None):
    """Rotary positions: (q', k') with the first 2 * len(freqs) columns of every row turned,
    pair i by position * freqs[i] (float64, see rope_frequencies()), and scaled by
    `magnitude`; the other columns are copied. Pairs are the columns (i, i + r/2), or
    (2 i, 2 i + 1) when `interleaved`. q and k (None: only q) are bf16/fp16 CUDA tensors in
    `layout`, of any strides with a dense last dimension; positions are int32 [N] or [B, N]
    (None: 0 .. N-1). q_out and k_out may be q and k."""
    return _rope(q, k, freqs, positions, magnitude, interleaved, layout, q_out, k_out, stream, 0)


def rope_backward(dq, dk, freqs, positions=None, magnitude: float = 1.0,
                  interleaved: bool = False, layout="bhnd", q_out=None, k_out=None, stream=None):
    """The gradients of rope()'s inputs from those of its outputs: the same rotation turned
    the other way. Arguments as in rope()."""
    return _rope(dq, dk, freqs, positions, magnitude, interleaved, layout, q_out, k_out, stream,
                 1)


def _paged_cache(x, name, device, k_pages, v_pages, page_table, cu_q, seq_k, page_layout):
    """The fields of the fa_paged_cache of these tensors for the packed rows x [T, H, d]."""
    dtype, i32 = x.dtype, _torch.int32
    code = _codes.get(dtype)
    if code is None:
        raise FaError(FA_ERR_UNSUPPORTED, f"dtype {dtype}")
    if x.dim() != 3:
        raise _bad(f"{name} is not a packed [T, H, d] tensor")
    if k_pages.get_device() != device or v_pages.get_device() != device or \
            k_pages.dtype != dtype or v_pages.dtype != dtype:
        raise _bad(f"k_pages or v_pages: not of {name}'s device or dtype")
    if page_table.get_device() != device or cu_q.get_device() != device or \
            seq_k.get_device() != device or page_table.dtype != i32 or cu_q.dtype != i32 or \
            seq_k.dtype != i32:
        raise _bad(f"page_table, cu_q or seq_k: not int32 tensors on {name}'s device")
    if page_layout not in LAYOUTS:
        raise _bad(f"layout {page_layout!r}")
    h, n = (1, 2) if page_layout == "bhnd" else (2, 1)
    shape, table = k_pages.shape, page_table.shape
    if len(shape) != 4 or v_pages.shape != shape:
        raise _bad("k_pages and v_pages are not 4-D tensors of one shape")
    batch = seq_k.shape[0] if seq_k.dim() == 1 else -1
    if len(table) != 2 or table[0] != batch or cu_q.shape != (batch + 1,) or \
            shape[3] != x.shape[2]:
        raise _bad("page_table, cu_q, seq_k or the head dims do not fit")
    st = page_table.stride()
    if not (cu_q.is_contiguous() and seq_k.is_contiguous()) or (table[1] > 1 and st[1] != 1):
        raise _bad("page_table, cu_q or seq_k is not dense")
    return (k_pages.data_ptr(), v_pages.data_ptr(), *_strides3(k_pages, 0, h, n, "k_pages"),
            *_strides3(v_pages, 0, h, n, "v_pages"), page_table.data_ptr(), cu_q.data_ptr(),
            seq_k.data_ptr(), st[0] if batch > 1 else 0, table[1], shape[0], shape[n], shape[h],
            shape[3], batch, x.shape[0], code)


def paged_append(k, v, k_pages, v_pages, page_table, cu_q, seq_k, q=None, freqs=None,
                 magnitude: float = 1.0, interleaved: bool = False, positions=None, q_out=None,
                 page_layout="bnhd", stream=None):
    """Write the new tokens' keys and values into a paged cache, in place.

    k and v [T, Hkv, d] are the packed new rows; sequence b owns rows cu_q[b] ..
    cu_q[b+1] - 1 and holds seq_k[b] keys with them. The cache is k_pages and v_pages
    ([P, page, Hkv, d], or [P, Hkv, page, d] for page_layout "bhnd") with page_table
    [B, W]: key j of sequence b is row j % page of page page_table[b, j // page]. All of
    page_table, cu_q and seq_k are int32 CUDA tensors. With `freqs` the keys are rotated on
    the way as in rope(), each at its position in the sequence (or at positions [T]), and so
    is q [T, Hq, d], if given; returns the rotated q (q_out, which may be q), or None."""
    if stream is not None:
        return _on_stream(stream, k, paged_append, k, v, k_pages, v_pages, page_table, cu_q, seq_k,
                          q, freqs, magnitude, interleaved, positions, q_out, page_layout)
    lib = _paged_lib or load_paged()
    torch = _torch
    device = _place(k, "k")
    if device != torch.cuda.current_device():
        with torch.cuda.device(device):
            return paged_append(k, v, k_pages, v_pages, page_table, cu_q, seq_k, q, freqs,
                                magnitude, interleaved, positions, q_out, page_layout)
    cache = _paged_cache(k, "k", device, k_pages, v_pages, page_table, cu_q, seq_k, page_layout)
    T, heads, d = k.shape
    if v.get_device() != device or v.dtype != k.dtype or v.shape != k.shape or heads != cache[15]:
        raise _bad("k, v and the cache have different devices, dtypes, shapes or heads")
    rot = 0 if freqs is None else _check_freqs(freqs, device)
    where = 0
    if positions is not None:
        where = positions.data_ptr()
        if positions.get_device() != device or positions.dtype != torch.int32 or \
                positions.shape != (T,) or not positions.is_contiguous():
            raise _bad("positions is not a dense int32 [T] tensor on the device of the others")
    rows = _NO_ROWS
    if q is not None:
        if freqs is None:
            raise _bad("q without freqs: there is nothing to do to it")
        if q.dim() != 3 or q.shape[0] != T or q.shape[2] != d:
            raise _bad("q is not [T, Hq, d]")
        q_out, rows = _rope_rows(q, q_out, "q", device, k.dtype, -1, 1, 0)
    rc = lib.fa_paged_append(
        _pack(_APPEND_ARGS, *cache, k.data_ptr(), v.data_ptr(), *_strides3(k, -1, 1, 0, "k"),
              *_strides3(v, -1, 1, 0, "v"), *rows, where,
              0 if freqs is None else freqs.data_ptr(), rot, 1 if interleaved else 0, magnitude),
        _raw_stream(device))
    if rc != FA_OK:
        raise FaError(rc, "fa_paged_append")
    return None if q is None else q_out


@functools.lru_cache(maxsize=256)
def paged_workspace_size(tokens: int, max_q: int, heads_q: int, heads: int, d: int) -> int:
    """Bytes of workspace of paged_attention() for these sizes (whatever the lengths)."""
    return int(load_paged().fa_paged_workspace_size(tokens, max_q, heads_q, heads, d))


def paged_attention(q, k_pages, v_pages, page_table, cu_q, seq_k, max_q: int | None = None,
                    causal: bool = True, scale: float | None = None, window=None,
                    page_layout="bnhd", out=None, lse=None, workspace=None, stream=None):
    """(O [T, Hq, d], L [Hq, T]) = attention of the packed new tokens q [T, Hq, d] over
    everything their sequence has in the cache (arguments as in paged_append(), which has
    to have written the new keys). Hq is a multiple of Hkv: query head h reads key head
    h // (Hq // Hkv). The mask is forward()'s, bottom-right aligned over each sequence's
    seq_k keys; here `causal` is the default. max_q: the most new tokens that any sequence
    has (None: T); 1 for a decode step. It picks the kernel for the whole batch and sizes the
    workspace, so leaving it out costs time: 64 single tokens take 186 us without, 162 us
    with it (32 heads over 8, 300 to 16,384 keys). Rows behind the last sequence are not
    written."""
    if stream is not None:
        return _on_stream(stream, q, paged_attention, q, k_pages, v_pages, page_table, cu_q, seq_k,
                          max_q, causal, scale, window, page_layout, out, lse, workspace)
    lib = _paged_lib or load_paged()
    torch = _torch
    device = _place(q, "q")
    if device != torch.cuda.current_device():
        with torch.cuda.device(device):
            return paged_attention(q, k_pages, v_pages, page_table, cu_q, seq_k, max_q, causal,
                                   scale, window, page_layout, out, lse, workspace)
    cache = _paged_cache(q, "q", device, k_pages, v_pages, page_table, cu_q, seq_k, page_layout)
    T, H, d = q.shape
    wl, wr = _window(causal, window)
    if max_q is None:
        max_q = T
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    qs = _strides3(q, -1, 1, 0, "q")
    if out is None:
        out = torch.empty_like(q)
        os_ = qs if out.stride() == q.stride() else _strides3(out, -1, 1, 0, "out")
    else:
        if out.get_device() != device or out.dtype != q.dtype or out.shape != q.shape:
            raise _bad("out: not of q's device, dtype or shape")
        os_ = _strides3(out, -1, 1, 0, "out")
    if lse is None:
        lse = torch.empty((H, T), device=q.device, dtype=torch.float32)
    elif lse.get_device() != device or lse.dtype != torch.float32 or lse.shape != (H, T) or \
            not lse.is_contiguous():
        raise _bad("lse is not a dense float32 [Hq, T] tensor on q's device")
    need = paged_workspace_size(T, max_q, H, cache[15], d)
    ws = 0
    if workspace is not None:
        if workspace.get_device() != device or not workspace.is_contiguous():
            raise _bad("workspace is not a dense tensor on q's device")
        ws, need = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    elif 0 < need < 1 << 62:
        workspace = torch.empty(need, device=q.device, dtype=torch.uint8)
        ws = workspace.data_ptr()
    rc = lib.fa_paged_attention(
        _pack(_ATTENTION_ARGS, *cache, q.data_ptr(), out.data_ptr(), lse.data_ptr(), *qs, *os_, H,
              max_q, wl, wr, scale, ws, need),
        _raw_stream(device))
    if rc != FA_OK:
        raise FaError(rc, "fa_paged_attention")
    return out, lse


def device_status(stream=None) -> int:
    """Synchronise the stream and return (and clear) the device error word: the first
    library's, or, where that holds none, the paged library's (if it has been loaded). An
    error in each is returned by two calls, one after the other."""
    status = int(load().fa_get_device_status(_stream_handle(stream)))
    if status == FA_OK and _paged_lib is not None:
        status = int(_paged_lib.fa_paged_device_status(_stream_handle(stream)))
    return status
