"""ctypes binding of libfa.so (include/fa.h) and libfa_paged.so (include/fa_paged.h):
argument marshalling only.

Every step of the attention computation runs in the library's CUDA kernels; this
module turns torch tensors into device pointers and the current CUDA stream, and
turns status codes into exceptions. It never computes attention itself, and it
raises if the library is missing -- there is no fallback path.
"""

from __future__ import annotations

import ctypes
import math
import os

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


class _Strides(ctypes.Structure):
    """fa_strides: element strides of batch, head and row."""
    _fields_ = [("b", ctypes.c_longlong), ("h", ctypes.c_longlong), ("n", ctypes.c_longlong)]


class _PagedCache(ctypes.Structure):
    """fa_paged_cache."""
    _fields_ = ([(n, _vp) for n in ("k_pages", "v_pages")]
                + [(n, ctypes.c_longlong) for n in ("k_page", "k_head", "k_row", "v_page",
                                                    "v_head", "v_row")]
                + [(n, _vp) for n in ("table", "cu_q", "seq_k")]
                + [(n, _int) for n in ("table_row", "table_width", "num_pages", "page_size",
                                       "heads", "d", "batch", "tokens", "dtype")])


# Every symbol include/fa_paged.h declares, with its ctypes signature.
_st, _pc = ctypes.POINTER(_Strides), ctypes.POINTER(_PagedCache)
PAGED_SIGNATURES = {
    "fa_rope": (_int, [_vp, _st, _vp, _st, _int] * 2 + [_vp, ctypes.c_longlong, _vp, _int, _f32]
                + [_int] * 6 + [_vp]),
    "fa_paged_append": (_int, [_pc, _vp, _st, _vp, _st, _vp, _st, _vp, _st, _int, _vp, _vp, _int,
                               _f32, _int, _vp]),
    "fa_paged_workspace_size": (_sz, [_int] * 5),
    "fa_paged_attention": (_int, [_pc, _vp, _st, _vp, _st, _vp, _int, _int, _int, _int, _f32, _vp,
                                  _sz, _vp]),
    "fa_paged_device_status": (_int, [_vp]),
}

_lib = None
_paged_lib = None


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
    global _paged_lib
    if _paged_lib is None:
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


def _strides_of(t, b, h, n, name):
    """The fa_strides of dimensions b, h, n of t (None: absent) whose last one is dense."""
    st, shape = t.stride(), t.shape
    if st[-1] != 1 and shape[-1] != 1:
        raise FaError(FA_ERR_INVALID, f"{name}: the last dimension is not dense")
    # a dimension of one row is never stepped over
    return _Strides(*(0 if i is None or shape[i] == 1 else st[i] for i in (b, h, n)))


def _same(t, name, like, dtype=None):
    """t lies on like's device and has its (or the given) dtype."""
    if t.get_device() != like.get_device() or not t.is_cuda:
        raise FaError(FA_ERR_INVALID, f"{name} is not on the device of the others")
    if t.dtype != (like.dtype if dtype is None else dtype):
        raise FaError(FA_ERR_INVALID, f"{name} has dtype {t.dtype}")


def _check_freqs(freqs, like):
    import torch
    _same(freqs, "freqs", like, torch.float64)
    if freqs.dim() != 1 or not freqs.is_contiguous():
        raise FaError(FA_ERR_INVALID, "freqs is not a dense vector")
    return 2 * freqs.shape[0]


class _Launch:
    """The device and stream of a call: the tensors' device becomes the current one, and
    tensors allocated for the call are kept for a stream that is not the current one."""

    __slots__ = ("device", "before", "stream", "other")

    def __init__(self, like, stream):
        self.device, self.stream, self.before = like.get_device(), stream, None

    def __enter__(self):
        import torch
        cuda = torch.cuda
        now = cuda.current_device()
        if now != self.device:
            self.before = now
            cuda.set_device(self.device)
        current = cuda.current_stream()
        self.other = self.stream is not None and self.stream != current
        if self.stream is None:
            self.stream = current
        elif self.stream.device_index != self.device:
            self.__exit__()
            raise FaError(FA_ERR_INVALID, "the stream is of another device than the tensors")
        return self

    def keep(self, *tensors):
        if self.other:
            for t in tensors:
                t.record_stream(self.stream)

    def __exit__(self, *exc):
        if self.before is not None:
            import torch
            torch.cuda.set_device(self.before)
            self.before = None


def _rope(q, k, freqs, positions, magnitude, interleaved, layout, q_out, k_out, stream, inverse):
    import torch
    lib = load_paged()
    dtype = _dtype_code(q)
    if not q.is_cuda:
        raise FaError(FA_ERR_INVALID, "q is not a CUDA tensor")
    B, H, N, d = _dims(q, layout)
    h, n = (1, 2) if layout == "bhnd" else (2, 1)
    rot = _check_freqs(freqs, q)
    Hk = 0
    if k is not None:
        _same(k, "k", q)
        Bk, Hk, Nk, dk = _dims(k, layout)
        if (Bk, Nk, dk) != (B, N, d):
            raise FaError(FA_ERR_INVALID, "k batch, length or head dim differ from q")
    pos_row = 0
    if positions is not None:
        _same(positions, "positions", q, torch.int32)
        if positions.shape == (B, N) and (N <= 1 or positions.stride(1) == 1):
            pos_row = positions.stride(0) if B > 1 else 0
        elif positions.shape != (N,) or (N > 1 and positions.stride(0) != 1):
            raise FaError(FA_ERR_INVALID, "positions is not a dense [N] or [B, N] tensor")
    with _Launch(q, stream) as at:
        outs = []
        for x, y, name in ((q, q_out, "q_out"), (k, k_out, "k_out")):
            if x is None:
                outs.append(None)
                continue
            if y is None:
                y = torch.empty(x.shape, device=x.device, dtype=x.dtype)
                at.keep(y)
            else:
                _same(y, name, x)
                if y.shape != x.shape:
                    raise FaError(FA_ERR_INVALID, f"{name} has another shape")
            outs.append(y)
        q_out, k_out = outs
        args = [q.data_ptr(), _strides_of(q, 0, h, n, "q"), q_out.data_ptr(),
                _strides_of(q_out, 0, h, n, "q_out"), H]
        if k is None:
            args += [None, None, None, None, 0]
        else:
            args += [k.data_ptr(), _strides_of(k, 0, h, n, "k"), k_out.data_ptr(),
                     _strides_of(k_out, 0, h, n, "k_out"), Hk]
        rc = lib.fa_rope(*args, _ptr_or_none(positions), pos_row, freqs.data_ptr(), rot,
                         magnitude, 1 if interleaved else 0, inverse, B, N, d, dtype,
                         at.stream.cuda_stream)
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


def _paged_cache(x, name, k_pages, v_pages, page_table, cu_q, seq_k, page_layout):
    """The fa_paged_cache of these tensors for the packed rows x [T, H, d]."""
    import torch
    dtype = _dtype_code(x)
    if not x.is_cuda or x.dim() != 3:
        raise FaError(FA_ERR_INVALID, f"{name} is not a packed [T, H, d] CUDA tensor")
    _same(k_pages, "k_pages", x)
    _same(v_pages, "v_pages", x)
    i32 = torch.int32
    _same(page_table, "page_table", x, i32)
    _same(cu_q, "cu_q", x, i32)
    _same(seq_k, "seq_k", x, i32)
    if k_pages.dim() != 4 or v_pages.shape != k_pages.shape:
        raise FaError(FA_ERR_INVALID, "k_pages and v_pages are not 4-D tensors of one shape")
    if page_layout not in LAYOUTS:
        raise FaError(FA_ERR_INVALID, f"layout {page_layout!r}")
    h, n = (1, 2) if page_layout == "bhnd" else (2, 1)
    shape = k_pages.shape
    batch = seq_k.shape[0] if seq_k.dim() == 1 else -1
    if page_table.dim() != 2 or page_table.shape[0] != batch or cu_q.shape != (batch + 1,) or \
            shape[3] != x.shape[2]:
        raise FaError(FA_ERR_INVALID, "page_table, cu_q, seq_k or the head dims do not fit")
    width = page_table.shape[1]
    if not (cu_q.is_contiguous() and seq_k.is_contiguous()) or \
            (width > 1 and page_table.stride(1) != 1):
        raise FaError(FA_ERR_INVALID, "page_table, cu_q or seq_k is not dense")
    ks, vs = _strides_of(k_pages, 0, h, n, "k_pages"), _strides_of(v_pages, 0, h, n, "v_pages")
    return _PagedCache(k_pages.data_ptr(), v_pages.data_ptr(), ks.b, ks.h, ks.n, vs.b, vs.h, vs.n,
                       page_table.data_ptr(), cu_q.data_ptr(), seq_k.data_ptr(),
                       page_table.stride(0) if batch > 1 else 0, width, shape[0], shape[n],
                       shape[h], shape[3], batch, x.shape[0], dtype)


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
    import torch
    lib = load_paged()
    cache = _paged_cache(k, "k", k_pages, v_pages, page_table, cu_q, seq_k, page_layout)
    _same(v, "v", k)
    T, heads, d = k.shape
    if v.shape != k.shape or heads != cache.heads:
        raise FaError(FA_ERR_INVALID, "k, v and the cache have different shapes or heads")
    rot = 0 if freqs is None else _check_freqs(freqs, k)
    if positions is not None:
        _same(positions, "positions", k, torch.int32)
        if positions.shape != (T,) or not positions.is_contiguous():
            raise FaError(FA_ERR_INVALID, "positions is not a dense [T] tensor")
    if q is not None and freqs is None:
        raise FaError(FA_ERR_INVALID, "q without freqs: there is nothing to do to it")
    with _Launch(k, stream) as at:
        args = [None, None, None, None, 0]
        if q is not None:
            _same(q, "q", k)
            if q.dim() != 3 or q.shape[0] != T or q.shape[2] != d:
                raise FaError(FA_ERR_INVALID, "q is not [T, Hq, d]")
            if q_out is None:
                q_out = torch.empty(q.shape, device=q.device, dtype=q.dtype)
                at.keep(q_out)
            else:
                _same(q_out, "q_out", q)
                if q_out.shape != q.shape:
                    raise FaError(FA_ERR_INVALID, "q_out has another shape")
            args = [q.data_ptr(), _strides_of(q, None, 1, 0, "q"), q_out.data_ptr(),
                    _strides_of(q_out, None, 1, 0, "q_out"), q.shape[1]]
        rc = lib.fa_paged_append(cache, k.data_ptr(), _strides_of(k, None, 1, 0, "k"),
                                 v.data_ptr(), _strides_of(v, None, 1, 0, "v"), *args,
                                 _ptr_or_none(positions), _ptr_or_none(freqs), rot, magnitude,
                                 1 if interleaved else 0, at.stream.cuda_stream)
    if rc != FA_OK:
        raise FaError(rc, "fa_paged_append")
    return None if q is None else q_out


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
    has (None: T); 1 for a decode step. Rows behind the last sequence are not written."""
    import torch
    lib = load_paged()
    cache = _paged_cache(q, "q", k_pages, v_pages, page_table, cu_q, seq_k, page_layout)
    T, H, d = q.shape
    wl, wr = _window(causal, window)
    if max_q is None:
        max_q = T
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    with _Launch(q, stream) as at:
        if out is None:
            out = torch.empty(q.shape, device=q.device, dtype=q.dtype)
            at.keep(out)
        else:
            _same(out, "out", q)
            if out.shape != q.shape:
                raise FaError(FA_ERR_INVALID, "out has another shape")
        if lse is None:
            lse = torch.empty((H, T), device=q.device, dtype=torch.float32)
            at.keep(lse)
        else:
            _same(lse, "lse", q, torch.float32)
            if lse.shape != (H, T) or not lse.is_contiguous():
                raise FaError(FA_ERR_INVALID, "lse is not a dense [Hq, T] tensor")
        need = lib.fa_paged_workspace_size(T, max_q, H, cache.heads, d)
        ws = None
        if workspace is not None:
            _same(workspace, "workspace", q, workspace.dtype)
            ws, need = workspace.data_ptr(), workspace.numel() * workspace.element_size()
        elif 0 < need < 1 << 62:
            workspace = torch.empty(need, device=q.device, dtype=torch.uint8)
            at.keep(workspace)
            ws = workspace.data_ptr()
        rc = lib.fa_paged_attention(cache, q.data_ptr(), _strides_of(q, None, 1, 0, "q"),
                                    out.data_ptr(), _strides_of(out, None, 1, 0, "out"),
                                    lse.data_ptr(), H, max_q, wl, wr, scale, ws, need,
                                    at.stream.cuda_stream)
    if rc != FA_OK:
        raise FaError(rc, "fa_paged_attention")
    return out, lse


def device_status(stream=None) -> int:
    """Synchronise the stream and return (and clear) the device error word: the first
    library's, or, where that holds none, the paged library's (if it has been loaded)."""
    status = int(load().fa_get_device_status(_stream_handle(stream)))
    if _paged_lib is not None:
        paged = int(_paged_lib.fa_paged_device_status(_stream_handle(stream)))
        status = status if status != FA_OK else paged
    return status
