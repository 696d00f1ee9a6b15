"""Python binding of ``libkvdecode.so`` -- the GB300 KV-cached decoder-step library.

Argument marshalling only: every function passes ``torch.Tensor.data_ptr()`` values,
sizes and the current CUDA stream to the C entry point of the same name declared in
``include/kvdecode.h``; all work happens in the library's CUDA kernels. There is no
fallback: if the library has not been built (``python -m kv_cached_decode_gb300.build``)
or a call fails, an exception is raised.

Tensors: caches are ``[batch, n_kv_heads, capacity, 64]`` fp16/bf16 CUDA tensors with
the last axis contiguous; queries/outputs are contiguous ``[batch, n_q_heads, qlen, 64]``;
lengths, drafts, parents and outputs of ``kvd_greedy_accept`` are int32 CUDA tensors;
logits are contiguous fp32 ``[batch, k+1, vocab]`` (``kvd_greedy_accept``) or
``[windows*beam, vocab]`` (``kvd_beam_select``). ``kvd_qk_norm_rope`` reads strided head
rows and ``kvd_sample_filtered`` strided logit rows. A 4-bit cache is a ``Q4Cache`` over
``[batch, n_kv_heads, capacity, 32]`` uint8 data and ``[..., 4]`` int16 parameters.
"""

from __future__ import annotations

import ctypes
import os
import threading

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libkvdecode.so")

KVD_OK = 0
STATUS_NAMES = {0: "KVD_OK", 1: "KVD_ERR_INVALID_ARG", 2: "KVD_ERR_UNSUPPORTED",
                3: "KVD_ERR_WORKSPACE", 4: "KVD_ERR_CUDA", 16: "KVD_ERR_LEN_OVERFLOW",
                17: "KVD_ERR_BAD_INDEX", 18: "KVD_ERR_BAD_TOKEN", 19: "KVD_ERR_NAN",
                20: "KVD_ERR_TIMEOUT", 21: "KVD_ERR_BAD_PARAM"}
KVD_F16, KVD_BF16 = 0, 1
KVD_OP_DECODE_ATTN, KVD_OP_VERIFY_ATTN, KVD_OP_GREEDY_ACCEPT, KVD_OP_SAMPLE_ACCEPT = 0, 1, 2, 3
KVD_OP_WINDOW_ATTN, KVD_OP_Q4_ATTN = 4, 5
KVD_FLAG_PDL, KVD_FLAG_EARLY_KV = 1, 2
KVD_FLAG_TEST_STALL = 1 << 8  # test only: see include/kvdecode.h
KVD_WS_COUNTER_BYTES = 65536
HEAD_DIM = 64

EXPORTED = ("kvd_kv_append", "kvd_decode_attn", "kvd_verify_attn", "kvd_greedy_accept",
            "kvd_beam_reorder_kv", "kvd_workspace_size", "kvd_status_string", "kvd_version",
            "kvd_decode_attn_noalloc", "kvd_prefill_attn", "kvd_rope", "kvd_beam_select",
            "kvd_kv_append_rope", "kvd_sample_accept", "kvd_noalloc_test_fill_counters",
            "kvd_qk_norm_rope", "kvd_window_attn", "kvd_prefill_window_attn", "kvd_q4_append",
            "kvd_q4_dequant", "kvd_q4_attn", "kvd_sample_filtered")


class KvdError(RuntimeError):
    def __init__(self, status: int, call: str):
        self.status = status
        super().__init__(f"{call} failed: {STATUS_NAMES.get(status, status)}")


class Cache(ctypes.Structure):
    """Mirror of ``kvd_cache``: one layer's K and V buffers with shared strides."""

    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
                ("stride_b", ctypes.c_int64), ("stride_h", ctypes.c_int64),
                ("stride_t", ctypes.c_int64), ("batch", ctypes.c_int32),
                ("n_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("capacity", ctypes.c_int32)]


class NewTokens(ctypes.Structure):
    """Mirror of ``kvd_new_tokens``: new K/V appended inside an attention call."""

    _fields_ = [("k_new", ctypes.c_void_p), ("v_new", ctypes.c_void_p),
                ("lens_out", ctypes.c_void_p), ("rope_base", ctypes.c_float)]


class HeadRows(ctypes.Structure):
    """Mirror of ``kvd_head_rows``: one tensor of head rows for ``kvd_qk_norm_rope``."""

    _fields_ = [("x", ctypes.c_void_p), ("stride_b", ctypes.c_int64),
                ("stride_h", ctypes.c_int64), ("stride_t", ctypes.c_int64),
                ("weight", ctypes.c_void_p), ("out", ctypes.c_void_p),
                ("n_heads", ctypes.c_int32)]


class Q4Cache(ctypes.Structure):
    """Mirror of ``kvd_q4_cache``: one layer's K and V held in 4 bits."""

    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("params", ctypes.c_void_p),
                ("stride_b", ctypes.c_int64), ("stride_h", ctypes.c_int64),
                ("batch", ctypes.c_int32), ("n_kv_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("capacity", ctypes.c_int32)]


_lock = threading.Lock()
_lib = None


def load_library(path: str = LIB_PATH):
    """Load the CUDA library (raises if it was never built)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(path):
            raise RuntimeError(
                f"{path} is missing: build it with `python -m kv_cached_decode_gb300.build` "
                "(there is no CPU fallback)")
        lib = ctypes.CDLL(path)
        P, I32, U32, F, SZ = (ctypes.c_void_p, ctypes.c_int32, ctypes.c_uint32, ctypes.c_float,
                              ctypes.c_size_t)
        CP = ctypes.POINTER(Cache)
        NP = ctypes.POINTER(NewTokens)
        QP = ctypes.POINTER(Q4Cache)
        sig = {
            "kvd_kv_append": [I32, CP, I32, I32, P, P, P, P, U32, P, P],
            "kvd_decode_attn": [I32, I32, I32, P, CP, P, I32, NP, I32, F, P, P, SZ, U32, P, P],
            "kvd_decode_attn_noalloc": [I32, I32, I32, P, CP, P, I32, NP, I32, F, P, U32, P, P],
            "kvd_noalloc_test_fill_counters": [ctypes.c_uint8, P],
            "kvd_verify_attn": [I32, I32, I32, I32, P, CP, P, I32, NP, I32, I32, F, P, P, SZ,
                                U32, P, P],
            "kvd_prefill_attn": [I32, I32, I32, I32, P, CP, P, P, P, P, P, F, F, P, U32, P, P],
            "kvd_kv_append_rope": [I32, CP, I32, I32, P, P, P, P, F, U32, P, P],
            "kvd_sample_accept": [P, P, P, I32, I32, I32, F, P, P, P, P, P, SZ, U32, P, P],
            "kvd_rope": [I32, I32, I32, P, I32, P, I32, P, F, U32, P, P],
            "kvd_greedy_accept": [P, I32, I32, I32, P, P, P, P, P, P, SZ, U32, P, P],
            "kvd_beam_reorder_kv": [I32, CP, I32, I32, I32, P, P, I32, U32, P, P],
            "kvd_beam_select": [P, I32, I32, I32, P, P, I32, P, I32, I32, I32, P, P, P, P, P,
                                P, P, P, U32, P, P],
            "kvd_qk_norm_rope": [I32, I32, I32, ctypes.POINTER(HeadRows),
                                 ctypes.POINTER(HeadRows), P, F, F, U32, P, P],
            "kvd_window_attn": [I32, I32, I32, I32, P, CP, P, I32, NP, I32, I32, F, P, P, SZ,
                                U32, P, P],
            "kvd_prefill_window_attn": [I32, I32, I32, I32, P, CP, P, P, P, P, P, I32, I32, F,
                                        F, P, U32, P, P],
            "kvd_q4_append": [I32, QP, I32, I32, P, P, P, P, P, U32, P, P],
            "kvd_q4_dequant": [I32, QP, I32, I32, P, P, P, U32, P, P],
            "kvd_q4_attn": [I32, I32, I32, I32, P, QP, P, I32, I32, I32, I32, F, P, P, SZ, U32,
                            P, P],
            "kvd_sample_filtered": [P, ctypes.c_int64, I32, I32, P, P, P, P, P, P, P, P, U32,
                                    P, P],
            "kvd_workspace_size": [I32, I32, I32, I32, I32, I32, I32, I32],
            "kvd_status_string": [I32],
            "kvd_version": [],
        }
        for name, args in sig.items():
            fn = getattr(lib, name)
            fn.argtypes = args
            fn.restype = I32
        lib.kvd_workspace_size.restype = SZ
        lib.kvd_status_string.restype = ctypes.c_char_p
        _lib = lib
        return lib


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.float16:
        return KVD_F16
    if t.dtype == torch.bfloat16:
        return KVD_BF16
    raise TypeError(f"expected float16 or bfloat16, got {t.dtype}")


_I32, _F32 = torch.int32, torch.float32


def _ptr(t, dtype=None, what="tensor"):
    """The device address of a contiguous CUDA tensor (None stays None). Anything else is
    refused here: the library would read a host address or a strided view as a dense
    device array."""
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError(f"{what} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{what} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{what} must be {dtype}, got {t.dtype}")
    return ctypes.c_void_p(t.data_ptr())


def _dev(t, what):
    return _ptr(t, None, what)


def _i32(t, what):
    return _ptr(t, _I32, what)


def _f32(t, what):
    return _ptr(t, _F32, what)


def _stream(stream):
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _append_arg(append):
    """``append`` is None or ``(k_new, v_new, lens_out_or_None[, rope_base])``: device
    tensors, and the rotary base (0 or absent: no rotation)."""
    if append is None:
        return None
    k_new, v_new, lens_out = append[:3]
    rope_base = float(append[3]) if len(append) > 3 else 0.0
    kp, vp = _dev(k_new, "k_new"), _dev(v_new, "v_new")
    lp = _i32(lens_out, "lens_out")
    return ctypes.byref(NewTokens(kp.value, vp.value, None if lp is None else lp.value,
                                  rope_base))


def _check(status: int, call: str):
    if status != KVD_OK:
        raise KvdError(status, call)


def make_cache(k: torch.Tensor, v: torch.Tensor) -> Cache:
    """Describe one layer's ``[batch, heads, capacity, 64]`` K/V tensors for the C ABI."""
    shape, st = k.shape, k.stride()
    if shape != v.shape or st != v.stride() or k.dtype != v.dtype:
        raise ValueError("K and V must share shape, strides and dtype")
    if len(shape) != 4 or shape[3] != HEAD_DIM or st[3] != 1:
        raise ValueError("cache must be [batch, heads, capacity, 64] with the last axis contiguous")
    if not (k.is_cuda and v.is_cuda):
        raise ValueError("cache tensors must be CUDA tensors")
    if k.get_device() != v.get_device():
        raise ValueError("K and V must be on one device")
    B, H, cap, D = shape
    c = Cache(k.data_ptr(), v.data_ptr(), st[0], st[1], st[2], B, H, D, cap)
    c._tensors = (k, v)  # the struct holds raw pointers: keep the tensors alive with it
    return c


def kvd_version() -> int:
    return load_library().kvd_version()


def kvd_status_string(status: int) -> str:
    return load_library().kvd_status_string(status).decode()


def kvd_workspace_size(op: int, batch: int, n_q_heads: int = 1, n_kv_heads: int = 1,
                       rows_per_kv: int = 1, qlen: int = 1, max_len: int = 0,
                       vocab: int = 0) -> int:
    return load_library().kvd_workspace_size(op, batch, n_q_heads, n_kv_heads, rows_per_kv, qlen,
                                             max_len, vocab)


def new_workspace(nbytes: int, device=None) -> torch.Tensor:
    """A zero-filled device workspace (the counter region must start at zero)."""
    return torch.zeros(max(int(nbytes), KVD_WS_COUNTER_BYTES), dtype=torch.uint8,
                       device=device or "cuda")


def kvd_kv_append(cache: Cache, k_new, v_new, lens_in, lens_out=None, flags: int = 0,
                  dev_err=None, stream=None):
    B, H, q, D = k_new.shape
    _check(load_library().kvd_kv_append(_dtype_code(k_new), ctypes.byref(cache), B, q,
                                        _dev(k_new, "k_new"), _dev(v_new, "v_new"),
                                        _i32(lens_in, "lens_in"), _i32(lens_out, "lens_out"), flags,
                                        _i32(dev_err, "dev_err"), _stream(stream)), "kvd_kv_append")


def kvd_kv_append_rope(cache: Cache, k_new, v_new, lens_in, lens_out=None,
                       rope_base: float = 10000.0, flags: int = 0, dev_err=None, stream=None):
    B, H, q, D = k_new.shape
    _check(load_library().kvd_kv_append_rope(_dtype_code(k_new), ctypes.byref(cache), B, q,
                                             _dev(k_new, "k_new"), _dev(v_new, "v_new"),
                                             _i32(lens_in, "lens_in"), _i32(lens_out, "lens_out"),
                                             rope_base, flags, _i32(dev_err, "dev_err"),
                                             _stream(stream)), "kvd_kv_append_rope")


def kvd_decode_attn(q, cache: Cache, out, workspace, lens=None, fixed_len: int = 0,
                    rows_per_kv: int = 1, scale: float = 0.125, flags: int = 0,
                    dev_err=None, stream=None, append=None):
    B, Hq, ql, D = q.shape
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(load_library().kvd_decode_attn(_dtype_code(q), B, Hq, _dev(q, "q"), ctypes.byref(cache),
                                          _i32(lens, "lens"), fixed_len, _append_arg(append),
                                          rows_per_kv, scale, _dev(out, "out"),
                                          _dev(workspace, "workspace"), ws_bytes, flags,
                                          _i32(dev_err, "dev_err"), _stream(stream)),
           "kvd_decode_attn")


def kvd_decode_attn_noalloc(q, cache: Cache, out, lens=None, fixed_len: int = 0,
                            rows_per_kv: int = 1, scale: float = 0.125, flags: int = 0,
                            dev_err=None, stream=None, append=None):
    """kvd_decode_attn without a workspace: the library's built-in scratch is used."""
    B, Hq, ql, D = q.shape
    _check(load_library().kvd_decode_attn_noalloc(_dtype_code(q), B, Hq, _dev(q, "q"),
                                                  ctypes.byref(cache), _i32(lens, "lens"),
                                                  fixed_len, _append_arg(append), rows_per_kv,
                                                  scale, _dev(out, "out"), flags,
                                                  _i32(dev_err, "dev_err"), _stream(stream)),
           "kvd_decode_attn_noalloc")


def kvd_noalloc_test_fill_counters(byte_value: int, stream=None):
    """Test support: fill the built-in scratch's arrival counters with ``byte_value``."""
    _check(load_library().kvd_noalloc_test_fill_counters(byte_value, _stream(stream)),
           "kvd_noalloc_test_fill_counters")


def kvd_verify_attn(q, cache: Cache, out, workspace, lens=None, fixed_len: int = 0,
                    rows_per_kv: int = 1, causal: bool = True, scale: float = 0.125,
                    flags: int = 0, dev_err=None, stream=None, append=None):
    B, Hq, ql, D = q.shape
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(load_library().kvd_verify_attn(_dtype_code(q), B, Hq, ql, _dev(q, "q"),
                                          ctypes.byref(cache), _i32(lens, "lens"), fixed_len,
                                          _append_arg(append), rows_per_kv, int(bool(causal)),
                                          scale, _dev(out, "out"), _dev(workspace, "workspace"),
                                          ws_bytes, flags, _i32(dev_err, "dev_err"),
                                          _stream(stream)), "kvd_verify_attn")


def kvd_prefill_attn(q, cache: Cache, k_new, v_new, plens, out, lens_in=None, lens_out=None,
                     scale: float = 0.125, rope_base: float = 0.0, flags: int = 0,
                     dev_err=None, stream=None):
    """Prefill: append the prompt's K/V (rows j < plens[b]) and run causal attention of
    the prompt. q, out: [batch, n_q_heads, max_len, 64]; k_new, v_new: [batch,
    n_kv_heads, max_len, 64]. rope_base > 0: rotary encoding of the prompt."""
    B, Hq, T, D = q.shape
    _check(load_library().kvd_prefill_attn(_dtype_code(q), B, Hq, T, _dev(q, "q"),
                                           ctypes.byref(cache), _dev(k_new, "k_new"),
                                           _dev(v_new, "v_new"), _i32(lens_in, "lens_in"),
                                           _i32(plens, "plens"), _i32(lens_out, "lens_out"), scale,
                                           rope_base, _dev(out, "out"), flags,
                                           _i32(dev_err, "dev_err"), _stream(stream)),
           "kvd_prefill_attn")


def kvd_rope(q=None, k=None, pos0=None, base: float = 10000.0, flags: int = 0, dev_err=None,
             stream=None):
    """Rotary encoding, in place, of q [batch, n_q_heads, n, 64] and/or k [batch,
    n_k_heads, n, 64]; token j of row b at position pos0[b] + j."""
    ref = q if q is not None else k
    B, _, n, _ = ref.shape
    _check(load_library().kvd_rope(_dtype_code(ref), B, n, _dev(q, "q"),
                                   0 if q is None else q.shape[1], _dev(k, "k"),
                                   0 if k is None else k.shape[1], _i32(pos0, "pos0"), base, flags,
                                   _i32(dev_err, "dev_err"), _stream(stream)), "kvd_rope")


def kvd_greedy_accept(logits, draft, n_accepted, next_token, workspace, n_min=None,
                      argmax=None, flags: int = 0, dev_err=None, stream=None):
    B, k1, V = logits.shape
    ws_bytes = workspace.numel() * workspace.element_size()
    _check(load_library().kvd_greedy_accept(_f32(logits, "logits"), B, k1 - 1, V,
                                            _i32(draft, "draft"), _i32(n_accepted, "n_accepted"),
                                            _i32(next_token, "next_token"), _i32(n_min, "n_min"),
                                            _i32(argmax, "argmax"), _dev(workspace, "workspace"),
                                            ws_bytes, flags, _i32(dev_err, "dev_err"),
                                            _stream(stream)), "kvd_greedy_accept")


def kvd_beam_reorder_kv(caches, rows: int, beam: int, parent, lens=None, fixed_len: int = 0,
                        dtype=torch.float16, flags: int = 0, dev_err=None, stream=None):
    arr = (Cache * len(caches))(*caches)
    code = KVD_F16 if dtype == torch.float16 else KVD_BF16
    _check(load_library().kvd_beam_reorder_kv(code, arr, len(caches), rows, beam,
                                              _i32(parent, "parent"), _i32(lens, "lens"), fixed_len,
                                              flags, _i32(dev_err, "dev_err"), _stream(stream)),
           "kvd_beam_reorder_kv")


def kvd_beam_select(logits, beam: int, *, cum=None, suppress=None, blank=None,
                    eot: int = 0, first_step: bool = False, row_token=None, row_logprob=None,
                    parent=None, token=None, new_cum=None, n_finished=None, fin_parent=None,
                    fin_score=None, flags: int = 0, dev_err=None, stream=None):
    """Logit filters + one beam-search selection step over ``logits [windows*beam, V]``.

    ``suppress``/``blank`` are int32 CUDA tensors of ids; the walk outputs (``parent``
    ... ``fin_score``) are all given or all None.
    """
    rows, V = logits.shape
    n_sup = 0 if suppress is None else suppress.numel()
    n_blank = 0 if blank is None else blank.numel()
    _check(load_library().kvd_beam_select(_f32(logits, "logits"), rows // beam, beam, V,
                                          _f32(cum, "cum"), _i32(suppress, "suppress"), n_sup,
                                          _i32(blank, "blank"), n_blank, eot, int(bool(first_step)),
                                          _i32(row_token, "row_token"),
                                          _f32(row_logprob, "row_logprob"), _i32(parent, "parent"),
                                          _i32(token, "token"), _f32(new_cum, "new_cum"),
                                          _i32(n_finished, "n_finished"),
                                          _i32(fin_parent, "fin_parent"),
                                          _f32(fin_score, "fin_score"), flags,
                                          _i32(dev_err, "dev_err"), _stream(stream)),
           "kvd_beam_select")


def kvd_sample_accept(target, u, n_accepted, next_token, workspace, temperature: float = 1.0,
                      draft=None, drafts=None, r=None, flags: int = 0, dev_err=None,
                      stream=None):
    """Temperature sampling (target [B, 1, V]) or stochastic speculative acceptance of k
    drafts (target [B, k+1, V], draft [B, k, V], drafts and r [B, k]); u: [B] uniforms;
    workspace: kvd_workspace_size(KVD_OP_SAMPLE_ACCEPT, B, qlen=k, vocab=V) bytes."""
    B, k1, V = target.shape
    ws_bytes = workspace.numel() * workspace.element_size()
    _check(load_library().kvd_sample_accept(_f32(target, "target"), _f32(draft, "draft"),
                                            _i32(drafts, "drafts"), B, k1 - 1, V, temperature,
                                            _f32(r, "r"), _f32(u, "u"),
                                            _i32(n_accepted, "n_accepted"),
                                            _i32(next_token, "next_token"),
                                            _dev(workspace, "workspace"), ws_bytes, flags,
                                            _i32(dev_err, "dev_err"), _stream(stream)),
           "kvd_sample_accept")


# The current device and its current stream as plain numbers: torch.cuda.current_stream()
# builds a Stream object, 3 us of a decode step's launch.
_raw_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda dev: torch.cuda.current_stream(dev).cuda_stream)


def _refuse(t, dtype, shape, what, dev):
    if not t.is_cuda:
        raise ValueError(f"{what} must be a CUDA tensor")
    if t.get_device() != dev:
        raise ValueError(f"{what} must be on the current device (cuda:{dev})")
    if t.dtype != dtype:
        raise TypeError(f"{what} must be {dtype}, got {t.dtype}")
    if shape is not None and tuple(t.shape) != shape:
        raise ValueError(f"{what} must be {list(shape)}, got {list(t.shape)}")
    raise ValueError(f"{what} must be contiguous")


def _at(t, dtype, shape, what, dev):
    """The address (an int, 0 for None) of a contiguous CUDA tensor of this type and shape on
    device ``dev``; the argument checks of the calls below."""
    if t is None:
        return 0
    if (t.get_device() != dev or t.dtype != dtype or (shape is not None and t.shape != shape)
            or not t.is_contiguous()):
        _refuse(t, dtype, shape, what, dev)
    return t.data_ptr()


def _scratch(workspace, dev):
    if workspace is None:
        return 0, 0
    if workspace.get_device() != dev or not workspace.is_contiguous():
        _refuse(workspace, workspace.dtype, None, "workspace", dev)
    return workspace.data_ptr(), workspace.nbytes


def _device_of(t, what):
    """The tensor's device index, which must be the current device: kernels are launched
    there."""
    dev = t.get_device()
    if dev < 0:
        raise ValueError(f"{what} must be a CUDA tensor")
    if dev != _raw_device():
        raise ValueError(f"{what} is on cuda:{dev}, which is not the current device")
    return dev


def _on(stream, dev):
    if stream is None:
        return _raw_stream(dev)
    if stream.device_index != dev:
        raise ValueError(f"the stream is on cuda:{stream.device_index}, the tensors on cuda:{dev}")
    return stream.cuda_stream


def _cache_on(cache, dev, dtype=None):
    """The cache's tensors (kept with the struct) are on the current device and of this
    type."""
    held = getattr(cache, "_tensors", None)
    if held is not None:  # they share device and type
        t = held[0]
        if t.get_device() != dev:
            raise ValueError(f"cache must be on the current device (cuda:{dev})")
        if dtype is not None and t.dtype != dtype:
            raise TypeError(f"cache must be {dtype}, got {t.dtype}")
    return ctypes.byref(cache)


def _strides(t):
    """Element strides of the first three axes of a 4-D tensor; 0 for an axis of size 1 (its
    stride is arbitrary and never used)."""
    st, sh = t.stride(), t.shape
    return tuple(0 if sh[i] == 1 else st[i] for i in range(3))


def make_q4_cache(k: torch.Tensor, v: torch.Tensor, params: torch.Tensor) -> Q4Cache:
    """Describe one layer's 4-bit K/V for the C ABI: ``k`` and ``v`` uint8 ``[batch, heads,
    capacity, 32]`` (dims 2j and 2j+1 in the low and high half of byte j), ``params`` int16
    ``[batch, heads, capacity, 4]`` (the bits of K's step and zero point, V's step and zero
    point). Positions of a head must be consecutive; the three share their layout."""
    if k.dtype != torch.uint8 or v.dtype != torch.uint8 or params.dtype != torch.int16:
        raise TypeError("k and v must be uint8, params int16")
    shape = k.shape
    if (len(shape) != 4 or shape[3] != HEAD_DIM // 2 or v.shape != shape
            or params.shape != (*shape[:3], 4)):
        raise ValueError("k and v must be [batch, heads, capacity, 32], params [batch, heads, "
                         "capacity, 4]")
    dev = k.get_device()
    if dev < 0 or v.get_device() != dev or params.get_device() != dev:
        raise ValueError("cache tensors must be CUDA tensors on one device")
    if k.is_contiguous() and v.is_contiguous() and params.is_contiguous():
        row = (shape[1] * shape[2], shape[2])
    else:
        rows = []
        for t in (k, v, params):
            sb, sh, st = _strides(t)
            n = t.shape[3]
            if t.stride(3) != 1 or (shape[2] > 1 and st != n) or sb % n or sh % n:
                raise ValueError("a head's positions must be consecutive rows")
            rows.append((sb // n, sh // n))
        if rows[0] != rows[1] or rows[0] != rows[2]:
            raise ValueError("k, v and params must share their strides")
        row = rows[0]
    B, H, cap, _ = k.shape
    c = Q4Cache(k.data_ptr(), v.data_ptr(), params.data_ptr(), row[0], row[1], B, H, HEAD_DIM, cap)
    c._tensors = (k, v, params)  # the struct holds raw pointers: keep the tensors alive
    return c


def new_q4_cache(batch: int, n_kv_heads: int, capacity: int, device=None) -> Q4Cache:
    """A zero-filled 4-bit cache (its tensors: ``cache._tensors``)."""
    dev = device or "cuda"
    shape = (batch, n_kv_heads, capacity)
    return make_q4_cache(torch.zeros(*shape, HEAD_DIM // 2, dtype=torch.uint8, device=dev),
                         torch.zeros(*shape, HEAD_DIM // 2, dtype=torch.uint8, device=dev),
                         torch.zeros(*shape, 4, dtype=torch.int16, device=dev))


def _head_rows(x, out, weight, dtype, n, what, dev):
    if x is None:
        if out is not None or weight is not None:
            raise ValueError(f"{what}_out and {what}_weight need {what}")
        return None
    if x.get_device() != dev:
        raise ValueError(f"{what} must be on the current device (cuda:{dev})")
    if x.dtype != dtype:
        raise TypeError(f"{what} must be {dtype}, got {x.dtype}")
    shape, st = x.shape, x.stride()
    if len(shape) != 4 or shape[3] != HEAD_DIM or st[3] != 1:
        raise ValueError(f"{what} must be [batch, heads, n, 64] with the last axis contiguous")
    B, H = shape[0], shape[1]
    # (the stride of an axis of size 1 is arbitrary and never used)
    return HeadRows(x.data_ptr(), st[0] if B > 1 else 0, st[1] if H > 1 else 0,
                    st[2] if n > 1 else 0, _at(weight, dtype, (HEAD_DIM,), what + "_weight", dev),
                    _at(out, dtype, (B, H, n, HEAD_DIM), what + "_out", dev), H)


def kvd_qk_norm_rope(q=None, k=None, q_out=None, k_out=None, q_weight=None, k_weight=None,
                     pos0=None, eps: float = 1e-6, base: float = 10000.0, flags: int = 0,
                     dev_err=None, stream=None):
    """RMS norm of each query and key head, then the rotation at position ``pos0[b] + j``, in
    one pass: ``q [batch, n_q_heads, n, 64]`` and/or ``k [batch, n_k_heads, n, 64]`` of any
    strides (a view of a fused projection) into contiguous ``q_out`` / ``k_out`` (``q`` and
    ``k`` themselves when contiguous). ``base`` 0: norm only."""
    ref = q if q is not None else k
    if ref is None:
        raise ValueError("q or k is needed")
    if ref.dim() != 4:
        raise ValueError("q and k must be [batch, heads, n, 64]")
    dev = _device_of(ref, "q" if q is not None else "k")
    B, _, n, _ = ref.shape
    if q is not None and k is not None and (k.shape[0] != B or k.shape[2] != n):
        raise ValueError("q and k must share batch and n")
    if (q is not None and q_out is None) or (k is not None and k_out is None):
        raise ValueError("q_out (k_out) is needed with q (k)")
    rq = _head_rows(q, q_out, q_weight, ref.dtype, n, "q", dev)
    rk = _head_rows(k, k_out, k_weight, ref.dtype, n, "k", dev)
    _check(load_library().kvd_qk_norm_rope(
        _dtype_code(ref), B, n, None if rq is None else ctypes.byref(rq),
        None if rk is None else ctypes.byref(rk), _at(pos0, _I32, (B,), "pos0", dev), eps, base,
        flags, _at(dev_err, _I32, None, "dev_err", dev), _on(stream, dev)), "kvd_qk_norm_rope")


def _query_shape(q, out, dev):
    shape = q.shape
    if len(shape) != 4 or shape[3] != HEAD_DIM:
        raise ValueError("q must be [batch, n_q_heads, qlen, 64]")
    if not q.is_contiguous():  # (its device is dev)
        raise ValueError("q must be contiguous")
    return shape, q.data_ptr(), _at(out, q.dtype, shape, "out", dev)


def kvd_window_attn(q, cache: Cache, out, workspace, window: int, n_sinks: int = 0, lens=None,
                    fixed_len: int = 0, scale: float = 0.125, flags: int = 0, dev_err=None,
                    stream=None, append=None):
    """``kvd_decode_attn`` (one query token per row) or the causal ``kvd_verify_attn`` (up to
    16) through a sliding window: the query at position p sees t <= p with t < n_sinks or
    t > p - window. workspace: kvd_workspace_size(KVD_OP_WINDOW_ATTN, ...) bytes."""
    dev = _device_of(q, "q")
    (B, Hq, ql, _), qp, op = _query_shape(q, out, dev)
    ws, ws_bytes = _scratch(workspace, dev)
    if append is not None:
        for t, what in zip(append[:3], ("k_new", "v_new", "lens_out")):
            dt, sh = (_I32, (B,)) if what == "lens_out" else (
                q.dtype, (B, cache.n_kv_heads, ql, HEAD_DIM))
            _at(t, dt, sh, what, dev)
    _check(load_library().kvd_window_attn(
        _dtype_code(q), B, Hq, ql, qp, _cache_on(cache, dev, q.dtype),
        _at(lens, _I32, (B,), "lens", dev), fixed_len, _append_arg(append), window, n_sinks, scale,
        op, ws, ws_bytes, flags, _at(dev_err, _I32, None, "dev_err", dev), _on(stream, dev)),
        "kvd_window_attn")


def kvd_prefill_window_attn(q, cache: Cache, k_new, v_new, plens, out, window: int,
                            n_sinks: int = 0, lens_in=None, lens_out=None, scale: float = 0.125,
                            rope_base: float = 0.0, flags: int = 0, dev_err=None, stream=None):
    """``kvd_prefill_attn`` through a sliding window with sinks."""
    dev = _device_of(q, "q")
    (B, Hq, T, _), qp, op = _query_shape(q, out, dev)
    kv = (B, cache.n_kv_heads, T, HEAD_DIM)
    _check(load_library().kvd_prefill_window_attn(
        _dtype_code(q), B, Hq, T, qp, _cache_on(cache, dev, q.dtype),
        _at(k_new, q.dtype, kv, "k_new", dev), _at(v_new, q.dtype, kv, "v_new", dev),
        _at(lens_in, _I32, (B,), "lens_in", dev), _at(plens, _I32, (B,), "plens", dev),
        _at(lens_out, _I32, (B,), "lens_out", dev), window, n_sinks, scale, rope_base, op, flags,
        _at(dev_err, _I32, None, "dev_err", dev), _on(stream, dev)), "kvd_prefill_window_attn")


def kvd_q4_append(cache: Q4Cache, k_new, v_new, lens_in=None, lens_out=None, counts=None,
                  flags: int = 0, dev_err=None, stream=None):
    """Quantise ``k_new``, ``v_new`` ``[batch, n_kv_heads, q, 64]`` and write row b's first
    ``counts[b]`` tokens (all q without ``counts``) at positions ``lens_in[b]`` on."""
    dev = _device_of(k_new, "k_new")
    if k_new.dim() != 4:
        raise ValueError("k_new must be [batch, n_kv_heads, q, 64]")
    B, _, n, _ = k_new.shape
    shape = (B, cache.n_kv_heads, n, HEAD_DIM)
    _check(load_library().kvd_q4_append(
        _dtype_code(k_new), _cache_on(cache, dev), B, n,
        _at(k_new, k_new.dtype, shape, "k_new", dev), _at(v_new, k_new.dtype, shape, "v_new", dev),
        _at(lens_in, _I32, (B,), "lens_in", dev), _at(counts, _I32, (B,), "counts", dev),
        _at(lens_out, _I32, (B,), "lens_out", dev), flags,
        _at(dev_err, _I32, None, "dev_err", dev), _on(stream, dev)), "kvd_q4_append")


def kvd_q4_dequant(cache: Q4Cache, k_out=None, v_out=None, pos0=None, flags: int = 0,
                   dev_err=None, stream=None):
    """Read positions ``pos0[b] ..`` of a 4-bit cache back into ``k_out`` and/or ``v_out``,
    ``[batch, n_kv_heads, n, 64]``."""
    ref = k_out if k_out is not None else v_out
    if ref is None or ref.dim() != 4:
        raise ValueError("k_out or v_out [batch, n_kv_heads, n, 64] is needed")
    dev = _device_of(ref, "k_out" if k_out is not None else "v_out")
    B, _, n, _ = ref.shape
    shape = (B, cache.n_kv_heads, n, HEAD_DIM)
    _check(load_library().kvd_q4_dequant(
        _dtype_code(ref), _cache_on(cache, dev), B, n, _at(k_out, ref.dtype, shape, "k_out", dev),
        _at(v_out, ref.dtype, shape, "v_out", dev), _at(pos0, _I32, (B,), "pos0", dev), flags,
        _at(dev_err, _I32, None, "dev_err", dev), _on(stream, dev)), "kvd_q4_dequant")


def kvd_q4_attn(q, cache: Q4Cache, out, workspace=None, lens=None, fixed_len: int = 0,
                causal: bool = True, window: int = 0, n_sinks: int = 0, scale: float = 0.125,
                flags: int = 0, dev_err=None, stream=None):
    """Attention of 1..16 query tokens per row over a 4-bit cache (the block's K/V already
    appended). ``window`` > 0: a sliding window with ``n_sinks`` sinks. workspace:
    kvd_workspace_size(KVD_OP_Q4_ATTN, ...) bytes; calls with much work (many rows over a large
    capacity) need it, for the others it may be None."""
    dev = _device_of(q, "q")
    (B, Hq, ql, _), qp, op = _query_shape(q, out, dev)
    ws, ws_bytes = _scratch(workspace, dev)
    _check(load_library().kvd_q4_attn(
        _dtype_code(q), B, Hq, ql, qp, _cache_on(cache, dev), _at(lens, _I32, (B,), "lens", dev),
        fixed_len, int(bool(causal)), window, n_sinks, scale, op, ws, ws_bytes, flags,
        _at(dev_err, _I32, None, "dev_err", dev), _on(stream, dev)), "kvd_q4_attn")


def kvd_sample_filtered(logits, u, token, temperature=None, top_k=None, top_p=None, min_p=None,
                        logprob=None, n_kept=None, flags: int = 0, dev_err=None, stream=None):
    """Draw one token per row of ``logits [batch, vocab]`` (rows may be strided) after
    temperature, top-k, top-p and min-p, each an optional ``[batch]`` tensor; ``u [batch]``
    are the caller's uniforms in [0, 1)."""
    if logits.dim() != 2 or logits.stride(1) != 1:
        raise ValueError("logits must be [batch, vocab] with contiguous rows")
    if logits.dtype != _F32:
        raise TypeError(f"logits must be {_F32}, got {logits.dtype}")
    dev = _device_of(logits, "logits")
    B, V = logits.shape
    row = logits.stride(0) if B > 1 else V
    b = (B,)
    _check(load_library().kvd_sample_filtered(
        logits.data_ptr(), row, B, V, _at(temperature, _F32, b, "temperature", dev),
        _at(top_k, _I32, b, "top_k", dev), _at(top_p, _F32, b, "top_p", dev),
        _at(min_p, _F32, b, "min_p", dev), _at(u, _F32, b, "u", dev),
        _at(token, _I32, b, "token", dev), _at(logprob, _F32, b, "logprob", dev),
        _at(n_kept, _I32, b, "n_kept", dev), flags, _at(dev_err, _I32, None, "dev_err", dev),
        _on(stream, dev)), "kvd_sample_filtered")
