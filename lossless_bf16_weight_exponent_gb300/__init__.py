"""Python binding of ``libuw.so`` - the C ABI declared in ``include/uw.h``.

Argument marshalling only: every step of the codec and the matmul runs in the
library's own host code and CUDA kernels.  PyTorch is used by callers for device
memory and streams; this module accepts torch tensors (or raw integer device
addresses) and passes plain pointers.  There is no CPU fallback: if the library
is missing, importing works but the first call raises.
"""
from __future__ import annotations

import ctypes
import os
import re

import numpy as np

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libuw.so")
HEADER = os.path.join(os.path.dirname(_HERE), "include", "uw.h")

# enums (mirrors of include/uw.h)
OK, ERR_INVALID_ARG, ERR_SHAPE, ERR_UNSUPPORTED, ERR_CORRUPT = 0, 1, 2, 3, 4
ERR_NO_MEMORY, ERR_WORKSPACE, ERR_CUDA, ERR_TIMEOUT, ERR_BUFFER_TOO_SMALL = 5, 6, 7, 8, 9
CODEC_PALETTE, CODEC_HUFFMAN = 0, 1
STRAT_AUTO, STRAT_FULL_DECODE, STRAT_EXP_ONLY, STRAT_PALETTE_TRANSCODE, STRAT_DIRECT_PALETTE = 0, 1, 2, 3, 4
STRAT_HUFFMAN_DIRECT = 5
STRATEGIES = {"full_decode": 1, "exp_only": 2, "palette_transcode": 3, "direct_palette": 4, "huffman_direct": 5}
OUT_F32, OUT_BF16 = 0, 1
KERNEL_AUTO, KERNEL_GEMV, KERNEL_TC = 0, 1, 2
RESIDENT_HUFFMAN, RESIDENT_BOTH, RESIDENT_PALETTE = 0, 1, 2
RESIDENT = {"huffman": RESIDENT_HUFFMAN, "both": RESIDENT_BOTH, "palette": RESIDENT_PALETTE}
SCORE_SOFTMAX, SCORE_SIGMOID = 0, 1
SCORE_CHOOSES = 16  # added to either: the choice is by score + bias in place of logit + bias
ROTARY_HALF, ROTARY_INTERLEAVED = 0, 1
ROTARY_PLAIN, ROTARY_LINEAR, ROTARY_STRETCHED, ROTARY_BANDS, ROTARY_RAMP = 0, 1, 2, 3, 4
SEQ_DIRECT = -1  # uw_sequence_run schedule: no side-stream transcode, every step its own AUTO plan
STEP_CONCURRENT = 1  # uw_step flag: the step may overlap the step before it
SEQ_GROUPS = 65536  # added to a uw_sequence_run schedule: overlap the groups of STEP_CONCURRENT steps


class UwError(RuntimeError):
    def __init__(self, status: int, where: str, message: str):
        super().__init__(f"{where}: status {status} ({message})")
        self.status = status
        self.message = message


class EncodeOpts(ctypes.Structure):
    _fields_ = [("codec", ctypes.c_uint32), ("chunk_weights", ctypes.c_uint32), ("max_code_len", ctypes.c_uint32)]


class Plan(ctypes.Structure):
    _fields_ = [("strategy", ctypes.c_int32), ("kernel", ctypes.c_int32), ("split_k", ctypes.c_int32),
                ("variant", ctypes.c_int32)]

    def as_tuple(self):
        return (self.strategy, self.kernel, self.split_k, self.variant)

    def __repr__(self):
        return f"Plan(strategy={self.strategy}, kernel={self.kernel}, split_k={self.split_k}, variant={self.variant})"


class Step(ctypes.Structure):
    _fields_ = [("m", ctypes.c_void_p), ("x", ctypes.c_void_p), ("y", ctypes.c_void_p), ("out_dtype", ctypes.c_int32),
                ("flags", ctypes.c_int32)]


class Info(ctypes.Structure):
    _fields_ = [("N", ctypes.c_int64), ("K", ctypes.c_int64), ("codec", ctypes.c_uint32), ("n_pal", ctypes.c_uint32),
                ("palette", ctypes.c_uint8 * 16), ("code_len", ctypes.c_uint8 * 16),
                ("n_blocks", ctypes.c_uint64), ("n_verbatim", ctypes.c_uint64), ("n_chunks", ctypes.c_uint64),
                ("total_bits", ctypes.c_uint64), ("blob_bytes", ctypes.c_uint64), ("device_bytes", ctypes.c_uint64),
                ("has_palette_form", ctypes.c_int32), ("chunk_weights", ctypes.c_int32),
                ("max_code_len", ctypes.c_int32), ("has_huffman_stream", ctypes.c_int32)]

    def as_dict(self):
        d = {f: getattr(self, f) for f, _ in self._fields_}
        d["palette"] = list(self.palette)
        d["code_len"] = list(self.code_len)
        return d


class GroupInfo(ctypes.Structure):
    _fields_ = [("N", ctypes.c_int64), ("K", ctypes.c_int64), ("experts", ctypes.c_int32), ("gated", ctypes.c_int32),
                ("n_verbatim", ctypes.c_uint64), ("device_bytes", ctypes.c_uint64)]

    def as_dict(self):
        return {f: getattr(self, f) for f, _ in self._fields_}


class RouterDesc(ctypes.Structure):
    _fields_ = [("experts", ctypes.c_int32), ("topk", ctypes.c_int32), ("score", ctypes.c_int32),
                ("renormalize", ctypes.c_int32), ("scale", ctypes.c_float), ("bias", ctypes.c_void_p)]


class NormDesc(ctypes.Structure):
    _fields_ = [("dim", ctypes.c_int64), ("post_weight", ctypes.c_void_p), ("gate", ctypes.c_void_p),
                ("gate_every", ctypes.c_int64), ("pre_weight", ctypes.c_void_p), ("res_scale", ctypes.c_float),
                ("out_scale", ctypes.c_float), ("eps", ctypes.c_float), ("res_dtype", ctypes.c_int32),
                ("block_dtype", ctypes.c_int32)]


class RotaryDesc(ctypes.Structure):
    _fields_ = [("dim", ctypes.c_int32), ("layout", ctypes.c_int32), ("freq", ctypes.c_void_p), ("scale", ctypes.c_float)]


class KVDesc(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("pages", ctypes.c_int64), ("page_stride", ctypes.c_int64),
                ("slot_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64), ("page_size", ctypes.c_int32), ("kv_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32)]


class KVBatchDesc(ctypes.Structure):
    _fields_ = [("sequences", ctypes.c_int32), ("starts", ctypes.c_void_p), ("lengths", ctypes.c_void_p), ("pages", ctypes.c_void_p),
                ("ld_pages", ctypes.c_int64), ("max_pages", ctypes.c_int64)]


class LogitEditsDesc(ctypes.Structure):
    _fields_ = [("tokens", ctypes.c_void_p), ("ld_tokens", ctypes.c_int64), ("max_tokens", ctypes.c_int64), ("lengths", ctypes.c_void_p),
                ("prompt_lengths", ctypes.c_void_p), ("repetition", ctypes.c_void_p), ("frequency", ctypes.c_void_p), ("presence", ctypes.c_void_p),
                ("bias_ids", ctypes.c_void_p), ("bias", ctypes.c_void_p), ("bias_lengths", ctypes.c_void_p), ("max_bias", ctypes.c_int64),
                ("allowed", ctypes.c_void_p), ("ld_allowed", ctypes.c_int64), ("mask_count", ctypes.c_int64), ("mask_rows", ctypes.c_void_p)]


_lib = None
_VP, _SZ, _I64, _INT = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int64, ctypes.c_int

_SIGS = {
    "uw_encode": [_VP, _I64, _I64, ctypes.POINTER(EncodeOpts), _VP, _SZ, ctypes.POINTER(_SZ)],
    "uw_load": [_VP, _SZ, _INT, _VP, ctypes.POINTER(_VP)],
    "uw_blob_validate": [_VP, _SZ, ctypes.POINTER(Info)],
    "uw_free": [_VP],
    "uw_get_info": [_VP, ctypes.POINTER(Info)],
    "uw_decode": [_VP, _VP, _VP],
    "uw_workspace_size": [_VP, _I64, _INT, ctypes.POINTER(_SZ)],
    "uw_matmul": [_VP, _VP, _I64, _VP, _INT, _INT, _VP, _SZ, _VP],
    "uw_matmul_plan": [_VP, _VP, _I64, _VP, _INT, ctypes.POINTER(Plan), _VP, _SZ, _VP],
    "uw_plan_workspace_size": [_VP, _I64, ctypes.POINTER(Plan), ctypes.POINTER(_SZ)],
    "uw_plan_for": [_VP, _I64, ctypes.POINTER(Plan)],
    "uw_matmul_host": [_VP, _VP, _I64, _VP, _INT, _VP, _SZ, _VP],
    "uw_matmul_host_async": [_VP, _VP, _I64, _VP, _INT, _VP, _SZ, _VP],
    "uw_host_workspace_size": [_VP, _I64, _INT, ctypes.POINTER(_SZ)],
    "uw_autotune": [_VP, ctypes.POINTER(_I64), _INT, _VP, _SZ, _VP],
    "uw_autotune_workspace_size": [_VP, ctypes.POINTER(_I64), _INT, ctypes.POINTER(_SZ)],
    "uw_tune_save": [_VP, ctypes.c_char_p, _SZ, ctypes.POINTER(_SZ)],
    "uw_tune_load": [_VP, ctypes.c_char_p],
    "uw_check": [_VP, _VP],
    "uw_matmul_noalloc": [_VP, _VP, _I64, _VP, _INT, _VP],
    "uw_sequence_workspace_size": [ctypes.POINTER(Step), _INT, _I64, ctypes.POINTER(_SZ)],
    "uw_sequence_run": [ctypes.POINTER(Step), _INT, _I64, _VP, _SZ, _VP, _VP, _INT],
    "uw_sequence_tune": [ctypes.POINTER(Step), _INT, _I64, _VP, _SZ, _VP, _VP, ctypes.POINTER(_INT)],
    "uw_group_create": [ctypes.POINTER(_VP), ctypes.POINTER(_VP), _INT, _VP, ctypes.POINTER(_VP)],
    "uw_group_create_dense": [_VP, _VP, _INT, _I64, _I64, _VP, ctypes.POINTER(_VP)],
    "uw_group_free": [_VP],
    "uw_group_get_info": [_VP, ctypes.POINTER(GroupInfo)],
    "uw_group_decode": [_VP, _INT, _INT, _VP, _VP],
    "uw_group_matmul": [_VP, _VP, _I64, _I64, _VP, _VP, _I64, _VP, _I64, _INT, _VP],
    "uw_group_check": [_VP, _VP],
    "uw_route_workspace_size": [ctypes.POINTER(RouterDesc), _I64, ctypes.POINTER(_SZ)],
    "uw_route": [ctypes.POINTER(RouterDesc), _VP, _INT, _I64, _I64, _VP, _VP, _VP, _VP, _VP, _VP, _SZ, _VP],
    "uw_block_norm": [ctypes.POINTER(NormDesc), _I64, _VP, _VP, _VP, _I64, _VP, _VP, _INT, _VP, _VP],
    "uw_token_logprobs": [_VP, _INT, _I64, _I64, _I64, ctypes.c_float, _VP, _VP, _VP, _INT, _VP, _VP, _VP],
    "uw_rotary_frequencies": [_INT, ctypes.c_double, _INT, ctypes.c_double, ctypes.c_double, ctypes.c_double, _I64, _VP,
                              ctypes.POINTER(ctypes.c_float)],
    "uw_kv_create": [ctypes.POINTER(KVDesc), ctypes.POINTER(_VP)],
    "uw_kv_free": [_VP],
    "uw_kv_append": [_VP, ctypes.POINTER(KVBatchDesc), ctypes.POINTER(RotaryDesc), _I64, _INT, _VP, _I64, _INT, _VP, _I64, _VP, _I64, _VP, _VP, _I64,
                     _VP],
    "uw_kv_attend_workspace_size": [_VP, _INT, _I64, _INT, ctypes.POINTER(_SZ)],
    "uw_kv_attend": [_VP, ctypes.POINTER(KVBatchDesc), _I64, _VP, _I64, _INT, ctypes.c_float, _INT, _I64, _VP, _I64, _VP, _VP, _SZ, _VP],
    "uw_kv_check": [_VP, _VP],
    "uw_edit_logits": [ctypes.POINTER(LogitEditsDesc), _VP, _INT, _I64, _I64, _I64, _VP, _INT, _I64, _VP],
    "uw_status_string": [_INT],
    "uw_last_error": [],
    "uw_version": [],
}


def lib():
    """The loaded ``libuw.so``; raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with __graft_entry__.build()")
        L = ctypes.CDLL(LIB_PATH)
        for name, args in _SIGS.items():
            f = getattr(L, name)
            f.argtypes = args
            f.restype = _INT
        L.uw_free.restype = None
        L.uw_group_free.restype = None
        L.uw_kv_free.restype = None
        L.uw_status_string.restype = ctypes.c_char_p
        L.uw_last_error.restype = ctypes.c_char_p
        L.uw_version.restype = ctypes.c_char_p
        _lib = L
    return _lib


def header_symbols():
    """Entry points declared in include/uw.h."""
    text = open(HEADER).read()
    return sorted(set(re.findall(r"\b(uw_[a-z_0-9]+)\s*\(", text)))


def _check(status: int, where: str):
    if status != OK:
        raise UwError(status, where, lib().uw_last_error().decode(errors="replace"))


def _ptr(t) -> int:
    if t is None:
        return 0
    if isinstance(t, int):
        return t
    return t.data_ptr()


_ELEMENTS = {}  # element types of the tensors that a call of this type (OUT_F32, OUT_BF16) takes


def _typed(what: str, t, dtype: int) -> int:
    """_ptr of a tensor of the type that the call reads or writes; one of another type is refused.  Addresses pass, and so
    do types that the library refuses."""
    if t is None:
        return 0
    if isinstance(t, int):
        return t
    if not _ELEMENTS:
        import torch
        _ELEMENTS.update({OUT_F32: (torch.float32,), OUT_BF16: (torch.bfloat16, torch.int16, torch.uint16)})
    takes = _ELEMENTS.get(dtype)
    if takes and t.dtype not in takes:
        raise ValueError(f"{what} is {t.dtype}, the call's type is {('fp32', 'bf16')[dtype]}")
    return t.data_ptr()


_raw_stream = None  # the current stream's address by torch's own binding, a tenth of current_stream()'s cost, and that of the device


def _current_stream():
    global _raw_stream
    if _raw_stream is None:
        import torch
        torch.cuda.current_device()  # sets CUDA up
        raw, device = (getattr(torch._C, n, None) for n in ("_cuda_getCurrentRawStream", "_cuda_getDevice"))
        _raw_stream = (lambda: raw(device())) if raw and device else (lambda: torch.cuda.current_stream().cuda_stream)
    return _raw_stream()


def _stream(stream) -> int:
    if stream is None:
        return _current_stream()
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def encode(w: np.ndarray, codec: int = CODEC_PALETTE, chunk: int = 256, max_len: int = 12) -> bytes:
    """Host encode of W[N,K] (numpy uint16 bf16 bit patterns)."""
    w = np.ascontiguousarray(w, dtype=np.uint16)
    N, K = w.shape
    opts = EncodeOpts(codec, chunk, max_len)
    size = ctypes.c_size_t(0)
    _check(lib().uw_encode(w.ctypes.data, N, K, ctypes.byref(opts), None, 0, ctypes.byref(size)), "uw_encode")
    out = np.empty(size.value, np.uint8)
    _check(lib().uw_encode(w.ctypes.data, N, K, ctypes.byref(opts), out.ctypes.data, size.value, ctypes.byref(size)),
           "uw_encode")
    return out.tobytes()


def validate(blob: bytes) -> dict:
    info = Info()
    buf = np.frombuffer(blob, np.uint8)
    _check(lib().uw_blob_validate(buf.ctypes.data if len(blob) else None, len(blob), ctypes.byref(info)),
           "uw_blob_validate")
    return info.as_dict()


class Matrix:
    """A compressed matrix resident on the current CUDA device (owns a ``uw_matrix``)."""

    def __init__(self, blob: bytes, want_palette_form: bool = False, stream=None, resident=None):
        """resident: "huffman", "both" or "palette" (uw_resident); if None, want_palette_form picks "both" (True)
        or "huffman" (False)."""
        mode = RESIDENT[resident] if resident is not None else (RESIDENT_BOTH if want_palette_form else RESIDENT_HUFFMAN)
        buf = np.frombuffer(blob, np.uint8)
        h = ctypes.c_void_p()
        _check(lib().uw_load(buf.ctypes.data, len(blob), mode, _stream(stream), ctypes.byref(h)), "uw_load")
        self._h = h
        info = Info()
        _check(lib().uw_get_info(self._h, ctypes.byref(info)), "uw_get_info")
        self.info = info.as_dict()
        self.N, self.K = self.info["N"], self.info["K"]

    def close(self):
        if getattr(self, "_h", None):
            lib().uw_free(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    @property
    def handle(self):
        return self._h

    def decode(self, out, stream=None):
        _check(lib().uw_decode(self._h, _ptr(out), _stream(stream)), "uw_decode")

    def workspace_size(self, B: int, strategy: int = STRAT_AUTO) -> int:
        n = ctypes.c_size_t(0)
        _check(lib().uw_workspace_size(self._h, B, strategy, ctypes.byref(n)), "uw_workspace_size")
        return n.value

    def plan_workspace_size(self, B: int, plan: Plan) -> int:
        n = ctypes.c_size_t(0)
        _check(lib().uw_plan_workspace_size(self._h, B, ctypes.byref(plan), ctypes.byref(n)), "uw_plan_workspace_size")
        return n.value

    def matmul(self, x, B: int, y, out_dtype: int = OUT_F32, strategy: int = STRAT_AUTO, workspace=None,
               ws_bytes: int = 0, stream=None):
        _check(lib().uw_matmul(self._h, _ptr(x), B, _ptr(y), out_dtype, strategy, _ptr(workspace), ws_bytes,
                               _stream(stream)), "uw_matmul")

    def matmul_plan(self, x, B: int, y, plan: Plan, out_dtype: int = OUT_F32, workspace=None, ws_bytes: int = 0,
                    stream=None):
        _check(lib().uw_matmul_plan(self._h, _ptr(x), B, _ptr(y), out_dtype, ctypes.byref(plan), _ptr(workspace),
                                    ws_bytes, _stream(stream)), "uw_matmul_plan")

    def plan_for(self, B: int) -> Plan:
        p = Plan()
        _check(lib().uw_plan_for(self._h, B, ctypes.byref(p)), "uw_plan_for")
        return p

    def host_workspace_size(self, B: int, out_dtype: int = OUT_F32) -> int:
        n = ctypes.c_size_t(0)
        _check(lib().uw_host_workspace_size(self._h, B, out_dtype, ctypes.byref(n)), "uw_host_workspace_size")
        return n.value

    def matmul_host(self, x_host, B: int, y_host, out_dtype: int, workspace, ws_bytes: int, stream=None):
        _check(lib().uw_matmul_host(self._h, _ptr(x_host), B, _ptr(y_host), out_dtype, _ptr(workspace), ws_bytes,
                                    _stream(stream)), "uw_matmul_host")

    def matmul_host_async(self, x_host, B: int, y_host, out_dtype: int, workspace, ws_bytes: int, stream=None):
        _check(lib().uw_matmul_host_async(self._h, _ptr(x_host), B, _ptr(y_host), out_dtype, _ptr(workspace),
                                          ws_bytes, _stream(stream)), "uw_matmul_host_async")

    def autotune_workspace_size(self, batches) -> int:
        arr = (ctypes.c_int64 * len(batches))(*batches)
        n = ctypes.c_size_t(0)
        _check(lib().uw_autotune_workspace_size(self._h, arr, len(batches), ctypes.byref(n)), "uw_autotune_workspace_size")
        return n.value

    def autotune(self, batches, workspace, ws_bytes: int, stream=None):
        arr = (ctypes.c_int64 * len(batches))(*batches)
        _check(lib().uw_autotune(self._h, arr, len(batches), _ptr(workspace), ws_bytes, _stream(stream)), "uw_autotune")

    def tune_save(self) -> str:
        n = ctypes.c_size_t(0)
        _check(lib().uw_tune_save(self._h, None, 0, ctypes.byref(n)), "uw_tune_save")
        buf = ctypes.create_string_buffer(n.value + 1)
        _check(lib().uw_tune_save(self._h, buf, n.value + 1, ctypes.byref(n)), "uw_tune_save")
        return buf.value.decode()

    def tune_load(self, text: str):
        _check(lib().uw_tune_load(self._h, text.encode()), "uw_tune_load")

    def matmul_noalloc(self, x, B: int, y, out_dtype: int = OUT_F32, stream=None):
        _check(lib().uw_matmul_noalloc(self._h, _ptr(x), B, _ptr(y), out_dtype, _stream(stream)), "uw_matmul_noalloc")

    def check(self, stream=None):
        _check(lib().uw_check(self._h, _stream(stream)), "uw_check")


def _steps(steps):
    arr = (Step * max(1, len(steps)))()
    for i, st in enumerate(steps):
        m, x, y = st[0], st[1], st[2]
        od = st[3] if len(st) > 3 else OUT_F32
        fl = st[4] if len(st) > 4 else 0
        arr[i] = Step(m.handle.value if isinstance(m, Matrix) else m, _ptr(x), _ptr(y), od, fl)
    return arr


def sequence_workspace_size(steps, B: int) -> int:
    """Workspace bytes of uw_sequence_run; steps: (Matrix, x, y[, out_dtype[, flags]]) tuples."""
    n = ctypes.c_size_t(0)
    _check(lib().uw_sequence_workspace_size(_steps(steps), len(steps), B, ctypes.byref(n)), "uw_sequence_workspace_size")
    return n.value


def sequence_run(steps, B: int, workspace, ws_bytes: int, stream=None, side_stream=None, decode_sms: int = 0):
    """uw_sequence_run: the steps in order on `stream`, hard steps' transcodes on `side_stream` (on `decode_sms`
    SMs beside the matmuls when it is > 0; SEQ_DIRECT: no transcode, every step its own AUTO plan)."""
    _check(lib().uw_sequence_run(_steps(steps), len(steps), B, _ptr(workspace), ws_bytes, _stream(stream),
                                 _stream(side_stream), decode_sms), "uw_sequence_run")


def sequence_tune(steps, B: int, workspace, ws_bytes: int, stream=None, side_stream=None) -> int:
    """uw_sequence_tune: the fastest decode SM split for these steps."""
    d = ctypes.c_int(0)
    _check(lib().uw_sequence_tune(_steps(steps), len(steps), B, _ptr(workspace), ws_bytes, _stream(stream),
                                  _stream(side_stream), ctypes.byref(d)), "uw_sequence_tune")
    return d.value


class Group:
    """The weight matrices of a layer's experts, compressed on the current CUDA device (owns a ``uw_group``).

    w: bf16 tensor [experts, N, K] on the device, or a list of loaded ``Matrix``; w_up: the same for the up matrices of
    a gated group, whose product is silu(W x) * (W_up x)."""

    def __init__(self, w, w_up=None, stream=None):
        h = ctypes.c_void_p()
        if isinstance(w, (list, tuple)):
            arr = [(ctypes.c_void_p * len(v))(*[m.handle for m in v]) if v is not None else None for v in (w, w_up)]
            if w_up is not None and len(w_up) != len(w):
                raise ValueError("w and w_up differ in length")
            _check(lib().uw_group_create(arr[0], arr[1], len(w), _stream(stream), ctypes.byref(h)), "uw_group_create")
        else:
            for t in (w, w_up):
                if t is not None and (t.dim() != 3 or t.shape != w.shape or not t.is_contiguous() or not t.is_cuda):
                    raise ValueError("weights must be contiguous tensors [experts, N, K] of one shape on the device")
                _typed("weights", t, OUT_BF16)
            E, N, K = w.shape
            _check(lib().uw_group_create_dense(_ptr(w), _ptr(w_up), E, N, K, _stream(stream), ctypes.byref(h)),
                   "uw_group_create_dense")
        self._h = h
        info = GroupInfo()
        _check(lib().uw_group_get_info(self._h, ctypes.byref(info)), "uw_group_get_info")
        self.info = info.as_dict()
        self.N, self.K, self.experts = self.info["N"], self.info["K"], self.info["experts"]

    def close(self):
        if getattr(self, "_h", None):
            lib().uw_group_free(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    @property
    def handle(self):
        return self._h

    def decode(self, expert: int, out, up: bool = False, stream=None):
        _check(lib().uw_group_decode(self._h, expert, int(up), _ptr(out), _stream(stream)), "uw_group_decode")

    def matmul(self, x, offsets, rows: int, y, row_src=None, x_rows=None, out_dtype: int = OUT_BF16, ldx: int = 0,
               ldy: int = 0, stream=None):
        """uw_group_matmul; x_rows None: rows of x (a tensor).  y is bf16 unless out_dtype is OUT_F32."""
        _check(lib().uw_group_matmul(self._h, _ptr(x), x.shape[0] if x_rows is None else x_rows, ldx, _ptr(row_src),
                                     _ptr(offsets), rows, _typed("y", y, out_dtype), ldy, out_dtype, _stream(stream)), "uw_group_matmul")

    def check(self, stream=None):
        _check(lib().uw_group_check(self._h, _stream(stream)), "uw_group_check")


class Router:
    """How a layer's router chooses its experts (a ``uw_router``); bias: fp32 [experts] on the device, for the choice
    alone, added to the logits, or to the scores with a score of SCORE_SIGMOID + SCORE_CHOOSES (or SCORE_SOFTMAX + ...)."""

    def __init__(self, experts: int, topk: int, score: int = SCORE_SOFTMAX, bias=None, renormalize: bool = True, scale: float = 1.0):
        self._bias = bias  # keeps it alive
        self.desc = RouterDesc(experts, topk, score, int(renormalize), scale, _ptr(bias) or None)
        self._ref = ctypes.byref(self.desc)

    def workspace_size(self, tokens: int) -> int:
        n = ctypes.c_size_t(0)
        _check(lib().uw_route_workspace_size(ctypes.byref(self.desc), tokens, ctypes.byref(n)), "uw_route_workspace_size")
        return n.value

    def route(self, logits, tokens: int, ids, weights, offsets, row_src, pos, dtype: int = OUT_F32, ld: int = 0, workspace=None,
              ws_bytes: int = 0, stream=None):
        """uw_route: ids, row_src, pos and offsets int32, weights fp32."""
        _check(lib().uw_route(self._ref, _typed("logits", logits, dtype), dtype, tokens, ld, _ptr(ids), _ptr(weights), _ptr(offsets),
                              _ptr(row_src), _ptr(pos), _ptr(workspace), ws_bytes, _stream(stream)), "uw_route")


class BlockNorm:
    """What stands between one block's output and the next block's input (a ``uw_norm``): the norm after the block, its
    gate, the residual, the norm before the next block.  Weights and gate are bf16 tensors on the device."""

    def __init__(self, dim: int, post_weight=None, gate=None, gate_every: int = 1, pre_weight=None, res_scale: float = 1.0,
                 out_scale: float = 1.0, eps: float = 1e-5, res_dtype: int = OUT_BF16, block_dtype: int = OUT_BF16):
        self._keep = (post_weight, gate, pre_weight)
        self.desc = NormDesc(dim, _ptr(post_weight) or None, _ptr(gate) or None, gate_every, _ptr(pre_weight) or None, res_scale,
                             out_scale, eps, res_dtype, block_dtype)
        self._ref, self._res, self._block = ctypes.byref(self.desc), res_dtype, block_dtype

    def run(self, rows: int, h, h_out, y=None, pos=None, weights=None, topk: int = 0, y_rows: int = 0, u=None, stream=None):
        """uw_block_norm; topk > 0: y holds expert rows, joined by pos and weights [rows, topk]."""
        _check(lib().uw_block_norm(self._ref, rows, _typed("h", h, self._res), _typed("h_out", h_out, self._res),
                                   _typed("y", y, self._block), y_rows, _ptr(pos), _ptr(weights), topk, _typed("u", u, OUT_BF16),
                                   _stream(stream)), "uw_block_norm")


def token_logprobs(logits, rows: int, vocab: int, logprob=None, targets=None, entropy=None, n_top: int = 0, top_ids=None,
                   top_logprobs=None, dtype: int = OUT_F32, ld: int = 0, temperature: float = 1.0, stream=None):
    """uw_token_logprobs: log probabilities of `targets` (int32), entropies and the n_top most probable tokens."""
    _check(lib().uw_token_logprobs(_typed("logits", logits, dtype), dtype, rows, vocab, ld, temperature, _ptr(targets), _ptr(logprob), _ptr(entropy),
                                   n_top, _ptr(top_ids), _ptr(top_logprobs), _stream(stream)), "uw_token_logprobs")


_KINDS = {}  # names of element types -> torch's types


def _kinds():
    import torch
    _KINDS.update(f32={torch.float32}, i32={torch.int32}, bf16={torch.bfloat16, torch.int16, torch.uint16}, bits={torch.int32, torch.uint32},
                  any={torch.float32, torch.bfloat16, torch.int16, torch.uint16})
    return _KINDS


_KIND_OF = {OUT_F32: "f32", OUT_BF16: "bf16"}  # of a call's dtype; another one is the library's to refuse


def _wrong(what, t, kind, device):
    if t.dtype not in _KINDS[kind]:
        raise ValueError(f"{what} is {t.dtype}, the call takes {' or '.join(sorted(str(d) for d in _KINDS[kind]))}")
    if t.get_device() != device:
        raise ValueError(f"{what} is on {t.device}, the call is on CUDA device {device}")
    raise ValueError(f"{what}: its last dimension is not dense, or its shape is another than the call's")


def _at(what: str, t, kind: str, device: int) -> int:
    """_ptr of a tensor of this kind on this CUDA device; addresses pass."""
    if t is None:
        return 0
    if t.__class__ is int:
        return t
    if t.dtype not in (_KINDS or _kinds())[kind] or t.get_device() != device:
        _wrong(what, t, kind, device)
    return t.data_ptr()


def _of_rows(what: str, t, rows: int, kind: str, device: int) -> int:
    """_at of a dense tensor of a number for each row."""
    if t is None:
        return 0
    if t.__class__ is int:
        return t
    if t.dtype not in (_KINDS or _kinds())[kind] or t.get_device() != device or t.numel() < rows or not t.is_contiguous():
        _wrong(what, t, kind, device)
    return t.data_ptr()


_get_device = None


def _device() -> int:
    """The current CUDA device."""
    global _get_device
    if _get_device is None:
        import torch
        torch.cuda.current_device()  # sets CUDA up
        _get_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
    return _get_device()


def _shared(what: str):
    """Of rows that share memory: their stride of 0 would be the library's word for dense rows, which end far behind the tensor."""
    raise ValueError(f"{what}: its rows share memory (a broadcast tensor); pass a contiguous copy")


def _heads(what: str, t, rows: int, dim: int, kind: str, device: int):
    """Address, elements from row to row (0: dense) and heads of a tensor [rows, heads, dim] or [rows, heads * dim]."""
    if t is None:
        return 0, 0, 0
    if t.__class__ is int:
        return t, 0, 0
    if t.dtype not in (_KINDS or _kinds())[kind] or t.get_device() != device:
        _wrong(what, t, kind, device)
    shape, stride = t.shape, t.stride()
    if len(shape) == 3:
        n, heads, d = shape
        ok = d == dim and stride[2] == 1 and (stride[1] == dim or heads == 1)
    elif len(shape) == 2:
        n, width = shape
        heads = width // dim
        ok = heads * dim == width and stride[1] == 1
    else:
        n, heads, ok = 0, 0, False
    if not ok or n < rows:
        raise ValueError(f"{what} must be [rows, heads, {dim}] or [rows, heads * {dim}], a row's heads dense")
    if rows > 1 and stride[0] < heads * dim:
        _shared(what)
    return t.data_ptr(), stride[0] if n > 1 else 0, heads


def _room(what: str, t, size: int, device: int) -> int:
    """_ptr of a dense tensor of any type with that many bytes on this CUDA device; addresses pass."""
    if t is None:
        return 0
    if t.__class__ is int:
        return t
    if t.get_device() != device or not t.is_contiguous() or t.numel() * t.element_size() < size:
        raise ValueError(f"{what} must be dense, on CUDA device {device} (it is on {t.device}) and have {size} bytes (it has {t.numel() * t.element_size()})")
    return t.data_ptr()


class Rotary:
    """Rotary positions (a ``uw_rotary``): the first `dim` elements of a head, in pairs `layout` apart, by frequencies of `base`
    scaled for long contexts (ROTARY_LINEAR, ...: uw_rotary_frequencies), held on the current CUDA device.  low and high None: as
    rotary_frequencies has them.  freq: the caller's own frequencies in place of these, dim / 2 of them in radians a position; scale: the
    caller's own factor on cos and sin."""

    def __init__(self, dim: int, base: float = 10000.0, layout: int = ROTARY_HALF, scaling: int = ROTARY_PLAIN, factor: float = 1.0,
                 low=None, high=None, original: int = 8192, freq=None, scale=None):
        import torch
        if freq is None:
            self.freq, own = rotary_frequencies(dim, base, scaling, factor, low, high, original)
        else:
            self.freq, own = np.array(freq.detach().cpu().numpy() if isinstance(freq, torch.Tensor) else freq, np.float64), 1.0
            if self.freq.shape != (dim // 2,) or not np.isfinite(self.freq).all():
                raise ValueError(f"freq must be {dim // 2} finite numbers")
        self.scale = own if scale is None else float(scale)
        if not np.isfinite(self.scale):
            raise ValueError(f"scale {scale}")
        self._dev = torch.from_numpy(self.freq).cuda()
        self.device = self._dev.get_device()
        self.desc = RotaryDesc(dim, layout, self._dev.data_ptr(), self.scale)
        self._ref = ctypes.byref(self.desc)


def rotary_frequencies(dim: int, base: float = 10000.0, scaling: int = ROTARY_PLAIN, factor: float = 1.0, low=None, high=None, original: int = 8192):
    """uw_rotary_frequencies: (float64 array [dim / 2] in radians a position, factor on cos and sin).  low and high, in turns over the
    original length, are by default those of the scaling's method: 1 and 4 by bands, 1 and 32 on a ramp."""
    low = 1.0 if low is None else low
    high = (32.0 if scaling == ROTARY_RAMP else 4.0) if high is None else high
    f, s = np.zeros(max(1, dim // 2)), ctypes.c_float(0)
    _check(lib().uw_rotary_frequencies(dim, base, scaling, factor, low, high, original, f.ctypes.data, ctypes.byref(s)), "uw_rotary_frequencies")
    return f, s.value


class KVBatch:
    """The new tokens of a step (a ``uw_kv_batch``), int32 on the device: sequence s brings rows [starts[s], starts[s + 1]) and
    holds lengths[s] tokens with them, in the pages pages[s] (a tensor [sequences, max_pages])."""

    def __init__(self, starts, lengths, pages):
        if any(not t.is_cuda or (t.shape[-1] > 1 and t.stride(-1) != 1) for t in (starts, lengths, pages)):
            raise ValueError("starts, lengths and rows of pages must be dense and in device memory")
        if pages.dim() != 2 or lengths.dim() != 1 or starts.dim() != 1 or pages.shape[0] != lengths.shape[0] or starts.shape[0] != lengths.shape[0] + 1:
            raise ValueError("starts [sequences + 1], lengths [sequences], pages [sequences, max_pages]")
        if pages.shape[0] > 1 and pages.stride(0) < pages.shape[1]:
            _shared("pages")
        self._keep = (starts, lengths, pages)
        self.sequences = lengths.shape[0]
        self.device = starts.get_device()
        self.desc = KVBatchDesc(self.sequences, *(_at(w, x, "i32", self.device) for w, x in (("starts", starts), ("lengths", lengths), ("pages", pages))),
                                pages.stride(0) if self.sequences > 1 else 0, pages.shape[1])
        self._ref = ctypes.byref(self.desc)


class KVCache:
    """Keys and values in pages (a ``uw_kv_cache`` on the current CUDA device): k and v bf16 tensors [pages, page_size, kv_heads,
    head_dim] of the same strides (head_dim dense; a transposed [pages, kv_heads, page_size, head_dim] is one)."""

    def __init__(self, k, v):
        self._h = None
        if k.dim() != 4 or k.shape != v.shape or k.stride() != v.stride() or k.stride(3) != 1:
            raise ValueError("k and v must be [pages, page_size, kv_heads, head_dim] with the same strides")
        self._keep = (k, v)
        self.pages, self.page_size, self.kv_heads, self.head_dim = k.shape
        self._scale = self.head_dim ** -0.5 if self.head_dim else 0.0
        self._device = _device() if k.is_cuda else -2
        d = KVDesc(_at("k", k, "bf16", self._device), _at("v", v, "bf16", self._device), self.pages, k.stride(0), k.stride(1), k.stride(2), self.page_size, self.kv_heads,
                   self.head_dim)
        h = ctypes.c_void_p()
        _check(lib().uw_kv_create(ctypes.byref(d), ctypes.byref(h)), "uw_kv_create")
        self._h = h

    def close(self):
        if getattr(self, "_h", None):
            lib().uw_kv_free(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    @property
    def handle(self):
        return self._h

    def append(self, batch, rows: int, k=None, v=None, q=None, q_out=None, q_heads: int = 0, rotary=None, positions=None, dtype: int = OUT_BF16,
               ldq: int = 0, ldk: int = 0, ldv: int = 0, ldq_out: int = 0, stream=None):
        """uw_kv_append: q, k, v of `dtype`, tensors [rows, heads, head_dim] (their strides and heads are taken from them) or
        addresses; q_out bf16."""
        D = self.head_dim
        kind = _KIND_OF.get(dtype, "any")
        dev = self._device
        pq, sq, hq = _heads("q", q, rows, D, kind, dev)
        po, so, ho = _heads("q_out", q_out, rows, D, "bf16", dev)
        pk, sk, hk = _heads("k", k, rows, D, kind, dev)
        pv, sv, hv = _heads("v", v, rows, D, kind, dev)
        if batch.device != dev or (rotary is not None and rotary.device != dev):
            raise ValueError(f"the batch or the rotary is on another device than the cache's {dev}")
        q_heads = q_heads or hq or ho
        if (hq and hq != q_heads) or (ho and ho != q_heads) or (hk and hk != self.kv_heads) or (hv and hv != self.kv_heads):
            raise ValueError(f"heads: q {hq}, q_out {ho} of {q_heads}, k {hk}, v {hv} of {self.kv_heads}")
        s = lib().uw_kv_append(self._h, batch._ref, rotary._ref if rotary is not None else None, rows, dtype, pq, ldq or sq, q_heads, pk, ldk or sk, pv,
                               ldv or sv, _of_rows("positions", positions, rows, "i32", dev), po, ldq_out or so, _stream(stream))
        if s:
            _check(s, "uw_kv_append")

    def workspace_size(self, batch, rows: int, q_heads: int) -> int:
        n = ctypes.c_size_t(0)
        _check(lib().uw_kv_attend_workspace_size(self._h, batch.sequences, rows, q_heads, ctypes.byref(n)), "uw_kv_attend_workspace_size")
        return n.value

    def attend(self, batch, rows: int, q, out, q_heads: int = 0, scale=None, causal: bool = True, window: int = 0, lse=None, workspace=None,
               ws_bytes: int = 0, ldq: int = 0, ldo: int = 0, stream=None):
        """uw_kv_attend: q and out bf16 [rows, q_heads, head_dim] (or addresses, with q_heads); scale None: head_dim ** -0.5;
        workspace: a tensor of at least ws_bytes bytes (or an address)."""
        dev = self._device
        pq, sq, hq = _heads("q", q, rows, self.head_dim, "bf16", dev)
        po, so, ho = _heads("out", out, rows, self.head_dim, "bf16", dev)
        if batch.device != dev:
            raise ValueError(f"the batch is on device {batch.device}, the cache on {dev}")
        q_heads = q_heads or hq or ho
        if (hq and hq != q_heads) or (ho and ho != q_heads):
            raise ValueError(f"heads: q {hq}, out {ho} of {q_heads}")
        if lse is not None and lse.__class__ is not int and (not lse.is_contiguous() or lse.numel() < rows * q_heads):
            raise ValueError("lse must be dense [rows, q_heads]")
        s = lib().uw_kv_attend(self._h, batch._ref, rows, pq, ldq or sq, q_heads, self._scale if scale is None else scale, causal, window, po, ldo or so,
                               _at("lse", lse, "f32", dev), _room("workspace", workspace, ws_bytes, dev), ws_bytes, _stream(stream))
        if s:
            _check(s, "uw_kv_attend")

    def check(self, stream=None):
        _check(lib().uw_kv_check(self._h, _stream(stream)), "uw_kv_check")


def edit_logits(logits, rows: int, vocab: int, out, tokens=None, lengths=None, prompt_lengths=None, repetition=None, frequency=None, presence=None,
                bias_ids=None, bias=None, bias_lengths=None, allowed=None, mask_rows=None, dtype: int = OUT_F32, out_dtype=None, ld: int = 0,
                ld_out: int = 0, stream=None):
    """uw_edit_logits on tensors: logits and out [rows, vocab or more] (or addresses, with ld), tokens int32 [rows, max_tokens], lengths and
    prompt_lengths int32 [rows], penalties fp32 [rows], bias_ids int32 and bias fp32 [rows, max_bias], allowed int32 words
    [masks, words].  out_dtype None: dtype."""
    out_dtype = dtype if out_dtype is None else out_dtype
    dev = _device()
    p, po = _at("logits", logits, _KIND_OF.get(dtype, "any"), dev), _at("out", out, _KIND_OF.get(out_dtype, "any"), dev)
    ld, ld_out = ld or _pitch("logits", logits, rows, vocab), ld_out or _pitch("out", out, rows, vocab)
    max_tokens = max_bias = ld_tokens = ld_allowed = masks = 0
    pt = _at("tokens", tokens, "i32", dev)
    if tokens is not None:
        ld_tokens, max_tokens = _pitch("tokens", tokens, rows, 0), tokens.shape[1]
        if max_tokens == 0:  # no history: no penalties
            pt, repetition, frequency, presence = 0, None, None, None
    pi, pb = _at("bias_ids", bias_ids, "i32", dev), _at("bias", bias, "f32", dev)
    if bias is not None and bias_ids is not None:
        if bias_ids.shape != bias.shape or bias.dim() != 2 or bias.shape[0] < rows or not bias.is_contiguous() or not bias_ids.is_contiguous():
            raise ValueError("bias_ids and bias must be contiguous [rows, max_bias]")
        max_bias = bias.shape[1]
    pa = _at("allowed", allowed, "bits", dev)
    if allowed is not None:
        if allowed.dim() != 2 or allowed.shape[1] * 32 < vocab or allowed.stride(1) != 1:
            raise ValueError("allowed must be [masks, ceil(vocab / 32)]")
        masks = allowed.shape[0]
        if masks > 1 and allowed.stride(0) * 32 < vocab:
            _shared("allowed")
        ld_allowed = allowed.stride(0) if masks > 1 else 0
    d = LogitEditsDesc(pt, ld_tokens, max_tokens, _of_rows("lengths", lengths, rows, "i32", dev), _of_rows("prompt_lengths", prompt_lengths, rows, "i32", dev),
                       _of_rows("repetition", repetition, rows, "f32", dev), _of_rows("frequency", frequency, rows, "f32", dev),
                       _of_rows("presence", presence, rows, "f32", dev), pi, pb, _of_rows("bias_lengths", bias_lengths, rows, "i32", dev), max_bias, pa, ld_allowed,
                       masks, _of_rows("mask_rows", mask_rows, rows, "i32", dev))
    s = lib().uw_edit_logits(ctypes.byref(d), p, dtype, rows, vocab, ld, po, out_dtype, ld_out, _stream(stream))
    if s:
        _check(s, "uw_edit_logits")


def _pitch(what: str, t, rows: int, width: int) -> int:
    """Elements from row to row (0: dense) of a tensor [rows, width or more]; 0 for an address."""
    if t is None or t.__class__ is int:
        return 0
    shape, stride = t.shape, t.stride()
    if len(shape) != 2 or shape[0] < rows or shape[1] < width or (stride[1] != 1 and shape[1] > 1):
        raise ValueError(f"{what} must be [rows, {width} or more], its rows dense")
    if rows > 1 and stride[0] < (width or shape[1]):
        _shared(what)
    return stride[0] if rows > 1 else 0
