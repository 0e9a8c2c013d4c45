"""ctypes binding of libcp.so (include/cp.h): argument marshalling only.

Every step of the frame runs in the library's CUDA kernels; this module only
turns torch tensors into raw pointers and stream handles and maps status codes
to exceptions. It fails loudly when the library has not been built.
"""
from __future__ import annotations

import ctypes as C
import os

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "_lib", "libcp.so")

CP_OK = 0
STATUS = {0: "CP_OK", 1: "CP_ERR_INVALID_ARG", 2: "CP_ERR_UNSUPPORTED", 3: "CP_ERR_RESIDENCY",
          4: "CP_ERR_CUDA", 5: "CP_ERR_TIMEOUT", 6: "CP_ERR_DEVICE_BOUNDS", 7: "CP_ERR_NOMEM",
          8: "CP_ERR_PLAN", 9: "CP_ERR_SCRATCH_LIMIT", 10: "CP_ERR_RANGE"}
CP_ERR_TIMEOUT = 5
CP_ERR_PLAN = 8
CP_ERR_SCRATCH_LIMIT = 9
CP_ERR_RANGE = 10

EXPORTS = ["cp_create", "cp_frame", "cp_frame_split", "cp_debug_logits", "cp_debug_state", "cp_status",
           "cp_clear_status", "cp_get_info", "cp_trace", "cp_destroy", "cp_strerror",
           "cp_plan_check", "cp_test_philox", "cp_test_draw", "cp_frame_static",
           "cp_cache_create", "cp_cache_append", "cp_cache_read", "cp_cache_attend", "cp_cache_status",
           "cp_cache_clear_status", "cp_cache_destroy", "cp_cache_check", "cp_test_slot", "cp_cache_copy",
           "cp_pages_create", "cp_pages_fork", "cp_pages_grow", "cp_pages_trim", "cp_pages_compact", "cp_pages_status",
           "cp_pages_clear_status", "cp_pages_destroy", "cp_pages_check",
           "cp_linear_create", "cp_linear_apply", "cp_linear_status", "cp_linear_clear_status", "cp_linear_unpack", "cp_linear_destroy", "cp_linear_check",
           "cp_verify", "cp_verify_check"]


class Shape(C.Structure):
    _fields_ = [("layers", C.c_int), ("hidden", C.c_int), ("q_heads", C.c_int), ("kv_heads", C.c_int),
                ("head_dim", C.c_int), ("ffn", C.c_int), ("positions", C.c_int), ("vocab", C.c_int),
                ("talker_hidden", C.c_int), ("max_rows", C.c_int), ("rms_eps", C.c_float),
                ("rope_base", C.c_float), ("qk_norm", C.c_int)]


_PP = C.POINTER(C.c_void_p)


class Weights(C.Structure):
    _fields_ = [("in_proj", C.c_void_p), ("embed", _PP), ("attn_norm", _PP), ("mlp_norm", _PP),
                ("q_norm", _PP), ("k_norm", _PP), ("w_qkv", _PP), ("w_o", _PP), ("w_gate", _PP),
                ("w_up", _PP), ("w_down", _PP), ("final_norm", C.c_void_p), ("heads", _PP)]


class Sampler(C.Structure):
    _fields_ = [("temperature", C.c_void_p), ("top_k", C.c_void_p), ("top_p", C.c_void_p),
                ("seed", C.c_void_p), ("offset", C.c_void_p)]


class Options(C.Structure):
    _fields_ = [("cluster", C.c_int), ("max_ctas", C.c_int), ("timeout_ns", C.c_int64), ("trace", C.c_int),
                ("n_cuts", C.c_int), ("cuts", C.POINTER(C.c_int)), ("debug_stall_task", C.c_int),
                ("debug_stall_staging", C.c_int), ("generic_kernel", C.c_int), ("phase_waits", C.c_int)]


class Info(C.Structure):
    _fields_ = [("grid", C.c_int), ("cluster", C.c_int), ("threads", C.c_int), ("smem_bytes", C.c_int),
                ("phases", C.c_int), ("tasks", C.c_int), ("weight_bytes", C.c_int64),
                ("max_cta_weight_bytes", C.c_int64), ("min_cta_weight_bytes", C.c_int64),
                ("scratch_bytes", C.c_int64), ("sm_count", C.c_int), ("specialized", C.c_int)]


class PlanStats(C.Structure):
    _fields_ = [("phases", C.c_int), ("tasks", C.c_int), ("counters", C.c_int), ("weight_bytes", C.c_int64),
                ("max_cta_weight_bytes", C.c_int64), ("min_cta_weight_bytes", C.c_int64),
                ("max_tasks_per_cta", C.c_int), ("message", C.c_char * 160)]


class CacheDesc(C.Structure):
    _fields_ = [("dtype", C.c_int), ("kv_heads", C.c_int), ("head_dim", C.c_int), ("page_size", C.c_int),
                ("pages", C.c_int), ("k", C.c_void_p), ("v", C.c_void_p), ("page_stride", C.c_int64),
                ("head_stride", C.c_int64), ("token_stride", C.c_int64), ("k_scale", C.c_void_p),
                ("v_scale", C.c_void_p), ("scale_page_stride", C.c_int64), ("scale_head_stride", C.c_int64),
                ("scale_token_stride", C.c_int64), ("timeout_ns", C.c_int64), ("debug_stall", C.c_int)]


class BatchDesc(C.Structure):
    _fields_ = [("sequences", C.c_int), ("rows", C.c_int), ("max_new", C.c_int), ("max_length", C.c_int),
                ("table_width", C.c_int), ("table_stride", C.c_int64), ("start", C.c_void_p), ("length", C.c_void_p),
                ("page_table", C.c_void_p)]


class AppendArgs(C.Structure):
    _fields_ = [("qkv", C.c_void_p), ("qkv_stride", C.c_int64), ("q_out", C.c_void_p), ("q_stride", C.c_int64),
                ("q_heads", C.c_int), ("q_norm", C.c_void_p), ("k_norm", C.c_void_p), ("rms_eps", C.c_float),
                ("rope_base", C.c_float)]


class AttendArgs(C.Structure):
    _fields_ = [("q", C.c_void_p), ("out", C.c_void_p), ("q_stride", C.c_int64), ("q_head_stride", C.c_int64),
                ("out_stride", C.c_int64), ("out_head_stride", C.c_int64), ("q_heads", C.c_int), ("scale", C.c_float),
                ("causal", C.c_int), ("window", C.c_int)]


class PagesDesc(C.Structure):
    _fields_ = [("pages", C.c_int), ("page_size", C.c_int), ("sequences", C.c_int), ("table_width", C.c_int),
                ("table_stride", C.c_int64), ("refs", C.c_void_p), ("page_table", C.c_void_p), ("length", C.c_void_p)]


class LinearDesc(C.Structure):
    _fields_ = [("features", C.c_int), ("width", C.c_int), ("group", C.c_int), ("gated", C.c_int), ("q", C.c_void_p),
                ("scale", C.c_void_p), ("zero", C.c_void_p), ("timeout_ns", C.c_int64), ("debug_stall", C.c_int)]


class LinearArgs(C.Structure):
    _fields_ = [("x", C.c_void_p), ("x_stride", C.c_int64), ("rows", C.c_int), ("out_dtype", C.c_int), ("out", C.c_void_p),
                ("out_stride", C.c_int64), ("add", C.c_void_p), ("add_stride", C.c_int64)]


class VerifyArgs(C.Structure):
    _fields_ = [("sequences", C.c_int), ("rows", C.c_int), ("vocab", C.c_int), ("dtype", C.c_int), ("start", C.c_void_p),
                ("logits", C.c_void_p), ("logits_stride", C.c_int64), ("draft_logits", C.c_void_p), ("draft_stride", C.c_int64),
                ("draft", C.c_void_p), ("temperature", C.c_void_p), ("u_accept", C.c_void_p), ("u_token", C.c_void_p),
                ("accepted", C.c_void_p), ("token", C.c_void_p), ("prob", C.c_void_p)]


class CPError(RuntimeError):
    def __init__(self, code: int, what: str):
        self.code = code
        super().__init__(f"{what}: {STATUS.get(code, code)}")


_lib = None


def lib() -> C.CDLL:
    """The loaded library; raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                               "persistent_megakernel_streaming_gb300.build.build()")
        L = C.CDLL(LIB_PATH)
        vp, i, st = C.c_void_p, C.c_int, C.c_void_p
        L.cp_create.argtypes = [C.POINTER(Shape), C.POINTER(Weights), i, C.POINTER(Options), C.POINTER(vp)]
        for name in ("cp_frame", "cp_frame_split", "cp_frame_static"):
            getattr(L, name).argtypes = [vp, vp, vp, C.POINTER(Sampler), i, vp, vp, st]
        L.cp_debug_logits.argtypes = [vp, i, vp, st]
        L.cp_debug_state.argtypes = [vp, i, i, i, vp, st]
        L.cp_status.argtypes = [vp]
        L.cp_clear_status.argtypes = [vp]
        L.cp_get_info.argtypes = [vp, C.POINTER(Info)]
        L.cp_trace.argtypes = [vp, vp, st]
        L.cp_destroy.argtypes = [vp]
        L.cp_destroy.restype = None
        L.cp_strerror.argtypes = [i]
        L.cp_strerror.restype = C.c_char_p
        L.cp_plan_check.argtypes = [C.POINTER(Shape), i, i, i, i, C.POINTER(PlanStats)]
        L.cp_test_philox.argtypes = [vp, vp, i, i, vp, st]
        L.cp_test_draw.argtypes = [vp, i, i, C.POINTER(Sampler), i, vp, st]
        L.cp_cache_create.argtypes = [C.POINTER(CacheDesc), i, C.POINTER(vp)]
        L.cp_cache_append.argtypes = [vp, C.POINTER(BatchDesc), C.POINTER(AppendArgs), st]
        L.cp_cache_read.argtypes = [vp, C.POINTER(BatchDesc), vp, vp, st]
        L.cp_cache_attend.argtypes = [vp, C.POINTER(BatchDesc), C.POINTER(AttendArgs), vp, C.c_size_t, st]
        L.cp_cache_status.argtypes = [vp]
        L.cp_cache_clear_status.argtypes = [vp]
        L.cp_cache_destroy.argtypes = [vp]
        L.cp_cache_destroy.restype = None
        L.cp_cache_check.argtypes = [C.POINTER(CacheDesc), C.POINTER(BatchDesc), C.POINTER(AppendArgs),
                                     C.POINTER(AttendArgs), C.POINTER(C.c_size_t)]
        L.cp_cache_copy.argtypes = [vp, vp, i, vp, st]
        L.cp_pages_create.argtypes = [C.POINTER(PagesDesc), i, C.POINTER(vp)]
        L.cp_pages_fork.argtypes = [vp, vp, vp, i, st]
        L.cp_pages_grow.argtypes = [vp, vp, vp, i, vp, st]
        L.cp_pages_trim.argtypes = [vp, vp, st]
        L.cp_pages_compact.argtypes = [vp, vp, i, vp, st]
        L.cp_pages_status.argtypes = [vp]
        L.cp_pages_clear_status.argtypes = [vp]
        L.cp_pages_destroy.argtypes = [vp]
        L.cp_pages_destroy.restype = None
        L.cp_pages_check.argtypes = [C.POINTER(PagesDesc)]
        L.cp_linear_create.argtypes = [C.POINTER(LinearDesc), i, C.POINTER(vp)]
        L.cp_linear_apply.argtypes = [vp, C.POINTER(LinearArgs), st]
        L.cp_linear_unpack.argtypes = [vp, vp, st]
        L.cp_linear_status.argtypes = [vp]
        L.cp_linear_clear_status.argtypes = [vp]
        L.cp_linear_destroy.argtypes = [vp]
        L.cp_linear_destroy.restype = None
        L.cp_linear_check.argtypes = [C.POINTER(LinearDesc), C.POINTER(LinearArgs)]
        L.cp_verify.argtypes = [C.POINTER(VerifyArgs), i, vp, C.c_size_t, st]
        L.cp_verify_check.argtypes = [C.POINTER(VerifyArgs), C.POINTER(C.c_size_t)]
        L.cp_test_slot.argtypes = [C.POINTER(CacheDesc), C.POINTER(C.c_int32), i, i, i]
        L.cp_test_slot.restype = C.c_int64
        _lib = L
    return _lib


def _check(code: int, what: str):
    if code != CP_OK:
        raise CPError(code, what)


def make_shape(d: dict) -> Shape:
    return Shape(d["layers"], d["hidden"], d["q_heads"], d["kv_heads"], d["head_dim"], d["ffn"],
                 d["positions"], d["vocab"], d["talker_hidden"], d.get("max_rows", 64),
                 float(d["rms_eps"]), float(d["rope_base"]), int(d["qk_norm"]))


def plan_check(shape: dict, grid: int, cluster: int, corrupt: int = 0, chunk_waits: bool = False):
    """Host-only schedule build and check (no GPU). Returns (status, stats)."""
    ps = PlanStats()
    code = lib().cp_plan_check(C.byref(make_shape(shape)), grid, cluster, int(chunk_waits), corrupt, C.byref(ps))
    return code, ps


def _ptr(t) -> int:
    return 0 if t is None else int(t.data_ptr())


def _stream(stream) -> int:
    if stream is None:
        import torch
        return int(torch.cuda.current_stream().cuda_stream)
    return int(getattr(stream, "cuda_stream", stream))


def _sampler(samp: dict) -> Sampler:
    return Sampler(_ptr(samp["temperature"]), _ptr(samp["top_k"]), _ptr(samp["top_p"]),
                   _ptr(samp["seed"]), _ptr(samp["offset"]))


class Frame:
    """A handle (cp_create) with the frame calls bound to torch tensors.

    ``weights``: dict of tensors (host or device) holding bf16 bit patterns in
    the layouts of include/cp.h (per-layer / per-position lists as stacked
    leading dimensions)."""

    def __init__(self, shape: dict, weights: dict, device: int = 0, cluster: int = 0, max_ctas: int = 0,
                 timeout_ns: int = 0, trace: bool = False, cuts=None, debug_stall_task: int = 0,
                 debug_stall_staging: bool = False, generic_kernel: bool = False, phase_waits: bool = False):
        self.shape = dict(shape)
        L, P = shape["layers"], shape["positions"]
        keep = []

        def one(t):
            keep.append(t)
            return C.c_void_p(_ptr(t))

        def many(t, n):
            arr = (C.c_void_p * n)(*[_ptr(t[i]) for i in range(n)])
            keep.append(t)
            keep.append(arr)
            return C.cast(arr, _PP)

        w = Weights(one(weights["in_proj"]), many(weights["embed"], P), many(weights["attn_norm"], L),
                    many(weights["mlp_norm"], L), many(weights["q_norm"], L), many(weights["k_norm"], L),
                    many(weights["w_qkv"], L), many(weights["w_o"], L), many(weights["w_gate"], L),
                    many(weights["w_up"], L), many(weights["w_down"], L), one(weights["final_norm"]),
                    many(weights["heads"], P - 1))
        cuts = list(cuts or [])
        cut_arr = (C.c_int * max(1, len(cuts)))(*cuts)
        opt = Options(cluster, max_ctas, _int64(timeout_ns, "timeout_ns"), int(trace), len(cuts), cut_arr, debug_stall_task,
                      int(debug_stall_staging), int(generic_kernel), int(phase_waits))
        h = C.c_void_p()
        _check(lib().cp_create(C.byref(make_shape(shape)), C.byref(w), device, C.byref(opt), C.byref(h)),
               "cp_create")
        self._h = h
        self.info = Info()
        _check(lib().cp_get_info(h, C.byref(self.info)), "cp_get_info")

    def _call(self, fn, h, c0, samp, rows, codes, emb_sum, stream):
        sp = _sampler(samp)
        _check(fn(self._h, _ptr(h), _ptr(c0), C.byref(sp), int(rows), _ptr(codes), _ptr(emb_sum),
                  _stream(stream)), fn.__name__)

    def frame(self, h, c0, samp, rows, codes, emb_sum=None, stream=None):
        self._call(lib().cp_frame, h, c0, samp, rows, codes, emb_sum, stream)

    def frame_split(self, h, c0, samp, rows, codes, emb_sum=None, stream=None):
        self._call(lib().cp_frame_split, h, c0, samp, rows, codes, emb_sum, stream)

    def frame_static(self, h, c0, samp, rows, codes, emb_sum=None, stream=None):
        """cp_frame with its working set in the library's static scratch array."""
        self._call(lib().cp_frame_static, h, c0, samp, rows, codes, emb_sum, stream)

    def debug_logits(self, group, dst, stream=None):
        _check(lib().cp_debug_logits(self._h, int(group), _ptr(dst), _stream(stream)), "cp_debug_logits")

    def debug_state(self, what, a, b, dst, stream=None):
        _check(lib().cp_debug_state(self._h, int(what), int(a), int(b), _ptr(dst), _stream(stream)),
               "cp_debug_state")

    def trace(self, dst, stream=None):
        _check(lib().cp_trace(self._h, _ptr(dst), _stream(stream)), "cp_trace")

    def status(self) -> int:
        return lib().cp_status(self._h)

    def clear_status(self):
        _check(lib().cp_clear_status(self._h), "cp_clear_status")

    def close(self):
        if getattr(self, "_h", None):
            lib().cp_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def _stride(t, axis: int) -> int:
    """Elements between t's entries along `axis`; 0 (the C side's "contiguous") where there is one at most."""
    if t.shape[axis] <= 1:
        return 0
    if t.stride(axis) <= 0:
        raise ValueError("a tensor whose entries share memory (an expanded one)")
    return t.stride(axis)


def _int32(x, what: str) -> int:
    """x as the C side's int; ctypes would keep its low 32 bits and say nothing."""
    if not -2 ** 31 <= int(x) < 2 ** 31:
        raise ValueError(f"{what}: {x} is past 32 bits")
    return int(x)


def _int64(x, what: str) -> int:
    """x as the C side's int64_t, likewise."""
    if not -2 ** 63 <= int(x) < 2 ** 63:
        raise ValueError(f"{what}: {x} is past 64 bits")
    return int(x)


def _not_lost(x: float, what: str):
    """x is not one that fp32 turns into zero, which the C side takes for "none given"."""
    if 0 < abs(x) < 2.0 ** -149:
        raise ValueError(f"{what}: {x} is zero in fp32")


_torch = None        # torch, once there are tensors to look at: an import statement costs a call 0.2 us


def _with_torch():
    global _torch
    if _torch is None:
        import torch
        _torch = torch
    return _torch


def _stream_on(index: int, stream) -> int:
    """The raw stream: torch's current one of that device, if none is given."""
    if stream is None:
        return (_torch or _with_torch())._C._cuda_getCurrentRawStream(index)
    return _stream(stream)


def _workspace(device, size: int, stream):
    """Device bytes, allocated on the stream that uses them, so that the allocator hands them on in that stream's order."""
    torch = _torch or _with_torch()
    if stream is None:
        return torch.empty(size, dtype=torch.uint8, device=device)
    if not hasattr(stream, "cuda_stream"):
        stream = torch.cuda.ExternalStream(int(stream), device=device)
    with torch.cuda.stream(stream):
        return torch.empty(size, dtype=torch.uint8, device=device)


def _array(t, what: str, dtype, shape, index: int) -> int:
    """Address of a contiguous device array of that type, shape and device."""
    if t.dtype is not dtype or t.shape != shape or t.get_device() != index or not t.is_contiguous():
        raise ValueError(f"{what}: {dtype} {list(shape)}, contiguous, on cuda:{index}; got {t.dtype} {list(t.shape)} on {t.device}")
    return t.data_ptr()


class Batch:
    """A ragged batch (cp_batch): row ``start[i] + j`` of the calls' row arrays is sequence i's new row j.

    ``start`` int32 [sequences + 1], ``length`` int32 [sequences] (cached positions, the new rows' own included),
    ``pages`` int32 [sequences][width]; device tensors, read when a call runs on the device. ``rows`` is the row
    arrays' length, ``max_new`` and ``max_len`` bound the new rows and the length of any sequence (0: no bound
    but the arrays' own). What a batch was made of stays: new lengths or pages are written into the tensors, other
    tensors or bounds are another batch."""

    def __setattr__(self, name, value):
        # the C side keeps the addresses and the bounds that the checks were made for
        if self.__dict__.get(name, value) is not value:        # (batch.length += 1 sets what is there)
            raise AttributeError(f"{name}: fixed when the batch is made")
        super().__setattr__(name, value)

    def __init__(self, start, length, pages, rows: int, max_new: int = 0, max_len: int = 0):
        import torch
        for name, t in (("start", start), ("length", length), ("pages", pages)):
            if t.dtype != torch.int32 or t.stride(-1) != 1 and t.shape[-1] > 1:
                raise ValueError(f"{name}: int32, contiguous")
        if length.dim() != 1 or start.dim() != 1 or pages.dim() != 2 or start.numel() != length.numel() + 1 or \
                pages.shape[0] != length.numel():
            raise ValueError("start [n + 1], length [n] and pages [n][width]")
        if not start.device == length.device == pages.device:
            raise ValueError("start, length and pages on one device")
        self.start, self.length, self.pages, self.rows = start, length, pages, _int32(rows, "rows")
        self.device_index = start.get_device()
        self.plans = {}     # attend's workspace sizes by what they depend on
        self.desc = BatchDesc(_int32(length.numel(), "sequences"), self.rows, _int32(max_new, "max_new"),
                              _int32(max_len, "max_len"), _int32(pages.shape[1], "width"), _stride(pages, 0), _ptr(start), _ptr(length), _ptr(pages))
        self.ref = C.byref(self.desc)


class Cache:
    """A paged K/V cache (cp_cache_create) over the caller's tensors.

    ``k``, ``v``: [pages][kv_heads][page_size][head_dim] bf16 (or int16 bit patterns), or e4m3 (or uint8) with
    ``k_scale``, ``v_scale`` uint8 [pages][kv_heads][page_size]; both of the same strides. See include/cp.h for
    what the calls compute."""

    def __init__(self, k, v, k_scale=None, v_scale=None, timeout_ns: int = 0, debug_stall: bool = False):
        import torch
        self.kinds = (torch.bfloat16, torch.int16)      # other 16-bit types would be read as bf16
        size = k.element_size()
        if k.dim() != 4 or k.shape != v.shape or k.stride() != v.stride() or k.device != v.device or \
                k.device.type != "cuda":
            raise ValueError("k and v: [pages][kv_heads][page_size][head_dim] of the same strides, on one GPU")
        if size == 2 and (k.dtype not in self.kinds or v.dtype not in self.kinds):
            raise ValueError("k and v: bf16 (or its bits as int16), or e4m3")
        if size == 1 and (k.dtype not in (torch.uint8, torch.float8_e4m3fn) or v.dtype != k.dtype):
            raise ValueError("k and v: e4m3 (or its bits as uint8), or bf16")
        if size not in (1, 2) or (size == 1) != (k_scale is not None) or (k_scale is None) != (v_scale is None):
            raise ValueError("bf16 pages without scales, or e4m3 pages with k_scale and v_scale")
        if k.stride(3) != 1:
            raise ValueError("k and v: the last axis contiguous")
        scale_strides = (0, 0, 0)
        if size == 1:
            for t in (k_scale, v_scale):
                if t.element_size() != 1 or t.shape != k.shape[:3] or t.stride() != k_scale.stride() or t.device != k.device:
                    raise ValueError("scales: uint8 [pages][kv_heads][page_size] of the same strides")
            scale_strides = [_stride(k_scale, i) for i in range(3)]
        self.pages, self.kv_heads, self.page_size, self.head_dim = (_int32(n, "k and v") for n in k.shape)
        self.keep = (k, v, k_scale, v_scale)
        self.device, self.device_index = k.device, k.get_device()
        self.layout = (size, self.kv_heads, self.head_dim, self.page_size)
        self.desc = CacheDesc(int(size == 1), self.kv_heads, self.head_dim, self.page_size, self.pages, _ptr(k), _ptr(v),
                              *(_stride(k, i) for i in range(3)), _ptr(k_scale), _ptr(v_scale), *scale_strides,
                              _int64(timeout_ns, "timeout_ns"), int(debug_stall))
        h = C.c_void_p()
        _check(lib().cp_cache_create(C.byref(self.desc), k.device.index, C.byref(h)), "cp_cache_create")
        self._h = h

    def append(self, batch: Batch, qkv, q_out=None, q_norm=None, k_norm=None, rms_eps: float = 1e-6,
               rope_base: float = 0.0, stream=None):
        """qkv [rows][(q_heads + 2 kv_heads) * head_dim] into the cache, its q into q_out [rows][q_heads][head_dim]."""
        d = self.head_dim
        heads = 0 if q_out is None else q_out.shape[1]
        x, st = self._rows(batch, qkv, "qkv", (batch.rows, (heads + 2 * self.kv_heads) * d))
        q, qs = 0, (0, 0)
        if q_out is not None:
            q, qs = self._rows(batch, q_out, "q_out", (batch.rows, heads, d))
            if qs[1] not in (0, d):
                raise ValueError("q_out: contiguous heads")
        _not_lost(rope_base, "rope_base")
        a = AppendArgs(x, st[0], q, qs[0], heads, self._gain(q_norm), self._gain(k_norm), rms_eps, rope_base)
        code = lib().cp_cache_append(self._h, batch.ref, C.byref(a), self._stream(stream))
        if code:
            raise CPError(code, "cp_cache_append")

    def read(self, batch: Batch, k_out=None, v_out=None, stream=None):
        """The batch's rows' cached keys and values as bf16 [rows][kv_heads][head_dim], contiguous."""
        at = [0, 0]
        for i, t in enumerate((k_out, v_out)):
            if t is not None:
                at[i], _ = self._rows(batch, t, "k_out, v_out", (batch.rows, self.kv_heads, self.head_dim))
                if not t.is_contiguous():
                    raise ValueError("k_out, v_out: contiguous")
        code = lib().cp_cache_read(self._h, batch.ref, at[0], at[1], self._stream(stream))
        if code:
            raise CPError(code, "cp_cache_read")

    def copy(self, moves, count, stream=None):
        """Whole pages, keys, values and scales, from moves[i][0] to moves[i][1] for i below count[0]: int32 [capacity][2]
        and [1], as Pages.grow and Pages.compact write them."""
        a, capacity, n = _moves(moves, count, self.device_index)
        code = lib().cp_cache_copy(self._h, a, capacity, n, self._stream(stream))
        if code:
            raise CPError(code, "cp_cache_copy")

    def attend(self, batch: Batch, q, out, scale: float = 0.0, causal: bool = True, window: int = 0, workspace=None,
               stream=None):
        """Attention of q [rows][q_heads][head_dim] over the cache into out (the same shape). Without a
        ``workspace`` (device bytes, see workspace_bytes) one is taken from torch's allocator for this call."""
        heads = q.shape[1]
        shape = (batch.rows, heads, self.head_dim)
        x, qs = self._rows(batch, q, "q", shape)
        y, os_ = self._rows(batch, out, "out", shape)
        _not_lost(scale, "scale")
        need = self._need(batch, heads, causal, window)
        a = AttendArgs(x, y, qs[0], qs[1], os_[0], os_[1], heads, scale, causal, window)
        at, size = 0, 0
        if workspace is not None:
            if workspace.get_device() != self.device_index or not workspace.is_contiguous():
                raise ValueError("workspace: contiguous, on the cache's device")
            at, size = workspace.data_ptr(), workspace.numel() * workspace.element_size()
        elif need:
            workspace = self._workspace(need, stream)
            at, size = workspace.data_ptr(), need
        code = lib().cp_cache_attend(self._h, batch.ref, C.byref(a), at, size, self._stream(stream))
        if code:
            raise CPError(code, "cp_cache_attend")

    def workspace_bytes(self, batch: Batch, q_heads: int, causal: bool = True, window: int = 0) -> int:
        """What ``attend`` needs for this batch, whatever its arrays hold."""
        return self._need(batch, int(q_heads), causal, window)

    def _need(self, batch, heads, causal, window):
        key = (self.layout, heads, bool(causal), window)
        if key not in batch.plans:
            _int32(window, "window")
            a = AttendArgs(16, 32, 0, 0, 0, 0, heads, 0.0, causal, window)
            need = C.c_size_t()
            _check(lib().cp_cache_check(C.byref(self.desc), batch.ref, None, C.byref(a), C.byref(need)), "cp_cache_attend")
            batch.plans[key] = need.value
        return batch.plans[key]

    def _rows(self, batch, t, what, shape):
        """Address of a row array and the strides of its axes but the last (0 where it has one entry at most)."""
        strides = t.stride()
        if t.shape != shape or t.dtype not in self.kinds or strides[-1] != 1 and shape[-1] > 1:
            raise ValueError(f"{what}: bf16 (or int16) {list(shape)}, the last axis contiguous; got {list(t.shape)}, "
                             f"strides {strides}, {t.dtype}")
        if t.get_device() != self.device_index or batch.device_index != self.device_index:
            raise ValueError(f"{what}, or the batch: on another device than the cache's")
        if shape[0] > 1 and strides[0] > 0 < strides[-2]:
            return t.data_ptr(), strides
        if any(n > 1 and s <= 0 for n, s in zip(shape, strides)):
            raise ValueError(f"{what}: entries that share memory (an expanded tensor)")
        return t.data_ptr(), tuple(s if n > 1 else 0 for n, s in zip(shape, strides))

    def _gain(self, t):
        if t is None:
            return 0
        if t.shape != (self.head_dim,) or t.dtype not in self.kinds or t.stride(0) != 1 or t.get_device() != self.device_index:
            raise ValueError("q_norm, k_norm: bf16 [head_dim] on the cache's device")
        return t.data_ptr()

    def _stream(self, stream) -> int:
        return _stream_on(self.device_index, stream)

    def _workspace(self, size, stream):
        return _workspace(self.device, size, stream)

    def status(self) -> int:
        return lib().cp_cache_status(self._h)

    def clear_status(self):
        _check(lib().cp_cache_clear_status(self._h), "cp_cache_clear_status")

    def close(self):
        if getattr(self, "_h", None):
            lib().cp_cache_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def _moves(moves, count, index: int):
    i32, shape = (_torch or _with_torch()).int32, moves.shape
    if moves.dtype is not i32 or len(shape) != 2 or shape[1] != 2 or not moves.is_contiguous() or moves.get_device() != index:
        raise ValueError(f"moves: int32 [capacity][2], contiguous, on cuda:{index}")
    return moves.data_ptr(), _int32(shape[0], "moves"), _array(count, "count", i32, (1,), index)


class Pages:
    """Which pages of a cache, or of several of the same page count and size, hold what (cp_pages_create).

    ``refs`` int32 [pages]: how many table entries name a page (0: free). ``table`` int32 [sequences][width] and
    ``length`` int32 [sequences]: as a Batch's pages and length. Device tensors that the calls read and write; what
    the calls want moved inside the pages stands in ``moves`` (int32 [capacity][2]) and ``count`` (int32 [1]), for
    Cache.copy of each cache."""

    def __init__(self, refs, table, length, page_size: int):
        import torch
        for name, t, dims in (("refs", refs, 1), ("table", table, 2), ("length", length, 1)):
            if t.dtype != torch.int32 or t.dim() != dims or t.device.type != "cuda" or t.device != refs.device or \
                    t.shape[-1] > 1 and t.stride(-1) != 1:
                raise ValueError(f"{name}: int32, {dims} axes, contiguous, on one GPU")
        if table.shape[0] != length.shape[0]:
            raise ValueError("table [sequences][width] and length [sequences]")
        self.keep = (refs, table, length)
        self.device_index = refs.get_device()
        self.sequences, self.pages = length.shape[0], refs.shape[0]
        self.i32, self.each = torch.int32, (length.shape[0],)
        _with_torch()
        self.desc = PagesDesc(_int32(refs.shape[0], "refs"), _int32(page_size, "page_size"), _int32(length.shape[0], "length"),
                              _int32(table.shape[1], "table"), _stride(table, 0), _ptr(refs), _ptr(table), _ptr(length))
        h = C.c_void_p()
        _check(lib().cp_pages_create(C.byref(self.desc), self.device_index, C.byref(h)), "cp_pages_create")
        self._h = h

    def fork(self, src, dst, stream=None):
        """Sequences dst[i], which hold nothing, become copies of src[i] that share its pages (int32 [n] each)."""
        shape, index = (dst.numel(),), self.device_index
        code = lib().cp_pages_fork(self._h, _array(src, "src", self.i32, shape, index), _array(dst, "dst", self.i32, shape, index),
                                   shape[0], _stream_on(index, stream))
        if code:
            raise CPError(code, "cp_pages_fork")

    def grow(self, add, moves, count, stream=None):
        """Room for add[i] (int32 [sequences]) more positions each; count[0] below 0: the pool lacks that many pages, and
        nothing was changed."""
        m, capacity, n = _moves(moves, count, self.device_index)
        code = lib().cp_pages_grow(self._h, _array(add, "add", self.i32, self.each, self.device_index), m, capacity, n,
                                   _stream_on(self.device_index, stream))
        if code:
            raise CPError(code, "cp_pages_grow")

    def trim(self, keep, stream=None):
        """Each sequence cut to at most keep[i] (int32 [sequences]) positions, pages past them given up."""
        code = lib().cp_pages_trim(self._h, _array(keep, "keep", self.i32, self.each, self.device_index),
                                   _stream_on(self.device_index, stream))
        if code:
            raise CPError(code, "cp_pages_trim")

    def compact(self, moves, count, stream=None):
        """The held pages moved to the pool's front."""
        m, capacity, n = _moves(moves, count, self.device_index)
        code = lib().cp_pages_compact(self._h, m, capacity, n, _stream_on(self.device_index, stream))
        if code:
            raise CPError(code, "cp_pages_compact")

    def status(self) -> int:
        return lib().cp_pages_status(self._h)

    def clear_status(self):
        _check(lib().cp_pages_clear_status(self._h), "cp_pages_clear_status")

    def close(self):
        if getattr(self, "_h", None):
            lib().cp_pages_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class Linear:
    """A projection with 4-bit weights (cp_linear_create), laid out once into memory of its own.

    ``q`` uint8 [features][width / 2], two weights a byte, the even input in the low half; ``scale`` bf16
    [features][width / group] and ``zero`` uint8 of the same shape (None: 8). ``gated``: the first half of the rows is a
    gate projection's, the second an up projection's."""

    def __init__(self, q, scale, zero=None, gated: bool = False, timeout_ns: int = 0, debug_stall: bool = False):
        import torch
        if q.dtype != torch.uint8 or q.dim() != 2 or scale.dim() != 2 or scale.dtype not in (torch.bfloat16, torch.int16) or \
                q.device.type != "cuda":
            raise ValueError("q: uint8 [features][width / 2], scale: bf16 [features][width / group], on a GPU")
        n, half = q.shape
        index = q.get_device()
        if scale.shape[0] != n or not scale.shape[1] or 2 * half % scale.shape[1]:
            raise ValueError("q [features][width / 2] and scale [features][width / group]")
        _array(q, "q", torch.uint8, (n, half), index)
        _array(scale, "scale", scale.dtype, scale.shape, index)
        if zero is not None:
            _array(zero, "zero", torch.uint8, scale.shape, index)
        self.features, self.width, self.group, self.gated = n, 2 * half, 2 * half // scale.shape[1], bool(gated)
        self.outs = n // 2 if gated else n
        self.device_index = index
        self.desc = LinearDesc(_int32(n, "features"), _int32(self.width, "width"), self.group, int(self.gated), _ptr(q), _ptr(scale),
                               _ptr(zero) or None, _int64(timeout_ns, "timeout_ns"), int(debug_stall))
        self.dtypes = {torch.bfloat16: 0, torch.float32: 1}
        self.x_dtypes = (torch.bfloat16, torch.int16)
        h = C.c_void_p()
        _check(lib().cp_linear_create(C.byref(self.desc), index, C.byref(h)), "cp_linear_create")
        self._h = h

    def apply(self, x, out, add=None, stream=None):
        """x bf16 [rows][width] into out [rows][features, or half of them if gated], bf16 or fp32; ``add`` of out's type is
        added before the result is rounded."""
        index, rows, out_dtype = self.device_index, x.shape[0], out.dtype
        shape = (rows, self.width)
        if x.dtype not in self.x_dtypes or x.shape != shape or x.get_device() != index:
            raise ValueError(f"x: bf16 [rows][{self.width}] on the weights' device")
        kind = self.dtypes.get(out_dtype)
        if kind is None or out.get_device() != index:
            raise ValueError("out: bf16 or fp32 on the weights' device")
        x_row = 0 if x.is_contiguous() else self._row(x, "x", shape)
        shape = (rows, self.outs)
        if out.shape != shape:
            raise ValueError(f"out: {list(shape)}; got {list(out.shape)}")
        a = LinearArgs(x.data_ptr(), x_row, rows, kind, out.data_ptr(), 0 if out.is_contiguous() else self._row(out, "out", shape))
        if add is not None:
            if add.dtype is not out_dtype or add.get_device() != index:
                raise ValueError("add: of out's type and device")
            a.add, a.add_stride = add.data_ptr(), self._row(add, "add", shape)
        code = lib().cp_linear_apply(self._h, C.byref(a), _stream_on(index, stream))
        if code:
            raise CPError(code, "cp_linear_apply")

    def _row(self, t, what, shape):
        """The stride of t's rows (0 for a single one)."""
        if t.shape != shape:
            raise ValueError(f"{what}: {list(shape)}; got {list(t.shape)}")
        row, one = t.stride()
        if one != 1 and shape[1] > 1:
            raise ValueError(f"{what}: the last axis contiguous")
        if shape[0] <= 1:
            return 0
        if row <= 0:
            raise ValueError(f"{what}: rows that share memory (an expanded tensor)")
        return row

    def unpack(self, out, stream=None):
        """The weights as the bf16 numbers that they stand for, into out [features][width]."""
        if out.dtype not in self.x_dtypes:
            raise ValueError("out: bf16")
        a = _array(out, "out", out.dtype, (self.features, self.width), self.device_index)
        code = lib().cp_linear_unpack(self._h, a, _stream_on(self.device_index, stream))
        if code:
            raise CPError(code, "cp_linear_unpack")

    def status(self) -> int:
        return lib().cp_linear_status(self._h)

    def clear_status(self):
        _check(lib().cp_linear_clear_status(self._h), "cp_linear_clear_status")

    def close(self):
        if getattr(self, "_h", None):
            lib().cp_linear_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


_verify_needs: dict = {}


def verify_workspace_bytes(sequences: int, rows: int, vocab: int) -> int:
    """What ``verify`` needs, whatever its arrays hold."""
    key = (sequences, rows, vocab)
    need = _verify_needs.get(key)
    if need is None:
        a = VerifyArgs(_int32(sequences, "sequences"), _int32(rows, "rows"), _int32(vocab, "vocab"), 0, 16, 16, 0, None, 0, 16, 16, 16,
                       16, 16, 16, None)
        n = C.c_size_t()
        _check(lib().cp_verify_check(C.byref(a), C.byref(n)), "cp_verify")
        if len(_verify_needs) > 4096:
            _verify_needs.clear()
        need = _verify_needs[key] = n.value
    return need


def verify(logits, draft, start, u_accept, u_token, temperature, accepted, token, prob=None, draft_logits=None, workspace=None,
           stream=None):
    """Verification of drafted tokens (cp_verify): how many of each sequence's are taken, and the token behind them.

    ``logits`` bf16 or fp32 [rows][vocab], the target's, and ``draft_logits`` the draft's (None: its tokens were certain);
    ``draft`` int32, ``u_accept`` and ``prob`` fp32 [rows]; ``start`` int32 [sequences + 1]; ``u_token`` and ``temperature`` fp32,
    ``accepted`` and ``token`` int32 [sequences]. Without a ``workspace`` (device bytes, see verify_workspace_bytes) one
    is taken from torch's allocator for this call."""
    torch = _torch or _with_torch()
    f32, i32, index = torch.float32, torch.int32, logits.get_device()
    dtype, shape = logits.dtype, logits.shape
    if dtype is not f32 and dtype is not torch.bfloat16 or index < 0 or len(shape) != 2:
        raise ValueError("logits: bf16 or fp32 [rows][vocab] on a GPU")
    rows, vocab = shape
    n = accepted.numel()
    by_row, by_seq = (rows,), (n,)
    # one expression: a call for each array takes the host longer than a small batch takes the GPU
    if not (start.dtype is i32 and draft.dtype is i32 and accepted.dtype is i32 and token.dtype is i32 and temperature.dtype is f32 and
            u_accept.dtype is f32 and u_token.dtype is f32 and start.shape == (n + 1,) and draft.shape == by_row and
            u_accept.shape == by_row and temperature.shape == by_seq and u_token.shape == by_seq and accepted.shape == by_seq and
            token.shape == by_seq and start.get_device() == index and draft.get_device() == index and
            u_accept.get_device() == index and temperature.get_device() == index and u_token.get_device() == index and
            accepted.get_device() == index and token.get_device() == index and start.is_contiguous() and draft.is_contiguous() and
            u_accept.is_contiguous() and temperature.is_contiguous() and u_token.is_contiguous() and accepted.is_contiguous() and
            token.is_contiguous()):
        for t, what, kind, each in ((start, "start", i32, (n + 1,)), (draft, "draft", i32, by_row), (u_accept, "u_accept", f32, by_row),
                                    (temperature, "temperature", f32, by_seq), (u_token, "u_token", f32, by_seq),
                                    (accepted, "accepted", i32, by_seq), (token, "token", i32, by_seq)):
            _array(t, what, kind, each, index)                # which of them it is
    row = 0 if logits.is_contiguous() else _logits_row(logits)
    draft_at, draft_row = None, 0
    if draft_logits is not None:
        if draft_logits.dtype is not dtype or draft_logits.shape != shape or draft_logits.get_device() != index:
            raise ValueError("draft_logits: of the logits' type, shape and device")
        draft_at, draft_row = draft_logits.data_ptr(), 0 if draft_logits.is_contiguous() else _logits_row(draft_logits)
    need = _verify_needs.get((n, rows, vocab))
    if need is None:
        need = verify_workspace_bytes(n, rows, vocab)
    a = VerifyArgs(n, rows, vocab, 0 if dtype is f32 else 1, start.data_ptr(), logits.data_ptr(), row, draft_at, draft_row,
                   draft.data_ptr(), temperature.data_ptr(), u_accept.data_ptr(), u_token.data_ptr(), accepted.data_ptr(),
                   token.data_ptr(), None if prob is None else _array(prob, "prob", f32, by_row, index))
    at, size = 0, 0
    if workspace is not None:
        if workspace.get_device() != index or not workspace.is_contiguous():
            raise ValueError("workspace: contiguous, on the logits' device")
        at, size = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    elif need:
        workspace = _workspace(logits.device, need, stream)
        at, size = workspace.data_ptr(), need
    code = lib().cp_verify(C.byref(a), index, at, size, _stream_on(index, stream))
    if code:
        raise CPError(code, "cp_verify")


def _logits_row(t) -> int:
    """Elements from row to row; 0 for a single one."""
    row, one = t.stride()
    if t.shape[1] > 1 and one != 1 or t.shape[0] > 1 and row <= 0:
        raise ValueError("logits, draft_logits: the last axis contiguous, rows that share no memory")
    return row if t.shape[0] > 1 else 0


def test_philox(ctr, key, use_curand: bool, out, stream=None):
    n = ctr.shape[0]
    _check(lib().cp_test_philox(_ptr(ctr), _ptr(key), n, int(use_curand), _ptr(out), _stream(stream)),
           "cp_test_philox")


def test_draw(logits, samp: dict, group: int, codes, stream=None):
    rows, vocab = logits.shape
    sp = _sampler(samp)
    _check(lib().cp_test_draw(_ptr(logits), rows, vocab, C.byref(sp), int(group), _ptr(codes),
                              _stream(stream)), "cp_test_draw")
