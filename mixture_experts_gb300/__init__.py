"""GB300-native forward pass of one sparse Mixture-of-Experts layer.

Thin ctypes binding over ``libcoli_moe.so`` (the C ABI in
``include/coli_moe.h``). Every function keeps the C name and argument order;
tensors are passed as device pointers, ``None`` as NULL. Marshalling only:
every step of the layer runs in the library's CUDA kernels, and calling any
of these without the built library raises instead of falling back.

Build with ``mixture_experts_gb300.build()`` (nvcc, sm_103a).
"""
from __future__ import annotations

import ctypes
import os
import re
import threading

F32, BF16, I4G128, MXFP8, MXFP4 = 0, 1, 2, 3, 4
PATH_AUTO, PATH_DECODE, PATH_PREFILL = 0, 1, 2
ROPE_HALF, ROPE_INTERLEAVED = 0, 1
ROPE_NONE, ROPE_LINEAR, ROPE_NTK, ROPE_YARN, ROPE_YARN_INDEX = 0, 1, 2, 3, 19
STATUS = {0: "COLI_OK", -1: "COLI_EINVAL", -2: "COLI_ENOMEM", -3: "COLI_ECUDA",
          -4: "COLI_EUNSUPPORTED", -5: "COLI_EDEVICE", -6: "COLI_ETIMEOUT"}
COLI_OK, COLI_EINVAL, COLI_ENOMEM, COLI_ECUDA = 0, -1, -2, -3
COLI_EUNSUPPORTED, COLI_EDEVICE, COLI_ETIMEOUT = -4, -5, -6
COLI_PERMUTE_STATIC_SCRATCH_BYTES = 65536
COLI_PAGED_DIRECT_TOKENS = 1024

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libcoli_moe.so")
HEADER = os.path.join(os.path.dirname(_HERE), "include", "coli_moe.h")
_lock = threading.Lock()
_lib = None


class ColiError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(f"{STATUS.get(status, status)}: {msg}")
        self.status = status


class coli_moe_config(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in (
        "d_model", "d_ff", "n_experts", "top_k", "max_tokens", "act_dtype", "weight_dtype",
        "has_router_bias", "path", "expert_slots", "max_promotions")]


class coli_moe_weights(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in (
        "w_router", "b_router", "w_gate", "w_up", "w_down", "s_gate", "s_up", "s_down")]


class coli_rope_config(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("rot_dim", "scaling", "original_positions")] + [
        (n, ctypes.c_double) for n in ("base", "factor", "beta_fast", "beta_slow", "amplitude")]


class coli_rotary(ctypes.Structure):
    _fields_ = [("table", ctypes.c_void_p)] + [(n, ctypes.c_int32) for n in (
        "n_positions", "rot_dim", "layout", "inverse")]


class coli_kv_cache(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("k", "v", "k_scale", "v_scale")] + [
        (n, ctypes.c_int32) for n in ("n_pages", "page_size", "n_kv_heads", "head_dim", "dtype")]


class coli_attn_config(ctypes.Structure):
    _fields_ = [("n_q_heads", ctypes.c_int32), ("window", ctypes.c_int32),
                ("scale", ctypes.c_float)]


def build(force: bool = False) -> str:
    from ._build import build as _b
    return _b(force=force)


_SIGS = {
    # name: (restype, [argtypes])  — P pointer, I int32, Z size_t
    "coli_version": ("s", []),
    "coli_status_string": ("s", ["I"]),
    "coli_last_error": ("s", []),
    "coli_device_status": ("I", ["P", "P", "Z"]),
    "coli_moe_create": ("I", ["P", "P", "P", "P", "P", "Z"]),
    "coli_moe_forward": ("I", ["P", "P", "I", "P", "P", "P", "Z"]),
    "coli_moe_forward_host": ("I", ["P", "P", "I", "P", "P", "P", "Z"]),
    "coli_moe_device_status": ("I", ["P", "P", "P", "Z"]),
    "coli_moe_debug_buffers": ("I", ["P"] * 8),
    "coli_moe_copy_debug": ("I", ["P", "I", "P", "P", "P", "P", "P", "P", "P", "P"]),
    "coli_moe_path_for": ("I", ["P", "I"]),
    "coli_moe_residency": ("I", ["P", "P", "P", "P"]),
    "coli_moe_set_timing": ("I", ["P", "I"]),
    "coli_moe_stage_times": ("I", ["P", "P", "I", "P", "P"]),
    "coli_moe_destroy": (None, ["P"]),
    "coli_route_scratch_bytes": ("Z", ["I", "I", "I"]),
    "coli_route_topk": ("I", ["P", "P", "P", "I", "I", "I", "I", "I", "P", "P", "P", "P", "Z",
                              "P"]),
    "coli_permute_scratch_bytes": ("Z", ["I", "I", "I"]),
    "coli_permute": ("I", ["P", "P", "I", "I", "I", "I", "I", "P", "P", "P", "P", "P", "P", "Z",
                           "P"]),
    "coli_expert_ffn": ("I", ["P", "P", "P", "I", "P", "P"]),
    "coli_combine": ("I", ["P", "P", "P", "I", "I", "I", "I", "P", "P"]),
    "coli_selftest_bounded_wait": ("I", ["I", "P"]),
    "coli_permute_noalloc": ("I", ["P", "P", "I", "I", "I", "I", "I", "P", "P", "P", "P", "P",
                                   "P"]),
    "coli_rope_table": ("I", ["P", "I", "P", "P"]),
    "coli_rope_apply": ("I", ["P", "P", "I", "I", "I"] + ["P", "Z", "I", "P", "Z"] * 2 + ["P"]),
    "coli_kv_append": ("I", ["P", "P", "Z", "P", "Z", "P", "I", "P", "P", "P", "Z", "I", "P", "Z",
                             "P"]),
    "coli_kv_read": ("I", ["P", "P", "I", "P", "Z", "P", "Z", "P"]),
    "coli_paged_attention_scratch_bytes": ("Z", ["P", "I", "I"]),
    "coli_paged_attention": ("I", ["P", "P", "P", "Z", "I", "P", "I", "P", "P", "Z", "P", "P",
                                   "Z", "P"]),
}
_CT = {"P": ctypes.c_void_p, "I": ctypes.c_int32, "Z": ctypes.c_size_t, "s": ctypes.c_char_p,
       None: None}


def lib():
    """The loaded library; raises if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise RuntimeError(f"{LIB_PATH} is missing: run mixture_experts_gb300.build()")
            h = ctypes.CDLL(LIB_PATH)
            for name, (res, args) in _SIGS.items():
                fn = getattr(h, name)
                fn.restype = _CT[res]
                fn.argtypes = [_CT[a] for a in args]
            _lib = h
    return _lib


def header_functions() -> list[str]:
    """Names of the functions declared in include/coli_moe.h."""
    text = open(HEADER).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return sorted(set(re.findall(r"\b(coli_\w+)\s*\(", text)))


def _ptr(t):
    if t is None:
        return None
    if isinstance(t, int):
        return t
    if hasattr(t, "data_ptr"):
        return t.data_ptr()
    if isinstance(t, ctypes.c_void_p):
        return t.value
    raise TypeError(f"cannot pass {type(t)} as a pointer")


def _stream(s):
    if s is None:
        import torch
        if not torch.cuda.is_available():
            return 0  # argument validation still runs; nothing is launched
        return torch.cuda.current_stream().cuda_stream
    if isinstance(s, int):
        return s
    return s.cuda_stream


def _check(rc: int, what: str, msg: str | None = None):
    if rc != 0:
        raise ColiError(rc, f"{what}: {msg if msg is not None else last_error()}")


def last_error() -> str:
    return lib().coli_last_error().decode()


# ---- same names as the C ABI ------------------------------------------------------
def coli_version() -> str:
    return lib().coli_version().decode()


def coli_status_string(status: int) -> str:
    return lib().coli_status_string(status).decode()


def coli_device_status(stream=None) -> int:
    buf = ctypes.create_string_buffer(256)
    return lib().coli_device_status(_stream(stream), buf, 256)


def coli_route_scratch_bytes(T: int, d: int, E: int) -> int:
    return lib().coli_route_scratch_bytes(T, d, E)


def coli_route_topk(x, w_router, b_router, T, d, E, k, act, topk_idx, topk_w, gap=None,
                    scratch=None, scratch_bytes=0, stream=None) -> int:
    return lib().coli_route_topk(_ptr(x), _ptr(w_router), _ptr(b_router), T, d, E, k, act,
                                 _ptr(topk_idx), _ptr(topk_w), _ptr(gap), _ptr(scratch),
                                 scratch_bytes, _stream(stream))


def coli_permute_scratch_bytes(T: int, k: int, E: int) -> int:
    return lib().coli_permute_scratch_bytes(T, k, E)


def coli_permute(topk_idx, x, T, d, E, k, act, counts, offsets, row_token, assign_row, x_perm,
                 scratch=None, scratch_bytes=0, stream=None) -> int:
    return lib().coli_permute(_ptr(topk_idx), _ptr(x), T, d, E, k, act, _ptr(counts),
                              _ptr(offsets), _ptr(row_token), _ptr(assign_row), _ptr(x_perm),
                              _ptr(scratch), scratch_bytes, _stream(stream))


def coli_expert_ffn(h, x_perm, offsets, n_rows, y_perm, stream=None) -> int:
    return lib().coli_expert_ffn(_ptr(h), _ptr(x_perm), _ptr(offsets), n_rows, _ptr(y_perm),
                                 _stream(stream))


def coli_combine(y_perm, assign_row, topk_w, T, k, d, out, y, stream=None) -> int:
    return lib().coli_combine(_ptr(y_perm), _ptr(assign_row), _ptr(topk_w), T, k, d, out, _ptr(y),
                              _stream(stream))


def coli_moe_create(cfg: coli_moe_config, weights: coli_moe_weights, stream=None):
    """Returns (status, handle, message)."""
    h = ctypes.c_void_p()
    buf = ctypes.create_string_buffer(512)
    rc = lib().coli_moe_create(ctypes.byref(cfg), ctypes.byref(weights), _stream(stream),
                               ctypes.byref(h), buf, 512)
    return rc, h, buf.value.decode()


def coli_moe_forward(h, x, T, y, stream=None) -> int:
    return lib().coli_moe_forward(_ptr(h), _ptr(x), T, _ptr(y), _stream(stream), None, 0)


def coli_moe_forward_host(h, x_host, T, y_host, stream=None) -> int:
    return lib().coli_moe_forward_host(_ptr(h), _ptr(x_host), T, _ptr(y_host), _stream(stream),
                                       None, 0)


def coli_moe_device_status(h, stream=None) -> int:
    return lib().coli_moe_device_status(_ptr(h), _stream(stream), None, 0)


def coli_moe_copy_debug(h, T, topk_idx=None, topk_w=None, gap=None, counts=None, offsets=None,
                        row_token=None, assign_row=None, stream=None) -> int:
    return lib().coli_moe_copy_debug(_ptr(h), T, _ptr(topk_idx), _ptr(topk_w), _ptr(gap),
                                     _ptr(counts), _ptr(offsets), _ptr(row_token),
                                     _ptr(assign_row), _stream(stream))


def coli_moe_residency(h, n_experts: int, stream=None):
    """(status, slot of each expert (-1: read from host memory), promotions
    since create) of a handle's residency tier; synchronises the stream."""
    slots = (ctypes.c_int32 * n_experts)()
    n = ctypes.c_int64()
    rc = lib().coli_moe_residency(_ptr(h), slots, ctypes.byref(n), _stream(stream))
    return rc, list(slots), n.value


def coli_moe_path_for(h, T) -> int:
    return lib().coli_moe_path_for(_ptr(h), T)


def coli_moe_set_timing(h, enable: bool) -> int:
    return lib().coli_moe_set_timing(_ptr(h), int(bool(enable)))


def coli_moe_stage_times(h):
    """(per-stage ms summed over timed forwards, forwards, kernel launches)."""
    ms = (ctypes.c_float * 5)()
    nf = ctypes.c_int32()
    nl = ctypes.c_int64()
    _check(lib().coli_moe_stage_times(_ptr(h), ms, 5, ctypes.byref(nf), ctypes.byref(nl)),
           "coli_moe_stage_times")
    return list(ms), nf.value, nl.value


def coli_moe_destroy(h) -> None:
    lib().coli_moe_destroy(_ptr(h))


def coli_permute_noalloc(topk_idx, x, T, d, E, k, act, counts, offsets, row_token, assign_row,
                         x_perm, stream=None) -> int:
    """coli_permute without caller scratch, for callers that cannot allocate
    device memory at the call site; its scratch is a fixed area inside the
    library (COLI_PERMUTE_STATIC_SCRATCH_BYTES), shared by all calls."""
    return lib().coli_permute_noalloc(_ptr(topk_idx), _ptr(x), T, d, E, k, act, _ptr(counts),
                                      _ptr(offsets), _ptr(row_token), _ptr(assign_row),
                                      _ptr(x_perm), _stream(stream))


def coli_selftest_bounded_wait(spin_limit: int, stream=None) -> int:
    return lib().coli_selftest_bounded_wait(spin_limit, _stream(stream))


def _ref(struct):
    return None if struct is None else ctypes.byref(struct)


def coli_rope_table(cfg: coli_rope_config, n_positions, table, stream=None) -> int:
    return lib().coli_rope_table(_ref(cfg), n_positions, _ptr(table), _stream(stream))


def coli_rope_apply(rotary: coli_rotary, positions, T, head_dim, act, q, q_stride, n_q_heads,
                    q_out, q_out_stride, k=None, k_stride=0, n_kv_heads=0, k_out=None,
                    k_out_stride=0, stream=None) -> int:
    return lib().coli_rope_apply(_ref(rotary), _ptr(positions), T, head_dim, act, _ptr(q),
                                 q_stride, n_q_heads, _ptr(q_out), q_out_stride, _ptr(k),
                                 k_stride, n_kv_heads, _ptr(k_out), k_out_stride,
                                 _stream(stream))


def coli_kv_append(cache: coli_kv_cache, k, k_stride, v, v_stride, slots, T, rotary=None,
                   positions=None, q=None, q_stride=0, n_q_heads=0, q_out=None, q_out_stride=0,
                   stream=None) -> int:
    return lib().coli_kv_append(_ref(cache), _ptr(k), k_stride, _ptr(v), v_stride, _ptr(slots), T,
                                _ref(rotary), _ptr(positions), _ptr(q), q_stride, n_q_heads,
                                _ptr(q_out), q_out_stride, _stream(stream))


def coli_kv_read(cache: coli_kv_cache, slots, N, k_out, k_out_stride, v_out, v_out_stride,
                 stream=None) -> int:
    return lib().coli_kv_read(_ref(cache), _ptr(slots), N, _ptr(k_out), k_out_stride, _ptr(v_out),
                              v_out_stride, _stream(stream))


def coli_paged_attention_scratch_bytes(cache: coli_kv_cache, B: int, n_q_heads: int) -> int:
    return lib().coli_paged_attention_scratch_bytes(_ref(cache), B, n_q_heads)


def coli_paged_attention(cache: coli_kv_cache, cfg: coli_attn_config, q, q_stride, B, block_table,
                         max_pages, seq_lens, out, out_stride, lse=None, scratch=None,
                         scratch_bytes=0, stream=None) -> int:
    return lib().coli_paged_attention(_ref(cache), _ref(cfg), _ptr(q), q_stride, B,
                                      _ptr(block_table), max_pages, _ptr(seq_lens), _ptr(out),
                                      out_stride, _ptr(lse), _ptr(scratch), scratch_bytes,
                                      _stream(stream))


# ---- convenience -------------------------------------------------------------------
class MoELayer:
    """One MoE layer on the current CUDA device (weights copied at creation).

    ``weights``: dict with w_router, b_router (or None), w_gate, w_up, w_down
    and for int4 s_gate, s_up, s_down — CUDA tensors in the canonical layouts.
    """

    def __init__(self, d_model, d_ff, n_experts, top_k, max_tokens, act_dtype, weight_dtype,
                 weights: dict, path: int = PATH_AUTO, stream=None, expert_slots: int = 0,
                 max_promotions: int = 0):
        import torch
        self.cfg = coli_moe_config(d_model, d_ff, n_experts, top_k, max_tokens, act_dtype,
                                   weight_dtype, int(weights.get("b_router") is not None), path,
                                   expert_slots, max_promotions)
        w = coli_moe_weights(*[_ptr(weights.get(n)) for n in (
            "w_router", "b_router", "w_gate", "w_up", "w_down", "s_gate", "s_up", "s_down")])
        rc, h, msg = coli_moe_create(self.cfg, w, stream)
        _check(rc, "coli_moe_create", msg)
        self.h = h
        self._torch = torch
        self.act_torch = torch.float32 if act_dtype == F32 else torch.bfloat16

    def forward(self, x, y=None, stream=None):
        T = x.shape[0]
        if y is None:
            y = self._torch.empty_like(x)
        _check(coli_moe_forward(self.h, x, T, y, stream), "coli_moe_forward")
        return y

    __call__ = forward

    def forward_host(self, x_host, y_host, stream=None):
        _check(coli_moe_forward_host(self.h, x_host, x_host.shape[0], y_host, stream),
               "coli_moe_forward_host")
        return y_host

    def debug(self, T: int, stream=None) -> dict:
        torch = self._torch
        c = self.cfg
        dev = torch.device("cuda")
        out = {
            "topk_idx": torch.empty(T, c.top_k, dtype=torch.int32, device=dev),
            "topk_w": torch.empty(T, c.top_k, dtype=torch.float32, device=dev),
            "gap": torch.empty(T, dtype=torch.float32, device=dev),
            "counts": torch.empty(c.n_experts, dtype=torch.int32, device=dev),
            "offsets": torch.empty(c.n_experts + 1, dtype=torch.int32, device=dev),
            "row_token": torch.empty(T * c.top_k, dtype=torch.int32, device=dev),
            "assign_row": torch.empty(T * c.top_k, dtype=torch.int32, device=dev),
        }
        _check(coli_moe_copy_debug(self.h, T, out["topk_idx"], out["topk_w"], out["gap"],
                                   out["counts"], out["offsets"], out["row_token"],
                                   out["assign_row"], stream), "coli_moe_copy_debug")
        return out

    def path_for(self, T: int) -> int:
        return coli_moe_path_for(self.h, T)

    def residency(self, stream=None):
        """(slot of each expert, -1 = host memory; promotions since create)."""
        rc, slots, n = coli_moe_residency(self.h, self.cfg.n_experts, stream)
        _check(rc, "coli_moe_residency")
        return slots, n

    def status(self, stream=None) -> int:
        return coli_moe_device_status(self.h, stream)

    def close(self):
        if getattr(self, "h", None) is not None and self.h.value:
            coli_moe_destroy(self.h)
            self.h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


_torch = None


def _t():
    """torch, imported at the first use of a wrapper that takes tensors."""
    global _torch
    if _torch is None:
        import torch
        _torch = torch
    return _torch


def _current_stream(x) -> int:
    """Raw handle of the current stream of tensor x's device: what
    torch.cuda.current_stream(x.device).cuda_stream gives, without building the
    stream object (a decode step's small calls are bound by the host)."""
    return _torch._C._cuda_getCurrentRawStream(x.get_device())


def _current_device() -> int:
    return _torch._C._cuda_getDevice()


def _device_of(name, x) -> int:
    """Index of x's device, which has to be the current one: that is where the library
    launches, and a stream's raw handle does not say whose it is."""
    dev = x.get_device()
    if dev < 0:
        raise ValueError(f"{name}: need a CUDA tensor, got {x.device}")
    if dev != _current_device():
        raise ValueError(f"{name} is on cuda:{dev}, but the current device is "
                         f"cuda:{_current_device()}")
    return dev


def _head_rows(name, x, n_heads, head_dim, dtype, dev=None) -> int:
    """Token stride (elements) of x [T][n_heads][head_dim], whose heads are
    contiguous; raises ValueError on anything the kernels would misread. dev: the
    device of the call."""
    at = x.get_device()
    if x.dim() != 3 or x.dtype is not dtype or at < 0:
        raise ValueError(f"{name}: need a CUDA {dtype} tensor [T][heads][head_dim], got "
                         f"{x.device} {x.dtype} {tuple(x.shape)}")
    if at != dev and dev is not None:
        raise ValueError(f"{name} is on cuda:{at}, not on cuda:{dev}")
    T, h, d = x.shape
    if h != n_heads or d != head_dim:
        raise ValueError(f"{name}: shape {tuple(x.shape)} does not fit {n_heads} heads of "
                         f"{head_dim}")
    s0, s1, s2 = x.stride()
    if (s2 != 1 and d > 1) or (s1 != d and h > 1):
        raise ValueError(f"{name}: a token's heads must be contiguous, strides {x.stride()}")
    return s0 if T > 1 else h * d


def _rank(name, x, n, shape):
    if x.dim() != n:
        raise ValueError(f"{name}: need {shape}, got {tuple(x.shape)}")


def _ids(name, x, n, dev) -> int:
    """Address of a contiguous int32 vector of n entries on device dev."""
    if x.dtype is not _torch.int32 or x.get_device() != dev or x.dim() != 1 or \
            x.shape[0] != n or not x.is_contiguous():
        raise ValueError(f"{name}: need a contiguous int32 vector of {n} on cuda:{dev}, got "
                         f"{x.device} {x.dtype} {tuple(x.shape)}")
    return x.data_ptr()


def _on(stream):
    """Context in which `stream` (a torch stream or a raw handle) is the current
    one, so that what a call allocates belongs to the stream that uses it."""
    import torch
    if isinstance(stream, int):
        stream = torch.cuda.ExternalStream(stream) if stream else torch.cuda.default_stream()
    return torch.cuda.stream(stream)


def _used_here(*tensors):
    """Tells the allocator that work on the current stream uses tensors of other streams,
    whose memory it would otherwise give away as soon as their owner lets go of them."""
    stream = _torch.cuda.current_stream()
    for x in tensors:
        if x is not None:
            x.record_stream(stream)


class Rotary:
    """A rotary table ([n_positions][rot_dim/2][2] f32, cosines and sines) with
    the layout it is applied in: "half" or "interleaved" (or ROPE_*). It serves calls
    on its own device, which has to be the current one."""

    def __init__(self, table, layout="half"):
        torch = _t()
        lay = {"half": ROPE_HALF, "interleaved": ROPE_INTERLEAVED}.get(layout, layout)
        if lay not in (ROPE_HALF, ROPE_INTERLEAVED):
            raise ValueError(f"layout: {layout!r} is not 'half' or 'interleaved'")
        if table.dim() != 3 or table.shape[2] != 2 or not table.is_contiguous() or \
                table.dtype is not torch.float32 or not table.is_cuda:
            raise ValueError("table: need a contiguous f32 CUDA tensor [n_positions][rot/2][2]")
        self.table, self._dev = table, table.get_device()
        self.c = coli_rotary(table.data_ptr(), table.shape[0], 2 * table.shape[1], lay, 0)
        self.c_inverse = coli_rotary(table.data_ptr(), table.shape[0], 2 * table.shape[1], lay, 1)
        self._ref, self._ref_inverse = ctypes.byref(self.c), ctypes.byref(self.c_inverse)

    @classmethod
    def build(cls, rot_dim, n_positions, base=10000.0, layout="half", scaling=ROPE_NONE,
              factor=1.0, original_positions=0, beta_fast=32.0, beta_slow=1.0, amplitude=1.0,
              stream=None):
        """Builds the table (coli_rope_table) and keeps it. ROPE_YARN blends over the turns a
        pair makes, as published; ROPE_YARN_INDEX over its index, as most checkpoints need."""
        torch = _t()
        if stream is not None:
            with _on(stream):
                return cls.build(rot_dim, n_positions, base, layout, scaling, factor,
                                 original_positions, beta_fast, beta_slow, amplitude)
        table = torch.empty(n_positions, rot_dim // 2, 2, dtype=torch.float32, device="cuda")
        cfg = coli_rope_config(rot_dim, scaling, original_positions, base, factor, beta_fast,
                               beta_slow, amplitude)
        _check(coli_rope_table(cfg, n_positions, table), "coli_rope_table")
        return cls(table, layout)


def rope(rotary: Rotary, positions, q, k=None, q_out=None, k_out=None, inverse=False,
         stream=None):
    """Rotated q and k (or (q, None)); q_out / k_out may be q / k themselves.
    inverse=True turns back, which is also the gradient with respect to q and k."""
    if stream is not None:
        with _on(stream):
            out = rope(rotary, positions, q, k, q_out, k_out, inverse)
            _used_here(rotary.table, positions, q, k, q_out, k_out)
            return out
    torch = _torch
    dt = q.dtype
    if dt is torch.bfloat16:
        act = BF16
    elif dt is torch.float32:
        act = F32
    else:
        raise ValueError(f"q: need f32 or bf16, got {dt}")
    _rank("q", q, 3, "[T][heads][head_dim]")
    T, hq, d = q.shape
    dev = _device_of("q", q)
    if rotary._dev != dev:
        raise ValueError(f"the rotary table is on cuda:{rotary._dev}, not on cuda:{dev}")
    qs = _head_rows("q", q, hq, d, dt, dev)
    if q_out is None:
        q_out = torch.empty((T, hq, d), dtype=dt, device=q.device)
        qos = hq * d
    else:
        qos = _head_rows("q_out", q_out, hq, d, dt, dev)
        if q_out.shape[0] != T:
            raise ValueError("q and q_out need the same number of tokens")
    pp = _ids("positions", positions, T, dev)
    kp = kop = None
    hk = ks = kos = 0
    if k is not None:
        _rank("k", k, 3, "[T][heads][head_dim]")
        hk = k.shape[1]
        ks = _head_rows("k", k, hk, d, dt, dev)
        if k_out is None:
            k_out = torch.empty((k.shape[0], hk, d), dtype=dt, device=q.device)
            kos = hk * d
        else:
            kos = _head_rows("k_out", k_out, hk, d, dt, dev)
        if k.shape[0] != T or k_out.shape[0] != T:
            raise ValueError("q and k need the same number of tokens")
        kp, kop = k.data_ptr(), k_out.data_ptr()
    rc = lib().coli_rope_apply(rotary._ref_inverse if inverse else rotary._ref, pp, T, d, act,
                               q.data_ptr(), qs, hq, q_out.data_ptr(), qos, kp, ks, hk, kop, kos,
                               _current_stream(q))
    if rc:
        _check(rc, "coli_rope_apply")
    return q_out, k_out


class PagedKVCache:
    """Pages of keys and values in the caller's tensors: k, v
    [n_pages][n_kv_heads][page_size][row] of float32, bfloat16 or (MX) uint8,
    with MX scales [..][page_size][S] uint8, S = head_dim/32 rounded up to a
    multiple of 4. The format follows from the type and the row length. Calls take
    tensors of the pages' device, which has to be the current one."""

    def __init__(self, k, v, k_scale=None, v_scale=None, head_dim=None):
        torch = _t()
        if k.dim() != 4 or k.shape != v.shape or k.dtype != v.dtype or \
                not (k.is_contiguous() and v.is_contiguous() and k.is_cuda) or \
                v.get_device() != k.get_device():
            raise ValueError("k and v: need equal contiguous CUDA tensors "
                             "[n_pages][n_kv_heads][page_size][row] on one device")
        n_pages, hk, page, row = k.shape
        head_dim = row if head_dim is None else head_dim
        dtype = {(torch.float32, head_dim): F32, (torch.bfloat16, head_dim): BF16,
                 (torch.uint8, head_dim): MXFP8, (torch.uint8, head_dim // 2): MXFP4}.get(
                     (k.dtype, row))
        if dtype is None:
            raise ValueError(f"rows of {row} x {k.dtype} hold no format of head_dim {head_dim}")
        if dtype in (MXFP8, MXFP4):
            want = (n_pages, hk, page, (head_dim // 32 + 3) // 4 * 4)
            for s in (k_scale, v_scale):
                if s is None or tuple(s.shape) != want or s.dtype != torch.uint8 or \
                        not s.is_contiguous() or s.get_device() != k.get_device():
                    raise ValueError(f"k_scale and v_scale: need contiguous uint8 {want} on the "
                                     "device of k and v")
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.n_kv_heads, self.head_dim, self.page_size = hk, head_dim, page
        self._dev = k.get_device()
        self.act_torch = torch.float32 if dtype == F32 else torch.bfloat16
        self.c = coli_kv_cache(_ptr(k), _ptr(v), _ptr(k_scale), _ptr(v_scale), n_pages, page, hk,
                               head_dim, dtype)
        self._ref = ctypes.byref(self.c)
        self._calls = {}

    @classmethod
    def empty(cls, n_pages, page_size, n_kv_heads, head_dim, dtype=BF16):
        """A zeroed pool in format F32, BF16, MXFP8 or MXFP4."""
        torch = _t()
        shape = (n_pages, n_kv_heads, page_size)
        t = {F32: torch.float32, BF16: torch.bfloat16}.get(dtype, torch.uint8)
        row = head_dim // 2 if dtype == MXFP4 else head_dim
        pools = [torch.zeros(*shape, row, dtype=t, device="cuda") for _ in range(2)]
        if dtype in (MXFP8, MXFP4):
            s = (head_dim // 32 + 3) // 4 * 4
            pools += [torch.zeros(*shape, s, dtype=torch.uint8, device="cuda") for _ in range(2)]
        return cls(*pools, head_dim=head_dim)

    def _pools(self):
        return self.k, self.v, self.k_scale, self.v_scale

    def _device(self) -> int:
        """The pool's device, which has to be the current one (see _device_of)."""
        if self._dev != _current_device():
            raise ValueError(f"the cache is on cuda:{self._dev}, but the current device is "
                             f"cuda:{_current_device()}")
        return self._dev

    def append(self, k, v, slots, rotary: Rotary = None, positions=None, q=None, q_out=None,
               stream=None):
        """Stores token t's k[t], v[t] at slots[t] (-1: skipped), keys rotated
        when `rotary` is given; returns the rotated q (None without q)."""
        if stream is not None:
            with _on(stream):
                out = self.append(k, v, slots, rotary, positions, q, q_out)
                _used_here(*self._pools(), k, v, slots, rotary and rotary.table, positions, q,
                           q_out)
                return out
        _rank("k", k, 3, "[T][heads][head_dim]")
        T, hk, d, dt = k.shape[0], self.n_kv_heads, self.head_dim, self.act_torch
        dev = self._device()
        ks = _head_rows("k", k, hk, d, dt, dev)
        vs = _head_rows("v", v, hk, d, dt, dev)
        if v.shape[0] != T:
            raise ValueError("k and v need the same number of tokens")
        at = _ids("slots", slots, T, dev)
        rp = pp = qp = qop = None
        hq = qs = qos = 0
        if rotary is not None:
            if positions is None:
                raise ValueError("a rotary needs positions")
            if rotary._dev != dev:
                raise ValueError(f"the rotary table is on cuda:{rotary._dev}, not on cuda:{dev}")
            rp, pp = rotary._ref, _ids("positions", positions, T, dev)
        if q is not None:
            _rank("q", q, 3, "[T][heads][head_dim]")
            hq = q.shape[1]
            qs = _head_rows("q", q, hq, d, dt, dev)
            if q_out is None:
                q_out = _torch.empty((q.shape[0], hq, d), dtype=dt, device=q.device)
                qos = hq * d
            else:
                qos = _head_rows("q_out", q_out, hq, d, dt, dev)
            if q.shape[0] != T or q_out.shape[0] != T:
                raise ValueError("q and k need the same number of tokens")
            qp, qop = q.data_ptr(), q_out.data_ptr()
        rc = lib().coli_kv_append(self._ref, k.data_ptr(), ks, v.data_ptr(), vs, at, T, rp, pp, qp,
                                  qs, hq, qop, qos, _current_stream(k))
        if rc:
            _check(rc, "coli_kv_append")
        return q_out if q is not None else None

    def read(self, slots, stream=None):
        """(k, v) rows [N][n_kv_heads][head_dim] of slots, zeros for -1."""
        if stream is not None:
            with _on(stream):
                out = self.read(slots)
                _used_here(*self._pools(), slots)
                return out
        _rank("slots", slots, 1, "a vector")
        N, h, d = slots.shape[0], self.n_kv_heads, self.head_dim
        at = _ids("slots", slots, N, self._device())
        k = _torch.empty((N, h, d), dtype=self.act_torch, device=slots.device)
        v = _torch.empty((N, h, d), dtype=self.act_torch, device=slots.device)
        rc = lib().coli_kv_read(self._ref, at, N, k.data_ptr(), h * d, v.data_ptr(), h * d,
                                _current_stream(k))
        if rc:
            _check(rc, "coli_kv_read")
        return k, v

    def attend(self, q, block_table, seq_lens, scale=None, window=0, out=None, return_lse=False,
               stream=None):
        """Attention of one new token a sequence: q [B][n_q_heads][head_dim],
        block_table [B][max_pages] int32, seq_lens [B] int32 -> out like q
        (and lse [B][n_q_heads] f32). scale defaults to head_dim^-0.5."""
        if stream is not None:
            with _on(stream):
                got = self.attend(q, block_table, seq_lens, scale, window, out, return_lse)
                _used_here(*self._pools(), q, block_table, seq_lens, out)
                return got
        torch, d, dt = _torch, self.head_dim, self.act_torch
        _rank("q", q, 3, "[B][heads][head_dim]")
        B, hq = q.shape[0], q.shape[1]
        dev = self._device()
        qs = _head_rows("q", q, hq, d, dt, dev)
        if out is None:
            out = torch.empty((B, hq, d), dtype=dt, device=q.device)
            os_ = hq * d
        else:
            os_ = _head_rows("out", out, hq, d, dt, dev)
            if out.shape[0] != B:
                raise ValueError("q and out need the same number of sequences")
        if block_table.dim() != 2 or block_table.shape[0] != B or \
                block_table.get_device() != dev or block_table.dtype is not torch.int32 or \
                not block_table.is_contiguous():
            raise ValueError(f"block_table: need a contiguous int32 tensor [{B}][max_pages] on "
                             f"cuda:{dev}")
        lens = _ids("seq_lens", seq_lens, B, dev)
        lse = torch.empty((B, hq), dtype=torch.float32, device=q.device) if return_lse else None
        L = lib()
        pages = block_table.shape[1]
        call = self._calls.get((hq, window, scale, B, pages))
        if call is None:  # the call's settings and scratch size, kept for the next step
            cfg = coli_attn_config(hq, window, d ** -0.5 if scale is None else scale)
            n = 0 if B == 0 or pages * self.page_size <= COLI_PAGED_DIRECT_TOKENS else \
                L.coli_paged_attention_scratch_bytes(self._ref, B, hq)
            if len(self._calls) >= 64:
                self._calls.clear()
            call = self._calls[(hq, window, scale, B, pages)] = (cfg, ctypes.byref(cfg), n)
        _, cfg_ref, n = call
        scratch = torch.empty((n,), dtype=torch.uint8, device=q.device) if n else None
        rc = L.coli_paged_attention(self._ref, cfg_ref, q.data_ptr(), qs, B,
                                    block_table.data_ptr(), pages, lens, out.data_ptr(), os_,
                                    None if lse is None else lse.data_ptr(),
                                    None if scratch is None else scratch.data_ptr(), n,
                                    _current_stream(q))
        if rc:
            _check(rc, "coli_paged_attention")
        return (out, lse) if return_lse else out
