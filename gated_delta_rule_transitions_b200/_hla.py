"""ctypes binding of libhla.so (argument marshalling only).

Every function here forwards to the C entry point of the same name in
``include/hla.h``.  Tensors are passed as raw device pointers; PyTorch supplies
device memory and the current CUDA stream.  There is no CPU fallback: if the
library or a CUDA device is missing, calls raise.
"""
from __future__ import annotations

import ctypes
import math
import os

import torch

_LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libhla.so")

HLA_OK = 0
HLA_ERR_INVALID_ARG = 1
HLA_ERR_UNSUPPORTED = 2
HLA_ERR_WORKSPACE = 3
HLA_ERR_CUDA = 4
HLA_ERR_TIMEOUT = 5
STATUS_NAMES = {0: "HLA_OK", 1: "HLA_ERR_INVALID_ARG", 2: "HLA_ERR_UNSUPPORTED", 3: "HLA_ERR_WORKSPACE",
                4: "HLA_ERR_CUDA", 5: "HLA_ERR_TIMEOUT"}

HLA_F32 = 0
HLA_BF16 = 1
HLA_CACHE_DENSE = 0
HLA_CACHE_FACTORED = 1
HLA_CACHE_INT8 = 2
CACHE_FORMATS = {"dense": HLA_CACHE_DENSE, "factored": HLA_CACHE_FACTORED, "int8": HLA_CACHE_INT8}
GATE_MODES = {"routed": 0, "one": 1, "zero": 2, "user": 3}
DECAY_MODES = {"scalar": 0, "channel": 1}


class HlaConfig(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int32), ("H", ctypes.c_int32), ("T", ctypes.c_int32), ("C", ctypes.c_int32),
                ("dk", ctypes.c_int32), ("dv", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("gate_mode", ctypes.c_int32), ("cache_format", ctypes.c_int32), ("tau", ctypes.c_float),
                ("bias", ctypes.c_float), ("skip_threshold", ctypes.c_float), ("pool_window", ctypes.c_int32),
                ("decay_mode", ctypes.c_int32)]


class HlaCache(ctypes.Structure):
    _fields_ = [("max_chunks", ctypes.c_int32), ("B", ctypes.c_int32), ("H", ctypes.c_int32),
                ("C", ctypes.c_int32), ("d", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("format", ctypes.c_int32), ("pool_window", ctypes.c_int32), ("decay_mode", ctypes.c_int32),
                ("A", ctypes.c_void_p), ("Bm", ctypes.c_void_p), ("Kf", ctypes.c_void_p), ("Wf", ctypes.c_void_p),
                ("Uf", ctypes.c_void_p), ("df", ctypes.c_void_p), ("rk", ctypes.c_void_p),
                ("buf_k", ctypes.c_void_p), ("buf_v", ctypes.c_void_p), ("buf_qr", ctypes.c_void_p),
                ("buf_kr", ctypes.c_void_p), ("buf_alpha", ctypes.c_void_p), ("buf_beta", ctypes.c_void_p),
                ("n_chunks", ctypes.c_void_p), ("m_partial", ctypes.c_void_p), ("mass", ctypes.c_void_p)]


class GdnConfig(ctypes.Structure):
    _fields_ = [("n_seq", ctypes.c_int32), ("Hk", ctypes.c_int32), ("H", ctypes.c_int32), ("dk", ctypes.c_int32),
                ("dv", ctypes.c_int32), ("dtype", ctypes.c_int32), ("decay_mode", ctypes.c_int32),
                ("n_slots", ctypes.c_int32)]


class HlaError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(f"{STATUS_NAMES.get(status, status)}: {msg}")
        self.status = status


_lib = None

_P = ctypes.c_void_p
_SIGS = {
    "hla_last_error": ([], ctypes.c_char_p),
    "hla_cache_bytes": ([ctypes.POINTER(HlaConfig), ctypes.c_int32], ctypes.c_size_t),
    "hla_cache_init": ([ctypes.POINTER(HlaConfig), ctypes.c_int32, _P, ctypes.c_size_t, ctypes.POINTER(HlaCache), _P],
                       ctypes.c_int),
    "hla_cache_slice": ([ctypes.POINTER(HlaCache), ctypes.c_int32, ctypes.c_int32, ctypes.POINTER(HlaCache)],
                        ctypes.c_int),
    "hla_cache_track_mass": ([ctypes.POINTER(HlaCache), _P, _P], ctypes.c_int),
    "hla_gate_mass": ([ctypes.POINTER(HlaConfig), _P, _P, _P], ctypes.c_int),
    "hla_cache_evict": ([ctypes.POINTER(HlaConfig), ctypes.POINTER(HlaCache), ctypes.POINTER(HlaCache),
                         ctypes.c_int32, ctypes.c_int32, _P, _P], ctypes.c_int),
    "gdn_workspace_bytes": ([ctypes.POINTER(GdnConfig), ctypes.c_int32], ctypes.c_size_t),
    "gdn_forward": ([ctypes.POINTER(GdnConfig), _P, _P, _P, _P, _P, _P, ctypes.c_int32, _P, _P, _P, _P, _P,
                     ctypes.c_size_t, _P], ctypes.c_int),
    "gdn_step": ([ctypes.POINTER(GdnConfig), _P, _P, _P, _P, _P, _P, _P, _P, _P], ctypes.c_int),
    "hla_prefill_workspace_bytes": ([ctypes.POINTER(HlaConfig)], ctypes.c_size_t),
    "hla_decode_workspace_bytes": ([ctypes.POINTER(HlaConfig), ctypes.c_int32], ctypes.c_size_t),
    "gdn_chunk_transitions": ([ctypes.POINTER(HlaConfig), _P, _P, _P, _P, _P, _P, _P], ctypes.c_int),
    "hla_routing": ([ctypes.POINTER(HlaConfig), _P, _P, _P, _P, _P, _P, _P, _P], ctypes.c_int),
    "hla_gate_support": ([ctypes.POINTER(HlaConfig), _P, _P, _P, _P], ctypes.c_int),
    "hla_prefill": ([ctypes.POINTER(HlaConfig), _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P,
                     ctypes.POINTER(HlaCache), _P, ctypes.c_size_t, _P], ctypes.c_int),
    "hla_decode_step": ([ctypes.POINTER(HlaConfig), ctypes.POINTER(HlaCache), _P, _P, _P, _P, _P, _P, _P, _P, _P,
                         ctypes.c_size_t, _P], ctypes.c_int),
    "hla_decode_step_static": ([ctypes.POINTER(HlaConfig), ctypes.POINTER(HlaCache), _P, _P, _P, _P, _P, _P, _P,
                                _P, _P], ctypes.c_int),
    "hla_device_status": ([ctypes.c_int32, ctypes.POINTER(ctypes.c_uint32)], ctypes.c_int),
    "hla_check_bounded_wait": ([ctypes.c_uint32, ctypes.c_int32, _P], ctypes.c_int),
    "hla_profile_enable": ([ctypes.c_int32], ctypes.c_int),
    "hla_profile_read": ([_P, _P, ctypes.c_int32], ctypes.c_int),
}

STAGES = ("pools", "gates", "transitions", "compose", "readout", "cache", "decode", "decode_close", "chain")

# Every symbol that include/hla.h declares (checked by the CPU tests).
EXPORTS = tuple(_SIGS)


def lib():
    """Load libhla.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(_LIB_PATH):
            raise RuntimeError(f"libhla.so not built at {_LIB_PATH}; run "
                               "`python -m gated_delta_rule_transitions_b200.build`")
        L = ctypes.CDLL(_LIB_PATH)
        for name, (args, res) in _SIGS.items():
            fn = getattr(L, name)
            fn.argtypes = args
            fn.restype = res
        _lib = L
    return _lib


def last_error() -> str:
    return lib().hla_last_error().decode()


def _check(status: int):
    if status != HLA_OK:
        raise HlaError(status, last_error())


def make_config(B, H, T, C=64, d=128, dtype="bf16", gate_mode="routed", tau=1.0, bias=0.0,
                skip_threshold=0.0, cache_format="dense", pool_window=0, decay="scalar") -> HlaConfig:
    dt = {"bf16": HLA_BF16, "f32": HLA_F32, torch.bfloat16: HLA_BF16, torch.float32: HLA_F32}[dtype]
    gm = GATE_MODES[gate_mode] if isinstance(gate_mode, str) else int(gate_mode)
    cf = CACHE_FORMATS[cache_format] if isinstance(cache_format, str) else int(cache_format)
    dm = DECAY_MODES[decay] if isinstance(decay, str) else int(decay)
    return HlaConfig(B, H, T, C, d, d, dt, gm, cf, tau, bias, skip_threshold, pool_window, dm)


def _ptr(t):
    if t is None:
        return None
    if not isinstance(t, torch.Tensor):
        raise TypeError("expected a torch.Tensor")
    if not t.is_cuda:
        raise ValueError("libhla takes CUDA device tensors only (no CPU path)")
    if not t.is_contiguous():
        raise ValueError("tensors must be contiguous")
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _scratch(nbytes, device, stream):
    """Device memory for the kernels of one call on `stream` (None: the current one): the allocator
    hands memory out, and on to the next, in the order of the stream that it is asked on."""
    with torch.cuda.stream(stream):
        return torch.empty(max(nbytes, 256), dtype=torch.uint8, device=device)


def _kept(shape, dtype, device, stream):
    """Device memory that a call on `stream` clears and the caller keeps: taken from that stream,
    and, once it is let go, not handed on while the stream that is current here still uses it."""
    with torch.cuda.stream(stream):
        t = torch.empty(shape, dtype=dtype, device=device)
    if stream is not None:
        t.record_stream(torch.cuda.current_stream(t.get_device()))
    return t


def cache_bytes(cfg: HlaConfig, max_chunks: int) -> int:
    return int(lib().hla_cache_bytes(ctypes.byref(cfg), max_chunks))


def prefill_workspace_bytes(cfg: HlaConfig) -> int:
    return int(lib().hla_prefill_workspace_bytes(ctypes.byref(cfg)))


def decode_workspace_bytes(cfg: HlaConfig, max_chunks: int) -> int:
    return int(lib().hla_decode_workspace_bytes(ctypes.byref(cfg), max_chunks))


def _arg(t, name, dtype, shape, device):
    """Device pointer of a tensor argument of the given dtype and shape (or, flattened or split,
    as many elements in another number of dimensions) on CUDA device number `device` (None stays
    None)."""
    if t is None:
        return None
    # the checks in one expression first: a step's binding is most of its time (8 arguments, a
    # launch of 3.5 us: 9.9 us in all with a check of the type and a Stream object, 7.8 without)
    try:
        if t.get_device() == device and t.dtype is dtype and t.shape == shape and t.is_contiguous():
            return t.data_ptr()  # (a CPU tensor's device is -1)
    except AttributeError:
        pass
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name}: libhla takes CUDA device tensors only (no CPU path)")
    if t.get_device() != device:
        raise ValueError(f"{name} is on {t.device}, the call's other tensors on cuda:{device}")
    if t.dtype != dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if t.dim() == len(shape) and t.shape != shape:
        raise ValueError(f"{name}: expected {tuple(shape)}, got {tuple(t.shape)}")
    if t.numel() != math.prod(shape):
        raise ValueError(f"{name}: expected {math.prod(shape)} elements, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _device(t, name):
    """CUDA device number of the tensor that says where a call runs."""
    if type(t) is torch.Tensor and (device := t.get_device()) >= 0:
        return device
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name}: libhla takes CUDA device tensors only (no CPU path)")
    return t.get_device()


# the current device's number (tensors on a device exist, so CUDA is up: no look at that) and the
# handle of a device's current stream: without a Stream object where torch offers that
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda device: torch.cuda.current_stream(device).cuda_stream)


def _run(device, stream, fn, *args):
    """Call fn(*args, stream) with CUDA device number `device` current, on its current stream
    by default."""
    if stream is None:
        s = _raw_stream(device)
    elif stream.device.index != device:
        raise ValueError(f"the stream is on {stream.device}, the tensors on cuda:{device}")
    else:
        s = stream.cuda_stream
    if device == _current_device():
        st = fn(*args, s)
    else:
        with torch.cuda.device(device):
            st = fn(*args, s)
    if st != HLA_OK:
        _check(st)


_F32, _I32 = torch.float32, torch.int32
_DTYPES = {HLA_F32: _F32, HLA_BF16: torch.bfloat16}


class CacheSlice:
    """Sequences [b0, b0 + nb) of a Cache (see Cache.slice)."""

    def __init__(self):
        self.struct = HlaCache()
        self.parent = None
        self.mass = None  # the weights that it points at (the parent may be tracked anew)
        self.max_chunks = 0

    @property
    def device_index(self):
        return self.parent.device_index


class Cache:
    """A decode cache: one caller-owned device block plus the C struct of views."""

    def __init__(self, cfg: HlaConfig, max_chunks: int, device="cuda", stream=None):
        nbytes = cache_bytes(cfg, max_chunks)
        if nbytes == 0:
            raise HlaError(HLA_ERR_UNSUPPORTED, "unsupported cache config")
        self.mass = None  # the weights that it keeps, if any (track_mass)
        self.mem = _kept(nbytes, torch.uint8, device, stream)
        self.struct = HlaCache()
        _run(self.mem.get_device(), stream, lib().hla_cache_init, ctypes.byref(cfg), max_chunks, _ptr(self.mem),
             nbytes, ctypes.byref(self.struct))
        self.cfg = cfg
        self.max_chunks = max_chunks

    @classmethod
    def from_tensors(cls, cfg: HlaConfig, max_chunks: int, **buffers):
        """A cache over the caller's own tensors, one per field of the C struct that the
        format uses (include/hla.h has the shapes), with the state that they hold: nothing
        is copied or cleared.  `mass` is optional (see track_mass)."""
        if not isinstance(max_chunks, int) or max_chunks < 1 or cache_bytes(cfg, max_chunks) == 0:
            raise HlaError(HLA_ERR_UNSUPPORTED, "unsupported cache config")
        B, H, C, d = cfg.B, cfg.H, cfg.C, cfg.dk
        if cfg.cache_format == HLA_CACHE_FACTORED and not (cfg.dtype == HLA_BF16 and d == 128 and C == 64):
            raise HlaError(HLA_ERR_UNSUPPORTED, "a factored cache needs bf16, d = 128 and C = 64")
        dt, f32, i32 = _DTYPES[cfg.dtype], torch.float32, torch.int32
        n = (B, H, max_chunks)
        reps = C // cfg.pool_window if cfg.pool_window else 1
        want = {"rk": (f32, n + (reps, d)), "buf_alpha": (f32, (B, H, C, d) if cfg.decay_mode else (B, H, C)),
                "buf_beta": (f32, (B, H, C)), "n_chunks": (i32, (B,)), "m_partial": (i32, (B,)), "mass": (f32, n)}
        want.update({f: (dt, (B, H, C, d)) for f in ("buf_k", "buf_v", "buf_qr", "buf_kr")})
        if cfg.cache_format == HLA_CACHE_FACTORED:
            want.update({f: (dt, n + (C, d)) for f in ("Kf", "Wf", "Uf")}, df=(f32, n + (C + 4,)))
        elif cfg.cache_format == HLA_CACHE_INT8:
            want.update(A=(torch.int8, n + (d, d)), Bm=(torch.int8, n + (d, d)), df=(f32, n + (4,)))
        else:
            want.update(A=(dt, n + (d, d)), Bm=(dt, n + (d, d)))
        if set(buffers) - set(want) or set(want) - set(buffers) - {"mass"}:
            raise ValueError(f"expected the buffers {sorted(set(want) - {'mass'})} (and mass), got {sorted(buffers)}")
        self = cls.__new__(cls)
        self.struct = HlaCache()
        st = self.struct
        st.max_chunks, st.B, st.H, st.C, st.d, st.dtype = max_chunks, B, H, C, d, cfg.dtype
        st.format, st.pool_window, st.decay_mode = cfg.cache_format, cfg.pool_window, cfg.decay_mode
        device = _device(buffers["rk"], "rk")
        for name, t in buffers.items():
            if t is None and name != "mass":
                raise TypeError(f"{name}: expected a torch.Tensor")
            setattr(st, name, _arg(t, name, *want[name], device))
        self.mem = None
        self.buffers = dict(buffers)  # keeps the memory alive
        self.mass = buffers.get("mass")
        self.cfg = cfg
        self.max_chunks = max_chunks
        return self

    @property
    def device_index(self):
        return (self.mem if self.mem is not None else self.buffers["rk"]).get_device()

    def track_mass(self, mass=None, stream=None):
        """Accumulate every closed chunk's gate weight from now on; returns the
        [B, H, max_chunks] float32 tensor that holds it (given or made here, zeroed).
        untrack_mass stops it."""
        s = self.struct
        device = self.device_index
        shape = (s.B, s.H, s.max_chunks)
        if mass is None:
            mass = _kept(shape, torch.float32, torch.device("cuda", device), stream)
        p = _arg(mass, "mass", torch.float32, shape, device)
        _run(device, stream, lib().hla_cache_track_mass, ctypes.byref(s), p)
        self.mass = mass
        return mass

    def untrack_mass(self, stream=None):
        """Stop accumulating weights (slices taken before go on with theirs)."""
        _run(self.device_index, stream, lib().hla_cache_track_mass, ctypes.byref(self.struct), None)
        self.mass = None

    def slice(self, b0: int, nb: int):
        """The cache of sequences [b0, b0 + nb) (shares this cache's memory)."""
        sub = CacheSlice()
        sub.parent = self
        sub.mass = self.mass
        sub.max_chunks = self.max_chunks
        _check(lib().hla_cache_slice(ctypes.byref(self.struct), b0, nb, ctypes.byref(sub.struct)))
        return sub

    def view(self, field: str, shape, dtype):
        """Torch view of one cache buffer (for tests and inspection)."""
        if field == "mass" or self.mem is None:
            return (self.mass if field == "mass" else self.buffers[field]).view(dtype).view(*shape)
        off = getattr(self.struct, field) - self.mem.data_ptr()
        n = 1
        for s in shape:
            n *= s
        es = torch.empty((), dtype=dtype).element_size()
        return self.mem[off:off + n * es].view(dtype).view(*shape)


def gdn_chunk_transitions(cfg, k, v, alpha, beta, A_out, B_out, stream=None):
    _run(_device(k, "k"), stream, lib().gdn_chunk_transitions, ctypes.byref(cfg), _ptr(k), _ptr(v), _ptr(alpha),
         _ptr(beta), _ptr(A_out), _ptr(B_out))


def hla_routing(cfg, q_route, k_route, rq_out, rk_out, gates_out=None, active_idx_out=None,
                active_cnt_out=None, stream=None):
    _run(_device(q_route, "q_route"), stream, lib().hla_routing, ctypes.byref(cfg), _ptr(q_route), _ptr(k_route),
         _ptr(rq_out), _ptr(rk_out), _ptr(gates_out), _ptr(active_idx_out), _ptr(active_cnt_out))


def hla_gate_support(cfg, gates, mass_out=None, support_out=None, stream=None):
    """Routing mass and effective support per query chunk from a gate matrix."""
    _run(_device(gates, "gates"), stream, lib().hla_gate_support, ctypes.byref(cfg), _ptr(gates), _ptr(mass_out),
         _ptr(support_out))


def hla_gate_mass(cfg, gates, mass_out, stream=None):
    """Weight that every chunk carried over a prompt, from its gate matrix."""
    n = (cfg.T + cfg.C - 1) // cfg.C if cfg.C > 0 else 0
    dev = _device(gates, "gates")
    g = _arg(gates, "gates", torch.float32, (cfg.B, cfg.H, n, n), dev)
    m = _arg(mass_out, "mass_out", torch.float32, (cfg.B, cfg.H, n), dev)
    _run(dev, stream, lib().hla_gate_mass, ctypes.byref(cfg), g, m)
    return mass_out


def hla_cache_evict(cfg, src, dst, keep, recent, kept_out, stream=None):
    """Keep per (sequence, head) the `recent` last chunks of `src` and the heaviest others,
    `keep` in all; `dst` is `src` (in place) or another cache."""
    dev = _device(kept_out, "kept_out")
    for name, c in (("src", src), ("dst", dst)):
        if c.device_index != dev:
            raise ValueError(f"{name} is on cuda:{c.device_index}, kept_out on cuda:{dev}")
    p = _arg(kept_out, "kept_out", torch.int32, (cfg.B, cfg.H, keep), dev)
    _run(dev, stream, lib().hla_cache_evict, ctypes.byref(cfg), ctypes.byref(src.struct),
         ctypes.byref(dst.struct), keep, recent, p)
    return kept_out


def make_gdn_config(n_seq, H, d=128, dtype="bf16", Hk=None, n_slots=None, decay="scalar") -> GdnConfig:
    dt = {"bf16": HLA_BF16, "f32": HLA_F32, torch.bfloat16: HLA_BF16, torch.float32: HLA_F32}[dtype]
    dm = DECAY_MODES[decay] if isinstance(decay, str) else int(decay)
    return GdnConfig(n_seq, H if Hk is None else Hk, H, d, d, dt, dm, n_seq if n_slots is None else n_slots)


def gdn_workspace_bytes(cfg: GdnConfig, T: int) -> int:
    return int(lib().gdn_workspace_bytes(ctypes.byref(cfg), T))


def _gdn_args(cfg, T, H, d, dev, q, k, v, alpha, beta, o):
    dt, hk, hv, h = _DTYPES.get(cfg.dtype), (T, cfg.Hk, d), (T, H, d), (T, H)
    return (_arg(q, "q", dt, hk, dev), _arg(k, "k", dt, hk, dev), _arg(v, "v", dt, hv, dev),
            _arg(alpha, "alpha", _F32, hv if cfg.decay_mode else h, dev), _arg(beta, "beta", _F32, h, dev),
            _arg(o, "o", dt, hv, dev))


def gdn_forward(cfg: GdnConfig, q, k, v, alpha, beta, cu_seqlens, o, state_in=None, state_out=None, slots=None,
                workspace=None, stream=None):
    """Ragged sequences through the gated delta rule, states in and out (include/hla.h)."""
    T, dev, n, H, d = v.shape[0], _device(q, "q"), cfg.n_seq, cfg.H, cfg.dk
    pq, pk, pv, pa, pb, po = _gdn_args(cfg, T, H, d, dev, q, k, v, alpha, beta, o)
    states = (cfg.n_slots, H, cfg.dv, d)
    if workspace is None:
        workspace = _scratch(gdn_workspace_bytes(cfg, T), q.device, stream)
    nb = workspace.numel() * workspace.element_size()
    _run(dev, stream, lib().gdn_forward, ctypes.byref(cfg), pq, pk, pv, pa, pb,
         _arg(cu_seqlens, "cu_seqlens", _I32, (n + 1,), dev), T, _arg(slots, "slots", _I32, (n,), dev),
         _arg(state_in, "state_in", _F32, states, dev), _arg(state_out, "state_out", _F32, states, dev), po,
         _arg(workspace, "workspace", workspace.dtype, workspace.shape, dev), nb)
    return o


def gdn_step(cfg: GdnConfig, q, k, v, alpha, beta, state, o, slots=None, stream=None):
    """One token per sequence through the gated delta rule, the states updated in place."""
    dev, n, H, d = _device(q, "q"), cfg.n_seq, cfg.H, cfg.dk
    pq, pk, pv, pa, pb, po = _gdn_args(cfg, n, H, d, dev, q, k, v, alpha, beta, o)
    _run(dev, stream, lib().gdn_step, ctypes.byref(cfg), pq, pk, pv, pa, pb, _arg(slots, "slots", _I32, (n,), dev),
         _arg(state, "state", _F32, (cfg.n_slots, H, cfg.dv, d), dev), po)
    return o


def hla_prefill(cfg, q, k, v, alpha, beta, o, q_route=None, k_route=None, user_gates=None, gates_out=None,
                active_idx_out=None, active_cnt_out=None, cache: Cache | None = None, workspace=None,
                stream=None):
    dev = _device(q, "q")
    if workspace is None:
        workspace = _scratch(prefill_workspace_bytes(cfg), q.device, stream)
    _run(dev, stream, lib().hla_prefill, ctypes.byref(cfg), _ptr(q), _ptr(k), _ptr(v), _ptr(alpha), _ptr(beta),
         _ptr(q_route), _ptr(k_route), _ptr(user_gates), _ptr(o), _ptr(gates_out), _ptr(active_idx_out),
         _ptr(active_cnt_out), ctypes.byref(cache.struct) if cache is not None else None, _ptr(workspace),
         workspace.numel() * workspace.element_size())
    return o


def hla_decode_step(cfg, cache: Cache, q, k, v, alpha, beta, o, q_route=None, k_route=None, workspace=None,
                    stream=None):
    dev = _device(q, "q")
    if workspace is None:
        workspace = _scratch(decode_workspace_bytes(cfg, cache.max_chunks), q.device, stream)
    _run(dev, stream, lib().hla_decode_step, ctypes.byref(cfg), ctypes.byref(cache.struct), _ptr(q), _ptr(k), _ptr(v),
         _ptr(alpha), _ptr(beta), _ptr(q_route), _ptr(k_route), _ptr(o), _ptr(workspace),
         workspace.numel() * workspace.element_size())
    return o


def hla_decode_step_static(cfg, cache: Cache, q, k, v, alpha, beta, o, q_route=None, k_route=None, stream=None):
    """hla_decode_step with the library's fixed device scratch array: allocates nothing."""
    _run(_device(q, "q"), stream, lib().hla_decode_step_static, ctypes.byref(cfg), ctypes.byref(cache.struct), _ptr(q),
         _ptr(k), _ptr(v), _ptr(alpha), _ptr(beta), _ptr(q_route), _ptr(k_route), _ptr(o))
    return o


def hla_device_status(clear: bool = True):
    code = ctypes.c_uint32(0)
    st = lib().hla_device_status(1 if clear else 0, ctypes.byref(code))
    return st, int(code.value)


def hla_check_bounded_wait(limit_us: int, complete: bool, stream=None):
    """Enqueue the library's bounded-wait check (see include/hla.h)."""
    _check(lib().hla_check_bounded_wait(int(limit_us), 1 if complete else 0, _stream(stream)))


def hla_profile_enable(on: bool = True):
    _check(lib().hla_profile_enable(1 if on else 0))


def hla_profile_read(reset: bool = True):
    """Accumulated per-stage device milliseconds and kernel launches since the last reset."""
    n = len(STAGES)
    ms = (ctypes.c_float * n)()
    la = (ctypes.c_int32 * n)()
    _check(lib().hla_profile_read(ctypes.cast(ms, ctypes.c_void_p), ctypes.cast(la, ctypes.c_void_p),
                                  1 if reset else 0))
    return {STAGES[i]: (float(ms[i]), int(la[i])) for i in range(n)}
