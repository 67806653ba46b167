"""GB300 (sm_103a) causal linear attention with a fixed matrix state.

Thin ctypes binding over the C ABI in ``include/la.h``. Every step of the
operator runs in the CUDA library built from ``csrc/``. This module only
marshals arguments: torch supplies device memory and streams. There is no
fallback. If the library has not been built, or no GB300 is present, the
calls raise.

Low level (same names as the C ABI): ``la_create``, ``la_forward``, ``la_forward_host``,
``la_decode_step``, ``la_status``, ``la_destroy``, ``la_last_error``,
``la_last_launches``, ``la_version``, ``la_forward_noalloc``, ``la_noalloc_status``,
and the ``la_packed_*`` calls (the gated delta rule over packed requests).
Convenience: ``Handle`` and ``PackedHandle`` take torch tensors.
"""
from __future__ import annotations

import ctypes
import os
import threading

from ._build import LIB as LIB_PATH, build  # noqa: F401  (build() compiles in-tree)

LA_NORM_ELU1, LA_GLA, LA_GDN, LA_NORM_DECAY, LA_KDA = 0, 1, 2, 3, 4
LA_BF16, LA_FP32 = 0, 1
LA_OK, LA_ERR_INVALID_ARG, LA_ERR_UNSUPPORTED, LA_ERR_MISALIGNED, LA_ERR_CUDA, LA_ERR_TIMEOUT = range(6)
LA_FLAG_IDENTITY_PHI = 0x1
LA_FLAG_SEQUENTIAL_CHUNKS = 0x2
LA_FLAG_TEST_TIMEOUT = 0x100
LA_PLAN_FAULT_ROWS, LA_PLAN_FAULT_FREE, LA_PLAN_FAULT_SLOT = 1, 2, 4
LA_PLAN_FAULT_OWNER, LA_PLAN_FAULT_STATE, LA_PLAN_FAULT_OVERFLOW = 8, 16, 32

VARIANTS = {"norm": LA_NORM_ELU1, "gla": LA_GLA, "gdn": LA_GDN, "norm_decay": LA_NORM_DECAY, "kda": LA_KDA}
ERRORS = {1: "LA_ERR_INVALID_ARG", 2: "LA_ERR_UNSUPPORTED", 3: "LA_ERR_MISALIGNED",
          4: "LA_ERR_CUDA", 5: "LA_ERR_TIMEOUT"}


class la_config(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int), ("H", ctypes.c_int), ("d_k", ctypes.c_int), ("d_v", ctypes.c_int),
                ("io", ctypes.c_int), ("flags", ctypes.c_uint), ("device", ctypes.c_int)]


class la_packed_config(ctypes.Structure):
    _fields_ = [("max_requests", ctypes.c_int), ("max_tokens", ctypes.c_int), ("slots", ctypes.c_int),
                ("H_k", ctypes.c_int), ("H_v", ctypes.c_int), ("d_k", ctypes.c_int), ("d_v", ctypes.c_int),
                ("io", ctypes.c_int), ("flags", ctypes.c_uint), ("device", ctypes.c_int)]


class LAError(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__(f"{ERRORS.get(code, code)}: {msg}")
        self.code = code


_lock = threading.Lock()
_lib = None


def lib() -> ctypes.CDLL:
    """The loaded CUDA library. Raises if it has not been built."""
    global _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise RuntimeError(
                    f"CUDA library {LIB_PATH} is missing: build it with "
                    "gated_delta_rule_causal_gb300.build() (nvcc, sm_103a)")
            L = ctypes.CDLL(LIB_PATH)
            vp, fp, i = ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int
            L.la_create.argtypes = [ctypes.POINTER(la_config), ctypes.POINTER(ctypes.c_void_p)]
            L.la_create.restype = i
            L.la_forward.argtypes = [vp, vp, vp, vp, fp, fp, fp, vp, fp, fp, i, i, i, vp]
            L.la_forward.restype = i
            L.la_forward_host.argtypes = [vp, vp, vp, vp, fp, fp, fp, vp, fp, fp, i, i, i, vp]
            L.la_forward_host.restype = i
            L.la_decode_step.argtypes = [vp, vp, vp, vp, fp, fp, fp, vp, fp, fp, i, vp]
            L.la_backward.restype = i
            L.la_backward.argtypes = [vp, vp, vp, vp, fp, vp, fp, vp, vp, vp, fp, i, i, vp]
            L.la_backward_gated.restype = i
            L.la_backward_gated.argtypes = [vp, vp, vp, vp, fp, fp, fp, vp, fp, vp, vp, vp, fp, fp, fp, i, i, vp]
            L.la_decode_step.restype = i
            L.la_status.argtypes = [vp, vp]
            L.la_status.restype = i
            L.la_destroy.argtypes = [vp]
            L.la_destroy.restype = None
            L.la_last_error.argtypes = [vp]
            L.la_last_error.restype = ctypes.c_char_p
            L.la_last_launches.argtypes = [vp]
            L.la_last_launches.restype = i
            L.la_version.argtypes = []
            L.la_version.restype = i
            L.la_forward_noalloc.argtypes = [ctypes.POINTER(la_config), vp, vp, vp, fp, fp, fp, vp, fp, fp, i, i, vp]
            L.la_forward_noalloc.restype = i
            L.la_noalloc_status.argtypes = [i, vp]
            L.la_noalloc_status.restype = i
            ll = ctypes.c_longlong
            L.la_packed_plan_words.argtypes = [ctypes.POINTER(la_packed_config)]
            L.la_packed_plan_words.restype = ll
            L.la_packed_create.argtypes = [ctypes.POINTER(la_packed_config), ctypes.POINTER(ctypes.c_void_p)]
            L.la_packed_create.restype = i
            L.la_packed_destroy.argtypes = [vp]
            L.la_packed_destroy.restype = None
            L.la_packed_plan.argtypes = [vp, vp, vp, vp, vp, vp, vp, i, i, vp]
            L.la_packed_plan.restype = i
            L.la_packed_forward.argtypes = [vp, vp, vp, vp, vp, fp, fp, fp, vp, i, i, ll, ll, ll, i, vp]
            L.la_packed_forward.restype = i
            L.la_packed_decode_step.argtypes = [vp, vp, vp, vp, vp, fp, fp, fp, vp, i, i, ll, ll, ll, vp]
            L.la_packed_decode_step.restype = i
            L.la_packed_status.argtypes = [vp, vp]
            L.la_packed_status.restype = i
            L.la_packed_last_error.argtypes = [vp]
            L.la_packed_last_error.restype = ctypes.c_char_p
            L.la_packed_last_launches.argtypes = [vp]
            L.la_packed_last_launches.restype = i
            _lib = L
    return _lib


# ------------------------------------------------------------------ raw ABI

def la_version() -> int:
    return lib().la_version()


def la_create(B, H, d_k, d_v, io=LA_BF16, flags=0, device=0) -> tuple[int, ctypes.c_void_p]:
    h = ctypes.c_void_p()
    cfg = la_config(B, H, d_k, d_v, io, flags, device)
    rc = lib().la_create(ctypes.byref(cfg), ctypes.byref(h))
    return rc, h


def la_forward(h, q, k, v, gate, beta, state_in, out, state_out, den_out, variant, T, chunk, stream) -> int:
    return lib().la_forward(h, q, k, v, gate, beta, state_in, out, state_out, den_out, variant, T, chunk, stream)


def la_forward_host(h, q, k, v, gate, beta, state_in, out, state_out, den_out, variant, T, chunk, stream) -> int:
    """la_forward with every tensor in (page-locked) host memory (see la.h)."""
    return lib().la_forward_host(h, q, k, v, gate, beta, state_in, out, state_out, den_out, variant, T, chunk, stream)


def la_decode_step(h, q, k, v, gate, beta, state_in, out, state_out, den_out, variant, stream) -> int:
    return lib().la_decode_step(h, q, k, v, gate, beta, state_in, out, state_out, den_out, variant, stream)


def la_forward_noalloc(cfg: la_config, q, k, v, gate, beta, state_in, out, state_out, den_out,
                       variant, T, stream) -> int:
    """Prefill without any device allocation by the library (see la.h)."""
    return lib().la_forward_noalloc(ctypes.byref(cfg), q, k, v, gate, beta, state_in, out, state_out,
                                    den_out, variant, T, stream)


def la_noalloc_status(device: int, stream) -> int:
    """Read and clear the status word of la_forward_noalloc calls on `device` (see la.h)."""
    return lib().la_noalloc_status(device, stream)


def la_status(h, stream) -> int:
    return lib().la_status(h, stream)


def la_destroy(h) -> None:
    lib().la_destroy(h)


def la_last_error(h) -> str:
    s = lib().la_last_error(h)
    return s.decode() if s else ""


def la_last_launches(h) -> int:
    return lib().la_last_launches(h)


# ------------------------------------------------------------------ torch marshalling

def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream_ptr(stream):
    import torch
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def state_size(variant: str, d_k: int, d_v: int) -> int:
    """fp32 elements of one sequence-head's state (norm and norm_decay append z)."""
    return d_k * d_v + (d_k if variant in ("norm", "norm_decay") else 0)


class Handle:
    """One configured operator instance (B, H, d_k, d_v, io dtype, device)."""

    def __init__(self, B, H, d_k, d_v, io="bf16", flags=0, device=None):
        import torch
        dev = torch.device("cuda", torch.cuda.current_device() if device is None else device)
        self.B, self.H, self.d_k, self.d_v = B, H, d_k, d_v
        self.io = io
        self.dtype = torch.bfloat16 if io == "bf16" else torch.float32
        self.device = dev
        rc, h = la_create(B, H, d_k, d_v, LA_BF16 if io == "bf16" else LA_FP32, flags, dev.index)
        if rc != LA_OK:
            raise LAError(rc, "la_create failed")
        self._h = h

    def close(self):
        if getattr(self, "_h", None):
            la_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def _check(self, rc):
        if rc != LA_OK:
            raise LAError(rc, la_last_error(self._h))

    def _expect(self, name, t, shape, dtype):
        import torch
        if t is None:
            return
        if not isinstance(t, torch.Tensor) or t.device != self.device or t.dtype != dtype:
            raise ValueError(f"{name}: expected a {dtype} tensor on {self.device}")
        if tuple(t.shape) != tuple(shape) or not t.is_contiguous():
            raise ValueError(f"{name}: expected contiguous shape {tuple(shape)}, got {tuple(t.shape)}")

    def forward(self, q, k, v, gate=None, beta=None, state_in=None, *, variant="gdn", chunk=0,
                out=None, state_out=None, den_out=None, return_state=True, stream=None):
        """Prefill: q,k [B,H,T,d_k], v [B,H,T,d_v]. Returns (out, state_out, den_out)."""
        import torch
        var = VARIANTS[variant]
        B, H, T = q.shape[0], q.shape[1], q.shape[2]
        if (B, H) != (self.B, self.H):
            raise ValueError("q batch/heads differ from the handle's")
        self._expect("q", q, (B, H, T, self.d_k), self.dtype)
        self._expect("k", k, (B, H, T, self.d_k), self.dtype)
        self._expect("v", v, (B, H, T, self.d_v), self.dtype)
        if var == LA_GLA:
            self._expect("gate", gate, (B, H, T, self.d_k), torch.float32)
        elif var == LA_KDA:
            self._expect("gate", gate, (B, H, T, self.d_k), torch.float32)
            self._expect("beta", beta, (B, H, T), torch.float32)
        elif var == LA_NORM_DECAY:
            self._expect("gate", gate, (B, H), torch.float32)
        elif var == LA_GDN:
            self._expect("gate", gate, (B, H, T), torch.float32)
            self._expect("beta", beta, (B, H, T), torch.float32)
        ss = state_size(variant, self.d_k, self.d_v)
        self._expect("state_in", state_in, (B, H, ss), torch.float32)
        if out is None:
            out = torch.empty((B, H, T, self.d_v), dtype=self.dtype, device=self.device)
        if state_out is None and return_state:
            state_out = torch.empty((B, H, ss), dtype=torch.float32, device=self.device)
        rc = la_forward(self._h, _ptr(q), _ptr(k), _ptr(v), _ptr(gate), _ptr(beta), _ptr(state_in),
                        _ptr(out), _ptr(state_out), _ptr(den_out), var, T, chunk, _stream_ptr(stream))
        self._check(rc)
        return out, state_out, den_out

    def forward_host(self, q, k, v, gate=None, beta=None, state_in=None, *, variant="gdn", chunk=0,
                     out=None, state_out=None, den_out=None, return_state=True, stream=None):
        """Prefill from pinned host tensors (CPU, ``pin_memory()``); the outputs
        are pinned host tensors too. The copies overlap the kernels inside the
        library. Returns (out, state_out, den_out), complete once ``stream``
        (default: the current stream) reaches the end of the call."""
        import torch
        var = VARIANTS[variant]
        B, H, T = q.shape[0], q.shape[1], q.shape[2]
        if (B, H) != (self.B, self.H):
            raise ValueError("q batch/heads differ from the handle's")
        cpu = torch.device("cpu")

        def chk(name, t, shape, dtype):
            if t is None:
                return
            if not isinstance(t, torch.Tensor) or t.device != cpu or t.dtype != dtype:
                raise ValueError(f"{name}: expected a {dtype} host tensor")
            if tuple(t.shape) != tuple(shape) or not t.is_contiguous():
                raise ValueError(f"{name}: expected contiguous shape {tuple(shape)}, got {tuple(t.shape)}")

        chk("q", q, (B, H, T, self.d_k), self.dtype)
        chk("k", k, (B, H, T, self.d_k), self.dtype)
        chk("v", v, (B, H, T, self.d_v), self.dtype)
        if var == LA_GLA:
            chk("gate", gate, (B, H, T, self.d_k), torch.float32)
        elif var == LA_KDA:
            chk("gate", gate, (B, H, T, self.d_k), torch.float32)
            chk("beta", beta, (B, H, T), torch.float32)
        elif var == LA_NORM_DECAY:
            chk("gate", gate, (B, H), torch.float32)
        elif var == LA_GDN:
            chk("gate", gate, (B, H, T), torch.float32)
            chk("beta", beta, (B, H, T), torch.float32)
        ss = state_size(variant, self.d_k, self.d_v)
        chk("state_in", state_in, (B, H, ss), torch.float32)
        if out is None:
            out = torch.empty((B, H, T, self.d_v), dtype=self.dtype).pin_memory()
        if state_out is None and return_state:
            state_out = torch.empty((B, H, ss), dtype=torch.float32).pin_memory()
        chk("out", out, (B, H, T, self.d_v), self.dtype)
        chk("state_out", state_out, (B, H, ss), torch.float32)
        rc = la_forward_host(self._h, _ptr(q), _ptr(k), _ptr(v), _ptr(gate), _ptr(beta), _ptr(state_in),
                             _ptr(out), _ptr(state_out), _ptr(den_out), var, T, chunk, _stream_ptr(stream))
        self._check(rc)
        return out, state_out, den_out

    def decode_step(self, q, k, v, gate=None, beta=None, state_in=None, *, variant="gdn",
                    out=None, state_out=None, den_out=None, stream=None):
        """One token: q,k [B,H,d_k], v [B,H,d_v]; state_out may be state_in (in place)."""
        import torch
        var = VARIANTS[variant]
        B, H = self.B, self.H
        self._expect("q", q, (B, H, self.d_k), self.dtype)
        self._expect("k", k, (B, H, self.d_k), self.dtype)
        self._expect("v", v, (B, H, self.d_v), self.dtype)
        ss = state_size(variant, self.d_k, self.d_v)
        if out is None:
            out = torch.empty((B, H, self.d_v), dtype=self.dtype, device=self.device)
        if state_out is None:
            state_out = torch.empty((B, H, ss), dtype=torch.float32, device=self.device)
        rc = la_decode_step(self._h, _ptr(q), _ptr(k), _ptr(v), _ptr(gate), _ptr(beta), _ptr(state_in),
                            _ptr(out), _ptr(state_out), _ptr(den_out), var, _stream_ptr(stream))
        self._check(rc)
        return out, state_out, den_out

    def backward(self, q, k, v, dout, state_in=None, dstate_out=None, *, variant="norm",
                 dq=None, dk=None, dv=None, dstate_in=None, return_dstate=True, stream=None):
        """Gradients of a normalized prefill: q,k [B,H,T,d_k], v and dout
        [B,H,T,d_v]; dstate_out optional. Returns (dq, dk, dv, dstate_in)."""
        import torch
        var = VARIANTS[variant]
        B, H, T = q.shape[0], q.shape[1], q.shape[2]
        if (B, H) != (self.B, self.H):
            raise ValueError("q batch/heads differ from the handle's")
        for name, t, d in (("q", q, self.d_k), ("k", k, self.d_k), ("v", v, self.d_v), ("dout", dout, self.d_v)):
            self._expect(name, t, (B, H, T, d), self.dtype)
        ss = state_size(variant, self.d_k, self.d_v)
        self._expect("state_in", state_in, (B, H, ss), torch.float32)
        self._expect("dstate_out", dstate_out, (B, H, ss), torch.float32)
        dq = torch.empty_like(q) if dq is None else dq
        dk = torch.empty_like(k) if dk is None else dk
        dv = torch.empty_like(v) if dv is None else dv
        if dstate_in is None and return_dstate:
            dstate_in = torch.empty((B, H, ss), dtype=torch.float32, device=self.device)
        rc = lib().la_backward(self._h, _ptr(q), _ptr(k), _ptr(v), _ptr(state_in), _ptr(dout), _ptr(dstate_out),
                               _ptr(dq), _ptr(dk), _ptr(dv), _ptr(dstate_in), var, T, _stream_ptr(stream))
        self._check(rc)
        return dq, dk, dv, dstate_in

    def backward_gated(self, q, k, v, gate, beta, dout, state_in=None, dstate_out=None, *, variant="gdn",
                       return_dstate=True, stream=None):
        """Gradients of a gated delta rule prefill (variant "gdn": gate
        [B,H,T]; "kda": gate [B,H,T,d_k]; beta [B,H,T]), of a per-channel
        gated one ("gla": gate [B,H,T,d_k]) or of a normalized one with a fixed
        decay ("norm_decay": gate [B,H]); the last two take no beta. Returns
        (dq, dk, dv, dgate, dbeta, dstate_in); dbeta is None without beta."""
        import torch
        var = VARIANTS[variant]
        B, H, T = q.shape[0], q.shape[1], q.shape[2]
        if (B, H) != (self.B, self.H):
            raise ValueError("q batch/heads differ from the handle's")
        for name, t, d in (("q", q, self.d_k), ("k", k, self.d_k), ("v", v, self.d_v), ("dout", dout, self.d_v)):
            self._expect(name, t, (B, H, T, d), self.dtype)
        gshape = ((B, H, T, self.d_k) if variant in ("kda", "gla") else (B, H) if variant == "norm_decay"
                  else (B, H, T))
        self._expect("gate", gate, gshape, torch.float32)
        if variant in ("gla", "norm_decay"):
            beta = None
        self._expect("beta", beta, (B, H, T), torch.float32)
        ss = state_size(variant, self.d_k, self.d_v)
        self._expect("state_in", state_in, (B, H, ss), torch.float32)
        self._expect("dstate_out", dstate_out, (B, H, ss), torch.float32)
        dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
        dgate = torch.empty_like(gate)
        dbeta = None if beta is None else torch.empty_like(beta)
        dstate_in = torch.empty((B, H, ss), dtype=torch.float32, device=self.device) if return_dstate else None
        rc = lib().la_backward_gated(self._h, _ptr(q), _ptr(k), _ptr(v), _ptr(gate), _ptr(beta), _ptr(state_in),
                                     _ptr(dout), _ptr(dstate_out), _ptr(dq), _ptr(dk), _ptr(dv), _ptr(dgate),
                                     _ptr(dbeta), _ptr(dstate_in), var, T, _stream_ptr(stream))
        self._check(rc)
        return dq, dk, dv, dgate, dbeta, dstate_in

    def last_launches(self) -> int:
        """Kernels the last forward / decode_step call enqueued."""
        return la_last_launches(self._h)

    def status(self, stream=None) -> int:
        """Synchronize the stream and return (and clear) the device status."""
        return la_status(self._h, _stream_ptr(stream))


class PackedPlan:
    """The plan of a step (see la.h): one int32 buffer on the device and its
    sections as views. The views follow the step the plan was last made for."""

    def __init__(self, cfg: la_packed_config, words, device):
        import torch
        self.words = torch.empty(words, dtype=torch.int32, device=device)
        self.cfg = cfg
        self._maxima = cfg.max_requests, cfg.max_tokens, cfg.slots
        self.requests = self.tokens = 0
        self._views = None

    def _set(self, requests, tokens):
        if (requests, tokens) != (self.requests, self.tokens) or self._views is None:
            self.requests, self.tokens = requests, tokens
            pad = lambda n: (n + 3) // 4 * 4   # noqa: E731
            R, N, w = self.cfg.max_requests, self.cfg.max_tokens, self.words
            offsets = 8
            slots = offsets + pad(R + 1)
            order = slots + pad(R)
            treq = order + pad(R) + 4 * R
            tpos = treq + pad(N)
            self._views = (w[:4], w[offsets:offsets + requests + 1], w[slots:slots + requests],
                           w[order:order + requests], w[treq:treq + tokens], w[tpos:tpos + tokens])

    def _section(self, i):
        if self._views is None:
            raise ValueError("plan: no step has been planned in this buffer yet")
        return self._views[i]

    @property
    def counts(self):
        """int32 [4]: rows used, requests taking part, free slots left, faults (LA_PLAN_FAULT_* bits)."""
        return self._section(0)

    @property
    def offsets(self):
        """int32 [requests + 1]: first row of every request."""
        return self._section(1)

    @property
    def state_slots(self):
        """int32 [requests]: state slot of a request that takes part, else -1."""
        return self._section(2)

    @property
    def order(self):
        """int32 [requests]: the order in which the prefill walks the requests."""
        return self._section(3)

    @property
    def token_request(self):
        """int32 [tokens]: every row's request, -1 in rows of none."""
        return self._section(4)

    @property
    def token_position(self):
        """int32 [tokens]: every row's position in its request (tokens seen before included), -1 in rows of none."""
        return self._section(5)


class PackedHandle:
    """The gated delta rule over packed requests with a pool of states: one
    configuration (head counts and sizes, io dtype, the largest step). The
    device is the current one unless given; calls run on ``stream`` or the
    device's current stream."""

    def __init__(self, *, max_requests, max_tokens, slots, H_k, H_v, d_k, d_v, io="bf16", device=None):
        import torch
        if io not in ("bf16", "fp32"):
            raise ValueError(f"io: expected 'bf16' or 'fp32', got {io!r}")
        dev = torch.device("cuda", torch.cuda.current_device() if device is None else device)
        self.device = dev
        self.dtype = torch.bfloat16 if io == "bf16" else torch.float32
        self.H_k, self.H_v, self.d_k, self.d_v, self.slots = H_k, H_v, d_k, d_v, slots
        # what every call looks up: a step of a few tokens takes the GPU less time than its enqueueing takes the host
        self._index, self._i32, self._f32 = dev.index, torch.int32, torch.float32
        self._pool = (slots, H_v, d_v, d_k)
        self._empty, self._cuda = torch.empty, torch.cuda
        self._current_stream = torch._C._cuda_getCurrentRawStream   # the number in torch.cuda.current_stream(device)
        self._lib = lib()
        self.cfg = la_packed_config(max_requests, max_tokens, slots, H_k, H_v, d_k, d_v,
                                    LA_BF16 if io == "bf16" else LA_FP32, 0, dev.index)
        h = ctypes.c_void_p()
        rc = lib().la_packed_create(ctypes.byref(self.cfg), ctypes.byref(h))
        if rc != LA_OK:
            raise LAError(rc, "la_packed_create failed")
        self._h = h
        self._words = lib().la_packed_plan_words(ctypes.byref(self.cfg))
        self._maxima = max_requests, max_tokens, slots

    def close(self):
        if getattr(self, "_h", None):
            lib().la_packed_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def _check(self, rc):
        if rc != LA_OK:
            raise LAError(rc, lib().la_packed_last_error(self._h).decode())

    def _stream(self, stream):
        return self._current_stream(self._index) if stream is None else stream.cuda_stream

    def _expect(self, name, t, shape, dtype):
        if t.dtype is not dtype or t.get_device() != self._index:
            raise ValueError(f"{name}: expected a {dtype} tensor on {self.device}")
        if t.shape != shape or not t.is_contiguous():
            raise ValueError(f"{name}: expected contiguous shape {tuple(shape)}, got {tuple(t.shape)}")

    def _rows(self, name, t, tokens, heads, d):
        """A packed tensor's row stride in elements; heads and channels of a row lie together."""
        if t.dtype is not self.dtype or t.get_device() != self._index:
            raise ValueError(f"{name}: expected a {self.dtype} tensor on {self.device}")
        if t.shape != (tokens, heads, d):
            raise ValueError(f"{name}: expected shape {(tokens, heads, d)}, got {tuple(t.shape)}")
        st = t.stride()
        if tokens and ((st[2] != 1 and d > 1) or (st[1] != d and heads > 1)):
            raise ValueError(f"{name}: the heads and channels of a row have to lie together, got strides {st}")
        return st[0] if tokens > 1 else heads * d

    def new_plan(self) -> PackedPlan:
        """A plan buffer of this handle's maxima; reusable, step after step."""
        return PackedPlan(self.cfg, self._words, self.device)

    def plan(self, lengths, seen, slots, free_slots, free_count, *, tokens, plan=None, stream=None) -> PackedPlan:
        """The plan of a step, made on the device: lengths, seen, slots int32
        [requests], free_slots int32 [slots], free_count int32 [1]; slots and
        the free stack are updated in place. ``tokens``: rows of the step's
        packed tensors. Returns ``plan`` (a new one if None)."""
        if plan is not None:
            self._own(plan)
        elif stream is None:
            plan = self.new_plan()
        else:
            with self._cuda.stream(stream):   # the memory belongs to the stream that writes it
                plan = self.new_plan()
        requests = lengths.numel()
        i32, expect = self._i32, self._expect
        expect("lengths", lengths, (requests,), i32)
        expect("seen", seen, (requests,), i32)
        expect("slots", slots, (requests,), i32)
        expect("free_slots", free_slots, (self.slots,), i32)
        expect("free_count", free_count, (1,), i32)
        self._check(self._lib.la_packed_plan(self._h, lengths.data_ptr(), seen.data_ptr(), slots.data_ptr(),
                                             free_slots.data_ptr(), free_count.data_ptr(), plan.words.data_ptr(), requests,
                                             tokens, self._stream(stream)))
        plan._set(requests, tokens)
        return plan

    def _own(self, plan):
        if plan._maxima != self._maxima or plan.words.get_device() != self._index:
            raise ValueError("plan: made by a handle of another configuration or device")

    def _step(self, call, plan, q, k, v, gate, beta, states, out, stream, *more):
        n, hk, hv, dk, dv = plan.tokens, self.H_k, self.H_v, self.d_k, self.d_v
        index, dtype, f32 = self._index, self.dtype, self._f32
        key, value, scalar = (n, hk, dk), (n, hv, dv), (n, hv)
        qs, ks, vs = q.stride(), k.stride(), v.stride()
        # the usual case in one go; anything else goes through the checks one by one
        if (plan._maxima == self._maxima and plan.words.get_device() == index and n > 1 and
                q.dtype is dtype and q.get_device() == index and q.shape == key and qs[1] == dk and qs[2] == 1 and
                k.dtype is dtype and k.get_device() == index and k.shape == key and ks[1] == dk and ks[2] == 1 and
                v.dtype is dtype and v.get_device() == index and v.shape == value and vs[1] == dv and vs[2] == 1 and
                gate.dtype is f32 and gate.get_device() == index and gate.shape == scalar and gate.is_contiguous() and
                beta.dtype is f32 and beta.get_device() == index and beta.shape == scalar and beta.is_contiguous() and
                states.dtype is f32 and states.get_device() == index and states.shape == self._pool and states.is_contiguous()):
            qs, ks, vs = qs[0], ks[0], vs[0]
        else:
            self._own(plan)
            plan._section(0)   # (refuses a buffer that no plan was made in)
            qs = self._rows("q", q, n, hk, dk)
            ks = self._rows("k", k, n, hk, dk)
            vs = self._rows("v", v, n, hv, dv)
            self._expect("gate", gate, scalar, f32)
            self._expect("beta", beta, scalar, f32)
            self._expect("states", states, self._pool, f32)
        if out is not None:
            self._expect("out", out, value, dtype)
        elif stream is None:
            out = self._empty(value, dtype=dtype, device=self.device)
        else:
            with self._cuda.stream(stream):   # the memory belongs to the stream that writes it
                out = self._empty(value, dtype=dtype, device=self.device)
        rc = call(self._h, plan.words.data_ptr(), q.data_ptr(), k.data_ptr(), v.data_ptr(), gate.data_ptr(),
                  beta.data_ptr(), states.data_ptr(), out.data_ptr(), plan.requests, n, qs, ks, vs, *more,
                  self._current_stream(index) if stream is None else stream.cuda_stream)
        if rc != LA_OK:
            self._check(rc)
        return out

    def forward(self, plan, q, k, v, gate, beta, states, *, chunk=0, out=None, stream=None):
        """Every token of every request of the plan: q, k [tokens, H_k, d_k],
        v [tokens, H_v, d_v] (rows may be strided), gate, beta fp32 [tokens,
        H_v], states fp32 [slots, H_v, d_v, d_k] updated in place. Returns out
        [tokens, H_v, d_v]; rows of no request are not written. ``chunk``: 0
        the default, 1 token by token, 32 or 64 (d_v 128) in blocks of so
        many tokens. By default the form, and with it a request's last bits,
        goes by the whole step's size; chunk 1 and 64 give the same bits in
        any step."""
        return self._step(self._lib.la_packed_forward, plan, q, k, v, gate, beta, states, out, stream, chunk)

    def decode_step(self, plan, q, k, v, gate, beta, states, *, out=None, stream=None):
        """The same for one or a few tokens per request: token by token, each
        state read and written once. States are those after the last token;
        to take tokens back, copy the slots before."""
        return self._step(self._lib.la_packed_decode_step, plan, q, k, v, gate, beta, states, out, stream)

    def last_launches(self) -> int:
        """Kernels the last call enqueued."""
        return lib().la_packed_last_launches(self._h)

    def status(self, stream=None) -> int:
        """Synchronize the stream and return (and clear) the device status."""
        return lib().la_packed_status(self._h, self._stream(stream))
