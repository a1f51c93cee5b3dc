"""ARL2 hybrid attention layer on B200: Python binding of libarl2.so.

Argument marshalling only: every step of the layer runs in the CUDA
kernels of ``libarl2.so`` (C ABI in ``include/arl2.h``).  PyTorch supplies
device memory and streams.  If the library is missing, importing this
package raises; there is no other implementation to fall back on.

The layer ("Attend Locally, Remember Linearly", technical summary §2.1 and
§2.2), per stream b and head h of one latent frame and denoising pass:

    out = softmax(Q K^T / sqrt(d)) V + (Q W_q[h]) S_{N-1}
    clean pass only, after the read:
    S_N = alpha S_{N-1} + K'^T diag(beta) (V' - K' S_{N-1}),
    K' = rownorm(K W_k[h]), V' = V W_v[h]

and the softmax teacher layer it replaces (TeacherLayer, technical summary
§1 "KV Cache Growth"): frame N attends to the clean keys/values of frames
0..N-1, kept in a KV cache, and bidirectionally to its own.

For softmax layers whose sequences differ in length there is a paged cache
(PagedCache, PagedBatch): new keys and values are written into pages, as they
are or quantised to 8 bits, and attended to with an optional rolling window
and sinks.  RotaryAxes gives q and k rotary positions with up to four axes.
"""
from __future__ import annotations

import ctypes
import os

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libarl2.so")

ARL2_OK = 0
ARL2_ERR_TIMEOUT = -6
ARL2_BF16, ARL2_FP32 = 0, 1
ARL2_IMPL_AUTO, ARL2_IMPL_SIMT = 0, 1
ARL2_GATE_HEADWISE, ARL2_GATE_ELEMENTWISE = 0, 1
ARL2_ACCESS_FRAME, ARL2_ACCESS_TOKEN = 0, 1
ARL2_PAIRS_ADJACENT, ARL2_PAIRS_HALVES = 0, 1
ARL2_FREQS_PER_AXIS, ARL2_FREQS_SHARED = 0, 1
ARL2_CACHE_NATIVE, ARL2_CACHE_E4M3 = 0, 1

EXPORTED = (
    "arl2_create", "arl2_frame_forward", "arl2_frame_forward_host", "arl2_state_reset",
    "arl2_state_get", "arl2_state_set", "arl2_phi_apply", "arl2_device_status",
    "arl2_device_bytes", "arl2_kernel_launches", "arl2_state_update_noalloc", "arl2_destroy",
    "arl2_status_string", "arl2_version", "arl2_gates_apply", "arl2_frame_forward_hidden",
    "arl2_frame_forward_hidden_host", "arl2_selftest_wait_timeout",
    "arl2_kv_create", "arl2_kv_frame_forward", "arl2_kv_frame_forward_host", "arl2_kv_reset",
    "arl2_kv_frames", "arl2_kv_cache_get", "arl2_kv_cache_set", "arl2_kv_device_status", "arl2_kv_device_bytes",
    "arl2_kv_cache_bytes", "arl2_kv_kernel_launches", "arl2_kv_destroy",
    "arl2_rotary_create", "arl2_rotary_apply", "arl2_rotary_destroy",
    "arl2_paged_create", "arl2_paged_write", "arl2_paged_read", "arl2_paged_attend", "arl2_paged_forward",
    "arl2_paged_device_status", "arl2_paged_device_bytes", "arl2_paged_kernel_launches", "arl2_paged_destroy",
)
NOALLOC_MAX_ELEMENTS = 1 << 22


class Arl2Config(ctypes.Structure):
    _fields_ = [
        ("batch", ctypes.c_int), ("heads", ctypes.c_int), ("head_dim", ctypes.c_int),
        ("tokens_per_frame", ctypes.c_int), ("dtype", ctypes.c_int),
        ("w_q", ctypes.c_void_p), ("w_k", ctypes.c_void_p), ("w_v", ctypes.c_void_p),
        ("softmax_scale", ctypes.c_float), ("host_staging", ctypes.c_int), ("impl", ctypes.c_int),
        ("max_ctas", ctypes.c_int), ("gating", ctypes.c_int), ("access", ctypes.c_int),
        ("hidden_dim", ctypes.c_int), ("w_gate", ctypes.c_void_p), ("b_gate", ctypes.c_void_p),
    ]


class Arl2KvConfig(ctypes.Structure):
    _fields_ = [
        ("batch", ctypes.c_int), ("heads", ctypes.c_int), ("head_dim", ctypes.c_int),
        ("tokens_per_frame", ctypes.c_int), ("max_frames", ctypes.c_int), ("dtype", ctypes.c_int),
        ("softmax_scale", ctypes.c_float), ("host_staging", ctypes.c_int), ("impl", ctypes.c_int),
        ("max_ctas", ctypes.c_int),
    ]


class Arl2RotaryConfig(ctypes.Structure):
    _fields_ = [
        ("head_dim", ctypes.c_int), ("axes", ctypes.c_int), ("axis_dim", ctypes.c_int * 4),
        ("base", ctypes.c_double), ("pairs", ctypes.c_int), ("freqs", ctypes.c_int),
    ]


class Arl2PagedConfig(ctypes.Structure):
    _fields_ = [
        ("q_heads", ctypes.c_int), ("kv_heads", ctypes.c_int), ("head_dim", ctypes.c_int),
        ("pages", ctypes.c_int), ("page_tokens", ctypes.c_int), ("dtype", ctypes.c_int),
        ("format", ctypes.c_int), ("softmax_scale", ctypes.c_float), ("impl", ctypes.c_int),
        ("max_ctas", ctypes.c_int),
    ]


class Arl2PagedPool(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
                ("k_scale", ctypes.c_void_p), ("v_scale", ctypes.c_void_p)]


class Arl2PagedBatch(ctypes.Structure):
    _fields_ = [
        ("seqs", ctypes.c_int), ("tokens", ctypes.c_int), ("max_pages", ctypes.c_int), ("max_new", ctypes.c_int),
        ("q_offsets", ctypes.c_void_p), ("kv_lens", ctypes.c_void_p), ("page_table", ctypes.c_void_p),
    ]


def _load() -> ctypes.CDLL:
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is missing: build it with "
                          "`python hybrid_softmax_gated_b200/build.py`")
    lib = ctypes.CDLL(LIB_PATH)
    P, I, S = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
    H = ctypes.c_void_p
    LL = ctypes.c_longlong
    sig = {
        "arl2_create": ([ctypes.POINTER(Arl2Config), P, ctypes.POINTER(H)], I),
        "arl2_frame_forward": ([H, P, P, P, P, P, I, P, P], I),
        "arl2_frame_forward_host": ([H, P, P, P, P, P, I, P, P], I),
        "arl2_state_reset": ([H, P], I),
        "arl2_state_get": ([H, P, P], I),
        "arl2_state_set": ([H, P, P], I),
        "arl2_phi_apply": ([H, I, P, P, P], I),
        "arl2_device_status": ([H, P], I),
        "arl2_device_bytes": ([H], S),
        "arl2_kernel_launches": ([H], ctypes.c_ulonglong),
        "arl2_state_update_noalloc": ([I, I, I, I, I, P, P, P, P, P, P, P, P], I),
        "arl2_destroy": ([H], None),
        "arl2_status_string": ([I], ctypes.c_char_p),
        "arl2_version": ([], I),
        "arl2_gates_apply": ([H, P, P, P, P], I),
        "arl2_frame_forward_hidden": ([H, P, P, P, P, I, P, P], I),
        "arl2_frame_forward_hidden_host": ([H, P, P, P, P, I, P, P], I),
        "arl2_selftest_wait_timeout": ([H, ctypes.c_uint, P], I),
        "arl2_kv_create": ([ctypes.POINTER(Arl2KvConfig), P, ctypes.POINTER(H)], I),
        "arl2_kv_frame_forward": ([H, P, P, P, I, P, P], I),
        "arl2_kv_frame_forward_host": ([H, P, P, P, I, P, P], I),
        "arl2_kv_reset": ([H], I),
        "arl2_kv_frames": ([H], I),
        "arl2_kv_cache_get": ([H, P, P, P], I),
        "arl2_kv_cache_set": ([H, P, P, I, P], I),
        "arl2_kv_device_status": ([H, P], I),
        "arl2_kv_device_bytes": ([H], S),
        "arl2_kv_cache_bytes": ([H], S),
        "arl2_kv_kernel_launches": ([H], ctypes.c_ulonglong),
        "arl2_kv_destroy": ([H], None),
        "arl2_rotary_create": ([ctypes.POINTER(Arl2RotaryConfig), ctypes.POINTER(H)], I),
        "arl2_rotary_apply": ([H, I, I, P, I, P, LL, P, LL, I, P, LL, P, LL, I, P], I),
        "arl2_rotary_destroy": ([H], None),
        "arl2_paged_create": ([ctypes.POINTER(Arl2PagedConfig), P, ctypes.POINTER(H)], I),
        "arl2_paged_write": ([H, P, P, P, LL, P, LL, P], I),
        "arl2_paged_read": ([H, P, I, I, I, P, P, P, P, P, P], I),
        "arl2_paged_attend": ([H, P, P, I, I, I, P, LL, P, P], I),
        "arl2_paged_forward": ([H, P, P, H, P, I, I, I, P, LL, P, LL, P, LL, P, P, P], I),
        "arl2_paged_device_status": ([H, P], I),
        "arl2_paged_device_bytes": ([H], S),
        "arl2_paged_kernel_launches": ([H], ctypes.c_ulonglong),
        "arl2_paged_destroy": ([H], None),
    }
    for name, (args, res) in sig.items():
        f = getattr(lib, name)
        f.argtypes = args
        f.restype = res
    return lib


_lib = _load()


class Arl2Error(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {_lib.arl2_status_string(status).decode()} ({status})")


def _check(status: int, what: str) -> None:
    if status != ARL2_OK:
        raise Arl2Error(status, what)


def _stream(stream) -> int:
    if stream is None:  # the current device's current stream (its handle alone: a Stream object costs 5 us)
        return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())
    return int(stream.cuda_stream) if hasattr(stream, "cuda_stream") else int(stream)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def state_update_noalloc(k, v, w_k, w_v, alpha, beta, state, stream=None) -> None:
    """arl2_state_update_noalloc: the clean-pass update in place on a
    caller-owned fp32 state [B, H, d, d], allocating no device memory."""
    B, L, H, d = k.shape
    dt = ARL2_BF16 if k.dtype == torch.bfloat16 else ARL2_FP32
    _check(_lib.arl2_state_update_noalloc(B, H, d, L, dt, _ptr(k), _ptr(v), _ptr(w_k), _ptr(w_v),
                                          _ptr(alpha), _ptr(beta), _ptr(state), _stream(stream)),
           "arl2_state_update_noalloc")


def library_path() -> str:
    return LIB_PATH


def version() -> int:
    return _lib.arl2_version()


class Arl2Layer:
    """One ARL2 hybrid attention layer: B streams, H heads, width d, L tokens.

    w_q, w_k, w_v: CUDA tensors [H, d, d] in the layer dtype (bf16 or fp32),
    row = input feature.  The handle copies them and owns the fp32 state
    S [B, H, d, d] (zero at creation).  host_staging: 0 none, 1 staging
    buffers for the host-buffer calls, 2 two sets of them whose copies
    overlap the neighbouring calls' work (arl2_config.host_staging).
    """

    def __init__(self, batch: int, heads: int, head_dim: int, tokens: int, w_q, w_k, w_v, *,
                 dtype: torch.dtype = torch.bfloat16, softmax_scale: float = 0.0,
                 host_staging: int = 0, impl: str = "auto", max_ctas: int = 0,
                 gating: str = "headwise", access: str = "frame", gate_weights=None, stream=None):
        if dtype not in (torch.bfloat16, torch.float32):
            raise ValueError("dtype must be torch.bfloat16 or torch.float32")
        for w in (w_q, w_k, w_v):
            if not (w.is_cuda and w.is_contiguous() and w.dtype == dtype):
                raise ValueError("feature maps must be contiguous CUDA tensors of the layer dtype")
            if tuple(w.shape) != (heads, head_dim, head_dim):
                raise ValueError("feature maps must be [H, d, d]")
        self.shape = (batch, tokens, heads, head_dim)
        self.dtype = dtype
        self.device = w_q.device
        self.hidden_dim = 0
        w_gate = b_gate = None
        if gate_weights is not None:
            w_gate, b_gate = gate_weights
            if not (w_gate.is_cuda and w_gate.is_contiguous() and w_gate.dtype == dtype and w_gate.dim() == 2
                    and w_gate.shape[1] == 2 * heads):
                raise ValueError("gate weights must be a contiguous CUDA tensor [D, 2H] of the layer dtype")
            if not (b_gate.is_cuda and b_gate.is_contiguous() and b_gate.dtype == torch.float32
                    and tuple(b_gate.shape) == (2 * heads,)):
                raise ValueError("gate bias must be a contiguous fp32 CUDA tensor [2H]")
            self.hidden_dim = int(w_gate.shape[0])
        cfg = Arl2Config(batch, heads, head_dim, tokens,
                         ARL2_BF16 if dtype == torch.bfloat16 else ARL2_FP32,
                         w_q.data_ptr(), w_k.data_ptr(), w_v.data_ptr(), float(softmax_scale),
                         int(host_staging),
                         {"auto": ARL2_IMPL_AUTO, "simt": ARL2_IMPL_SIMT}[impl], int(max_ctas),
                         {"headwise": ARL2_GATE_HEADWISE, "elementwise": ARL2_GATE_ELEMENTWISE}[gating],
                         {"frame": ARL2_ACCESS_FRAME, "token": ARL2_ACCESS_TOKEN}[access],
                         self.hidden_dim, None if w_gate is None else w_gate.data_ptr(),
                         None if b_gate is None else b_gate.data_ptr())
        self.token_level = access == "token"
        self.alpha_shape = lambda B, H: (B, H, head_dim) if gating == "elementwise" else (B, H)
        h = ctypes.c_void_p()
        with torch.cuda.device(self.device):
            _check(_lib.arl2_create(ctypes.byref(cfg), _stream(stream), ctypes.byref(h)), "arl2_create")
        self._h = h

    # -- helpers --------------------------------------------------------
    def _tok(self, t, name):
        if not (t.is_cuda and t.is_contiguous() and t.dtype == self.dtype):
            raise ValueError(f"{name} must be a contiguous CUDA tensor of the layer dtype")
        if tuple(t.shape) != self.shape:
            raise ValueError(f"{name} must have shape {self.shape}")
        return t

    @property
    def handle(self):
        if self._h is None:
            raise RuntimeError("layer is closed")
        return self._h

    # -- C ABI calls ----------------------------------------------------
    def forward(self, q, k, v, alpha=None, beta=None, clean_pass: bool = False, out=None,
                stream=None):
        """One denoising pass; returns out [B, L, H, d].  alpha [B, H] ([B, H, d]
        with elementwise gating) and beta [B, H, L] (fp32 CUDA) are needed on
        the clean pass only."""
        self._tok(q, "q"), self._tok(k, "k"), self._tok(v, "v")
        if out is None:
            out = torch.empty_like(q)
        self._tok(out, "out")
        B, L, H, _ = self.shape
        gates = clean_pass or self.token_level  # token-level access reads the gates on every pass
        if gates:
            if alpha is None or beta is None:
                raise ValueError("this pass needs alpha and beta")
            if not (alpha.is_cuda and alpha.dtype == torch.float32 and alpha.is_contiguous()
                    and tuple(alpha.shape) == self.alpha_shape(B, H)):
                raise ValueError(f"alpha must be a contiguous fp32 CUDA tensor {list(self.alpha_shape(B, H))}")
            if not (beta.is_cuda and beta.dtype == torch.float32 and beta.is_contiguous()
                    and tuple(beta.shape) == (B, H, L)):
                raise ValueError("beta must be a contiguous fp32 CUDA tensor [B, H, L]")
        _check(_lib.arl2_frame_forward(self.handle, _ptr(q), _ptr(k), _ptr(v),
                                       _ptr(alpha) if gates else None,
                                       _ptr(beta) if gates else None,
                                       1 if clean_pass else 0, _ptr(out), _stream(stream)),
               "arl2_frame_forward")
        return out

    def forward_host(self, q, k, v, alpha, beta, clean_pass: bool, out, stream=None):
        """arl2_frame_forward_host: q, k, v, alpha, beta, out are host (pinned) tensors."""
        for t in (q, k, v, out):
            if t.is_cuda or not t.is_contiguous() or tuple(t.shape) != self.shape or t.dtype != self.dtype:
                raise ValueError("host token tensors must be contiguous CPU tensors of the layer shape")
        gates = clean_pass or self.token_level
        if gates and (alpha is None or beta is None or alpha.is_cuda or beta.is_cuda):
            raise ValueError("this pass needs host alpha and beta")
        _check(_lib.arl2_frame_forward_host(self.handle, _ptr(q), _ptr(k), _ptr(v),
                                            _ptr(alpha) if gates else None,
                                            _ptr(beta) if gates else None,
                                            1 if clean_pass else 0, _ptr(out), _stream(stream)),
               "arl2_frame_forward_host")
        return out

    def _hidden(self, x):
        B, L, _, _ = self.shape
        if not (x.is_cuda and x.is_contiguous() and x.dtype == self.dtype
                and tuple(x.shape) == (B, L, self.hidden_dim)):
            raise ValueError(f"x must be a contiguous CUDA tensor [B, L, D] = {[B, L, self.hidden_dim]}")
        return x

    def gates_apply(self, x, stream=None):
        """arl2_gates_apply: (alpha [B, H], beta [B, H, L]) projected from the
        hidden states x [B, L, D]."""
        B, L, H, _ = self.shape
        self._hidden(x)
        alpha = torch.empty(B, H, dtype=torch.float32, device=self.device)
        beta = torch.empty(B, H, L, dtype=torch.float32, device=self.device)
        _check(_lib.arl2_gates_apply(self.handle, _ptr(x), _ptr(alpha), _ptr(beta), _stream(stream)),
               "arl2_gates_apply")
        return alpha, beta

    def forward_hidden(self, q, k, v, x=None, clean_pass: bool = False, out=None, stream=None):
        """One pass with the gates projected from x [B, L, D] (needed on the
        clean pass, and on every pass with token-level access)."""
        self._tok(q, "q"), self._tok(k, "k"), self._tok(v, "v")
        if out is None:
            out = torch.empty_like(q)
        self._tok(out, "out")
        if x is not None:
            self._hidden(x)
        elif clean_pass or self.token_level:
            raise ValueError("this pass needs the hidden states x")
        _check(_lib.arl2_frame_forward_hidden(self.handle, _ptr(q), _ptr(k), _ptr(v), _ptr(x),
                                              1 if clean_pass else 0, _ptr(out), _stream(stream)),
               "arl2_frame_forward_hidden")
        return out

    def forward_hidden_host(self, q, k, v, x, clean_pass: bool, out, stream=None):
        """arl2_frame_forward_hidden_host: q, k, v, x, out are host (pinned) tensors."""
        B, L, _, _ = self.shape
        for t in (q, k, v, out):
            if t.is_cuda or not t.is_contiguous() or tuple(t.shape) != self.shape or t.dtype != self.dtype:
                raise ValueError("host token tensors must be contiguous CPU tensors of the layer shape")
        if x is not None and (x.is_cuda or not x.is_contiguous() or x.dtype != self.dtype
                              or tuple(x.shape) != (B, L, self.hidden_dim)):
            raise ValueError("x must be a contiguous CPU tensor [B, L, D] of the layer dtype")
        _check(_lib.arl2_frame_forward_hidden_host(self.handle, _ptr(q), _ptr(k), _ptr(v), _ptr(x),
                                                   1 if clean_pass else 0, _ptr(out), _stream(stream)),
               "arl2_frame_forward_hidden_host")
        return out

    def state_reset(self, stream=None) -> None:
        _check(_lib.arl2_state_reset(self.handle, _stream(stream)), "arl2_state_reset")

    def state_get(self, out=None, stream=None):
        B, _, H, d = self.shape
        if out is None:
            out = torch.empty(B, H, d, d, dtype=torch.float32, device=self.device)
        _check(_lib.arl2_state_get(self.handle, _ptr(out), _stream(stream)), "arl2_state_get")
        return out

    def state_set(self, src, stream=None) -> None:
        B, _, H, d = self.shape
        if not (src.is_cuda and src.dtype == torch.float32 and src.is_contiguous()
                and tuple(src.shape) == (B, H, d, d)):
            raise ValueError("state must be a contiguous fp32 CUDA tensor [B, H, d, d]")
        _check(_lib.arl2_state_set(self.handle, _ptr(src), _stream(stream)), "arl2_state_set")

    def phi_apply(self, which: str, x, out=None, stream=None):
        """which in {"q", "k", "v"}: x W_q, rownorm(x W_k) or x W_v."""
        self._tok(x, "x")
        if out is None:
            out = torch.empty_like(x)
        self._tok(out, "out")
        _check(_lib.arl2_phi_apply(self.handle, {"q": 0, "k": 1, "v": 2}[which], _ptr(x), _ptr(out),
                                   _stream(stream)), "arl2_phi_apply")
        return out

    def selftest_wait_timeout(self, limit_us: int, stream=None) -> None:
        """arl2_selftest_wait_timeout: a bounded wait on a word nothing sets,
        which gives up after limit_us and sets the error word."""
        _check(_lib.arl2_selftest_wait_timeout(self.handle, int(limit_us), _stream(stream)),
               "arl2_selftest_wait_timeout")

    def device_status(self, stream=None) -> int:
        """Synchronise and return the device status code (0, or ARL2_ERR_TIMEOUT)."""
        return _lib.arl2_device_status(self.handle, _stream(stream))

    def device_bytes(self) -> int:
        return int(_lib.arl2_device_bytes(self.handle))

    def kernel_launches(self) -> int:
        """Kernels this layer has enqueued (or recorded into a graph) so far."""
        return int(_lib.arl2_kernel_launches(self.handle))

    def close(self) -> None:
        if getattr(self, "_h", None) is not None:
            _lib.arl2_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.close()


class TeacherLayer:
    """The softmax teacher layer with a KV cache (arl2_kv_* in the C ABI).

    One pass of frame N: out = softmax([Q Kc^T, Q K^T] scale) [Vc; V], where
    (Kc, Vc) are the clean keys/values of frames 0..N-1 (the cache) and
    (K, V) the pass's own; a clean pass appends its k, v.  The cache holds up
    to max_frames frames, allocated at creation.
    """

    def __init__(self, batch: int, heads: int, head_dim: int, tokens: int, max_frames: int, *,
                 dtype: torch.dtype = torch.bfloat16, softmax_scale: float = 0.0,
                 host_staging: bool = False, impl: str = "auto", max_ctas: int = 0,
                 device=None, stream=None):
        if dtype not in (torch.bfloat16, torch.float32):
            raise ValueError("dtype must be torch.bfloat16 or torch.float32")
        self.shape = (batch, tokens, heads, head_dim)
        self.dtype = dtype
        self.device = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
        cfg = Arl2KvConfig(batch, heads, head_dim, tokens, max_frames,
                           ARL2_BF16 if dtype == torch.bfloat16 else ARL2_FP32, float(softmax_scale),
                           1 if host_staging else 0,
                           {"auto": ARL2_IMPL_AUTO, "simt": ARL2_IMPL_SIMT}[impl], int(max_ctas))
        h = ctypes.c_void_p()
        with torch.cuda.device(self.device):
            _check(_lib.arl2_kv_create(ctypes.byref(cfg), _stream(stream), ctypes.byref(h)), "arl2_kv_create")
        self._h = h

    def _tok(self, t, name):
        if not (t.is_cuda and t.is_contiguous() and t.dtype == self.dtype):
            raise ValueError(f"{name} must be a contiguous CUDA tensor of the layer dtype")
        if tuple(t.shape) != self.shape:
            raise ValueError(f"{name} must have shape {self.shape}")
        return t

    @property
    def handle(self):
        if self._h is None:
            raise RuntimeError("layer is closed")
        return self._h

    def forward(self, q, k, v, clean_pass: bool = False, out=None, stream=None):
        """One pass of the current frame; returns out [B, L, H, d]."""
        self._tok(q, "q"), self._tok(k, "k"), self._tok(v, "v")
        if out is None:
            out = torch.empty_like(q)
        self._tok(out, "out")
        _check(_lib.arl2_kv_frame_forward(self.handle, _ptr(q), _ptr(k), _ptr(v), 1 if clean_pass else 0,
                                          _ptr(out), _stream(stream)), "arl2_kv_frame_forward")
        return out

    def forward_host(self, q, k, v, clean_pass: bool, out, stream=None):
        """arl2_kv_frame_forward_host: q, k, v, out are host (pinned) tensors."""
        for t in (q, k, v, out):
            if t.is_cuda or not t.is_contiguous() or tuple(t.shape) != self.shape or t.dtype != self.dtype:
                raise ValueError("host token tensors must be contiguous CPU tensors of the layer shape")
        _check(_lib.arl2_kv_frame_forward_host(self.handle, _ptr(q), _ptr(k), _ptr(v), 1 if clean_pass else 0,
                                               _ptr(out), _stream(stream)), "arl2_kv_frame_forward_host")
        return out

    def reset(self) -> None:
        _check(_lib.arl2_kv_reset(self.handle), "arl2_kv_reset")

    def frames(self) -> int:
        return int(_lib.arl2_kv_frames(self.handle))

    def cache_get(self, stream=None):
        """(k, v) in the cache: [B, frames * L, H, d] each."""
        B, L, H, d = self.shape
        n = self.frames() * L
        kc = torch.empty(B, n, H, d, dtype=self.dtype, device=self.device)
        vc = torch.empty_like(kc)
        _check(_lib.arl2_kv_cache_get(self.handle, _ptr(kc), _ptr(vc), _stream(stream)), "arl2_kv_cache_get")
        return kc, vc

    def cache_set(self, k, v, stream=None) -> None:
        """Load the cache from (k, v), [B, n * L, H, d] each (n whole frames)."""
        B, L, H, d = self.shape
        for t in (k, v):
            if not (t.is_cuda and t.is_contiguous() and t.dtype == self.dtype and t.dim() == 4
                    and t.shape[0] == B and t.shape[2:] == (H, d) and t.shape[1] % L == 0):
                raise ValueError("cache tensors must be contiguous CUDA tensors [B, n * L, H, d]")
        if k.shape != v.shape:
            raise ValueError("k and v must have the same shape")
        _check(_lib.arl2_kv_cache_set(self.handle, _ptr(k), _ptr(v), k.shape[1] // L, _stream(stream)),
               "arl2_kv_cache_set")

    def device_status(self, stream=None) -> int:
        return _lib.arl2_kv_device_status(self.handle, _stream(stream))

    def device_bytes(self) -> int:
        return int(_lib.arl2_kv_device_bytes(self.handle))

    def cache_bytes(self) -> int:
        return int(_lib.arl2_kv_cache_bytes(self.handle))

    def kernel_launches(self) -> int:
        return int(_lib.arl2_kv_kernel_launches(self.handle))

    def close(self) -> None:
        if getattr(self, "_h", None) is not None:
            _lib.arl2_kv_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.close()


def _dtype(t: torch.dtype) -> int:
    if t not in (torch.bfloat16, torch.float32):
        raise ValueError("dtype must be torch.bfloat16 or torch.float32")
    return ARL2_BF16 if t == torch.bfloat16 else ARL2_FP32


def _head_rows(t, name, heads, d, dtype, device, tokens=None):
    """A [tokens, heads, d] tensor whose tokens may be strided (a slice of a
    joint qkv projection); returns it."""
    shape = t.shape
    if len(shape) != 3 or shape[1] != heads or shape[2] != d or (tokens is not None and shape[0] != tokens):
        raise ValueError(f"{name} must be [{'tokens' if tokens is None else tokens}, {heads}, {d}]")
    if t.dtype != dtype or t.device != device:
        raise ValueError(f"{name} must be a CUDA tensor of the layer's dtype and device")
    if not t.is_contiguous() and t.numel() and ((d > 1 and t.stride(2) != 1) or (heads > 1 and t.stride(1) != d)
                                                or (shape[0] > 1 and t.stride(0) < heads * d)):
        raise ValueError(f"{name} must have contiguous heads (tokens may be strided)")
    return t


def _token_stride(t) -> int:
    # (the stride of a single token says nothing: dense)
    return 0 if t.is_contiguous() or t.shape[0] <= 1 else t.stride(0)


def _table(t, name, shape, device):
    good = t.dtype == torch.int32 and t.device == device and t.is_contiguous() and t.dim() == len(shape)
    if good:
        for want, n in zip(shape, t.shape):
            good = good and (want is None or want == n)
    if not good:
        raise ValueError(f"{name} must be a contiguous int32 CUDA tensor {['n' if w is None else w for w in shape]}")
    return t


def _side(stream, device):
    """The torch stream that a call's `stream` (a Stream, a raw handle, None)
    stands for, or None if that is the current one."""
    if stream is None:
        return None
    handle = _stream(stream)
    if handle == torch._C._cuda_getCurrentRawStream(device.index):
        return None
    if isinstance(stream, torch.cuda.Stream):
        return stream
    return torch.cuda.ExternalStream(handle, device=device) if handle else torch.cuda.default_stream(device)


def _empty(like, shape, dtype, stream):
    """Memory for a call on `stream`: allocated there, so that it is neither in
    use by the current stream nor given to it while the call runs; the current
    stream, where the caller uses it, is recorded."""
    side = _side(stream, like.device)
    if side is None:
        return like.new_empty(shape, dtype=dtype)
    current = torch.cuda.current_stream(like.device)
    with torch.cuda.stream(side):
        t = like.new_empty(shape, dtype=dtype)
    t.record_stream(current)
    return t


def _like(t, stream):
    if stream is None and t.is_contiguous():
        return torch.empty_like(t)
    return _empty(t, t.shape, t.dtype, stream)


def _mask(block, window, sinks):
    """The mask's sizes as C integers: positions stay below 2^30, so what is
    larger than an int means the same as the largest one (ctypes would take its
    low 32 bits)."""
    if (block | window | sinks) >> 31:  # (a negative one, too: refused by the call)
        block, window, sinks = (max(-1, min(x, 2 ** 31 - 1)) for x in (block, window, sinks))
    return block, window, sinks


class RotaryAxes:
    """Rotary positions with up to four axes (arl2_rotary_* in the C ABI).

    axis_dims: features of a head that each axis turns, in order (even; what
    is left of head_dim passes through).  pairs: "adjacent" (2p, 2p + 1) or
    "halves" (p, p + R/2).  freqs: "per_axis" (each axis runs through all
    frequencies) or "shared" (one run over all axes' pairs).  A plan holds no
    device memory and may be used on any device, stream and thread.  Nothing is
    recorded for autograd: a backward pass calls apply with inverse=True on the
    gradients.
    """

    def __init__(self, head_dim: int, axis_dims, *, base: float = 10000.0, pairs: str = "adjacent",
                 freqs: str = "per_axis"):
        dims = [int(a) for a in axis_dims]
        cfg = Arl2RotaryConfig(head_dim, len(dims), (ctypes.c_int * 4)(*dims[:4]), float(base),
                               {"adjacent": ARL2_PAIRS_ADJACENT, "halves": ARL2_PAIRS_HALVES}[pairs],
                               {"per_axis": ARL2_FREQS_PER_AXIS, "shared": ARL2_FREQS_SHARED}[freqs])
        h = ctypes.c_void_p()
        _check(_lib.arl2_rotary_create(ctypes.byref(cfg), ctypes.byref(h)), "arl2_rotary_create")
        self._h = h
        self.head_dim, self.axes = head_dim, len(dims)

    @property
    def handle(self):
        if self._h is None:
            raise RuntimeError("plan is closed")
        return self._h

    def apply(self, q, k, positions, *, inverse: bool = False, q_out=None, k_out=None, stream=None):
        """(q, k) turned by positions (int32 [tokens, axes]): [tokens, heads, d]
        each, k may be None.  inverse turns back, which is also the gradient.
        q_out, k_out may be q, k (in place)."""
        if not q.is_cuda:
            raise ValueError("q must be a CUDA tensor")
        d, shape, dtype, device = self.head_dim, q.shape, q.dtype, q.device
        tokens, qh = (shape[0], shape[1]) if len(shape) == 3 else (0, 0)
        dt = _dtype(dtype)
        _head_rows(q, "q", qh, d, dtype, device)
        _table(positions, "positions", (tokens, self.axes), device)
        if q_out is None:
            q_out = _like(q, stream)
        else:
            _head_rows(q_out, "q_out", qh, d, dtype, device, tokens)
        kh, ks, kos, kp, kop = 0, 0, 0, None, None
        if k is None:
            k_out = None
        else:
            kh = k.shape[1] if k.dim() == 3 else 0
            _head_rows(k, "k", kh, d, dtype, device, tokens)
            if k_out is None:
                k_out = _like(k, stream)
            else:
                _head_rows(k_out, "k_out", kh, d, dtype, device, tokens)
            ks, kos, kp, kop = _token_stride(k), _token_stride(k_out), k.data_ptr(), k_out.data_ptr()
        if device.index != torch._C._cuda_getDevice():
            raise Arl2Error(-1, "arl2_rotary_apply: the current device is not the tensors'")
        _check(_lib.arl2_rotary_apply(self.handle, dt, tokens, positions.data_ptr(), qh, q.data_ptr(),
                                      _token_stride(q), q_out.data_ptr(), _token_stride(q_out), kh, kp, ks, kop, kos,
                                      1 if inverse else 0,
                                      _stream(stream)), "arl2_rotary_apply")
        return q_out, k_out

    def close(self) -> None:
        if getattr(self, "_h", None) is not None:
            _lib.arl2_rotary_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class PagedBatch:
    """The sequences of a step and their chunks of new tokens (arl2_paged_batch).

    q_offsets: int32 [seqs + 1], rows of each sequence's new tokens in the
    token tensors; kv_lens: int32 [seqs], lengths with the new tokens;
    page_table: int32 [seqs, max_pages].  max_new: the largest number of new
    tokens of a sequence, if known (it picks the kernel).  The tensors are
    read when the kernels run and are kept alive by this object.
    """

    def __init__(self, q_offsets, kv_lens, page_table, *, max_new: int = 0):
        if not q_offsets.is_cuda:
            raise ValueError("q_offsets must be a CUDA tensor")
        self.device = q_offsets.device
        seqs = int(kv_lens.shape[0])
        _table(q_offsets, "q_offsets", (seqs + 1,), self.device)
        _table(kv_lens, "kv_lens", (seqs,), self.device)
        _table(page_table, "page_table", (seqs, None), self.device)
        self.tensors = (q_offsets, kv_lens, page_table)
        self.seqs, self.max_new, self.max_pages = seqs, min(int(max_new), 2 ** 31 - 1), int(page_table.shape[1])
        self._c = {}

    def struct(self, tokens: int):
        c = self._c.get(tokens)
        if c is None:
            q, kv, pt = self.tensors
            c = Arl2PagedBatch(self.seqs, tokens, self.max_pages, self.max_new, q.data_ptr(), kv.data_ptr(),
                               pt.data_ptr())
            self._c = {tokens: c}
        return ctypes.byref(c)


def _check_pool(pool, shape, store, e4m3):
    """A given pool (k_pages, v_pages, k_scales, v_scales), all on one device."""
    k, v, ks, vs = pool
    for t, name, want, sh in ((k, "k_pages", store, shape), (v, "v_pages", store, shape),
                              (ks, "k_scales", torch.float32, shape[:4]), (vs, "v_scales", torch.float32, shape[:4])):
        if name.endswith("scales") and not e4m3:
            if t is not None:
                raise ValueError(f"{name}: this format has none")
        elif t is None or t.dtype != want or tuple(t.shape) != tuple(sh) or not t.is_cuda or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous CUDA tensor {list(sh)} of {want}")
        elif t.device != k.device:
            raise ValueError(f"{name} must be on k_pages' device")
    return k, v, ks, vs


class PagedCache:
    """A paged KV cache and the attention that reads it (arl2_paged_*).

    The pools are tensors of this object: k_pages, v_pages [layers, pages,
    kv_heads, page_tokens, d] in dtype or, with cache_format="e4m3", 8-bit
    codes with k_scales, v_scales fp32 [layers, pages, kv_heads, page_tokens].
    pool: existing ones instead, (k_pages, v_pages, k_scales, v_scales).

    Calls take a stream (a torch stream or a raw handle; default: the current
    one).  What they return may be used on that stream and, once the caller has
    made it wait, on the current one; what they are given has to outlive the
    kernels (record_stream, for a tensor of another stream).  The calls of one
    cache share its workspace: on different streams, or in graphs replayed side
    by side, they must not overlap (two caches may share a pool).  Nothing is
    recorded for autograd.
    """

    def __init__(self, q_heads: int, kv_heads: int, head_dim: int, pages: int, page_tokens: int, *, layers: int = 1,
                 dtype: torch.dtype = torch.bfloat16, cache_format: str = "native", softmax_scale: float = 0.0,
                 impl: str = "auto", max_ctas: int = 0, pool=None, device=None, stream=None):
        dt = _dtype(dtype)
        e4m3 = {"native": False, "e4m3": True}[cache_format]
        self.device = torch.device("cuda" if device is None else device)
        if self.device.type != "cuda":
            raise ValueError("device must be a CUDA device")
        if self.device.index is None:
            self.device = torch.device("cuda", torch.cuda.current_device())
        self.heads, self.head_dim, self.dtype, self.layers = (q_heads, kv_heads), head_dim, dtype, layers
        cfg = Arl2PagedConfig(q_heads, kv_heads, head_dim, pages, page_tokens, dt,
                              ARL2_CACHE_E4M3 if e4m3 else ARL2_CACHE_NATIVE, float(softmax_scale),
                              {"auto": ARL2_IMPL_AUTO, "simt": ARL2_IMPL_SIMT}[impl], int(max_ctas))
        shape = (layers, pages, kv_heads, page_tokens, head_dim)
        store = torch.float8_e4m3fn if e4m3 else dtype
        if pool is not None:
            k, v, ks, vs = _check_pool(pool, shape, store, e4m3)
            self.device = k.device
        h = ctypes.c_void_p()
        with torch.cuda.device(self.device):
            _check(_lib.arl2_paged_create(ctypes.byref(cfg), _stream(stream), ctypes.byref(h)), "arl2_paged_create")
        self._h = h
        if pool is None:  # (cleared on the given stream, like the handle's own memory)
            near = torch.empty(0, device=self.device)
            k, v = (_empty(near, shape, torch.uint8 if e4m3 else dtype, stream) for _ in range(2))
            ks, vs = (_empty(near, shape[:4], torch.float32, stream) if e4m3 else None for _ in range(2))
            side = _side(stream, self.device)
            with torch.cuda.stream(side) if side is not None else torch.cuda.device(self.device):
                for t in (k, v, ks, vs):
                    if t is not None:
                        t.zero_()
            k, v = k.view(store), v.view(store)
        self.k_pages, self.v_pages, self.k_scales, self.v_scales = k, v, ks, vs
        self._pools = [Arl2PagedPool(k[i].data_ptr(), v[i].data_ptr(), None if ks is None else ks[i].data_ptr(),
                                     None if vs is None else vs[i].data_ptr()) for i in range(layers)]

    @property
    def handle(self):
        if self._h is None:
            raise RuntimeError("cache is closed")
        return self._h

    def _pool(self, layer: int):
        if not 0 <= layer < self.layers:
            raise ValueError(f"layer must be in 0..{self.layers - 1}")
        return ctypes.byref(self._pools[layer])

    def _batch(self, batch, tokens):
        if batch.device != self.device:
            raise ValueError("the batch's tables must be on the cache's device")
        return batch.struct(tokens)

    def _rows(self, t, name, kv, tokens=None):
        return _head_rows(t, name, self.heads[kv], self.head_dim, self.dtype, self.device, tokens)

    def _out(self, out, q, stream):
        if out is None:
            return _like(q, stream)
        if not out.is_contiguous():
            raise ValueError("out must be contiguous")
        return self._rows(out, "out", 0, q.shape[0])

    def write(self, k, v, batch: PagedBatch, *, layer: int = 0, stream=None) -> None:
        """The batch's new keys and values ([tokens, kv_heads, d]) into their pages."""
        tokens = k.shape[0]
        self._rows(k, "k", 1), self._rows(v, "v", 1, tokens)
        _check(_lib.arl2_paged_write(self.handle, self._pool(layer), self._batch(batch, tokens), k.data_ptr(),
                                     _token_stride(k), v.data_ptr(), _token_stride(v), _stream(stream)),
               "arl2_paged_write")

    def read(self, page_table, offsets, tokens: int, *, starts=None, layer: int = 0, k_out=None, v_out=None,
             stream=None):
        """(k, v) [tokens, kv_heads, d] read back: rows offsets[s] .. offsets[s + 1]
        - 1 are sequence s's positions from starts[s] (default 0) on."""
        seqs = page_table.shape[0]
        _table(page_table, "page_table", (None, None), self.device)
        _table(offsets, "offsets", (seqs + 1,), self.device)
        if starts is not None:
            _table(starts, "starts", (seqs,), self.device)
        shape = (tokens, self.heads[1], self.head_dim)
        outs = []
        for t, name in ((k_out, "k_out"), (v_out, "v_out")):
            if t is None:
                t = _empty(page_table, shape, self.dtype, stream)
            elif not self._rows(t, name, 1, tokens).is_contiguous():
                raise ValueError(f"{name} must be contiguous")
            outs.append(t)
        _check(_lib.arl2_paged_read(self.handle, self._pool(layer), seqs, tokens, page_table.shape[1],
                                    offsets.data_ptr(), None if starts is None else starts.data_ptr(),
                                    page_table.data_ptr(), outs[0].data_ptr(), outs[1].data_ptr(), _stream(stream)),
               "arl2_paged_read")
        return tuple(outs)

    def attend(self, q, batch: PagedBatch, *, block: int = 1, window: int = 0, sinks: int = 0, layer: int = 0,
               out=None, stream=None):
        """Attention of the new tokens q [tokens, q_heads, d] over their
        sequences' keys: up to the end of their own block of `block` tokens,
        from `window` blocks back (0: from the start), the first `sinks` blocks
        always.  Returns out [tokens, q_heads, d]; rows of no sequence are left
        as they were."""
        self._rows(q, "q", 0)
        out = self._out(out, q, stream)
        _check(_lib.arl2_paged_attend(self.handle, self._pool(layer), self._batch(batch, q.shape[0]),
                                      *_mask(block, window, sinks), q.data_ptr(), _token_stride(q), out.data_ptr(), _stream(stream)),
               "arl2_paged_attend")
        return out

    def forward(self, q, k, v, batch: PagedBatch, *, rotary: RotaryAxes = None, positions=None, block: int = 1,
                window: int = 0, sinks: int = 0, layer: int = 0, out=None, stream=None):
        """One softmax layer's step: q and k turned by `rotary` at `positions`
        (int32 [tokens, axes]; None: not turned), k and v written, then the
        attention of the turned q.  Bit for bit apply, write and attend."""
        tokens = q.shape[0]
        self._rows(q, "q", 0), self._rows(k, "k", 1, tokens), self._rows(v, "v", 1, tokens)
        turned = None
        if rotary is not None:
            if positions is None or rotary.head_dim != self.head_dim:
                raise ValueError("rotary needs positions and the cache's head_dim")
            _table(positions, "positions", (tokens, rotary.axes), self.device)
            turned = _empty(q, (tokens, sum(self.heads), self.head_dim), self.dtype, stream)
        out = self._out(out, q, stream)
        _check(_lib.arl2_paged_forward(self.handle, self._pool(layer), self._batch(batch, tokens),
                                       None if rotary is None else rotary.handle,
                                       None if rotary is None else positions.data_ptr(),
                                       *_mask(block, window, sinks), q.data_ptr(), _token_stride(q), k.data_ptr(), _token_stride(k), v.data_ptr(),
                                       _token_stride(v), None if turned is None else turned.data_ptr(),
                                       out.data_ptr(), _stream(stream)), "arl2_paged_forward")
        return out

    def device_status(self, stream=None) -> int:
        """Synchronise and return the device status code: 0, ARL2_ERR_TIMEOUT,
        or -1 if a batch's tables were wrong."""
        return _lib.arl2_paged_device_status(self.handle, _stream(stream))

    def device_bytes(self) -> int:
        return int(_lib.arl2_paged_device_bytes(self.handle))

    def kernel_launches(self) -> int:
        return int(_lib.arl2_paged_kernel_launches(self.handle))

    def close(self) -> None:
        if getattr(self, "_h", None) is not None:
            _lib.arl2_paged_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.close()
