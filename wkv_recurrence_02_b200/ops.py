"""Thin ctypes binding of libwkv.so (include/rwkv_wkv.h) for torch CUDA tensors.

Argument marshalling only: every step of the recurrences runs in the library's CUDA
kernels.  There is no CPU fallback -- if the library is not built, or a tensor is
not on a CUDA device, the call raises.

Functions mirror the C entry points:
  wkv4_forward(w, u, k, v, s0=None, want_state=False)   -> y            | (y, sT)
  wkv6_forward(r, k, v, w, u, s0=None, want_state=True) -> (y, sT)      | y
  delta_forward(q, k, v, g, beta, s0=None, ...)         -> (o, sT)      | o
  delta_backward(q, k, v, g, beta, do, ...)             -> dict of gradients
  state_copy(pool, src, dst), state_compact(pool, live) -> None, (new_index, count)
The calls are asynchronous on torch's current CUDA stream.
"""
import contextlib
import ctypes
import functools
import os
import re

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libwkv.so")
HEADER = os.path.join(os.path.dirname(_HERE), "include", "rwkv_wkv.h")

RWKV_OK = 0
STATUS_NAMES = {0: "RWKV_OK", -1: "RWKV_ERR_NULL", -2: "RWKV_ERR_SHAPE", -3: "RWKV_ERR_UNSUPPORTED",
                -4: "RWKV_ERR_ALIAS", -5: "RWKV_ERR_CUDA", -6: "RWKV_ERR_TIMEOUT",
                -7: "RWKV_ERR_ALIGN", -8: "RWKV_ERR_ARG", -9: "RWKV_ERR_BOUNDS"}
ALGOS = {"auto": 0, "serial": 1, "chunked": 2}

_i64 = ctypes.c_int64
_vp = ctypes.c_void_p
_lib = None


class WkvError(RuntimeError):
    def __init__(self, code, msg):
        super().__init__(f"{STATUS_NAMES.get(code, code)}: {msg}")
        self.code = code


def declared_functions(header: str = HEADER):
    """Names of the functions include/rwkv_wkv.h declares."""
    with open(header) as f:
        text = f.read()
    return sorted(set(re.findall(r"\b(rwkv_[a-z0-9_]+)\s*\(", text)))


def load(path: str = LIB_PATH):
    """Load libwkv.so (once) and declare its signatures.  Raises if it is missing."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is not built: run `python -m wkv_recurrence_02_b200.build`")
    lib = ctypes.CDLL(path)
    wkv4 = [_i64, _i64, _i64, _vp, _vp, _vp, _vp, _vp]
    wkv4s = [_i64, _i64, _i64, _vp, _vp, _vp, _vp, _vp, _vp, _vp]
    wkv6 = [_i64, _i64, _i64, _i64, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp]
    for name, args in [("rwkv_wkv4_forward", wkv4), ("rwkv_wkv4_forward_bf16", wkv4),
                       ("rwkv_wkv4_forward_state", wkv4s), ("rwkv_wkv4_forward_state_bf16", wkv4s),
                       ("rwkv_wkv6_forward", wkv6), ("rwkv_wkv6_forward_bf16", wkv6)]:
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = ctypes.c_int
    lib.rwkv_set_stream.argtypes = [_vp]
    lib.rwkv_set_stream.restype = None
    lib.rwkv_get_stream.argtypes = []
    lib.rwkv_get_stream.restype = _vp
    lib.rwkv_set_wkv6_algo.argtypes = [ctypes.c_int]
    lib.rwkv_set_wkv6_algo.restype = ctypes.c_int
    lib.rwkv_get_wkv6_algo.argtypes = []
    lib.rwkv_get_wkv6_algo.restype = ctypes.c_int
    lib.rwkv_wkv6_forward_bf16_noalloc.argtypes = wkv6 + [ctypes.c_int]
    lib.rwkv_wkv6_forward_gated_bf16.argtypes = wkv6[:10] + [_vp, _vp, _vp, ctypes.c_float] + wkv6[10:]
    lib.rwkv_wkv6_forward_gated_bf16.restype = ctypes.c_int
    lib.rwkv_wkv6_forward_omega_bf16.argtypes = wkv6[:10] + [_vp, _vp, _vp, ctypes.c_float] + wkv6[10:]
    lib.rwkv_wkv6_forward_omega_bf16.restype = ctypes.c_int
    bwd = [_i64] * 4 + [_vp] * 14 + [_vp, ctypes.c_size_t]
    for name in ("rwkv_wkv6_backward", "rwkv_wkv6_backward_bf16", "rwkv_wkv6_backward_omega_bf16"):
        fn = getattr(lib, name)
        fn.argtypes = bwd
        fn.restype = ctypes.c_int
    lib.rwkv_wkv6_backward_workspace_bytes.argtypes = [_i64] * 4 + [ctypes.POINTER(ctypes.c_size_t)]
    lib.rwkv_wkv6_backward_workspace_bytes.restype = ctypes.c_int
    lib.rwkv_wkv6_forward_bf16_noalloc.restype = ctypes.c_int
    delta = [_i64] * 5 + [_vp] * 5 + [ctypes.c_float, _i64, _vp]
    for name in ("rwkv_delta_forward", "rwkv_delta_forward_bf16"):
        fn = getattr(lib, name)
        fn.argtypes = delta + [_i64, _vp, _vp, _vp, _vp, _vp, ctypes.c_size_t]
        fn.restype = ctypes.c_int
    for name in ("rwkv_delta_backward", "rwkv_delta_backward_bf16"):
        fn = getattr(lib, name)
        fn.argtypes = delta + [_vp] * 10 + [ctypes.c_size_t]
        fn.restype = ctypes.c_int
    for name in ("rwkv_delta_forward_workspace_bytes", "rwkv_delta_backward_workspace_bytes"):
        fn = getattr(lib, name)
        fn.argtypes = [_i64] * 6 + [ctypes.c_int, ctypes.c_int, ctypes.POINTER(ctypes.c_size_t)]
        fn.restype = ctypes.c_int
    lib.rwkv_state_copy.argtypes = [_i64, _i64, _i64, _vp, _i64, _vp, _vp]
    lib.rwkv_state_copy.restype = ctypes.c_int
    lib.rwkv_state_compact.argtypes = [_i64, _i64, _i64, _vp, _vp, _vp, _vp]
    lib.rwkv_state_compact.restype = ctypes.c_int
    lib.rwkv_set_wkv6_segments.argtypes = [ctypes.c_int]
    lib.rwkv_set_wkv6_segments.restype = ctypes.c_int
    lib.rwkv_get_wkv6_segments.argtypes = []
    lib.rwkv_get_wkv6_segments.restype = ctypes.c_int
    lib.rwkv_debug_inject_timeout.argtypes = [ctypes.c_int]
    lib.rwkv_debug_inject_timeout.restype = ctypes.c_int
    lib.rwkv_get_device_status.argtypes = []
    lib.rwkv_get_device_status.restype = ctypes.c_int
    lib.rwkv_status_string.argtypes = [ctypes.c_int]
    lib.rwkv_status_string.restype = ctypes.c_char_p
    lib.rwkv_last_error.argtypes = []
    lib.rwkv_last_error.restype = ctypes.c_char_p
    lib.rwkv_abi_version.argtypes = []
    lib.rwkv_abi_version.restype = ctypes.c_int
    lib.rwkv_debug_bounds.argtypes = []
    lib.rwkv_debug_bounds.restype = ctypes.c_int
    _lib = lib
    return lib


@contextlib.contextmanager
def using_library(path: str):
    """Route the calls of this module to another build of the library (e.g. the bounds-checked
    debug build, libwkv_debug.so) inside the block; the default library is restored after."""
    global _lib
    prev = _lib
    _lib = None
    try:
        yield load(path)
    finally:
        _lib = prev


def _check(rc):
    if rc != RWKV_OK:
        lib = load()
        raise WkvError(rc, (lib.rwkv_last_error() or b"").decode() or
                       lib.rwkv_status_string(rc).decode())


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _cuda(t, name, dtype=None, shape=None):
    if t is None:
        return None
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    return t


def _use_current_stream(lib, device):
    lib.rwkv_set_stream(ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream))


def wkv4_forward(w, u, k, v, s0=None, want_state=False, y=None, sT=None):
    """RWKV-4 WKV.  k, v: [B,T,C] fp32|bf16; w, u: [C] fp32; s0: [B,3,C] fp32 or None."""
    lib = load()
    _cuda(k, "k")
    B, T, C = k.shape
    dt = k.dtype
    if dt not in (torch.float32, torch.bfloat16):
        raise TypeError("k must be float32 or bfloat16")
    _cuda(v, "v", dt, (B, T, C))
    _cuda(w, "w", torch.float32, (C,))
    _cuda(u, "u", torch.float32, (C,))
    _cuda(s0, "s0", torch.float32, (B, 3, C))
    if y is None:
        y = torch.empty_like(k)
    _cuda(y, "y", dt, (B, T, C))
    stateful = want_state or s0 is not None or sT is not None
    if stateful and sT is None and want_state:
        sT = torch.empty(B, 3, C, device=k.device, dtype=torch.float32)
    _cuda(sT, "sT", torch.float32, (B, 3, C))
    _use_current_stream(lib, k.device)
    bf = dt == torch.bfloat16
    if stateful:
        fn = lib.rwkv_wkv4_forward_state_bf16 if bf else lib.rwkv_wkv4_forward_state
        _check(fn(B, T, C, _ptr(w), _ptr(u), _ptr(k), _ptr(v), _ptr(s0), _ptr(y), _ptr(sT)))
    else:
        fn = lib.rwkv_wkv4_forward_bf16 if bf else lib.rwkv_wkv4_forward
        _check(fn(B, T, C, _ptr(w), _ptr(u), _ptr(k), _ptr(v), _ptr(y)))
    return (y, sT) if want_state else y


def wkv6_forward(r, k, v, w, u, s0=None, want_state=True, y=None, sT=None, algo=None,
                 segments=None):
    """Eagle/Finch WKV-6.  r,k,v,w: [B,T,H,N] fp32|bf16; u: [H,N] fp32; s0: [B,H,N,N] fp32.

    algo: None (library default), "auto", "serial" or "chunked" (this call only).
    segments: None (library default), 0 (auto), 1 (no sequence split) or n (at most n).
    """
    lib = load()
    _cuda(r, "r")
    B, T, H, N = r.shape
    dt = r.dtype
    if dt not in (torch.float32, torch.bfloat16):
        raise TypeError("r must be float32 or bfloat16")
    for name, t in (("k", k), ("v", v), ("w", w)):
        _cuda(t, name, dt, (B, T, H, N))
    _cuda(u, "u", torch.float32, (H, N))
    _cuda(s0, "s0", torch.float32, (B, H, N, N))
    if y is None:
        y = torch.empty_like(r)
    _cuda(y, "y", dt, (B, T, H, N))
    if sT is None and want_state:
        sT = torch.empty(B, H, N, N, device=r.device, dtype=torch.float32)
    _cuda(sT, "sT", torch.float32, (B, H, N, N))
    _use_current_stream(lib, r.device)
    fn = lib.rwkv_wkv6_forward_bf16 if dt == torch.bfloat16 else lib.rwkv_wkv6_forward
    prev = prev_seg = None
    if algo is not None:
        prev = lib.rwkv_get_wkv6_algo()
        _check(lib.rwkv_set_wkv6_algo(ALGOS[algo]))
    if segments is not None:
        prev_seg = lib.rwkv_get_wkv6_segments()
        _check(lib.rwkv_set_wkv6_segments(int(segments)))
    try:
        _check(fn(B, T, H, N, _ptr(r), _ptr(k), _ptr(v), _ptr(w), _ptr(u), _ptr(s0), _ptr(y),
                  _ptr(sT)))
    finally:
        if prev is not None:
            lib.rwkv_set_wkv6_algo(prev)
        if prev_seg is not None:
            lib.rwkv_set_wkv6_segments(prev_seg)
    return (y, sT) if want_state else y


def wkv6_forward_gated(r, k, v, w, u, g, ln_w, ln_b, eps=1e-5, s0=None, want_state=True, y=None,
                       sT=None):
    """WKV-6 (bf16) with the fused output stage: y = SiLU(g) * LayerNorm_head(o; ln_w, ln_b, eps).

    r,k,v,w,g: [B,T,H,N] bf16; u, ln_w, ln_b: [H,N] fp32; s0: [B,H,N,N] fp32.
    """
    lib = load()
    _cuda(r, "r", torch.bfloat16)
    B, T, H, N = r.shape
    for name, t in (("k", k), ("v", v), ("w", w), ("g", g)):
        _cuda(t, name, torch.bfloat16, (B, T, H, N))
    for name, t in (("u", u), ("ln_w", ln_w), ("ln_b", ln_b)):
        _cuda(t, name, torch.float32, (H, N))
    _cuda(s0, "s0", torch.float32, (B, H, N, N))
    if y is None:
        y = torch.empty_like(r)
    _cuda(y, "y", torch.bfloat16, (B, T, H, N))
    if sT is None and want_state:
        sT = torch.empty(B, H, N, N, device=r.device, dtype=torch.float32)
    _cuda(sT, "sT", torch.float32, (B, H, N, N))
    _use_current_stream(lib, r.device)
    _check(lib.rwkv_wkv6_forward_gated_bf16(B, T, H, N, _ptr(r), _ptr(k), _ptr(v), _ptr(w), _ptr(u),
                                             _ptr(s0), _ptr(g), _ptr(ln_w), _ptr(ln_b), float(eps),
                                             _ptr(y), _ptr(sT)))
    return (y, sT) if want_state else y


def wkv6_forward_omega(r, k, v, omega, u, s0=None, g=None, ln_w=None, ln_b=None, eps=1e-5,
                       want_state=True, y=None, sT=None, algo=None):
    """WKV-6 (bf16) fed the decay logit omega_t; the kernels form w_t = exp(-exp(omega_t)).

    r,k,v,omega (and g): [B,T,H,N] bf16; u (and ln_w, ln_b): [H,N] fp32; s0: [B,H,N,N] fp32.
    With g, ln_w and ln_b the fused head LayerNorm + SiLU gate is applied as in
    wkv6_forward_gated.  algo (plain output only): as in wkv6_forward.
    """
    lib = load()
    _cuda(r, "r", torch.bfloat16)
    B, T, H, N = r.shape
    for name, t in (("k", k), ("v", v), ("omega", omega), ("g", g)):
        _cuda(t, name, torch.bfloat16, (B, T, H, N))
    for name, t in (("u", u), ("ln_w", ln_w), ("ln_b", ln_b)):
        _cuda(t, name, torch.float32, (H, N))
    _cuda(s0, "s0", torch.float32, (B, H, N, N))
    if y is None:
        y = torch.empty_like(r)
    _cuda(y, "y", torch.bfloat16, (B, T, H, N))
    if sT is None and want_state:
        sT = torch.empty(B, H, N, N, device=r.device, dtype=torch.float32)
    _cuda(sT, "sT", torch.float32, (B, H, N, N))
    _use_current_stream(lib, r.device)
    prev = None
    if algo is not None:
        prev = lib.rwkv_get_wkv6_algo()
        _check(lib.rwkv_set_wkv6_algo(ALGOS[algo]))
    try:
        _check(lib.rwkv_wkv6_forward_omega_bf16(B, T, H, N, _ptr(r), _ptr(k), _ptr(v), _ptr(omega),
                                                 _ptr(u), _ptr(s0), _ptr(g), _ptr(ln_w), _ptr(ln_b),
                                                 float(eps), _ptr(y), _ptr(sT)))
    finally:
        if prev is not None:
            lib.rwkv_set_wkv6_algo(prev)
    return (y, sT) if want_state else y


def wkv6_backward_workspace_bytes(B, T, H, N=64) -> int:
    """Device scratch (bytes) that a WKV-6 backward call of this shape needs."""
    lib = load()
    out = ctypes.c_size_t(0)
    _check(lib.rwkv_wkv6_backward_workspace_bytes(int(B), int(T), int(H), int(N), ctypes.byref(out)))
    return int(out.value)


def wkv6_backward(r, k, v, w, u, dy, s0=None, dsT=None, omega=False, want_ds0=True, workspace=None,
                  algo=None):
    """WKV-6 backward: gradients of a loss with dL/dy = dy and dL/dsT = dsT (None = 0).

    r,k,v,w,dy: [B,T,H,N] fp32|bf16 (with omega=True, w holds omega_t and bf16 is required);
    u: [H,N] fp32; s0, dsT: [B,H,N,N] fp32.  Returns a dict of fp32 tensors dr, dk, dv,
    dw (or domega), du, and ds0 (when want_ds0).  workspace: optional uint8 CUDA tensor of at
    least wkv6_backward_workspace_bytes bytes; allocated here when not given.
    algo: None (library default: bf16 inputs take the chunked tensor-core path), "auto",
    "serial" (the exact fp32 walks) or "chunked" (this call only).
    """
    lib = load()
    _cuda(r, "r")
    B, T, H, N = r.shape
    dt = r.dtype
    if dt not in (torch.float32, torch.bfloat16):
        raise TypeError("r must be float32 or bfloat16")
    if omega and dt != torch.bfloat16:
        raise TypeError("the logit backward takes bf16 inputs")
    for name, t in (("k", k), ("v", v), ("w", w), ("dy", dy)):
        _cuda(t, name, dt, (B, T, H, N))
    _cuda(u, "u", torch.float32, (H, N))
    _cuda(s0, "s0", torch.float32, (B, H, N, N))
    _cuda(dsT, "dsT", torch.float32, (B, H, N, N))
    dev = r.device
    out = {n: torch.empty(B, T, H, N, device=dev, dtype=torch.float32) for n in ("dr", "dk", "dv")}
    dwn = "domega" if omega else "dw"
    out[dwn] = torch.empty(B, T, H, N, device=dev, dtype=torch.float32)
    out["du"] = torch.empty(H, N, device=dev, dtype=torch.float32)
    out["ds0"] = torch.empty(B, H, N, N, device=dev, dtype=torch.float32) if want_ds0 else None
    need = wkv6_backward_workspace_bytes(B, T, H, N)
    if workspace is None:
        workspace = torch.empty(max(need, 16), device=dev, dtype=torch.uint8)
    _cuda(workspace, "workspace", torch.uint8)
    _use_current_stream(lib, dev)
    fn = (lib.rwkv_wkv6_backward_omega_bf16 if omega else
          lib.rwkv_wkv6_backward_bf16 if dt == torch.bfloat16 else lib.rwkv_wkv6_backward)
    prev = None
    if algo is not None:
        prev = lib.rwkv_get_wkv6_algo()
        _check(lib.rwkv_set_wkv6_algo(ALGOS[algo]))
    try:
        _check(fn(B, T, H, N, _ptr(r), _ptr(k), _ptr(v), _ptr(w), _ptr(u), _ptr(s0), _ptr(dy), _ptr(dsT),
                  _ptr(out["dr"]), _ptr(out["dk"]), _ptr(out["dv"]), _ptr(out[dwn]), _ptr(out["du"]),
                  _ptr(out["ds0"]), _ptr(workspace), ctypes.c_size_t(workspace.numel())))
    finally:
        if prev is not None:
            lib.rwkv_set_wkv6_algo(prev)
    if not want_ds0:
        del out["ds0"]
    return out


def _call(lib, device, fn, *args):
    """fn(*args) on the tensors' device and its current torch stream; raises on an error status."""
    index = device.index
    if index != torch._C._cuda_getDevice():
        with torch.cuda.device(device):
            return _call(lib, device, fn, *args)
    lib.rwkv_set_stream(torch._C._cuda_getCurrentRawStream(index))
    _check(fn(*args))


def _at(t):
    return None if t is None else t.data_ptr()


def _tensor(t, name, dtype, shape, device):
    """Like _cuda, for the operators whose calls take microseconds: one pass over what is usual."""
    if t is None:
        return
    if (t.__class__ is not torch.Tensor and not isinstance(t, torch.Tensor)) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, not on {device}")


def _delta_shapes(q, k, v, g, beta, offsets):
    """(B, T, Hk, H, N, sequences, dtype) of a delta-rule call, its inputs checked."""
    _cuda(q, "q")
    _cuda(v, "v")
    if q.dim() != 4 or v.dim() != 4:
        raise ValueError("q and v must have shape [B, T, heads, N]")
    B, T, Hk, N = q.shape
    H, dt, dev = v.shape[2], q.dtype, q.device
    if dt not in (torch.float32, torch.bfloat16):
        raise TypeError("q must be float32 or bfloat16")
    _tensor(k, "k", dt, q.shape, dev)
    _tensor(v, "v", dt, (B, T, H, N), dev)
    _tensor(g, "g", dt, (B, T, H), dev)
    _tensor(beta, "beta", dt, (B, T, H), dev)
    nseq = B
    if offsets is not None:
        _tensor(offsets, "offsets", torch.int32, None, dev)
        if offsets.dim() != 1 or offsets.numel() < 1:
            raise ValueError("offsets must have shape [sequences + 1]")
        nseq = offsets.numel() - 1
    return B, T, Hk, H, N, nseq, dt


@functools.lru_cache(maxsize=1024)
def _delta_workspace(name, B, T, Hk, H, N, nseq, packed, bf16):
    out = ctypes.c_size_t(0)
    _check(getattr(load(), name)(B, T, Hk, H, N, nseq, packed, bf16, ctypes.byref(out)))
    return out.value


def delta_forward_workspace_bytes(B, T, Hk, H, N=64, nseq=None, packed=False, bf16=True) -> int:
    """Device scratch (bytes) that a delta-rule forward call of this shape needs."""
    return _delta_workspace("rwkv_delta_forward_workspace_bytes", B, T, Hk, H, N, B if nseq is None else nseq, packed,
                            bf16)


def delta_forward(q, k, v, g, beta, scale=None, s0=None, offsets=None, slots=None, want_state=True, o=None, sT=None,
                  workspace=None):
    """Gated delta rule: S' = exp(g) S, u = beta (v - k S'), S = S' + k^T u, o = scale q S.

    q, k: [B,T,Hk,N] fp32|bf16; v: [B,T,H,N]; g, beta: [B,T,H] (Hk divides H).  scale: default
    1/sqrt(N).  offsets: int32 [sequences+1], the runs of tokens of a packed call (B = 1).
    s0: [sequences,H,N,N] fp32 or None (zero); with slots (int32 [sequences]), a pool
    [P,H,N,N] whose slot slots[i] is sequence i's state, updated in place unless another pool
    is given as sT; a negative slot is a sequence without a state.  Slots without a pool (s0 and
    sT None, want_state False) are not looked at: every sequence starts from zero.  Returns (o, sT),
    or o; an o allocated here is not set for tokens outside every sequence.

    bf16 sequences of 24 tokens or more on average run in chunks on the tensor cores (o is formed from
    bf16 operands); shorter ones, and inputs cast to fp32, token by token in fp32.  A long sequence
    packed with many short ones is faster in a call of its own, over slices of the same tensors.
    """
    lib = load()
    B, T, Hk, H, N, nseq, dt = _delta_shapes(q, k, v, g, beta, offsets)
    dev = q.device
    if slots is not None:
        _tensor(slots, "slots", torch.int32, (nseq,), dev)
        if sT is None and want_state:
            if s0 is None:
                raise ValueError("slots need a pool: s0, sT or both")
            sT = s0
    pool = s0 if s0 is not None else sT
    if pool is None:  # no state to find or to keep: the slots name nothing
        slots = None
    nslots = nseq if slots is None else pool.shape[0]
    state = (nslots, H, N, N)
    _tensor(s0, "s0", torch.float32, state, dev)
    if o is None:
        o = torch.empty_like(v)
    else:
        _tensor(o, "o", dt, v.shape, dev)
    if sT is None and want_state:
        sT = torch.empty(state, device=dev, dtype=torch.float32)
    elif sT is not s0:
        _tensor(sT, "sT", torch.float32, state, dev)
    bf = dt == torch.bfloat16
    if workspace is None:
        need = _delta_workspace("rwkv_delta_forward_workspace_bytes", B, T, Hk, H, N, nseq, offsets is not None, bf)
        if need:
            workspace = torch.empty(need, device=dev, dtype=torch.uint8)
    _tensor(workspace, "workspace", torch.uint8, None, dev)
    _call(lib, dev, lib.rwkv_delta_forward_bf16 if bf else lib.rwkv_delta_forward, B, T, Hk, H, N, q.data_ptr(),
          k.data_ptr(), v.data_ptr(), g.data_ptr(), beta.data_ptr(), N ** -0.5 if scale is None else float(scale), nseq,
          _at(offsets), nslots, _at(slots), _at(s0), o.data_ptr(), _at(sT), _at(workspace),
          0 if workspace is None else workspace.numel())
    return (o, sT) if want_state else o


def delta_backward_workspace_bytes(B, T, Hk, H, N=64, nseq=None, packed=False, bf16=True) -> int:
    """Device scratch (bytes) that a delta-rule backward call of this shape needs."""
    return _delta_workspace("rwkv_delta_backward_workspace_bytes", B, T, Hk, H, N, B if nseq is None else nseq,
                            packed, bf16)


def delta_backward(q, k, v, g, beta, do, scale=None, s0=None, dsT=None, offsets=None, want_ds0=True, workspace=None):
    """Gradients of delta_forward for a loss with dL/do = do and dL/dsT = dsT (None = 0).

    Inputs as in delta_forward (no slots); do: [B,T,H,N]; dsT: [sequences,H,N,N] fp32.  Returns
    a dict of dq, dk, dv, dg, dbeta (type of the inputs) and ds0 (fp32, when want_ds0).
    Gradients of tokens outside every sequence are zero.  workspace: optional uint8 CUDA tensor
    of at least delta_backward_workspace_bytes bytes; allocated here when not given.
    """
    lib = load()
    B, T, Hk, H, N, nseq, dt = _delta_shapes(q, k, v, g, beta, offsets)
    dev, state = q.device, (nseq, H, N, N)
    _tensor(do, "do", dt, v.shape, dev)
    _tensor(s0, "s0", torch.float32, state, dev)
    _tensor(dsT, "dsT", torch.float32, state, dev)
    make = torch.empty_like if offsets is None else torch.zeros_like
    out = {"dq": make(q), "dk": make(k), "dv": make(v), "dg": make(g), "dbeta": make(beta)}
    if want_ds0:
        out["ds0"] = torch.empty(state, device=dev, dtype=torch.float32)
    bf = dt == torch.bfloat16
    if workspace is None:
        need = _delta_workspace("rwkv_delta_backward_workspace_bytes", B, T, Hk, H, N, nseq, offsets is not None, bf)
        workspace = torch.empty(max(need, 16), device=dev, dtype=torch.uint8)
    _tensor(workspace, "workspace", torch.uint8, None, dev)
    _call(lib, dev, lib.rwkv_delta_backward_bf16 if bf else lib.rwkv_delta_backward, B, T, Hk, H, N, q.data_ptr(),
          k.data_ptr(), v.data_ptr(), g.data_ptr(), beta.data_ptr(), N ** -0.5 if scale is None else float(scale), nseq,
          _at(offsets), _at(s0), do.data_ptr(), _at(dsT), *(out[n].data_ptr() for n in ("dq", "dk", "dv", "dg", "dbeta")),
          _at(out.get("ds0")), workspace.data_ptr(), workspace.numel())
    return out


def _pool_shape(pool, slot_dim):
    """(layers, slots, bytes of a slot) of a pool whose dimension slot_dim counts the slots."""
    _cuda(pool, "pool")
    if not 0 <= slot_dim < pool.dim():
        raise ValueError("slot_dim must be a dimension of the pool")
    layers = slot = 1
    for n in pool.shape[:slot_dim]:
        layers *= n
    for n in pool.shape[slot_dim + 1:]:
        slot *= n
    return layers, pool.shape[slot_dim], slot * pool.element_size()


def state_copy(pool, src, dst, slot_dim=0):
    """Copy, fork and free slots of a pool of states, in place: for every pair, slot dst[i] <-
    slot src[i] as it was before the call (src[i] < 0: zeros; dst[i] < 0: the pair is left out;
    of several pairs with one dst the last counts).

    pool: any CUDA tensor whose dimension slot_dim counts the slots and whose earlier ones count
    layers, e.g. [P,H,N,N], or [L,P,H,N,N] with slot_dim=1.  src, dst: int32 [n], n <= 4096.
    """
    lib = load()
    layers, nslots, slot_bytes = _pool_shape(pool, slot_dim)
    _tensor(src, "src", torch.int32, None, pool.device)
    _tensor(dst, "dst", torch.int32, src.shape, pool.device)
    _call(lib, pool.device, lib.rwkv_state_copy, layers, nslots, slot_bytes, pool.data_ptr(), src.numel(), src.data_ptr(),
          dst.data_ptr())


def state_compact(pool, live, slot_dim=0):
    """Move the live slots of a pool of states to its front, in order and in place.

    pool, slot_dim: as in state_copy, at most 16384 slots; live: bool or uint8 [P].  Returns
    (new_index, count): int32 [P], the place each slot went to (-1 if it is not live), and
    int32 [1], both on the device.  Slots from count on keep what they hold.
    """
    lib = load()
    layers, nslots, slot_bytes = _pool_shape(pool, slot_dim)
    if isinstance(live, torch.Tensor) and live.dtype not in (torch.bool, torch.uint8):
        raise TypeError("live must be bool or uint8")
    _tensor(live, "live", getattr(live, "dtype", None), (nslots,), pool.device)
    new_index = torch.empty(nslots, device=pool.device, dtype=torch.int32)
    count = torch.empty(1, device=pool.device, dtype=torch.int32)
    _call(lib, pool.device, lib.rwkv_state_compact, layers, nslots, slot_bytes, pool.data_ptr(), live.data_ptr(),
          new_index.data_ptr(), count.data_ptr())
    return new_index, count


def device_status() -> int:
    """Synchronise the current stream and return/clear the device status word."""
    lib = load()
    _use_current_stream(lib, torch.cuda.current_device())
    return int(lib.rwkv_get_device_status())
