"""Thin ctypes binding of libsot (include/sot.h), same names as the C ABI.

Only argument marshalling lives here: every step of the computation runs in
the CUDA kernels of libsot.  Tensors must be float32, contiguous and on the
current CUDA device (the language-model losses take logits in three types and
with a row stride); the calls are stream-ordered on
``torch.cuda.current_stream()`` unless a stream is given.  Outputs are
allocated with torch when not supplied (plain device memory, no compute).
A missing or unloadable libsot raises at once: there is no CPU fallback.
"""
from __future__ import annotations

import ctypes as C
import os
import re

import torch

from . import build as _build

SOT_OK = 0
SOT_ERR_INVALID_ARG = -1
SOT_ERR_NONFINITE = -2
SOT_ERR_CAPACITY = -3
SOT_ERR_TIMEOUT = -4
SOT_ERR_CUDA = -5
SOT_ERR_UNSUPPORTED = -6
SOT_ERR_NOMEM = -7

SOT_PREC_AUTO = 0
SOT_PREC_FP32 = 1
SOT_PREC_F16X3 = 2
SOT_WARM_START = 1 << 4
SOT_STAGE_EARLY_EXIT = 1 << 5
SOT_TC_NO_SCREEN = 1 << 6
SOT_NO_CLUSTER = 1 << 7
SOT_COST_COSINE = 1 << 8

SOT_F32, SOT_F16, SOT_BF16, SOT_I32, SOT_I64 = range(5)  # sot_dtype
_FLOATS = {torch.float32: SOT_F32, torch.float16: SOT_F16, torch.bfloat16: SOT_BF16}
_INDICES = {torch.int32: SOT_I32, torch.int64: SOT_I64}

HEADER = os.path.join(_build.ROOT, "include", "sot.h")


class SotError(RuntimeError):
    def __init__(self, status: int, func: str, detail: str):
        super().__init__(f"{func}: {detail} (status {status})")
        self.status = status


class sot_schedule(C.Structure):
    _fields_ = [("eps", C.c_float), ("eps_init", C.c_float), ("eps_factor", C.c_float),
                ("iters_per_stage", C.c_int), ("max_iters", C.c_int), ("tol", C.c_float), ("flags", C.c_int)]


class sot_stats(C.Structure):
    _fields_ = [("iters_done", C.c_int), ("stages_done", C.c_int), ("converged", C.c_int), ("final_eps", C.c_float),
                ("err_host", C.POINTER(C.c_float)), ("stage_iters_host", C.POINTER(C.c_int)),
                ("stage_iters_cap", C.c_int)]


_lib = None
_fp = C.c_void_p


def declared_functions() -> list[str]:
    """Names of the functions declared in include/sot.h."""
    txt = open(HEADER).read()
    txt = re.sub(r"/\*.*?\*/", "", txt, flags=re.S)
    return sorted(set(re.findall(r"\b(sot_[a-z_0-9]+)\s*\(", txt)))


def load(path: str | None = None):
    """Load libsot.so (built in-tree by ``build.build()``); raises if absent."""
    global _lib
    if _lib is not None and path is None:
        return _lib
    p = path or _build.LIB
    if not os.path.exists(p):
        raise RuntimeError(f"libsot.so not found at {p}: run sinkhorn_point_cloud_gb300.build.build()")
    L = C.CDLL(p)
    P = _fp
    i, f, ll = C.c_int, C.c_float, C.c_longlong
    sig = {
        "sot_potentials": [P, P, P, P, i, i, i, i, f, i, P, P, P],
        "sot_potentials_ex": [P, P, P, P, i, i, i, i, C.POINTER(sot_schedule), P, P, C.POINTER(sot_stats), P],
        "sot_plan_apply": [P, P, P, P, i, i, i, i, P, P, f, P, P, P, i, P],
        "sot_cost": [P, P, P, P, i, i, i, i, P, P, f, P, P],
        "sot_grad_x": [P, P, P, P, i, i, i, i, P, P, f, P, P],
        "sot_cost_grad": [P, P, P, P, i, i, i, i, P, P, f, P, P, P],
        "sot_plan_coo": [P, P, P, P, i, i, i, i, P, P, f, f, i, ll, P, P, P, P, C.POINTER(ll), P],
        "sot_grad_x_coo": [P, P, i, i, i, i, P, P, P, P, P, P],
        "sot_check_inputs": [P, P, P, P, i, i, i, i, P],
        "sot_profile_enable": [i],
        "sot_profile_read": [C.POINTER(ll), C.POINTER(C.c_double)],
        "sot_profile_read_kinds": [C.POINTER(ll), C.POINTER(C.c_double)],
        "sot_status_string": [i],
        "sot_last_error": [],
        "sot_version": [],
        "sot_kernel_launches": [],
        "sot_select_path": [i, i],
        "sot_potentials_noalloc": [P, P, P, P, i, i, i, i, f, i, P, P, P],
        "sot_transport_apply": [P, P, P, P, i, i, i, i, P, P, f, P, i, i, P, i, P],
        "sot_grad_y": [P, P, P, P, i, i, i, i, P, P, f, P, i, P],
        "sot_apml_coo": [P, P, P, P, i, i, i, i, P, P, P, ll, f, i, P, P, P, P],
        "sot_async_status": [P],
        "sot_hvp": [P, P, P, P, i, i, i, i, P, P, f, P, i, f, P, i, P],
        "sot_test_hold_tile": [i, i, ll],
        "sot_test_hold_routed": [i, ll],
        "sot_plan_coo_operands": [P, P, P, P, i, i, i, i, P, P, f, f, P, P, P, P, P, P, P, P,
                                  C.POINTER(C.c_float), P],
        "sot_token_logprob": [P, ll, i, ll, i, f, P, i, P, P, P],
        "sot_token_logprob_grad": [P, ll, i, ll, i, f, P, i, P, P, P, ll, P],
        "sot_distill_topk": [P, ll, i, ll, i, f, P, i, P, i, i, i, P, P, P, ll, P],
        "sot_policy_loss": [P, ll, i, ll, i, f, P, i, P, P, P, P, f, f, f, P, P, P, P, ll, P],
        "sot_preference_loss": [P, P, P, i, P, i, ll, f, f, i, f, P, P, P, P],
        "sot_balance_loss": [P, ll, i, ll, i, P, i, i, P, f, f, P, P, P, ll, P],
        "sot_token_topk": [P, ll, i, ll, i, f, P, i, i, P, P, P, P, P, P],
        "sot_token_topk_grad": [P, ll, i, ll, i, f, P, i, P, P, P, P, P, i, P, P, ll, P],
        "sot_embed": [P, i, i, ll, i, P, i, ll, f, P, ll, i, P],
        "sot_embed_grad": [P, ll, i, ll, i, P, i, i, f, i, P, ll, i, P],
        "sot_routed_layer": [P, i, i, ll, i, P, P, i, P, P, i, i, i, f, P, ll, P, P, P, P],
    }
    for name, args in sig.items():
        fn = getattr(L, name)
        fn.argtypes = args
        fn.restype = C.c_char_p if name in ("sot_status_string", "sot_last_error") else \
            (C.c_longlong if name == "sot_kernel_launches" else C.c_int)
    if path is None:
        _lib = L
    return L


def _check(rc: int, func: str):
    if rc != SOT_OK:
        L = load()
        raise SotError(rc, func, L.sot_last_error().decode() or L.sot_status_string(rc).decode())


def _ptr(t):
    if t is None:
        return None
    if not isinstance(t, torch.Tensor):
        raise TypeError("expected a torch.Tensor")
    if t.dtype != torch.float32 and t.dtype not in (torch.int32, torch.int64):
        raise TypeError(f"expected float32, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError("tensor must be on a CUDA device")
    if not t.is_contiguous():
        raise ValueError("tensor must be contiguous")
    return C.c_void_p(t.data_ptr())


def _stream(stream):
    s = torch.cuda.current_stream() if stream is None else stream
    return C.c_void_p(s.cuda_stream)


def _want(t, name, count, dev, dtype=torch.float32):
    """A tensor the caller supplies must be contiguous, of ``dtype``, on ``dev``
    and hold exactly ``count`` elements (None: any count), since the library
    reads or writes that many."""
    if t is None:
        return t
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if count is not None and t.numel() != count:
        raise ValueError(f"{name} must hold {count} elements, got shape {tuple(t.shape)}")
    if t.device != dev:
        raise ValueError(f"{name} must be on {dev}, got {t.device}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t


def _shapes(X, Y, a, b):
    if not isinstance(X, torch.Tensor) or not isinstance(Y, torch.Tensor):
        raise TypeError("X and Y must be torch.Tensors")
    if X.dim() == 2:
        X = X.unsqueeze(0)
    if Y.dim() == 2:
        Y = Y.unsqueeze(0)
    if X.dim() != 3 or Y.dim() != 3:
        raise ValueError("X must be [B,n,d] or [n,d], Y [B,m,d] or [m,d]")
    B, n, d = X.shape
    B2, m, d2 = Y.shape
    if B != B2 or d != d2:
        raise ValueError("X [B,n,d] and Y [B,m,d] disagree")
    if a is not None and tuple(a.shape) not in ((B, n), (n,) if B == 1 else (B, n)):
        raise ValueError("a must be [B, n]")
    if b is not None and tuple(b.shape) not in ((B, m), (m,) if B == 1 else (B, m)):
        raise ValueError("b must be [B, m]")
    dev = X.device
    _want(X, "X", B * n * d, dev)
    _want(Y, "Y", B * m * d, dev)
    _want(a, "a", B * n, dev)
    _want(b, "b", B * m, dev)
    return X, Y, B, n, m, d


def _potentials_args(f, g, B, n, m, dev):
    return _want(f, "f", B * n, dev), _want(g, "g", B * m, dev)


def sot_version() -> int:
    return int(load().sot_version())


def sot_kernel_launches() -> int:
    return int(load().sot_kernel_launches())


def sot_select_path(d: int, flags: int = 0) -> int:
    """0 = fp32 point kernels, 1 = fp32 dense kernels, 2 = tensor-core kernels (negative: none)."""
    return int(load().sot_select_path(int(d), int(flags)))


def sot_status_string(status: int) -> str:
    return load().sot_status_string(int(status)).decode()


def sot_potentials(X, Y, a=None, b=None, eps=0.1, iters=100, f=None, g=None, stream=None):
    """Fixed schedule from f = g = 0; returns (f [B,n], g [B,m])."""
    X, Y, B, n, m, d = _shapes(X, Y, a, b)
    f = torch.empty(B, n, device=X.device, dtype=torch.float32) if f is None else f
    g = torch.empty(B, m, device=X.device, dtype=torch.float32) if g is None else g
    _potentials_args(f, g, B, n, m, X.device)
    rc = load().sot_potentials(_ptr(X), _ptr(Y), _ptr(a), _ptr(b), B, n, m, d, float(eps), int(iters), _ptr(f),
                               _ptr(g), _stream(stream))
    _check(rc, "sot_potentials")
    return f, g


def sot_potentials_noalloc(X, Y, a=None, b=None, eps=0.1, iters=100, f=None, g=None, stream=None):
    """sot_potentials for d <= 3 using the library's static scratch (no device
    allocation inside the call; see include/sot.h).  Pass preallocated f, g to
    keep this call path free of allocations on the Python side too."""
    X, Y, B, n, m, d = _shapes(X, Y, a, b)
    f = torch.empty(B, n, device=X.device, dtype=torch.float32) if f is None else f
    g = torch.empty(B, m, device=X.device, dtype=torch.float32) if g is None else g
    _potentials_args(f, g, B, n, m, X.device)
    rc = load().sot_potentials_noalloc(_ptr(X), _ptr(Y), _ptr(a), _ptr(b), B, n, m, d, float(eps), int(iters),
                                       _ptr(f), _ptr(g), _stream(stream))
    _check(rc, "sot_potentials_noalloc")
    return f, g


def sot_potentials_ex(X, Y, a=None, b=None, eps=0.1, eps_init=None, eps_factor=0.5, iters_per_stage=100,
                      max_iters=0, tol=0.0, flags=0, f=None, g=None, stats=False, stream=None):
    """General schedule (see sot_schedule in sot.h).  With ``flags & SOT_WARM_START``
    the given f, g are the initial potentials.  Returns (f, g) or (f, g, stats dict)."""
    X, Y, B, n, m, d = _shapes(X, Y, a, b)
    if flags & SOT_WARM_START and (f is None or g is None):
        raise ValueError("warm start needs f and g")
    f = torch.empty(B, n, device=X.device, dtype=torch.float32) if f is None else f
    g = torch.empty(B, m, device=X.device, dtype=torch.float32) if g is None else g
    _potentials_args(f, g, B, n, m, X.device)
    s = sot_schedule(float(eps), float(eps if eps_init is None else eps_init), float(eps_factor),
                     int(iters_per_stage), int(max_iters), float(tol), int(flags))
    st = None
    if stats:
        cap = 100000
        err = (C.c_float * max(B, 1))()
        si = (C.c_int * cap)()
        st = sot_stats(0, 0, 0, 0.0, C.cast(err, C.POINTER(C.c_float)), C.cast(si, C.POINTER(C.c_int)), cap)
    rc = load().sot_potentials_ex(_ptr(X), _ptr(Y), _ptr(a), _ptr(b), B, n, m, d, C.byref(s), _ptr(f), _ptr(g),
                                  C.byref(st) if st is not None else None, _stream(stream))
    _check(rc, "sot_potentials_ex")
    if not stats:
        return f, g
    info = dict(iters_done=st.iters_done, stages_done=st.stages_done, converged=bool(st.converged),
                final_eps=st.final_eps, err=[err[k] for k in range(B)],
                stage_iters=[si[k] for k in range(st.stages_done)])
    return f, g, info


def sot_plan_apply(X, Y, a, b, f, g, eps, cost=True, grad=True, rowsum=False, flags=0, stream=None):
    """Returns (cost [B] or None, grad [B,n,d] or None, rowsum [B,n] or None).
    Each of cost, grad, rowsum is True (allocate), False/None (skip) or a
    preallocated tensor to write into."""
    X, Y, B, n, m, d = _shapes(X, Y, a, b)
    dev = X.device
    pick = lambda want, shape: torch.empty(*shape, device=dev, dtype=torch.float32) if want is True else \
        (None if want is None or want is False else want)
    c, gr, r = pick(cost, (B,)), pick(grad, (B, n, d)), pick(rowsum, (B, n))
    _potentials_args(f, g, B, n, m, dev)
    _want(c, "cost", B, dev)
    _want(gr, "grad", B * n * d, dev)
    _want(r, "rowsum", B * n, dev)
    rc = load().sot_plan_apply(_ptr(X), _ptr(Y), _ptr(a), _ptr(b), B, n, m, d, _ptr(f), _ptr(g), float(eps),
                               _ptr(c), _ptr(gr), _ptr(r), int(flags), _stream(stream))
    _check(rc, "sot_plan_apply")
    return c, gr, r


def sot_transport_apply(X, Y, a, b, f, g, eps, V, side=0, flags=0, out=None, stream=None):
    """Transport-matrix product: side 0 -> P V with V [B,m,c] (out [B,n,c]);
    side 1 -> P^T V with V [B,n,c] (out [B,m,c]).  A [B,rows] V is one column."""
    X, Y, B, n, m, d = _shapes(X, Y, a, b)
    vec = V.dim() == 2
    V3 = V.unsqueeze(-1) if vec else V
    if V3.dtype != torch.float32 or not V3.is_contiguous() or V3.device != X.device:
        raise ValueError("V must be a contiguous float32 tensor on the device of X")
    rows_in, rows_out = (m, n) if side == 0 else (n, m)
    if V3.shape[0] != B or V3.shape[1] != rows_in:
        raise ValueError(f"V must have shape [B, {rows_in}, c] for side {side}")
    c = V3.shape[2]
    o = torch.empty(B, rows_out, c, device=X.device, dtype=torch.float32) if out is None else out
    _potentials_args(f, g, B, n, m, X.device)
    _want(o, "out", B * rows_out * c, X.device)
    rc = load().sot_transport_apply(_ptr(X), _ptr(Y), _ptr(a), _ptr(b), B, n, m, d, _ptr(f), _ptr(g),
                                    float(eps), _ptr(V3), int(c), int(side), _ptr(o), int(flags), _stream(stream))
    _check(rc, "sot_transport_apply")
    return o[..., 0] if vec else o


def sot_grad_y(X, Y, a, b, f, g, eps, flags=0, out=None, stream=None):
    """Gradient with respect to Y: 2 (b_j y_j - sum_i P_ij x_i), [B, m, d]."""
    X, Y, B, n, m, d = _shapes(X, Y, a, b)
    o = torch.empty(B, m, d, device=X.device, dtype=torch.float32) if out is None else out
    _potentials_args(f, g, B, n, m, X.device)
    _want(o, "out", B * m * d, X.device)
    rc = load().sot_grad_y(_ptr(X), _ptr(Y), _ptr(a), _ptr(b), B, n, m, d, _ptr(f), _ptr(g), float(eps), _ptr(o),
                           int(flags), _stream(stream))
    _check(rc, "sot_grad_y")
    return o


def sot_hvp(X, Y, a, b, f, g, eps, V, cg_iters=300, cg_tol=1e-5, out=None, stream=None):
    """Hessian-vector product of the entropic OT loss with respect to X at the
    potentials (f, g), applied to V [B, n, d]; returns H V [B, n, d]."""
    X, Y, B, n, m, d = _shapes(X, Y, a, b)
    _potentials_args(f, g, B, n, m, X.device)
    _want(V, "V", B * n * d, X.device)
    o = torch.empty(B, n, d, device=X.device, dtype=torch.float32) if out is None else out
    _want(o, "out", B * n * d, X.device)
    rc = load().sot_hvp(_ptr(X), _ptr(Y), _ptr(a), _ptr(b), B, n, m, d, _ptr(f), _ptr(g), float(eps), _ptr(V),
                        int(cg_iters), float(cg_tol), _ptr(o), 0, _stream(stream))
    _check(rc, "sot_hvp")
    return o


def sot_apml_coo(X, Y, a, b, coo, T, iters=10, loss=True, grad=True, stream=None):
    """Sparse APML on a stored support (``coo`` as sot_plan_coo returns it):
    returns (vals [nnz], loss [B] or None, grad [B,n,d] or None)."""
    X, Y, B, n, m, d = _shapes(X, Y, a, b)
    nnz = int(coo["nnz"])
    _want(coo["rows"], "coo rows", nnz, X.device, torch.int32)
    _want(coo["cols"], "coo cols", nnz, X.device, torch.int32)
    _want(coo["batch_offsets"], "coo batch_offsets", B + 1, X.device, torch.int64)
    vals = torch.empty(max(nnz, 1), device=X.device, dtype=torch.float32)
    lo = torch.empty(B, device=X.device, dtype=torch.float32) if loss else None
    gr = torch.empty(B, n, d, device=X.device, dtype=torch.float32) if grad else None
    rc = load().sot_apml_coo(_ptr(X), _ptr(Y), _ptr(a), _ptr(b), B, n, m, d, _ptr(coo["rows"]), _ptr(coo["cols"]),
                             _ptr(coo["batch_offsets"]), nnz, float(T), int(iters), _ptr(vals), _ptr(lo), _ptr(gr),
                             _stream(stream))
    _check(rc, "sot_apml_coo")
    return vals[:nnz], lo, gr


def sot_cost(X, Y, a, b, f, g, eps, stream=None):
    return sot_plan_apply(X, Y, a, b, f, g, eps, cost=True, grad=False, stream=stream)[0]


def sot_grad_x(X, Y, a, b, f, g, eps, stream=None):
    return sot_plan_apply(X, Y, a, b, f, g, eps, cost=False, grad=True, stream=stream)[1]


def sot_cost_grad(X, Y, a, b, f, g, eps, stream=None):
    c, gr, _ = sot_plan_apply(X, Y, a, b, f, g, eps, cost=True, grad=True, stream=stream)
    return c, gr


def sot_plan_coo(X, Y, a, b, f, g, eps, threshold=1e-8, dirs=3, capacity=None, stream=None):
    """Thresholded COO plan; returns dict(rows, cols, vals, batch_offsets, nnz).
    With capacity None the call runs twice if needed (count, then write)."""
    X, Y, B, n, m, d = _shapes(X, Y, a, b)
    dev = X.device
    _potentials_args(f, g, B, n, m, dev)
    L = load()
    off = torch.empty(B + 1, device=dev, dtype=torch.int64)
    nnz = C.c_longlong(0)
    cap = int(capacity) if capacity is not None else 0
    rows = torch.empty(max(cap, 1), device=dev, dtype=torch.int32)
    cols = torch.empty(max(cap, 1), device=dev, dtype=torch.int32)
    vals = torch.empty(max(cap, 1), device=dev, dtype=torch.float32)
    args = lambda: (_ptr(X), _ptr(Y), _ptr(a), _ptr(b), B, n, m, d, _ptr(f), _ptr(g), float(eps), float(threshold),
                    int(dirs), cap, _ptr(rows), _ptr(cols), _ptr(vals), _ptr(off), C.byref(nnz), _stream(stream))
    rc = L.sot_plan_coo(*args())
    if rc == SOT_ERR_CAPACITY and capacity is None:
        cap = int(nnz.value)
        rows = torch.empty(max(cap, 1), device=dev, dtype=torch.int32)
        cols = torch.empty(max(cap, 1), device=dev, dtype=torch.int32)
        vals = torch.empty(max(cap, 1), device=dev, dtype=torch.float32)
        rc = L.sot_plan_coo(*args())
    if rc == SOT_ERR_CAPACITY:
        raise SotError(rc, "sot_plan_coo", f"capacity {cap} < nnz {nnz.value}")
    _check(rc, "sot_plan_coo")
    k = int(nnz.value)
    return dict(rows=rows[:k], cols=cols[:k], vals=vals[:k], batch_offsets=off, nnz=k)


def sot_plan_coo_operands(X, Y, a, b, f, g, eps, threshold=1e-8, stream=None):
    """The fp32 operands sot_plan_coo decides its support from; returns
    dict(xc, lwx, Lx, yc, lwy, Ly, Mr, Mc, kappa, log2tau)."""
    X, Y, B, n, m, d = _shapes(X, Y, a, b)
    dev = X.device
    _potentials_args(f, g, B, n, m, dev)
    L = load()
    new = lambda *shape: torch.empty(*shape, device=dev, dtype=torch.float32)  # noqa: E731
    out = dict(xc=new(B, n, d), lwx=new(B, n), Lx=new(B, n), yc=new(B, m, d), lwy=new(B, m), Ly=new(B, m), Mr=new(B, n),
               Mc=new(B, m))
    sc = (C.c_float * 2)()
    rc = L.sot_plan_coo_operands(_ptr(X), _ptr(Y), _ptr(a), _ptr(b), B, n, m, d, _ptr(f), _ptr(g), float(eps),
                                 float(threshold), *(_ptr(out[k]) for k in ("xc", "lwx", "Lx", "yc", "lwy", "Ly",
                                                                            "Mr", "Mc")),
                                 sc, _stream(stream))
    _check(rc, "sot_plan_coo_operands")
    out["kappa"], out["log2tau"] = float(sc[0]), float(sc[1])
    return out


def sot_grad_x_coo(X, Y, rows, cols, vals, batch_offsets, grad=None, stream=None):
    X, Y, B, n, m, d = _shapes(X, Y, None, None)
    dev = X.device
    _want(rows, "rows", None, dev, torch.int32)
    _want(cols, "cols", rows.numel(), dev, torch.int32)
    _want(vals, "vals", rows.numel(), dev)
    _want(batch_offsets, "batch_offsets", B + 1, dev, torch.int64)
    grad = torch.empty(B, n, d, device=X.device, dtype=torch.float32) if grad is None else grad
    _want(grad, "grad", B * n * d, dev)
    rc = load().sot_grad_x_coo(_ptr(X), _ptr(Y), B, n, m, d, _ptr(rows), _ptr(cols), _ptr(vals),
                               _ptr(batch_offsets), _ptr(grad), _stream(stream))
    _check(rc, "sot_grad_x_coo")
    return grad


# ---- language-model training losses ---------------------------------------------------------------------------------
# A call on a handful of tokens takes the GPU 4 to 6 us, so these marshal with
# as few interpreter steps as the checks allow: each helper answers with the
# tensor's address once everything about it is right, and only what is wrong is
# looked at again to say what.
_F32 = torch.float32
# (the handle without a stream object around it; a torch without CUDA has neither)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (lambda dev: torch.cuda.current_stream(dev).cuda_stream)


def _logits(x, name="logits"):
    """(address, rows, columns, row stride, sot_dtype, device index) of [rows, columns] whose rows are contiguous."""
    try:
        dt = _FLOATS[x.dtype]
        T, V = x.shape
        ld, inner = x.stride()
        dev = x.get_device()
        if dev >= 0 and (inner == 1 or V == 1) and (ld >= V or T <= 1):
            return x.data_ptr(), T, V, ld if T > 1 else V, dt, dev
    except (AttributeError, KeyError, ValueError):
        pass
    if not isinstance(x, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if x.dtype not in _FLOATS:
        raise TypeError(f"{name} must be float32, float16 or bfloat16, got {x.dtype}")
    if x.dim() != 2:
        raise ValueError(f"{name} must be [rows, columns], got shape {tuple(x.shape)}")
    if not x.is_cuda:
        raise ValueError(f"{name} must be on a CUDA device")
    if x.shape[1] > 1 and x.stride(1) != 1:
        raise ValueError(f"{name}: the elements of a row must be contiguous")
    raise ValueError(f"{name}: rows must not overlap (row stride {x.stride(0)}, {x.shape[1]} columns)")


def _floats(t, name, n, dev, dtype=_F32):
    """Address of a contiguous tensor of n elements of this type on this device; None for None."""
    if t is None:
        return None
    try:
        if t.dtype is dtype and t.numel() == n and t.get_device() == dev and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        pass
    _want(t, name, n, torch.device("cuda", dev), dtype)


def _needed(t, name, n, dev):
    if t is None:
        raise TypeError(f"{name} must be a torch.Tensor")
    return _floats(t, name, n, dev)


def _indices(t, name, shape, dev):
    """(address, sot_dtype) of a contiguous int32 or int64 tensor of this shape on this device."""
    try:
        ty = _INDICES[t.dtype]
        if t.shape == shape and t.get_device() == dev and t.is_contiguous():
            return t.data_ptr(), ty
    except (AttributeError, KeyError):
        pass
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype not in _INDICES:
        raise TypeError(f"{name} must be int32 or int64, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.get_device() != dev:
        raise ValueError(f"{name} must be on cuda:{dev}, got {t.device}")
    raise ValueError(f"{name} must be contiguous")


def _pairs(t, name, T, dev):
    """(address, sot_dtype, columns) of an index tensor [T, columns]."""
    if not isinstance(t, torch.Tensor) or t.dim() != 2:
        raise ValueError(f"{name} must be [rows, entries]")
    K = t.shape[1]
    return *_indices(t, name, (T, K), dev), K


def _grad_of(grad, logits, T, V, ld, dt, dev):
    """(tensor or None, address, row stride) of a gradient asked for as True, False, None or a tensor."""
    if grad is True:
        g = torch.empty_like(logits) if ld == V else torch.empty((T, V), dtype=logits.dtype, device=logits.device)
        return g, g.data_ptr(), V
    if grad is None or grad is False:
        return None, None, 0
    at, gT, gV, gld, gdt, gdev = _logits(grad, "grad")
    if (gT, gV, gdt, gdev) != (T, V, dt, dev):
        raise ValueError(f"grad must be {logits.dtype} of shape {(T, V)} on {logits.device}")
    return grad, at, gld


def _on(stream, call):
    """call(handle) on the given stream: what it allocates is then the stream's own,
    not memory that another stream's work may still be using."""
    with torch.cuda.stream(stream):
        return call(stream.cuda_stream)


def sot_token_logprob(logits, target, temperature=1.0, logp=None, lse=None, stream=None):
    """Log-probability of one token per row: (logp [T], lse [T]) float32 of logits
    [T, V] (float32, float16 or bfloat16, any row stride) and target [T].  A
    target outside [0, V) leaves its row out (both values 0)."""
    x, T, V, ld, dt, dev = _logits(logits)
    tg, ty = _indices(target, "target", (T,), dev)
    _floats(logp, "logp", T, dev)
    _floats(lse, "lse", T, dev)

    def call(s):
        p = torch.empty(T, dtype=_F32, device=logits.device) if logp is None else logp
        q = torch.empty_like(p) if lse is None else lse
        rc = load().sot_token_logprob(x, T, V, ld, dt, temperature, tg, ty, p.data_ptr(), q.data_ptr(), s)
        if rc:
            _check(rc, "sot_token_logprob")
        return p, q
    return call(_raw_stream(dev)) if stream is None else _on(stream, call)


def sot_token_logprob_grad(logits, target, lse, grad_logp, temperature=1.0, grad=True, stream=None):
    """Gradient [T, V] (the logits' type) of sum_t grad_logp[t] logp[t], from the lse of
    sot_token_logprob.  ``grad`` may be a tensor to write, the logits included."""
    x, T, V, ld, dt, dev = _logits(logits)
    tg, ty = _indices(target, "target", (T,), dev)
    l, g = _needed(lse, "lse", T, dev), _needed(grad_logp, "grad_logp", T, dev)

    def call(s):
        out, at, ldg = _grad_of(grad, logits, T, V, ld, dt, dev)
        rc = load().sot_token_logprob_grad(x, T, V, ld, dt, temperature, tg, ty, l, g, at, ldg, s)
        if rc:
            _check(rc, "sot_token_logprob_grad")
        return out
    return call(_raw_stream(dev)) if stream is None else _on(stream, call)


def sot_distill_topk(logits, ids, teacher, weight=None, temperature=1.0, tail=False, grad=True, loss=None, stream=None):
    """Distillation from a teacher's top entries: (loss [T], grad [T, V] or None).
    ids and teacher are [T, K]; an id outside [0, V) is an unused entry.  Without
    ``tail`` the teacher values are logits; with it they are log-probabilities and
    the mass outside the entries is one more outcome.  weight [T] (None = 1/T), 0
    leaves a row out.  ``grad``: True, False or a tensor (the logits included)."""
    x, T, V, ld, dt, dev = _logits(logits)
    i, ty, K = _pairs(ids, "ids", T, dev)
    tt = _FLOATS.get(teacher.dtype) if isinstance(teacher, torch.Tensor) else None
    if tt is None:
        raise TypeError("teacher must be a float32, float16 or bfloat16 torch.Tensor")
    if teacher.dim() > 1 and teacher.shape != ids.shape:
        raise ValueError(f"teacher must have the shape of ids, {(T, K)}, got {tuple(teacher.shape)}")
    z = _floats(teacher, "teacher", T * K, dev, teacher.dtype)
    w = _floats(weight, "weight", T, dev)
    _floats(loss, "loss", T, dev)

    def call(s):
        lo = torch.empty(T, dtype=_F32, device=logits.device) if loss is None else loss
        g, at, ldg = _grad_of(grad, logits, T, V, ld, dt, dev)
        rc = load().sot_distill_topk(x, T, V, ld, dt, temperature, i, ty, z, tt, K, 1 if tail else 0, w, lo.data_ptr(), at,
                                     ldg, s)
        if rc:
            _check(rc, "sot_distill_topk")
        return lo, g
    return call(_raw_stream(dev)) if stream is None else _on(stream, call)


def sot_policy_loss(logits, target, old_logp, advantage, ref_logp=None, weight=None, temperature=1.0, clip_low=0.2,
                    clip_high=0.2, kl_coef=0.0, grad=True, stream=None):
    """Clipped policy loss with a KL term: (loss [T], logp [T], kl [T], grad [T, V] or
    None).  old_logp, advantage, ref_logp and weight are [T]; weight None = 1/T, 0
    leaves a row out, as does a target outside [0, V).  Without ref_logp, kl_coef
    takes no part.  ``grad``: True, False or a tensor (the logits included)."""
    x, T, V, ld, dt, dev = _logits(logits)
    tg, ty = _indices(target, "target", (T,), dev)
    old, adv = _needed(old_logp, "old_logp", T, dev), _needed(advantage, "advantage", T, dev)
    ref, w = _floats(ref_logp, "ref_logp", T, dev), _floats(weight, "weight", T, dev)

    def call(s):
        loss = torch.empty_like(old_logp)
        logp, kl = torch.empty_like(loss), torch.empty_like(loss)
        g, at, ldg = _grad_of(grad, logits, T, V, ld, dt, dev)
        rc = load().sot_policy_loss(x, T, V, ld, dt, temperature, tg, ty, old, ref, adv, w, clip_low, clip_high,
                                    0.0 if ref is None else kl_coef, loss.data_ptr(), logp.data_ptr(), kl.data_ptr(), at,
                                    ldg, s)
        if rc:
            _check(rc, "sot_policy_loss")
        return loss, logp, kl, g
    return call(_raw_stream(dev)) if stream is None else _on(stream, call)


def sot_preference_loss(logp, offsets, ref_logp=None, target=None, beta=0.1, label_smoothing=0.0, average=False,
                        scale=None, stream=None):
    """Paired preference loss on token log-probabilities [T]: (loss [P], margin [P],
    grad_logp [T]).  offsets [2P+1] int64 packs chosen, rejected, chosen, ...; a
    token whose target is negative takes no part.  scale None = 1/P."""
    if not isinstance(logp, torch.Tensor) or not isinstance(offsets, torch.Tensor):
        raise TypeError("logp and offsets must be torch.Tensors")
    if not logp.is_cuda:
        raise ValueError("logp must be on a CUDA device")
    dev, T, n = logp.get_device(), logp.numel(), offsets.numel()
    lp = _floats(logp, "logp", T, dev)
    if n % 2 == 0:
        raise ValueError("offsets must hold 2 P + 1 elements")
    off = _floats(offsets, "offsets", n, dev, torch.int64)
    P = n // 2
    ref = _floats(ref_logp, "ref_logp", T, dev)
    tg, ty = (None, SOT_I32) if target is None else _indices(target, "target", (T,), dev)
    if scale is None:
        scale = 1.0 / max(P, 1)

    def call(s):
        loss = torch.empty(P, dtype=_F32, device=logp.device)
        margin, g = torch.empty_like(loss), torch.empty_like(logp)
        rc = load().sot_preference_loss(lp, ref, tg, ty, off, P, T, beta, label_smoothing, 1 if average else 0, scale,
                                        loss.data_ptr(), margin.data_ptr(), g.data_ptr(), s)
        if rc:
            _check(rc, "sot_preference_loss")
        return loss, margin, g
    return call(_raw_stream(dev)) if stream is None else _on(stream, call)


def sot_balance_loss(logits, ids, mask=None, balance_coef=1.0, z_coef=0.0, grad=True, stream=None):
    """A router's balance and z losses with per-expert counts: (counts [E] int32,
    loss [2], grad [T, E] or None) of router logits [T, E] and the experts chosen,
    ids [T, K] (outside [0, E): dropped).  mask [T] bool: False leaves a token out."""
    x, T, E, ld, dt, dev = _logits(logits)
    i, ty, K = _pairs(ids, "ids", T, dev)
    m = _floats(mask, "mask", T, dev, torch.bool)

    def call(s):
        counts = torch.empty(E, dtype=torch.int32, device=logits.device)
        loss = torch.empty(2, dtype=_F32, device=logits.device)
        g, at, ldg = _grad_of(grad, logits, T, E, ld, dt, dev)
        rc = load().sot_balance_loss(x, T, E, ld, dt, i, ty, K, m, balance_coef, z_coef, counts.data_ptr(),
                                     loss.data_ptr(), at, ldg, s)
        if rc:
            _check(rc, "sot_balance_loss")
        return counts, loss, g
    return call(_raw_stream(dev)) if stream is None else _on(stream, call)


# ---- language-model operators around the losses ---------------------------------------------------------------------
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _run(dev, stream, call):
    """call(handle) on the given stream, or on the current stream of the tensors' device, with that device current."""
    if stream is not None:
        if stream.device.index != dev:
            raise ValueError(f"the stream belongs to {stream.device}, the tensors to cuda:{dev}")
        return _on(stream, call)
    if _current_device() == dev:
        return call(_raw_stream(dev))
    with torch.cuda.device(dev):
        return call(_raw_stream(dev))


def _count(n, name, least):
    """A whole number that the library takes in 32 bits (ctypes would cut a larger one off without a word)."""
    n = int(n)
    if not least <= n < 1 << 31:
        raise ValueError(f"{name} must satisfy {least} <= {name} < 2^31, got {n}")
    return n


def sot_token_topk(logits, K, target=None, temperature=1.0, stream=None):
    """Scores of given tokens with entropies and the best alternatives: (logp [T] or None, lse [T], entropy [T],
    ids [T, K] int32, top_logp [T, K]) of logits [T, V].  ids are the columns of the K largest logits, largest first,
    lower columns first among equal ones; entries that do not exist (masked by -inf, beyond V) are -1 with -inf.
    They are what sot_distill_topk takes as its teacher.  A target outside [0, V) leaves its row out (0, ids -1);
    without target every row takes part and logp is None."""
    x, T, V, ld, dt, dev = _logits(logits)
    tg, ty = (None, SOT_I32) if target is None else _indices(target, "target", (T,), dev)
    K = _count(K, "K", 0)

    def call(s):
        lse = torch.empty(T, dtype=_F32, device=logits.device)
        entropy = torch.empty_like(lse)
        logp = None if target is None else torch.empty_like(lse)
        top = torch.empty((T, K), dtype=_F32, device=logits.device)
        ids = torch.empty((T, K), dtype=torch.int32, device=logits.device)
        rc = load().sot_token_topk(x, T, V, ld, dt, temperature, tg, ty, K, None if logp is None else logp.data_ptr(),
                                   lse.data_ptr(), entropy.data_ptr(), ids.data_ptr(), top.data_ptr(), s)
        if rc:
            _check(rc, "sot_token_topk")
        return logp, lse, entropy, ids, top
    return _run(dev, stream, call)


def sot_token_topk_grad(logits, lse, entropy=None, target=None, grad_logp=None, grad_entropy=None, ids=None, grad_top=None,
                        temperature=1.0, grad=True, stream=None):
    """Gradient [T, V] (the logits' type) of sot_token_topk's outputs, from the lse and entropy it gave and the gradients
    with respect to logp [T], entropy [T] and top_logp [T, K] (None: 0; grad_top needs the ids, int32).  ``grad`` may be a
    tensor to write, the logits included."""
    x, T, V, ld, dt, dev = _logits(logits)
    tg, ty = (None, SOT_I32) if target is None else _indices(target, "target", (T,), dev)
    l, h = _needed(lse, "lse", T, dev), _floats(entropy, "entropy", T, dev)
    gl, gh = _floats(grad_logp, "grad_logp", T, dev), _floats(grad_entropy, "grad_entropy", T, dev)
    i, K, gt = None, 0, None
    if grad_top is not None:
        if ids is None:
            raise TypeError("grad_top needs ids")
        i, ity, K = _pairs(ids, "ids", T, dev)
        if ity != SOT_I32:
            raise TypeError("ids must be int32")
        gt = _indices_like(grad_top, "grad_top", ids)
    if grad is None or grad is False:
        raise TypeError("grad must be True or a tensor")

    def call(s):
        out, at, ldg = _grad_of(grad, logits, T, V, ld, dt, dev)
        rc = load().sot_token_topk_grad(x, T, V, ld, dt, temperature, tg, ty, l, h, gl, gh, i, K, gt, at, ldg, s)
        if rc:
            _check(rc, "sot_token_topk_grad")
        return out
    return _run(dev, stream, call)


def _indices_like(t, name, ids):
    """Address of a float32 tensor of the shape of ids."""
    if isinstance(t, torch.Tensor) and t.shape != ids.shape:
        raise ValueError(f"{name} must have the shape of ids, {tuple(ids.shape)}, got {tuple(t.shape)}")
    return _floats(t, name, ids.numel(), ids.get_device())


def _matrix(t, name, rows, D, dev):
    """(address, row stride, sot_dtype) of a tensor [rows, D] whose rows are contiguous, on this device."""
    at, n, d, ld, dt, on = _logits(t, name)
    if (n, d) != (rows, D):
        raise ValueError(f"{name} must have shape {(rows, D)}, got {(n, d)}")
    if on != dev:
        raise ValueError(f"{name} must be on cuda:{dev}, got {t.device}")
    return at, ld, dt


def _float_type(dtype, default):
    """sot_dtype of a torch float type; the default for None."""
    if dtype is None:
        return default
    try:
        return _FLOATS[dtype]
    except (KeyError, TypeError):
        raise TypeError(f"dtype must be float32, float16 or bfloat16, got {dtype}") from None


def sot_embed(table, ids, scale=1.0, dtype=None, out=None, stream=None):
    """Embedding lookup with scaling: out [T, D] = scale table[ids] in 32 bits, rounded; rows of zeros for ids outside
    [0, V).  table [V, D] may have a row stride, ids is [T]; ``dtype`` (default the table's) is the type of a new out."""
    x, V, D, ld, dt, dev = _logits(table, "table")
    V = _count(V, "V", 1)
    if not isinstance(ids, torch.Tensor) or ids.dim() != 1:
        raise ValueError("ids must be a torch.Tensor of shape [T]")
    T = ids.shape[0]
    i, ty = _indices(ids, "ids", (T,), dev)
    ot = _float_type(dtype, dt)
    if out is not None:
        at, ldo, ot = _matrix(out, "out", T, D, dev)

    def call(s):
        if out is not None:
            o, to, ld_out = out, at, ldo
        else:
            o = torch.empty((T, D), dtype=dtype or table.dtype, device=table.device)
            to, ld_out = o.data_ptr(), D
        rc = load().sot_embed(x, V, D, ld, dt, i, ty, T, scale, to, ld_out, ot, s)
        if rc:
            _check(rc, "sot_embed")
        return o
    return _run(dev, stream, call)


def sot_embed_grad(grad_out, ids, V, scale=1.0, dtype=None, grad=None, accumulate=False, stream=None):
    """Gradient [V, D] of sot_embed with respect to the table: scale times the sums of grad_out [T, D] over the tokens
    of each row, tokens sorted by row, the same bits on every call.  ``grad`` may be a tensor to write; with ``accumulate``
    the sums are added to it and rows that no token names stay untouched (with weights tied to the output head, its
    gradient).  ``dtype`` (default grad_out's) is the type of a new gradient."""
    x, T, D, ld, dt, dev = _logits(grad_out, "grad_out")
    i, ty = _indices(ids, "ids", (T,), dev)
    V = _count(V, "V", 1)
    if accumulate and grad is None:
        raise TypeError("accumulate needs a gradient to add to")
    gt = _float_type(dtype, dt)
    if grad is not None:
        at, ldg, gt = _matrix(grad, "grad", V, D, dev)

    def call(s):
        if grad is not None:
            g, to, ld_grad = grad, at, ldg
        else:
            g = torch.empty((V, D), dtype=dtype or grad_out.dtype, device=grad_out.device)
            to, ld_grad = g.data_ptr(), D
        rc = load().sot_embed_grad(x, T, D, ld, dt, i, ty, V, scale, 1 if accumulate else 0, to, ld_grad, gt, s)
        if rc:
            _check(rc, "sot_embed_grad")
        return g
    return _run(dev, stream, call)


def sot_routed_layer(x, router, gate_up, down, K, bias=None, renorm=True, scale=1.0, out=None, stream=None):
    """A routed layer for a few tokens (at most 128): (out [T, H], logits [T, E] float32, ids [T, K] int32, weights [T, K]
    float32) of x [T, H], router [E, H], gate_up [E, 2 F, H], down [E, H, F] (one type) and bias [E] float32.
    out = sum over a token's K best experts of weight * down (silu(gate x) * up x).  logits and ids go on to
    sot_balance_loss.  The tensor cores take float16 and bfloat16 with H, F and x's row stride multiples of 8 and x, gate_up
    and down at 16-byte addresses; anything else is right too, but many times slower (x.contiguous() before the call)."""
    at, T, H, ld, dt, dev = _logits(x, "x")
    K = int(K)
    try:
        E, F = router.shape[0], down.shape[2]
        agree = router.shape == (E, H) and gate_up.shape == (E, 2 * F, H) and down.shape == (E, H, F)
    except (AttributeError, IndexError):
        agree = False
    if not agree:
        raise ValueError("x [T, H], router [E, H], gate_up [E, 2 F, H] and down [E, H, F] must be torch.Tensors that agree, got "
                         + ", ".join(str(tuple(getattr(t, "shape", ()))) for t in (x, router, gate_up, down)))
    r = _floats(router, "router", E * H, dev, x.dtype)
    gu, dn = _floats(gate_up, "gate_up", E * 2 * F * H, dev, x.dtype), _floats(down, "down", E * H * F, dev, x.dtype)
    b = _floats(bias, "bias", E, dev)
    if K < 1 or K > E:
        raise ValueError(f"K must satisfy 1 <= K <= {E}")
    if out is not None:
        to, ld_out, ot = _matrix(out, "out", T, H, dev)
        if ot != dt:
            raise TypeError(f"out must be {x.dtype}, got {out.dtype}")

    def call(s):
        if out is not None:
            o, oat, ldo = out, to, ld_out
        else:
            o = torch.empty((T, H), dtype=x.dtype, device=x.device)
            oat, ldo = o.data_ptr(), H
        logits = torch.empty((T, E), dtype=_F32, device=x.device)
        ids = torch.empty((T, K), dtype=torch.int32, device=x.device)
        weights = torch.empty((T, K), dtype=_F32, device=x.device)
        rc = load().sot_routed_layer(at, T, H, ld, dt, r, b, E, gu, dn, F, K, 1 if renorm else 0, scale, oat, ldo,
                                     logits.data_ptr(), ids.data_ptr(), weights.data_ptr(), s)
        if rc:
            _check(rc, "sot_routed_layer")
        return o, logits, ids, weights
    return _run(dev, stream, call)


def sot_async_status(stream=None):
    """Raises SotError(SOT_ERR_TIMEOUT) when a bounded device-side wait gave up
    in an asynchronous call since the last check on this device; clears it."""
    _check(load().sot_async_status(_stream(stream)), "sot_async_status")


def sot_test_hold_tile(tile: int, after_launches: int = 0, wait_ns: int = 0):
    """Testing hook: after `after_launches` more tensor-core launches, those
    kernels withhold column tile `tile` of their chunk onward (tile < 0: off),
    so their waits run out after wait_ns nanoseconds."""
    _check(load().sot_test_hold_tile(int(tile), int(after_launches), int(wait_ns)), "sot_test_hold_tile")


def sot_test_hold_routed(what: int, wait_ns: int = 0):
    """Testing hook: a CTA of the routed layer's tensor-core kernel withholds its arrival at a meeting (what = 0 to 3) or its
    weights from unit what - 4 on (what < 0: off), so that waits run out after wait_ns nanoseconds."""
    _check(load().sot_test_hold_routed(int(what), int(wait_ns)), "sot_test_hold_routed")


def sot_check_inputs(X, Y, a=None, b=None, stream=None) -> int:
    """Returns the status code (0 ok, SOT_ERR_NONFINITE, ...) without raising."""
    X, Y, B, n, m, d = _shapes(X, Y, a, b)
    return int(load().sot_check_inputs(_ptr(X), _ptr(Y), _ptr(a), _ptr(b), B, n, m, d, _stream(stream)))


def sot_profile_enable(on: bool = True):
    _check(load().sot_profile_enable(int(bool(on))), "sot_profile_enable")


def sot_profile_read():
    """(half-step launches, total milliseconds) since the last read."""
    n = C.c_longlong(0)
    ms = C.c_double(0)
    _check(load().sot_profile_read(C.byref(n), C.byref(ms)), "sot_profile_read")
    return int(n.value), float(ms.value)


def sot_profile_read_kinds():
    """{"full": (half-steps, ms), "screened": (...), "cluster": (...)} since the last read."""
    n = (C.c_longlong * 3)()
    ms = (C.c_double * 3)()
    _check(load().sot_profile_read_kinds(n, ms), "sot_profile_read_kinds")
    return {"full": (int(n[0]), float(ms[0])), "screened": (int(n[1]), float(ms[1])),
            "cluster": (int(n[2]), float(ms[2]))}
