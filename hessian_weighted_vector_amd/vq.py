"""Python binding of libvq (ctypes).  Argument marshalling only.

Every function takes torch tensors that already live on the GPU (PyTorch is
used for device memory and streams), passes their device pointers and the
current stream to the C ABI declared in include/vq.h, and raises VQError on
a non-zero status.  There is no fallback: if libvq.so is missing or no
gfx950 device is present the call fails.
"""
import ctypes
import functools
import math
import os
import weakref

import numpy as np
import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libvq.so")

VQ_OK, VQ_ERR_INVALID, VQ_ERR_WORKSPACE, VQ_ERR_INIT, VQ_ERR_DEVICE, VQ_ERR_UNSUPPORTED = range(6)
STATUS_NAMES = {0: "VQ_OK", 1: "VQ_ERR_INVALID", 2: "VQ_ERR_WORKSPACE", 3: "VQ_ERR_INIT",
                4: "VQ_ERR_DEVICE", 5: "VQ_ERR_UNSUPPORTED"}


class VQError(RuntimeError):
    def __init__(self, status, msg):
        super().__init__("%s: %s" % (STATUS_NAMES.get(status, status), msg))
        self.status = status


_P = ctypes.c_void_p
_I64 = ctypes.c_int64
_I = ctypes.c_int
_SZ = ctypes.c_size_t
_D = ctypes.c_double


class FitParams(ctypes.Structure):
    _fields_ = [("M", _I64), ("N", _I64), ("d", _I), ("K1", _I), ("iters1", _I), ("K2", _I),
                ("iters2", _I), ("outlier_frac", _D), ("binorm", _I), ("mask_outliers", _I)]


class FitInputs(ctypes.Structure):
    _fields_ = [("W", _P), ("h", _P), ("perm1", _P), ("perm2", _P), ("C1_init", _P), ("C2_init", _P)]


class FitOutputs(ctypes.Structure):
    _fields_ = [("idx1", _P), ("C1", _P), ("idx2", _P), ("C2", _P), ("row_ptr", _P), ("col", _P),
                ("val", _P), ("mask", _P), ("Wp", _P), ("rscale", _P), ("cscale", _P), ("hcol", _P),
                ("rho", _P), ("W_hat", _P), ("J_hist", _P), ("bpw", _P), ("empty_hist", _P)]


class GroupedParams(ctypes.Structure):
    _fields_ = [("fit", FitParams), ("n_out", _I64), ("d0", _I), ("K0", _I), ("iters0", _I), ("n_groups", _I)]


class GroupedInputs(ctypes.Structure):
    _fields_ = [("W", _P), ("h", _P), ("perm1", _P), ("perm2", _P)]


class GroupedOutputs(ctypes.Structure):
    _fields_ = [("cols", _P), ("idx", _P), ("codebooks", _P), ("row_ptr", _P), ("col", _P), ("val", _P),
                ("mask", _P), ("W_hat", _P), ("J_hist", _P), ("bpw", _P)]


class QMatrixStruct(ctypes.Structure):
    _fields_ = [("M", _I64), ("N", _I64), ("d", _I), ("K1", _I), ("K2", _I), ("C1", _P), ("idx1", _P), ("C2", _P),
                ("idx2", _P), ("rscale", _P), ("cscale", _P), ("row_ptr", _P), ("col", _P), ("delta", _P)]


class I8MatrixStruct(ctypes.Structure):
    _fields_ = [("M", _I64), ("N", _I64), ("q", _P), ("ldq", _I64), ("scale", _P)]


class AdamWTensor(ctypes.Structure):
    _fields_ = [("param", _P), ("grad", _P), ("master", _P), ("m", _P), ("v", _P), ("m_scale", _P), ("v_scale", _P),
                ("n", _I64)]


class AdamWPlan(ctypes.Structure):
    _fields_ = [("table", _P), ("count", _I64), ("chunks", _I64), ("param_dtype", _I), ("grad_dtype", _I),
                ("has_master", _I), ("state_bits", _I), ("known", _P)]


# name -> (restype, argtypes); every symbol declared in include/vq.h
SIGNATURES = {
    "vq_version": (ctypes.c_char_p, []),
    "vq_last_error": (ctypes.c_char_p, []),
    "vq_workspace_bytes": (_SZ, [_I64, _I64, _I, _I, _I, _I64]),
    "vq_sparse_select": (_I, [_P, _P, _I64, _I64, _I, _I64, _P, _P, _P, _P, _P, _SZ, _P]),
    "vq_binorm": (_I, [_P, _P, _I64, _I64, _P, _P, _P, _P, _P, _P, _SZ, _P]),
    "vq_init": (_I, [_P, _I64, _I64, _I, _P, _I, _P, _P, _SZ, _P]),
    "vq_assign": (_I, [_P, _P, _P, _P, _I64, _I64, _I, _P, _I, _P, _P, _P, _SZ, _P]),
    "vq_assign_noalloc": (_I, [_P, _P, _P, _P, _I64, _I64, _I, _P, _I, _P, _P, _P]),
    "vq_assign_exact_count": (_I, [_P, _SZ, _I64, _I, _P]),
    "vq_assign_exact_list": (_I64, [_P, _SZ, _I64, _I, _P, _I64, _P]),
    "vq_nnz": (_I64, [_I64, _I64, _D]),
    "vq_update": (_I, [_P, _P, _P, _P, _I64, _I64, _I, _P, _I, _P, _P, _P, _P, _SZ, _P]),
    "vq_objective": (_I, [_P, _P, _P, _P, _I64, _I64, _I, _P, _I, _P, _P, _P, _SZ, _P]),
    "vq_residual": (_I, [_P, _I64, _I64, _I, _P, _I, _P, _P, _P]),
    "vq_reconstruct": (_I, [_I64, _I64, _I, _P, _I, _P, _P, _I, _P, _P, _P, _P, _P, _P, _P, _P]),
    "vq_select_subvectors": (_I, [_P, _P, _I64, _I64, _I, _I64, _P, _P, _SZ, _P]),
    "vq_select_residual": (_I, [_P, _P, _P, _I64, _I64, _I, _I64, _P, _P, _SZ, _P]),
    "vq_mask_to_csr": (_I, [_P, _P, _I64, _I64, _I, _I64, _P, _P, _P, _P, _SZ, _P]),
    "vq_hessian_factor_workspace_bytes": (_SZ, [_I64]),
    "vq_hessian_factor": (_I, [_P, _I64, _D, _P, _P, _SZ, _P]),
    "vq_vptq_workspace_bytes": (_SZ, [_I64, _I64, _I]),
    "vq_vptq": (_I, [_P, _P, _I64, _I64, _I, _P, _I, _I, _P, _P, _P, _P, _SZ, _P]),
    "vq_qgemv_workspace_bytes": (_SZ, [_I64, _I64, _I, _I64]),
    "vq_qgemv": (_I, [_I64, _I64, _I, _P, _I, _P, _P, _I, _P, _P, _P, _P, _P, _P, _P, _I64, _P, _P, _SZ,
                      _P]),
    "vq_fit": (_I, [ctypes.POINTER(FitParams), ctypes.POINTER(FitInputs), ctypes.POINTER(FitOutputs),
                    _P, _SZ, _P]),
    "vq_grouped_sizes": (_SZ, [ctypes.POINTER(GroupedParams), ctypes.POINTER(_I64), ctypes.POINTER(_I64),
                               ctypes.POINTER(_I64), ctypes.POINTER(_I64), ctypes.POINTER(_I64)]),
    "vq_fit_grouped": (_I, [ctypes.POINTER(GroupedParams), ctypes.POINTER(GroupedInputs),
                            ctypes.POINTER(GroupedOutputs), _P, _SZ, _P]),
    "vq_bits_per_weight_grouped": (_D, [ctypes.POINTER(GroupedParams)]),
    "vq_bits_per_weight": (_D, [_I64, _I64, _I, _I, _I, _I64, _I, _I]),
    "vq_linear_workspace_bytes": (_SZ, [_I64, _I64, _I64, _P, _I64, _P, _I64]),
    "vq_linear": (_I, [_I64, _I64, _I64, _I, _I, _P, _I64, _P, _I64, _P, _P, _I64, _P, _I64, _P, _I64, _P, _SZ, _P]),
    "vq_linear_backward_workspace_bytes": (_SZ, [_I64, _I64, _I64, _I, _P, _I64, _P, _I64, _P, _I64, _I, _I, _I]),
    "vq_linear_backward": (_I, [_I64, _I64, _I64, _I, _I, _P, _I64, _P, _I64, _P, _I64, _P, _I64, _P, _I64, _P, _I64,
                                _P, _P, _SZ, _P]),
    "vq_gated_workspace_bytes": (_SZ, [_I64, _I64, _I64, _P, _I64, _P, _P, _I64]),
    "vq_gated": (_I, [_I64, _I64, _I64, _I, _I, _P, _I64, _P, _P, _I64, _P, _P, _P, _I64, _P, _P, _I64, _P, _SZ, _P]),
    "vq_gated_backward_workspace_bytes": (_SZ, [_I64, _I64, _I64, _I, _P, _I64, _P, _I64, _P, _P, _I64, _I, _I, _I]),
    "vq_gated_backward": (_I, [_I64, _I64, _I64, _I, _I, _P, _I64, _P, _I64, _P, _P, _I64, _P, _P, _I64, _P, _I64,
                               _P, _P, _I64, _P, _P, _P, _SZ, _P]),
    "vq_sparse_delta": (_I, [_P, _P, _P, _P]),
    "vq_qlinear_workspace_bytes": (_SZ, [_I64, _I64, _I, _I64]),
    "vq_qlinear": (_I, [_P, _I64, _I, _I, _P, _I64, _P, _P, _I64, _P, _I64, _P, _SZ, _P]),
    "vq_qgated_workspace_bytes": (_SZ, [_I64, _I64, _I, _I64]),
    "vq_qgated": (_I, [_P, _P, _I64, _I, _I, _P, _I64, _P, _P, _P, _I64, _P, _SZ, _P]),
    "vq_linear_i8_workspace_bytes": (_SZ, [_I64, _I64, _I64]),
    "vq_linear_i8": (_I, [_P, _I64, _I, _I, _P, _I64, _P, _P, _I64, _P, _I64, _P, _SZ, _P]),
    "vq_gated_i8_workspace_bytes": (_SZ, [_I64, _I64, _I64]),
    "vq_gated_i8": (_I, [_P, _P, _I64, _I, _I, _P, _I64, _P, _P, _P, _I64, _P, _SZ, _P]),
    "vq_quantize_rows": (_I, [_I64, _I64, _I, _P, _I64, _P, _I64, _P, _P]),
    "vq_cross_entropy_workspace_bytes": (_SZ, [_I64, _I64, _I64, _P, _I64]),
    "vq_cross_entropy": (_I, [_I64, _I64, _I64, _I, _P, _I64, _P, _I64, _P, _I64, _P, _P, _P, _SZ, _P]),
    "vq_cross_entropy_backward_workspace_bytes": (_SZ, [_I64, _I64, _I64, _P, _I64, _I, _I]),
    "vq_cross_entropy_backward": (_I, [_I64, _I64, _I64, _I, _P, _P, _I64, _P, _I64, _P, _I64, _P, _P, _I64, _P, _I64,
                                       _P, _SZ, _P]),
    "vq_adamw_plan_bytes": (_SZ, [_P, _I64]),
    "vq_adamw_plan": (_I, [_P, _I64, _I, _I, _I, _I, _P, _SZ, _P, _P]),
    "vq_adamw_plan_free": (None, [_P]),
    "vq_adamw_grads": (_I, [_P, _P, _I64, _P]),
    "vq_adamw": (_I, [_P, _D, _D, _D, _D, _D, _I64, _P, _P, _P, _P]),
    "vq_timing_enable": (None, [_I]),
    "vq_timing_count": (_I, []),
    "vq_timing_get": (_I, [_I, ctypes.c_char_p, _I, ctypes.POINTER(_I), ctypes.POINTER(_I64),
                           ctypes.POINTER(_D), ctypes.POINTER(_D), ctypes.POINTER(_D)]),
}

_lib = None


def load(path=None):
    """Loads libvq.so; raises if it has not been built."""
    global _lib
    if _lib is not None and path is None:
        return _lib
    p = path or LIB_PATH
    if not os.path.exists(p):
        raise RuntimeError("libvq.so is not built (%s); run __graft_entry__.build() or "
                           "python hessian_weighted_vector_amd/build.py" % p)
    lib = ctypes.CDLL(p)
    for name, (res, args) in SIGNATURES.items():
        f = getattr(lib, name)
        f.restype = res
        f.argtypes = args
    if path is None:
        _lib = lib
    return lib


def _check(st):
    if st != VQ_OK:
        raise VQError(st, load().vq_last_error().decode())


def _ptr(t):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("tensor must be on the GPU")
    if not t.is_contiguous():
        raise ValueError("tensor must be contiguous")
    return t.data_ptr()


def _public_stream(device):
    return torch.cuda.current_stream(device).cuda_stream


# The current device's index and the raw handle of its current stream: torch's own entries
# make no Stream object (0.2 us against 1.5); a torch without them gives the same publicly.
_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", _public_stream)


def _stream():
    return _raw_stream(_device())


def _dtype(t, dt, name):
    if t is not None and t.dtype != dt:
        raise TypeError("%s must be %s, got %s" % (name, dt, t.dtype))


def workspace_bytes(M, N, d, K1, K2=0, nnz=0):
    return int(load().vq_workspace_bytes(M, N, d, K1, K2, nnz))


def workspace(M, N, d, K1, K2=0, nnz=0, device="cuda"):
    """A byte tensor large enough for every call with these sizes."""
    return torch.empty(max(workspace_bytes(M, N, d, K1, K2, nnz), 256), dtype=torch.uint8, device=device)


def nnz_of(M, N, p):
    """The library's salient count for an M x N matrix and fraction p."""
    n = int(load().vq_nnz(M, N, float(p)))
    if n < 0:
        raise VQError(VQ_ERR_INVALID, load().vq_last_error().decode())
    return n


def sparse_select(W, h, d, nnz, ws):
    _dtype(W, torch.float32, "W")
    M, N = W.shape
    dev = W.device
    row_ptr = torch.empty(M + 1, dtype=torch.int32, device=dev)
    col = torch.empty(max(nnz, 1), dtype=torch.int32, device=dev)
    val = torch.empty(max(nnz, 1), dtype=torch.float32, device=dev)
    mask = torch.empty(M * N // d, dtype=torch.uint8, device=dev)
    _check(load().vq_sparse_select(_ptr(W), _ptr(h), M, N, d, nnz, _ptr(row_ptr), _ptr(col), _ptr(val),
                                   _ptr(mask), _ptr(ws), ws.numel(), _stream()))
    return row_ptr, col[:nnz], val[:nnz], mask


def binorm(W, h, ws):
    M, N = W.shape
    Wp = torch.empty_like(W)
    r = torch.empty(M, dtype=torch.float32, device=W.device)
    c = torch.empty(N, dtype=torch.float32, device=W.device)
    hcol = torch.empty(N, dtype=torch.float32, device=W.device)
    rho = torch.empty(M, dtype=torch.float32, device=W.device)
    _check(load().vq_binorm(_ptr(W), _ptr(h), M, N, _ptr(Wp), _ptr(r), _ptr(c), _ptr(hcol), _ptr(rho),
                            _ptr(ws), ws.numel(), _stream()))
    return Wp, r, c, hcol, rho


def init(X, d, perm_host, K, ws):
    """perm_host: numpy int32 array (host)."""
    M, N = X.shape
    perm = np.ascontiguousarray(perm_host, dtype=np.int32)
    C = torch.empty((K, d), dtype=torch.float32, device=X.device)
    _check(load().vq_init(_ptr(X), M, N, d, perm.ctypes.data, K, _ptr(C), _ptr(ws), ws.numel(), _stream()))
    return C


def assign(X, hcol, rho, mask, d, C, ws, want_dist=False, idx=None, dist=None):
    _dtype(X, torch.float32, "X")
    _dtype(C, torch.float32, "C")
    _dtype(mask, torch.uint8, "mask")
    M, N = X.shape
    K = C.shape[0]
    n_sub = M * N // d
    if idx is None:
        idx = torch.empty(n_sub, dtype=torch.uint16, device=X.device)
    if want_dist and dist is None:
        dist = torch.empty(n_sub, dtype=torch.float32, device=X.device)
    _check(load().vq_assign(_ptr(X), _ptr(hcol), _ptr(rho), _ptr(mask), M, N, d, _ptr(C), K, _ptr(idx),
                            _ptr(dist) if want_dist else None, _ptr(ws), ws.numel(), _stream()))
    return (idx, dist) if want_dist else idx


def assign_exact_count(ws, n_sub, K):
    return int(load().vq_assign_exact_count(_ptr(ws), ws.numel(), n_sub, K, _stream()))


def assign_exact_list(ws, n_sub, K):
    """Sorted ids (numpy int32) of the sub-vectors the last assign re-searched exactly."""
    lib = load()
    n = int(lib.vq_assign_exact_list(_ptr(ws), ws.numel(), n_sub, K, None, 0, _stream()))
    if n < 0:
        raise VQError(VQ_ERR_INVALID, lib.vq_last_error().decode())
    out = np.zeros(max(n, 1), np.int32)
    m = int(lib.vq_assign_exact_list(_ptr(ws), ws.numel(), n_sub, K, out.ctypes.data, n, _stream()))
    if m != n:
        raise VQError(VQ_ERR_DEVICE, "exact-path list changed between reads")
    return np.sort(out[:n])


def update(X, hcol, rho, mask, d, idx, C, ws, want_counts=True, want_J=True):
    """In place on C; returns (counts, J tensor [1] float64)."""
    M, N = X.shape
    K = C.shape[0]
    counts = torch.empty(K, dtype=torch.int32, device=X.device) if want_counts else None
    J = torch.empty(1, dtype=torch.float64, device=X.device) if want_J else None
    _check(load().vq_update(_ptr(X), _ptr(hcol), _ptr(rho), _ptr(mask), M, N, d, _ptr(idx), K, _ptr(C),
                            _ptr(counts), _ptr(J), _ptr(ws), ws.numel(), _stream()))
    return counts, J


def objective(X, hcol, rho, mask, d, C, idx, ws):
    M, N = X.shape
    J = torch.empty(1, dtype=torch.float64, device=X.device)
    _check(load().vq_objective(_ptr(X), _ptr(hcol), _ptr(rho), _ptr(mask), M, N, d, _ptr(C), C.shape[0],
                               _ptr(idx), _ptr(J), _ptr(ws), ws.numel(), _stream()))
    return J


def residual(X, d, C, idx):
    M, N = X.shape
    R = torch.empty_like(X)
    _check(load().vq_residual(_ptr(X), M, N, d, _ptr(C), C.shape[0], _ptr(idx), _ptr(R), _stream()))
    return R


def reconstruct(M, N, d, C1, idx1, C2=None, idx2=None, rscale=None, cscale=None, row_ptr=None, col=None,
                val=None, out=None):
    W_hat = out if out is not None else torch.empty((M, N), dtype=torch.float32, device=C1.device)
    _check(load().vq_reconstruct(M, N, d, _ptr(C1), C1.shape[0], _ptr(idx1), _ptr(C2),
                                 0 if C2 is None else C2.shape[0], _ptr(idx2), _ptr(rscale), _ptr(cscale),
                                 _ptr(row_ptr), _ptr(col), _ptr(val), _ptr(W_hat), _stream()))
    return W_hat


def select_subvectors(W, h, d, n_sel, mask, ws):
    """OR every bit of the n_sel most salient sub-vectors into mask (in place)."""
    M, N = W.shape
    _check(load().vq_select_subvectors(_ptr(W), _ptr(h), M, N, d, int(n_sel), _ptr(mask), _ptr(ws), ws.numel(),
                                       _stream()))
    return mask


def select_residual(W, W_hat, h, d, n_sel, mask, ws):
    """OR the n_sel largest weighted residuals among clear positions into mask (in place)."""
    M, N = W.shape
    _check(load().vq_select_residual(_ptr(W), _ptr(W_hat), _ptr(h), M, N, d, int(n_sel), _ptr(mask), _ptr(ws),
                                     ws.numel(), _stream()))
    return mask


def mask_to_csr(W, mask, d, nnz_cap, ws):
    """(row_ptr, col, val) of the held positions; row_ptr[M] is the full count."""
    M, N = W.shape
    row_ptr = torch.empty(M + 1, dtype=torch.int32, device=W.device)
    col = torch.empty(max(int(nnz_cap), 1), dtype=torch.int32, device=W.device)
    val = torch.empty(max(int(nnz_cap), 1), dtype=torch.float32, device=W.device)
    _check(load().vq_mask_to_csr(_ptr(W), _ptr(mask), M, N, d, int(nnz_cap), _ptr(row_ptr), _ptr(col), _ptr(val),
                                 _ptr(ws), ws.numel(), _stream()))
    return row_ptr, col, val


def hessian_factor(H, damp=0.01, ws=None):
    """U [N, N] (float32, upper): U^T U = (H + damp mean(diag H) I)^-1."""
    N = H.shape[0]
    U = torch.empty_like(H)
    if ws is None:
        ws = torch.empty(max(int(load().vq_hessian_factor_workspace_bytes(N)), 256), dtype=torch.uint8,
                         device=H.device)
    _check(load().vq_hessian_factor(_ptr(H), N, float(damp), _ptr(U), _ptr(ws), ws.numel(), _stream()))
    return U


def vptq(W, U, V, C, B=128, want_E=False, ws=None):
    """Algorithm 1 (column sub-vectors of length V): returns idx [N, M/V], W_hat [M, N]
    and, with want_E, E [M, N]."""
    M, N = W.shape
    dev = W.device
    idx = torch.empty((N, M // V), dtype=torch.uint16, device=dev)
    W_hat = torch.empty_like(W)
    E = torch.empty_like(W) if want_E else None
    if ws is None:
        ws = torch.empty(max(int(load().vq_vptq_workspace_bytes(M, N, V)), 256), dtype=torch.uint8, device=dev)
    _check(load().vq_vptq(_ptr(W), _ptr(U), M, N, V, _ptr(C), C.shape[0], int(B), _ptr(idx), _ptr(W_hat),
                          _ptr(E), _ptr(ws), ws.numel(), _stream()))
    return idx, W_hat, E


def qgemv_workspace_bytes(M, N, d, B):
    return int(load().vq_qgemv_workspace_bytes(M, N, d, B))


def qgemv(M, N, d, C1, idx1, X, C2=None, idx2=None, rscale=None, cscale=None, row_ptr=None, col=None,
          val=None, out=None, ws=None):
    """Y = X W_hat^T from the compressed form (X [B x N] -> Y [B x M], float32)."""
    B = X.shape[0]
    Y = out if out is not None else torch.empty((B, M), dtype=torch.float32, device=X.device)
    need = qgemv_workspace_bytes(M, N, d, B)
    if ws is None and need > 0:
        ws = torch.empty(need, dtype=torch.uint8, device=X.device)
    _check(load().vq_qgemv(M, N, d, _ptr(C1), C1.shape[0], _ptr(idx1), _ptr(C2),
                           0 if C2 is None else C2.shape[0], _ptr(idx2), _ptr(rscale), _ptr(cscale),
                           _ptr(row_ptr), _ptr(col), _ptr(val), _ptr(X), B, _ptr(Y), _ptr(ws),
                           0 if ws is None else ws.numel(), _stream()))
    return Y


def grouped_params(M, N, d, K1, iters1, K2, iters2, outlier_frac, binorm, mask_outliers, n_out, d0, K0, iters0,
                   n_groups):
    return GroupedParams(FitParams(M, N, d, K1, iters1, K2, iters2, float(outlier_frac), int(bool(binorm)),
                                   int(bool(mask_outliers))), int(n_out), d0, K0, iters0, n_groups)


def grouped_sizes(params):
    """(workspace bytes, n_idx, n_codebook, n_J, n_perm1, n_perm2)."""
    v = [_I64(0) for _ in range(5)]
    ws = load().vq_grouped_sizes(ctypes.byref(params), *[ctypes.byref(x) for x in v])
    return (int(ws),) + tuple(int(x.value) for x in v)


def fit_grouped(W, h, params, perm1, perm2=None, ws=None):
    """The grouped fit; returns a dict of the outputs (device tensors; J and bpw on the host)."""
    M, N = W.shape
    dev = W.device
    wsb, n_idx, n_cb, n_J, n_p1, n_p2 = grouped_sizes(params)
    if wsb == 0:
        raise ValueError("the column groups do not split these sizes")
    nnz = nnz_of(M, N, params.fit.outlier_frac)
    o = {"cols": torch.empty(N, dtype=torch.int32, device=dev),
         "idx": torch.empty(max(n_idx, 1), dtype=torch.uint16, device=dev),
         "codebooks": torch.empty(max(n_cb, 1), dtype=torch.float32, device=dev),
         "row_ptr": torch.empty(M + 1, dtype=torch.int32, device=dev),
         "col": torch.empty(max(nnz, 1), dtype=torch.int32, device=dev),
         "val": torch.empty(max(nnz, 1), dtype=torch.float32, device=dev),
         "mask": torch.empty(M * N // params.fit.d, dtype=torch.uint8, device=dev),
         "W_hat": torch.empty_like(W)}
    J = np.zeros(max(n_J, 1), np.float64)
    bpw = np.zeros(1, np.float64)
    p1 = np.ascontiguousarray(perm1, dtype=np.int32)
    p2 = None if perm2 is None else np.ascontiguousarray(perm2, dtype=np.int32)
    if ws is None:
        ws = torch.empty(wsb, dtype=torch.uint8, device=dev)
    inputs = GroupedInputs(_ptr(W), _ptr(h), p1.ctypes.data, None if p2 is None else p2.ctypes.data)
    outputs = GroupedOutputs(_ptr(o["cols"]), _ptr(o["idx"]), _ptr(o["codebooks"]), _ptr(o["row_ptr"]),
                             _ptr(o["col"]), _ptr(o["val"]), _ptr(o["mask"]), _ptr(o["W_hat"]), J.ctypes.data,
                             bpw.ctypes.data)
    _check(load().vq_fit_grouped(ctypes.byref(params), ctypes.byref(inputs), ctypes.byref(outputs), _ptr(ws),
                                 ws.numel(), _stream()))
    o["col"] = o["col"][:nnz]
    o["val"] = o["val"][:nnz]
    o["J"] = J[:n_J]
    o["bpw"] = float(bpw[0])
    return o


def timing_enable(on=True):
    load().vq_timing_enable(int(bool(on)))


def timing_records():
    """[(name, K, launches, total_ms, min_ms, max_ms)] of the recorded step timings."""
    lib = load()
    out = []
    for i in range(lib.vq_timing_count()):
        buf = ctypes.create_string_buffer(64)
        K, n = _I(0), _I64(0)
        tot, mn, mx = _D(0), _D(0), _D(0)
        if lib.vq_timing_get(i, buf, 64, ctypes.byref(K), ctypes.byref(n), ctypes.byref(tot),
                             ctypes.byref(mn), ctypes.byref(mx)) == 0:
            out.append((buf.value.decode(), K.value, n.value, tot.value, mn.value, mx.value))
    return out


def bits_per_weight(M, N, d, K1, K2, nnz, cb_bits=32, binorm=False):
    return float(load().vq_bits_per_weight(M, N, d, K1, K2, nnz, cb_bits, int(bool(binorm))))


def fit(W, h, d, K1, iters1, K2=0, iters2=0, outlier_frac=0.0, binorm=False, mask_outliers=True,
        perm1=None, perm2=None, C1_init=None, C2_init=None, ws=None):
    """The whole pipeline on the GPU; returns a dict of device tensors + host J/bpw."""
    M, N = W.shape
    dev = W.device
    n_sub = M * N // d
    nnz = nnz_of(M, N, outlier_frac)
    if ws is None:
        ws = workspace(M, N, d, K1, K2, nnz, dev)
    o = {
        "idx1": torch.empty(n_sub, dtype=torch.uint16, device=dev),
        "C1": torch.empty((K1, d), dtype=torch.float32, device=dev),
        "idx2": torch.empty(n_sub if K2 > 0 else 1, dtype=torch.uint16, device=dev),
        "C2": torch.empty((max(K2, 1), d), dtype=torch.float32, device=dev),
        "row_ptr": torch.empty(M + 1, dtype=torch.int32, device=dev),
        "col": torch.empty(max(nnz, 1), dtype=torch.int32, device=dev),
        "val": torch.empty(max(nnz, 1), dtype=torch.float32, device=dev),
        "mask": torch.empty(n_sub, dtype=torch.uint8, device=dev),
        "W_hat": torch.empty((M, N), dtype=torch.float32, device=dev),
    }
    if binorm:
        o.update({"Wp": torch.empty_like(W), "rscale": torch.empty(M, dtype=torch.float32, device=dev),
                  "cscale": torch.empty(N, dtype=torch.float32, device=dev),
                  "hcol": torch.empty(N, dtype=torch.float32, device=dev),
                  "rho": torch.empty(M, dtype=torch.float32, device=dev)})
    nJ = iters1 + 1 + (iters2 + 1 if K2 > 0 else 0)
    J = np.zeros(nJ, np.float64)
    bpw = np.zeros(1, np.float64)
    empty = np.zeros(max(iters1 + (iters2 if K2 > 0 else 0), 1), np.int64)
    p1 = None if perm1 is None else np.ascontiguousarray(perm1, dtype=np.int32)
    p2 = None if perm2 is None else np.ascontiguousarray(perm2, dtype=np.int32)
    params = FitParams(M, N, d, K1, iters1, K2, iters2, float(outlier_frac), int(bool(binorm)),
                       int(bool(mask_outliers)))
    inputs = FitInputs(_ptr(W), _ptr(h), None if p1 is None else p1.ctypes.data,
                       None if p2 is None else p2.ctypes.data, _ptr(C1_init), _ptr(C2_init))
    g = lambda k: _ptr(o[k]) if k in o else None  # noqa: E731
    outputs = FitOutputs(g("idx1"), g("C1"), g("idx2"), g("C2"), g("row_ptr"), g("col"), g("val"), g("mask"),
                         g("Wp"), g("rscale"), g("cscale"), g("hcol"), g("rho"), g("W_hat"),
                         J.ctypes.data, bpw.ctypes.data, empty.ctypes.data)
    _check(load().vq_fit(ctypes.byref(params), ctypes.byref(inputs), ctypes.byref(outputs), _ptr(ws),
                         ws.numel(), _stream()))
    o["col"] = o["col"][:nnz]
    o["val"] = o["val"][:nnz]
    o["J"] = J
    o["empty"] = empty[:iters1 + (iters2 if K2 > 0 else 0)]
    o["bpw"] = float(bpw[0])
    o["nnz"] = nnz
    if K2 == 0:
        o["C2"] = None
        o["idx2"] = None
    return o


# ---- dense feed-forward calls ------------------------------------------------
# Outputs carry no autograd graph, also where an input requires gradients: the backward
# passes are calls of their own (linear_backward, gated_backward).

ACTIVATIONS = {"none": 0, "relu": 1, "silu": 2, "gelu": 3, "gelu_tanh": 4, "sigmoid": 5}
_DTYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}


def _act(act):
    try:
        return ACTIVATIONS[act]
    except KeyError:
        raise ValueError("act must be one of %s, got %r" % (", ".join(ACTIVATIONS), act)) from None


def _half(t, name):
    """The library's code of a 16-bit tensor's type."""
    code = _DTYPES.get(t.dtype)
    if code is None or code > 1:
        raise TypeError("%s must be torch.bfloat16 or torch.float16, got %s" % (name, t.dtype))
    return code


def _home(X, name="X"):
    """The index of the current GPU, where the launches go; X has to be on it."""
    dev = X.get_device()
    if dev < 0 or dev != _device():
        _elsewhere(X, name)
    return dev


def _elsewhere(t, name):
    if not t.is_cuda:
        raise ValueError("%s must be on the GPU" % name)
    raise ValueError("%s must be on the current GPU %d, is on %d" % (name, _device(), t.get_device()))


def _matrix(t, rows, cols, dtype, dev, name):
    """(pointer, leading dimension) of a [rows x cols] tensor on GPU dev with unit column stride; None passes."""
    if t is None:
        return None, 0
    if t.dtype != dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if t.get_device() != dev:
        _elsewhere(t, name)
    if t.shape != (rows, cols):
        raise ValueError("%s must be [%d x %d], got %s" % (name, rows, cols, list(t.shape)))
    s0, s1 = t.stride()
    if s1 != 1 and cols > 1:
        raise ValueError("%s must have contiguous rows" % name)
    if s0 < cols:
        if rows > 1:
            raise ValueError("%s must have rows that do not overlap" % name)
        s0 = cols
    return t.data_ptr(), s0


def _output(out, X, rows, cols, dev):
    """(tensor, pointer, leading dimension) of a caller's output or of a new one of X's type."""
    if out is None:
        out = X.new_empty((rows, cols))
        return out, out.data_ptr(), cols
    return (out,) + _matrix(out, rows, cols, X.dtype, dev, "out")


def _vector(t, n, dtype, dev, name):
    if t is None:
        return None
    if t.dtype != dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if t.dim() != 1 or t.shape[0] != n:
        raise ValueError("%s must be [%d], got %s" % (name, n, list(t.shape)))
    if t.get_device() != dev:
        _elsewhere(t, name)
    return _ptr(t)


def _scratch(need, ws, X, dev):
    """(pointer, bytes, tensor) of a workspace of at least `need` bytes."""
    if ws is None:
        if need == 0:
            return None, 0, None
        ws = torch.empty(need, dtype=torch.uint8, device=X.device)
    elif ws.get_device() != dev:
        _elsewhere(ws, "ws")
    return _ptr(ws), ws.numel(), ws


# Workspace sizes by sizes, leading dimensions and alignments (an address stands for its last four bits).
@functools.lru_cache(maxsize=4096)
def _linear_need(T, M, N, x, ldx, w, ldw):
    return load().vq_linear_workspace_bytes(T, M, N, x, ldx, w, ldw)


@functools.lru_cache(maxsize=4096)
def _gated_need(T, M, N, x, ldx, wg, wu, ldw):
    return load().vq_gated_workspace_bytes(T, M, N, x, ldx, wg, wu, ldw)


@functools.lru_cache(maxsize=4096)
def _linear_backward_need(*args):
    return load().vq_linear_backward_workspace_bytes(*args)


@functools.lru_cache(maxsize=4096)
def _gated_backward_need(*args):
    return load().vq_gated_backward_workspace_bytes(*args)


@functools.lru_cache(maxsize=4096)
def _qlinear_need(M, N, d, T):
    return load().vq_qlinear_workspace_bytes(M, N, d, T)


@functools.lru_cache(maxsize=4096)
def _qgated_need(M, N, d, T):
    return load().vq_qgated_workspace_bytes(M, N, d, T)


def _dims(X, W):
    if X.dim() != 2 or W.dim() != 2:
        raise ValueError("X and W must be matrices")
    return X.shape[0], W.shape[0], W.shape[1]


def linear(X, W, bias=None, residual=None, act="none", want_pre=False, out=None, ws=None):
    """Y = act(X W^T + bias) + residual: X [T, N], W [M, N], bfloat16 or float16 (one type).

    With want_pre returns (Y, Z), Z = X W^T + bias (linear_backward's `pre`).
    Rows may be strided.  `out` may be the residual itself.
    """
    T, M, N = _dims(X, W)
    dt, a, dev = _half(X, "X"), _act(act), _home(X)
    x, ldx = _matrix(X, T, N, X.dtype, dev, "X")
    w, ldw = _matrix(W, M, N, X.dtype, dev, "W")
    b = _vector(bias, M, X.dtype, dev, "bias")
    r, ldr = _matrix(residual, T, M, X.dtype, dev, "residual")
    Y, y, ldy = _output(out, X, T, M, dev)
    Z, z, ldz = _output(None, X, T, M, dev) if want_pre else (None, None, 0)
    lib = load()
    p, n, ws = _scratch(_linear_need(T, M, N, x & 15, ldx, w & 15, ldw), ws, X, dev)
    _check(lib.vq_linear(T, M, N, dt, a, x, ldx, w, ldw, b, r, ldr, y, ldy, z, ldz, p, n, _stream()))
    return (Y, Z) if want_pre else Y


def linear_backward(dY, X, W, pre=None, act="none", want_dx=True, want_dw=True, want_db=False, ws=None):
    """(dX, dW, db) of linear for the incoming gradient dY [T, M]; None where not wanted.

    `pre` is the Z that linear returned (needed unless act is "none").  The
    residual's gradient is dY itself.
    """
    T, M, N = _dims(X, W)
    dt, a = _half(X, "X"), _act(act)
    if a != 0 and pre is None:
        raise ValueError("pre is needed for the activation's gradient")
    dev = _home(X)
    g, ldg = _matrix(dY, T, M, X.dtype, dev, "dY")
    x, ldx = _matrix(X, T, N, X.dtype, dev, "X")
    w, ldw = _matrix(W, M, N, X.dtype, dev, "W")
    z, ldz = _matrix(pre, T, M, X.dtype, dev, "pre")
    dX = X.new_empty((T, N)) if want_dx else None
    dW = X.new_empty((M, N)) if want_dw else None
    db = X.new_empty(M) if want_db else None
    lib = load()
    p, n, ws = _scratch(_linear_backward_need(T, M, N, a, g & 15, ldg, x & 15, ldx, w & 15, ldw, want_dx, want_dw, want_db),
                        ws, X, dev)
    _check(lib.vq_linear_backward(T, M, N, dt, a, g, ldg, x, ldx, w, ldw, z, ldz, _ptr(dX), N, _ptr(dW), N, _ptr(db),
                                  p, n, _stream()))
    return dX, dW, db


def gated(X, W_gate, W_up, bias_gate=None, bias_up=None, act="silu", want_pre=False, out=None, ws=None):
    """H = act(G) * U, G = X W_gate^T + bias_gate, U = X W_up^T + bias_up, in one kernel.

    X [T, N], W_gate and W_up [M, N], bfloat16 or float16.  With want_pre
    returns (H, G, U), which gated_backward takes.
    """
    T, M, N = _dims(X, W_gate)
    dt, a, dev = _half(X, "X"), _act(act), _home(X)
    x, ldx = _matrix(X, T, N, X.dtype, dev, "X")
    wg, ldw = _matrix(W_gate, M, N, X.dtype, dev, "W_gate")
    wu, ldu = _matrix(W_up, M, N, X.dtype, dev, "W_up")
    if ldw != ldu:
        raise ValueError("W_gate and W_up must have the same row stride")
    bg = _vector(bias_gate, M, X.dtype, dev, "bias_gate")
    bu = _vector(bias_up, M, X.dtype, dev, "bias_up")
    H, h, ldh = _output(out, X, T, M, dev)
    G = X.new_empty((T, M)) if want_pre else None
    U = X.new_empty((T, M)) if want_pre else None
    lib = load()
    p, n, ws = _scratch(_gated_need(T, M, N, x & 15, ldx, wg & 15, wu & 15, ldw), ws, X, dev)
    _check(lib.vq_gated(T, M, N, dt, a, x, ldx, wg, wu, ldw, bg, bu, h, ldh, _ptr(G), _ptr(U), M, p, n, _stream()))
    return (H, G, U) if want_pre else H


def gated_backward(dH, X, W_gate, W_up, G, U, act="silu", want_dx=True, want_dw=True, want_db=False, ws=None):
    """(dX, dW_gate, dW_up, db_gate, db_up) of gated; None where not wanted."""
    T, M, N = _dims(X, W_gate)
    dt, a, dev = _half(X, "X"), _act(act), _home(X)
    dh, lddh = _matrix(dH, T, M, X.dtype, dev, "dH")
    x, ldx = _matrix(X, T, N, X.dtype, dev, "X")
    wg, ldw = _matrix(W_gate, M, N, X.dtype, dev, "W_gate")
    wu, ldu = _matrix(W_up, M, N, X.dtype, dev, "W_up")
    g, ldz = _matrix(G, T, M, X.dtype, dev, "G")
    u, ldz2 = _matrix(U, T, M, X.dtype, dev, "U")
    if ldw != ldu or ldz != ldz2:
        raise ValueError("W_gate and W_up, and G and U, must have the same row stride")

    def new(on, *shape):
        return X.new_empty(shape) if on else None

    dX, dWg, dWu = new(want_dx, T, N), new(want_dw, M, N), new(want_dw, M, N)
    dbg, dbu = new(want_db, M), new(want_db, M)
    lib = load()
    p, n, ws = _scratch(_gated_backward_need(T, M, N, a, dh & 15, lddh, x & 15, ldx, wg & 15, wu & 15, ldw, want_dx, want_dw,
                                             want_db), ws, X, dev)
    _check(lib.vq_gated_backward(T, M, N, dt, a, dh, lddh, x, ldx, wg, wu, ldw, g, u, ldz, _ptr(dX), N, _ptr(dWg),
                                 _ptr(dWu), N, _ptr(dbg), _ptr(dbu), p, n, _stream()))
    return dX, dWg, dWu, dbg, dbu


# ---- feed-forward calls on compressed matrices --------------------------------

class QMatrix:
    """A compressed matrix as a serving program keeps it.

    Takes the arrays of a fit (codebooks, indices, scales, sparse correction)
    and makes the sparse part's differences to the decoded weights once, on the
    current stream.  Holds references to the arrays; call refresh() after
    changing any of them in place.
    """

    def __init__(self, M, N, d, C1, idx1, C2=None, idx2=None, rscale=None, cscale=None, row_ptr=None, col=None, val=None):
        n_sub = M * N // d if d else 0
        for t, dt, n, name in ((C1, torch.float32, None, "C1"), (C2, torch.float32, None, "C2"),
                               (idx1, torch.uint16, n_sub, "idx1"), (idx2, torch.uint16, n_sub, "idx2"),
                               (rscale, torch.float32, M, "rscale"), (cscale, torch.float32, N, "cscale"),
                               (row_ptr, torch.int32, M + 1, "row_ptr"), (col, torch.int32, None, "col"),
                               (val, torch.float32, None, "val")):
            _dtype(t, dt, name)
            if t is not None and n is not None and t.numel() != n:
                raise ValueError("%s must have %d elements, got %d" % (name, n, t.numel()))
        for t, name in ((C1, "C1"), (C2, "C2")):
            if t is not None and (t.dim() != 2 or t.shape[1] != d):
                raise ValueError("%s must be [K x %d], got %s" % (name, d, list(t.shape)))
        if (C2 is None) != (idx2 is None):
            raise ValueError("C2 and idx2 come together")
        for t, name in ((C1, "C1"), (idx1, "idx1"), (C2, "C2"), (idx2, "idx2"), (rscale, "rscale"), (cscale, "cscale"),
                        (row_ptr, "row_ptr"), (col, "col"), (val, "val")):
            if t is not None:
                _home(t, name)
        sparse = row_ptr is not None and col is not None and col.numel() > 0
        if sparse and (val is None or val.numel() != col.numel()):
            raise ValueError("val must have as many elements as col")
        self.M, self.N, self.d = int(M), int(N), int(d)
        self.val = val if sparse else None
        self.delta = torch.empty_like(val) if sparse else None
        self._keep = (C1, idx1, C2, idx2, rscale, cscale, row_ptr, col)
        self._struct = QMatrixStruct(M, N, d, C1.shape[0], 0 if C2 is None else C2.shape[0], _ptr(C1), _ptr(idx1),
                                     _ptr(C2), _ptr(idx2), _ptr(rscale), _ptr(cscale), _ptr(row_ptr) if sparse else None,
                                     _ptr(col) if sparse else None, _ptr(self.delta))
        self._ref = ctypes.addressof(self._struct)
        self.device = C1.device
        self.index = C1.get_device()
        self.refresh()

    @classmethod
    def from_fit(cls, out, M, N, d):
        """From the dict that fit returns."""
        return cls(M, N, d, out["C1"], out["idx1"], out["C2"], out["idx2"], out.get("rscale"), out.get("cscale"),
                   out["row_ptr"], out["col"], out["val"])

    def refresh(self):
        """Makes the sparse differences again (current stream)."""
        if self.index != _device():
            _elsewhere(self._keep[0], "the matrix")
        if self.delta is not None:
            _check(load().vq_sparse_delta(self._ref, _ptr(self.val), _ptr(self.delta), _stream()))


def _any_dtype(t, name):
    code = _DTYPES.get(t.dtype)
    if code is None:
        raise TypeError("%s must be torch.bfloat16, torch.float16 or torch.float32, got %s" % (name, t.dtype))
    return code


def qlinear(Q, X, bias=None, residual=None, act="none", out=None, ws=None):
    """Y = act(X W^T + bias) + residual with W = the QMatrix Q, never decoded to memory.

    X [T, N] of bfloat16, float16 or float32; the other tensors have its type.  For a few
    tokens: every 32 read the matrix anew.
    """
    if X.dim() != 2:
        raise ValueError("X must be a matrix")
    T, M, N = X.shape[0], Q.M, Q.N
    dt, a, dev = _any_dtype(X, "X"), _act(act), _home(X)
    if Q.index != dev:
        _elsewhere(Q._keep[0], "Q")
    x, ldx = _matrix(X, T, N, X.dtype, dev, "X")
    b = _vector(bias, M, X.dtype, dev, "bias")
    r, ldr = _matrix(residual, T, M, X.dtype, dev, "residual")
    Y, y, ldy = _output(out, X, T, M, dev)
    lib = load()
    p, n, ws = _scratch(_qlinear_need(M, N, Q.d, T), ws, X, dev)
    _check(lib.vq_qlinear(Q._ref, T, dt, a, x, ldx, b, r, ldr, y, ldy, p, n, _stream()))
    return Y


def qgated(Q_gate, Q_up, X, bias_gate=None, bias_up=None, act="silu", out=None, ws=None):
    """H = act(X Wg^T + bias_gate) * (X Wu^T + bias_up) with both compressed matrices in one launch (tokens as in qlinear)."""
    if X.dim() != 2:
        raise ValueError("X must be a matrix")
    T, M, N = X.shape[0], Q_gate.M, Q_gate.N
    dt, a, dev = _any_dtype(X, "X"), _act(act), _home(X)
    if Q_gate.index != dev:
        _elsewhere(Q_gate._keep[0], "Q_gate")
    if Q_up.index != dev:
        _elsewhere(Q_up._keep[0], "Q_up")
    x, ldx = _matrix(X, T, N, X.dtype, dev, "X")
    bg = _vector(bias_gate, M, X.dtype, dev, "bias_gate")
    bu = _vector(bias_up, M, X.dtype, dev, "bias_up")
    H, h, ldh = _output(out, X, T, M, dev)
    lib = load()
    p, n, ws = _scratch(_qgated_need(M, N, Q_gate.d, T), ws, X, dev)
    _check(lib.vq_qgated(Q_gate._ref, Q_up._ref, T, dt, a, x, ldx, bg, bu, h, ldh, p, n, _stream()))
    return H


# ---- feed-forward calls in 8-bit integers --------------------------------------------

def quantize_rows(X):
    """(q, scale): int8 [T, N] and float32 [T] with X[t, j] near scale[t] q[t, j], q the integer nearest to 127 X[t, j] / max |X[t]|.

    X [T, N] is bfloat16, float16 or float32; a row that is not finite has a NaN scale.  q's
    rows begin every multiple of 64 bytes, as Int8Matrix takes them in place.
    """
    if X.dim() != 2:
        raise ValueError("X must be a matrix")
    T, N = X.shape
    dt, dev = _any_dtype(X, "X"), _home(X)
    x, ldx = _matrix(X, T, N, X.dtype, dev, "X")
    ldq = -(-N // 64) * 64
    q = torch.empty((T, ldq), dtype=torch.int8, device=X.device)
    scale = torch.empty(T, dtype=torch.float32, device=X.device)
    _check(load().vq_quantize_rows(T, N, dt, x, ldx, q.data_ptr(), ldq, scale.data_ptr(), _stream()))
    return q[:, :N], scale


class Int8Matrix:
    """A matrix in 8-bit codes with a scale a row: W[i, j] = scale[i] q[i, j].

    q int8 [M, N], scale float32 [M].  q is kept in place where its rows are laid out as the
    kernels read them (16-byte aligned, every multiple of 64 bytes, readable to the next one),
    else copied once on the current stream.
    """

    def __init__(self, q, scale):
        if q.dim() != 2 or q.dtype != torch.int8:
            raise TypeError("q must be an int8 matrix")
        M, N = q.shape
        self.index = _home(q, "q")
        _vector(scale, M, torch.float32, self.index, "scale")
        ld = q.stride(0) if M > 1 else -(-N // 64) * 64
        end = q.storage_offset() + (M - 1) * ld + -(-N // 64) * 64
        if (N > 1 and q.stride(1) != 1) or ld % 64 or ld < N or q.data_ptr() % 16 or end > q.untyped_storage().nbytes():
            ld = -(-N // 64) * 64
            copy = torch.empty((M, ld), dtype=torch.int8, device=q.device)
            copy[:, :N].copy_(q)
            q = copy[:, :N]
        self.M, self.N, self.q, self.scale = M, N, q, scale
        self._struct = I8MatrixStruct(M, N, q.data_ptr(), ld, scale.data_ptr())
        self._ref = ctypes.addressof(self._struct)

    def compact(self):
        """The matrix with its codes' rows as near as they can be (each begins at the next multiple of 64 bytes): itself, or a copy."""
        ld = -(-self.N // 64) * 64
        if self._struct.ldq == ld:
            return self
        copy = torch.empty((self.M, ld), dtype=torch.int8, device=self.q.device)
        copy[:, :self.N].copy_(self.q)
        return type(self)(copy[:, :self.N], self.scale)

    @classmethod
    def from_dense(cls, W):
        """From a dense matrix (bfloat16, float16 or float32), its rows brought to 8 bits."""
        return cls(*quantize_rows(W))


@functools.lru_cache(maxsize=4096)
def _linear_i8_need(M, N, T):
    return load().vq_linear_i8_workspace_bytes(M, N, T)


@functools.lru_cache(maxsize=4096)
def _gated_i8_need(M, N, T):
    return load().vq_gated_i8_workspace_bytes(M, N, T)


def linear_i8(Q, X, bias=None, residual=None, act="none", out=None, ws=None):
    """Y = act(X W^T + bias) + residual with W = the Int8Matrix Q and X brought to 8 bits, a scale a token.

    X [T, N] is bfloat16 or float16; the other tensors have its type.  `out` may be the residual itself.
    """
    if X.dim() != 2:
        raise ValueError("X must be a matrix")
    T, M, N = X.shape[0], Q.M, Q.N
    dt, a, dev = _half(X, "X"), _act(act), _home(X)
    if Q.index != dev:
        _elsewhere(Q.q, "Q")
    x, ldx = _matrix(X, T, N, X.dtype, dev, "X")
    b = _vector(bias, M, X.dtype, dev, "bias")
    r, ldr = _matrix(residual, T, M, X.dtype, dev, "residual")
    Y, y, ldy = _output(out, X, T, M, dev)
    lib = load()
    p, n, ws = _scratch(_linear_i8_need(M, N, T), ws, X, dev)
    _check(lib.vq_linear_i8(Q._ref, T, dt, a, x, ldx, b, r, ldr, y, ldy, p, n, _stream()))
    return Y


def gated_i8(Q_gate, Q_up, X, bias_gate=None, bias_up=None, act="silu", out=None, ws=None):
    """H = act(X Wg^T + bias_gate) * (X Wu^T + bias_up) with two Int8Matrix of one shape in one launch (tokens as in linear_i8).

    Their codes' rows are equally far apart: with one kept in place in wider rows, take compact() of both.
    """
    if X.dim() != 2:
        raise ValueError("X must be a matrix")
    T, M, N = X.shape[0], Q_gate.M, Q_gate.N
    dt, a, dev = _half(X, "X"), _act(act), _home(X)
    if Q_gate.index != dev:
        _elsewhere(Q_gate.q, "Q_gate")
    if Q_up.index != dev:
        _elsewhere(Q_up.q, "Q_up")
    if Q_gate._struct.ldq != Q_up._struct.ldq and (Q_up.M, Q_up.N) == (M, N):
        raise ValueError("Q_gate and Q_up must have rows that are equally far apart: take compact() of both")
    x, ldx = _matrix(X, T, N, X.dtype, dev, "X")
    bg = _vector(bias_gate, M, X.dtype, dev, "bias_gate")
    bu = _vector(bias_up, M, X.dtype, dev, "bias_up")
    H, h, ldh = _output(out, X, T, M, dev)
    lib = load()
    p, n, ws = _scratch(_gated_i8_need(M, N, T), ws, X, dev)
    _check(lib.vq_gated_i8(Q_gate._ref, Q_up._ref, T, dt, a, x, ldx, bg, bu, h, ldh, p, n, _stream()))
    return H


# ---- the loss over a vocabulary ---------------------------------------------------

@functools.lru_cache(maxsize=4096)
def _cross_entropy_need(T, V, N, w, ldw):
    return load().vq_cross_entropy_workspace_bytes(T, V, N, w, ldw)


@functools.lru_cache(maxsize=4096)
def _cross_entropy_backward_need(*args):
    return load().vq_cross_entropy_backward_workspace_bytes(*args)


def cross_entropy(X, W, labels, ignore_index=-100, ws=None):
    """(loss, lse), float32 [T] each: loss = lse - z[label], lse = log sum exp z, z = X W^T never kept.

    X [T, N] and W [V, N] are bfloat16 or float16 (one type, rows may be strided), labels int64
    [T].  Tokens whose label is ignore_index take no part: loss and lse are 0 there, whatever
    X holds.  Another label outside [0, V) gives a NaN loss.  The reduction is the caller's:
    loss.sum() / n, with dloss = 1 / n for cross_entropy_backward.
    """
    T, V, N = _dims(X, W)
    dt, dev = _half(X, "X"), _home(X)
    x, ldx = _matrix(X, T, N, X.dtype, dev, "X")
    w, ldw = _matrix(W, V, N, X.dtype, dev, "W")
    lab = _vector(labels, T, torch.int64, dev, "labels")
    loss, lse = (torch.empty(T, dtype=torch.float32, device=X.device) for _ in range(2))
    lib = load()
    p, n, ws = _scratch(_cross_entropy_need(T, V, N, w & 15, ldw), ws, X, dev)
    _check(lib.vq_cross_entropy(T, V, N, dt, x, ldx, w, ldw, lab, ignore_index, loss.data_ptr(), lse.data_ptr(), p, n, _stream()))
    return loss, lse


def cross_entropy_backward(dloss, X, W, labels, lse, ignore_index=-100, want_dx=True, want_dw=True, ws=None):
    """(dX, dW) of sum(dloss * loss), dloss float32 [T], for the lse that cross_entropy returned; None where not wanted."""
    T, V, N = _dims(X, W)
    dt, dev = _half(X, "X"), _home(X)
    x, ldx = _matrix(X, T, N, X.dtype, dev, "X")
    w, ldw = _matrix(W, V, N, X.dtype, dev, "W")
    g = _vector(dloss, T, torch.float32, dev, "dloss")
    lab = _vector(labels, T, torch.int64, dev, "labels")
    ls = _vector(lse, T, torch.float32, dev, "lse")
    dX = X.new_empty((T, N)) if want_dx else None
    dW = X.new_empty((V, N)) if want_dw else None
    lib = load()
    p, n, ws = _scratch(_cross_entropy_backward_need(T, V, N, w & 15, ldw, want_dx, want_dw), ws, X, dev)
    _check(lib.vq_cross_entropy_backward(T, V, N, dt, g, x, ldx, w, ldw, lab, ignore_index, ls, _ptr(dX), N, _ptr(dW), N, p, n,
                                         _stream()))
    return dX, dW


# ---- the optimizer's step -------------------------------------------------------

def _free_plan(plan):
    load().vq_adamw_plan_free(ctypes.addressof(plan))


class AdamW:
    """AdamW over many tensors in one launch, in place.

        m = beta1 m + (1 - beta1) g,  v = beta2 v + (1 - beta2) g^2,  g = grad_scale * grad,
        p = (1 - lr wd) p - lr / (1 - beta1^t) * m / (sqrt(v) / sqrt(1 - beta2^t) + eps)

    params: contiguous tensors of one type (bfloat16, float16 or float32); grads: of the same
    sizes and of one type, kept by the caller and filled before each step, or given to step();
    they share no memory with what a step writes.
    masters: float32 tensors that hold the values of 16-bit params.  state_bits 8 keeps the
    moments as float8_e4m3fn codes of m and sqrt(v) with a float32 scale for each 256
    elements.  `state` (a dict of lists m, v and, in 8 bits, m_scale, v_scale, as the
    attribute of that name holds them) and `steps` continue an earlier run; `state` is used
    in place.  capturable keeps the step's number (`steps`, int64) and the learning rate
    (`lr`, float32) on the GPU: a captured step() replays as consecutive steps, with the
    gradients that it was given when captured, or without any with those of the last step before
    each replay (captured after a step that was given its own: with the last ones given outside of
    a graph until then).
    Outside of a graph step() without gradients takes the last ones given outside of one.
    The first gradients of a type are given outside of a capture.  Those of captured steps are
    kept until release().
    """

    BLOCK = 256

    def __init__(self, params, grads=None, masters=None, lr=1e-3, betas=(0.9, 0.999), eps=1e-8, weight_decay=0.01,
                 state_bits=32, state=None, steps=0, capturable=False):
        self.params, self.masters = list(params), None if masters is None else list(masters)
        if not self.params:
            raise ValueError("params must not be empty")
        if state_bits not in (8, 32):
            raise ValueError("state_bits must be 8 or 32, got %r" % (state_bits,))
        self.index = _home(self.params[0], "params[0]")
        self.dtype = _any_dtype(self.params[0], "params[0]")
        self._same(self.params, self.params[0].dtype, "params")
        if self.masters is not None:
            if self.dtype == 2:
                raise ValueError("float32 params have no masters")
            self._same(self.masters, torch.float32, "masters")
        self.betas, self.eps, self.weight_decay = (float(betas[0]), float(betas[1])), float(eps), float(weight_decay)
        self.state_bits = state_bits
        dev = self.params[0].device
        if state is None:
            state = self._new_state(dev)
        self.state = {k: None if state.get(k) is None else list(state[k]) for k in ("m", "v", "m_scale", "v_scale")}
        kind = torch.float32 if state_bits == 32 else torch.float8_e4m3fn
        for k in ("m", "v"):
            self._same(self.state[k], kind, "state[%r]" % k)
        for k in ("m_scale", "v_scale"):
            if state_bits == 8:
                self._same(self.state[k], torch.float32, "state[%r]" % k, blocks=True)
            elif self.state[k] is not None:
                raise ValueError("32-bit moments have no scales")
        self.capturable = bool(capturable)
        if capturable:
            self.steps = torch.full((1,), int(steps), dtype=torch.int64, device=dev)
            self.lr = torch.full((1,), float(lr), dtype=torch.float32, device=dev)
        else:
            self.steps, self.lr = int(steps), float(lr)
        self.grads = None
        self._tables = {}                                     # by the gradients' type: plan, table, its stream, gradients
        self._captured = []                                   # gradients that graphs put into the tables
        if grads is not None:
            self._bind(grads)

    def _new_state(self, dev):
        """Zero moments: one buffer each, every tensor from a block's border on."""
        starts, at = [], 0
        for p in self.params:
            starts.append(at)
            at += -(-p.numel() // self.BLOCK)
        kind = torch.float32 if self.state_bits == 32 else torch.uint8
        out = {}
        for k in ("m", "v"):
            flat = torch.zeros(at * self.BLOCK, dtype=kind, device=dev)
            flat = flat if self.state_bits == 32 else flat.view(torch.float8_e4m3fn)
            out[k] = [flat[s * self.BLOCK:s * self.BLOCK + p.numel()].view(p.shape) for s, p in zip(starts, self.params)]
            if self.state_bits == 8:
                scale = torch.zeros(at, dtype=torch.float32, device=dev)
                out[k + "_scale"] = [scale[s:s - (-p.numel() // self.BLOCK)] for s, p in zip(starts, self.params)]
        return out

    def _same(self, ts, dtype, name, blocks=False):
        """Checks a list against params: type, sizes, device, contiguity."""
        if ts is None or len(ts) != len(self.params):
            raise ValueError("%s must have %d tensors" % (name, len(self.params)))
        for i, (t, p) in enumerate(zip(ts, self.params)):
            n = -(-p.numel() // self.BLOCK) if blocks else p.numel()
            if t.dtype != dtype:
                raise TypeError("%s[%d] must be %s, got %s" % (name, i, dtype, t.dtype))
            if t.get_device() != self.index:
                _elsewhere(t, "%s[%d]" % (name, i))
            if t.numel() != n:
                raise ValueError("%s[%d] must have %d elements, got %d" % (name, i, n, t.numel()))
            if not t.is_contiguous():
                raise ValueError("%s[%d] must be contiguous" % (name, i))

    def _bind(self, grads):
        """A type's table on the GPU with these gradients: made once, which waits for the stream, then changed in stream order.

        A graph may have been captured with any table: they stay, and what they point to.
        """
        grads = list(grads)
        if not grads:
            raise ValueError("grads must have %d tensors" % len(self.params))
        code = _any_dtype(grads[0], "grads[0]")
        self._same(grads, grads[0].dtype, "grads")
        captured = torch.cuda.is_current_stream_capturing()
        if code in self._tables:
            plan = self._tables[code][0]
            self._put(plan, grads)
        elif captured:
            raise ValueError("the first gradients of a type must be given outside of a capture")
        else:
            plan = self._table(grads, code)
        self._plan, self._ref, self._memory, self._made_on = plan, ctypes.addressof(plan), *self._tables[code][1:3]
        if captured:
            self._captured.append(grads)
        else:
            self.grads = self._tables[code][3] = grads

    def _put(self, plan, grads):
        """Gradients into a plan's table, in stream order."""
        _check(load().vq_adamw_grads(ctypes.addressof(plan), (_P * len(grads))(*[g.data_ptr() for g in grads]), len(grads), _stream()))

    def _table(self, grads, code):
        n = len(self.params)
        none = [None] * n
        s = self.state
        rows = (AdamWTensor * n)(*[
            AdamWTensor(p.data_ptr(), g.data_ptr(), w.data_ptr() if w is not None else None, m.data_ptr(), v.data_ptr(),
                        ms.data_ptr() if ms is not None else None, vs.data_ptr() if vs is not None else None, p.numel())
            for p, g, w, m, v, ms, vs in zip(self.params, grads, self.masters or none, s["m"], s["v"], s["m_scale"] or none,
                                             s["v_scale"] or none)])
        lib = load()
        need = lib.vq_adamw_plan_bytes(rows, n)
        table = torch.empty(need, dtype=torch.uint8, device=self.params[0].device)
        plan = AdamWPlan()
        _check(lib.vq_adamw_plan(rows, n, self.dtype, code, self.masters is not None, self.state_bits, table.data_ptr(), need,
                                 ctypes.addressof(plan), _stream()))
        weakref.finalize(self, _free_plan, plan)
        self._tables[code] = [plan, table, _stream(), grads]
        return plan

    def release(self):
        """Drops the gradients that captured steps were given: for when none of their graphs will replay again.

        Until then each capture keeps its own, and a step() without gradients outside of a graph
        puts the last ones given there back into the table first, one launch for each 448 tensors.
        """
        if self.index != _device():
            _elsewhere(self.params[0], "params[0]")
        if torch.cuda.is_current_stream_capturing():
            raise ValueError("gradients are released outside of a capture")
        if self._captured:
            for plan, _, _, grads in self._tables.values():   # each may hold what is dropped
                self._put(plan, grads)
            self._bind(self.grads)
            self._captured = []

    def step(self, grads=None, grad_scale=None):
        """One step.  grads replace those of the last step; grad_scale: a float32 tensor of one element on
        the GPU that the gradients are multiplied by."""
        if self.index != _device():
            _elsewhere(self.params[0], "params[0]")
        if not self.capturable and torch.cuda.is_current_stream_capturing():
            raise ValueError("a captured step would replay as one and the same: capturable is needed")
        if grads is not None:
            self._bind(grads)
        elif self.grads is None:
            raise ValueError("grads are needed")
        elif self._captured:                                  # a replay may have put its own into the table
            self._bind(self.grads)
        gs = None
        if grad_scale is not None:
            gs = _vector(grad_scale.reshape(-1), 1, torch.float32, self.index, "grad_scale")
        st = _stream()
        if st != self._made_on:                               # the table's memory waits for this stream too
            self._memory.record_stream(torch.cuda.current_stream())
        b1, b2 = self.betas
        if self.capturable:
            _check(load().vq_adamw(self._ref, 0.0, b1, b2, self.eps, self.weight_decay, 0, self.steps.data_ptr(),
                                   self.lr.data_ptr(), gs, st))
        else:
            _check(load().vq_adamw(self._ref, self.lr, b1, b2, self.eps, self.weight_decay, self.steps + 1, None, None, gs, st))
            self.steps += 1
