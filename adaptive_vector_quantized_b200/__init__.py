"""B200-native forward pass of AVQ-Attention (Adaptive Vector-Quantized Attention).

Thin Python binding over the C ABI of ``libavq.so`` (declared in
``include/avq.h``).  The functions keep the C names and only marshal
arguments: they check tensor dtypes/shapes/devices, allocate outputs with
torch when the caller passes none, and hand raw device pointers and the
current CUDA stream to the library.  Every step of the computation runs in
the library's CUDA kernels; there is no CPU or PyTorch fallback -- if the
library is missing the import of the first call raises.

Stage 1, ``avq_quantize``: full-tree key quantisation and aggregation
("AVQ-Attention: Adaptive Vector-Quantized Attention", Sec. 4.2, Algorithm 1).
Stage 2, ``avq_attention``: count-weighted attention over the parents with
top-P child refinement per query block (Sec. 4.3, Algorithm 2).

Beside them, exact operators of the same layers, each with its gradient:
``avq_rotary`` and ``avq_qk_norm`` (queries and keys before they are
quantised) and ``avq_cross_attention`` (over another sequence).
"""
from __future__ import annotations

import ctypes
import os
import threading

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libavq.so")

AVQ_OK, AVQ_ERR_INVALID_ARG, AVQ_ERR_UNSUPPORTED, AVQ_ERR_CUDA = 0, 1, 2, 3
AVQ_ERR_DEVICE, AVQ_ERR_TIMEOUT, AVQ_ERR_WORKSPACE = 4, 5, 6
AVQ_F32, AVQ_BF16 = 0, 1
AVQ_PATH_AUTO, AVQ_PATH_SIMT, AVQ_PATH_TC = 0, 1, 2
AVQ_DENOM_AUTO, AVQ_DENOM_TWO_PASS, AVQ_DENOM_EXTRAPOLATED = 0, 1, 2
AVQ_NORM_NONE, AVQ_NORM_RMS, AVQ_NORM_LAYER = 0, 1, 2
AVQ_ROTARY_HALF, AVQ_ROTARY_INTERLEAVED = 0, 1
AVQ_ROTARY_PLAIN, AVQ_ROTARY_LINEAR, AVQ_ROTARY_NTK, AVQ_ROTARY_YARN = 0, 1, 2, 3


class AVQError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(f"{status_string(status)}: {msg}")
        self.status = status


class avq_dims(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int), ("H", ctypes.c_int), ("N", ctypes.c_int),
                ("d", ctypes.c_int), ("M0", ctypes.c_int), ("C", ctypes.c_int)]


class avq_strides(ctypes.Structure):
    _fields_ = [("b", ctypes.c_int64), ("h", ctypes.c_int64), ("n", ctypes.c_int64)]


class avq_qk_dims(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_int) for n in ("B", "N", "Hq", "Hk", "d", "rot", "axes", "pos_batch", "layout",
                                             "norm")]
                + [("eps", ctypes.c_float), ("mscale", ctypes.c_float)])


class avq_cross_dims(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in ("B", "Bk", "Hq", "Hk", "Nq", "Nk", "d")] + [("scale", ctypes.c_float)]


_lib = None
_lib_lock = threading.Lock()
_vp = ctypes.c_void_p


def lib() -> ctypes.CDLL:
    """The loaded libavq.so; raises if it has not been built."""
    global _lib
    if _lib is None:
        with _lib_lock:
            if _lib is None:
                if not os.path.exists(LIB_PATH):
                    raise ImportError(
                        f"{LIB_PATH} is missing: build it with "
                        "`python -m adaptive_vector_quantized_b200.build`")
                L = ctypes.CDLL(LIB_PATH)
                P = ctypes.POINTER
                L.avq_quantize.argtypes = [P(avq_dims), ctypes.c_int, _vp, _vp, _vp, _vp, _vp, _vp,
                                           _vp, ctypes.c_int, _vp, ctypes.c_size_t, _vp]
                L.avq_quantize_noalloc.argtypes = [P(avq_dims), ctypes.c_int, _vp, _vp, _vp, _vp,
                                                   _vp, _vp, _vp, _vp]
                L.avq_attention.argtypes = [P(avq_dims), ctypes.c_int, _vp, _vp, _vp, _vp, _vp,
                                            ctypes.c_int, ctypes.c_int, ctypes.c_float, ctypes.c_int,
                                            _vp, _vp, _vp, _vp, ctypes.c_size_t, _vp]
                L.avq_quantize3.argtypes = [P(avq_dims), ctypes.c_int] + [_vp] * 8 + [_vp]
                L.avq_attention3.argtypes = ([P(avq_dims), ctypes.c_int] + [_vp] * 6
                                             + [ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.c_float]
                                             + [_vp] * 5 + [_vp])
                L.avq_codebook_update.argtypes = [P(avq_dims), ctypes.c_int, ctypes.c_float, _vp, _vp,
                                                  _vp, _vp, _vp, _vp, _vp]
                L.avq_permute.argtypes = [_vp, _vp, _vp, ctypes.c_int, ctypes.c_int, ctypes.c_int,
                                          ctypes.c_int, _vp]
                L.avq_hilbert_order.argtypes = [ctypes.c_int, _vp]
                L.avq_gilbert_order.argtypes = [ctypes.c_int, ctypes.c_int, _vp]
                st = P(avq_strides)
                L.avq_rotary.argtypes = [P(avq_qk_dims), ctypes.c_int, _vp, st, _vp, st, _vp, _vp, ctypes.c_int,
                                         _vp, _vp, _vp]
                L.avq_qk_norm.argtypes = [P(avq_qk_dims), ctypes.c_int, _vp, st, _vp, st] + [_vp] * 9
                L.avq_qk_norm_backward.argtypes = ([P(avq_qk_dims), ctypes.c_int] + [_vp, st] * 4 + [_vp] * 10
                                                   + [_vp, ctypes.c_size_t, _vp])
                L.avq_qk_norm_workspace_size.argtypes = [P(avq_qk_dims), ctypes.c_int]
                L.avq_qk_norm_workspace_size.restype = ctypes.c_size_t
                L.avq_rotary_freqs.argtypes = [ctypes.c_int, ctypes.c_int, ctypes.c_double, ctypes.c_int,
                                               ctypes.c_double, ctypes.c_int, ctypes.c_double, ctypes.c_double,
                                               _vp, _vp]
                L.avq_cross_attention.argtypes = ([P(avq_cross_dims), ctypes.c_int] + [_vp, st] * 3
                                                  + [_vp, _vp, _vp, st, _vp, _vp, ctypes.c_size_t, _vp])
                L.avq_cross_attention_backward.argtypes = ([P(avq_cross_dims), ctypes.c_int] + [_vp, st] * 5
                                                           + [_vp] * 7 + [ctypes.c_size_t, _vp])
                L.avq_cross_workspace_size.argtypes = [P(avq_cross_dims), ctypes.c_int, ctypes.c_int]
                L.avq_cross_workspace_size.restype = ctypes.c_size_t
                L.avq_selftest_wait.argtypes = [ctypes.c_int, _vp]
                L.avq_selftest_exp2.argtypes = [_vp, _vp, ctypes.c_int64, _vp]
                L.avq_workspace_size.argtypes = [P(avq_dims), ctypes.c_int, ctypes.c_int,
                                                 ctypes.c_int, ctypes.c_int, ctypes.c_int]
                L.avq_workspace_size.restype = ctypes.c_size_t
                L.avq_check_device.argtypes = [_vp]
                L.avq_set_path.argtypes = [ctypes.c_int]
                L.avq_set_path.restype = ctypes.c_int
                for name in ("avq_status_string", "avq_last_error", "avq_last_kernels"):
                    getattr(L, name).restype = ctypes.c_char_p
                L.avq_status_string.argtypes = [ctypes.c_int]
                L.avq_version.restype = ctypes.c_int
                for name in ("avq_quantize", "avq_quantize_noalloc", "avq_attention", "avq_permute",
                             "avq_quantize3", "avq_attention3",
                             "avq_hilbert_order", "avq_gilbert_order", "avq_check_device",
                             "avq_codebook_update", "avq_selftest_wait", "avq_selftest_exp2",
                             "avq_rotary", "avq_qk_norm", "avq_qk_norm_backward", "avq_rotary_freqs",
                             "avq_cross_attention", "avq_cross_attention_backward"):
                    getattr(L, name).restype = ctypes.c_int
                _lib = L
    return _lib


def status_string(status: int) -> str:
    return lib().avq_status_string(int(status)).decode()


def last_error() -> str:
    return lib().avq_last_error().decode()


def last_kernels() -> str:
    return lib().avq_last_kernels().decode()


def avq_set_path(path: int) -> int:
    old = lib().avq_set_path(int(path))
    if old < 0:
        raise ValueError(f"unknown path {path}")
    return old


def _check(status: int):
    if status != AVQ_OK:
        raise AVQError(status, last_error())


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.float32:
        return AVQ_F32
    if t.dtype == torch.bfloat16:
        return AVQ_BF16
    raise TypeError(f"unsupported dtype {t.dtype}; use float32 or bfloat16")


def _ptr(t):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("tensors must be CUDA tensors")
    if not t.is_contiguous():
        raise ValueError("tensors must be contiguous")
    return _vp(t.data_ptr())


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return _vp(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def _expect(t, name, shape, dtype, device):
    """Raise unless `t` is a contiguous CUDA tensor of this shape, dtype and device."""
    if t is None:
        return
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device} (all tensors on one GPU)")


def _dims(Q_like: torch.Tensor, parents: torch.Tensor, children) -> avq_dims:
    B, H, N, d = Q_like.shape
    Hp, M0, dp = parents.shape
    C = 0 if children is None else children.shape[2]
    if Hp != H or dp != d:
        raise ValueError("parents must be [H, M0, d]")
    if children is not None and tuple(children.shape) != (H, M0, C, d):
        raise ValueError("children must be [H, M0, C, d]")
    return avq_dims(B, H, N, d, M0, C)


def avq_workspace_size(dims: avq_dims, dtype: int, deterministic=False, two_pass=False,
                       P: int = 0, block: int = 128) -> int:
    return int(lib().avq_workspace_size(ctypes.byref(dims), int(dtype), int(bool(deterministic)),
                                        int(two_pass), int(P), int(block)))


def workspace(dims: avq_dims, dtype: int, device, deterministic=False, two_pass=False, P=0,
              block=128):
    """A device byte tensor of the size the library asks for (None when 0)."""
    n = avq_workspace_size(dims, dtype, deterministic, two_pass, P, block)
    if n == 0:
        return None
    return torch.empty(n + 256, dtype=torch.uint8, device=device)


def _ws_ptr(ws, device=None):
    if ws is None:
        return None, 0
    if device is not None and ws.device != device:
        raise ValueError(f"workspace is on {ws.device}, expected {device}")
    p = ws.data_ptr()
    off = (-p) % 256
    return _vp(p + off), ws.numel() - off


def _check_stage1(K, V, parents, children, assign, vsum, counts, Mt):
    """Shapes, dtypes and devices of stage 1's tensors: every tensor on K's
    device, V like K, codebook in K's dtype, outputs of the stated layout."""
    B, H, N, d = K.shape
    dev = K.device
    _expect(V, "V", K.shape, K.dtype, dev)
    _expect(parents, "parents", parents.shape, K.dtype, dev)
    _expect(children, "children", children.shape if children is not None else (), K.dtype, dev)
    _expect(assign, "assign", (B, H, N), torch.int32, dev)
    _expect(vsum, "vsum", (B, H, Mt, d), torch.float32, dev)
    _expect(counts, "counts", (B, H, Mt), torch.int32, dev)


def avq_quantize(K, V, parents, children, assign=None, vsum=None, counts=None,
                 deterministic=False, ws=None, stream=None):
    """Stage 1.  K, V [B,H,N,d]; parents [H,M0,d]; children [H,M0,C,d] (or None
    for C = 0).  Returns (assign [B,H,N] int32, vsum [B,H,Mt,d] fp32,
    counts [B,H,Mt] int32)."""
    dims = _dims(K, parents, children)
    dt = _dtype_code(K)
    B, H, N, d = K.shape
    Mt = dims.M0 * (1 + dims.C)
    dev = K.device
    _check_stage1(K, V, parents, children, assign, vsum, counts, Mt)
    if assign is None:
        assign = torch.empty((B, H, N), dtype=torch.int32, device=dev)
    if vsum is None:
        vsum = torch.empty((B, H, Mt, d), dtype=torch.float32, device=dev)
    if counts is None:
        counts = torch.empty((B, H, Mt), dtype=torch.int32, device=dev)
    if ws is None:
        ws = workspace(dims, dt, dev, deterministic=deterministic)
    wp, wn = _ws_ptr(ws, dev)
    with torch.cuda.device(dev):  # the library launches on the current device
        _check(lib().avq_quantize(ctypes.byref(dims), dt, _ptr(K), _ptr(V), _ptr(parents),
                                  _ptr(children), _ptr(assign), _ptr(vsum), _ptr(counts),
                                  int(bool(deterministic)), wp, wn, _stream(stream)))
    return assign, vsum, counts


def avq_quantize_noalloc(K, V, parents, children, assign=None, vsum=None, counts=None, stream=None):
    """Stage 1 through the library's static scratch instead of a workspace
    (no device memory is allocated by the call; pass `assign`, `vsum` and
    `counts` to keep this wrapper from allocating the outputs).  Calls whose
    executions may overlap on one device race on that scratch."""
    dims = _dims(K, parents, children)
    dt = _dtype_code(K)
    B, H, N, d = K.shape
    Mt = dims.M0 * (1 + dims.C)
    dev = K.device
    _check_stage1(K, V, parents, children, assign, vsum, counts, Mt)
    if assign is None:
        assign = torch.empty((B, H, N), dtype=torch.int32, device=dev)
    if vsum is None:
        vsum = torch.empty((B, H, Mt, d), dtype=torch.float32, device=dev)
    if counts is None:
        counts = torch.empty((B, H, Mt), dtype=torch.int32, device=dev)
    with torch.cuda.device(dev):  # the scratch array and the launch are the current device's
        _check(lib().avq_quantize_noalloc(ctypes.byref(dims), dt, _ptr(K), _ptr(V), _ptr(parents),
                                          _ptr(children), _ptr(assign), _ptr(vsum), _ptr(counts),
                                          _stream(stream)))
    return assign, vsum, counts


def avq_attention(Q, parents, children, vsum, counts, P: int, block: int = 128, scale=None,
                  two_pass=False, O=None, sel=None, importance=False, ws=None, stream=None):
    """Stage 2.  Returns (O [B,H,N,d], sel [B,H,nblk,P] int32, importance
    [B,H,nblk,M0] fp32 or None).  `importance=True` asks for the importance
    output; a tensor is written in place.  `two_pass`: AVQ_DENOM_AUTO (or
    False), AVQ_DENOM_TWO_PASS (or True) or AVQ_DENOM_EXTRAPOLATED."""
    dims = _dims(Q, parents, children)
    dt = _dtype_code(Q)
    B, H, N, d = Q.shape
    nblk = (N + block - 1) // block
    dev = Q.device
    if scale is None:
        scale = d ** -0.5
    Mt = dims.M0 * (1 + dims.C)
    _expect(parents, "parents", parents.shape, Q.dtype, dev)
    _expect(children, "children", children.shape if children is not None else (), Q.dtype, dev)
    _expect(vsum, "vsum", (B, H, Mt, d), torch.float32, dev)
    _expect(counts, "counts", (B, H, Mt), torch.int32, dev)
    _expect(O, "O", Q.shape, Q.dtype, dev)
    _expect(sel, "sel", (B, H, nblk, max(P, 0)), torch.int32, dev)
    if isinstance(importance, torch.Tensor):
        _expect(importance, "importance", (B, H, nblk, dims.M0), torch.float32, dev)
    if O is None:
        O = torch.empty_like(Q)
    if sel is None:
        sel = torch.empty((B, H, nblk, max(P, 0)), dtype=torch.int32, device=dev)
    imp = None
    if isinstance(importance, torch.Tensor):
        imp = importance
    elif importance:
        imp = torch.empty((B, H, nblk, dims.M0), dtype=torch.float32, device=dev)
    if ws is None:
        ws = workspace(dims, dt, dev, two_pass=two_pass, P=P, block=block)
    wp, wn = _ws_ptr(ws, dev)
    with torch.cuda.device(dev):
        _check(lib().avq_attention(ctypes.byref(dims), dt, _ptr(Q), _ptr(parents), _ptr(children),
                                   _ptr(vsum), _ptr(counts), int(P), int(block), float(scale),
                                   int(two_pass), _ptr(O), _ptr(sel) if P > 0 else None,
                                   _ptr(imp), wp, wn, _stream(stream)))
    return O, sel, imp


def m_total3(M0: int, C: int) -> int:
    """Codes of a depth-3 tree: M0 parents, M0*C children, M0*C*C grandchildren."""
    return M0 + M0 * C + M0 * C * C


def _dims3(X, parents, children, grandchildren):
    B, H, N, d = X.shape
    Hp, M0, dp = parents.shape
    if Hp != H or dp != d:
        raise ValueError("parents must be [H, M0, d]")
    C = children.shape[2]
    if tuple(children.shape) != (H, M0, C, d):
        raise ValueError("children must be [H, M0, C, d]")
    if tuple(grandchildren.shape) != (H, M0, C, C, d):
        raise ValueError("grandchildren must be [H, M0, C, C, d]")
    return avq_dims(B, H, N, d, M0, C)


def avq_quantize3(K, V, parents, children, grandchildren, assign=None, vsum=None, counts=None,
                  stream=None):
    """Stage 1 over a depth-3 tree.  K, V [B,H,N,d]; parents [H,M0,d];
    children [H,M0,C,d]; grandchildren [H,M0,C,C,d].  Returns (assign [B,H,N]
    int32, vsum [B,H,Mt3,d] fp32, counts [B,H,Mt3] int32), Mt3 = m_total3."""
    dims = _dims3(K, parents, children, grandchildren)
    dt = _dtype_code(K)
    B, H, N, d = K.shape
    Mt = m_total3(dims.M0, dims.C)
    dev = K.device
    _expect(V, "V", K.shape, K.dtype, dev)
    for t, nm in ((parents, "parents"), (children, "children"), (grandchildren, "grandchildren")):
        _expect(t, nm, t.shape, K.dtype, dev)
    _expect(assign, "assign", (B, H, N), torch.int32, dev)
    _expect(vsum, "vsum", (B, H, Mt, d), torch.float32, dev)
    _expect(counts, "counts", (B, H, Mt), torch.int32, dev)
    if assign is None:
        assign = torch.empty((B, H, N), dtype=torch.int32, device=dev)
    if vsum is None:
        vsum = torch.empty((B, H, Mt, d), dtype=torch.float32, device=dev)
    if counts is None:
        counts = torch.empty((B, H, Mt), dtype=torch.int32, device=dev)
    with torch.cuda.device(dev):
        _check(lib().avq_quantize3(ctypes.byref(dims), dt, _ptr(K), _ptr(V), _ptr(parents), _ptr(children),
                                   _ptr(grandchildren), _ptr(assign), _ptr(vsum), _ptr(counts),
                                   _stream(stream)))
    return assign, vsum, counts


def avq_attention3(Q, parents, children, grandchildren, vsum, counts, P: int, P2: int, block: int = 128,
                   scale=None, O=None, importance=False, stream=None):
    """Stage 2 over a depth-3 tree.  Returns (O [B,H,N,d], sel [B,H,nblk,P]
    parents, sel2 [B,H,nblk,P2] child codes, importance [B,H,nblk,M0] or None,
    importance2 [B,H,nblk,P*C] or None)."""
    dims = _dims3(Q, parents, children, grandchildren)
    dt = _dtype_code(Q)
    B, H, N, d = Q.shape
    M0, C = dims.M0, dims.C
    Mt = m_total3(M0, C)
    nblk = (N + block - 1) // block
    dev = Q.device
    if scale is None:
        scale = d ** -0.5
    for t, nm in ((parents, "parents"), (children, "children"), (grandchildren, "grandchildren")):
        _expect(t, nm, t.shape, Q.dtype, dev)
    _expect(vsum, "vsum", (B, H, Mt, d), torch.float32, dev)
    _expect(counts, "counts", (B, H, Mt), torch.int32, dev)
    _expect(O, "O", Q.shape, Q.dtype, dev)
    if O is None:
        O = torch.empty_like(Q)
    sel = torch.empty((B, H, nblk, max(P, 0)), dtype=torch.int32, device=dev)
    sel2 = torch.empty((B, H, nblk, max(P2, 0)), dtype=torch.int32, device=dev)
    imp = imp2 = None
    if importance:
        imp = torch.empty((B, H, nblk, M0), dtype=torch.float32, device=dev)
        imp2 = torch.empty((B, H, nblk, max(P * C, 1)), dtype=torch.float32, device=dev)
    with torch.cuda.device(dev):
        _check(lib().avq_attention3(ctypes.byref(dims), dt, _ptr(Q), _ptr(parents), _ptr(children),
                                    _ptr(grandchildren), _ptr(vsum), _ptr(counts), int(P), int(P2),
                                    int(block), float(scale), _ptr(O), _ptr(sel) if P > 0 else None,
                                    _ptr(sel2) if P2 > 0 else None, _ptr(imp), _ptr(imp2), _stream(stream)))
    return O, sel, sel2, imp, imp2


def avq_codebook_update(ksum, counts, S, Nst, parents, children, lam: float, stream=None):
    """Codebook update (EMA statistics and constraint projection).  ksum
    [B,H,Mt,d] fp32 and counts [B,H,Mt] int32: avq_quantize's statistics of
    the keys; S [H,Mt,d] and Nst [H,Mt] fp32: EMA state, updated in place;
    parents [H,M0,d] and children [H,M0,C,d]: codebook, rewritten in place."""
    B, H, Mt, d = ksum.shape
    Hp, M0, dp = parents.shape
    C = 0 if children is None else children.shape[2]
    if Hp != H or dp != d or Mt != M0 * (1 + C):
        raise ValueError("ksum must be [B, H, M0*(1+C), d] for parents [H, M0, d]")
    if children is not None and tuple(children.shape) != (H, M0, C, d):
        raise ValueError("children must be [H, M0, C, d]")
    dims = avq_dims(B, H, 1, d, M0, C)
    dt = _dtype_code(parents)
    dev = parents.device
    _expect(ksum, "ksum", (B, H, Mt, d), torch.float32, dev)
    _expect(counts, "counts", (B, H, Mt), torch.int32, dev)
    _expect(S, "S", (H, Mt, d), torch.float32, dev)
    _expect(Nst, "Nst", (H, Mt), torch.float32, dev)
    _expect(children, "children", (H, M0, C, d), parents.dtype, dev)
    with torch.cuda.device(dev):
        _check(lib().avq_codebook_update(ctypes.byref(dims), dt, float(lam), _ptr(ksum), _ptr(counts),
                                         _ptr(S), _ptr(Nst), _ptr(parents), _ptr(children),
                                         _stream(stream)))
    return S, Nst, parents, children


def avq_permute(X, idx, inverse=False, Y=None, stream=None):
    """Gather (inverse=False: Y[b,i] = X[b,idx[i]]) or scatter back along dim -2
    of a [..., rows, cols] tensor; idx is an int32 CUDA tensor."""
    rows = X.shape[-2]
    batch = X.numel() // (rows * X.shape[-1])
    row_bytes = X.shape[-1] * X.element_size()
    _expect(idx, "idx", (rows,), torch.int32, X.device)
    _expect(Y, "Y", X.shape, X.dtype, X.device)
    if Y is None:
        Y = torch.empty_like(X)
    with torch.cuda.device(X.device):
        _check(lib().avq_permute(_ptr(X), _ptr(idx), _ptr(Y), int(batch), int(rows), int(row_bytes),
                                 int(bool(inverse)), _stream(stream)))
    return Y


def avq_hilbert_order(side: int) -> torch.Tensor:
    """Raster index of the t-th cell along a Hilbert curve (host tensor, int32)."""
    out = torch.empty(side * side, dtype=torch.int32)
    _check(lib().avq_hilbert_order(int(side), _vp(out.data_ptr())))
    return out


def avq_gilbert_order(width: int, height: int) -> torch.Tensor:
    """Raster index (y*width + x) of the t-th cell along a generalised Hilbert
    curve over a width x height grid (host tensor, int32)."""
    out = torch.empty(max(1, int(width) * int(height)), dtype=torch.int32)  # sizes checked by the library
    _check(lib().avq_gilbert_order(int(width), int(height), _vp(out.data_ptr())))
    return out


def _view(t, name, shape=None, dtype=None, device=None):
    """Address and strides of a [B,H,N,d] CUDA tensor whose last dimension is
    contiguous (any view of that kind: heads inside a joint projection)."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dim() != 4:
        raise ValueError(f"{name} must be [B, H, N, d], got {tuple(t.shape)}")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device} (all tensors on one GPU)")
    b, h, n, d = t.stride()
    if d != 1:
        raise ValueError(f"the last dimension of {name} must be contiguous")
    return t.data_ptr(), avq_strides(b, h, n)


_NO_VIEW = (None, avq_strides(0, 0, 0))


def _dense_like(t):
    return torch.empty_like(t, memory_format=torch.contiguous_format)


def _addr(t):
    """Address of a contiguous CUDA tensor, None for None."""
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("tensors must be CUDA tensors")
    if not t.is_contiguous():
        raise ValueError("tensors must be contiguous")
    return t.data_ptr()


class _Launch:
    """Context in which a call allocates and launches, as the raw stream handle:
    `dev` current and, when the caller names a stream, that stream current too,
    so that outputs and workspaces made inside come from (and go back to) that
    stream's memory.  Where both are current already nothing is switched: the
    smallest calls are bound by the host."""
    __slots__ = ("inner", "index")

    def __init__(self, dev, stream):
        self.index = dev.index
        if stream is not None:
            if not isinstance(stream, torch.cuda.Stream):
                handle = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
                stream = torch.cuda.ExternalStream(handle, device=dev)
            if stream.device != dev:
                raise ValueError(f"the stream is on {stream.device}, expected {dev}")
            self.inner = torch.cuda.stream(stream)
        else:
            self.inner = None if torch.cuda.current_device() == dev.index else torch.cuda.device(dev)

    def __enter__(self):
        if self.inner is not None:
            self.inner.__enter__()
        return torch._C._cuda_getCurrentRawStream(self.index)

    def __exit__(self, *exc):
        if self.inner is not None:
            self.inner.__exit__(*exc)


_NORMS = {"rms": AVQ_NORM_RMS, "layer": AVQ_NORM_LAYER}
_LAYOUTS = {"half": AVQ_ROTARY_HALF, "interleaved": AVQ_ROTARY_INTERLEAVED}
_SCALINGS = {"none": AVQ_ROTARY_PLAIN, "linear": AVQ_ROTARY_LINEAR, "ntk": AVQ_ROTARY_NTK, "yarn": AVQ_ROTARY_YARN}


def _choice(table, value, name):
    if value not in table:
        raise ValueError(f"{name} must be one of {sorted(table)}, got {value!r}")
    return table[value]


def _qk_dims(Q, K, norm, eps, freqs, positions, layout, mscale, axes):
    """Dims, position and frequency tensors of a norm or rotation call, checked."""
    if not isinstance(Q, torch.Tensor) or Q.dim() != 4:
        raise ValueError("Q must be a [B, H, N, d] tensor")
    B, Hq, N, d = Q.shape
    Hk = 0
    if K is not None:
        shape = K.shape if isinstance(K, torch.Tensor) else ()
        if len(shape) != 4 or shape[0] != B or shape[2] != N or shape[3] != d:
            raise ValueError("K must be [B, Hk, N, d] like Q")
        Hk = shape[1]
    rot, pos_batch = 0, 0
    if freqs is not None:
        pairs = freqs.numel()
        rot, dev = 2 * pairs, Q.device
        _expect(freqs, "freqs", (pairs,), torch.float64, dev)
        if positions is not None:
            tail = (2,) if axes == 2 else ()
            pos_batch = int(positions.dim() == 2 + len(tail))
            _expect(positions, "positions", ((B, N) if pos_batch else (N,)) + tail, torch.int32, dev)
    elif positions is not None:
        raise ValueError("positions need freqs")
    dims = avq_qk_dims(B, N, Hq, Hk, d, rot, int(axes), pos_batch, _choice(_LAYOUTS, layout, "layout"), norm,
                       float(eps), float(mscale))
    return dims, (positions if freqs is not None else None)


def _qk_outputs(Q, K, Yq, Yk):
    if Yq is None:
        Yq = _dense_like(Q)
    else:
        _expect(Yq, "the queries' output", Q.shape, Q.dtype, Q.device)
    if K is None:
        return Yq, None
    if Yk is None:
        Yk = _dense_like(K)
    else:
        _expect(Yk, "the keys' output", K.shape, Q.dtype, Q.device)
    return Yq, Yk


def avq_rotary_freqs(rot: int, base: float = 10000.0, axes: int = 1, scaling: str = "none", factor: float = 1.0,
                     trained: int = 4096, turns_low: float = 1.0, turns_high: float = 32.0, device="cpu"):
    """Frequencies of a rotation of `rot` elements (float64 [rot/2], on `device`)
    and the factor on sine and cosine.  scaling: "none", "linear", "ntk" or
    "yarn", stretching positions by `factor` beyond the `trained` range."""
    out = torch.empty(max(1, int(rot) // 2), dtype=torch.float64)
    m = ctypes.c_float(1.0)
    _check(lib().avq_rotary_freqs(int(rot), int(axes), float(base), _choice(_SCALINGS, scaling, "scaling"),
                                  float(factor), int(trained), float(turns_low), float(turns_high),
                                  _vp(out.data_ptr()), ctypes.byref(m)))
    return out.to(device), m.value


def avq_rotary(Q, K=None, freqs=None, positions=None, layout="half", mscale=1.0, axes=1, inverse=False, Yq=None,
               Yk=None, stream=None):
    """Rotation by position of Q [B,Hq,N,d] and K [B,Hk,N,d] (or None), views
    with a contiguous last dimension.  freqs float64 [rot/2] on the GPU: the
    leading `rot` elements of each head turn; positions int32 [N] or [B,N],
    with axes=2 [N,2] or [B,N,2] (None: 0..N-1); layout "half" or
    "interleaved".  Returns dense (Yq, Yk).  `inverse` turns the other way:
    the gradient of the forward call."""
    if freqs is None:
        raise ValueError("freqs is needed")
    dims, positions = _qk_dims(Q, K, AVQ_NORM_NONE, 0.0, freqs, positions, layout, mscale, axes)
    dt, dev = _dtype_code(Q), Q.device
    qp, qs = _view(Q, "Q")
    kp, ks = _NO_VIEW if K is None else _view(K, "K", dtype=Q.dtype, device=dev)
    with _Launch(dev, stream) as st:
        Yq, Yk = _qk_outputs(Q, K, Yq, Yk)
        _check(lib().avq_rotary(ctypes.byref(dims), dt, qp, ctypes.byref(qs), kp, ctypes.byref(ks),
                                _addr(positions), _addr(freqs), int(bool(inverse)), _addr(Yq), _addr(Yk),
                                st))
    return Yq, Yk


def avq_qk_norm(Q, K=None, q_weight=None, k_weight=None, q_bias=None, k_bias=None, norm="rms", eps=1e-6, freqs=None,
                positions=None, layout="half", mscale=1.0, axes=1, Yq=None, Yk=None, stream=None):
    """RMS or LayerNorm (norm "rms" or "layer") of every head of Q [B,Hq,N,d] and
    K [B,Hk,N,d] (or None), then, with freqs, the rotation of avq_rotary, in
    one pass.  Weights and biases [d] in Q's dtype, or None.  Returns dense
    (Yq, Yk)."""
    dims, positions = _qk_dims(Q, K, _choice(_NORMS, norm, "norm"), eps, freqs, positions, layout, mscale, axes)
    dt, dev = _dtype_code(Q), Q.device
    qp, qs = _view(Q, "Q")
    kp, ks = _NO_VIEW if K is None else _view(K, "K", dtype=Q.dtype, device=dev)
    shape = (dims.d,)
    for t, n in ((q_weight, "q_weight"), (k_weight, "k_weight"), (q_bias, "q_bias"), (k_bias, "k_bias")):
        if t is not None:
            _expect(t, n, shape, Q.dtype, dev)
    with _Launch(dev, stream) as st:
        Yq, Yk = _qk_outputs(Q, K, Yq, Yk)
        _check(lib().avq_qk_norm(ctypes.byref(dims), dt, qp, ctypes.byref(qs), kp, ctypes.byref(ks), _addr(q_weight),
                                 _addr(k_weight), _addr(q_bias), _addr(k_bias), _addr(positions), _addr(freqs), _addr(Yq),
                                 _addr(Yk), st))
    return Yq, Yk


def avq_qk_norm_backward(dYq, dYk, Q, K=None, q_weight=None, k_weight=None, norm="rms", eps=1e-6, bias=False,
                         freqs=None, positions=None, layout="half", mscale=1.0, axes=1, dQ=None, dK=None, ws=None,
                         stream=None):
    """Gradients of avq_qk_norm.  Returns (dQ, dK, dq_weight, dk_weight, dq_bias,
    dk_bias): dQ, dK dense in Q's dtype, the others float32 [d] (the weights'
    where a weight was given, the biases' with bias=True, else None)."""
    dims, positions = _qk_dims(Q, K, _choice(_NORMS, norm, "norm"), eps, freqs, positions, layout, mscale, axes)
    if (dYk is None) != (K is None):
        raise ValueError("dYk and K go together")
    dt, dev = _dtype_code(Q), Q.device
    gqp, gqs = _view(dYq, "dYq", Q.shape, Q.dtype, dev)
    gkp, gks = _NO_VIEW if K is None else _view(dYk, "dYk", K.shape, Q.dtype, dev)
    qp, qs = _view(Q, "Q")
    kp, ks = _NO_VIEW if K is None else _view(K, "K", dtype=Q.dtype, device=dev)
    for t, n in ((q_weight, "q_weight"), (k_weight, "k_weight")):
        if t is not None:
            _expect(t, n, (dims.d,), Q.dtype, dev)
    wanted = (q_weight is not None, K is not None and k_weight is not None, bool(bias), bool(bias) and K is not None)
    with _Launch(dev, stream) as st:
        dQ, dK = _qk_outputs(Q, K, dQ, dK)
        sums = iter(torch.empty((sum(wanted), dims.d), dtype=torch.float32, device=dev).unbind(0) if any(wanted) else ())
        dwq, dwk, dbq, dbk = (next(sums) if w else None for w in wanted)
        if ws is None:
            n = int(lib().avq_qk_norm_workspace_size(ctypes.byref(dims), dt))
            ws = torch.empty(n + 256, dtype=torch.uint8, device=dev)
        wp, wn = _ws_ptr(ws, dev)
        _check(lib().avq_qk_norm_backward(ctypes.byref(dims), dt, gqp, ctypes.byref(gqs), gkp, ctypes.byref(gks), qp,
                                          ctypes.byref(qs), kp, ctypes.byref(ks), _addr(q_weight), _addr(k_weight),
                                          _addr(positions), _addr(freqs), _addr(dQ), _addr(dK), _addr(dwq), _addr(dwk),
                                          _addr(dbq), _addr(dbk), wp, wn, st))
    return dQ, dK, dwq, dwk, dbq, dbk


def _cross_dims(Q, K, V, kv_lens, key_mask, scale):
    """Dims of a cross attention call and its inputs' pointers and strides."""
    if not isinstance(Q, torch.Tensor) or Q.dim() != 4:
        raise ValueError("Q must be a [B, Hq, Nq, d] tensor")
    B, Hq, Nq, d = Q.shape
    dev = Q.device
    views = [_view(Q, "Q"), _view(K, "K", None, Q.dtype, dev), _view(V, "V", K.shape, Q.dtype, dev)]
    Bk, Hk, Nk, dk = K.shape
    if dk != d:
        raise ValueError(f"K must be [Bk, Hk, Nk, {d}], got {tuple(K.shape)}")
    if Bk < 1 or Hk < 1 or B % Bk or Hq % Hk:
        raise ValueError(f"Q's batch and heads ({B}, {Hq}) must be multiples of K's ({Bk}, {Hk})")
    _expect(kv_lens, "kv_lens", (Bk,), torch.int32, dev)
    if key_mask is not None:
        if not isinstance(key_mask, torch.Tensor) or key_mask.dtype not in (torch.bool, torch.uint8):
            raise TypeError("key_mask must be a bool or uint8 tensor")
        _expect(key_mask, "key_mask", (Bk, Nk), None, dev)
    scale = d ** -0.5 if scale is None else float(scale)
    return avq_cross_dims(B, Bk, Hq, Hk, Nq, Nk, d, scale), views


def avq_cross_workspace_size(dims: avq_cross_dims, dtype: int, backward=False) -> int:
    return int(lib().avq_cross_workspace_size(ctypes.byref(dims), int(dtype), int(bool(backward))))


def _cross_ws(dims, dt, backward, ws, dev):
    if ws is None:
        n = avq_cross_workspace_size(dims, dt, backward)
        ws = torch.empty(n + 256, dtype=torch.uint8, device=dev) if n else None
    return ws, *_ws_ptr(ws, dev)


def avq_cross_attention(Q, K, V, kv_lens=None, key_mask=None, scale=None, O=None, lse=False, ws=None, stream=None):
    """Exact attention of Q [B,Hq,Nq,d] over another sequence's K, V
    [Bk,Hk,Nk,d] (views with a contiguous last dimension; B a multiple of Bk,
    Hq of Hk).  kv_lens int32 [Bk]: keys from there on are left out; key_mask
    bool [Bk,Nk]: keys where it is False are left out.  Rows with no key give
    0.  Returns (O [B,Hq,Nq,d], lse float32 [B,Hq,Nq] or None); `O` may be a
    view; `lse=True` asks for the log-sum-exp that the backward call needs, a
    tensor is written in place."""
    dims, ((qp, qs), (kp, ks), (vp, vs)) = _cross_dims(Q, K, V, kv_lens, key_mask, scale)
    dt, dev = _dtype_code(Q), Q.device
    with _Launch(dev, stream) as st:
        if O is None:
            O = _dense_like(Q)
        op, os_ = _view(O, "O", Q.shape, Q.dtype, dev)
        if isinstance(lse, torch.Tensor):
            _expect(lse, "lse", Q.shape[:3], torch.float32, dev)
        else:
            lse = torch.empty(Q.shape[:3], dtype=torch.float32, device=dev) if lse else None
        ws, wp, wn = _cross_ws(dims, dt, False, ws, dev)
        _check(lib().avq_cross_attention(ctypes.byref(dims), dt, qp, ctypes.byref(qs), kp, ctypes.byref(ks), vp,
                                         ctypes.byref(vs), _addr(kv_lens), _addr(key_mask), op, ctypes.byref(os_),
                                         _addr(lse), wp, wn, st))
    return O, lse


def avq_cross_attention_backward(dO, Q, K, V, O, lse, kv_lens=None, key_mask=None, scale=None, dQ=None, dK=None,
                                 dV=None, ws=None, stream=None):
    """Gradients of avq_cross_attention from its inputs, its outputs O and lse and
    the gradient dO of O.  Returns dense (dQ [B,Hq,Nq,d], dK, dV [Bk,Hk,Nk,d]),
    dK and dV summed over the heads and batch entries that share them."""
    dims, ((qp, qs), (kp, ks), (vp, vs)) = _cross_dims(Q, K, V, kv_lens, key_mask, scale)
    dt, dev = _dtype_code(Q), Q.device
    gp, gs = _view(dO, "dO", Q.shape, Q.dtype, dev)
    op, os_ = _view(O, "O", Q.shape, Q.dtype, dev)
    if lse is None:
        raise ValueError("lse is needed: call the forward pass with lse=True")
    _expect(lse, "lse", Q.shape[:3], torch.float32, dev)
    for t, name, like in ((dQ, "dQ", Q), (dK, "dK", K), (dV, "dV", K)):
        if t is not None:
            _expect(t, name, like.shape, Q.dtype, dev)
    with _Launch(dev, stream) as st:
        dQ, dK, dV = (_dense_like(like) if t is None else t
                      for t, like in ((dQ, Q), (dK, K), (dV, K)))
        ws, wp, wn = _cross_ws(dims, dt, True, ws, dev)
        _check(lib().avq_cross_attention_backward(
            ctypes.byref(dims), dt, gp, ctypes.byref(gs), qp, ctypes.byref(qs), kp, ctypes.byref(ks), vp,
            ctypes.byref(vs), op, ctypes.byref(os_), _addr(lse), _addr(kv_lens), _addr(key_mask), _addr(dQ), _addr(dK),
            _addr(dV), wp, wn, st))
    return dQ, dK, dV


def avq_selftest_wait(timeout_us: int = 2000, stream=None):
    """Launch the bounded-wait self-test: the next avq_check_device raises
    AVQError with status AVQ_ERR_TIMEOUT."""
    _check(lib().avq_selftest_wait(int(timeout_us), _stream(stream)))


def avq_selftest_exp2(x, y=None, stream=None):
    """The FMA-pipe 2^x of the attention kernel on a contiguous fp32 CUDA
    tensor with an even number of elements; returns y (allocated if None)."""
    if not (isinstance(x, torch.Tensor) and x.is_cuda and x.dtype == torch.float32):
        raise TypeError("x must be a float32 CUDA tensor")
    if y is None:
        y = torch.empty_like(x)
    _expect(y, "y", x.shape, torch.float32, x.device)
    with torch.cuda.device(x.device):
        _check(lib().avq_selftest_exp2(_ptr(x), _ptr(y), int(x.numel()), _stream(stream)))
    return y


def avq_check_device(stream=None):
    """Synchronise the stream and raise if a kernel recorded a device-side error."""
    _check(lib().avq_check_device(_stream(stream)))


def avq_version() -> int:
    return int(lib().avq_version())
