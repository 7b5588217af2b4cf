"""Binding of libmxs (the C ABI in include/mxs.h), same entry-point names: ctypes,
and for the ordinary form of the serving calls a small extension module where
one is built for the torch at hand (the general path gives the same results).

Argument marshalling only: every step of the path runs in the library's CUDA
kernels.  torch supplies device memory (inputs, outputs, workspaces) and
streams.  The library must be built (``python -m mx_microscaling_mixed_b200.build``);
if it is missing this module raises on import -- there is no fallback.
"""
from __future__ import annotations

import ctypes
import importlib.util
import os
from dataclasses import dataclass, field
from typing import List, Optional, Sequence

import torch

from . import build as _build

_LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libmxs.so")
if not os.path.exists(_LIB_PATH):
    raise ImportError(f"libmxs.so not built at {_LIB_PATH}; run python -m mx_microscaling_mixed_b200.build")
_lib = ctypes.CDLL(_LIB_PATH)


def _load_binding():
    """The extension that marshals the serving calls' arguments in C++ (linked
    against libmxs.so), or None."""
    path = _build.binding_path()
    if not os.path.exists(path):
        return None
    spec = importlib.util.spec_from_file_location(__package__ + "._binding", path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


_binding = _load_binding()

MXS_F32, MXS_BF16 = 0, 1
MXS_ALLOC_FRACTIONS, MXS_ALLOC_BUDGET, MXS_ALLOC_LAYER = 0, 1, 2
SEG_BITS = (8, 6, 4)

STATUS = {0: "MXS_OK", 1: "MXS_ERR_ARG", 2: "MXS_ERR_SHAPE", 3: "MXS_ERR_ALIGN", 4: "MXS_ERR_DTYPE",
          5: "MXS_ERR_BUDGET", 6: "MXS_ERR_CUDA", 7: "MXS_ERR_TIMEOUT", 8: "MXS_ERR_DEVICE",
          9: "MXS_ERR_WORKSPACE"}


class MxsError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {_lib.mxs_status_str(status).decode()}")


class Segment(ctypes.Structure):
    _fields_ = [("bits", ctypes.c_int32), ("k_real", ctypes.c_int64), ("k_pad", ctypes.c_int64),
                ("k_off", ctypes.c_int64)]


class LayoutC(ctypes.Structure):
    _fields_ = [("K", ctypes.c_int64), ("K_pad", ctypes.c_int64), ("seg", Segment * 3),
                ("perm", ctypes.c_void_p)]


class MXTensorC(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("lay", LayoutC), ("codes", ctypes.c_void_p * 3),
                ("code_pitch", ctypes.c_int64 * 3), ("scales", ctypes.c_void_p * 3),
                ("scale_pitch", ctypes.c_int64 * 3)]


class StackC(ctypes.Structure):
    _fields_ = [("n_blocks", ctypes.c_int32), ("hidden", ctypes.c_int32), ("n_heads", ctypes.c_int32),
                ("n_kv_heads", ctypes.c_int32), ("mlp", ctypes.c_int32), ("rms_eps", ctypes.c_float),
                ("rope_theta", ctypes.c_float), ("W", ctypes.c_void_p)]


class BudgetC(ctypes.Structure):
    _fields_ = [("mode", ctypes.c_int32), ("num", ctypes.c_int64), ("den", ctypes.c_int64),
                ("p8_num", ctypes.c_int64), ("p8_den", ctypes.c_int64), ("p6_num", ctypes.c_int64),
                ("p6_den", ctypes.c_int64), ("fixed8", ctypes.c_int64)]


class RopeScalingC(ctypes.Structure):
    _fields_ = [("kind", ctypes.c_int32), ("factor", ctypes.c_double), ("low", ctypes.c_double),
                ("high", ctypes.c_double), ("orig_len", ctypes.c_int64)]


class RopePlanC(ctypes.Structure):
    _fields_ = [("rot", ctypes.c_int32), ("layout", ctypes.c_int32), ("gain", ctypes.c_double),
                ("step", ctypes.c_uint64 * 128)]


class KVCacheC(ctypes.Structure):
    _fields_ = [("K", MXTensorC), ("V", MXTensorC), ("n_kvh", ctypes.c_int64)]


class TreeBatchC(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int64), ("rows", ctypes.c_int64), ("max_q", ctypes.c_int64),
                ("max_len", ctypes.c_int64), ("q_start", ctypes.c_void_p), ("length", ctypes.c_void_p),
                ("pages", ctypes.c_void_p), ("ldp", ctypes.c_int64), ("page_size", ctypes.c_int64),
                ("mask", ctypes.c_void_p), ("ldm", ctypes.c_int64)]


_P = ctypes.c_void_p
_I64 = ctypes.c_int64
_SZ = ctypes.c_size_t
_ST = ctypes.c_int


def _sig(name, args, res=_ST):
    f = getattr(_lib, name)
    f.argtypes = args
    f.restype = res
    return f


_sig("mxs_status_str", [_ST], ctypes.c_char_p)
_sig("mxs_launch_count", [], _I64)
_sig("mxs_sync", [_P])
_sig("mxs_set_wait_limit", [_I64])
_sig("mxs_layout_make", [_I64, _P, _P, ctypes.POINTER(LayoutC)])
_sig("mxs_mxtensor_bytes", [_I64, ctypes.POINTER(LayoutC), _P, _P, _P, _P])
_sig("mxs_sensitivity_workspace_bytes", [_I64, _I64, _I64, ctypes.POINTER(_SZ)])
_sig("mxs_sensitivity", [_P, _ST, _I64, _I64, _I64, _P, _ST, _I64, _I64, _P, _P, _P, _P, _SZ, _P])
_sig("mxs_sensitivity_noalloc", [_P, _ST, _I64, _I64, _I64, _P, _ST, _I64, _I64, _P, _P, _P, _P])
_sig("mxs_allocate_workspace_bytes", [ctypes.c_int32, _P, ctypes.POINTER(_SZ)])
_sig("mxs_allocate", [ctypes.c_int32, _P, _P, _P, _P, ctypes.POINTER(BudgetC), _P, _P, _P, _SZ, _P])
_sig("mxs_quantize_weight", [_P, _ST, _I64, _I64, ctypes.POINTER(MXTensorC), _P])
_sig("mxs_quantize_act", [_P, _ST, _I64, _I64, ctypes.POINTER(MXTensorC), _P])
_sig("mxs_dequantize", [ctypes.POINTER(MXTensorC), _P, _I64, _P])
_sig("mxs_gemm_workspace_bytes", [ctypes.POINTER(MXTensorC), ctypes.POINTER(MXTensorC), ctypes.POINTER(_SZ)])
_sig("mxs_gemm", [ctypes.POINTER(MXTensorC), ctypes.POINTER(MXTensorC), _P, _I64, _P, _SZ, _P])
_sig("mxs_layer_scores_workspace_bytes", [ctypes.POINTER(StackC), _I64, ctypes.POINTER(_SZ)])
_sig("mxs_layer_scores", [ctypes.POINTER(StackC), _P, _I64, _I64, _P, _P, _SZ, _P])
_sig("mxs_attn_decode_workspace_bytes", [_I64, _I64, _I64, _I64, ctypes.POINTER(_SZ)])
_sig("mxs_attn_decode", [_P, _I64, _I64, ctypes.POINTER(MXTensorC), ctypes.POINTER(MXTensorC), _I64, _I64,
                         ctypes.c_float, _P, _I64, _P, _SZ, _P])
_sig("mxs_rope_plan_make", [ctypes.c_int32, ctypes.c_int32, ctypes.c_double, _P, _P])
_sig("mxs_rope", [_P, _ST, _I64, _I64, _I64, _I64, _I64, _P, _P, ctypes.c_int32, _P, _ST, _I64, _I64, _P])
_sig("mxs_kv_write", [_P, _I64, _I64, _P, _I64, _I64, _ST, _I64, _P, _P, _P, _P, _P])
_sig("mxs_kv_read", [_P, _I64, _P, _P, _I64, _I64, _P, _I64, _I64, _ST, _P])
_sig("mxs_attn_tree_workspace_bytes", [_P, _P, _I64, _ST, _P])
_sig("mxs_attn_tree", [_P, _I64, _I64, _I64, _P, _P, ctypes.c_float, _P, _ST, _I64, _I64, _P, _P, _SZ, _P])

EXPORTS = ["mxs_status_str", "mxs_launch_count", "mxs_sync", "mxs_set_wait_limit", "mxs_layout_make", "mxs_mxtensor_bytes",
           "mxs_sensitivity_workspace_bytes", "mxs_sensitivity", "mxs_sensitivity_noalloc",
           "mxs_allocate_workspace_bytes",
           "mxs_allocate", "mxs_quantize_weight", "mxs_quantize_act", "mxs_dequantize",
           "mxs_gemm_workspace_bytes", "mxs_gemm", "mxs_attn_decode_workspace_bytes", "mxs_attn_decode",
           "mxs_layer_scores_workspace_bytes", "mxs_layer_scores", "mxs_rope_plan_make", "mxs_rope", "mxs_kv_write",
           "mxs_kv_read", "mxs_attn_tree_workspace_bytes", "mxs_attn_tree"]


def _check(st: int, where: str):
    if st != 0:
        raise MxsError(st, where)


def _stream(stream) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


_DT = {torch.float32: MXS_F32, torch.bfloat16: MXS_BF16}


def _dt(t: torch.Tensor) -> int:
    d = _DT.get(t.dtype)
    if d is None:
        raise TypeError(f"unsupported dtype {t.dtype}")
    return d


def _rowmajor(t: torch.Tensor) -> int:
    if t.dim() != 2 or t.stride(1) != 1:
        raise ValueError("expected a 2-D tensor with unit stride along K")
    return t.stride(0)


def _workspace(nbytes: int, device) -> torch.Tensor:
    # 1024 extra bytes so the base can be aligned to 1024 inside
    return torch.empty(int(nbytes) + 1024, dtype=torch.uint8, device=device)


def _aligned_ptr(buf: torch.Tensor, align: int = 1024) -> int:
    p = buf.data_ptr()
    return (p + align - 1) // align * align


# ------------------------------------------------------------------ layouts
@dataclass
class Layout:
    c: LayoutC
    counts: tuple
    perm: Optional[torch.Tensor] = None      # keeps the device permutation alive

    @property
    def K(self) -> int:
        return int(self.c.K)

    @property
    def K_pad(self) -> int:
        return int(self.c.K_pad)


def mxs_layout_make(K: int, counts: Sequence[int], perm: Optional[torch.Tensor] = None) -> Layout:
    arr = (ctypes.c_int64 * 3)(*[int(c) for c in counts])
    lay = LayoutC()
    if perm is not None:
        assert perm.dtype == torch.int32 and perm.is_cuda and perm.is_contiguous() and perm.numel() == K
    _check(_lib.mxs_layout_make(int(K), arr, None if perm is None else ctypes.c_void_p(perm.data_ptr()),
                                ctypes.byref(lay)), "mxs_layout_make")
    return Layout(lay, tuple(int(c) for c in counts), perm)


def mxs_mxtensor_bytes(rows: int, layout: Layout):
    cp, cb, sp, sb = [(ctypes.c_int64 * 3)() for _ in range(4)]
    _check(_lib.mxs_mxtensor_bytes(int(rows), ctypes.byref(layout.c), cp, cb, sp, sb), "mxs_mxtensor_bytes")
    return list(cp), list(cb), list(sp), list(sb)


@dataclass
class MXTensor:
    """A quantised matrix: per-segment code and scale buffers (torch uint8)."""
    rows: int
    layout: Layout
    codes: List[Optional[torch.Tensor]]
    scales: List[Optional[torch.Tensor]]
    c: MXTensorC = field(default_factory=MXTensorC)

    def code_rows(self, g: int) -> torch.Tensor:
        """Compact (rows x payload bytes) view of segment g's codes."""
        kp = self.layout.c.seg[g].k_pad
        return self.codes[g][:, :kp * SEG_BITS[g] // 8] if kp else torch.empty(self.rows, 0, dtype=torch.uint8)

    def scale_rows(self, g: int) -> torch.Tensor:
        kp = self.layout.c.seg[g].k_pad
        return self.scales[g][:, :kp // 32] if kp else torch.empty(self.rows, 0, dtype=torch.uint8)


def mxtensor_empty(rows: int, layout: Layout, device="cuda") -> MXTensor:
    cp, cb, sp, sb = mxs_mxtensor_bytes(rows, layout)
    codes, scales = [], []
    c = MXTensorC()
    c.rows = rows
    c.lay = layout.c
    for g in range(3):
        if cb[g] or (layout.c.seg[g].k_pad and rows):
            ct = torch.zeros((rows, cp[g]), dtype=torch.uint8, device=device)
            st = torch.zeros((rows, sp[g]), dtype=torch.uint8, device=device)
        else:
            ct = st = None
        codes.append(ct)
        scales.append(st)
        c.codes[g] = ct.data_ptr() if ct is not None else None
        c.scales[g] = st.data_ptr() if st is not None else None
        c.code_pitch[g] = cp[g]
        c.scale_pitch[g] = sp[g]
    return MXTensor(rows, layout, codes, scales, c)


# ------------------------------------------------------------- sensitivity
def mxs_sensitivity_workspace_bytes(T: int, N: int, K: int) -> int:
    need = _SZ(0)
    _check(_lib.mxs_sensitivity_workspace_bytes(T, N, K, ctypes.byref(need)), "mxs_sensitivity_workspace_bytes")
    return need.value


def mxs_sensitivity(X: torch.Tensor, W: torch.Tensor, stream=None, workspace: Optional[torch.Tensor] = None,
                    out=None):
    """(H, E, s) fp64 device tensors for calibration X (T x K) and weight W (N x K)."""
    T, K = X.shape
    N, K2 = W.shape
    assert K == K2
    need = _SZ(mxs_sensitivity_workspace_bytes(T, N, K))
    ws = workspace if workspace is not None else _workspace(need.value, X.device)
    if out is None:
        H = torch.empty(K, dtype=torch.float64, device=X.device)
        E = torch.empty_like(H)
        s = torch.empty_like(H)
    else:
        H, E, s = out
    _check(_lib.mxs_sensitivity(X.data_ptr(), _dt(X), T, K, _rowmajor(X), W.data_ptr(), _dt(W), N,
                                _rowmajor(W), H.data_ptr(), E.data_ptr(), s.data_ptr(),
                                _aligned_ptr(ws), need.value, _stream(stream)), "mxs_sensitivity")
    return H, E, s


NOALLOC_SCRATCH_BYTES = 16 << 20


def mxs_sensitivity_noalloc(X: torch.Tensor, W: torch.Tensor, out, stream=None):
    """mxs_sensitivity with the library's fixed device scratch instead of a
    workspace; `out` = (H, E, s) caller-allocated fp64 tensors of K."""
    T, K = X.shape
    N, K2 = W.shape
    assert K == K2
    H, E, s = out
    _check(_lib.mxs_sensitivity_noalloc(X.data_ptr(), _dt(X), T, K, _rowmajor(X), W.data_ptr(), _dt(W), N,
                                        _rowmajor(W), H.data_ptr(), E.data_ptr(), s.data_ptr(), _stream(stream)),
           "mxs_sensitivity_noalloc")
    return H, E, s


# --------------------------------------------------------------- allocation
def make_budget(mode: str, budget=(9, 2), p8=(5, 100), p6=(15, 100), fixed8: int = 32) -> BudgetC:
    b = BudgetC()
    b.mode = {"fractions": MXS_ALLOC_FRACTIONS, "budget": MXS_ALLOC_BUDGET, "layer": MXS_ALLOC_LAYER}[mode]
    b.num, b.den = int(budget[0]), int(budget[1])
    b.p8_num, b.p8_den = int(p8[0]), int(p8[1])
    b.p6_num, b.p6_den = int(p6[0]), int(p6[1])
    b.fixed8 = int(fixed8)
    return b


def mxs_allocate(s_list: Sequence[torch.Tensor], N_list: Sequence[int], *, mode: str, budget=(9, 2),
                 p8=(5, 100), p6=(15, 100), fixed8: int = 32, layer_w=None, stream=None,
                 perms: Optional[List[torch.Tensor]] = None, workspace: Optional[torch.Tensor] = None):
    """Returns (perms: list of device int32 tensors, counts: list of (n8, n6, n4)).
    mode: "fractions", "budget" or "layer" (layer_w = the layer scores).
    Synchronises the stream only in multi-layer budget mode."""
    L = len(s_list)
    dev = s_list[0].device
    K = (ctypes.c_int64 * L)(*[int(s.numel()) for s in s_list])
    N = (ctypes.c_int64 * L)(*[int(n) for n in N_list])
    sp = (ctypes.c_void_p * L)(*[s.data_ptr() for s in s_list])
    if perms is None:
        perms = [torch.empty(int(s.numel()), dtype=torch.int32, device=dev) for s in s_list]
    pp = (ctypes.c_void_p * L)(*[p.data_ptr() for p in perms])
    counts = (ctypes.c_int64 * (3 * L))()
    w = None if layer_w is None else (ctypes.c_double * L)(*[float(x) for x in layer_w])
    need = _SZ(0)
    _check(_lib.mxs_allocate_workspace_bytes(L, K, ctypes.byref(need)), "mxs_allocate_workspace_bytes")
    ws = workspace if workspace is not None else _workspace(need.value, dev)
    b = make_budget(mode, budget, p8, p6, fixed8)
    _check(_lib.mxs_allocate(L, K, N, sp, w, ctypes.byref(b), pp, counts, _aligned_ptr(ws), need.value,
                             _stream(stream)), "mxs_allocate")
    return perms, [tuple(counts[3 * l:3 * l + 3]) for l in range(L)]


# --------------------------------------------------------------- quantisers
def _quantize(fn, name, src: torch.Tensor, out: MXTensor, stream):
    _check(fn(src.data_ptr(), _dt(src), src.shape[0], _rowmajor(src), ctypes.byref(out.c), _stream(stream)), name)
    return out


def mxs_quantize_weight(W: torch.Tensor, out: MXTensor, stream=None) -> MXTensor:
    return _quantize(_lib.mxs_quantize_weight, "mxs_quantize_weight", W, out, stream)


def mxs_quantize_act(A: torch.Tensor, out: MXTensor, stream=None) -> MXTensor:
    return _quantize(_lib.mxs_quantize_act, "mxs_quantize_act", A, out, stream)


def mxs_dequantize(t: MXTensor, stream=None) -> torch.Tensor:
    dev = next(x.device for x in t.codes if x is not None)
    out = torch.empty((t.rows, t.layout.K_pad), dtype=torch.float32, device=dev)
    _check(_lib.mxs_dequantize(ctypes.byref(t.c), out.data_ptr(), out.stride(0), _stream(stream)), "mxs_dequantize")
    return out


# -------------------------------------------------------------------- GEMM
def mxs_gemm_workspace_bytes(A: MXTensor, W: MXTensor) -> int:
    need = _SZ(0)
    _check(_lib.mxs_gemm_workspace_bytes(ctypes.byref(A.c), ctypes.byref(W.c), ctypes.byref(need)),
           "mxs_gemm_workspace_bytes")
    return need.value


def mxs_gemm(A: MXTensor, W: MXTensor, Y: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
             stream=None) -> torch.Tensor:
    dev = next(x.device for x in A.codes if x is not None)
    if Y is None:
        Y = torch.empty((A.rows, W.rows), dtype=torch.bfloat16, device=dev)
    need = mxs_gemm_workspace_bytes(A, W)
    ws = workspace if workspace is not None else _workspace(need, dev)
    _check(_lib.mxs_gemm(ctypes.byref(A.c), ctypes.byref(W.c), Y.data_ptr(), Y.stride(0), _aligned_ptr(ws), need,
                         _stream(stream)), "mxs_gemm")
    return Y


# -------------------------------------------------------- decode attention
def mxs_attn_decode_workspace_bytes(T: int, n_qh: int, n_kvh: int, d: int = 128) -> int:
    need = _SZ(0)
    _check(_lib.mxs_attn_decode_workspace_bytes(T, n_qh, n_kvh, d, ctypes.byref(need)),
           "mxs_attn_decode_workspace_bytes")
    return need.value


def mxs_attn_decode(q: torch.Tensor, K: MXTensor, V: MXTensor, T: int, n_kvh: int, sm_scale: float,
                    out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                    stream=None) -> torch.Tensor:
    """fp32 (n_qh x 128) output of one decode step of grouped-query attention
    over the MXINT4 K/V caches K and V (T*n_kvh rows each, token-major)."""
    if q.dtype != torch.bfloat16:
        raise TypeError("q must be bf16")
    n_qh = q.shape[0]
    if out is None:
        out = torch.empty((n_qh, q.shape[1]), dtype=torch.float32, device=q.device)
    need = mxs_attn_decode_workspace_bytes(T, n_qh, n_kvh, q.shape[1])
    ws = workspace if workspace is not None else _workspace(need, q.device)
    _check(_lib.mxs_attn_decode(q.data_ptr(), n_qh, _rowmajor(q), ctypes.byref(K.c), ctypes.byref(V.c), T, n_kvh,
                                float(sm_scale), out.data_ptr(), _rowmajor(out), _aligned_ptr(ws, 256), need,
                                _stream(stream)), "mxs_attn_decode")
    return out


# ------------------------------------------- serving around the K/V cache
# Every tensor of these calls must be on one device, which need not be the
# current one; memory the binding allocates is held for the stream it is used
# on.
class _On:
    """The stream handle and the device of a call; makes that device current
    for the call where it is not."""
    __slots__ = ("dev", "index", "stream", "given")

    def __init__(self, dev: torch.device, stream, others=()):
        if dev.type != "cuda":
            raise ValueError("expected CUDA tensors")
        for t in others:
            if t is not None and t.device != dev:
                raise ValueError(f"tensors on {dev} and {t.device}")
        index = dev.index
        self.dev, self.index, self.given = dev, index, stream is not None
        if stream is None:
            self.stream = _current_stream(index)
        else:
            self.stream = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)

    def call(self, f, *args) -> int:
        """f(*args) with the call's device current; its status."""
        cur = torch._C._cuda_getDevice()
        if cur == self.index:
            return f(*args)
        torch.cuda.set_device(self.index)
        try:
            return f(*args)
        finally:
            torch.cuda.set_device(cur)

    def empty(self, shape, dtype) -> torch.Tensor:
        """Memory for use on the call's stream."""
        if not self.given:
            return torch.empty(shape, dtype=dtype, device=self.dev)
        with torch.cuda.stream(torch.cuda.ExternalStream(self.stream, device=self.dev)):
            return torch.empty(shape, dtype=dtype, device=self.dev)

    def empty_like(self, t: torch.Tensor, dtype) -> torch.Tensor:
        """The same, of t's shape (cheaper to ask for)."""
        if not self.given:
            if dtype is None or dtype == t.dtype:
                return torch.empty_like(t, memory_format=torch.contiguous_format)
            return torch.empty_like(t, dtype=dtype, memory_format=torch.contiguous_format)
        return self.empty(t.shape, dtype or t.dtype)


# the current stream's handle by device index, without the object around it
_current_stream = torch._C._cuda_getCurrentRawStream


def _heads(t: torch.Tensor, what: str):
    s = t.stride()
    if len(s) != 3 or (s[2] != 1 and t.shape[2] > 1):
        raise ValueError(f"{what}: expected (tokens, heads, d) with unit stride along d")
    return s[0], s[1]


def _index(t: torch.Tensor, dtype, n: int, what: str) -> int:
    if t.dtype != dtype or t.dim() != 1 or t.numel() != n or not t.is_contiguous():
        raise ValueError(f"{what}: expected {n} contiguous {dtype} values")
    return t.data_ptr()


def _result(r, where: str):
    """What the extension gave: the call's results, or the status of its refusal."""
    if isinstance(r, int):
        raise MxsError(r, where)
    return r


_ROPE_KINDS = {"linear": 1, "parts": 2, "yarn": 3}


class RopePlan:
    """Frequencies of a rotary embedding (mxs_rope_plan_make)."""
    __slots__ = ("c", "ptr")

    def __init__(self, c: RopePlanC):
        self.c, self.ptr = c, ctypes.addressof(c)


def mxs_rope_plan(rot: int, theta: float = 500000.0, layout: str = "half", scaling: Optional[dict] = None) -> RopePlan:
    """Plan for the first `rot` positions of a head.  layout: "half" (pairs
    i, i + rot/2) or "interleaved" (2i, 2i + 1).  scaling: None, or a dict of
    kind "linear" (factor), "parts" (factor, low, high, orig_len) or "yarn"
    (factor, orig_len, beta_fast = 32, beta_slow = 1)."""
    layouts = {"half": 0, "interleaved": 1}
    if layout not in layouts:
        raise ValueError(f"unknown rope layout {layout!r}")
    sc = None
    if scaling is not None:
        p = dict(scaling)
        kind = p.pop("kind", None)
        if kind not in _ROPE_KINDS:
            raise ValueError(f"unknown rope scaling {kind!r}")
        if kind == "yarn":
            p["low"], p["high"] = p.pop("beta_slow", 1.0), p.pop("beta_fast", 32.0)
        need = {"factor"} if kind == "linear" else {"factor", "low", "high", "orig_len"}
        if set(p) != need:
            raise ValueError(f"rope scaling {kind!r} takes {sorted(need)}, got {sorted(p)}")
        sc = RopeScalingC(_ROPE_KINDS[kind], float(p["factor"]), float(p.get("low", 0.0)), float(p.get("high", 0.0)),
                          int(p.get("orig_len", 0)))
    c = RopePlanC()
    _check(_lib.mxs_rope_plan_make(int(rot), layouts[layout], float(theta),
                                   None if sc is None else ctypes.addressof(sc), ctypes.addressof(c)),
           "mxs_rope_plan_make")
    return RopePlan(c)


def mxs_rope(x: torch.Tensor, pos: torch.Tensor, plan: RopePlan, *, inverse: bool = False,
             dtype: Optional[torch.dtype] = None, out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """x (tokens, heads, d; bf16 or fp32) turned to its positions pos (int64),
    as `dtype` (x's by default); out may be x.  inverse turns back: the
    gradient of x from that of the result."""
    if _binding is not None and out is None and stream is None:
        r = _binding.rope(x, pos, plan.ptr, inverse, dtype)
        if r is not None:
            return _result(r, "mxs_rope")
    ldxt, ldxh = _heads(x, "x")
    T, heads, d = x.shape
    on = _On(x.device, stream, (pos, out))
    p = _index(pos, torch.int64, T, "pos")
    if out is None:
        out = on.empty_like(x, dtype)
        ldot, ldoh = heads * d, d
    else:
        if out.shape != x.shape or (dtype is not None and out.dtype != dtype):
            raise ValueError("out: another shape or type than asked for")
        ldot, ldoh = _heads(out, "out")
    st = on.call(_lib.mxs_rope, x.data_ptr(), _dt(x), T, heads, d, ldxt, ldxh, p, plan.ptr, bool(inverse),
                 out.data_ptr(), _dt(out), ldot, ldoh, on.stream)
    if st:
        raise MxsError(st, "mxs_rope")
    return out


class KVCache:
    """A pool of token slots: K and V are MXTensors of n_slots * n_kvh rows
    (row slot * n_kvh + head) in the same 4- or 8-bit identity layout."""

    def __init__(self, K: MXTensor, V: MXTensor, n_kvh: int):
        self.K, self.V, self.n_kvh = K, V, int(n_kvh)
        self.c = KVCacheC(K.c, V.c, int(n_kvh))
        self.ptr = ctypes.addressof(self.c)
        self.n_slots, self.d = K.rows // int(n_kvh), K.layout.K
        dev = [t.device for m in (K, V) for t in (*m.codes, *m.scales) if t is not None]
        self.device = dev[0] if dev else torch.device("cuda", torch.cuda.current_device())
        if any(x != self.device for x in dev):
            raise ValueError("K and V on different devices")
        self.index = -1 if self.device.index is None else self.device.index


def kv_cache_empty(n_slots: int, n_kvh: int, d: int, bits: int = 4, device="cuda") -> KVCache:
    """A cache of n_slots zeroed token slots; bits 4 or 8."""
    if bits not in (4, 8):
        raise ValueError("a K/V cache has 4 or 8 bits")
    lay = mxs_layout_make(d, (0, 0, d) if bits == 4 else (d, 0, 0))
    return KVCache(mxtensor_empty(n_slots * n_kvh, lay, device), mxtensor_empty(n_slots * n_kvh, lay, device), n_kvh)


def mxs_kv_write(k: torch.Tensor, v: torch.Tensor, cache: KVCache, slot: torch.Tensor, *,
                 pos: Optional[torch.Tensor] = None, rope: Optional[RopePlan] = None, stream=None) -> None:
    """Codes the tokens k, v (tokens, n_kvh, d) into their slots (int64; a
    negative one skips the token).  With `rope` the keys are turned to pos
    (int64) first."""
    if _binding is not None and stream is None:
        r = _binding.kv_write(k, v, cache.ptr, cache.index, slot, pos, None if rope is None else rope.ptr)
        if r is not None:
            return _check(r, "mxs_kv_write")
    ldkt, ldkh = _heads(k, "k")
    ldvt, ldvh = _heads(v, "v")
    T = k.shape[0]
    if k.shape != v.shape or k.shape[1:] != (cache.n_kvh, cache.d):
        raise ValueError(f"k, v: expected (tokens, {cache.n_kvh}, {cache.d})")
    if k.dtype != v.dtype:
        raise TypeError("k and v of different types")
    if (rope is None) != (pos is None):
        raise ValueError("rope and pos come together")
    on = _On(cache.device, stream, (k, v, slot, pos))
    s = _index(slot, torch.int64, T, "slot")
    p = None if pos is None else _index(pos, torch.int64, T, "pos")
    _check(on.call(_lib.mxs_kv_write, k.data_ptr(), ldkt, ldkh, v.data_ptr(), ldvt, ldvh, _dt(k), T, s, p,
                   None if rope is None else rope.ptr, cache.ptr, on.stream), "mxs_kv_write")


def mxs_kv_read(cache: KVCache, slot: torch.Tensor, *, dtype: torch.dtype = torch.bfloat16, out=None, stream=None):
    """(k, v), each (tokens, n_kvh, d): the values in the given slots (int64).
    A negative slot leaves its rows of `out` as they are (unspecified where
    the call makes them)."""
    if _binding is not None and out is None and stream is None:
        r = _binding.kv_read(cache.ptr, cache.index, slot, dtype)
        if r is not None:
            return _result(r, "mxs_kv_read")
    T = slot.numel()
    on = _On(cache.device, stream, (slot,) if out is None else (slot, *out))
    s = _index(slot, torch.int64, T, "slot")
    if out is None:
        h, d = cache.n_kvh, cache.d
        k = on.empty((T, h, d), dtype)
        v = on.empty_like(k, None)
        ldkt, ldkh = ldvt, ldvh = h * d, d
    else:
        k, v = out
        if k.shape != (T, cache.n_kvh, cache.d) or v.shape != k.shape or k.dtype != v.dtype:
            raise ValueError(f"out: expected two tensors of ({T}, {cache.n_kvh}, {cache.d}) and one type")
        ldkt, ldkh = _heads(k, "k")
        ldvt, ldvh = _heads(v, "v")
    st = on.call(_lib.mxs_kv_read, cache.ptr, T, s, k.data_ptr(), ldkt, ldkh, v.data_ptr(), ldvt, ldvh, _dt(k), on.stream)
    if st:
        raise MxsError(st, "mxs_kv_read")
    return k, v


class TreeBatch:
    """Drafted tokens of a batch of sequences over a paged cache."""
    __slots__ = ("c", "ptr", "rows", "tensors", "device", "index")

    def __init__(self, c: TreeBatchC, tensors):
        self.c, self.ptr, self.tensors = c, ctypes.addressof(c), tensors
        self.rows, self.device = int(c.rows), tensors[0].device
        self.index = -1 if self.device.index is None else self.device.index


def tree_batch(q_start: torch.Tensor, length: torch.Tensor, pages: torch.Tensor, page_size: int, *, max_q: int,
               max_len: int, mask: Optional[torch.Tensor] = None) -> TreeBatch:
    """q_start (B + 1) and length (B) int32, pages (B, per sequence) int32;
    mask: (rows, words) int32, bit j % 32 of word j / 32 set where the row
    sees drafted token j, or None for a chain.  max_q and max_len bound the
    drafted tokens and the tokens altogether of any sequence.  The tensors
    are read by each call, so their contents may change between calls.
    The batch covers q's rows as mask has them, else any number."""
    B = length.numel()
    if pages.dtype != torch.int32 or pages.dim() != 2 or pages.shape[0] != B or (pages.shape[1] > 1 and pages.stride(1) != 1):
        raise ValueError(f"pages: expected ({B}, pages of a sequence) int32 with unit stride")
    c = TreeBatchC(B, -1, int(max_q), int(max_len), _index(q_start, torch.int32, B + 1, "q_start"),
                   _index(length, torch.int32, B, "length"), pages.data_ptr(),
                   pages.stride(0) if B > 1 else pages.shape[1], int(page_size), None, 0)
    if mask is not None:
        if mask.dtype != torch.int32 or mask.dim() != 2 or (mask.shape[1] > 1 and mask.stride(1) != 1):
            raise ValueError("mask: expected (rows, words) int32 with unit stride")
        if mask.shape[1] * 32 < max_q:
            raise MxsError(2, "tree_batch")
        c.mask, c.ldm, c.rows = mask.data_ptr(), mask.stride(0) if mask.shape[0] > 1 else mask.shape[1], mask.shape[0]
    if max_len > page_size * pages.shape[1]:
        raise MxsError(2, "tree_batch")
    dev = length.device
    for t in (q_start, pages, mask):
        if t is not None and t.device != dev:
            raise ValueError(f"tensors on {dev} and {t.device}")
    return TreeBatch(c, (length, q_start, pages, mask))


def _tree_rows(q: torch.Tensor, batch: TreeBatch) -> TreeBatchC:
    c = batch.c
    if c.mask is not None:
        if batch.rows != q.shape[0]:
            raise ValueError(f"q has {q.shape[0]} rows, mask {batch.rows}")
    elif c.rows != q.shape[0]:
        c = TreeBatchC.from_buffer_copy(c)
        c.rows = q.shape[0]
    return c


def mxs_attn_tree_workspace_bytes(q: torch.Tensor, cache: KVCache, batch: TreeBatch,
                                  dtype: torch.dtype = torch.bfloat16) -> int:
    need = _SZ(0)
    c = _tree_rows(q, batch)
    _check(_lib.mxs_attn_tree_workspace_bytes(cache.ptr, ctypes.addressof(c), q.shape[1],
                                              MXS_F32 if dtype == torch.float32 else MXS_BF16,
                                              ctypes.addressof(need)), "mxs_attn_tree_workspace_bytes")
    return need.value


def attn_tree_workspace(q: torch.Tensor, cache: KVCache, batch: TreeBatch) -> torch.Tensor:
    """A workspace for mxs_attn_tree calls of these sizes, of either output
    type; calls that may overlap need one each."""
    return _workspace(max(mxs_attn_tree_workspace_bytes(q, cache, batch, t) for t in (torch.bfloat16, torch.float32)),
                      cache.device)


def mxs_attn_tree(q: torch.Tensor, cache: KVCache, batch: TreeBatch, sm_scale: float, *,
                  dtype: torch.dtype = torch.bfloat16, out: Optional[torch.Tensor] = None, return_lse: bool = False,
                  workspace: Optional[torch.Tensor] = None, stream=None):
    """Attention of the drafted tokens q (rows, n_qh, d) bf16 over the cache:
    (rows, n_qh, d) as `dtype` (bf16 or fp32), and with return_lse the fp32
    (rows, n_qh) logarithms of the sums.  Rows of no sequence stay as they
    are in `out` (unspecified where the call makes it)."""
    if q.dtype != torch.bfloat16:
        raise TypeError("q must be bf16")
    if _binding is not None and out is None and stream is None:
        r = _binding.attn_tree(q, cache.ptr, cache.index, batch.ptr, batch.index, sm_scale, dtype, return_lse, workspace)
        if r is not None:
            return _result(r, "mxs_attn_tree")
    ldqt, ldqh = _heads(q, "q")
    rows, n_qh, d = q.shape
    if d != cache.d:
        raise ValueError(f"q has heads of {d}, the cache of {cache.d}")
    on = _On(cache.device, stream, (q, out, workspace, batch))
    c = _tree_rows(q, batch)
    cp = ctypes.addressof(c)
    if out is None:
        out = on.empty_like(q, dtype)
        ldot, ldoh = n_qh * d, d
    elif out.shape != q.shape:
        raise ValueError("out: another shape than q")
    else:
        ldot, ldoh = _heads(out, "out")
    ot = _dt(out)
    if workspace is None:
        need = _SZ(0)
        _check(on.call(_lib.mxs_attn_tree_workspace_bytes, cache.ptr, cp, n_qh, ot, ctypes.addressof(need)), "mxs_attn_tree")
        workspace = on.empty(need.value + 1024, torch.uint8)
    ws = _aligned_ptr(workspace, 256)
    ws_bytes = workspace.numel() * workspace.element_size() - (ws - workspace.data_ptr())
    lse = on.empty((rows, n_qh), torch.float32) if return_lse else None
    st = on.call(_lib.mxs_attn_tree, q.data_ptr(), n_qh, ldqt, ldqh, cache.ptr, cp, sm_scale, out.data_ptr(), ot, ldot,
                 ldoh, None if lse is None else lse.data_ptr(), ws, max(ws_bytes, 0), on.stream)
    if st:
        raise MxsError(st, "mxs_attn_tree")
    return (out, lse) if return_lse else out


# ---------------------------------------------------------- layer scores
LINEARS = ("q", "k", "v", "o", "gate", "up", "down")


def _stack_c(blocks, hidden, n_heads, n_kv_heads, mlp, rms_eps, rope_theta):
    ptrs = (ctypes.c_void_p * (7 * len(blocks)))()
    for b, Ws in enumerate(blocks):
        for j, w in enumerate(Ws):
            if w.dtype != torch.bfloat16 or not w.is_contiguous():
                raise TypeError("stack weights must be contiguous bf16")
            ptrs[7 * b + j] = w.data_ptr()
    m = StackC(len(blocks), hidden, n_heads, n_kv_heads, mlp, rms_eps, rope_theta,
               ctypes.cast(ptrs, ctypes.c_void_p))
    return m, ptrs


def mxs_layer_scores_workspace_bytes(n_blocks: int, hidden: int, n_heads: int, n_kv_heads: int, mlp: int,
                                     T: int, rms_eps: float = 1e-5, rope_theta: float = 500000.0) -> int:
    m = StackC(n_blocks, hidden, n_heads, n_kv_heads, mlp, rms_eps, rope_theta, ctypes.c_void_p(1 << 20))
    need = _SZ(0)
    _check(_lib.mxs_layer_scores_workspace_bytes(ctypes.byref(m), T, ctypes.byref(need)),
           "mxs_layer_scores_workspace_bytes")
    return need.value


def mxs_layer_scores(x: torch.Tensor, blocks, *, n_heads: int, n_kv_heads: int, rms_eps: float = 1e-5,
                     rope_theta: float = 500000.0, workspace: Optional[torch.Tensor] = None, stream=None):
    """Layer-wise sensitivity scores (7 per block: q, k, v, o, gate, up, down)
    of the decoder stack `blocks` (a list of 7-tuples of bf16 weights) for the
    fp32 hidden states x (T x hidden).  Synchronises the stream."""
    import numpy as np
    T, hidden = x.shape
    mlp = blocks[0][4].shape[0]
    m, ptrs = _stack_c(blocks, hidden, n_heads, n_kv_heads, mlp, rms_eps, rope_theta)
    need = _SZ(0)
    _check(_lib.mxs_layer_scores_workspace_bytes(ctypes.byref(m), T, ctypes.byref(need)),
           "mxs_layer_scores_workspace_bytes")
    ws = workspace if workspace is not None else _workspace(need.value, x.device)
    out = np.zeros(7 * len(blocks))
    if x.dtype != torch.float32:
        raise TypeError("x must be fp32")
    _check(_lib.mxs_layer_scores(ctypes.byref(m), x.data_ptr(), T, _rowmajor(x),
                                 out.ctypes.data_as(ctypes.c_void_p), _aligned_ptr(ws, 256), need.value,
                                 _stream(stream)), "mxs_layer_scores")
    return out


def mxs_sync(stream=None) -> None:
    _check(_lib.mxs_sync(_stream(stream)), "mxs_sync")


def mxs_set_wait_limit(cycles: int) -> None:
    """Diagnostic: the spin limit (SM cycles) of the pipeline waits of the
    prefill GEMM and mxs_attn_tree kernels on the current device; 0 restores
    the default."""
    _check(_lib.mxs_set_wait_limit(int(cycles)), "mxs_set_wait_limit")


def mxs_launch_count() -> int:
    return int(_lib.mxs_launch_count())


def mxs_status_str(st: int) -> str:
    return _lib.mxs_status_str(st).decode()
