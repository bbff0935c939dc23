"""Python entry points: marshal torch tensors into the C ABI of librb.so."""
from __future__ import annotations

import ctypes
from typing import Optional, Sequence

import torch

from . import _lib
from ._lib import GemvDesc, Layout, check

_DT = {torch.float32: _lib.RB_F32, torch.float16: _lib.RB_F16}


def _stream(device: torch.device) -> ctypes.c_void_p:
    return ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)


def _p(t: Optional[torch.Tensor]):
    return ctypes.c_void_p(t.data_ptr()) if t is not None else None


_ORDERS = {"rows": _lib.RB_ROWS, "sliced": _lib.RB_SLICED}


def layout(M: int, K: int, n_paths: int, group: int = 0, order: str = "rows") -> Layout:
    return Layout(M, K, n_paths, group, _ORDERS[order], 0)


def planes_words(M: int, K: int, n_paths: int, group: int = 0, order: str = "rows") -> int:
    return _lib.load().rb_planes_words(layout(M, K, n_paths, group, order))


def scales_count(M: int, K: int, n_paths: int, group: int = 0) -> int:
    return _lib.load().rb_scales_count(layout(M, K, n_paths, group))


def _planes_geometry(planes: torch.Tensor, K: int):
    """(N, M, order) of a planes tensor: [N, M, K/32] rows or [N, S, M, 16] sliced."""
    if planes.dim() == 3:
        N, M, W32 = planes.shape
        if W32 * 32 != K:
            raise ValueError("planes and x disagree on K")
        return N, M, "rows"
    if planes.dim() == 4:
        N, S, M, sixteen = planes.shape
        if sixteen != 16 or S != (K + 511) // 512:
            raise ValueError("sliced planes and x disagree on K")
        return N, M, "sliced"
    raise ValueError("planes must be [N, M, K/32] (rows) or [N, S, M, 16] (sliced)")


def _require_cuda(*ts: torch.Tensor) -> torch.device:
    dev = None
    for t in ts:
        if t is None:
            continue
        if not t.is_cuda:
            raise ValueError("tensors must live on a CUDA device")
        if dev is None:
            dev = t.device
        elif t.device != dev:
            raise ValueError("tensors are on different devices")
    return dev


def _mapped_host_ptr(t: torch.Tensor) -> int:
    """Device address of a pinned host tensor (the kernel writes it over the
    bus). Page-locked host memory is mapped into the device address space
    under unified addressing; the runtime is asked for the address rather
    than assuming it."""
    if t.is_cuda or not t.is_pinned():
        raise ValueError("expected a pinned host tensor")
    try:
        from cuda.bindings import runtime as rt
    except ImportError as e:   # pragma: no cover - cuda-python is part of the image
        raise ValueError("a pinned host output needs cuda-python (cuda.bindings)") from e
    base = t.untyped_storage().data_ptr()          # the allocation the runtime knows
    err, dptr = rt.cudaHostGetDevicePointer(base, 0)
    if int(err) != 0 or not dptr:
        raise ValueError(f"pinned host tensor is not mapped for the device (cudaHostGetDevicePointer: {err})")
    return int(dptr) + (t.data_ptr() - base)


def pack(W: torch.Tensor, n_paths: int = 2, group: int = 0, alpha_f16: bool = False, order: str = "rows",
         planes: Optional[torch.Tensor] = None, alpha: Optional[torch.Tensor] = None,
         alpha16: Optional[torch.Tensor] = None):
    """Derive N residual sign planes and scales from the shared weight W (M x K).

    Returns (planes, alpha fp32 [N, M, K/G], alpha16 fp16 [N, M, K/G] or None).
    planes holds uint32 words in an int32 tensor: [N, M, K/32] for
    order="rows", [N, ceil(K/512), M, 16] for order="sliced" (the order the
    matvec kernel streams fastest). Output tensors of those shapes may be
    passed in to be filled instead of allocated.
    """
    lib = _lib.load()
    dev = _require_cuda(W, planes, alpha, alpha16)
    if W.dim() != 2 or W.stride(1) != 1 or W.dtype not in _DT:
        raise ValueError("W must be a 2-D fp16/fp32 tensor with unit column stride")
    M, K = W.shape
    G = K if group == 0 else group
    shape = (n_paths, M, K // 32) if order == "rows" else (n_paths, (K + 511) // 512, M, 16)

    def out(t, shp, dt):
        if t is None:
            return torch.empty(shp, dtype=dt, device=dev)
        if tuple(t.shape) != tuple(shp) or t.dtype != dt or not t.is_contiguous():
            raise ValueError(f"output tensor must be contiguous {dt} of shape {shp}")
        return t
    planes = out(planes, shape, torch.int32)
    alpha = out(alpha, (n_paths, M, K // G), torch.float32)
    a16 = out(alpha16, (n_paths, M, K // G), torch.float16) if alpha_f16 else None
    with torch.cuda.device(dev):
        check(lib.rb_pack(_p(W), _DT[W.dtype], W.stride(0), layout(M, K, n_paths, group, order),
                          _p(planes), _p(alpha), _p(a16), _stream(dev)))
    return planes, alpha, a16


def gemv_workspace_bytes(M: int, K: int, n_paths: int, group: int, T: int) -> int:
    return _lib.load().rb_gemv_workspace_bytes(layout(M, K, n_paths, group), T)


def _x2d(x: torch.Tensor) -> torch.Tensor:
    if x.dim() == 1:
        x = x.unsqueeze(0)
    if x.dtype != torch.float16 or x.dim() != 2 or x.stride(1) != 1:
        raise ValueError("x must be fp16 [T, K] with unit column stride")
    return x


def gemv(planes: torch.Tensor, alpha: torch.Tensor, x: torch.Tensor, group: int = 0,
         y: Optional[torch.Tensor] = None, y_dtype: torch.dtype = torch.float16,
         workspace: Optional[torch.Tensor] = None, check_device: bool = False) -> torch.Tensor:
    """y[t] = sum_k alpha_k (.) (B_k x[t]) for T <= 64 tokens (CUDA-core table kernel).

    A caller-given workspace must have been zeroed once before its first use
    (torch.zeros); each call leaves it ready for the next. Without one, a
    zeroed workspace is allocated for the call. With check_device=True the
    call waits for the stream and raises if the kernel recorded a failure in
    its workspace (rb_gemv_check).
    """
    lib = _lib.load()
    x = _x2d(x)
    dev = _require_cuda(planes, alpha, x, y, workspace)
    K = x.shape[1]
    N, M, order = _planes_geometry(planes, K)
    T = x.shape[0]
    if y is None:
        y = torch.empty((T, M), dtype=y_dtype, device=dev)
    L = layout(M, K, N, group, order)
    need = lib.rb_gemv_workspace_bytes(L, T)
    if workspace is None or workspace.numel() * workspace.element_size() < need:
        workspace = torch.zeros(max(need, 16), dtype=torch.uint8, device=dev)
    with torch.cuda.device(dev):
        check(lib.rb_gemv(_p(planes), _p(alpha), _DT[alpha.dtype], L, _p(x), x.stride(0), T,
                          _p(y), _DT[y.dtype], y.stride(0), _p(workspace),
                          workspace.numel() * workspace.element_size(), _stream(dev)))
        if check_device:
            check(lib.rb_gemv_check(_p(workspace), _stream(dev)))
    return y


def gemv_swiglu_workspace_bytes(M: int, K: int, n_paths: int, group: int, T: int) -> int:
    return _lib.load().rb_gemv_swiglu_workspace_bytes(layout(M, K, n_paths, group), T)


def gemv_swiglu(planes: torch.Tensor, alpha: torch.Tensor, x: torch.Tensor, group: int = 0,
                h: Optional[torch.Tensor] = None, h_dtype: torch.dtype = torch.float16,
                workspace: Optional[torch.Tensor] = None, check_device: bool = False) -> torch.Tensor:
    """h[t] = silu(G x[t]) * (U x[t]) in one launch (rb_gemv_swiglu).

    planes / alpha hold the gate's N paths followed by the up projection's N
    paths (e.g. torch.cat of two pack() outputs along dim 0). The workspace
    contract is gemv()'s (zeroed once before its first use).
    """
    lib = _lib.load()
    x = _x2d(x)
    dev = _require_cuda(planes, alpha, x, h, workspace)
    K = x.shape[1]
    N2, M, order = _planes_geometry(planes, K)
    if N2 % 2:
        raise ValueError("planes must hold the gate's and the up projection's paths (an even count)")
    T = x.shape[0]
    if h is None:
        h = torch.empty((T, M), dtype=h_dtype, device=dev)
    L = layout(M, K, N2 // 2, group, order)
    need = lib.rb_gemv_swiglu_workspace_bytes(L, T)
    if workspace is None or workspace.numel() * workspace.element_size() < need:
        workspace = torch.zeros(max(need, 16), dtype=torch.uint8, device=dev)
    with torch.cuda.device(dev):
        check(lib.rb_gemv_swiglu(_p(planes), _p(alpha), _DT[alpha.dtype], L, _p(x), x.stride(0), T,
                                 _p(h), _DT[h.dtype], h.stride(0), _p(workspace),
                                 workspace.numel() * workspace.element_size(), _stream(dev)))
        if check_device:
            check(lib.rb_gemv_check(_p(workspace), _stream(dev)))
    return h


def mlp_gemv(gu_planes: torch.Tensor, gu_alpha: torch.Tensor, d_planes: torch.Tensor, d_alpha: torch.Tensor,
             x: torch.Tensor, group: int = 0, y: Optional[torch.Tensor] = None,
             workspace: Optional[torch.Tensor] = None, check_device: bool = False):
    """The gated MLP block for decode tokens: y = D (silu(G x) * (U x)).

    Two launches on the current stream: rb_gemv_swiglu (gate and up, gated
    in the epilogue, h in fp16) and rb_gemv for the down projection D.
    Returns (y, h). One workspace (zeroed once) serves both launches.
    """
    x = _x2d(x)
    K = x.shape[1]
    _, M, order = _planes_geometry(gu_planes, K)
    Nd, Md, _ = _planes_geometry(d_planes, M)
    T = x.shape[0]
    need = max(gemv_swiglu_workspace_bytes(M, K, gu_planes.shape[0] // 2, group, T),
               gemv_workspace_bytes(Md, M, Nd, group, T), 16)
    if workspace is None or workspace.numel() * workspace.element_size() < need:
        workspace = torch.zeros(need, dtype=torch.uint8, device=x.device)
    h = gemv_swiglu(gu_planes, gu_alpha, x, group=group, workspace=workspace, check_device=check_device)
    y = gemv(d_planes, d_alpha, h, group=group, y=y, workspace=workspace, check_device=check_device)
    return y, h


class GroupedGemv:
    """One persistent launch over many (planes, alpha, x, y) matrices.

    The descriptor table is uploaded once at construction; call ``run()`` for
    every step (the x tensors are read and the y tensors written in place).
    An x or y tensor may also be a pinned host tensor: the kernel then reads
    x from, or writes y to, host memory over the bus (zero-copy), so a step
    needs no separate host-to-device or device-to-host copy.
    """

    def __init__(self, items: Sequence[tuple], n_paths: int, group: int = 0, T: int = 1):
        lib = _lib.load()
        self.n_paths, self.group, self.T = n_paths, group, T
        self.items = list(items)   # keep tensors alive
        n = len(self.items)
        self.host = (GemvDesc * n)()
        adt = ydt = order = None
        dev = None
        for i, (planes, alpha, x, y) in enumerate(self.items):
            host_x = not x.is_cuda and x.is_pinned()
            host_y = not y.is_cuda and y.is_pinned()
            dev = _require_cuda(planes, alpha, None if host_x else x, None if host_y else y)
            K = x.shape[-1]
            N, M, o = _planes_geometry(planes, K)
            order = o if order is None else order
            if N != n_paths or y.shape[-1] != M or o != order:
                raise ValueError(f"item {i}: inconsistent shapes or plane orders")
            if not (x.is_contiguous() and y.is_contiguous()):
                raise ValueError(f"item {i}: x and y must be contiguous [T, K] / [T, M]")
            # the descriptors are dense [T][K] / [T][M]: exactly T rows each
            if x.numel() != T * K or y.numel() != T * M:
                raise ValueError(f"item {i}: x must hold {T} x {K} and y {T} x {M} values")
            adt = alpha.dtype if adt is None else adt
            ydt = y.dtype if ydt is None else ydt
            if alpha.dtype != adt or y.dtype != ydt:
                raise ValueError("all items must share the scale and output dtypes")
            x_ptr = x.data_ptr() if x.is_cuda else _mapped_host_ptr(x)
            y_ptr = y.data_ptr() if y.is_cuda else _mapped_host_ptr(y)
            self.host[i] = GemvDesc(planes.data_ptr(), alpha.data_ptr(), x_ptr, y_ptr, M, K)
        self.device = dev
        raw = bytes(self.host)
        self.dev_descs = torch.frombuffer(bytearray(raw), dtype=torch.uint8).to(dev)
        self.alpha_dtype, self.y_dtype = _DT[adt], _DT[ydt]
        self.order = _ORDERS[order]
        need = lib.rb_gemv_grouped_workspace_bytes(self.host, n, n_paths, T)
        self.workspace = torch.zeros(max(need, 16), dtype=torch.uint8, device=dev)
        self.n = n

    def run(self) -> None:
        lib = _lib.load()
        with torch.cuda.device(self.device):
            check(lib.rb_gemv_grouped(ctypes.cast(self.host, ctypes.c_void_p), _p(self.dev_descs), self.n,
                                      self.n_paths, self.group, self.order, self.alpha_dtype, self.y_dtype, self.T,
                                      _p(self.workspace), self.workspace.numel(), _stream(self.device)))

    def check_device_flag(self) -> None:
        check(_lib.load().rb_gemv_check(_p(self.workspace), _stream(self.device)))


def gemm_workspace_bytes(M: int, K: int, n_paths: int, group: int, T: int) -> int:
    return _lib.load().rb_gemm_workspace_bytes(layout(M, K, n_paths, group), T)


def gemm(planes: torch.Tensor, alpha: torch.Tensor, X: torch.Tensor, group: int = 0,
         Y: Optional[torch.Tensor] = None, y_dtype: torch.dtype = torch.float16,
         workspace: Optional[torch.Tensor] = None, check_device: bool = False,
         reconstruct: bool = False) -> torch.Tensor:
    """Y[t] = sum_k alpha_k (.) (B_k X[t]) on the tcgen05 tensor cores (any T).

    reconstruct=True (two paths, per-row scales): one fp16 operand
    RN(alpha_0 B_0 + alpha_1 B_1) per weight and one MMA chain
    (rb_gemm_reconstruct). With check_device=True the call waits for the
    stream and raises if a kernel recorded a failure in its workspace
    (rb_gemm_check).
    """
    lib = _lib.load()
    X = _x2d(X)
    dev = _require_cuda(planes, alpha, X, Y, workspace)
    K = X.shape[1]
    N, M, order = _planes_geometry(planes, K)
    T = X.shape[0]
    if Y is None:
        Y = torch.empty((T, M), dtype=y_dtype, device=dev)
    L = layout(M, K, N, group, order)
    need = 256 if reconstruct else lib.rb_gemm_workspace_bytes(L, T)
    if workspace is None or workspace.numel() * workspace.element_size() < need:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=dev)
    fn = lib.rb_gemm_reconstruct if reconstruct else lib.rb_gemm
    with torch.cuda.device(dev):
        check(fn(_p(planes), _p(alpha), _DT[alpha.dtype], L, _p(X), X.stride(0), T,
                 _p(Y), _DT[Y.dtype], Y.stride(0), _p(workspace),
                 workspace.numel() * workspace.element_size(), _stream(dev)))
        if check_device:
            check(lib.rb_gemm_check(_p(workspace), _stream(dev)))
    return Y


def gemm_from_weight_workspace_bytes(M: int, K: int, n_paths: int, group: int, T: int, order: str = "sliced") -> int:
    return _lib.load().rb_gemm_from_weight_workspace_bytes(layout(M, K, n_paths, group, order), T)


def gemm_from_weight(W: torch.Tensor, X: torch.Tensor, n_paths: int = 2, group: int = 0, order: str = "sliced",
                     Y: Optional[torch.Tensor] = None, y_dtype: torch.dtype = torch.float16,
                     workspace: Optional[torch.Tensor] = None, check_device: bool = False) -> torch.Tensor:
    """Training forward: Y[t] = sum_k alpha_k (.) (B_k X[t]) with the planes
    and scales derived afresh from the full-precision weight W (M x K) in the
    same call (rb_gemm_from_weight: pack into the workspace, then rb_gemm)."""
    lib = _lib.load()
    X = _x2d(X)
    dev = _require_cuda(W, X, Y, workspace)
    if W.dim() != 2 or W.stride(1) != 1 or W.dtype not in _DT:
        raise ValueError("W must be a 2-D fp16/fp32 tensor with unit column stride")
    M, K = W.shape
    if X.shape[1] != K:
        raise ValueError("X must have K columns")
    T = X.shape[0]
    if Y is None:
        Y = torch.empty((T, M), dtype=y_dtype, device=dev)
    L = layout(M, K, n_paths, group, order)
    need = lib.rb_gemm_from_weight_workspace_bytes(L, T)
    if workspace is None or workspace.numel() * workspace.element_size() < need:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=dev)
    with torch.cuda.device(dev):
        check(lib.rb_gemm_from_weight(_p(W), _DT[W.dtype], W.stride(0), L, _p(X), X.stride(0), T, _p(Y),
                                      _DT[Y.dtype], Y.stride(0), _p(workspace),
                                      workspace.numel() * workspace.element_size(), _stream(dev)))
        if check_device:
            check(lib.rb_gemm_check(_p(workspace), _stream(dev)))
    return Y


def pack_fixed(W: torch.Tensor, h: torch.Tensor, g: Optional[torch.Tensor] = None, order: str = "rows",
               planes: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Sign planes of the dual-scale block for given scales: h fp32 [N, M]
    (output channels), g fp32 [N, K] (input channels) or None.
    B_k = sign(R_{k-1}), R_k = R_{k-1} - h_k[i] g_k[j] B_k."""
    lib = _lib.load()
    dev = _require_cuda(W, h, g, planes)
    if W.dim() != 2 or W.stride(1) != 1 or W.dtype not in _DT:
        raise ValueError("W must be a 2-D fp16/fp32 tensor with unit column stride")
    M, K = W.shape
    N = h.shape[0]
    if h.shape != (N, M) or h.dtype != torch.float32 or not h.is_contiguous():
        raise ValueError("h must be contiguous fp32 [N, M]")
    if g is not None and (g.shape != (N, K) or g.dtype != torch.float32 or not g.is_contiguous()):
        raise ValueError("g must be contiguous fp32 [N, K]")
    shape = (N, M, K // 32) if order == "rows" else (N, (K + 511) // 512, M, 16)
    if planes is None:
        planes = torch.empty(shape, dtype=torch.int32, device=dev)
    elif tuple(planes.shape) != shape or planes.dtype != torch.int32 or not planes.is_contiguous():
        raise ValueError(f"planes must be contiguous int32 of shape {shape}")
    with torch.cuda.device(dev):
        check(lib.rb_pack_fixed(_p(W), _DT[W.dtype], W.stride(0), layout(M, K, N, 0, order), _p(h), _p(g),
                                _p(planes), _stream(dev)))
    return planes


def dual_gemv(planes: torch.Tensor, h: torch.Tensor, g: Optional[torch.Tensor], x: torch.Tensor,
              y: Optional[torch.Tensor] = None, y_dtype: torch.dtype = torch.float16,
              workspace: Optional[torch.Tensor] = None, check_device: bool = False) -> torch.Tensor:
    """y[t] = sum_k h_k (.) (B_k RN_fp16(g_k (.) x[t])) for T <= 64 tokens."""
    lib = _lib.load()
    x = _x2d(x)
    dev = _require_cuda(planes, h, g, x, y, workspace)
    K = x.shape[1]
    N, M, order = _planes_geometry(planes, K)
    T = x.shape[0]
    if h.shape != (N, M) or h.dtype != torch.float32 or not h.is_contiguous():
        raise ValueError("h must be contiguous fp32 [N, M]")
    if g is not None and (g.shape != (N, K) or g.dtype != torch.float32 or not g.is_contiguous()):
        raise ValueError("g must be contiguous fp32 [N, K]")
    if y is None:
        y = torch.empty((T, M), dtype=y_dtype, device=dev)
    L = layout(M, K, N, 0, order)
    need = lib.rb_dual_gemv_workspace_bytes(L, T)
    if workspace is None or workspace.numel() * workspace.element_size() < need:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=dev)
    with torch.cuda.device(dev):
        check(lib.rb_dual_gemv(_p(planes), L, _p(h), _p(g), _p(x), x.stride(0), T, _p(y), _DT[y.dtype], y.stride(0),
                               _p(workspace), workspace.numel() * workspace.element_size(), _stream(dev)))
        if check_device:
            check(lib.rb_gemv_check(_p(workspace), _stream(dev)))
    return y


_DT8 = {torch.float32: _lib.RB_F32, torch.float16: _lib.RB_F16, torch.bfloat16: _lib.RB_BF16}
_E4M3 = torch.float8_e4m3fn
_GRAD_DT = (torch.float16, torch.bfloat16)
# A small call lasts a few microseconds on the GPU, so what surrounds it here
# counts: the raw stream handle is taken without a Stream object around it.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)

_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _call(dev: torch.device, fn, *args) -> None:
    """fn(*args, stream) on the current stream of `dev`, whichever device is current."""
    index = dev.index
    if _current_device() == index:
        status = fn(*args, _raw_stream(index))
    else:
        with torch.cuda.device(index):
            status = fn(*args, _raw_stream(index))
    if status:
        check(status)


def _cuda_device(*ts: Optional[torch.Tensor]) -> torch.device:
    """The one CUDA device that all tensors given are on."""
    dev = None
    for t in ts:
        if t is not None:
            d = t.device
            if dev is None:
                if d.type != "cuda":
                    raise ValueError("tensors must live on a CUDA device")
                dev = d
            elif d != dev:
                raise ValueError("tensors must live on one CUDA device")
    return dev


def _matrix(t: torch.Tensor, name: str, shape=None, dtypes=None) -> None:
    """Refuses t unless it is a 2-D tensor with unit column stride and rows that do not overlap."""
    if t.dim() != 2 or (shape is not None and t.shape != shape):
        raise ValueError(f"{name} must be a 2-D tensor" + (f" of shape {tuple(shape)}" if shape else ""))
    if dtypes is not None and t.dtype not in dtypes:
        raise ValueError(f"{name} has dtype {t.dtype}")
    if not t.is_contiguous() and ((t.stride(1) != 1 and t.shape[1] > 1) or (t.shape[0] > 1 and t.stride(0) < t.shape[1])):
        raise ValueError(f"{name} must have unit column stride and rows that do not overlap")


def _pitch(t: torch.Tensor) -> int:
    # the stride of a single row says nothing (torch may give any value): its
    # columns, rounded up to a 16-byte pitch
    return t.stride(0) if t.shape[0] > 1 else -(-t.shape[1] // 8) * 8


def _blocks8(codes: torch.Tensor, scales: torch.Tensor, block_rows: int, what: str):
    """(rows, K) of e4m3 codes [rows, K] with fp32 scales [ceil(rows / block_rows), K / 128]."""
    if codes.dtype != _E4M3 or codes.dim() != 2 or not codes.is_contiguous():
        raise ValueError(f"{what}: codes must be contiguous float8_e4m3fn [rows, K]")
    rows, K = codes.shape
    if block_rows not in (1, 128):
        raise ValueError(f"{what}: block_rows must be 1 or 128")
    if K % 128:
        raise ValueError(f"{what}: K={K} is not a multiple of 128")
    shape = (-(-rows // block_rows), K // 128)
    if scales.shape != shape or scales.dtype != torch.float32 or not scales.is_contiguous():
        raise ValueError(f"{what}: scales must be contiguous fp32 of shape {shape}")
    return rows, K


def _header(workspace: Optional[torch.Tensor], check_device: bool, dev: torch.device):
    """(workspace, its address, its bytes): the caller's, one for check_device, or none."""
    if workspace is None:
        if not check_device:
            return None, None, 0
        workspace = torch.empty(256, dtype=torch.uint8, device=dev)
    return workspace, workspace.data_ptr(), workspace.numel() * workspace.element_size()


def pack8(X: torch.Tensor, block_rows: int = 1, codes: Optional[torch.Tensor] = None,
          scales: Optional[torch.Tensor] = None):
    """e4m3 codes of X (fp16, bf16 or fp32 [rows, K]) with one power-of-two
    scale per 128 columns of a row (block_rows=1: activations, and their
    checkpoints) or per 128 x 128 block (block_rows=128: weights).

    Returns (codes float8_e4m3fn [rows, K], scales fp32
    [ceil(rows / block_rows), K / 128]); X ~= codes * scales. Output tensors of
    those shapes may be passed in to be filled. Values that are not finite
    become NaN codes and leave their block's scale alone.
    """
    lib = _lib._lib or _lib.load()
    dev = _cuda_device(X, codes, scales)
    _matrix(X, "X", dtypes=_DT8)
    rows, K = X.shape
    if block_rows not in (1, 128):
        raise ValueError("block_rows must be 1 or 128")
    given = codes is not None or scales is not None
    if codes is None:
        codes = torch.empty(rows, K, dtype=_E4M3, device=dev)
    if scales is None:
        scales = torch.empty(-(-rows // block_rows), K // 128, dtype=torch.float32, device=dev)
    if given and (_blocks8(codes, scales, block_rows, "pack8") != (rows, K)):
        raise ValueError(f"codes must have shape {(rows, K)}")
    _call(dev, lib.rb_pack8, X.data_ptr(), _DT8[X.dtype], _pitch(X), rows, K, block_rows, codes.data_ptr(),
          scales.data_ptr())
    return codes, scales


def unpack8(codes: torch.Tensor, scales: torch.Tensor, block_rows: int = 1, dtype: torch.dtype = torch.float16,
            X: Optional[torch.Tensor] = None) -> torch.Tensor:
    """X = codes * scales in `dtype` (fp16, bf16 or fp32; X's own where X is given)."""
    lib = _lib._lib or _lib.load()
    dev = _cuda_device(codes, scales, X)
    rows, K = _blocks8(codes, scales, block_rows, "unpack8")
    if X is None:
        if dtype not in _DT8:
            raise ValueError(f"dtype {dtype}")
        X = torch.empty(rows, K, dtype=dtype, device=dev)
    else:
        _matrix(X, "X", (rows, K), _DT8)
    _call(dev, lib.rb_unpack8, codes.data_ptr(), scales.data_ptr(), rows, K, block_rows, X.data_ptr(), _DT8[X.dtype],
          _pitch(X))
    return X


def gemm8(w: torch.Tensor, w_scales: torch.Tensor, x: torch.Tensor, x_scales: torch.Tensor,
          Y: Optional[torch.Tensor] = None, y_dtype: torch.dtype = torch.float16, pow2_scales: bool = True,
          workspace: Optional[torch.Tensor] = None, check_device: bool = False) -> torch.Tensor:
    """Y[t] = W x[t] from 8-bit blocks: w, w_scales = pack8(W, block_rows=128),
    x, x_scales = pack8(X). Any number of tokens.

    pow2_scales=True takes scales as pack8 writes them, powers of two, which
    the tensor cores apply; a scale that is none makes the outputs that it
    enters NaN (and check_device raise). pow2_scales=False takes any fp32
    scales. With check_device=True the call waits for the stream and raises
    if the kernel recorded a failure (rb_gemm_check)."""
    lib = _lib._lib or _lib.load()
    dev = _cuda_device(w, w_scales, x, x_scales, Y, workspace)
    M, K = _blocks8(w, w_scales, 128, "w")
    T, Kx = _blocks8(x, x_scales, 1, "x")
    if Kx != K:
        raise ValueError("w and x disagree on K")
    if Y is None:
        if y_dtype not in _DT8:
            raise ValueError(f"y_dtype {y_dtype}")
        Y = torch.empty(T, M, dtype=y_dtype, device=dev)
    else:
        _matrix(Y, "Y", (T, M), _DT8)
    workspace, ws, ws_bytes = _header(workspace, check_device, dev)
    _call(dev, lib.rb_gemm8, w.data_ptr(), w_scales.data_ptr(), x.data_ptr(), x_scales.data_ptr(), M, K, T,
          1 if pow2_scales else 0, Y.data_ptr(), _DT8[Y.dtype], _pitch(Y), ws, ws_bytes)
    if check_device:
        _call(dev, lib.rb_gemm_check, ws)
    return Y


def gemm_wgrad(dY: torch.Tensor, codes: torch.Tensor, scales: torch.Tensor, add: Optional[torch.Tensor] = None,
               dW: Optional[torch.Tensor] = None, dw_dtype: torch.dtype = torch.float32,
               workspace: Optional[torch.Tensor] = None, check_device: bool = False) -> torch.Tensor:
    """Weight gradient from an 8-bit checkpoint of the layer's input:
    dW = add + dY^T X with dY fp16 or bf16 [T, M] and codes, scales = pack8(X).

    `add` (of dW's type and row pitch) is dW itself (gradients summed over
    micro-batches) or apart from it. The products see X rounded to dY's type
    (exact for a checkpoint of a tensor of that type); sums are fp32, and dW is
    rounded once (fp32 dW: once for each 1024 or 2048 tokens, and sums below
    2^-126 may become zero).

    dY's rows must start on 16-byte boundaries. Where M is not a multiple of 8,
    that takes a buffer with longer rows, torch.empty(T, -(-M // 8) * 8)[:, :M].
    """
    lib = _lib._lib or _lib.load()
    dev = _cuda_device(dY, codes, scales, add, dW, workspace)
    T, K = _blocks8(codes, scales, 1, "checkpoint")
    _matrix(dY, "dY", dtypes=_GRAD_DT)
    if dY.shape[0] != T:
        raise ValueError("dY and the checkpoint disagree on the number of tokens")
    M = dY.shape[1]
    if dW is None:
        dt = dw_dtype if add is None else add.dtype
        if dt not in _DT8:
            raise ValueError(f"dw_dtype {dt}")
        dW = torch.empty(M, K, dtype=dt, device=dev)
    else:
        _matrix(dW, "dW", (M, K), _DT8)
    if add is not None:
        _matrix(add, "add", (M, K), (dW.dtype,))
        if _pitch(add) != _pitch(dW):
            raise ValueError("add must have dW's row pitch")
    workspace, ws, ws_bytes = _header(workspace, check_device, dev)
    _call(dev, lib.rb_gemm_wgrad, dY.data_ptr(), _DT8[dY.dtype], _pitch(dY), M, codes.data_ptr(), scales.data_ptr(), K, T,
          None if add is None else add.data_ptr(), dW.data_ptr(), _DT8[dW.dtype], _pitch(dW), ws, ws_bytes)
    if check_device:
        _call(dev, lib.rb_gemm_check, ws)
    return dW


def gemm_dgrad(planes: torch.Tensor, alpha: torch.Tensor, dY: torch.Tensor, K: int, group: int = 0,
               dX: Optional[torch.Tensor] = None, dx_dtype: torch.dtype = torch.float16,
               workspace: Optional[torch.Tensor] = None, check_device: bool = False) -> torch.Tensor:
    """Gradient of gemm() with respect to its input: dX = dY W^ with
    W^ = sum_k alpha_k (.) B_k taken straight from the planes, dY fp16 or bf16
    [T, M]. K is the layer's input width (sliced planes are padded to 512
    columns, so they do not say it).

    W^ is rounded once to dY's type (so dX is within eps / 2 of the sum of its
    terms' magnitudes); sums are fp32. dY's rows must start on 16-byte boundaries, as
    gemm_wgrad's."""
    lib = _lib._lib or _lib.load()
    dev = _cuda_device(planes, alpha, dY, dX, workspace)
    N, M, order = _planes_geometry(planes, K)
    if planes.dtype != torch.int32 or not planes.is_contiguous():
        raise ValueError("planes must be contiguous int32")
    G = K if group == 0 else group
    if alpha.dtype not in _DT or tuple(alpha.shape) != (N, M, K // G) or not alpha.is_contiguous():
        raise ValueError(f"alpha must be contiguous fp16 or fp32 of shape {(N, M, K // G)}")
    _matrix(dY, "dY", dtypes=_GRAD_DT)
    if dY.shape[1] != M:
        raise ValueError("dY must have M columns")
    T = dY.shape[0]
    if dX is None:
        if dx_dtype not in _DT8:
            raise ValueError(f"dx_dtype {dx_dtype}")
        dX = torch.empty(T, K, dtype=dx_dtype, device=dev)
    else:
        _matrix(dX, "dX", (T, K), _DT8)
    workspace, ws, ws_bytes = _header(workspace, check_device, dev)
    _call(dev, lib.rb_gemm_dgrad, planes.data_ptr(), alpha.data_ptr(), _DT[alpha.dtype], layout(M, K, N, group, order),
          dY.data_ptr(), _DT8[dY.dtype], _pitch(dY), T, dX.data_ptr(), _DT8[dX.dtype], _pitch(dX), ws, ws_bytes)
    if check_device:
        _call(dev, lib.rb_gemm_check, ws)
    return dX
