"""Residual-binary-weight linear layers on B200 (sm_100a).

A weight W (M x K) is stored as N bit-packed sign planes and scales,
W ~= sum_k alpha_k (.) B_k (RaBiT, arXiv 2602.05367, sections 4.1-4.2; QBB
grouped variant). This package is a thin binding over the C ABI of
``librb.so`` (include/rb_api.h): tensors are torch CUDA tensors, the stream is
torch's current stream, and every step of the computation runs in the
library's CUDA kernels.

    planes, alpha, alpha16 = pack(W, n_paths=2, group=0)
    y = gemv(planes, alpha, x, group=0)               # decode, T <= 64 tokens
    Y = gemm(planes, alpha, X, group=0)               # any batch, tcgen05 tensor cores

Backward pass, with the layer's input kept in 8 bits, and layers kept at 8 bits:

    c, s = pack8(X)                                   # e4m3 codes, a scale per 128 columns
    dX = gemm_dgrad(planes, alpha, dY, K)             # dY W^
    dW = gemm_wgrad(dY, c, s)                         # dY^T X
    Y = gemm8(*pack8(W, block_rows=128), c, s)
"""
from ._lib import RbError, load  # noqa: F401
from .api import (  # noqa: F401
    GroupedGemv,
    dual_gemv,
    gemm,
    gemm8,
    gemm_dgrad,
    gemm_from_weight,
    gemm_from_weight_workspace_bytes,
    gemm_wgrad,
    gemm_workspace_bytes,
    gemv,
    gemv_swiglu,
    gemv_swiglu_workspace_bytes,
    gemv_workspace_bytes,
    layout,
    mlp_gemv,
    pack,
    pack8,
    pack_fixed,
    planes_words,
    scales_count,
    unpack8,
)

__all__ = ["pack", "pack_fixed", "gemv", "gemv_swiglu", "mlp_gemv", "dual_gemv", "gemm", "gemm_from_weight",
           "GroupedGemv", "layout", "planes_words", "scales_count", "gemv_workspace_bytes",
           "gemv_swiglu_workspace_bytes", "gemm_workspace_bytes", "gemm_from_weight_workspace_bytes",
           "pack8", "unpack8", "gemm8", "gemm_wgrad", "gemm_dgrad", "RbError", "load"]
