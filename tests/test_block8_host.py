"""Refusals of the 8-bit block and gradient calls before anything is enqueued (CPU)."""
import ctypes

import pytest
import torch

import residual_binary_weight_b200 as rb
from residual_binary_weight_b200 import _lib
from residual_binary_weight_b200._lib import Layout

FAKE = 1 << 40          # a 16-byte aligned address that is never dereferenced
F32, F16, BF16 = 0, 1, 2


def _caller(fn, names, ok):
    def call(**kw):
        args = [kw.get(n, v) for n, v in zip(names, ok)]
        assert set(kw) <= set(names)
        args = [ctypes.c_void_p(a) if isinstance(a, int) and a >= FAKE else a for a in args]
        return _lib.STATUS_NAMES[getattr(_lib.load(), fn)(*args)]
    return call


def test_pack8_refusals():
    call = _caller("rb_pack8", ["X", "dt", "ldx", "rows", "K", "br", "codes", "scales", "s"],
                   (FAKE, F16, 256, 3, 256, 1, FAKE, FAKE, None))
    for k in ("X", "codes", "scales"):
        assert call(**{k: None}) == "RB_ERR_INVALID_ARG", k
    assert call(dt=3) == call(dt=-1) == "RB_ERR_INVALID_ARG"
    assert call(rows=0) == call(rows=-1) == call(K=0) == "RB_ERR_INVALID_ARG"
    assert call(K=200, ldx=256) == "RB_ERR_UNSUPPORTED"
    assert call(br=0) == call(br=64) == "RB_ERR_UNSUPPORTED"
    assert call(ldx=255) == "RB_ERR_INVALID_ARG"
    assert call(ldx=260) == "RB_ERR_ALIGNMENT"
    assert call(ldx=258, dt=F32) == "RB_ERR_ALIGNMENT"
    assert call(X=FAKE + 2) == call(codes=FAKE + 8) == call(scales=FAKE + 2) == "RB_ERR_ALIGNMENT"
    assert call(rows=1 << 31) == "RB_ERR_UNSUPPORTED"
    assert call(rows=1 << 30, K=256) == "RB_ERR_UNSUPPORTED"
    call(K=200, ldx=256)
    assert b"multiple of 128" in _lib.load().rb_last_error()


def test_unpack8_refusals():
    call = _caller("rb_unpack8", ["codes", "scales", "rows", "K", "br", "X", "dt", "ldx", "s"],
                   (FAKE, FAKE, 3, 256, 1, FAKE, F16, 256, None))
    for k in ("X", "codes", "scales"):
        assert call(**{k: None}) == "RB_ERR_INVALID_ARG", k
    assert call(dt=3) == call(rows=0) == call(ldx=128) == "RB_ERR_INVALID_ARG"
    assert call(K=130, ldx=256) == call(br=2) == "RB_ERR_UNSUPPORTED"
    assert call(ldx=260) == call(X=FAKE + 8) == call(codes=FAKE + 1) == call(scales=FAKE + 1) == "RB_ERR_ALIGNMENT"


def test_gemm8_refusals():
    call = _caller("rb_gemm8", ["w", "ws", "x", "xs", "M", "K", "T", "p2", "Y", "dt", "ldy", "wk", "wb", "s"],
                   (FAKE, FAKE, FAKE, FAKE, 100, 256, 5, 1, FAKE, F16, 100, FAKE, 256, None))
    for k in ("w", "ws", "x", "xs", "Y"):
        assert call(**{k: None}) == "RB_ERR_INVALID_ARG", k
    assert call(dt=3) == call(M=0) == call(ldy=99) == call(p2=2) == "RB_ERR_INVALID_ARG"
    assert call(T=0) == call(T=(1 << 22) + 1) == call(K=64) == "RB_ERR_UNSUPPORTED"
    assert call(w=FAKE + 4) == call(x=FAKE + 8) == call(ws=FAKE + 2) == call(xs=FAKE + 1) == "RB_ERR_ALIGNMENT"
    assert call(Y=FAKE + 1) == call(Y=FAKE + 2, dt=F32) == "RB_ERR_ALIGNMENT"
    assert call(wb=255) == call(wk=FAKE + 8) == "RB_ERR_WORKSPACE"
    assert call(T=1 << 22, M=1 << 24, K=128, ldy=1 << 24) == "RB_ERR_UNSUPPORTED"


def test_wgrad_refusals():
    call = _caller("rb_gemm_wgrad",
                   ["dY", "ddt", "ldd", "M", "codes", "scales", "K", "T", "add", "dW", "dt", "ldw", "wk", "wb", "s"],
                   (FAKE, F16, 104, 100, FAKE, FAKE, 256, 5, None, FAKE, F32, 256, FAKE, 256, None))
    for k in ("dY", "codes", "scales", "dW"):
        assert call(**{k: None}) == "RB_ERR_INVALID_ARG", k
    assert call(ddt=F32) == "RB_ERR_UNSUPPORTED"
    assert call(ddt=7) == call(dt=3) == call(M=0) == call(ldd=96) == call(ldw=255) == "RB_ERR_INVALID_ARG"
    assert call(T=0) == call(T=(1 << 22) + 1) == call(K=100) == "RB_ERR_UNSUPPORTED"
    assert call(ldd=100) == call(dY=FAKE + 8) == call(codes=FAKE + 8) == call(scales=FAKE + 2) == "RB_ERR_ALIGNMENT"
    assert call(dW=FAKE + 2) == call(add=FAKE + 2) == "RB_ERR_ALIGNMENT"
    assert call(wb=0) == "RB_ERR_WORKSPACE"
    # `add` that shares bytes with dW: half a row off, rows off, before it, in
    # the gap between dW's rows but longer than it
    for off in (512, 16, 1024 * 3, -1024 * 99, -4):
        assert call(add=FAKE + off) == "RB_ERR_INVALID_ARG", off
    assert call(ldw=400, add=FAKE + 256 * 4 - 4) == call(ldw=400, add=FAKE + 256 * 4) == "RB_ERR_INVALID_ARG"


def test_dgrad_refusals():
    call = _caller("rb_gemm_dgrad",
                   ["planes", "alpha", "adt", "L", "dY", "ddt", "ldd", "T", "dX", "dt", "ldx", "wk", "wb", "s"],
                   (FAKE, FAKE, F32, Layout(100, 256, 2, 0, 0, 0), FAKE, BF16, 104, 5, FAKE, BF16, 256, FAKE, 256, None))
    for k in ("planes", "alpha", "dY", "dX"):
        assert call(**{k: None}) == "RB_ERR_INVALID_ARG", k
    assert call(adt=BF16) == call(ddt=5) == call(dt=4) == call(ldd=96) == call(ldx=255) == "RB_ERR_INVALID_ARG"
    assert call(L=Layout(100, 256, 5, 0, 0, 0)) == call(L=Layout(100, 200, 2, 0, 0, 0)) == "RB_ERR_UNSUPPORTED"
    assert call(ddt=F32) == call(T=0) == "RB_ERR_UNSUPPORTED"
    assert call(L=Layout(100, 256, 2, 0, 3, 0)) == "RB_ERR_INVALID_ARG"
    assert call(ldd=100) == call(planes=FAKE + 4) == call(alpha=FAKE + 2) == call(dX=FAKE + 1) == "RB_ERR_ALIGNMENT"
    assert call(wb=16) == "RB_ERR_WORKSPACE"


@pytest.mark.parametrize("fn", ["rb_pack", "rb_gemv", "rb_gemm"])
def test_the_earlier_calls_refuse_bf16(fn):
    lib, p, L = _lib.load(), ctypes.c_void_p(FAKE), Layout(64, 256, 2, 0, 0, 0)
    if fn == "rb_pack":
        rc = lib.rb_pack(p, BF16, 256, L, p, p, None, None)
    else:
        rc = getattr(lib, fn)(p, p, F32, L, p, 256, 1, p, BF16, 64, p, 1 << 20, None)
    assert _lib.STATUS_NAMES[rc] == "RB_ERR_INVALID_ARG"


def test_binding_takes_no_cpu_tensors():
    x = torch.zeros(2, 128)
    c, s = torch.zeros(2, 128, dtype=torch.float8_e4m3fn), torch.ones(2, 1)
    for f in (lambda: rb.pack8(x), lambda: rb.unpack8(c, s), lambda: rb.gemm8(c, s[:1], c, s),
              lambda: rb.gemm_wgrad(x.half(), c, s),
              lambda: rb.gemm_dgrad(torch.zeros(1, 4, 4, dtype=torch.int32), torch.ones(1, 4, 1), x.half(), 128)):
        with pytest.raises(ValueError, match="CUDA"):
            f()
