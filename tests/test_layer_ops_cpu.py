"""Refusals of the 8-bit layer operators: found on the host before anything
is enqueued, so they need no GPU.  Addresses are made up and never read."""
import ctypes
import math

import pytest
import torch

import tiled_dense_int8_amd as t

X, R, W, S, Q, SC = (0x10000000 * (i + 1) for i in range(6))


def norm(fmt="s8", type=t.BF16, T=4, H=256, x=X, ldx=256, residual=R, ldr=256, weight=W, eps=1e-6, sum=S, ldsum=256,
         q=Q, ldq=256, scale=SC, lds=2):
    args = [type, T, H, x, ldx, residual, ldr, weight, eps, sum, ldsum, q, ldq, scale]
    return t.rmsnorm_quant_s8(*args) if fmt == "s8" else t.rmsnorm_quant_f8(*args, lds)


def act(fmt="s8", type=t.BF16, T=4, N=256, gate=X, ldg=256, up=R, ldu=256, q=Q, ldq=256, scale=SC, lds=2):
    args = [type, T, N, gate, ldg, up, ldu, q, ldq, scale]
    return t.swiglu_quant_s8(*args) if fmt == "s8" else t.swiglu_quant_f8(*args, lds)


@pytest.mark.parametrize("fmt", ["s8", "f8"])
def test_norm_refusals(fmt):
    bad = dict(type=3), dict(type=-1), dict(T=-1), dict(H=-1), dict(H=2 ** 30 + 1, ldx=2 ** 30 + 1, ldr=2 ** 30 + 1,
                                                                 ldsum=2 ** 30 + 1, ldq=2 ** 30 + 1, lds=2 ** 24), \
        dict(ldx=255), dict(ldr=255), dict(ldsum=255), dict(ldq=255), dict(eps=-1e-6), dict(eps=math.nan), \
        dict(eps=math.inf), dict(residual=None), dict(x=X + 1), dict(weight=W + 1), dict(scale=SC + 2), dict(sum=S + 1)
    for kw in bad:
        assert norm(fmt, **kw) == t.ERR_INVALID_VALUE, kw
    for kw in dict(x=None), dict(weight=None), dict(q=None), dict(scale=None):
        assert norm(fmt, **kw) == t.ERR_NULL_POINTER, kw
    for kw in dict(q=X), dict(q=R + 100), dict(q=W), dict(scale=X + 4 * 512 - 4), dict(sum=X, ldsum=257), \
            dict(sum=X + 2), dict(sum=R, ldr=300), dict(sum=W), dict(q=S), dict(scale=S), dict(scale=Q):
        assert norm(fmt, **kw) == t.ERR_ALIASING, kw
    if fmt == "f8":
        assert norm(fmt, lds=1) == t.ERR_INVALID_VALUE


@pytest.mark.parametrize("fmt", ["s8", "f8"])
def test_act_refusals(fmt):
    for kw in dict(type=9), dict(T=-1), dict(N=-2), dict(ldg=255), dict(ldu=255), dict(ldq=0), dict(gate=X + 1), \
            dict(up=R + 1), dict(scale=SC + 1):
        assert act(fmt, **kw) == t.ERR_INVALID_VALUE, kw
    for kw in dict(gate=None), dict(up=None), dict(q=None), dict(scale=None):
        assert act(fmt, **kw) == t.ERR_NULL_POINTER, kw
    for kw in dict(q=X), dict(q=R), dict(scale=X), dict(scale=Q):
        assert act(fmt, **kw) == t.ERR_ALIASING, kw


def test_empty_rows_enqueue_nothing():
    assert norm(T=0) == t.OK and norm(H=0, ldx=1) == t.OK and act(T=0) == t.OK and act(N=0) == t.OK
    assert norm(T=0, x=None, weight=None, q=None, scale=None) == t.OK


def test_ints_that_do_not_fit_are_refused():
    with pytest.raises(ValueError):
        norm(T=2 ** 32 + 1)
    with pytest.raises(ValueError):
        act(ldq=2 ** 31)


def test_wrappers_refuse():
    x = torch.zeros(4, 256)
    w = torch.zeros(256)
    with pytest.raises(ValueError, match="GPU"):
        t.rms_norm(x, w)
    with pytest.raises(ValueError, match="GPU"):
        t.swiglu(x, x)
    with pytest.raises(TypeError):
        t.rms_norm(x.double(), w.double())
    with pytest.raises(TypeError):
        t.rms_norm(x, w, residual=x.half())
    with pytest.raises(TypeError):
        t.swiglu(x, x.half())
    with pytest.raises(ValueError):
        t.rms_norm(x, w[:255])
    with pytest.raises(ValueError):
        t.rms_norm(x, w.half())
    with pytest.raises(ValueError):
        t.rms_norm(x.t(), torch.zeros(4))
    with pytest.raises(ValueError):
        t.rms_norm(x[:1].expand(4, 256), w)
    with pytest.raises(ValueError):
        t.rms_norm(x, w, sum_out=x)
    with pytest.raises(ValueError):
        t.swiglu(x, x[:, :128])
    with pytest.raises(ValueError):
        t.rms_norm(x[0], w)
