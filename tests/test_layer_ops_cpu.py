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


# ----- products ----------------------------------------------------------------------

C, BS, RO, OF = (0x100000000 * (i + 1) for i in range(4))


def grouped(type=t.BF16, G=4, M=32, N=64, K=128, A=X, lda=128, a_rows=16, a_scale=SC, rows=RO, offsets=OF, B=W,
            ldb=128, group_b=64 * 128, b_scale=BS, C=C, ldc=64):
    return t.gemm_s8s8_grouped(type, G, M, N, K, A, lda, a_rows, a_scale, rows, offsets, B, ldb, group_b, b_scale, C,
                               ldc)


def f8(type=t.BF16, M=32, N=200, K=300, A=X, lda=300, a_scale=SC, ldas=3, B=W, ldb=300, b_scale=BS, ldbs=3, C=C,
       ldc=200):
    return t.gemm_f8f8_block128(type, M, N, K, A, lda, a_scale, ldas, B, ldb, b_scale, ldbs, C, ldc)


def test_grouped_refusals():
    big = 2 ** 30 + 1
    for kw in dict(type=3), dict(type=-1), dict(G=-1), dict(M=-1), dict(N=-1), dict(K=-1), dict(lda=127), \
            dict(ldb=127), dict(ldc=63), dict(a_rows=-1), dict(a_rows=0), dict(K=131072, lda=131072, ldb=131072,
                                                                              group_b=2 ** 40), \
            dict(group_b=64 * 128 - 1), dict(group_b=-1), dict(rows=None, a_rows=31), dict(C=C + 1), \
            dict(type=t.F32, C=C + 2), dict(a_scale=SC + 1), dict(b_scale=BS + 2), dict(rows=RO + 2), \
            dict(offsets=OF + 1), dict(M=big), dict(N=big, ldc=big), dict(G=big):
        assert grouped(**kw) == t.ERR_INVALID_VALUE, kw
    for kw in dict(offsets=None), dict(A=None), dict(B=None), dict(a_scale=None), dict(b_scale=None), dict(C=None):
        assert grouped(**kw) == t.ERR_NULL_POINTER, kw
    for kw in dict(C=X), dict(C=W + 3 * 64 * 128), dict(C=SC), dict(C=BS + 4), dict(C=RO), dict(C=OF + 16):
        assert grouped(**kw) == t.ERR_ALIASING, kw
    for kw in dict(M=0), dict(N=0), dict(G=0), dict(M=0, A=None, C=None):
        assert grouped(**kw) == t.OK, kw
    with pytest.raises(ValueError):
        grouped(group_b=2 ** 63)
    with pytest.raises(ValueError):
        grouped(M=2 ** 32)


def test_f8_refusals():
    big = 2 ** 30 + 1
    for kw in dict(type=7), dict(M=-1), dict(N=-1), dict(K=-1), dict(lda=299), dict(ldb=299), dict(ldc=199), \
            dict(ldas=2), dict(ldbs=2), dict(C=C + 1), dict(a_scale=SC + 2), dict(b_scale=BS + 1), \
            dict(K=big, lda=big, ldb=big, ldas=2 ** 24, ldbs=2 ** 24):
        assert f8(**kw) == t.ERR_INVALID_VALUE, kw
    for kw in dict(A=None), dict(B=None), dict(a_scale=None), dict(b_scale=None), dict(C=None):
        assert f8(**kw) == t.ERR_NULL_POINTER, kw
    for kw in dict(C=X + 300), dict(C=W), dict(C=SC), dict(C=BS):
        assert f8(**kw) == t.ERR_ALIASING, kw
    assert f8(M=0) == t.OK and f8(N=0, ldc=1) == t.OK


def test_product_wrappers_refuse():
    A, s = torch.zeros(4, 256, dtype=torch.int8), torch.zeros(4)
    B, bs = torch.zeros(3, 8, 256, dtype=torch.int8), torch.zeros(3, 8)
    off = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError, match="GPU"):
        t.grouped_gemm(A, s, B, bs, off)
    with pytest.raises(TypeError):
        t.grouped_gemm(A.float(), s, B, bs, off)
    with pytest.raises(TypeError):
        t.grouped_gemm(A, s, B.float(), bs, off)
    for kw in dict(offsets=None), dict(offsets=off[:3]), dict(offsets=off.long()), dict(rows=off.long()), \
            dict(rows=off[::2]), dict(a_scale=s[:3]), dict(a_scale=s.double()), dict(b_scale=bs[:2]), \
            dict(b_scale=bs.t().contiguous().t()), dict(B=B[:, :, :255]), dict(B=B.transpose(1, 2)):
        with pytest.raises(ValueError):
            t.grouped_gemm(**{**dict(A=A, a_scale=s, B=B, b_scale=bs, offsets=off), **kw})
    F = torch.zeros(4, 256).to(torch.float8_e4m3fn)
    fs, gs = torch.zeros(4, 2), torch.zeros(1, 2)
    with pytest.raises(ValueError, match="GPU"):
        t.gemm_f8(F, fs, F, gs)
    with pytest.raises(TypeError):
        t.gemm_f8(F.view(torch.int8), fs, F, gs)
    for kw in dict(B=F[:, :128]), dict(a_scale=fs[:3]), dict(b_scale=gs[:, :1]), dict(a_scale=torch.zeros(2, 4).t()):
        with pytest.raises(ValueError):
            t.gemm_f8(**{**dict(A=F, a_scale=fs, B=F, b_scale=gs), **kw})


def test_native_calls_leave_others_to_python():
    """_calls makes no call it cannot: CPU tensors, other objects, other counts of arguments."""
    x, w = torch.zeros(2, 8), torch.ones(8)
    q = torch.zeros(2, 128).to(torch.float8_e4m3fn)
    s = torch.ones(2, 1)
    i8 = torch.zeros(2, 8, dtype=torch.int8)
    for name, args in (("rms_norm", (x, w, 1e-6, None, "s8", None, None, None)), ("swiglu", (x, x, "s8", None, None)),
                       ("gemm_f8", (q, s, q, s[:1], None, torch.float32)),
                       ("grouped_gemm", (i8, w[:2], i8, w[:2], None, None, None, torch.float32))):
        call = getattr(t._calls, name)
        assert call(*args, 0, 0) is None
        assert call(*args) is None and call() is None
        assert call(*args, None, "stream") is None
        for k in range(len(args)):
            for other in (None, 3, "x", [1], object()):
                assert call(*args[:k], other, *args[k + 1:], 0, 0) is None


# ----- the choice of a product's kernel ------------------------------------------------

def most_tiles(G, M, N):
    """Tiles of 64 x 128 results, the rows of each group that can have some filled up to 64."""
    groups = min(G, M)
    return (M + 63 * groups) // 64 * -(-N // 128)


# (f8, groups, M, N, K): few rows and very many columns, the reverse, groups of a row
HUGE = [(0, 1, 1, 70_000_000, 16), (0, 1, 1, 70_000_000, 1), (0, 1, 8, 68_000_000, 16), (0, 1, 4, 100_000_000, 8),
        (1, 1, 1, 70_000_000, 16), (1, 1, 8, 68_000_000, 16), (1, 1, 4, 100_000_000, 8), (0, 1, 1, 500_000_000, 1),
        (0, 1, 250_000_000, 1, 16), (1, 1, 250_000_000, 1, 7), (0, 1, 2 ** 21, 2 ** 13, 64),
        (0, 4_000_000, 4_000_000, 64, 32), (0, 4_000_000, 4_000_000, 128, 31), (0, 100_000, 200_000, 4096, 64)]


@pytest.mark.parametrize("type", [t.F32, t.BF16, t.F16])
@pytest.mark.parametrize("size", HUGE, ids=lambda s: "x".join(map(str, s)))
def test_products_of_many_results_have_a_grid(size, type):
    """A tile whose grid cannot be launched is passed over for one whose grid can."""
    f8, G, M, N, K = size
    assert most_tiles(G, M, N) <= 4_000_000
    for aligned in (K % 16 == 0, False):
        plan = t.scaled_product_plan(f8, type, G, M, N, K, aligned, 256)
        assert plan.form != t.SCALED_NONE
        assert plan.blocks * plan.threads < 2 ** 31
        tiles = (M + min(G, M) * (plan.block_m - 1)) // plan.block_m * -(-N // plan.block_n)
        assert plan.blocks == -(-tiles // 8) * 8


def test_products_without_a_grid_are_refused():
    for size in (0, 1, 2 ** 30, 2 ** 12, 64), (0, 1, 2 ** 30, 2 ** 30, 64), (0, 2 ** 26, 2 ** 26, 1024, 64):
        for aligned in (0, 1):
            f8, G, M, N, K = size
            assert most_tiles(G, M, N) > 4_000_000
            with pytest.raises(t.TDI8Error) as e:
                t.scaled_product_plan(f8, t.BF16, G, M, N, K, aligned, 256)
            assert e.value.status == t.ERR_INVALID_VALUE


def test_plan_of_ordinary_sizes():
    """The tiles of sizes whose measurements the code names."""
    for size, want in (((1, 1, 16, 4096, 4096, 1), (t.SCALED_STREAM, 16, 16)),
                       ((1, 1, 4096, 4096, 4096, 1), (t.SCALED_LDS, 256, 256)),
                       ((1, 1, 1000, 3000, 777, 0), (t.SCALED_STAGED, 64, 128)),
                       ((0, 8, 1000, 1501, 777, 0), (t.SCALED_STAGED, 64, 128)),
                       ((0, 64, 64, 4096, 2048, 1), (t.SCALED_STREAM, 16, 32)),
                       ((0, 16, 16384, 4096, 4096, 1), (t.SCALED_LDS, 256, 256))):
        f8, G, M, N, K, aligned = size
        plan = t.scaled_product_plan(f8, t.BF16, G, M, N, K, aligned, 256)
        assert (plan.form, plan.block_m, plan.block_n) == want, size
    for empty in (0, 0, 5, 5), (0, 3, 0, 5), (1, 1, 5, 0):
        assert t.scaled_product_plan(*empty[:1], t.F32, *empty[1:], 64, 1, 256).form == t.SCALED_NONE
    for bad in (0, 3, 1, 1, 1, 1, 1, 256), (1, 0, 2, 1, 1, 1, 1, 256), (0, 0, 1, 1, 1, 131072, 1, 256), \
            (0, 0, 1, -1, 1, 1, 1, 256), (0, 0, 1, 1, 1, 1, 1, 0):
        with pytest.raises(t.TDI8Error):
            t.scaled_product_plan(*bad)


def test_only_bf16_results_of_e4m3_take_the_256_wide_tile():
    """Results of fp16 and fp32 need sums in 32 bits, whose kernels have other tiles."""
    for type, want in ((t.BF16, (256, 256)), (t.F16, (128, 128)), (t.F32, (128, 128))):
        plan = t.scaled_product_plan(1, type, 1, 4096, 4096, 4096, 1, 256)
        assert plan.form == t.SCALED_LDS and (plan.block_m, plan.block_n) == want


def test_layer_code_hash_covers_every_layer_kernel():
    """The hash is that of all objects that hold layer kernels; with the configurations' it covers the library's."""
    import glob
    import hashlib
    import os
    import re
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    sys.path.insert(0, os.path.join(root, "tiled_dense_int8_amd"))
    import build as b
    h = t.tdi8_layer_code_hash()
    assert len(h) == 16 and int(h, 16) >= 0 and h != t.tdi8_kernel_code_hash()
    cos = [os.path.join(b.BUILD, name + ".o.co") for name in b.LAYER_OBJECTS]
    if all(os.path.exists(c) for c in cos):
        d = hashlib.sha256()
        for c in cos:
            d.update(open(c, "rb").read())
        assert d.hexdigest()[:16] == h
    # no source with a kernel's definition is built into an object of neither list
    sources = {os.path.splitext(os.path.basename(p))[0] for p in glob.glob(os.path.join(b.CSRC, "*.hip"))}
    listed = {re.sub("_(S8|F8|F8Wide|F32|Bf16|F16)$", "", name) for name in b.LAYER_OBJECTS}
    assert {s.replace("stream_product", "stream") for s in sources} == listed | {"instantiate", "ceilings"}


# ----- the package without its native calls ----------------------------------------------

WITHOUT_CALLS = """
import sys, types, warnings
sys.path.insert(0, {root!r})
if {other!r}:
    calls = types.ModuleType("tiled_dense_int8_amd._calls")
    calls.torch_version = {other!r}
    sys.modules["tiled_dense_int8_amd._calls"] = calls
else:
    class Missing:
        def find_spec(self, name, path=None, target=None):
            if name.endswith("._calls"):
                raise ModuleNotFoundError("no module named " + name, name=name)
    sys.meta_path.insert(0, Missing())
with warnings.catch_warnings(record=True) as seen:
    warnings.simplefilter("always")
    import tiled_dense_int8_amd as t
import torch
assert t._calls is None and [w.category for w in seen] == [RuntimeWarning] and "_calls" in str(seen[0].message)
assert t.tile_config_count() > 0 and t.gemm_s8s8s32(0, 4, 4, 0, 4, 0, 4, 0, 4, 0) == t.OK
x = torch.zeros(2, 8)
for call in (lambda: t.rms_norm(x, x[0]), lambda: t.swiglu(x, x)):
    try:
        call()
    except ValueError as e:
        assert "GPU" in str(e)
    else:
        raise AssertionError("not refused")
"""


@pytest.mark.parametrize("other", ["", "0.0.1"])
def test_package_without_its_native_calls(other):
    """Missing, or of another torch: the package imports with a warning and makes its calls by Python."""
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", WITHOUT_CALLS.format(root=root, other=other)], capture_output=True,
                       text=True, timeout=300)
    assert r.returncode == 0, r.stderr


def test_native_calls_are_of_this_torch():
    assert t._calls is not None and t._calls.torch_version == torch.__version__


def test_outputs_that_require_grad_are_refused():
    x, w = torch.zeros(4, 256), torch.zeros(256)
    leaf, s = torch.zeros(4, 256, requires_grad=True), torch.zeros(4, requires_grad=True)
    A, a, B, b = torch.zeros(4, 256, dtype=torch.int8), torch.zeros(4), torch.zeros(8, 256, dtype=torch.int8), torch.zeros(8)
    F = x.to(torch.float8_e4m3fn)
    y = torch.zeros(4, 8, requires_grad=True)
    calls = (lambda: t.rms_norm(x, w, residual=x, sum_out=leaf), lambda: t.rms_norm(x, w, scale=s),
             lambda: t.swiglu(x, x, scale=s), lambda: t.grouped_gemm(A, a, B, b, out=y),
             lambda: t.gemm_f8(F, torch.zeros(4, 2), F[:1], torch.zeros(1, 2), out=y[:, :1]))
    for call in calls:
        with pytest.raises(ValueError, match="requires grad"):
            call()
        with torch.no_grad(), pytest.raises(ValueError, match="GPU"):  # the next check
            call()


def test_operands_that_lie_wrong_are_refused_in_words():
    A, s = torch.zeros(4, 256, dtype=torch.int8), torch.zeros(4)
    B, bs = torch.zeros(3, 8, 256, dtype=torch.int8), torch.zeros(3, 8)
    off, rows = torch.zeros(4, dtype=torch.int32), torch.zeros(5, dtype=torch.int32)
    with pytest.raises(ValueError, match="groups overlap"):
        t.grouped_gemm(A, s, B[:1].expand(3, 8, 256), bs, off)
    with pytest.raises(ValueError, match="groups overlap"):
        t.grouped_gemm(A, s, torch.as_strided(B, (3, 8, 256), (255 + 7 * 256, 256, 1)), bs, off)
    with pytest.raises(ValueError, match="rows overlap"):
        t.grouped_gemm(A, s, torch.as_strided(B, (3, 8, 256), (2048, 255, 1)), bs, off)
    with pytest.raises(ValueError, match="no rows"):
        t.grouped_gemm(A[:0], s[:0], B, bs, off, rows=rows)
    # what lies apart, and calls of no rows, go on to the next check
    for args in ((A, s, torch.zeros(3, 9, 272, dtype=torch.int8)[:, :8, :256], bs, off),
                 (A[:0], s[:0], B[:1].expand(3, 8, 256), bs, off), (A[:0], s[:0], B, bs, off, rows[:0]),
                 (A[:, :0], s, B[:, :, :0], bs, off)):
        with pytest.raises(ValueError, match="GPU"):
            t.grouped_gemm(*args)


def negated(t_):
    """A view whose memory holds the values of the other sign."""
    view = torch._neg_view(t_)
    assert view.is_neg() or not t_.numel()
    return view


def test_lazily_negated_operands_are_refused():
    """Their memory holds other values than they show."""
    x, w, n = torch.ones(4, 256), torch.ones(256), negated
    column = torch.ones(4, 1, dtype=torch.complex64).conj().imag  # as ordinary code comes by one
    assert column.is_neg()
    A, a, B, b = torch.ones(4, 256, dtype=torch.int8), torch.ones(4), torch.ones(8, 256, dtype=torch.int8), torch.ones(8)
    F, f, g = x.to(torch.float8_e4m3fn), torch.ones(4, 2), torch.ones(1, 2)
    calls = [lambda: t.rms_norm(column, torch.ones(1)), lambda: t.swiglu(x[:, :1], column),
             lambda: t.rms_norm(n(x), w), lambda: t.rms_norm(x, n(w)), lambda: t.rms_norm(x, w, residual=n(x)),
             lambda: t.rms_norm(x, w, residual=x, sum_out=n(x)), lambda: t.swiglu(n(x), x), lambda: t.swiglu(x, n(x)),
             lambda: t.grouped_gemm(n(A), a, B, b), lambda: t.grouped_gemm(A, n(a), B, b),
             lambda: t.grouped_gemm(A, a, n(B), b), lambda: t.grouped_gemm(A, a, B, n(b)),
             lambda: t.gemm_f8(F, n(f), F, g), lambda: t.gemm_f8(F, f, F, n(g))]
    for call in calls:
        with pytest.raises(ValueError, match="negated lazily"):
            call()
