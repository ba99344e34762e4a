"""The layer operators' ordinary calls (module _calls) against the calls by Python, and what each refuses."""
import sys

import pytest
import torch

import tiled_dense_int8_amd as t

pytestmark = pytest.mark.gpu
F8 = torch.float8_e4m3fn


def gen(seed):
    return torch.Generator().manual_seed(seed)


def normal(g, *shape, dtype=torch.bfloat16):
    return torch.randn(*shape, generator=g).to(dtype).cuda()


def s8(g, *shape):
    return torch.randint(-128, 128, shape, generator=g, dtype=torch.int8).cuda()


def scales(g, *shape):
    return (torch.rand(*shape, generator=g) + 0.1).cuda()


def same(a, b):
    a, b = (x if isinstance(x, tuple) else (x,) for x in (a, b))
    assert len(a) == len(b)
    for x, y in zip(a, b):
        assert x.dtype == y.dtype and x.shape == y.shape and x.stride() == y.stride() and x.device == y.device
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))


def where():
    device = torch.cuda.current_device()
    return device, torch.cuda.current_stream().cuda_stream


def native(name, *args):
    """The call through _calls alone (None where it leaves the call to Python)."""
    return getattr(t._calls, name)(*args, *where())


@pytest.mark.parametrize("fmt", ["s8", "f8"])
@pytest.mark.parametrize("shape", [(0, 5), (1, 1), (1, 4096), (7, 130), (33, 1000)])
def test_rows_alike(shape, fmt):
    g = gen(sum(shape))
    stream = torch.cuda.current_stream()
    for dtype in (torch.float32, torch.bfloat16, torch.float16):
        x, r, w = normal(g, *shape, dtype=dtype), normal(g, *shape, dtype=dtype), normal(g, shape[1], dtype=dtype)
        got = native("rms_norm", x, w, 1e-5, r, fmt, None, None, None)
        assert got is not None
        same(got, t.rms_norm(x, w, 1e-5, residual=r, fmt=fmt, stream=stream))
        same(t.rms_norm(x, w, 1e-5, fmt=fmt), t.rms_norm(x, w, 1e-5, fmt=fmt, stream=stream))
        assert native("swiglu", x, r, fmt, None, None) is not None
        same(t.swiglu(x, r, fmt=fmt), t.swiglu(x, r, fmt=fmt, stream=stream))
        both = torch.cat((x, r), 1)
        same(t.swiglu(both[:, :shape[1]], both[:, shape[1]:], fmt=fmt), t.swiglu(x, r, fmt=fmt, stream=stream))
    torch.cuda.synchronize()


def test_products_alike():
    g = gen(3)
    stream = torch.cuda.current_stream()
    for M, N, K in ((1, 1, 1), (3, 40, 128), (20, 300, 777), (70, 129, 256)):
        kb, nb = -(-K // 128), -(-N // 128)
        A, B = (normal(g, *s, dtype=torch.float32).to(F8) for s in ((M, K), (N, K)))
        sa, sb = scales(g, M, kb), scales(g, nb, kb)
        A8, B8, ra, rb = s8(g, M, K), s8(g, 2, N, K), scales(g, M), scales(g, 2, N)
        off = torch.tensor([0, M // 2, M], dtype=torch.int32).cuda()
        rows = torch.randint(0, M, (M,), generator=g, dtype=torch.int32).cuda()
        for dtype in (torch.float32, torch.bfloat16, torch.float16):
            assert native("gemm_f8", A, sa, B, sb, None, dtype) is not None
            same(t.gemm_f8(A, sa, B, sb, dtype=dtype), t.gemm_f8(A, sa, B, sb, dtype=dtype, stream=stream))
            for o, r in ((off, rows), (off, None)):
                assert native("grouped_gemm", A8, ra, B8, rb, o, r, None, dtype) is not None
                same(t.grouped_gemm(A8, ra, B8, rb, o, rows=r, dtype=dtype),
                     t.grouped_gemm(A8, ra, B8, rb, o, rows=r, dtype=dtype, stream=stream))
            assert native("grouped_gemm", A8, ra, B8[0], rb[0], None, None, None, dtype) is not None
            same(t.grouped_gemm(A8, ra, B8[0], rb[0], dtype=dtype),
                 t.grouped_gemm(A8, ra, B8[:1], rb[:1], rows=None, dtype=dtype, stream=stream))
    torch.cuda.synchronize()


def test_outputs_of_the_caller():
    """Given outputs are the ones returned, written in place, and no reference is kept."""
    g = gen(4)
    x, r, w = normal(g, 5, 300), normal(g, 5, 300), normal(g, 300)
    want = t.rms_norm(x, w, residual=r, fmt="f8")
    out, scale, total = (torch.empty(5, 320, dtype=F8).cuda()[:, :300], torch.empty(5, 3).cuda(), r.clone())
    before = [sys.getrefcount(o) for o in (x, out, scale, total)]
    for _ in range(3):
        total.copy_(r)
        got = t.rms_norm(x, w, residual=total, fmt="f8", sum_out=total, out=out, scale=scale)
        assert got[0] is out and got[1] is scale and got[2] is total
        for a, b in zip(got, want):
            assert torch.equal(a.contiguous().view(torch.uint8), b.view(torch.uint8))
        del got, a
    assert [sys.getrefcount(o) for o in (x, out, scale, total)] == before
    A8, B8, ra, rb = s8(g, 4, 64), s8(g, 1, 30, 64), scales(g, 4), scales(g, 1, 30)
    y = torch.empty(4, 32).cuda()[:, :30]
    assert t.grouped_gemm(A8, ra, B8, rb, out=y) is y
    assert torch.equal(y, t.grouped_gemm(A8, ra, B8, rb, dtype=torch.float32))
    q = torch.empty(5, 300, dtype=torch.int8).cuda()
    assert t.swiglu(x, r, out=q)[0] is q


def test_left_to_python():
    """Calls that _calls does not make work all the same, or are refused by name."""
    g = gen(5)
    x, w = normal(g, 5, 300), normal(g, 300)
    want = t.rms_norm(x, w, 0.0)
    for eps in (0, torch.tensor(0.0)):  # not a Python float
        assert native("rms_norm", x, w, eps, None, "s8", None, None, None) is None
    same(t.rms_norm(x, w, 0), want)
    same(t.rms_norm(x, torch.nn.Parameter(w), 0.0), want)
    same(t.rms_norm(x.as_subclass(type("Mine", (torch.Tensor,), {})), w, 0.0), want)
    A, B, sa, sb = (normal(g, 4, 256, dtype=torch.float32).to(F8), normal(g, 30, 256, dtype=torch.float32).to(F8),
                    scales(g, 4, 2), scales(g, 1, 2))
    A8, B8, ra, rb = s8(g, 4, 64), s8(g, 2, 30, 64), scales(g, 4), scales(g, 2, 30)
    off = torch.tensor([0, 1, 4], dtype=torch.int32).cuda()
    refused = [
        (TypeError, lambda: t.rms_norm(x.double(), w)), (ValueError, lambda: t.rms_norm(x, w.float())),
        (ValueError, lambda: t.rms_norm(x, w[1:])), (ValueError, lambda: t.rms_norm(x.t(), w[:5])),
        (ValueError, lambda: t.rms_norm(x, w, fmt="int8")), (ValueError, lambda: t.rms_norm(x, w, sum_out=x)),
        (ValueError, lambda: t.rms_norm(x, w.cpu())), (TypeError, lambda: t.rms_norm(x, w, residual=x.float())),
        (ValueError, lambda: t.rms_norm(x[0], w)), (TypeError, lambda: t.rms_norm(x, w, out=torch.empty(5, 300).cuda())),
        (ValueError, lambda: t.rms_norm(x, w, scale=torch.empty(4).cuda())),
        (ValueError, lambda: t.swiglu(x, x[:4])), (ValueError, lambda: t.swiglu(x[:1].expand(5, 300), x)),
        (TypeError, lambda: t.gemm_f8(A.view(torch.int8), sa, B, sb)), (ValueError, lambda: t.gemm_f8(A, sa[:, :1], B, sb)),
        (ValueError, lambda: t.gemm_f8(A[:, :128], sa[:, :1], B, sb)), (TypeError, lambda: t.gemm_f8(A, sa, B, sb, dtype=torch.int8)),
        (ValueError, lambda: t.gemm_f8(A, sa, B, sb, out=torch.empty(4, 31).cuda())),
        (ValueError, lambda: t.grouped_gemm(A8, ra, B8, rb)), (ValueError, lambda: t.grouped_gemm(A8, ra, B8, rb, off[:2])),
        (ValueError, lambda: t.grouped_gemm(A8, ra, B8, rb, off.long())),
        (ValueError, lambda: t.grouped_gemm(A8, ra, B8, rb[:, ::2], off)),
        (ValueError, lambda: t.grouped_gemm(A8, ra[:3], B8, rb, off)),
        (TypeError, lambda: t.grouped_gemm(A8, ra, B8.float(), rb, off)),
    ]
    for k, (error, call) in enumerate(refused):
        with pytest.raises(error):
            call()
            print("not refused:", k)


def test_status_becomes_an_error():
    g = gen(6)
    A, sa = normal(g, 64, 128, dtype=torch.float32).to(F8), scales(g, 64, 1)
    with pytest.raises(t.TDI8Error) as e:
        t.gemm_f8(A, sa, A, scales(g, 1, 1), out=A.view(torch.float16))
    assert e.value.status == t.ERR_ALIASING
    x = normal(g, 4, 64)
    for call in (lambda: t.rms_norm(x, x[0], float("nan")), lambda: t.rms_norm(x, x[0], -1.0)):
        with pytest.raises(t.TDI8Error) as e:
            call()
        assert e.value.status == t.ERR_INVALID_VALUE
    x8 = torch.zeros(4, 64, dtype=torch.int8).cuda()
    with pytest.raises(t.TDI8Error):
        t.swiglu(x8.view(torch.float16), x8.view(torch.float16), out=x8[:, :32])


def test_other_streams_and_threads():
    """The current stream is the one used, in threads of their own too."""
    import threading
    g = gen(7)
    x, w = normal(g, 300, 4000), normal(g, 4000)
    want = t.rms_norm(x, w, fmt="f8")
    torch.cuda.synchronize()
    results = {}

    def work(k):
        with torch.cuda.stream(torch.cuda.Stream()):
            y = x + 0
            for _ in range(20):
                results[k] = t.rms_norm(y, w, fmt="f8")
            torch.cuda.current_stream().synchronize()

    threads = [threading.Thread(target=work, args=(k,)) for k in range(4)]
    for th in threads:
        th.start()
    for th in threads:
        th.join()
    for k in range(4):
        same(results[k], want)


def test_captured_with_outputs_of_their_own():
    """A layer's calls captured into a graph, outputs from the graph's memory, replayed over changing inputs."""
    g = gen(8)
    x, r, w = normal(g, 24, 512), normal(g, 24, 512), normal(g, 512)
    B, sb = s8(g, 3, 200, 512), scales(g, 3, 200)
    off = torch.tensor([0, 5, 5, 24], dtype=torch.int32).cuda()

    def layer():
        q, scale, h = t.rms_norm(x, w, residual=r)
        y = t.grouped_gemm(q, scale, B, sb, off)
        return (q, scale, h, y) + t.swiglu(y[:, :100], y[:, 100:], fmt="f8")

    layer()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        made = layer()
    for _ in range(4):
        x.copy_(normal(g, 24, 512))
        r.copy_(normal(g, 24, 512))
        graph.replay()
        torch.cuda.synchronize()
        same(made, layer())


def test_inference_mode_and_leaves():
    g = gen(9)
    x, w = normal(g, 6, 256), normal(g, 256)
    want = t.rms_norm(x, w)
    with torch.inference_mode():
        same(tuple(o.clone() for o in t.rms_norm(x, w)), want)
    got = t.rms_norm(x.clone().requires_grad_(), torch.nn.Parameter(w.clone()))
    same(got, want)
    assert not any(o.requires_grad for o in got)


def operator_calls(g):
    """(call of the outputs to write and a stream, those outputs) of every operator."""
    x, w = normal(g, 5, 300), normal(g, 300)
    q, q8 = torch.empty(5, 300, dtype=torch.int8).cuda(), torch.empty(5, 300, dtype=F8).cuda()
    s, s8_ = torch.empty(5).cuda(), torch.empty(5, 3).cuda()
    h = normal(g, 5, 300)
    A, B, ra, rb = s8(g, 5, 64), s8(g, 30, 64), scales(g, 5), scales(g, 30)
    A8, B8 = (normal(g, *k, dtype=torch.float32).to(F8) for k in ((5, 128), (30, 128)))
    sa, sb = scales(g, 5, 1), scales(g, 1, 1)
    y = torch.empty(5, 30).cuda()
    return [
        (lambda o, stream: t.rms_norm(x, w, residual=x, sum_out=o[0], out=o[1], scale=o[2], stream=stream), (h, q, s)),
        (lambda o, stream: t.rms_norm(x, w, fmt="f8", out=o[0], scale=o[1], stream=stream), (q8, s8_)),
        (lambda o, stream: t.swiglu(x, x, out=o[0], scale=o[1], stream=stream), (q, s)),
        (lambda o, stream: t.grouped_gemm(A, ra, B, rb, out=o[0], stream=stream), (y,)),
        (lambda o, stream: t.gemm_f8(A8, sa, B8, sb, out=o[0], stream=stream), (y,)),
    ]


def test_written_outputs_are_known_to_autograd():
    """A call's outputs count as written once, made natively or by Python; those of inference mode are left alone."""
    for call, outputs in operator_calls(gen(20)):
        for stream in (None, torch.cuda.current_stream()):
            before = [o._version for o in outputs]
            call(outputs, stream)
            assert [o._version for o in outputs] == [v + 1 for v in before]
            with torch.inference_mode():
                inner = [o.clone() for o in outputs]
                call(inner, stream)
            call(inner, stream)
            for a, b in zip(inner, outputs):
                assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    # the residual stream overwritten between a product and its backward pass
    g = gen(21)
    x, w, h = normal(g, 4, 64), normal(g, 64), normal(g, 4, 64)
    for stream in (None, torch.cuda.current_stream()):
        leaf = normal(g, 64).requires_grad_()
        loss = (h * leaf).sum()
        t.rms_norm(x, w, residual=h, sum_out=h, stream=stream)
        with pytest.raises(RuntimeError, match="inplace"):
            loss.backward()


def test_outputs_that_require_grad():
    """Refused while gradients are recorded, written under no_grad as torch's own operators write them."""
    for call, outputs in operator_calls(gen(22)):
        want = [o.clone() for o in outputs]
        call(want, None)
        for k, o in enumerate(outputs):
            if not o.dtype.is_floating_point:
                continue
            given = [p.clone().requires_grad_() if i == k else p for i, p in enumerate(outputs)]
            for stream in (None, torch.cuda.current_stream()):
                with pytest.raises(ValueError, match="requires grad"):
                    call(given, stream)
                with torch.no_grad():
                    call(given, stream)
                same(tuple(p.detach() for p in given), tuple(want))


def test_operands_that_lie_wrong():
    """Refused in words on the GPU as well, where the native calls leave them to Python."""
    g = gen(23)
    A, s, B, bs = s8(g, 4, 64), scales(g, 4), s8(g, 3, 8, 64), scales(g, 3, 8)
    off, rows = torch.tensor([0, 1, 2, 4], dtype=torch.int32).cuda(), torch.zeros(5, dtype=torch.int32).cuda()
    for stream in (None, torch.cuda.current_stream()):
        with pytest.raises(ValueError, match="groups overlap"):
            t.grouped_gemm(A, s, B[:1].expand(3, 8, 64), bs, off, stream=stream)
        with pytest.raises(ValueError, match="rows overlap"):
            t.grouped_gemm(A, s, torch.as_strided(B, (3, 8, 64), (512, 63, 1)), bs, off, stream=stream)
        with pytest.raises(ValueError, match="no rows"):
            t.grouped_gemm(A[:0], s[:0], B, bs, off, rows=rows, stream=stream)


def test_lazily_negated_operands_are_refused():
    x, w = torch.ones(4, 1, device="cuda"), torch.ones(1, device="cuda")
    column = torch.full((4, 1), 1 + 1j, device="cuda").conj().imag
    q, scale = torch.empty(4, 1, dtype=torch.int8, device="cuda"), torch._neg_view(torch.empty(4, device="cuda"))
    for stream in (None, torch.cuda.current_stream()):
        for call in (lambda: t.rms_norm(column, w, stream=stream), lambda: t.rms_norm(x, w, scale=scale, stream=stream),
                     lambda: t.swiglu(x, column, out=q, stream=stream)):
            with pytest.raises(ValueError, match="negated lazily"):
                call()
    same(t.rms_norm(column.resolve_neg(), w), t.rms_norm(-x, w))
