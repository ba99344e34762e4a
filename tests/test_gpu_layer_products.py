"""Grouped int8 products and block-scaled e4m3 products against 64-bit forms."""
import pytest
import torch

import tiled_dense_int8_amd as t
from helpers import note
from layer_helpers import TYPES, check_f8, check_grouped, f8_reference, grouped_reference, strided

pytestmark = pytest.mark.gpu
SENTINEL = 7.0


def gen(seed):
    return torch.Generator().manual_seed(seed)


def s8(g, *shape):
    return torch.randint(-128, 128, shape, generator=g, dtype=torch.int8)


def scales(g, *shape):
    return (torch.rand(*shape, generator=g) + 0.1) * 0.01


def run_grouped(g, counts, N, K, kind, T=None, rows="random", slack=0, ld=(0, 0, 0), start=(0, 0, 0), group_pad=0):
    """One call with the operands in padded buffers; rows: "random", "none" or a tensor."""
    G, used = len(counts), sum(counts)
    M = used + slack
    if isinstance(rows, str):
        rows = None if rows == "none" else torch.randint(0, T or max(M, 1), (M,), generator=g, dtype=torch.int32)
    T = max(M, 1) if T is None else T
    A, a_scale = s8(g, T, K), scales(g, T)
    B, b_scale = s8(g, G, N, K), scales(g, G, N)
    ends = [0]
    for c in counts:
        ends.append(ends[-1] + c)
    what = f"grouped {counts} N={N} K={K} {kind} T={T} rows={rows is not None} ld={ld} start={start}"
    note("[case] " + what)
    Av, _ = strided(A, K + ld[0], start[0])
    per = N * (K + ld[1]) + group_pad
    Bbuf = torch.full((start[1] + G * per + 64,), 55, dtype=torch.int8, device="cuda")
    Bv = Bbuf[start[1]:start[1] + G * per].view(G, per)[:, :N * (K + ld[1])].view(G, N, K + ld[1])[:, :, :K]
    Bv.copy_(B.cuda())
    out, obuf = strided(torch.full((M, N), SENTINEL, dtype=TYPES[kind]), N + ld[2], start[2])
    before = obuf.clone()
    got = t.grouped_gemm(Av, a_scale.cuda(), Bv, b_scale.cuda(), torch.tensor(ends, dtype=torch.int32).cuda(),
                         rows=None if rows is None else rows.cuda(), out=out)
    torch.cuda.synchronize()
    want, written = grouped_reference(A, a_scale, B, b_scale, ends, rows, M)
    check_grouped(got, want, written, SENTINEL, TYPES[kind], what)
    out.fill_(SENTINEL)
    assert torch.equal(obuf, before), f"{what}: wrote outside C"


COUNTS = [[1], [5, 0, 1], [16, 17, 0, 15], [0, 33, 64, 0], [65, 1, 0, 2, 130], [300, 7], [2] * 70, [0] * 66 + [3] * 67,
          [128, 256, 129], [700], [513, 0, 300, 1]]


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("counts", COUNTS, ids=lambda c: f"{len(c)}x{max(c)}")
def test_grouped_sizes(counts, kind):
    """Every row tile, groups that are empty or end inside tiles, aligned and odd K, odd N."""
    g = gen(len(counts) + max(counts))
    for N, K in ((1, 1), (5, 17), (16, 16), (64, 128), (100, 144), (257, 777), (128, 256), (300, 2064)):
        run_grouped(g, counts, N, K, kind)


@pytest.mark.parametrize("kind", list(TYPES))
def test_grouped_strides(kind):
    g = gen(5)
    for counts in ([3, 0, 20], [40, 90], [200, 300]):
        run_grouped(g, counts, 70, 128, kind, ld=(16, 32, 4), group_pad=16)           # aligned, padded
        run_grouped(g, counts, 70, 128, kind, ld=(1, 0, 1), start=(0, 0, 1))          # A's rows misaligned
        run_grouped(g, counts, 70, 128, kind, ld=(0, 3, 0), group_pad=5)              # B's
        run_grouped(g, counts, 70, 128, kind, start=(1, 0, 0))
        run_grouped(g, counts, 70, 128, kind, start=(0, 7, 3), ld=(0, 0, 5))


def test_grouped_rows():
    """No index (the rows themselves), the same one often, a few rows of A, and entries outside A."""
    g = gen(6)
    for N, K in ((64, 256), (33, 100)):
        for counts in ([5, 0, 30], [100, 50, 200]):
            M = sum(counts)
            run_grouped(g, counts, N, K, "f32", rows="none")
            run_grouped(g, counts, N, K, "bf16", T=1, rows=torch.zeros(M, dtype=torch.int32))
            rows = torch.randint(0, 9, (M,), generator=g, dtype=torch.int32)
            rows[0], rows[M // 2], rows[M - 1], rows[3] = -1, 9, 2 ** 31 - 1, -2 ** 31
            run_grouped(g, counts, N, K, "f16", T=9, rows=rows)


def test_grouped_rows_behind_the_last_group():
    g = gen(7)
    for counts in ([1, 2], [20, 0, 40], [150, 300]):
        for K in (128, 99):
            run_grouped(g, counts, 48, K, "bf16", slack=77)
            run_grouped(g, [0] * len(counts), 48, K, "bf16", slack=50)


def test_grouped_offsets_that_lead_nowhere():
    """Offsets past C, negative or falling reach no memory outside C's rows."""
    g = gen(8)
    A, B = s8(g, 40, 64).cuda(), s8(g, 3, 20, 64).cuda()
    sa, sb = scales(g, 40).cuda(), scales(g, 3, 20).cuda()
    for ends in ([0, 10, 20, 10 ** 9], [-5, 10, 2 ** 31 - 1, -2 ** 31], [0, 30, 5, 40], [39, 40, 41, 42]):
        buf = torch.full((60, 20), SENTINEL, device="cuda")
        t.grouped_gemm(A, sa, B, sb, torch.tensor(ends, dtype=torch.int32).cuda(), out=buf[10:50])
        torch.cuda.synchronize()
        assert (buf[:10] == SENTINEL).all() and (buf[50:] == SENTINEL).all()


def test_grouped_extreme_sums():
    """The longest K with every product at its largest: the sum is exact, no wrap."""
    K = 131071
    for counts, N in (([2, 1], 3), ([70], 20)):
        M = sum(counts)
        A = torch.full((M, K), -128, dtype=torch.int8)
        B = torch.full((len(counts), N, K), -128, dtype=torch.int8)
        A[1] = 127
        ends = [0] + torch.tensor(counts).cumsum(0).tolist()
        sa, sb = torch.ones(M), torch.ones(len(counts), N)
        got = t.grouped_gemm(A.cuda(), sa.cuda(), B.cuda(), sb.cuda(), torch.tensor(ends, dtype=torch.int32).cuda(),
                             dtype=torch.float32).cpu()
        assert (got[0] == float(128 * 128 * K)).all() and (got[1] == torch.tensor(-127.0 * 128 * K)).all()


def test_grouped_far_operands():
    """Groups, rows of A and rows of C that start past 2^31 bytes."""
    g = gen(9)
    G, N, K, M = 4, 40, 256, 90
    big = 2 ** 30 + 16
    Bbuf = torch.zeros(3 * big + N * K, dtype=torch.int8, device="cuda")
    Bv = torch.as_strided(Bbuf, (G, N, K), (big, K, 1))
    B = s8(g, G, N, K)
    Bv.copy_(B.cuda())
    lda = 2 ** 25
    Abuf = torch.zeros(M * lda, dtype=torch.int8, device="cuda")
    Av = Abuf.view(M, lda)[:, :K]
    A = s8(g, M, K)
    Av.copy_(A.cuda())
    ldc = 2 ** 25
    out = torch.full((M * ldc,), SENTINEL, dtype=torch.bfloat16, device="cuda").view(M, ldc)[:, :N]
    sa, sb = scales(g, M), scales(g, G, N)
    for ends in ([0, 3, 10, 11, 90], [0, 0, 0, 0, 90]):
        note(f"[case] far {ends}")
        out.fill_(SENTINEL)
        t.grouped_gemm(Av, sa.cuda(), Bv, sb.cuda(), torch.tensor(ends, dtype=torch.int32).cuda(), out=out)
        want, written = grouped_reference(A, sa, B, sb, ends, None, M)
        check_grouped(out, want, written, SENTINEL, torch.bfloat16, f"far {ends}")


def test_dense_form():
    """One group without offsets: the dense scaled product, weights 2-D or 3-D."""
    g = gen(10)
    for M, N, K in ((1, 300, 512), (20, 64, 99), (130, 200, 1024)):
        A, B, sa, sb = s8(g, M, K), s8(g, N, K), scales(g, M), scales(g, N)
        want, written = grouped_reference(A, sa, B[None], sb[None], [0, M], None, M)
        got = t.grouped_gemm(A.cuda(), sa.cuda(), B.cuda(), sb.cuda())
        check_grouped(got, want, written, SENTINEL, torch.bfloat16, "dense")
        assert torch.equal(got, t.grouped_gemm(A.cuda(), sa.cuda(), B.cuda()[None], sb.cuda()[None]))
        acc = t.gemm(A.cuda(), B.cuda(), True).cpu()
        one = t.grouped_gemm(A.cuda(), torch.ones(M).cuda(), B.cuda(), torch.ones(N).cuda(), dtype=torch.float32)
        assert torch.equal(one.cpu(), acc.float())


def test_grouped_no_k_and_no_rows():
    out = torch.full((6, 5), SENTINEL, device="cuda")
    off = torch.tensor([0, 2, 4], dtype=torch.int32).cuda()
    t.grouped_gemm(torch.empty(6, 0, dtype=torch.int8).cuda(), torch.ones(6).cuda(),
                   torch.empty(2, 5, 0, dtype=torch.int8).cuda(), torch.ones(2, 5).cuda(), off, out=out)
    assert (out[:4] == 0).all() and (out[4:] == SENTINEL).all()
    none = t.grouped_gemm(torch.empty(0, 16, dtype=torch.int8).cuda(), torch.empty(0).cuda(),
                          torch.ones(2, 5, 16, dtype=torch.int8).cuda(), torch.ones(2, 5).cuda(), off * 0)
    assert none.shape == (0, 5)


def test_grouped_graph_and_streams():
    """A captured call sees the offsets, rows and values of each replay; two calls at once on two streams."""
    g = gen(11)
    for M, N, K in ((40, 96, 256), (400, 128, 512)):
        T, G = 25, 6
        A, B, sa, sb = s8(g, T, K), s8(g, G, N, K), scales(g, T), scales(g, G, N)
        dA, dB, dsa, dsb = A.cuda(), B.cuda(), sa.cuda(), sb.cuda()
        off = torch.zeros(G + 1, dtype=torch.int32, device="cuda")
        rows = torch.zeros(M, dtype=torch.int32, device="cuda")
        out = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            t.grouped_gemm(dA, dsa, dB, dsb, off, rows=rows, out=out)
        side = torch.cuda.Stream()
        for k in range(4):
            ends = [0] + sorted(torch.randint(0, M + 1, (G,), generator=g).tolist())
            r = torch.randint(-1, T, (M,), generator=g, dtype=torch.int32)
            off.copy_(torch.tensor(ends, dtype=torch.int32))
            rows.copy_(r)
            out.fill_(SENTINEL)
            graph.replay()
            torch.cuda.synchronize()
            want, written = grouped_reference(A, sa, B, sb, ends, r, M)
            check_grouped(out, want, written, SENTINEL, torch.bfloat16, f"replay {k}")
            eager = torch.full_like(out, SENTINEL)
            other = torch.full_like(out, SENTINEL)
            side.wait_stream(torch.cuda.current_stream())
            t.grouped_gemm(dA, dsa, dB, dsb, off, rows=rows, out=other, stream=side)
            t.grouped_gemm(dA, dsa, dB, dsb, off, rows=rows, out=eager)
            torch.cuda.current_stream().wait_stream(side)
            assert torch.equal(out, eager) and torch.equal(out, other)


# ----- block-scaled e4m3 ---------------------------------------------------------------

def e4m3(g, *shape):
    return (torch.randn(*shape, generator=g) * 60).clamp(-448, 448).to(torch.float8_e4m3fn)


def run_f8(g, M, N, K, kind, ld=(0, 0, 0), start=(0, 0, 0), scale_pad=0):
    kb, nb = -(-K // 128), -(-N // 128)
    A, B = e4m3(g, M, K), e4m3(g, N, K)
    sa, sb = scales(g, M, kb), scales(g, nb, kb) - 0.002  # some negative
    what = f"f8 {M}x{N}x{K} {kind} ld={ld} start={start}"
    note("[case] " + what)
    Av, _ = strided(A, K + ld[0], start[0])
    Bv, _ = strided(B, K + ld[1], start[1])
    sav, _ = strided(sa, kb + scale_pad, scale_pad)
    sbv, _ = strided(sb, kb + 2 * scale_pad, scale_pad)
    out, obuf = strided(torch.full((M, N), SENTINEL, dtype=TYPES[kind]), N + ld[2], start[2])
    before = obuf.clone()
    got = t.gemm_f8(Av, sav, Bv, sbv, out=out)
    torch.cuda.synchronize()
    want = f8_reference(A, sa, B, sb)
    check_f8(got, want, K, TYPES[kind], what)
    out.fill_(SENTINEL)
    assert torch.equal(obuf, before), f"{what}: wrote outside C"


F8_SIZES = [(1, 1, 1), (1, 16, 128), (3, 100, 256), (16, 300, 384), (17, 5, 130), (31, 64, 1000), (33, 129, 640),
            (64, 257, 144), (65, 31, 127), (100, 384, 272), (128, 128, 128), (129, 256, 512), (200, 130, 777),
            (256, 256, 256), (257, 511, 1040), (300, 1000, 384), (513, 300, 2048), (700, 640, 129)]


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("size", F8_SIZES, ids=lambda s: "x".join(map(str, s)))
def test_f8_sizes(size, kind):
    run_f8(gen(sum(size)), *size, kind)


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("M", [5, 30, 90, 400])
def test_f8_strides(M, kind):
    g = gen(M)
    run_f8(g, M, 200, 256, kind, ld=(16, 32, 4), scale_pad=3)
    run_f8(g, M, 200, 256, kind, ld=(1, 0, 0))
    run_f8(g, M, 200, 256, kind, ld=(0, 5, 1), start=(0, 3, 1))
    run_f8(g, M, 200, 256, kind, start=(9, 0, 5), scale_pad=1)


def test_f8_no_k():
    for kind in TYPES.values():
        for M, N in ((3, 5), (40, 300), (300, 20000)):
            e = torch.empty(M, 0, dtype=torch.float8_e4m3fn, device="cuda")
            out = torch.full((M, N), SENTINEL, dtype=kind, device="cuda")
            t.gemm_f8(e, torch.empty(M, 0, device="cuda"), torch.empty(N, 0, dtype=e.dtype, device="cuda"),
                      torch.empty(-(-N // 128), 0, device="cuda"), out=out)
            assert (out == 0).all()


# (few rows; every LDS tile: 64 x 128 up to 256 x 256, in both forms; unaligned ones)
LARGE = [(70, 11008, 512), (256, 16384, 256), (1024, 4096, 640), (2100, 4096, 256), (4096, 4096, 384),
         (333, 16400, 272), (600, 8200, 200)]


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("size", LARGE, ids=lambda s: "x".join(map(str, s)))
def test_f8_large(size, kind):
    """Sizes at which the choice takes each kernel, with leading dimensions off the sizes."""
    run_f8(gen(sum(size)), *size, kind, ld=(16, 0, 8) if size[2] % 16 == 0 else (0, 0, 1))


@pytest.mark.parametrize("kind", ["f16", "f32"])
@pytest.mark.parametrize("case", [([3] * 40, 2048, 256), ([70, 0, 200, 31] * 8, 1024, 256), ([300, 900, 50, 0], 4096, 128),
                                  ([2500, 1, 1500, 60], 2048, 128), ([130] * 12, 1100, 200), ([1] * 150, 500, 512)],
                         ids=lambda c: f"{len(c[0])}x{max(c[0])}")
def test_grouped_large(case, kind):
    counts, N, K = case
    run_grouped(gen(N + K + len(counts)), counts, N, K, kind, T=100, slack=5)


def test_grouped_many_groups_and_bad_offsets():
    """More groups than a wave has lanes by far, and offsets whose groups all overlap."""
    g = gen(12)
    G, N, K = 5000, 16, 32
    run_grouped(g, [i % 7 == 0 for i in range(G)], N, K, "bf16")
    A, sa = s8(g, 4000, K).cuda(), scales(g, 4000).cuda()
    B, sb = s8(g, G, N, K).cuda(), scales(g, G, N).cuda()
    bad = (torch.arange(G + 1, dtype=torch.int32) % 2 * 4000).cuda()
    buf = torch.full((4100, N), SENTINEL, device="cuda")
    t.grouped_gemm(A, sa, B, sb, bad, out=buf[50:4050])
    torch.cuda.synchronize()
    assert (buf[:50] == SENTINEL).all() and (buf[4050:] == SENTINEL).all()


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("M", [2, 24, 60, 300, 3000])
def test_f8_special_values(M, kind):
    """NaN reaches its row or column, zero scales give zeros, the largest and smallest magnitudes hold."""
    g = gen(20 + M)
    N, K = 150, 400
    A, B = e4m3(g, M, K), e4m3(g, N, K)
    sa, sb = scales(g, M, 4), scales(g, 2, 4)
    sa[0] = 0
    bad = A.clone().view(torch.int8)
    bad[1, 399] = 0x7f
    got = t.gemm_f8(bad.view(torch.float8_e4m3fn).cuda(), sa.cuda(), B.cuda(), sb.cuda(), dtype=TYPES[kind]).cpu()
    assert got[1].isnan().all() and (got[0] == 0).all() and not got[torch.arange(M) != 1].isnan().any()
    badb = B.clone().view(torch.int8)
    badb[149, 0] = -1
    got = t.gemm_f8(A.cuda(), sa.cuda(), badb.view(torch.float8_e4m3fn).cuda(), sb.cuda(), dtype=TYPES[kind]).cpu()
    assert got[:, 149].isnan().all() and not got[:, :149].isnan().any()
    for value in (448.0, 2.0 ** -9):
        a = torch.full((M, K), value).to(torch.float8_e4m3fn)
        got = t.gemm_f8(a.cuda(), torch.ones(M, 4).cuda(), a[:1].expand(N, K).contiguous().cuda(),
                        torch.ones(2, 4).cuda(), dtype=TYPES[kind]).cpu()
        assert (got == torch.tensor(value * value * K).to(TYPES[kind])).all()


def test_f8_far_operands():
    g = gen(30)
    M, N, K, ld = 140, 260, 256, 2 ** 24 + 16
    A, B = e4m3(g, M, K), e4m3(g, N, K)
    Av = torch.zeros(M * ld, dtype=torch.int8, device="cuda").view(torch.float8_e4m3fn).view(M, ld)[:, :K]
    Bv = torch.zeros(N * ld, dtype=torch.int8, device="cuda").view(torch.float8_e4m3fn).view(N, ld)[:, :K]
    Av.copy_(A.cuda())
    Bv.copy_(B.cuda())
    sa, sb = scales(g, M, 2), scales(g, 3, 2)
    out = torch.zeros(M * ld, dtype=torch.bfloat16, device="cuda").view(M, ld)[:, :N]
    for rows in (M, 10):
        t.gemm_f8(Av[:rows], sa[:rows].cuda(), Bv, sb.cuda(), out=out[:rows])
        want = f8_reference(A[:rows], sa[:rows], B, sb)
        check_f8(out[:rows], want, K, torch.bfloat16, f"far {rows}")


def test_f8_graph_and_streams():
    g = gen(31)
    for M, N, K in ((9, 400, 512), (300, 256, 640)):
        A, sa = e4m3(g, M, K).cuda(), scales(g, M, K // 128).cuda()
        B, sb = e4m3(g, N, K).cuda(), scales(g, -(-N // 128), K // 128).cuda()
        out = torch.empty(M, N, dtype=torch.float16, device="cuda")
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            t.gemm_f8(A, sa, B, sb, out=out)
        side = torch.cuda.Stream()
        for k in range(4):
            A.copy_(e4m3(g, M, K))
            graph.replay()
            torch.cuda.synchronize()
            side.wait_stream(torch.cuda.current_stream())
            other = t.gemm_f8(A, sa, B, sb, dtype=torch.float16, stream=side)
            eager = t.gemm_f8(A, sa, B, sb, dtype=torch.float16)
            torch.cuda.current_stream().wait_stream(side)
            assert torch.equal(out, eager) and torch.equal(out, other)
        want = f8_reference(A.cpu(), sa.cpu(), B.cpu(), sb.cpu())
        check_f8(out, want, K, torch.float16, "last replay")


# ----- as a layer uses them together ---------------------------------------------------

def test_experts_layer():
    """Norm with the residual, the experts' first product, activation, second product."""
    g = gen(40)
    T, H, I, G, top = 37, 512, 384, 6, 2
    x, r = torch.randn(T, H, generator=g).bfloat16(), torch.randn(T, H, generator=g).bfloat16()
    w = torch.randn(H, generator=g).bfloat16()
    w1, s1 = s8(g, G, 2 * I, H), scales(g, G, 2 * I) * 0.02
    w2, s2 = s8(g, G, H, I), scales(g, G, H) * 0.02
    expert = torch.randint(0, G - 1, (T * top,), generator=g)  # the last expert gets no rows
    order = torch.argsort(expert, stable=True)
    rows = (torch.arange(T * top) // top)[order].int()
    ends = [0] + torch.bincount(expert, minlength=G).cumsum(0).tolist()
    off = torch.tensor(ends, dtype=torch.int32).cuda()

    q, s, h = t.rms_norm(x.cuda(), w.cuda(), residual=r.cuda())
    up = t.grouped_gemm(q, s, w1.cuda(), s1.cuda(), off, rows=rows.cuda())
    q2, sq2 = t.swiglu(up[:, :I], up[:, I:])
    out = t.grouped_gemm(q2, sq2, w2.cuda(), s2.cuda(), off, dtype=torch.float32)
    torch.cuda.synchronize()
    want, written = grouped_reference(q.cpu(), s.cpu(), w1, s1, ends, rows, T * top)
    check_grouped(up, want, written, 0, torch.bfloat16, "first product")
    want, written = grouped_reference(q2.cpu(), sq2.cpu(), w2, s2, ends, None, T * top)
    check_grouped(out, want, written, 0, torch.float32, "second product")
    # against the layer without 8-bit rounding: an 8-bit operand is off by at most half a step,
    # 1/254 of its row's largest value; with rows whose largest value is below 6 times their
    # root mean square that is 2.4% of the row's norm for each of the two operands at worst
    hf = (x.float() + r.float()).bfloat16().double()
    y = hf / torch.sqrt((hf * hf).mean(1, keepdim=True) + 1e-6) * w.double()
    assert torch.equal(h.cpu().double(), hf)
    ref = torch.zeros(T * top, H, dtype=torch.float64)
    for e in range(G):
        idx = rows[ends[e]:ends[e + 1]].long()
        u = y[idx] @ (w1[e].double() * s1[e].double()[:, None]).t()
        a = u[:, :I] / (1 + torch.exp(-u[:, :I])) * u[:, I:]
        ref[ends[e]:ends[e + 1]] = a @ (w2[e].double() * s2[e].double()[:, None]).t()
    assert (out.cpu().double() - ref).norm() < 0.05 * ref.norm()


def test_dense_layer_f8():
    """The same with e4m3 operands and dense products."""
    g = gen(41)
    T, H, I = 50, 640, 400
    x, w = torch.randn(T, H, generator=g).half(), torch.rand(H, generator=g).half()
    w1, s1 = e4m3(g, 2 * I, H), scales(g, -(-2 * I // 128), 5) * 0.01
    w2, s2 = e4m3(g, H, I), scales(g, 5, 4) * 0.01
    q, s = t.rms_norm(x.cuda(), w.cuda(), fmt="f8")
    up = t.gemm_f8(q, s, w1.cuda(), s1.cuda(), dtype=torch.float16)
    q2, sq2 = t.swiglu(up[:, :I], up[:, I:], fmt="f8")
    out = t.gemm_f8(q2, sq2, w2.cuda(), s2.cuda(), dtype=torch.float32)
    torch.cuda.synchronize()
    want = f8_reference(q.cpu(), s.cpu(), w1, s1)
    check_f8(up, want, H, torch.float16, "first product")
    want = f8_reference(q2.cpu(), sq2.cpu(), w2, s2)
    check_f8(out, want, I, torch.float32, "second product")


# For each stream kernel a product that it is taken for: rows and columns that
# end inside tiles, chunks of K that the waves share unevenly, a last one of 16
# bytes (aligned operands) or of 77.
STREAMED = [(5, 1999), (16, 4111), (30, 3999), (64, 3999), (128, 3999), (200, 3999)]
UNALIGNED = [(3, 4201), (16, 1999), (13, 5001), (30, 1501), (60, 1501), (100, 999), (150, 1501), (270, 1501)]
STREAM_CASES = [(M, N, 2832) for M, N in STREAMED] + [(M, N, 1101) for M, N in UNALIGNED]


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("size", STREAM_CASES, ids=lambda s: "x".join(map(str, s)))
def test_f8_streams(size, kind):
    run_f8(gen(sum(size)), *size, kind, ld=(32, 16, 1), scale_pad=1)


@pytest.mark.parametrize("size", STREAM_CASES, ids=lambda s: "x".join(map(str, s)))
def test_grouped_streams(size):
    """The same as one group, and shared by three of which one is empty."""
    M, N, K = size
    g = gen(sum(size))
    run_grouped(g, [M], N, K, "bf16", T=M + 3, ld=(16, 0, 3))
    run_grouped(g, [M // 2, 0, M - M // 2], N, K, "f32", T=M + 3)


@pytest.mark.parametrize("counts", [[1] * 40, [3, 0, 20, 16], [0, 1, 2, 33, 8, 0, 1, 1]], ids=lambda c: f"{len(c)}x{max(c)}")
def test_grouped_stream_of_few_rows(counts):
    g = gen(max(counts))
    for N, K in ((700, 2832), (699, 2832), (129, 112), (33, 4096)):
        run_grouped(g, counts, N, K, "f16", slack=5)


def test_streams_captured_together():
    """Two stream products on one captured stream, replayed over changing inputs."""
    g = gen(77)
    A, B = e4m3(g, 24, 2832).cuda(), e4m3(g, 999, 2832).cuda()
    sa, sb = scales(g, 24, 23).cuda(), scales(g, 8, 23).cuda()
    A8, B8 = s8(g, 24, 1024).cuda(), s8(g, 3, 500, 1024).cuda()
    ra, rb = scales(g, 24).cuda(), scales(g, 3, 500).cuda()
    off = torch.tensor([0, 4, 4, 24], dtype=torch.int32).cuda()
    y, z = torch.empty(24, 999, device="cuda"), torch.empty(24, 500, device="cuda")
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        t.gemm_f8(A, sa, B, sb, out=y)
        t.grouped_gemm(A8, ra, B8, rb, off, out=z)
    for k in range(4):
        A.copy_(e4m3(g, 24, 2832))
        A8.copy_(s8(g, 24, 1024))
        off.copy_(torch.tensor([0, 4 + k, 5 + k, 24], dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, t.gemm_f8(A, sa, B, sb, dtype=torch.float32))
        assert torch.equal(z, t.grouped_gemm(A8, ra, B8, rb, off, dtype=torch.float32))
        check_f8(y, f8_reference(A.cpu(), sa.cpu(), B.cpu(), sb.cpu()), 2832, torch.float32, f"replay {k}")


@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_more_columns_than_the_smallest_tile_has_a_grid_for(kind):
    """70 million columns of a row: the products of integers that fp32 holds, rounded once."""
    g = torch.Generator(device="cuda").manual_seed(50)
    N, K = 70_000_000, 16
    note(f"[case] 1 x {N} x {K} {kind}")
    A = torch.randint(-128, 128, (1, K), device="cuda", generator=g, dtype=torch.int8)
    B = torch.randint(-128, 128, (N, K), device="cuda", generator=g, dtype=torch.int8)
    ones = torch.ones(N, device="cuda")
    want = sum(B[:, k].float() * A[0, k].float() for k in range(K)).to(TYPES[kind])
    got = t.grouped_gemm(A, ones[:1], B, ones, dtype=TYPES[kind])
    assert torch.equal(got[0], want)
    # e4m3: the values 1 .. 8, so that 8 of their products keep within the instruction's 13 bits
    A8, B8 = ((x & 7).float() + 1 for x in (A, B))
    want = sum(B8[:, k] * A8[0, k] for k in range(K)).to(TYPES[kind])
    A8, B8 = A8.to(torch.float8_e4m3fn), B8.to(torch.float8_e4m3fn)
    blocks = ones[:-(-N // 128)][:, None]
    got = t.gemm_f8(A8, ones[:1, None], B8, blocks, dtype=TYPES[kind])
    assert torch.equal(got[0], want)


LOUD_CASES = STREAM_CASES + [(M, N, K) for M, N, K in LARGE if M * N < 10 ** 7] + \
    [(700, 640, 1408), (2100, 4096, 256), (1000, 1501, 1101)]


@pytest.mark.parametrize("kind", ["f16", "f32"])
@pytest.mark.parametrize("size", LOUD_CASES, ids=lambda s: "x".join(map(str, s)))
def test_f8_large_products_that_cancel(size, kind):
    """Two products of +-448^2 among each 16, the others 1: with sums in 32
    bits every partial sum is a whole number below 2^24, so the result is the
    exact one, rounded once to the type."""
    M, N, K = size
    note(f"[case] cancelling {size} {kind}")
    a, b = torch.ones(M, K), torch.ones(N, K)
    g = gen(sum(size))
    a[:, 0::16], b[:, 0::16] = 448, 448
    a[:, 5::16], b[:, 5::16] = -448, 448
    if K % 16 in range(1, 6):  # a last piece that holds the first of the two only
        a[:, K - K % 16] = 1
        b[:, K - K % 16] = 1
    some = torch.arange(K) % 16 == 9  # and values that differ from row to row
    a[:, some] = torch.randint(-8, 9, (M, int(some.sum())), generator=g).float()
    want = a.double().mm(b.double().t())
    kb, nb = -(-K // 128), -(-N // 128)
    f8 = torch.float8_e4m3fn
    got = t.gemm_f8(a.to(f8).cuda(), torch.ones(M, kb).cuda(), b.to(f8).cuda(), torch.ones(nb, kb).cuda(),
                    dtype=TYPES[kind])
    assert torch.equal(got.cpu(), want.to(TYPES[kind]))


@pytest.mark.parametrize("size", [(16, 300, 2832), (100, 999, 1101), (513, 640, 2048)], ids=lambda s: "x".join(map(str, s)))
def test_f8_bf16_sums_of_loud_channels(size):
    """bf16 results within the documented bound of the instruction's sums, loud channels or not."""
    M, N, K = size
    for loud in (1, 30):
        g = gen(sum(size))
        A, B = torch.randn(M, K, generator=g) * 8, e4m3(g, N, K)
        A[:, 7::128] *= loud
        A = A.clamp(-448, 448).to(torch.float8_e4m3fn)
        sa, sb = scales(g, M, -(-K // 128)), scales(g, -(-N // 128), -(-K // 128))
        got = t.gemm_f8(A.cuda(), sa.cuda(), B.cuda(), sb.cuda())
        want, size_of, _ = f8_reference(A, sa, B, sb)
        # 7 of 8 consecutive products, each by less than 2^-13 of the largest of
        # them; sums in 32 bits and the type's rounding as check_f8 has them
        # (127 * 2^-23 + 40 * 2^-24 < 2^-15)
        largest = [torch.nn.functional.pad(x.double().abs() * s.double().repeat_interleave(128, 1)[:, :K].abs(),
                                           (0, -K % 8)).view(x.shape[0], -1, 8).amax(2)
                   for x, s in ((A, sa), (B, sb.repeat_interleave(128, 0)[:N]))]
        off = (got.cpu().double() - want).abs()
        absolute = 7 * largest[0] @ largest[1].t() * 2.0 ** -13 + size_of * 2.0 ** -15
        assert (off <= absolute * (1 + 2.0 ** -8) + want.abs() * 2.0 ** -8).all()


def test_f8_bf16_products_beside_a_loud_one():
    """What a product of 448^2 does to small ones in bf16 results: cut toward
    zero to multiples of 8 among the same 8 consecutive ones, kept elsewhere.
    The loud one is taken back in the next block of 128, where sums are fp32."""
    M, K = 256, 256
    for loud in (0, 5, 15, 40, 127):
        for small in (1.0, -3.0, 8.0, 9.0, -15.0, 44.0):
            a, b = torch.zeros(M, K), torch.zeros(16, K)
            a[torch.arange(128), torch.arange(128)] = small
            a[:, loud], a[:, 128] = 448, -448
            b[:, :128], b[:, loud], b[:, 128] = 1, 448, 448
            one = torch.ones(M, 2).cuda()
            a, b = (x.to(torch.float8_e4m3fn).cuda() for x in (a, b))
            want = torch.full((128,), small)
            want[loud // 8 * 8:loud // 8 * 8 + 8] = float(torch.tensor(small / 8).trunc()) * 8
            want[loud] = 0  # the loud one itself
            got = t.gemm_f8(a, one, b, one[:1])
            assert torch.equal(got[:128].float().cpu(), want[:, None].expand(128, 16))
            want = torch.full((128,), small)
            want[loud] = 0
            for kind in (torch.float16, torch.float32):  # sums in 32 bits
                got = t.gemm_f8(a, one, b, one[:1], dtype=kind)
                assert torch.equal(got[:128].float().cpu(), want[:, None].expand(128, 16))
