"""RMS norm and gated activation with 8-bit outputs against 64-bit forms."""
import pytest
import torch

import tiled_dense_int8_amd as t
from helpers import note
from layer_helpers import (TYPES, act_values, check_quantised, e4m3_nearest, norm_steps, norm_sum, norm_values, quantise,
                           strided)

pytestmark = pytest.mark.gpu

# one of every row shape, its ends, odd lengths, and rows that are read twice
LENGTHS = [1, 7, 8, 100, 127, 128, 129, 511, 512, 513, 2047, 2048, 2049, 4096, 4100, 5000, 8192, 8193, 16384, 16385,
           20011, 40000]


def gen(seed):
    return torch.Generator().manual_seed(seed)


def run_norm(x, w, r, eps, fmt, what):
    note(f"[norm] {what}")
    got = t.rms_norm(x.cuda(), w.cuda(), eps, residual=None if r is None else r.cuda(), fmt=fmt)
    torch.cuda.synchronize()
    if r is not None:
        assert torch.equal(got[2].cpu().view(torch.int8), norm_sum(x, r).view(torch.int8)), what
    v, inv = norm_values(x, w, r, eps)
    check_quantised(got[0], got[1], v, inv, fmt, what, norm_steps(x))


@pytest.mark.parametrize("fmt", ["s8", "f8"])
@pytest.mark.parametrize("kind", list(TYPES))
def test_norm_lengths(kind, fmt):
    g = gen(1)
    for i, H in enumerate(LENGTHS):
        T = 1 + i % 5
        x = torch.randn(T, H, generator=g).to(TYPES[kind])
        w = (1 + 0.2 * torch.randn(H, generator=g)).to(TYPES[kind])
        r = torch.randn(T, H, generator=g).to(TYPES[kind]) * 3 if i % 3 else None
        run_norm(x, w, r, 1e-5, fmt, f"{kind} {fmt} T={T} H={H} residual={r is not None}")


@pytest.mark.parametrize("fmt", ["s8", "f8"])
@pytest.mark.parametrize("kind", list(TYPES))
def test_act_lengths(kind, fmt):
    g = gen(2)
    for i, N in enumerate(LENGTHS):
        T = 1 + i % 5
        both = (torch.randn(T, 2 * N, generator=g) * 4).to(TYPES[kind]).cuda()
        what = f"{kind} {fmt} T={T} N={N}"
        note(f"[act] {what}")
        q, scale = t.swiglu(both[:, :N], both[:, N:], fmt=fmt)
        v, inv = act_values(both[:, :N].cpu(), both[:, N:].cpu())
        check_quantised(q, scale, v, inv, fmt, what)


@pytest.mark.parametrize("fmt", ["s8", "f8"])
def test_many_rows(fmt):
    g = gen(3)
    x, r = torch.randn(3001, 1024, generator=g), torch.randn(3001, 1024, generator=g)
    w = torch.randn(1024, generator=g)
    run_norm(x.bfloat16(), w.bfloat16(), r.bfloat16(), 1e-6, fmt, f"{fmt} 3001 rows")
    run_norm(x[:, :300].contiguous(), w[:300].contiguous(), None, 1e-6, fmt, f"{fmt} 3001 short rows")


def test_s8_ties_go_to_even():
    """Quotients that lie exactly between two integers: max 254, odd values."""
    x = torch.arange(-127, 128, dtype=torch.float32)[None]
    x = torch.cat([x, torch.tensor([[254.0]])], 1)
    for kind in TYPES.values():
        for n in (0, 300, 9000):  # another row shape each, the rest zeros
            row = torch.cat([x, torch.zeros(1, n)], 1).to(kind)
            run_norm(row, torch.ones(row.shape[1], dtype=kind), None, 0.0, "s8", f"ties {kind} {n}")


@pytest.mark.parametrize("kind", list(TYPES))
def test_act_values_far_out(kind):
    """Gates so negative that the exponential overflows, large ones, zeros of both signs."""
    g = torch.tensor([-1e4, -200, -104, -100, -89, -88, -87.5, -81, -80, -79, -40, -20, -1, -0.0, 0.0, 1, 20, 80, 100,
                      1e4])
    gate = g.repeat(4, 30)[:, :577].to(TYPES[kind])
    up = torch.stack([torch.ones(577), torch.full((577,), 1e3), torch.full((577,), -3e-3),
                      torch.randn(577, generator=gen(4))]).to(TYPES[kind])
    only_small = gate.clamp(max=-85)  # every value of the row is tiny
    for a in (gate, only_small):
        for fmt in ("s8", "f8"):
            q, scale = t.swiglu(a.cuda(), up.cuda(), fmt=fmt)
            v, inv = act_values(a, up)
            note(f"[act] far out {kind} {fmt}")
            if fmt == "s8":
                want, s = quantise(v, inv, fmt)
                assert torch.equal(q.cpu().double(), want.round())
                # scales below fp32's normal range round to a multiple of 2^-149
                assert ((scale.cpu().double() - s[:, 0]).abs() <= s[:, 0] * 2.0 ** -23 + 2.0 ** -150).all()


@pytest.mark.parametrize("size", [1e-30, 1e-20, 1e18, 1e30])
def test_norm_extreme_magnitudes(size):
    """Products that leave fp32's range, squares that overflow it."""
    g = gen(5)
    for kind in ("f32", "bf16"):
        for H in (200, 3000, 17000):
            x = (torch.randn(2, H, generator=g) * size).to(TYPES[kind])
            w = (torch.randn(H, generator=g) * (size if size < 1 else 1)).to(TYPES[kind])
            h = x.double()
            v, inv = h * w.double(), 1 / torch.sqrt((h * h).mean(1) + 0.0)
            for fmt in ("s8", "f8"):
                note(f"[norm] {kind} {size} H={H} {fmt}")
                q, scale = t.rms_norm(x.cuda(), w.cuda(), 0.0, fmt=fmt)
                check_quantised(q, scale, v, inv, fmt, f"{kind} {size} {H} {fmt}", norm_steps(x))


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("H", [100, 1000, 20000])
def test_zeros_infinities_nan(kind, H):
    """Rows of zeros; rows (f8: blocks) that hold an infinity or NaN."""
    g = gen(6)
    x = torch.randn(6, H, generator=g).to(TYPES[kind])
    w = torch.ones(H, dtype=TYPES[kind])
    x[1] = 0
    x[2, H // 2] = float("inf")
    x[3, H - 1] = float("nan")
    x[4, 0] = float("-inf")
    for eps in (0.0, 1e-6):
        q, scale = t.rms_norm(x.cuda(), w.cuda(), eps)
        q, scale = q.cpu(), scale.cpu()
        assert (q[1:5] == 0).all() and scale[1] == 0 and scale[2:5].isnan().all()
        good = torch.tensor([0, 5])
        v, inv = norm_values(x[good], w, None, eps)
        check_quantised(q[good], scale[good], v, inv, "s8", "rows beside them", norm_steps(x))
        q, scale = t.rms_norm(x.cuda(), w.cuda(), eps, fmt="f8")
        q, scale = q.cpu().float(), scale.cpu()
        assert (q[1] == 0).all() and (scale[1] == 0).all()
        for row, col in ((2, H // 2), (3, H - 1), (4, 0)):
            b = col // 128
            assert (q[row, b * 128:(b + 1) * 128] == 0).all() and scale[row, b].isnan()
        assert scale[3].isnan().all()                      # NaN in the row's root
        rest = [b for b in range(scale.shape[1]) if b != H // 2 // 128]
        assert (scale[2, rest] == 0).all()                 # finite values over an infinite root
    for bad in (float("inf"), float("-inf"), float("nan")):
        for where in (0, 1):
            gate, up = x[[0, 5]].clone(), x[[5, 0]].clone()
            (gate, up)[where][1, H // 3] = bad
            q, scale = t.swiglu(gate.cuda(), up.cuda())
            assert (q[1] == 0).all() and scale[1].isnan() and scale[0].isfinite()
            q, scale = t.swiglu(gate.cuda(), up.cuda(), fmt="f8")
            b = H // 3 // 128
            assert (q[1, b * 128:(b + 1) * 128].float() == 0).all() and scale[1, b].isnan()
            assert scale.isnan().sum() == 1


@pytest.mark.parametrize("fmt", ["s8", "f8"])
@pytest.mark.parametrize("kind", list(TYPES))
def test_strides_and_offsets(kind, fmt):
    """Odd leading dimensions and starts, padding left as it was, in place."""
    g = gen(7)
    for T, H in ((5, 300), (3, 2051), (2, 17001)):
        x = torch.randn(T, H, generator=g).to(TYPES[kind])
        r = torch.randn(T, H, generator=g).to(TYPES[kind])
        w = torch.randn(H, generator=g).to(TYPES[kind])
        xv, _ = strided(x, H + 3, 1)
        rv, rbuf = strided(r, H + 5, 3)
        wv, _ = strided(w[None], None, 5)
        qd = torch.int8 if fmt == "s8" else torch.float8_e4m3fn
        qv, qbuf = strided(torch.zeros(T, H).to(qd), H + 7, 3)
        nb = -(-H // 128)
        scale = torch.zeros(T) if fmt == "s8" else torch.zeros(T, nb)
        if fmt == "f8":
            scale, _ = strided(scale, nb + 2, 1)
        else:
            scale = scale.cuda()
        before_r, before_q = rbuf.clone(), qbuf.clone()
        q, s, h = t.rms_norm(xv, wv[0], 1e-6, residual=rv, fmt=fmt, sum_out=rv, out=qv, scale=scale)
        assert h is rv and q is qv
        v, inv = norm_values(x, w, r, 1e-6)
        check_quantised(q, s, v, inv, fmt, f"{kind} {fmt} {T}x{H}", norm_steps(x))
        assert torch.equal(rv.cpu().view(torch.int8), norm_sum(x, r).view(torch.int8))
        # everything outside the windows is as it was
        rv.copy_(before_r[3:3 + T * (H + 5)].view(T, H + 5)[:, :H])
        assert torch.equal(rbuf.view(torch.int8), before_r.view(torch.int8))
        qv.view(torch.int8).copy_(before_q.view(torch.int8)[3:3 + T * (H + 7)].view(T, H + 7)[:, :H])
        assert torch.equal(qbuf.view(torch.int8), before_q.view(torch.int8))
        # x in place of the residual, and the sum thrown away
        x2 = x.cuda()
        _, _, h = t.rms_norm(x2, w.cuda(), 1e-6, residual=r.cuda(), fmt=fmt, sum_out=x2)
        assert h is x2 and torch.equal(x2.cpu().view(torch.int8), norm_sum(x, r).view(torch.int8))
        qa = torch.empty(T, H, dtype=qd, device="cuda")
        sa = torch.empty(s.shape, device="cuda")
        xc, rc, wc = x.cuda(), r.cuda(), w.cuda()
        args = [t._TYPES[x.dtype], T, H, xc.data_ptr(), H, rc.data_ptr(), H, wc.data_ptr(), 1e-6, None, 0,
                qa.data_ptr(), H, sa.data_ptr()]
        stream = torch.cuda.current_stream().cuda_stream
        assert (t.rmsnorm_quant_s8(*args, stream) if fmt == "s8" else t.rmsnorm_quant_f8(*args, nb, stream)) == t.OK
        check_quantised(qa, sa, v, inv, fmt, "sum not kept", norm_steps(x))


def test_rows_past_32_bit_offsets():
    """Rows that start past 2^31 elements of x, the sum and q."""
    T, H, ld = 5, 600, 2 ** 29 + 8
    x = torch.zeros(T * ld, dtype=torch.bfloat16, device="cuda").view(T, ld)[:, :H]
    q = torch.zeros(T * ld, dtype=torch.int8, device="cuda").view(T, ld)[:, :H]
    src = torch.randn(T, H, generator=gen(8)).bfloat16()
    x.copy_(src.cuda())
    w = torch.ones(H, dtype=torch.bfloat16)
    r = torch.randn(T, H, generator=gen(9)).bfloat16()
    got, scale, h = t.rms_norm(x, w.cuda(), residual=r.cuda(), sum_out=x, out=q)
    v, inv = norm_values(src, w, r, 1e-6)
    check_quantised(got, scale, v, inv, "s8", "far rows")
    assert torch.equal(x.cpu().view(torch.int16), norm_sum(src, r).view(torch.int16))


def test_graph_and_streams():
    """Captured and replayed on changed inputs, on a side stream, and two calls at once."""
    g = gen(10)
    H = 3000
    x = torch.randn(64, H, generator=g).bfloat16().cuda()
    r = torch.randn(64, H, generator=g).bfloat16().cuda()
    w = torch.randn(H, generator=g).bfloat16().cuda()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    on_side = t.rms_norm(x, w, residual=r, fmt="f8", stream=side)
    here = t.rms_norm(x, w, residual=r, fmt="f8")
    handle = t.rms_norm(x, w, residual=r, fmt="f8", stream=side.cuda_stream)
    torch.cuda.current_stream().wait_stream(side)
    for a, b, c in zip(on_side, here, handle):
        assert torch.equal(a.view(torch.int8), b.view(torch.int8)) and torch.equal(a.view(torch.int8), c.view(torch.int8))
    q = torch.empty(64, H, dtype=torch.int8, device="cuda")
    s = torch.empty(64, device="cuda")
    y = torch.empty_like(x)
    q2, s2 = torch.empty_like(q), torch.empty_like(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        t.rms_norm(x, w, residual=r, sum_out=y, out=q, scale=s)
        t.swiglu(y, x, out=q2, scale=s2)
    for k in range(4):
        x.copy_(torch.randn(64, H, generator=g).bfloat16())
        graph.replay()
        torch.cuda.synchronize()
        e = t.rms_norm(x, w, residual=r)
        e2 = t.swiglu(e[2], x)
        for a, b in ((q, e[0]), (s, e[1]), (y, e[2]), (q2, e2[0]), (s2, e2[1])):
            assert torch.equal(a, b)


def test_more_rows_than_a_grid_holds():
    """Rows past one launch's 2^31 threads; every row by its own length-1 definition: q = 127 sign(x)."""
    T = 2 ** 25 + 70_000
    x = torch.randn(T, 1, device="cuda")
    q, scale = t.rms_norm(x, torch.ones(1, device="cuda"), 0.0)
    assert torch.equal(q, (127 * torch.sign(x)).to(torch.int8))
    want = (x[:, 0] != 0).float()  # zeros, which so many normal values contain, have scale 0
    assert ((scale * 127 - want).abs() <= 2 ** -22).all()
    q, scale = t.swiglu(x, x, fmt="f8")
    assert torch.equal(q.float(), (448 * torch.sign(x * x)))
    assert scale.shape == (T, 1) and scale[-1] > 0 and scale.isfinite().all()


def test_f8_quotients_next_to_a_border_go_by_their_fp32_form():
    """Quotients above a border between two e4m3 values by less than 2^-25 of it count as on it: ties to even."""
    H, columns = 128, []
    for border, below in ((17.0, 16.0), (19.0, 20.0), (1.0625 * 256, 256.0), (2.125, 2.0)):  # and what its tie gives
        for i in range(1, 4000):
            w = 1 + i * 2.0 ** -23
            h = torch.tensor(border * (1 + 2.0 ** -22) / w, dtype=torch.float64).float().item()
            # v = h w in whole units of 2^-60: above the border's v = border (1 + 2^-22)?
            v = int(h * 2.0 ** 30) * int(w * 2.0 ** 30)
            at = int(border * 2.0 ** 30) * (2 ** 30 + 2 ** 8)
            if h * 2.0 ** 30 == int(h * 2.0 ** 30) and 0 < v - at < at >> 26:
                columns.append((h, w, below))
                if len(columns) % 20 == 0:
                    break
    assert len(columns) == 80
    x, weight, want = torch.zeros(1, H), torch.ones(H), torch.zeros(H)
    x[0, 0], weight[0], want[0] = 448.0, 1 + 2.0 ** -22, 448.0
    for k, (h, w, q) in enumerate(columns):
        x[0, 1 + k], weight[1 + k], want[1 + k] = h, w, q
    q, _ = t.rms_norm(x.cuda(), weight.cuda(), fmt="f8")
    assert torch.equal(q.float().cpu()[0], want)


@pytest.mark.parametrize("kind", list(TYPES))
def test_act_f8_values_far_out(kind):
    """The e4m3 form of gates whose exponential overflows, of large ones and of zeros of both signs."""
    g = torch.tensor([-1e4, -200, -104, -100, -89, -88, -87.5, -81, -80, -79, -40, -20, -1, -0.0, 0.0, 1, 20, 80, 100,
                      1e4])
    gate = g.repeat(4, 30)[:, :577].to(TYPES[kind])
    up = torch.stack([torch.ones(577), torch.full((577,), 1e3), torch.full((577,), -3e-3),
                      torch.randn(577, generator=gen(4))]).to(TYPES[kind])
    for a in (gate, gate.clamp(max=-85)):
        note(f"[act] f8 far out {kind}")
        q, scale = t.swiglu(a.cuda(), up.cuda(), fmt="f8")
        v, inv = act_values(a, up)
        want, s = quantise(v, inv, "f8")
        assert torch.equal(q.cpu().float().double(), e4m3_nearest(want))
        # the largest value may be a 32-bit one, off by 10 steps of 2^-24, before
        # the scale's rounding; scales below fp32's normal range round to a
        # multiple of 2^-149
        assert ((scale.cpu().double() - s).abs() <= s * 11 * 2.0 ** -24 + 2.0 ** -150).all()


# (gate, up) beside values of 2^-60: gates below -80 whose value is nothing all
# the same, and gates so small that their half is no normal fp32 number
BESIDE = [(-128.0, 2.0 ** 33), (-96.0, 2.0 ** 33), (-100.0, 2.0 ** 39), (-90.0, 2.0 ** 34), (-81.0, 2.0 ** 32),
          (-80.5, 2.0 ** 25), (-4096.0, 2.0 ** 20), (-80.0, -2.0 ** 33), (3 * 2.0 ** -149, 2.0 ** 89),
          (5 * 2.0 ** -149, -2.0 ** 88), (7 * 2.0 ** -149, 2.0 ** 39), (2.0 ** -133, 2.0 ** 72),
          (3 * 2.0 ** -130, 2.0 ** 60), (2.0 ** 100, 2.0 ** -160 * 3), (2.0 ** 90, 2.0 ** -149)]


@pytest.mark.parametrize("fmt", ["s8", "f8"])
@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_act_far_values_beside_small_ones(kind, fmt):
    """Values whose gate or other half is far out, where the largest of the row (block) is about 2^-60."""
    for N in (5, 300, 7000, 40000):
        # among others in a vector of eight, and vectors of nothing else
        for far in (torch.arange(N) % 97 == 3, torch.arange(N) // 8 % 12 == 1):
            gate = torch.ones(len(BESIDE), N)
            up = torch.rand(len(BESIDE), N, generator=gen(11)) * 2.0 ** -60 + 2.0 ** -60
            for row, (a, b) in enumerate(BESIDE):
                gate[row, far], up[row, far] = a, b
            gate, up = gate.to(TYPES[kind]), up.to(TYPES[kind])
            what = f"{kind} {fmt} N={N}"
            note(f"[act] beside {what}")
            q, scale = t.swiglu(gate.cuda(), up.cuda(), fmt=fmt)
            v, inv = act_values(gate, up)
            check_quantised(q, scale, v, inv, fmt, what)


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("H", [300, 2500, 20000])
def test_f8_norm_blocks_beside_an_infinity_or_nan(kind, H):
    """Values over a root that is infinite are zeros, over one that is NaN are NaN: of blocks of zeros too."""
    g = gen(12)
    x = torch.randn(4, H, generator=g).to(TYPES[kind])
    x[:, 128:200] = 0
    x[:, 256:] = x[:, 256:] * (torch.arange(256, H) % 2)
    x[1, 5], x[2, 5], x[3, 5] = float("inf"), float("nan"), float("-inf")
    w = (1 + torch.rand(H, generator=g)).to(TYPES[kind])
    x[:, 200:256] = 0  # block 1 holds only zeros
    for residual in (None, torch.zeros_like(x).cuda()):
        made = t.rms_norm(x.cuda(), w.cuda(), residual=residual, fmt="f8")
        q, scale = made[0].cpu().float(), made[1].cpu()
        assert (q[1:] == 0).all() and q[0].abs().max() == 448
        assert scale[0].isfinite().all() and scale[0, 1] == 0 and scale[0, 0] > 0
        assert scale[1:, 0].isnan().all()
        assert (scale[[1, 3], 1:] == 0).all() and scale[2].isnan().all()
