"""Plain 64-bit forms of the 8-bit layer operators and tensors for their tests."""
from __future__ import annotations

import torch

BLOCK = 128
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def strided(t, ld=None, offset=0):
    """t's values in a larger buffer on the GPU: rows `ld` elements apart,
    the first one `offset` elements in.  Returns (view, whole buffer)."""
    rows, cols = t.shape
    ld = cols if ld is None else ld
    buf = torch.full((offset + rows * ld + 16,), 7, dtype=torch.int8, device="cuda").to(t.dtype)
    view = buf[offset:offset + rows * ld].view(rows, ld)[:, :cols]
    view.copy_(t.cuda())
    return view, buf


def norm_sum(x, residual):
    """x + residual as the operator rounds it (CPU)."""
    return x if residual is None else (x.float() + residual.float()).to(x.dtype)


def norm_values(x, weight, residual, eps):
    """(v, inv): v = h w and the row's 1 / root, in 64 bits on the CPU."""
    h = norm_sum(x, residual).double()
    inv = 1 / torch.sqrt((h * h).mean(1) + eps)
    return h * weight.double(), inv


def norm_steps(x):
    """check_quantised's `steps` of the norm of x."""
    return 1 if x.dtype == torch.float32 else 0


def act_values(gate, up):
    g = gate.double()
    v = g / (1 + torch.exp(-g)) * up.double()
    return v, torch.ones(gate.shape[0], dtype=torch.float64)


def quantise(v, inv, fmt):
    """(quotients in 64 bits, scales in 64 bits) of finite rows v."""
    T, H = v.shape
    top, width = (127.0, max(H, 1)) if fmt == "s8" else (448.0, BLOCK)
    quotients, scales = torch.zeros_like(v), []
    for c in range(0, H, width):
        part = v[:, c:c + width]
        m = part.abs().amax(1, keepdim=True)
        quotients[:, c:c + width] = torch.where(m > 0, part * top / m, torch.zeros_like(part))
        scales.append(torch.where(m[:, 0] > 0, m[:, 0] * inv / top, torch.zeros_like(inv)))
    return quotients, torch.stack(scales, 1)


def e4m3_nearest(t):
    """64-bit values up to 448 rounded to fp32 and then to e4m3 (3 mantissa bits, exponents from -6 on), ties to even."""
    t = t.float().double()
    _, exponent = torch.frexp(t)  # t = f * 2^exponent, 1/2 <= |f| < 1
    step = torch.exp2(((exponent - 1).clamp(min=-6) - 3).double())
    return torch.round(t / step) * step


def check_quantised(q, scale, v, inv, fmt, what, steps=10):
    """q and scale against the quotients in 64 bits.

    q: equal to the integer nearest to the quotient, or the e4m3 value nearest
    to its fp32 form, ties to even.  scale: computed in 64 bits and rounded once to fp32, half a step =
    2^-24 relative (values in fp32's normal range), plus what two 64-bit
    computations differ by (< 2^-40).  f8: a block's largest value may be a
    32-bit one, off by `steps` times 2^-24: 10 for the activation, 1 for the
    norm's product of 32-bit values, 0 for that of 16-bit values, which is
    exact in 32 bits."""
    t, want = quantise(v, inv, fmt)
    nearest = t.round() if fmt == "s8" else e4m3_nearest(t)
    bad = (q.cpu().double() if fmt == "s8" else q.cpu().float().double()) != nearest
    assert not bad.any(), f"{what}: {bad.sum()} values differ, first at {bad.nonzero()[0].tolist()}"
    scale = scale.reshape(-1, 1) if fmt == "s8" else scale
    off = (scale.cpu().double() - want).abs()
    allowed = 2.0 ** -24 * (1 + (steps if fmt == "f8" else 0)) + 2.0 ** -40
    assert (off <= want * allowed).all(), f"{what}: scales off by {(off / want).max()}"


# ----- scaled products ---------------------------------------------------------------

def output_tolerance(want, dtype, absolute, relative):
    """Largest allowed difference from `want` (64 bits): `absolute` plus
    `relative` of it from the 32-bit arithmetic, then half a step of dtype
    (none more for float32, whose rounding the arithmetic counts)."""
    info = torch.finfo(dtype)
    half = 0.0 if dtype == torch.float32 else info.eps / 2
    return absolute + want.abs() * ((1 + relative) * (1 + half) - 1) + absolute * half + info.tiny * info.eps / 2


def grouped_reference(A, a_scale, B, b_scale, ends, rows, M):
    """(result in 64 bits, rows that are written) of the grouped product (CPU tensors)."""
    out = torch.zeros(M, B.shape[1], dtype=torch.float64)
    written = torch.zeros(M, dtype=torch.bool)
    T = A.shape[0]
    for g, (lo, hi) in enumerate(zip(ends, ends[1:])):
        if hi <= lo:
            continue
        idx = rows[lo:hi].long() if rows is not None else torch.arange(lo, hi)
        inside = (idx >= 0) & (idx < T)
        safe = torch.where(inside, idx, torch.zeros_like(idx))
        acc = A[safe].double() @ B[g].double().t()  # exact: below 2^53
        out[lo:hi] = acc * a_scale[safe].double()[:, None] * b_scale[g].double() * inside[:, None]
        written[lo:hi] = True
    return out, written


def check_grouped(got, want, written, sentinel, dtype, what):
    """Rows of the groups within the rounding of an exact sum to fp32, of the
    scales' product and of their product (2^-24 each; the fourth term covers
    their squares), then of dtype; other rows untouched."""
    got = got.cpu()
    tol = output_tolerance(want[written], dtype, 0.0, 3 * 2.0 ** -24 + 2.0 ** -44)
    off = (got[written].double() - want[written]).abs()
    bad = ~(off <= tol)
    assert not bad.any(), f"{what}: {bad.sum()} values off, first at {bad.nonzero()[0].tolist()}, by {off.max()}"
    rest = got[~written]
    assert (rest == sentinel).all(), f"{what}: rows outside the groups were written"


def f8_reference(A, a_scale, B, b_scale):
    """(result, the same with every term's magnitude, the same with every
    term replaced by the largest of its 16 consecutive ones at most), in 64
    bits, of the block-scaled product (CPU tensors)."""
    M, K = A.shape
    N = B.shape[0]
    a = A.double() * a_scale.double().repeat_interleave(BLOCK, 1)[:, :K]
    b = B.double() * b_scale.double().repeat_interleave(BLOCK, 0).repeat_interleave(BLOCK, 1)[:N, :K]

    def largest(x):
        return torch.nn.functional.pad(x.abs(), (0, -K % 16)).view(x.shape[0], -1, 16).amax(2)

    return a @ b.t(), a.abs() @ b.abs().t(), 16 * largest(a) @ largest(b).t()


def check_f8(got, reference, K, dtype, what):
    """Within the error of the sums.

    With `size` the sum of all terms' magnitudes: a block's 128 exact products
    are added with at most 127 roundings of a step (2^-23, so that truncation
    is allowed too) each relative to at most its part of `size`; the scales'
    product and the multiply-add of each of the ceil(K / 128) blocks, and the
    sum of up to 16 waves' parts, round by 2^-24.  16-bit results: each of 16
    consecutive products may lose up to 2^-13 of the largest's power of two
    before."""
    want, size, pieces = reference
    got = got.cpu().double()
    blocks = -(-K // BLOCK)
    absolute = size * (127 * 2.0 ** -23 + (blocks + 17) * 2.0 ** -24) * (1 + 2.0 ** -10)
    if dtype != torch.float32:
        absolute = absolute + pieces * 2.0 ** -13
    tol = output_tolerance(want, dtype, absolute, 0.0)
    off = (got - want).abs()
    bad = ~((off <= tol) | (want.isnan() & got.isnan()))
    assert not bad.any(), f"{what}: {bad.sum()} values off, first at {bad.nonzero()[0].tolist()}, by {off.max()}"
