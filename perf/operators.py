"""The 8-bit layer operators beside the int8 product, as cases that can be timed.

Each case is one call of an operator: RMS norm with the residual's addition
and an 8-bit output, the gated activation with an 8-bit output, int8 products
grouped by expert, and the 8-bit floating-point product with a scale for each
block of 128.  `own` False computes the operator's plain form in elementary
torch operations, True calls the library.
"""
import math

import torch

own = False

E4M3_MAX = 448.0
BLOCK = 128
EPS = 1e-6
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
BYTES = {"bf16": 2, "f16": 2, "f32": 4}


# ----- cases -----------------------------------------------------------------------

def listed():
    return [
        # one generated token's norm between two layers: latency of a single row
        {"name": "norm_s8_token", "op": "norm", "fmt": "s8", "T": 1, "H": 4096, "type": "bf16", "residual": True},
        # a batch of prompts through the residual stream of a wide layer
        {"name": "norm_s8_prompts", "op": "norm", "fmt": "s8", "T": 16384, "H": 8192, "type": "bf16",
         "residual": True},
        # rows whose length is no multiple of a block or of a vector, full precision in, no residual
        {"name": "norm_s8_odd", "op": "norm", "fmt": "s8", "T": 1000, "H": 2999, "type": "f32", "residual": False},
        # the operand of the block-scaled product, half precision, last block short
        {"name": "norm_f8_prompt", "op": "norm", "fmt": "f8", "T": 4096, "H": 5000, "type": "f16", "residual": True},
        # the experts' activations while sixteen sequences decode
        {"name": "act_s8_decode", "op": "act", "fmt": "s8", "T": 64, "N": 2048, "type": "bf16"},
        # a dense layer's activations of a prompt batch
        {"name": "act_f8_prompts", "op": "act", "fmt": "f8", "T": 8192, "N": 11008, "type": "bf16"},
        # sixteen tokens, four experts each: the experts' weights are read once
        {"name": "experts_decode", "op": "experts", "G": 64, "tokens": 16, "top": 4, "N": 4096, "K": 2048,
         "type": "bf16"},
        # a short prompt over a few experts, every size odd
        {"name": "experts_odd", "op": "experts", "G": 8, "tokens": 500, "top": 2, "N": 1501, "K": 777, "type": "f16"},
        # a large prompt batch through the experts
        {"name": "experts_prompts", "op": "experts", "G": 16, "tokens": 8192, "top": 2, "N": 4096, "K": 4096,
         "type": "bf16"},
        # sixteen sequences decoding through one dense layer
        {"name": "f8_decode", "op": "f8", "M": 16, "N": 4096, "K": 4096, "type": "bf16"},
        # a ragged product: sizes that end inside tiles and blocks
        {"name": "f8_odd", "op": "f8", "M": 1000, "N": 3000, "K": 777, "type": "f32"},
        # a prompt through one dense layer
        {"name": "f8_prompt", "op": "f8", "M": 4096, "N": 4096, "K": 4096, "type": "bf16"},
    ]


def _spread(rng, lo, hi, step=1):
    """A size between lo and hi, spread over the logarithm; a multiple of `step` two times in three."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    if step > 1 and rng.random() < 2 / 3:
        v = max(step, v // step * step)
    return max(lo, min(hi, v))


def draw(rng):
    op = rng.choice(["norm", "act", "experts", "f8"])
    kind = rng.choice(["bf16", "bf16", "f16", "f32"])
    if op in ("norm", "act"):
        H = _spread(rng, 64, 16384, 128)
        T = _spread(rng, 1, min(16384, 32_000_000 // H))
        fmt = rng.choice(["s8", "f8"])
        if op == "norm":
            return {"op": op, "fmt": fmt, "T": T, "H": H, "type": kind, "residual": rng.random() < 0.7}
        return {"op": op, "fmt": fmt, "T": T, "N": H, "type": kind}
    N, K = _spread(rng, 64, 8192, 128), _spread(rng, 64, 8192, 128)
    if op == "experts":
        G = _spread(rng, 1, 64)
        top = rng.randint(1, min(G, 8))
        tokens = _spread(rng, 1, max(1, min(8192 // top, 100_000_000 // (N * top))))
        return {"op": op, "G": G, "tokens": tokens, "top": top, "N": N, "K": K, "type": kind}
    return {"op": op, "M": _spread(rng, 1, 4096), "N": N, "K": K, "type": kind}


def _used(case):
    """Experts of a case that get rows: one in eight gets none."""
    return min(case["tokens"] * case["top"], case["G"] - case["G"] // 8)


def work(case):
    b = BYTES[case["type"]]
    if case["op"] == "norm":
        T, H = case["T"], case["H"]
        scales = T if case["fmt"] == "s8" else T * -(-H // BLOCK)
        return {"bytes": T * H * (b + (2 * b if case["residual"] else 0) + 1) + H * b + 4 * scales, "flops": 5 * T * H}
    if case["op"] == "act":
        T, N = case["T"], case["N"]
        scales = T if case["fmt"] == "s8" else T * -(-N // BLOCK)
        return {"bytes": T * N * (2 * b + 1) + 4 * scales, "flops": 6 * T * N}
    N, K = case["N"], case["K"]
    if case["op"] == "experts":
        R, E = case["tokens"] * case["top"], _used(case)
        return {"bytes": case["tokens"] * (K + 4) + 4 * R + E * N * (K + 4) + R * N * b + 4 * (case["G"] + 1),
                "flops": 2 * R * N * K}
    M, kb = case["M"], -(-K // BLOCK)
    return {"bytes": M * K + N * K + 4 * kb * (M + -(-N // BLOCK)) + M * N * b, "flops": 2 * M * N * K}


# ----- inputs ----------------------------------------------------------------------

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed) * 2 + 1)


def _normal(gen, *shape, dtype=torch.float32):
    return torch.randn(*shape, generator=gen, device="cuda", dtype=torch.float32).to(dtype)


def _rows_s8(gen, *shape):
    """Normal rows quantised to int8, with their scales."""
    x = torch.randn(*shape, generator=gen, device="cuda")
    scale = x.abs().amax(-1) / 127
    return (x / scale[..., None]).round().to(torch.int8), scale


def _prepare_experts(case, gen):
    G, T, top, N, K = case["G"], case["tokens"], case["top"], case["N"], case["K"]
    R, E = T * top, _used(case)
    A, a_scale = _rows_s8(gen, T, K)
    B = torch.empty(G, N, K, dtype=torch.int8, device="cuda")
    b_scale = torch.empty(G, N, device="cuda")
    for g in range(G):
        B[g], b_scale[g] = _rows_s8(gen, N, K)
    # the router's answer: every used expert has a row, the others get a
    # skewed share, and the rows are sorted by expert
    used = torch.randperm(G, generator=gen, device="cuda")[:E]
    share = torch.rand(E, generator=gen, device="cuda") + 0.25
    more = torch.multinomial(share, R - E, replacement=True, generator=gen) if R > E else used[:0]
    expert = used[torch.cat([torch.arange(E, device="cuda"), more])]
    token = torch.randperm(R, generator=gen, device="cuda") // top
    rows = token[torch.argsort(expert, stable=True)].to(torch.int32)
    counts = torch.bincount(expert, minlength=G)
    offsets = torch.zeros(G + 1, dtype=torch.int32, device="cuda")
    offsets[1:] = counts.cumsum(0)
    return {"A": A, "a_scale": a_scale, "B": B, "b_scale": b_scale * K ** -0.5, "rows": rows, "offsets": offsets,
            "most": int(counts.max())}


def _prepare_f8(case, gen):
    M, N, K = case["M"], case["N"], case["K"]
    mb, nb, kb = M, -(-N // BLOCK), -(-K // BLOCK)
    A = (_normal(gen, M, K) * 100).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    B = (_normal(gen, N, K) * 100).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    a_scale = torch.rand(mb, kb, generator=gen, device="cuda") * 0.02 + 0.002
    b_scale = (torch.rand(nb, kb, generator=gen, device="cuda") * 0.02 + 0.002) * K ** -0.5
    return {"A": A, "a_scale": a_scale, "B": B, "b_scale": b_scale}


def prepare(case, seed):
    gen, dtype = _gen(seed), TYPES[case["type"]]
    if case["op"] == "norm":
        T, H = case["T"], case["H"]
        # a few channels of the residual stream are far larger than the rest
        loud = 1 + 30 * (torch.rand(H, generator=gen, device="cuda") < 0.002)
        s = {"x": _normal(gen, T, H, dtype=dtype), "weight": (1 + 0.1 * _normal(gen, H)).to(dtype),
             "residual": (_normal(gen, T, H) * loud).to(dtype) if case["residual"] else None}
    elif case["op"] == "act":
        both = _normal(gen, case["T"], 2 * case["N"], dtype=dtype) * 2  # the gate's and the other half, side by side
        s = {"gate": both[:, :case["N"]], "up": both[:, case["N"]:]}
    elif case["op"] == "experts":
        s = _prepare_experts(case, gen)
    else:
        s = _prepare_f8(case, gen)
    return {**s, "case": dict(case), "dtype": dtype}


# ----- plain forms -----------------------------------------------------------------

def _quotient(v, most, top):
    """v * top / most, 0 where the row or block holds only zeros."""
    return torch.where(most > 0, v * top / most, torch.zeros_like(v))


def _blocks(v):
    """The last axis cut into blocks of 128, the last one filled up with zeros."""
    v = torch.nn.functional.pad(v, (0, -v.shape[-1] % BLOCK))
    return v.view(v.shape[0], -1, BLOCK)


def _to_s8(v):
    """Rows in 64 bits (an int8 value next to a border goes by their last bits) to int8 and their largest magnitudes."""
    most = v.abs().amax(-1, keepdim=True)
    return _quotient(v, most, 127.0).round().to(torch.int8), most[:, 0]


def _to_f8(v):
    b = _blocks(v)
    most = b.abs().amax(-1, keepdim=True)
    q = _quotient(b, most, E4M3_MAX).clamp(-E4M3_MAX, E4M3_MAX)
    return q.reshape(v.shape[0], -1)[:, :v.shape[1]].to(torch.float8_e4m3fn), most[..., 0]


def _plain_norm(x, weight, residual, fmt):
    # the norm is that of the sum as the residual stream keeps it, in x's type
    h = x if residual is None else (x.float() + residual.float()).to(x.dtype)
    mean = h.float().square().mean(-1, keepdim=True)
    inv = torch.rsqrt(mean + EPS)
    if fmt == "s8":
        q, most = _to_s8(h.double() * weight.double())
        scale = most.float() * inv[:, 0] / 127
    else:
        q, most = _to_f8(h.float() * weight.float())
        scale = most * inv / E4M3_MAX
    return (q, scale) if residual is None else (q, scale, h)


def _plain_act(gate, up, fmt):
    if fmt == "s8":
        g = gate.double()
        q, most = _to_s8(g / (1 + torch.exp(-g)) * up.double())
        return q, (most / 127).float()
    g = gate.float()
    q, most = _to_f8(g / (1 + torch.exp(-g)) * up.float())
    return q, most / E4M3_MAX


def _plain_experts(A, a_scale, B, b_scale, rows, offsets, most, dtype):
    # every expert's rows in a batch of equal sizes, the short ones filled up with zeros
    at = torch.arange(rows.numel(), device=A.device)
    expert = torch.searchsorted(offsets[1:].long(), at, right=True)
    place = at - offsets.long()[expert]
    rows = rows.long()
    batch = torch.zeros(B.shape[0], most, A.shape[1], device=A.device)
    batch[expert, place] = A.float()[rows]
    product = torch.bmm(batch, B.float().transpose(1, 2))[expert, place]
    return (product * (a_scale[rows][:, None] * b_scale[expert])).to(dtype)


def _plain_f8(A, a_scale, B, b_scale, dtype):
    M, K = A.shape
    N = B.shape[0]
    a = A.float() * a_scale.repeat_interleave(BLOCK, 1)[:, :K]
    b = B.float() * b_scale.repeat_interleave(BLOCK, 0).repeat_interleave(BLOCK, 1)[:N, :K]
    return (a @ b.t()).to(dtype)


def _plain(s):
    c = s["case"]
    if c["op"] == "norm":
        return _plain_norm(s["x"], s["weight"], s["residual"], c["fmt"])
    if c["op"] == "act":
        return _plain_act(s["gate"], s["up"], c["fmt"])
    if c["op"] == "experts":
        return _plain_experts(s["A"], s["a_scale"], s["B"], s["b_scale"], s["rows"], s["offsets"], s["most"],
                              s["dtype"])
    return _plain_f8(s["A"], s["a_scale"], s["B"], s["b_scale"], s["dtype"])


def _own(s):
    import tiled_dense_int8_amd as t
    c = s["case"]
    if c["op"] == "norm":
        return t.rms_norm(s["x"], s["weight"], EPS, residual=s["residual"], fmt=c["fmt"])
    if c["op"] == "act":
        return t.swiglu(s["gate"], s["up"], fmt=c["fmt"])
    if c["op"] == "experts":
        return t.grouped_gemm(s["A"], s["a_scale"], s["B"], s["b_scale"], s["offsets"], rows=s["rows"],
                              dtype=s["dtype"])
    return t.gemm_f8(s["A"], s["a_scale"], s["B"], s["b_scale"], dtype=s["dtype"])


def run(state):
    return _own(state) if own else _plain(state)


# ----- the definition in 64 bits ---------------------------------------------------

def _exact_rows(v, fmt):
    """(quantised rows, scales) of rows v in 64 bits, one row or block of 128 at a time."""
    T, H = v.shape
    width, top = (H, 127.0) if fmt == "s8" else (BLOCK, E4M3_MAX)
    parts, scales = [], []
    for start in range(0, H, width):
        part = v[:, start:start + width]
        largest = torch.linalg.vector_norm(part, ord=float("inf"), dim=1)
        scales.append(largest / top)
        parts.append(part / torch.where(largest == 0, 1.0, largest)[:, None] * top)
    q = torch.cat(parts, 1)
    if fmt == "s8":
        return torch.round(q).to(torch.int8), scales[0]
    return q.float().to(torch.float8_e4m3fn), torch.stack(scales, 1)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        h = s["x"].double()
        if s["residual"] is not None:
            h = h + s["residual"].double()
        kept = h.to(s["dtype"])
        k = kept.double()
        rms = torch.sqrt((k * k).sum(1) / case["H"] + EPS)
        q, scale = _exact_rows(k * s["weight"].double(), case["fmt"])
        scale = scale / (rms if case["fmt"] == "s8" else rms[:, None])
        return (q, scale) if s["residual"] is None else (q, scale, h)
    if case["op"] == "act":
        g, u = s["gate"].double(), s["up"].double()
        return _exact_rows(g * torch.sigmoid(g) * u, case["fmt"])
    if case["op"] == "experts":
        ends = s["offsets"].tolist()
        out = torch.zeros(s["rows"].numel(), case["N"], dtype=torch.float64, device="cuda")
        for g, (lo, hi) in enumerate(zip(ends, ends[1:])):
            idx = s["rows"][lo:hi].long()
            left = s["A"][idx].double() * s["a_scale"][idx].double()[:, None]
            right = s["B"][g].double() * s["b_scale"][g].double()[:, None]
            out[lo:hi] = torch.mm(left, right.t())
        return out
    out = torch.zeros(case["M"], case["N"], dtype=torch.float64, device="cuda")
    for kb, lo in enumerate(range(0, case["K"], BLOCK)):
        part = torch.mm(s["A"][:, lo:lo + BLOCK].double(), s["B"][:, lo:lo + BLOCK].double().t())
        out += part * s["a_scale"][:, kb, None].double() * torch.repeat_interleave(
            s["b_scale"][:, kb].double(), BLOCK)[:case["N"]]
    return out
