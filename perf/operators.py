"""Microscaled 4-bit floating point: what is measured of it, case by case, beside a plain form in elementary torch
operations.

Three operators, each reached through ``bit_gemm_w4_b200.mosaicq``:

  quantize   X [M, K] to E2M1 codes with a scale for each block of columns, and back to the values they stand for
             (``fp4_quantize(X, fmt)``, ``Fp4Tensor.dequantize(dtype)``);
  linear     Y = X W^T with W held in 4 bits and X quantised within the call (``Fp4Weight.linear(X)``);
  grouped    the same for the rows of each expert: row r of the ragged batch is X[rows[r]], and expert e owns the rows
             offsets[e] .. offsets[e + 1] - 1 (``Fp4Weight.linear_grouped(X, offsets, rows=rows)``).

Formats, both decided in 32 bits (all roundings to nearest, ties to even):

  mxfp4      blocks of 32 columns. With a = max |x| of the block and E the exponent field of a as a 32-bit float,
             s = max(E - 2, 0) and the scale is 2^(s - 127); code = e2m1(x * 2^(127 - s)), saturating at 6.
  nvfp4      blocks of 16 columns, and one 32-bit factor r for each row: r = max(max |row| * (1 / 2688), 2^-100); the
             block's scale is b = e4m3((a * (1 / 6)) * (1 / r)); code = e2m1(x * (1 / (b * r))), and 0 where b is 0.
"""

import math

import torch

own = False

_DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
_BLOCK = {"mxfp4": 32, "nvfp4": 16}


# ---------------------------------------------------------------- the cases
def listed():
    return [
        # one token's activations on the way into a 4-bit linear: latency alone
        dict(name="quantize nv 1x4096", op="quantize", fmt="nvfp4", dtype="bf16", M=1, K=4096),
        # a prefill batch of activations, wide enough to leave the L2 cache
        dict(name="quantize mx 8192x4096", op="quantize", fmt="mxfp4", dtype="bf16", M=8192, K=4096),
        # an odd width: rows that start at any 2-byte address, a last block that is not full
        dict(name="quantize nv 3001x11003", op="quantize", fmt="nvfp4", dtype="fp16", M=3001, K=11003),
        # a decoding step of a 7B-shaped model at one token: q, k, v or o
        dict(name="linear nv 1x4096x4096", op="linear", fmt="nvfp4", dtype="bf16", M=1, N=4096, K=4096),
        # batched decoding of a 70B-shaped MLP
        dict(name="linear mx 16x28672x8192", op="linear", fmt="mxfp4", dtype="bf16", M=16, N=28672, K=8192),
        # a handful of requests' tokens at odd sizes, between decoding and prefill
        dict(name="linear nv 77x11007x4100", op="linear", fmt="nvfp4", dtype="fp16", M=77, N=11007, K=4100),
        # prefill of 2048 tokens through the up projection
        dict(name="linear nv 2048x14336x4096", op="linear", fmt="nvfp4", dtype="bf16", M=2048, N=14336, K=4096),
        # a longer prefill through a down projection
        dict(name="linear mx 4096x4096x11008", op="linear", fmt="mxfp4", dtype="bf16", M=4096, N=4096, K=11008),
        # one token through 2 of 8 large experts
        dict(name="grouped nv 1 of 8x14336x4096", op="grouped", fmt="nvfp4", dtype="bf16", T=1, E=8, top=2, N=14336, K=4096),
        # a decoding batch spread over many small experts, most of them with a row or two
        dict(name="grouped mx 32 of 64x2048x2048", op="grouped", fmt="mxfp4", dtype="bf16", T=32, E=64, top=6, N=2048, K=2048),
        # experts of odd sizes with ragged shares of some hundred tokens
        dict(name="grouped nv 333 of 5x1111x2891", op="grouped", fmt="nvfp4", dtype="fp16", T=333, E=5, top=3, N=1111, K=2891),
        # prefill of 2048 tokens through 2 of 8 large experts
        dict(name="grouped mx 2048 of 8x14336x4096", op="grouped", fmt="mxfp4", dtype="bf16", T=2048, E=8, top=2, N=14336, K=4096),
    ]


def _spread(rng, low, high):
    """A whole number of low .. high, spread evenly over its logarithm."""
    return min(high, max(low, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def _width(rng, low, high):
    """A number of columns: most are multiples of 32, as a model's are; one in three is any number."""
    k = _spread(rng, low, high)
    return k if rng.random() < 1 / 3 else max(32, k // 32 * 32)


def draw(rng):
    op = rng.choice(["quantize", "linear", "linear", "grouped", "grouped"])
    c = dict(op=op, fmt=rng.choice(["mxfp4", "nvfp4"]), dtype=rng.choice(["bf16", "bf16", "fp16"]))
    if op == "quantize":
        c["K"] = _width(rng, 40, 16384)
        c["M"] = _spread(rng, 1, min(16384, 33_000_000 // c["K"]))
    elif op == "linear":
        c["N"], c["K"] = _spread(rng, 60, 28672), _width(rng, 40, 11008)
        c["M"] = _spread(rng, 1, min(4096, int(1.8e11) // (c["N"] * c["K"])))
    else:
        c["E"] = _spread(rng, 2, 128)
        c["top"] = rng.randint(1, min(c["E"], 8))
        c["K"] = _width(rng, 40, 5120)
        c["N"] = _spread(rng, 60, max(64, min(14336, 400_000_000 // (c["E"] * c["K"]))))
        c["T"] = _spread(rng, 1, max(1, min(2048, int(1.8e11) // (c["top"] * c["N"] * c["K"]))))
    return c


# ---------------------------------------------------------------- the plain form
def _pad(x, to):
    """Columns of zeros up to a multiple of `to`."""
    short = -x.shape[-1] % to
    return torch.nn.functional.pad(x, (0, short)) if short else x


def _e2m1(q):
    """Code 0 .. 7 of |q|, rounded to nearest with ties to the even code, plus 8 for a negative q."""
    a = q.abs()
    mag = (a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0)
    return mag + 8 * torch.signbit(q).to(torch.uint8)


def _quantize(X, fmt):
    """Codes [..., Kb, block] (0 .. 15), scale bytes [..., Kb] and, for nvfp4, the rows' factors [...]; K padded to whole blocks."""
    block = _BLOCK[fmt]
    x = _pad(X.float(), block)
    x = x.reshape(*x.shape[:-1], -1, block)
    a = x.abs().amax(-1)
    if fmt == "mxfp4":
        s = (((a.view(torch.int32) >> 23) & 255) - 2).clamp_min(0)
        inv = ((254 - s) << 23).view(torch.float32)  # 2^(127 - s)
        return _e2m1(x * inv[..., None]), s.to(torch.uint8), None
    r = (a.amax(-1) * (1 / 2688)).clamp_min(2.0**-100)
    b = (a * (1 / 6)) * (1.0 / r)[..., None]
    b = b.clamp_max(448.0).to(torch.float8_e4m3fn)
    p = b.float() * r[..., None]
    inv = torch.where(p > 0, 1.0 / p, 0.0)
    return _e2m1(x * inv[..., None]), b.view(torch.uint8), r


def _dequantize(codes, scales, r, K):
    """The values, in 32 bits, that _quantize's answer stands for, [..., K]."""
    mantissa, exponent = (codes & 1).float(), (codes >> 1) & 3
    v = torch.where(exponent > 0, (1 + 0.5 * mantissa) * (1 << exponent) * 0.5, 0.5 * mantissa)
    v = torch.where(codes > 7, -v, v)
    s = torch.ldexp(torch.ones_like(scales, dtype=torch.float32), scales.int() - 127) if r is None else scales.view(torch.float8_e4m3fn).float()
    v = v * s[..., None]
    if r is not None:
        v = v * r[..., None, None]
    return v.flatten(-2)[..., :K]


# ---------------------------------------------------------------- states
def _activations(M, K, dtype, g):
    """Normal values with a few large channels, as the inputs of a model's linear layers have."""
    x = torch.randn(M, K, generator=g, device="cuda")
    x[:, torch.randint(0, K, (4,), generator=g, device="cuda")] *= 20.0
    return x.to(dtype)


def _weight(N, K, g):
    """Normal values with outliers in one of 200 places."""
    w = torch.randn(N, K, generator=g, device="cuda") * 0.02
    return w * torch.where(torch.rand(N, K, generator=g, device="cuda") < 0.005, 8.0, 1.0)


def _bytes_of(codes, scales):
    """The packed form: two codes in a byte (the even column low), rows of codes and of scales padded to 16 bytes."""
    c = _pad(codes.flatten(-2), 32)
    return (c[..., 0::2] | (c[..., 1::2] << 4)).contiguous(), _pad(scales, 16).contiguous()


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    fmt, dtype, K = case["fmt"], _DTYPES[case["dtype"]], case["K"]
    if case["op"] == "quantize":
        return dict(op="quantize", fmt=fmt, X=_activations(case["M"], K, dtype, g))
    E, N, T = case.get("E", 1), case["N"], case["M"] if case["op"] == "linear" else case["T"]
    s = dict(op=case["op"], fmt=fmt, X=_activations(T, K, dtype, g))
    # the weight as a checkpoint holds it; a program keeps it as the framework's handle, or (plain form) as 32-bit values
    kept = []
    for _ in range(E):
        q = _quantize(_weight(N, K, g), fmt)
        kept.append((*_bytes_of(*q[:2]), q[2]) if own else _dequantize(*q, K))
    if own:
        from bit_gemm_w4_b200 import mosaicq

        codes, scales = (torch.stack([k[i] for k in kept]) for i in (0, 1))
        factors = torch.stack([k[2] for k in kept]) if fmt == "nvfp4" else None
        s["w"] = mosaicq.Fp4Weight.pack_codes(codes, scales, factors, K, fmt)
    else:
        s["W"] = kept
    if case["op"] == "grouped":
        # a router's choice: the largest `top` of E scores, some experts more popular than others
        score = torch.randn(T, E, generator=g, device="cuda") + 0.5 * torch.randn(E, generator=g, device="cuda")
        chosen = score.topk(case["top"], dim=1).indices.flatten()
        order = torch.sort(chosen, stable=True).indices
        s["rows"] = (order // case["top"]).int()
        s["offsets"] = torch.nn.functional.pad(torch.bincount(chosen, minlength=E).cumsum(0), (1, 0)).int()
        s["split"] = s["offsets"].tolist()
    return s


def run(state):
    X, fmt, op = state["X"], state["fmt"], state["op"]
    if own:
        from bit_gemm_w4_b200 import mosaicq

        if op == "quantize":
            return mosaicq.fp4_quantize(X, fmt).dequantize(X.dtype)
        if op == "linear":
            return state["w"].linear(X)
        return state["w"].linear_grouped(X, state["offsets"], rows=state["rows"])
    x = _dequantize(*_quantize(X, fmt), X.shape[1])
    if op == "quantize":
        return x.to(X.dtype)
    if op == "linear":
        return (x @ state["W"][0].T).to(X.dtype)
    # one product for each expert that has rows: padding them to one batch would charge for rows that are not there
    at = state["split"]
    parts = [x[state["rows"][a:b]] @ w.T for w, a, b in zip(state["W"], at, at[1:]) if b > a]
    return torch.cat(parts).to(X.dtype)


# ---------------------------------------------------------------- 64 bits
def _rounded(v, mantissa, least):
    """v (64 bits, >= 0) to the nearest number with `mantissa` bits behind the leading one and no exponent below `least`, ties to even."""
    _, e = torch.frexp(v)
    step = torch.exp2(((e - 1).clamp_min(least) - mantissa).double())
    return torch.round(v / step) * step


def _held(x, fmt):
    """The values that x [R, K] (32 bits) is held as, in 64 bits; the decisions are those of the definition, in 32 bits."""
    R, K = x.shape
    block = _BLOCK[fmt]
    whole = torch.zeros(R, -(-K // block) * block, dtype=torch.float32, device=x.device)
    whole[:, :K] = x
    parts = whole.view(R, -1, block)
    top = parts.abs().max(dim=2, keepdim=True).values
    if fmt == "mxfp4":
        exponent = torch.frexp(top.double()).exponent - 1  # floor(log2), where top > 0
        scale = torch.exp2(torch.where(top > 0, exponent - 2, -127).clamp_min(-127).double())
        scaled = parts.double() / scale
    else:
        r = top.max(dim=1, keepdim=True).values * torch.full((), 1 / 2688, dtype=torch.float32, device=x.device)
        r = torch.maximum(r, torch.full_like(r, 2.0**-100))
        b = (top * torch.full((), 1 / 6, dtype=torch.float32, device=x.device)) * torch.reciprocal(r)
        b = _rounded(b.double(), 3, -6).clamp_max(448.0)
        product = (b * r.double()).float()
        scaled = torch.where(product > 0, parts * torch.reciprocal(product), torch.zeros_like(parts)).double()
        scale = b * r.double()
    held = _rounded(scaled.abs(), 1, 0).clamp_max(6.0) * torch.sign(scaled) * scale
    return held.reshape(R, -1)[:, :K]


def exact(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    fmt, dtype, K = case["fmt"], _DTYPES[case["dtype"]], case["K"]
    if case["op"] == "quantize":
        return _held(_activations(case["M"], K, dtype, g).float(), fmt)
    E, N, T = case.get("E", 1), case["N"], case["M"] if case["op"] == "linear" else case["T"]
    x = _held(_activations(T, K, dtype, g).float(), fmt)
    if case["op"] == "linear":
        return x @ _held(_weight(N, K, g), fmt).T
    state = g.get_state()
    for _ in range(E):
        _weight(N, K, g)
    score = torch.randn(T, E, generator=g, device="cuda") + 0.5 * torch.randn(E, generator=g, device="cuda")
    _, chosen = score.topk(case["top"], dim=1)
    pairs = [(e, t) for t, of in enumerate(chosen.tolist()) for e in of]
    g.set_state(state)
    parts = []
    for e in range(E):
        w = _held(_weight(N, K, g), fmt)
        mine = [t for f, t in pairs if f == e]
        if mine:
            parts.append(x[mine] @ w.T)
    return torch.cat(parts)


# ---------------------------------------------------------------- what a pass cannot do without
def work(case):
    K, per = case["K"], 0.5 + 1 / _BLOCK[case["fmt"]]  # bytes of a held element: half a byte and its share of the scale
    if case["op"] == "quantize":
        n = case["M"] * K
        return {"bytes": 4 * n, "flops": 4 * n}  # X read, the values written; a maximum, a product and two roundings
    if case["op"] == "linear":
        M, N, read = case["M"], case["N"], 1.0
        T = M
    else:
        T, N = case["T"], case["N"]
        M = T * case["top"]
        read = case["E"] * (1 - (1 - case["top"] / case["E"]) ** T)  # experts that some token chooses
    return {"bytes": read * N * K * per + 2 * T * K + 2 * M * N, "flops": 2 * M * N * K}
