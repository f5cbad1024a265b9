"""The 4-bit and 8-bit feed-forward operators of libbsq as measured cases.

Three operators that run one after another around a (mixture-of-experts)
feed-forward layer whose operands are block-scaled:

* ``norm``   -- h = residual + residual_scale * (post-norm(x) * gate), then the
  RMS norm of h quantized for the next product; and its backward pass.
* ``swiglu`` -- silu(gate half) * up half of a fused gate/up product, quantized
  for the down product; and its backward pass.
* ``mm``     -- the product of two block-scaled operands, dense or grouped by
  expert with ragged token counts.

Each has a plain form in elementary torch operations and, in ``exact``, its
definition in 64 bits.  Values that are held in 8 bits are returned as torch's
8-bit floats (a view of the same bytes); 4-bit codes are looked up in a table
of the values they stand for, which costs the measured side that holds them
packed a few extra passes.
"""
import math

import numpy as np
import torch

own = False

BLOCK = {"nvfp4": 16, "mxfp4": 32, "mxfp8": 32}
CODE_BITS = {"nvfp4": 4, "mxfp4": 4, "mxfp8": 8}
EPS = 1e-6


# ------------------------------------------------------------------ cases ---

def listed():
    return [
        # one decoded token through one 4-bit projection: latency, and the weight bytes
        {"name": "mm nvfp4 T=1", "op": "mm", "a": "nvfp4", "w": "nvfp4", "T": 1, "E": 0, "N": 2048, "K": 7168, "tail": 0},
        # a ragged prompt through a dense 8-bit projection
        {"name": "mm mxfp8 T=777", "op": "mm", "a": "mxfp8", "w": "mxfp8", "T": 777, "E": 0, "N": 4104, "K": 2080, "tail": 0},
        # 64 decoded tokens routed over 32 experts, 8-bit activations on 4-bit weights: bound by the weights
        {"name": "mm w4a8 T=64 E=32", "op": "mm", "a": "mxfp8", "w": "mxfp4", "T": 64, "E": 32, "N": 2048, "K": 7168, "tail": 0},
        # a training batch over 32 skewed experts, 13 padding rows behind the last one
        {"name": "mm nvfp4 T=16384 E=32", "op": "mm", "a": "nvfp4", "w": "nvfp4", "T": 16384, "E": 32, "N": 2048, "K": 7168, "tail": 13},
        # the norm before a block for one decoded token
        {"name": "norm mxfp8 1x7168", "op": "norm", "fmt": "mxfp8", "rows": 1, "C": 7168, "dtype": "bf16", "residual": True, "post": False, "gate": False, "scale": 1.0},
        # the same for a training batch, with the norm after the block, its gate and a residual scale
        {"name": "norm mxfp8 16384x7168", "op": "norm", "fmt": "mxfp8", "rows": 16384, "C": 7168, "dtype": "bf16", "residual": True, "post": True, "gate": True, "scale": 0.22},
        # backward of that norm over a training batch
        {"name": "norm backward 4096x7168", "op": "norm_bwd", "rows": 4096, "C": 7168, "dtype": "bf16", "residual": True, "post": True, "gate": True, "scale": 0.22},
        # backward of the plain pre-norm, odd row count, fp32 stream
        {"name": "norm backward 333x2080", "op": "norm_bwd", "rows": 333, "C": 2080, "dtype": "fp32", "residual": True, "post": False, "gate": False, "scale": 1.0},
        # activation between the two expert products of a training batch
        {"name": "swiglu mxfp8 16384x2048", "op": "swiglu", "fmt": "mxfp8", "rows": 16384, "F": 2048, "dtype": "bf16"},
        # activation of a dense layer for a ragged prompt, 4-bit
        {"name": "swiglu nvfp4 77x18432", "op": "swiglu", "fmt": "nvfp4", "rows": 77, "F": 18432, "dtype": "bf16"},
        # backward of the activation over a training batch, and over a few fp32 rows
        {"name": "swiglu backward 16384x2048", "op": "swiglu_bwd", "rows": 16384, "F": 2048, "dtype": "bf16"},
        {"name": "swiglu backward 19x2064", "op": "swiglu_bwd", "rows": 19, "F": 2064, "dtype": "fp32"},
    ]


def _log_int(rng, lo, hi, step=1):
    """A multiple of `step` in [lo, hi], spread evenly over its logarithm."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))
    return max(lo, min(hi, int(v) // step * step))


def draw(rng):
    op = rng.choice(["mm", "mm", "mm", "norm", "norm_bwd", "swiglu", "swiglu_bwd"])
    if op == "mm":
        a, w = rng.choice([("nvfp4", "nvfp4"), ("mxfp4", "mxfp4"), ("mxfp8", "mxfp8"), ("mxfp8", "mxfp4")])
        E = rng.choice([0, 0, rng.randint(1, 8), _log_int(rng, 8, 64)])
        K = _log_int(rng, 128, 7168, 128 if a != w else 32)
        N = _log_int(rng, 128, 7168, 8)
        while max(E, 1) * N * K > 470_000_000:
            E = max(1, E // 2)
        T = _log_int(rng, 1, 16384)
        while 2.0 * T * N * K > 4.8e11:
            T = T // 2
        return {"op": "mm", "a": a, "w": w, "T": T, "E": E, "N": N, "K": K,
                "tail": rng.randint(0, T // 4) if E and rng.random() < 0.5 else 0}
    bf16 = rng.random() < 0.75
    rows = _log_int(rng, 1, 16384)
    if op in ("swiglu", "swiglu_bwd"):
        c = {"op": op, "rows": rows, "F": _log_int(rng, 64, 18432, 32), "dtype": "bf16" if bf16 else "fp32"}
        while c["rows"] * c["F"] > 16384 * 2048:
            c["rows"] //= 2
    else:
        c = {"op": op, "rows": rows, "C": _log_int(rng, 64, 18432, 32), "dtype": "bf16" if bf16 else "fp32",
             "residual": rng.random() < 0.8, "post": rng.random() < 0.4, "gate": rng.random() < 0.4,
             "scale": rng.choice([1.0, 0.22, 0.5])}
        while c["rows"] * c["C"] > (16384 if op == "norm" else 4096) * 7168 // (1 if bf16 else 2):
            c["rows"] //= 2
    if op in ("norm", "swiglu"):
        c["fmt"] = rng.choice(["nvfp4", "mxfp4", "mxfp8"])
    return c


def _alters(case):
    """Whether h differs from x (then it is an output of its own)."""
    return bool(case["residual"] or case["post"] or case["gate"] or case["scale"] != 1.0)


def work(case):
    op = case["op"]
    if op == "mm":
        T, N, K = case["T"], case["N"], case["K"]
        tokens = T - case["tail"]
        E = max(1, case["E"])
        hit = min(E, tokens)  # experts that can have a token: weights of the others need not be read
        per = {f: CODE_BITS[f] / 8 + 1 / BLOCK[f] for f in BLOCK}
        b = tokens * K * per[case["a"]] + hit * N * K * per[case["w"]] + 2 * T * N
        b += 4 * tokens * (case["a"] == "nvfp4") + 4 * hit * N * (case["w"] == "nvfp4")
        return {"bytes": b, "flops": 2.0 * tokens * N * K}
    es = 2 if case["dtype"] == "bf16" else 4
    rows = case["rows"]
    if op in ("norm", "swiglu"):
        out = CODE_BITS[case["fmt"]] / 8 + 1 / BLOCK[case["fmt"]]
    if op == "swiglu":
        n = rows * case["F"]
        return {"bytes": n * (2 * es + out), "flops": 8.0 * n}
    if op == "swiglu_bwd":
        n = rows * case["F"]
        return {"bytes": n * 5 * es, "flops": 12.0 * n}
    n = rows * case["C"]
    if op == "norm":
        b = n * es * (1 + case["residual"] + case["gate"] + _alters(case)) + n * out
        return {"bytes": b + 4 * case["C"] * (1 + case["post"]), "flops": (8.0 + 4 * case["post"] + 2 * case["gate"]) * n}
    # gradient of y, h and the gradient of the residual stream in, its gradient out ...
    b = n * es * (3 + 1)
    if case["post"] or case["gate"]:
        b += n * es * (1 + 1 + 2 * case["gate"])  # ... x and the gate in, their gradients out
    elif case["scale"] != 1.0:
        b += n * es
    return {"bytes": b + 8 * case["C"] * (1 + case["post"]), "flops": (10.0 + 8 * case["post"] + 3 * case["gate"]) * n}


# ---------------------------------------------- formats, in 32-bit torch ----

_E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, 0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0]


def _e2m1_code(q):
    """Nearest e2m1 code, ties to the even code, saturating at 6."""
    a = q.abs()
    m = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0))
    return m + ((q < 0) & (m > 0)).to(torch.uint8) * 8


def _exponent(amax, top):
    """floor(log2(amax)) - top, -127 for a block of zeros."""
    e = torch.frexp(amax).exponent - 1 - top
    return torch.where(amax == 0, torch.full_like(e, -127), e).clamp(-127, 127)


def _quantized(y, fmt):
    """codes (e2m1 codes 0..15, or e4m3 bytes as float8), scales as 8-bit floats, row scales (nvfp4)."""
    b = BLOCK[fmt]
    blocks = y.reshape(*y.shape[:-1], -1, b)
    amax = blocks.abs().amax(-1)
    if fmt == "nvfp4":
        g = y.abs().amax(-1) / 2688.0
        some = (g > 0)[..., None]
        s = torch.where(some, (amax / 6.0 / g[..., None]).clamp(2.0 ** -9, 448.0), torch.zeros((), device=y.device)).to(torch.float8_e4m3fn)
        d = s.float() * g[..., None]
        q = torch.where(some[..., None], blocks / d[..., None], torch.zeros((), device=y.device))
        return _e2m1_code(q).reshape(y.shape), s, g
    e = _exponent(amax, 2 if fmt == "mxfp4" else 8)
    scales = (e + 127).to(torch.uint8).view(torch.float8_e8m0fnu)
    half = torch.exp2((e.float() / 2).ceil())  # 2**e in two steps: 2**-127 and its inverse stay in range
    rest = torch.exp2((e.float() / 2).floor())
    q = blocks / half[..., None] / rest[..., None]
    if fmt == "mxfp4":
        return _e2m1_code(q).reshape(y.shape), scales, None
    return q.clamp(-448.0, 448.0).to(torch.float8_e4m3fn).reshape(y.shape), scales, None


def _packed(codes, fmt):
    """Codes as they are held: two e2m1 codes a byte, the even column low; or one e4m3 code a byte."""
    if fmt == "mxfp8":
        return codes.view(torch.uint8)
    return codes[..., 0::2] | (codes[..., 1::2] << 4)


def _unpacked(held, fmt, dtype):
    if fmt == "mxfp8":
        return held.view(torch.float8_e4m3fn).to(dtype)
    table = torch.tensor(_E2M1, dtype=dtype, device=held.device)
    return torch.stack((table[(held & 15).int()], table[(held >> 4).int()]), -1).flatten(-2)


def _scales(held, fmt):
    return held.view(torch.float8_e4m3fn if fmt == "nvfp4" else torch.float8_e8m0fnu)


def _dequantized(held, scales, row, fmt, dtype):
    v = _unpacked(held, fmt, dtype)
    s = _scales(scales, fmt).to(dtype)
    v = (v.reshape(*s.shape, BLOCK[fmt]) * s[..., None]).reshape(v.shape)
    return v if row is None else v * row.to(dtype)[..., None]


def _held_values(held, fmt):
    """What the held codes stand for, as 8-bit floats."""
    if fmt == "mxfp8":
        return held.view(torch.float8_e4m3fn)
    v = torch.tensor(_E2M1, device=held.device).to(torch.float8_e4m3fn).view(torch.uint8).short()
    pairs = (v[None, :] | (v[:, None] << 8)).flatten()  # byte -> the two values' bytes
    return pairs.index_select(0, held.flatten().int()).view(torch.float8_e4m3fn).reshape(*held.shape[:-1], -1)


def _code_values(codes, fmt):
    return codes if fmt == "mxfp8" else torch.tensor(_E2M1, device=codes.device).to(torch.float8_e4m3fn).view(torch.uint8)[codes.int()].view(torch.float8_e4m3fn)


# ---------------------------------------------------------------- inputs ----

def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda")


def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _routing(seed, T, E):
    """Zipf(1.1) shares of T tokens over E experts in a seeded order, the smallest left empty."""
    rng = np.random.default_rng(seed)
    p = (rng.permutation(E) + 1.0) ** -1.1
    n = rng.multinomial(T, p / p.sum())
    if E > 1:
        n[n.argmax()] += n.min()
        n[n.argmin()] = 0
        n[n.argmax()] += T - n.sum()
    return [int(v) for v in n]


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = {"case": case, "op": case["op"]}
    if case["op"] == "mm":
        T, N, K, E = case["T"], case["N"], case["K"], case["E"]
        a, w = case["a"], case["w"]
        # activations with outliers: channels of log-uniform scale
        x = _randn(g, T, K) * torch.exp(torch.rand(K, generator=g, device="cuda") * 2.0 - 1.0)
        codes, sc, s["a_row"] = _quantized(x, a)
        s["a"], s["a_scales"] = _packed(codes, a).contiguous(), sc.view(torch.uint8)
        held, scales, rows = [], [], []
        for _ in range(max(E, 1)):
            codes, sc, row = _quantized(_randn(g, N, K) * 0.02, w)
            held.append(_packed(codes, w))
            scales.append(sc.view(torch.uint8))
            rows.append(row)
        s["w"], s["w_scales"] = torch.stack(held), torch.stack(scales)
        s["w_row"] = torch.stack(rows) if w == "nvfp4" else None
        s["counts"] = _routing(seed, T - case["tail"], E) if E else [T]
        s["offs"] = torch.tensor(np.cumsum(s["counts"]), dtype=torch.int32, device="cuda") if E else None
        s["err"] = torch.zeros(1, dtype=torch.int32, device="cuda")
        return s
    dt = _dtype(case)
    rows = case["rows"]
    if case["op"] in ("swiglu", "swiglu_bwd"):
        s["x"] = (_randn(g, rows, 2 * case["F"]) * 1.5).to(dt)
        if case["op"] == "swiglu_bwd":
            s["grad_y"] = (_randn(g, rows, case["F"]) * 0.01).to(dt)
        return s
    C = case["C"]
    s["x"] = _randn(g, rows, C).to(dt)
    s["residual"] = (_randn(g, rows, C) * torch.exp(torch.rand(C, generator=g, device="cuda") * 3.0)).to(dt) if case["residual"] else None
    s["gate"] = (1.0 + 0.5 * _randn(g, rows, C)).to(dt) if case["gate"] else None
    s["weight"] = 1.0 + 0.1 * _randn(g, C)
    s["post_weight"] = 1.0 + 0.1 * _randn(g, C) if case["post"] else None
    if case["op"] == "norm_bwd":
        h, s["rstd"], s["post_rstd"] = _normed(s)
        s["h"] = h.to(dt)
        s["residual"] = None
        s["grad_y"] = (_randn(g, rows, C) * 0.01).to(dt)
        s["grad_h"] = (_randn(g, rows, C) * 0.01).to(dt)
    return s


# ------------------------------------------------------------ plain forms ---

def _normed(s):
    """The new residual stream in 32 bits, its reciprocal RMS, and the block output's."""
    v, post_rstd = s["x"].float(), None
    if s["post_weight"] is not None:
        post_rstd = torch.rsqrt(v.square().mean(-1) + EPS)
        v = v * post_rstd[:, None] * s["post_weight"]
    if s["gate"] is not None:
        v = v * s["gate"].float()
    h = v * s["case"]["scale"]
    if s["residual"] is not None:
        h = h + s["residual"].float()
    return h, torch.rsqrt(h.square().mean(-1) + EPS), post_rstd


def _norm_plain(s):
    h, rstd, post_rstd = _normed(s)
    fmt = s["case"]["fmt"]
    codes, scales, row = _quantized(h * rstd[:, None] * s["weight"], fmt)
    out = {"codes": _code_values(codes, fmt), "scales": scales, "rstd": rstd}
    return _norm_out(s, out, row, h.to(s["x"].dtype), post_rstd)


def _norm_out(s, out, row, h, post_rstd):
    if row is not None:
        out["row_scale"] = row
    if _alters(s["case"]):
        out["h"] = h
    if post_rstd is not None:
        out["post_rstd"] = post_rstd
    return out


def _norm_bwd_plain(s):
    c, dt = s["case"], s["x"].dtype
    gy, hhat = s["grad_y"].float(), s["h"].float() * s["rstd"][:, None]
    a = gy * s["weight"]
    dh = s["grad_h"].float() + s["rstd"][:, None] * (a - hhat * (a * hhat).mean(-1, keepdim=True))
    out = {"grad_residual": dh.to(dt), "grad_weight": (gy * hhat).sum(0)}
    if not (c["post"] or c["gate"] or c["scale"] != 1.0):
        return out
    du = dh * c["scale"]
    x = s["x"].float()
    xhat = x * s["post_rstd"][:, None] if c["post"] else x
    if c["gate"]:
        out["grad_gate"] = (du * (xhat * s["post_weight"] if c["post"] else xhat)).to(dt)
        du = du * s["gate"].float()
    if c["post"]:
        out["grad_post_weight"] = (du * xhat).sum(0)
        b = du * s["post_weight"]
        du = s["post_rstd"][:, None] * (b - xhat * (b * xhat).mean(-1, keepdim=True))
    out["grad_x"] = du.to(dt)
    return out


def _mm_plain(s):
    c = s["case"]
    a = _dequantized(s["a"], s["a_scales"], s["a_row"], c["a"], torch.float32)
    w = _dequantized(s["w"], s["w_scales"], s["w_row"], c["w"], torch.float32)
    parts = a[: sum(s["counts"])].split(s["counts"])
    padding = torch.zeros(c["tail"], c["N"], device=a.device)
    return torch.cat([*(p @ v.T for p, v in zip(parts, w)), padding]).to(torch.bfloat16)


def run(s):
    op = s["op"]
    if own:
        return _run_own(s, op)
    if op == "mm":
        return {"out": _mm_plain(s)}
    if op == "norm":
        return _norm_plain(s)
    if op == "norm_bwd":
        return _norm_bwd_plain(s)
    F = s["case"]["F"]
    gate, up = s["x"][:, :F].float(), s["x"][:, F:].float()
    sig = 1.0 / (1.0 + torch.exp(-gate))
    if op == "swiglu":
        fmt = s["case"]["fmt"]
        codes, scales, row = _quantized(gate * sig * up, fmt)
        out = {"codes": _code_values(codes, fmt), "scales": scales}
        return out if row is None else {**out, "row_scale": row}
    gy = s["grad_y"].float()
    return {"grad_x": torch.cat((gy * up * sig * (1.0 + gate * (1.0 - sig)), gy * gate * sig), -1).to(s["x"].dtype)}


def _run_own(s, op):
    """The calls a user makes."""
    from fp8_microscaling_quantization_b200 import bsq
    c = s["case"]
    fmts = {"nvfp4": bsq.Format.NVFP4, "mxfp4": bsq.Format.MXFP4, "mxfp8": bsq.Format.MXFP8}
    if op == "mm":
        out, _ = bsq.bsq_grouped_mm_scaled(fmts[c["a"]], s["a"], s["a_scales"], s["a_row"], fmts[c["w"]], s["w"],
                                           s["w_scales"], s["w_row"], s["offs"], err=s["err"])
        return {"out": out}
    if op == "norm":
        codes, scales, row, h, rstd, post_rstd = bsq.bsq_norm_quantize(
            s["x"], fmts[c["fmt"]], s["weight"], residual=s["residual"], gate=s["gate"], post_weight=s["post_weight"],
            residual_scale=c["scale"], eps=EPS)
        out = {"codes": _held_values(codes, c["fmt"]), "scales": _scales(scales, c["fmt"]), "rstd": rstd}
        return _norm_out(s, out, row, h, post_rstd)
    if op == "norm_bwd":
        got = bsq.bsq_norm_quantize_backward(
            s["grad_y"], s["h"], s["rstd"], s["weight"], grad_h=s["grad_h"], x=s["x"], gate=s["gate"],
            post_weight=s["post_weight"], post_rstd=s["post_rstd"], residual_scale=c["scale"])
        out = dict(zip(("grad_residual", "grad_x", "grad_gate", "grad_weight", "grad_post_weight"), got))
        if not (c["post"] or c["gate"] or c["scale"] != 1.0):
            del out["grad_x"]
        return {k: v for k, v in out.items() if v is not None}
    if op == "swiglu":
        codes, scales, row = bsq.bsq_swiglu_quantize(s["x"], fmts[c["fmt"]])
        out = {"codes": _held_values(codes, c["fmt"]), "scales": _scales(scales, c["fmt"])}
        return out if row is None else {**out, "row_scale": row}
    return {"grad_x": bsq.bsq_swiglu_backward(s["grad_y"], s["x"])}


# ------------------------------------------------ the definitions, 64 bits --

def _nearest(v, grid):
    """Nearest value of an ascending grid whose even places win ties; beyond its end the end."""
    grid = torch.tensor(grid, dtype=torch.float64, device=v.device)
    mids = (grid[1:] + grid[:-1]) / 2
    lo = torch.bucketize(v.abs(), mids)               # place with mids[lo - 1] < |v| <= mids[lo]
    tie = (lo < mids.numel()) & (v.abs() == mids[lo.clamp(max=mids.numel() - 1)]) & (lo % 2 == 1)
    return torch.sign(v) * grid[lo + tie.long()]


def _e4m3_grid():
    return [m * 2.0 ** -9 for m in range(8)] + [(8 + m) / 8 * 2.0 ** e for e in range(-6, 9) for m in range(8) if not (e == 8 and m == 7)]


def _exact_quantized(y, fmt):
    """(code values, scale values, row scales) of the format's definition."""
    n = BLOCK[fmt]
    z = y.unflatten(-1, (y.shape[-1] // n, n))
    top = z.abs().max(-1).values
    if fmt == "nvfp4":
        row = y.abs().max(-1).values / (6.0 * 448.0)
        live = (row > 0).unsqueeze(-1)
        unit = torch.where(live, row.unsqueeze(-1), torch.ones_like(row).unsqueeze(-1))
        scale = torch.where(live, _nearest(torch.clamp(top / 6.0 / unit, min=2.0 ** -9), _e4m3_grid()), torch.zeros_like(top))
        step = torch.where(live, scale * unit, torch.ones_like(top))
        return _nearest(z / step.unsqueeze(-1), _E2M1[:8]).flatten(-2), scale, row
    low = 2 if fmt == "mxfp4" else 8
    power = torch.floor(torch.log2(torch.where(top > 0, top, torch.ones_like(top))))
    power = power + (torch.exp2(power + 1) <= top).double() - (torch.exp2(power) > top).double()  # log2 next to a power of two
    power = torch.where(top > 0, power - low, torch.full_like(top, -127.0)).clamp(-127, 127)
    scale = torch.exp2(power)
    return _nearest(z / scale.unsqueeze(-1), _E2M1[:8] if fmt == "mxfp4" else _e4m3_grid()).flatten(-2), scale, None


def exact(case, seed):
    s = prepare(case, seed)
    d = {k: v.double() if isinstance(v, torch.Tensor) and v.is_floating_point() else v for k, v in s.items()}
    op = case["op"]
    if op == "mm":
        out = torch.zeros(case["T"], case["N"], dtype=torch.float64, device="cuda")
        begin = 0
        for e, n in enumerate(s["counts"]):
            if n:
                part = slice(begin, begin + n)
                x = _dequantized(s["a"][part], s["a_scales"][part], None if s["a_row"] is None else s["a_row"][part], case["a"], torch.float64)
                v = _dequantized(s["w"][e], s["w_scales"][e], None if s["w_row"] is None else s["w_row"][e], case["w"], torch.float64)
                out[part] = x @ v.T
            begin += n
        return {"out": out}
    if op in ("swiglu", "swiglu_bwd"):
        gate, up = d["x"].chunk(2, -1)
        sig = torch.sigmoid(gate)
        if op == "swiglu_bwd":
            slope = sig + gate * sig * (1 - sig)
            return {"grad_x": torch.cat([d["grad_y"] * up * slope, d["grad_y"] * gate * sig], -1)}
        codes, scales, row = _exact_quantized(gate * sig * up, case["fmt"])
        out = {"codes": codes, "scales": scales}
        return out if row is None else {**out, "row_scale": row}
    rms = lambda t: 1.0 / torch.sqrt((t * t).sum(-1) / t.shape[-1] + EPS)  # noqa: E731
    if op == "norm":
        v = d["x"]
        if case["post"]:
            v = v * rms(v).unsqueeze(-1) * d["post_weight"]
        if case["gate"]:
            v = v * d["gate"]
        h = v * case["scale"] + (d["residual"] if case["residual"] else 0.0)
        codes, scales, row = _exact_quantized(h * rms(h).unsqueeze(-1) * d["weight"], case["fmt"])
        return _norm_out(s, {"codes": codes, "scales": scales, "rstd": rms(h)}, row, h, rms(d["x"]) if case["post"] else None)
    # y = h r w with r = rstd(h): dL/dh = r (w gy - h r^2 <w gy, h> / C), on top of the stream's own gradient
    r, C = d["rstd"].unsqueeze(-1), case["C"]
    wg = d["weight"] * d["grad_y"]
    dh = d["grad_h"] + r * wg - d["h"] * r ** 3 * (wg * d["h"]).sum(-1, keepdim=True) / C
    out = {"grad_residual": dh, "grad_weight": (d["grad_y"] * d["h"] * r).sum(0)}
    if case["post"] or case["gate"] or case["scale"] != 1.0:
        p = d["post_rstd"].unsqueeze(-1) if case["post"] else 1.0
        u = d["x"] * p * (d["post_weight"] if case["post"] else 1.0)
        du = case["scale"] * dh * (d["gate"] if case["gate"] else 1.0)
        if case["gate"]:
            out["grad_gate"] = case["scale"] * dh * u
        if case["post"]:
            out["grad_post_weight"] = (du * d["x"] * p).sum(0)
            wd = d["post_weight"] * du
            du = p * wd - d["x"] * p ** 3 * (wd * d["x"]).sum(-1, keepdim=True) / C
        out["grad_x"] = du
    return out
