"""GPU tests of the gated activation's binary32 values, gates far from zero
included, against float64.

A row whose 16 gates are one value and whose up values are another has one y
in every place, and the NVFP4 row scale is RN(|y| / 2688): y itself, give or
take one rounding.  With u = 2**-24 (half a last place, relative), y carries
the exponential's 2 last places (4 u), its sum with 1 (1 u), the reciprocal's
last place (2 u), for bf16 the neglected square of the split product (at most
(87.3 * 4.9e-6)**2 / 2 = 1.6 u) and the fma that applies it (1 u), two products
(2 u) and the row scale's division (1 u): 13 u for bf16, 10 u for fp32, however
large the gate.  The backward pass divides (1 u) instead of the reciprocal:
its up half carries 4 + 1 + 1 + 2 = 8 u; its gate half, d u (s + g s (1 - s)),
that and 1 - s, which carries s's error in units of s, on each term."""
import numpy as np
import pytest
import torch

from gpu_util import dev, dev_bf16, host_bits

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


@pytest.fixture(scope="module")
def B():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from fp8_microscaling_quantization_b200 import bsq
    return bsq


def gates(dtype):
    """(device tensor, float64 values): -87 to 87, densest near zero."""
    from fp8_microscaling_quantization_b200 import synth
    rng = np.random.default_rng(3)
    v = np.concatenate([np.linspace(-87, 87, 2001), rng.standard_normal(2000) * 3, -np.exp(rng.uniform(-6, 4.46, 2000))])
    v = v.astype(np.float32)
    if dtype == "bf16":
        b = synth.to_bf16_bits(v)
        return dev_bf16(b), np.clip(synth.bf16_bits_to_f32(b).astype(np.float64), -88, 88)
    return dev(v), v.astype(np.float64)


@pytest.mark.parametrize("dtype,tol", [("bf16", 13), ("fp32", 10)])
def test_activation_of_any_gate_is_a_few_last_places_off(B, dtype, tol):
    t, g = gates(dtype)
    up = 1.5
    x = torch.cat([t[:, None].expand(-1, 16), torch.full((len(g), 16), up, dtype=t.dtype, device="cuda")], 1).contiguous()
    codes, scales, row = B.bsq_swiglu_quantize(x, B.Format.NVFP4)
    torch.cuda.synchronize()
    want = np.abs(g / (1 + np.exp(-g)) * up) / 2688.0
    off = np.abs(host_bits(row).astype(np.float64) - want) - tol * U * want
    # (a row scale below 2**-126 has fewer bits)
    assert np.all(off <= 2.0 ** -149), f"gate {g[np.argmax(off / np.maximum(want, 1e-300))]}: {np.max(off / np.maximum(want, 1e-300)) / U} u past"
    # all 16 values are the row's maximum: the largest code, the largest scale
    live = host_bits(row) > 0
    assert np.all(host_bits(scales)[live] == 0x7E) and np.all(host_bits(codes)[live] & 0x77 == 0x77)


def test_activation_backward_of_any_gate_is_a_few_last_places_off(B):
    t, g = gates("fp32")
    d, up = 0.75, 1.5
    x = torch.stack([t, torch.full_like(t, up)], 1)[:, :, None].expand(-1, -1, 8).reshape(len(g), 16).contiguous()
    gx = B.bsq_swiglu_backward(torch.full((len(g), 8), d, device="cuda"), x)
    torch.cuda.synchronize()
    got = host_bits(gx).astype(np.float64).reshape(len(g), 2, 8)
    assert np.all(got == got[:, :, :1])
    s = 1 / (1 + np.exp(-g))
    want = d * g * s
    assert np.all(np.abs(got[:, 1, 0] - want) <= 8 * U * np.abs(want) + 2.0 ** -148)
    want = d * up * (s + g * s * (1 - s))
    # s carries 6 u, g s 7 u, 1 - s half a last place of 1 at most and 6 u of s; three more products and the sum 4 u
    err = 10 * U * s + np.abs(g) * s * (11 * U * (1 - s) + 7 * U * s)
    assert np.all(np.abs(got[:, 0, 0] - want) <= d * up * err + 2.0 ** -148)


def test_gates_past_every_border_stay_finite(B):
    """The largest finite gates of either sign, and those around the borders of
    the exponential's and the reciprocal's range: y is g u or 0 (to 2**-110)."""
    top = float(torch.finfo(torch.bfloat16).max)
    g = [-top, -1e30, -1000.0, -129.0, -128.0, -100.0, -89.0, -88.0, 88.0, 89.0, 128.0, 1000.0, 1e30, top]
    for dt in (torch.bfloat16, torch.float32):
        t = torch.tensor(g, device="cuda").to(dt)
        x = torch.cat([t[:, None].expand(-1, 16), torch.ones(len(g), 16, dtype=dt, device="cuda")], 1).contiguous()
        row = B.bsq_swiglu_quantize(x, B.Format.NVFP4)[2].double() * 2688
        gx = B.bsq_swiglu_backward(torch.ones(len(g), 16, dtype=dt, device="cuda"), x).double()
        torch.cuda.synchronize()
        want = t.double().clamp(min=0)
        assert bool(torch.isfinite(gx).all())
        assert bool(((row - want).abs() <= 16 * U * want + 2.0 ** -110).all())
        assert bool(((gx[:, 16] - want).abs() <= 2.0 ** -8 * want + 2.0 ** -110).all())
        assert bool(((gx[:, 0] - (want > 0).double()).abs() <= 2.0 ** -8).all())


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("rows,F", [(1, 8), (700, 2064), (3, 18432)])
def test_activation_backward_in_place(B, dtype, rows, F):
    """grad_x may be x itself: the same bits as into a tensor of its own."""
    g = torch.Generator(device="cuda").manual_seed(F)
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    x = (2 * torch.randn(rows, 2 * F, generator=g, device="cuda")).to(dt)
    gy = torch.randn(rows, F, generator=g, device="cuda").to(dt)
    want = B.bsq_swiglu_backward(gy, x)
    got = B.bsq_swiglu_backward(gy, x, grad_x=x)
    torch.cuda.synchronize()
    assert got is x and torch.equal(got, want)
