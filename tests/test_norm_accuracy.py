"""GPU tests of the norms' row factors: what is common to all elements of a row
must carry no more than its own roundings.

Every step rounds to nearest, so errors average out.  With u = 2**-24, the
relative error of a row's rstd (a sum of squares, a division, a sum, a root, each
rounded) is within u or so of zero either way, and its mean over R rows within
6 u / sqrt(R) of zero.  One step does not average out: the mean square m lies on
binary32's grid, where m + eps is the same fraction of a step off for every m of
a binade (m in [1, 2), eps = 1e-6 = 8.39 steps: 0.39 of a step, 0.39 u of the
root), so the reference takes that step in binary32 as the formula does.  A factor 1 / C rounded beforehand would shift it for every
row (C = 7168: 0.37 u).  In h = scale * (x post_rstd post_weight gate) four
products round per element, each by up to u, so the mean relative error over a
row of C elements is within 6 * 4 u / sqrt(C) of zero; a product scale * post_rstd
rounded beforehand would shift the whole row by up to u.  And the row scale of
y = h rstd weight is its three roundings off at most (3 u)."""
import numpy as np
import pytest
import torch

from gpu_util import dev, host_bits

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


@pytest.fixture(scope="module")
def B():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from fp8_microscaling_quantization_b200 import bsq
    return bsq


def f64(t):
    return host_bits(t).astype(np.float64)


@pytest.mark.parametrize("rows,C", [(8192, 7168), (8192, 2080), (8192, 224), (2048, 10240), (1024, 28672)])
def test_row_factors_are_not_biased(B, rows, C):
    g = torch.Generator(device="cuda").manual_seed(C)
    x = torch.randn(rows, C, generator=g, device="cuda")
    w = 1 + 0.1 * torch.randn(C, generator=g, device="cuda")
    eps = 1e-6
    _, _, row, h, rstd, post = B.bsq_norm_quantize(x, B.Format.NVFP4, w, post_weight=w, residual_scale=0.22, eps=eps)
    torch.cuda.synchronize()
    hd = h.double()
    for got, v in ((post, x.double()), (rstd, hd)):
        want = ((v * v).mean(-1).float() + eps).double() ** -0.5
        off = float(((got.double() - want) / want).mean()) / U
        assert abs(off) <= 6 / np.sqrt(rows), f"mean relative error of a row factor: {off:.3f} u"
    y = ((hd * rstd.double()[:, None]).abs() * w.double().abs()).amax(-1) / 2688
    assert bool(((row.double() - y).abs() <= 3 * U * (1 + 2.0 ** -10) * y).all())


@pytest.mark.parametrize("rows,C", [(300, 7168), (50, 18432), (40, 28672)])
def test_rows_carry_the_factor_they_return(B, rows, C):
    g = torch.Generator(device="cuda").manual_seed(rows)
    x, z = (torch.randn(rows, C, generator=g, device="cuda") for _ in range(2))
    w, pw = (1 + 0.1 * torch.randn(C, generator=g, device="cuda") for _ in range(2))
    s = 0.22
    h, post = [B.bsq_norm_quantize(x, B.Format.MXFP8, w, gate=z, post_weight=pw, residual_scale=s)[i] for i in (3, 5)]
    torch.cuda.synchronize()
    want = x.double() * post.double()[:, None] * pw.double() * z.double() * float(np.float32(s))
    assert not bool(h[want == 0].any())  # (a normal sample may be 0)
    off = ((h.double() - want) / torch.where(want == 0, 1.0, want)).mean(-1).abs().max()
    assert float(off) / U <= 24 / np.sqrt(C), f"a row is {float(off) / U:.3f} u off as a whole"
