"""GPU tests of the product of two block-scaled operands over long
contractions, where the per-output bound of binary32 accumulation ((K + 2) 2**-23
of sum |a||w|, 7% of a typical output at K = 7168) would not see a scale block
left out or taken twice.

In norm it is seen.  Per token and per feature, |out - ref| is at most 2**-8 |ref|
for the rounding to bf16, plus the accumulation: at most a last place (2**-23) of
the running sum per MMA of 32 columns or more, K / 32 of them, and of random
signs the running sum stays below some 4 standard deviations of the output:
(7168 / 32) 2**-23 4 = 1.1e-4.  So 2**-8 + 2e-4 = 4.1e-3 holds, and one block of 32
of 7168 columns is sqrt(32 / 7168) = 6.7e-2, one of 16 4.7e-2."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

BOUND = 2.0 ** -8 + 2e-4


@pytest.fixture(scope="module")
def B():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from fp8_microscaling_quantization_b200 import bsq
    return bsq


def within(out, ref):
    """Whether out is within BOUND of ref in the norm of every row and column."""
    d = (out.double() - ref).square()
    r = ref.square()
    return all(bool((d.sum(i).sqrt() <= BOUND * r.sum(i).sqrt()).all()) for i in (0, 1))


@pytest.mark.parametrize("pair", ["nvfp4", "mxfp4", "mxfp8", "w4a8"])
@pytest.mark.parametrize("T,N,K", [(5, 2048, 7168),     # the contraction split over a cluster
                                   (128, 520, 7296),    # single CTAs; MXFP8's scale rows loaded by the warps
                                   (3000, 2048, 7168),  # pairs
                                   (2000, 1032, 7296)])
def test_every_block_counts_once(B, pair, T, N, K):
    from test_feed_forward_run import dequantize, quantize
    F = B.Format
    af, wf = {"nvfp4": (F.NVFP4, F.NVFP4), "mxfp4": (F.MXFP4, F.MXFP4), "mxfp8": (F.MXFP8, F.MXFP8), "w4a8": (F.MXFP8, F.MXFP4)}[pair]
    g = torch.Generator(device="cuda").manual_seed(T + K)
    a = quantize(B, af, torch.randn(T, K, generator=g, device="cuda").bfloat16())
    w = quantize(B, wf, torch.randn(N, K, generator=g, device="cuda").bfloat16())
    out, err = B.bsq_grouped_mm_scaled(af, *a, wf, *w)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    av, wv = dequantize(B, af, *a), dequantize(B, wf, *w)
    ref = av @ wv.T
    assert within(out, ref), f"{pair} {T} x {N} x {K}"
    # the bound sees a block that one side left out, or took twice, in one row alone
    n = 16 if pair == "nvfp4" else 32
    for k in (0, K // n // 2 * n, K - n):
        part = av[T // 2, k:k + n] @ wv[:, k:k + n].T
        for sign in (-1, 1):
            wrong = ref.clone()
            wrong[T // 2] += sign * part
            assert not within(out, wrong)
