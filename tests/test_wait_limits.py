"""GPU tests of the products' bounded waits: with the limit of each wait cut
short (BSQ_GMM_WAIT_NS) the kernel gives up somewhere in its pipeline, waits
for its loads in flight and returns; the context stays usable and the next call
is right.  A call that still finished in time has to be right itself.  (How the
loads are waited for is checked on the CPU first: test_pipeline_drain.py.)"""
import numpy as np
import pytest
import torch

from test_scaled_mm import call, check, problem

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def B():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from fp8_microscaling_quantization_b200 import bsq
    return bsq


# pair of formats, T, N, K, offs; whether a limit of 1 ns always runs out (a
# load takes far longer, but the clock that the limit is read from is coarse)
SCALED = [
    ("nvfp4", 3000, 2048, 2048, None, True),                        # pairs
    ("mxfp8", 3000, 2048, 1056, None, True),                        # pairs, scale rows loaded by the warps
    ("w4a8", 2000, 2048, 1024, [700, 700, 1400, 1990], True),       # pairs, grouped
    ("nvfp4", 700, 512, 256, None, False),                          # single CTAs, the contraction within the ring
    ("mxfp4", 700, 512, 4096, [100, 130, 600], True),               # single CTAs, grouped
    ("mxfp8", 600, 520, 1056, None, False),                         # single CTAs, scale rows loaded by the warps
    ("nvfp4", 1, 2048, 7168, None, False),                          # the contraction split over a cluster
    ("mxfp8", 20, 264, 2080, None, False),                          # the same, scale rows loaded by the warps
]


@pytest.mark.parametrize("pair,T,N,K,offs,sure", SCALED)
def test_block_scaled_product_gives_up_and_recovers(B, oracle, monkeypatch, pair, T, N, K, offs, sure):
    E = len(offs) if offs else 1
    af, wf, a, w = problem(oracle, B, pair, T, N, K, E, T + K)
    offs = np.array(offs, np.int32) if offs else None
    rows = np.unique(np.concatenate([np.arange(min(T, 40)), np.arange(max(0, T - 40), T)]))
    for ns in (1, 1, 300, 1000, 2000, 3000, 5000, 8000, 12000, 20000):
        monkeypatch.setenv("BSQ_GMM_WAIT_NS", str(ns))
        got, err = call(B, af, wf, a, w, offs)
        assert err in ((2,) if sure and ns == 1 else (0, 2)), f"limit {ns} ns: error word {err}"
        if err == 0:
            check(got, a, w, offs, T, f"in time at {ns} ns", rows)
    monkeypatch.delenv("BSQ_GMM_WAIT_NS")
    got, err = call(B, af, wf, a, w, offs)
    assert err == 0
    check(got, a, w, offs, T, "after timed-out calls", rows)


# CTA pairs or singles, format, T, N, K, experts, backward
DEQUANT = [
    ("1", "mxfp4", 2500, 512, 1024, 5, False),  # pairs, two MMAs per k-step
    ("1", "nvfp4", 700, 1024, 512, 3, True),
    ("1", "nvfp4", 300, 256, 128, 2, False),    # the contraction within the ring
    ("0", "nvfp4", 1500, 256, 1024, 4, False),  # single CTAs
    ("0", "mxfp4", 300, 128, 128, 2, True),
]


@pytest.mark.parametrize("cta_pair,name,T,N,K,E,backward", DEQUANT)
def test_dequantizing_product_gives_up_and_recovers(B, oracle, monkeypatch, cta_pair, name, T, N, K, E, backward):
    from test_parity_gemm import check_rows, make_problem, quantize_weights, run_gemm
    monkeypatch.setenv("BSQ_GMM_CTA_PAIR", cta_pair)
    x, w, go, offs = make_problem(T, K, N, E, T + K)
    fmt = oracle.FMT_MXFP4 if name == "mxfp4" else oracle.FMT_NVFP4
    packed, scales, g = quantize_weights(oracle, fmt, w)
    a = go if backward else x
    end = int(offs[-1])
    rows = np.unique(np.concatenate([np.arange(min(end, 40)), np.arange(max(0, end - 40), end)]))
    ref = oracle.grouped_mm_rows(fmt, backward, a, packed, scales, g, offs, rows)
    Wmax = max(np.abs(oracle.dequant_expert_f32(fmt, packed[e], scales[e], None if g is None else g[e])).max()
               for e in range(E))
    for ns in (1, 1, 300, 1000, 2000, 3000, 5000, 8000, 12000, 20000):
        monkeypatch.setenv("BSQ_GMM_WAIT_NS", str(ns))
        got, err = run_gemm(B, oracle, fmt, backward, a, packed, scales, g, offs)
        assert err in (0, 2), f"limit {ns} ns: error word {err}"
        if err == 0:
            check_rows(got[rows], ref, a, Wmax, N if backward else K, f"in time at {ns} ns")
    monkeypatch.delenv("BSQ_GMM_WAIT_NS")
    got, err = run_gemm(B, oracle, fmt, backward, a, packed, scales, g, offs)
    assert err == 0
    check_rows(got[rows], ref, a, Wmax, N if backward else K, "after timed-out calls")
