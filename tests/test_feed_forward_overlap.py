"""Outputs of the block-scaled feed-forward operators that share memory with an
input or with one another are refused (CPU: addresses only, nothing is
launched); what the documentation allows in place is not refused for it."""
import ctypes

import pytest

P, I64, F32, SZ = ctypes.c_void_p, ctypes.c_int64, ctypes.c_float, ctypes.c_size_t
INVALID = 1
MXFP4, NVFP4, MXFP8 = 1, 2, 3
ROWS, C = 4, 64
BASE, STEP = 0x100000, 0x10000  # operands far apart


@pytest.fixture(scope="module")
def lib():
    from fp8_microscaling_quantization_b200 import build
    l = ctypes.CDLL(build.build())
    l.bsq_last_error.restype = ctypes.c_char_p
    return l


def refused(lib, rc):
    return rc == INVALID and "overlap" in lib.bsq_last_error().decode()


def place(names):
    return {n: BASE + i * STEP for i, n in enumerate(names)}


# operand -> bytes, of 4 x 64 bf16 quantized to NVFP4 and so on
NORM = {"x": 512, "residual": 512, "gate": 512, "post_weight": 256, "weight": 256, "h": 512, "codes": 128, "scales": 16,
        "row_scale": 16, "rstd": 16, "post_rstd": 16}


def norm(lib, at):
    return lib.bsq_norm_quantize(NVFP4, *(P(at[n]) for n in ("x", "residual", "gate")), 0, I64(ROWS), I64(C), F32(1),
                                 P(at["post_weight"]), P(at["weight"]), F32(1e-6),
                                 *(P(at[n]) for n in ("h", "codes", "scales", "row_scale", "rstd", "post_rstd")), None)


@pytest.mark.parametrize("out", ["h", "codes", "scales", "row_scale", "rstd", "post_rstd"])
def test_norm_outputs(lib, out):
    for other in NORM:
        if other == out:
            continue
        for shift in (0, NORM[other] - 16):  # from its first byte, and over its last 16
            at = place(NORM)
            at[out] = at[other] + shift
            if out == "h" and other in ("x", "residual") and shift == 0:
                continue  # in place: allowed (not called here, it would launch)
            assert refused(lib, norm(lib, at)), (out, other, shift)


BWD = {"grad_y": 512, "grad_h": 512, "h": 512, "rstd": 16, "weight": 256, "x": 512, "gate": 512, "post_weight": 256,
       "post_rstd": 16, "grad_residual": 512, "grad_x": 512, "grad_gate": 512, "grad_weight": 256, "grad_post_weight": 256,
       "scratch": 2048}


def norm_bwd(lib, at):
    ins = ("grad_y", "grad_h", "h", "rstd", "weight", "x", "gate", "post_weight", "post_rstd")
    outs = ("grad_residual", "grad_x", "grad_gate", "grad_weight", "grad_post_weight", "scratch")
    return lib.bsq_norm_quantize_backward(*(P(at[n]) for n in ins), F32(1), 0, I64(ROWS), I64(C), *(P(at[n]) for n in outs),
                                          SZ(1 << 20), None)


@pytest.mark.parametrize("out", ["grad_residual", "grad_x", "grad_gate", "grad_weight", "grad_post_weight", "scratch"])
def test_norm_backward_outputs(lib, out):
    for other in BWD:
        if other == out:
            continue
        for shift in (0, BWD[other] - 16):
            at = place(BWD)
            at[out] = at[other] + shift
            assert refused(lib, norm_bwd(lib, at)), (out, other, shift)


ACT = {"x": 1024, "codes": 128, "scales": 16, "row_scale": 16}


@pytest.mark.parametrize("out", ["codes", "scales", "row_scale"])
def test_activation_outputs(lib, out):
    for other in ACT:
        if other == out:
            continue
        for shift in (0, ACT[other] - 16):
            at = place(ACT)
            at[out] = at[other] + shift
            assert refused(lib, lib.bsq_swiglu_quantize(NVFP4, P(at["x"]), 0, I64(ROWS), I64(C),
                                                        *(P(at[n]) for n in ("codes", "scales", "row_scale")), None))


# T 16, N 128, K 256, two experts, NVFP4
MM = {"a": 2048, "a_scales": 256, "a_row": 64, "w": 32768, "w_scales": 4096, "w_row": 1024, "offs": 8, "out": 4096}


def test_product_output(lib):
    for other in MM:
        if other == "out":
            continue
        for shift in (0, MM[other] // 16 * 16 - 16 if MM[other] > 16 else 0, -16):
            at = place(MM)
            at["out"] = at[other] + shift
            rc = lib.bsq_grouped_mm_scaled(NVFP4, NVFP4, *(P(at[n]) for n in ("a", "a_scales", "a_row", "w", "w_scales",
                                                                              "w_row", "offs")),
                                           2, I64(16), I64(128), I64(256), P(at["out"]), P(0x90000), None)
            assert refused(lib, rc), (other, shift)
