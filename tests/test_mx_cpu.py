"""The MX operators without a GPU: the oracle against values written down by
hand, and every refusal of the C entry points (validation runs before any HIP
call, so the fake pointers are never read)."""
import ctypes
import os

import numpy as np
import pytest

from oracle import mx


@pytest.fixture(scope="module")
def lib():
    from q4_packed_weight_amd import binding
    if not os.path.exists(binding.LIB_PATH):
        from q4_packed_weight_amd import build
        build.build()
    return binding.lib()


P = ctypes.c_void_p
A, B, C, D, E = (P(0x100000 * i) for i in range(1, 6))
ODD = P(0x100004)
F32, FP4, FP8 = 0, 4, 8
EPS = ctypes.c_float(1e-5)


# ------------------------------------------------------------ the oracle

def test_element_values():
    assert mx.E2M1.tolist() == [0, 0.5, 1, 1.5, 2, 3, 4, 6]
    assert mx.E4M3[1] == 2.0 ** -9 and mx.E4M3[8] == 2.0 ** -6 and mx.E4M3[126] == 448


def _row(values):
    x = np.zeros((1, 32))
    x[0, :len(values)] = values
    return x


def test_fp4_rounds_to_nearest_even_and_saturates():
    # amax 4..7.99 has scale 2^0
    vals = [7.9, 0.25, 0.26, 0.75, 1.25, 1.26, 1.75, 2.5, 2.51, 3.5, 5.0, 5.01, -0.25, -5.0]
    codes, scales = mx.quantize(_row(vals), "fp4")
    assert scales.tolist() == [[127]]
    got = mx.dequantize(codes, scales, "fp4")[0, :len(vals)]
    assert got.tolist() == [6, 0, 0.5, 1, 1, 1.5, 2, 2, 3, 4, 4, 6, 0, -4]


def test_fp8_rounds_to_nearest_even_and_saturates():
    # amax 256..511.9 has scale 2^0
    vals = [500.0, 449.0, 17.0, 19.0, 2.0 ** -9, 2.0 ** -10, 3 * 2.0 ** -10, -17.0]
    codes, scales = mx.quantize(_row(vals), "fp8")
    assert scales.tolist() == [[127]]
    got = mx.dequantize(codes, scales, "fp8")[0, :len(vals)]
    assert got.tolist() == [448, 448, 16, 20, 2.0 ** -9, 0, 2.0 ** -8, -16]


def test_special_blocks():
    x = np.zeros((5, 32))
    x[1, 3] = np.nan
    x[2, 4] = -np.inf
    x[3, 0] = 2.0 ** -140
    x[4, 0] = 2.0 ** 127
    for fmt in ("fp4", "fp8"):
        codes, scales = mx.quantize(x, fmt)
        assert scales[:, 0].tolist() == [0, 255, 255, 0, 254 - mx.SHIFT[fmt]]
        assert not codes[:3].any()
    assert np.isnan(mx.dequantize(*mx.quantize(x, "fp4"), "fp4")[1]).all()


def test_nibble_order():
    codes, scales = mx.quantize(_row([4.0, -1.5]), "fp4")
    assert codes[0, 0] == 6 | (11 << 4)
    assert mx.dequantize(codes, scales, "fp4")[0, :3].tolist() == [4, -1.5, 0]


def test_choice_takes_the_lower_index_of_equal_logits_and_nan_last():
    l = np.array([[1.0, 2.0, 2.0, np.nan, 0.5], [0.0, -0.0, 0.0, 0.0, 0.0],
                  [np.nan, -np.inf, np.nan, 1.0, np.nan]])
    assert mx.choose(l, 3).tolist() == [[1, 2, 0], [0, 1, 2], [3, 1, 0]]


# ------------------------------------------------------------ refusals

@pytest.mark.parametrize("K", [0, -32, 31, 33, 48, (1 << 24) + 32])
def test_rejects_bad_input_dim(lib, K):
    assert lib.mx_quantize(A, F32, FP4, 4, K, B, C, None) == -1
    assert lib.mx_dequantize(A, B, FP4, 4, K, C, F32, None) == -1
    assert lib.mx_rmsnorm(A, None, B, EPS, F32, 4, K, None, None, FP8, C, D, None) == -1
    assert lib.mxfp4_matmul(A, B, FP8, C, D, 4, K, 16, E, F32, None) == -1
    assert lib.mxfp4_moe(A, F32, B, None, C, D, C, D, 4, K, 64, 4, 2, E, A, 1 << 40, None) == -1
    assert lib.mxfp4_moe(A, F32, B, None, C, D, C, D, 4, 64, K, 4, 2, E, A, 1 << 40, None) == -1
    assert lib.mxfp4_moe_workspace_size(4, K, 64, 4, 2) == -1
    assert lib.mxfp4_moe_workspace_size(4, 64, K, 4, 2) == -1


@pytest.mark.parametrize("n", [0, -1, 1 << 31])
def test_rejects_bad_row_counts(lib, n):
    assert lib.mx_quantize(A, F32, FP4, n, 64, B, C, None) == -1
    assert lib.mx_dequantize(A, B, FP4, n, 64, C, F32, None) == -1
    assert lib.mx_rmsnorm(A, None, B, EPS, F32, n, 64, None, None, FP8, C, D, None) == -1
    assert lib.mxfp4_matmul(A, B, FP8, C, D, n, 64, 16, E, F32, None) == -1
    assert lib.mxfp4_matmul(A, B, FP8, C, D, 4, 64, n, E, F32, None) == -1
    assert lib.mxfp4_moe(A, F32, B, None, C, D, C, D, n, 64, 64, 4, 2, E, A, 1 << 40, None) == -1


def test_matmul_rejects_more_outputs_than_a_grid(lib):
    assert lib.mxfp4_matmul(A, B, FP8, C, D, 4, 64, (1 << 26) + 1, E, F32, None) == -1


@pytest.mark.parametrize("experts,top_k", [(0, 1), (257, 2), (4, 0), (4, 5), (64, 17), (-3, -4)])
def test_moe_rejects_bad_routing(lib, experts, top_k):
    assert lib.mxfp4_moe(A, F32, B, None, C, D, C, D, 4, 64, 64, experts, top_k, E, A, 1 << 40,
                         None) == -1
    assert lib.mxfp4_moe_workspace_size(4, 64, 64, experts, top_k) == -1


def test_rmsnorm_rejects_bad_eps(lib):
    for eps in (-1e-5, float("nan")):
        assert lib.mx_rmsnorm(A, None, B, ctypes.c_float(eps), F32, 4, 64, None, None, FP8, C, D,
                              None) == -1


@pytest.mark.parametrize("bad", [-1, 3, 5])
def test_rejects_unknown_types_and_formats(lib, bad):
    assert lib.mx_quantize(A, bad, FP4, 4, 64, B, C, None) == -6
    assert lib.mx_quantize(A, F32, bad, 4, 64, B, C, None) == -6
    assert lib.mx_dequantize(A, B, bad, 4, 64, C, F32, None) == -6
    assert lib.mx_dequantize(A, B, FP4, 4, 64, C, bad, None) == -6
    assert lib.mx_rmsnorm(A, None, B, EPS, bad, 4, 64, None, None, FP8, C, D, None) == -6
    assert lib.mx_rmsnorm(A, None, B, EPS, F32, 4, 64, None, None, bad, C, D, None) == -6
    assert lib.mxfp4_matmul(A, B, bad, C, D, 4, 64, 16, E, F32, None) == -6
    assert lib.mxfp4_matmul(A, B, FP8, C, D, 4, 64, 16, E, bad, None) == -6
    assert lib.mxfp4_moe(A, bad, B, None, C, D, C, D, 4, 64, 64, 4, 2, E, A, 1 << 40, None) == -6


def test_rejects_null_pointers(lib):
    for i in range(3):
        p = [A, B, C]
        p[i] = None
        assert lib.mx_quantize(p[0], F32, FP4, 4, 64, p[1], p[2], None) == -2
        assert lib.mx_dequantize(p[0], p[1], FP4, 4, 64, p[2], F32, None) == -2
    assert lib.mx_rmsnorm(None, A, B, EPS, F32, 4, 64, None, None, FP8, C, D, None) == -2
    assert lib.mx_rmsnorm(A, None, None, EPS, F32, 4, 64, None, None, FP8, C, D, None) == -2
    assert lib.mx_rmsnorm(A, None, B, EPS, F32, 4, 64, None, None, FP8, C, None, None) == -2
    assert lib.mx_rmsnorm(A, None, B, EPS, F32, 4, 64, None, None, FP8, None, D, None) == -2
    # nothing to write
    assert lib.mx_rmsnorm(A, None, B, EPS, F32, 4, 64, None, None, 0, None, None, None) == -2
    for i in range(5):
        p = [A, B, C, D, E]
        p[i] = None
        assert lib.mxfp4_matmul(p[0], p[1], FP8, p[2], p[3], 4, 64, 16, p[4], F32, None) == -2
    for i in range(8):
        p = [A, B, C, D, C, D, E, A]
        p[i] = None
        assert lib.mxfp4_moe(p[0], F32, p[1], None, *p[2:6], 4, 64, 64, 4, 2, p[6], p[7], 1 << 40,
                             None) == -2


def test_rejects_misaligned(lib):
    assert lib.mx_quantize(ODD, F32, FP4, 4, 64, B, C, None) == -3
    assert lib.mx_quantize(A, F32, FP4, 4, 64, ODD, C, None) == -3
    assert lib.mx_dequantize(ODD, B, FP4, 4, 64, C, F32, None) == -3
    assert lib.mx_dequantize(A, B, FP4, 4, 64, ODD, F32, None) == -3
    for i in range(6):
        p = [A, B, C, D, E, A]
        p[i] = ODD
        assert lib.mx_rmsnorm(p[0], p[1], p[2], EPS, F32, 4, 64, p[3], p[4], FP8, p[5], D,
                              None) == -3
    assert lib.mxfp4_matmul(ODD, B, FP8, C, D, 4, 64, 16, E, F32, None) == -3
    assert lib.mxfp4_matmul(A, B, FP8, ODD, D, 4, 64, 16, E, F32, None) == -3
    for i in (0, 1, 2, 4, 6, 7):
        p = [A, B, C, D, C, D, E, A]
        p[i] = ODD
        assert lib.mxfp4_moe(p[0], F32, p[1], None, *p[2:6], 4, 64, 64, 4, 2, p[6], p[7], 1 << 40,
                             None) == -3
    assert lib.mxfp4_moe(A, F32, B, P(0x100002), C, D, C, D, 4, 64, 64, 4, 2, E, A, 1 << 40,
                         None) == -3


def test_moe_workspace(lib):
    n = lib.mxfp4_moe_workspace_size(4, 64, 96, 4, 2)
    assert n > 0 and n % 256 == 0
    assert lib.mxfp4_moe(A, F32, B, None, C, D, C, D, 4, 64, 96, 4, 2, E, A, n - 1, None) == -5
    assert b"workspace" in lib.q4k_strerror(-5)
    # 64 tokens at a time (fewer where the logits would not fit): no growth beyond
    assert (lib.mxfp4_moe_workspace_size(64, 64, 96, 4, 2)
            == lib.mxfp4_moe_workspace_size(5000, 64, 96, 4, 2))
    assert (lib.mxfp4_moe_workspace_size(32, 64, 96, 256, 2)
            == lib.mxfp4_moe_workspace_size(64, 64, 96, 256, 2))


def test_errors_come_in_order_and_have_texts(lib):
    assert lib.mx_quantize(None, 9, FP4, 4, 33, ODD, C, None) == -1
    assert lib.mx_quantize(None, 9, FP4, 4, 64, ODD, C, None) == -6
    assert lib.mx_quantize(None, F32, FP4, 4, 64, ODD, C, None) == -2
    assert b"type" in lib.q4k_strerror(-6)


def test_binding_refuses_what_it_marshals():
    import torch
    from q4_packed_weight_amd import binding
    x = torch.zeros(2, 64)
    c = torch.zeros(2, 32, dtype=torch.uint8)
    s = torch.zeros(2, 2, dtype=torch.uint8)
    with pytest.raises(ValueError):
        binding.mx_quantize(x, 2, 64, "fp6", c, s)
    with pytest.raises(TypeError):
        binding.mx_quantize(x.double(), 2, 64, "fp4", c, s)
    with pytest.raises(ValueError):  # not a GPU tensor
        binding.mx_quantize(x, 2, 64, "fp4", c, s)
    with pytest.raises(ValueError):  # strided
        binding.mx_quantize(torch.zeros(64, 2).t(), 2, 64, "fp4", c, s)
    with pytest.raises(ValueError):
        binding.mx_quantize(None, 2, 64, "fp4", c, s)
    with pytest.raises(ValueError) as e:
        binding.mxfp4_moe_workspace_size(1, 33, 32, 4, 1)
    assert e.value.code == binding.Q4K_EINVAL_DIM
