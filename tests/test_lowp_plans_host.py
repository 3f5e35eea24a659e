"""The calls that tell how a projection on 8-bit or 4-bit operands runs refuse what the projections refuse,
without a GPU."""

import ctypes

import pytest

from qwen3_decoder_forward_gb300 import binding, build


@pytest.fixture(scope="module")
def lib():
    build.build()
    return binding.load_library()


def _refused(f, *args):
    with pytest.raises(binding.Qwen3Error) as e:
        f(*args)
    return e.value.code == binding.QWEN3_E_INVALID


@pytest.mark.parametrize("M,K,N", [(0, 16, 16), (-1, 16, 16), (2 ** 31 - 1, 16, 16), (1, 8, 16), (1, 24, 16), (1, 16, 0), (1, 16, 24)])
def test_gemm_q8_plan_refuses(lib, M, K, N):
    assert _refused(binding.qwen3_op_gemm_q8_plan, M, K, N)


@pytest.mark.parametrize("M,K,group,N", [(0, 64, 32, 8), (1, 48, 32, 8), (1, 0, 32, 8), (1, 65568, 32, 8), (1, 64, 32, 0),
                                         (1, 64, 48, 8), (1, 64, 0, 8), (1, 64, -32, 8)])
def test_gemv_w4_plan_refuses(lib, M, K, group, N):
    assert _refused(binding.qwen3_op_gemv_w4_plan, M, K, group, False, N)


def test_null_results_are_refused(lib):
    one = ctypes.c_int32()
    assert lib.qwen3_op_gemm_q8_plan(1, 16, 16, None, ctypes.byref(one)) == binding.QWEN3_E_INVALID
    assert lib.qwen3_op_gemv_w4_plan(1, 64, 32, 0, 8, None, None, None, None) == binding.QWEN3_E_INVALID
    assert "qwen3_op_gemv_w4_plan" in binding.qwen3_last_error(None)
