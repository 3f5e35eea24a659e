"""Every form that the projections on 8-bit and 4-bit operands choose between, against 64 bits: the sizes are checked to
reach the form that they stand for.  Tolerances as in test_gpu_lowp.py, whose checks these are."""

import pytest
import torch

import gpu_common as gc
from qwen3_decoder_forward_gb300 import binding
from test_gpu_lowp import F32, RESID, SWIGLU, _check, _codes, _out, _rand, _w4

pytestmark = pytest.mark.gpu

# (columns of a tile, CTAs sharing K): M, K, N with ragged ends
GEMM = {
    (256, 1): (4001, 272, 1040), (128, 1): (129, 1040, 6144), (128, 2): (1, 3856, 6144), (128, 4): (3, 2064, 3600),
    (128, 8): (3, 3856, 1040), (64, 1): (1, 144, 6144), (64, 2): (257, 3856, 1008), (64, 4): (40, 2064, 2064),
    (64, 8): (1, 2064, 512), (32, 1): (3, 144, 48), (32, 2): (129, 2064, 1008), (32, 4): (40, 2064, 512), (32, 8): (1, 2064, 16),
}
# single CTAs that go through several tiles, with 128, 64 and 32 columns
ROUNDS = {(128, 1): (2100, 528, 2064), (64, 1): (1, 128, 20240), (32, 1): (20, 128, 10160)}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    gc.ensure_library()


@pytest.mark.parametrize("form,size", [*GEMM.items(), *ROUNDS.items()])
@pytest.mark.parametrize("epi", [F32, RESID, SWIGLU])
def test_gemm_q8_form(form, size, epi):
    M, K, N = size
    assert binding.qwen3_op_gemm_q8_plan(M, K, N) == form
    xq, wq = _codes((M, K), M + K), _codes((N, K), N + K)
    xs, ws = _rand((M,), 5).abs() * 1e-3 + 1e-4, _rand((N,), 6).abs() * 1e-4 + 1e-5
    out, intact, base = _out(M, N, epi, 7)
    again = out.clone()
    binding.gemm_q8(xq, xs, wq, ws, epilogue=epi, out=out)
    binding.gemm_q8(xq, xs, wq, ws, epilogue=epi, out=again)
    a, b = xq.double() * xs.double()[:, None], wq.double() * ws.double()[:, None]
    _check(out, a @ b.T, a.abs() @ b.abs().T, K, epi, base)
    assert intact() and torch.equal(out, again)


# rounds of tiles: joined by no one, in a CTA, in a cluster, in both; 1 to 8, 9 to 16 and 17 to 32 rows of x
GEMV = [(1, 256, 79454, 64), (9, 256, 79454, 64), (20, 256, 40002, 64), (1, 8192, 20002, 128), (9, 448, 79454, 64),
        (16, 4096, 20002, 128), (20, 448, 40002, 64), (16, 8192, 14338, 64), (9, 8192, 20002, 64), (32, 2048, 20002, 64),
        (32, 4096, 12290, 128), (32, 4096, 14338, 128), (32, 8192, 8192, 64)]


def test_gemv_w4_sizes_reach_every_join():
    joins = set()
    for M, K, N, group in GEMV:
        warps, shares, cluster, rounds = binding.qwen3_op_gemv_w4_plan(M, K, group, (M + N // 2) % 2 == 1, N)
        assert rounds > 1, (M, K, N)
        joins.add((1 if M <= 8 else 2 if M <= 16 else 4, shares > 1, cluster > 1))
    assert joins >= {(t, shares, False) for t in (1, 2, 4) for shares in (False, True)}
    assert joins >= {(2, True, True), (4, True, True), (4, False, True)}


@pytest.mark.parametrize("M,K,N,group", GEMV)
@pytest.mark.parametrize("epi", [F32, RESID, SWIGLU])
def test_gemv_w4_rounds_of_tiles(M, K, N, group, epi):
    zeros, x8 = (M + N // 2) % 2 == 1, (M + K // group) % 2 == 1
    codes, scales, zp, w = _w4(N, K, group, zeros, M + K + N)
    x, xs = (_codes((M, K), 4), _rand((M,), 5).abs() * 1e-2 + 1e-3) if x8 else (_rand((M, K), 4, torch.bfloat16), None)
    xd = x.double() * xs.double()[:, None] if x8 else x.double()
    out, intact, base = _out(M, N, epi, 9)
    again = out.clone()
    binding.gemv_w4(x, codes, scales, group, zeros=zp, x_scale=xs, epilogue=epi, out=out)
    binding.gemv_w4(x, codes, scales, group, zeros=zp, x_scale=xs, epilogue=epi, out=again)
    _check(out, xd @ w.T, xd.abs() @ w.abs().T, K, epi, base)
    assert intact() and torch.equal(out, again)
