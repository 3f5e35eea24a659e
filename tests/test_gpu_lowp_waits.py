"""Failure detection of the kernels on 8-bit and 4-bit operands, without a fault: with a limit of one
cycle their bounded waits on copies and on the tensor cores give up for real.  Nothing traps or
hangs; every output is then what the call gives otherwise or NaN -- never what the buffer held
before -- and the next call with the default limit is right.
"""

import pytest
import torch

import gpu_common as gc
from qwen3_decoder_forward_gb300 import binding

F32, RESID, SWIGLU = binding.QWEN3_EPI_F32, binding.QWEN3_EPI_RESID_ADD, binding.QWEN3_EPI_SWIGLU
E4M3 = torch.float8_e4m3fn


@pytest.fixture
def limit():
    gc.ensure_library()
    yield binding.qwen3_op_set_wait_limit
    binding.qwen3_op_set_wait_limit(0)


def test_a_limit_is_a_number_of_cycles(limit):
    for bad in (-1, 2 ** 32):
        with pytest.raises(binding.Qwen3Error) as e:
            limit(bad)
        assert e.value.code == binding.QWEN3_E_INVALID
    limit(2 ** 32 - 1)
    limit(0)


def _codes(shape, seed):
    g = torch.Generator().manual_seed(seed)
    b = torch.randint(0, 256, shape, generator=g, dtype=torch.int32)
    return torch.where((b & 0x7F) == 0x7F, b - 1, b).to(torch.uint8).view(E4M3).cuda()


def _out(M, N, epi, base):
    if epi == RESID:
        return base.clone()
    return torch.full((M, N // 2 if epi == SWIGLU else N), 77.0, dtype=torch.bfloat16 if epi == SWIGLU else torch.float32,
                      device="cuda")


def _gives_up(call, M, N, epi, limit, before=lambda: None, surely=True):
    """call(out) with the default limit, then with one cycle and the default again, twice.  surely: a wait
    cannot but give up."""
    base = torch.randn(M, N, device="cuda") if epi == RESID else None
    want = call(_out(M, N, epi, base))
    assert bool(torch.isfinite(want).all())
    for _ in range(2):
        before()
        limit(1)
        got = call(_out(M, N, epi, base))
        torch.cuda.synchronize()
        nan = torch.isnan(got)
        assert bool(nan.any()) or not surely
        assert torch.equal(got[~nan], want[~nan])
        limit(0)
        assert torch.equal(call(_out(M, N, epi, base)), want)


# 256-wide pairs, 128-, 64- and 32-wide tiles of single CTAs, whole and with K shared by a cluster
@pytest.mark.gpu
@pytest.mark.parametrize("M,N,K", [(2100, 2064, 528), (4001, 1040, 2064), (23460, 1024, 144), (129, 6144, 1040), (300, 3600, 1040), (1, 6144, 144),
                                   (40, 272, 528), (40, 512, 2048), (3, 3600, 2048), (1, 512, 3856), (257, 512, 2048)])
@pytest.mark.parametrize("epi", [F32, RESID, SWIGLU])
def test_gemm_q8_wait_that_gives_up(M, N, K, epi, limit):
    xq, wq = _codes((M, K), M), _codes((N, K), N)
    xs, ws = torch.full((M,), 2.0 ** -9, device="cuda"), torch.full((N,), 2.0 ** -9, device="cuda")
    _gives_up(lambda out: binding.gemm_q8(xq, xs, wq, ws, epilogue=epi, out=out), M, N, epi, limit)


# rows stored by the warp that has their sums; shares joined in a CTA over several rounds of tiles, and in a
# cluster.  One row of x, so that it is staged before the first codes can be there (by a cluster, each of its
# share of the columns, they may be).
@pytest.mark.gpu
@pytest.mark.parametrize("M,N,K,group,zeros", [(1, 79454, 256, 64, True), (1, 79454, 1024, 64, False), (1, 20002, 8192, 128, False),
                                               (1, 1000, 8192, 64, True), (1, 2000, 65536, 128, False)])
@pytest.mark.parametrize("epi", [F32, RESID, SWIGLU])
def test_gemv_w4_wait_that_gives_up(M, N, K, group, zeros, epi, limit):
    g = torch.Generator().manual_seed(N)
    codes = torch.randint(0, 256, (N, K // 2), generator=g, dtype=torch.uint8).cuda()
    scales = torch.full((N, K // group), 2.0 ** -9, dtype=torch.bfloat16, device="cuda")
    zp = torch.randint(0, 16, (N, K // group), generator=g, dtype=torch.uint8).cuda() if zeros else None
    x = torch.randn(M, K, generator=g).bfloat16().cuda()
    flush = torch.empty(2 ** 28, dtype=torch.uint8, device="cuda")  # more than L2

    def cold():  # the weights out of L2, x in it: x is staged before the first codes can be there
        flush.fill_(1)
        x.clone()

    _gives_up(lambda out: binding.gemv_w4(x, codes, scales, group, zeros=zp, epilogue=epi, out=out), M, N, epi, limit, cold, surely=N > 2000)
