"""Edges of the single kernels on 8-bit and 4-bit operands: values far from 1, against their
definitions in 64 bits.

Tolerances: a projection's sums as in test_gpu_lowp.py, (K / 16 + 8) 2^-23 of the terms' magnitudes; a
rounding is half a step of its type.
"""

import pytest
import torch

import gpu_common as gc
from qwen3_decoder_forward_gb300 import binding

pytestmark = pytest.mark.gpu

F32, RESID, SWIGLU = binding.QWEN3_EPI_F32, binding.QWEN3_EPI_RESID_ADD, binding.QWEN3_EPI_SWIGLU
E4M3 = torch.float8_e4m3fn
BF16_HALF = torch.finfo(torch.bfloat16).eps / 2

# GEMM sizes (M, N, K) that run as pairs of CTAs, as single CTAs, and with K shared by a cluster
FORMS = [(4000, 3584, 128), (200, 512, 128), (40, 512, 2048)]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    gc.ensure_library()


def _gates():
    """Gates over the range in which silu leaves fp32's normal numbers, and ordinary ones."""
    return torch.cat([torch.linspace(-105, -80, 200, dtype=torch.float64), torch.linspace(-12, 100, 56, dtype=torch.float64)]).float()


def _check_swiglu(out, gate, up):
    """exp's error at |g| <= 105 is 126 ulp by CUDA's table (2 + 1.173 |g|), the division's and the products'
    a few: 2^-16 in all; a value below the normal numbers has steps of 2^-133 in bf16."""
    g, u = gate.double(), up.double()
    ref = g * torch.sigmoid(g) * u
    tol = (BF16_HALF + 2 ** -16) * ref.abs() + 2.0 ** -133
    # e^g itself is a subnormal of fp32 below -87.3, with steps of 2^-149, and so is a product with it
    tol = tol + 2.0 ** -149 * (g.abs() * u.abs() + u.abs() + 1)
    err = (out.double().cpu() - ref).abs()
    worst = int((err / tol).argmax())
    assert bool((err <= tol).all()), f"gate {float(g.flatten()[worst % g.numel()])}: error / tolerance {float((err / tol).max()):.3g}"


@pytest.mark.parametrize("M,N,K", FORMS)
@pytest.mark.parametrize("up", [1.0, -3e4, 1e30])
def test_gemm_q8_swiglu_over_the_range_of_gates(M, N, K, up):
    """One product of ones a row, so that gate and up are the weights' scales."""
    gates = _gates()
    xq, wq = torch.zeros(M, K), torch.zeros(N, K)
    xq[:, 1] = 1
    wq[:, 1] = 1
    gate = gates.repeat(N // 2 // gates.numel() + 1)[: N // 2]
    ws = torch.stack([gate, torch.full_like(gate, up)], dim=1).flatten()
    out = binding.gemm_q8(xq.to(E4M3).cuda(), torch.ones(M, device="cuda"), wq.to(E4M3).cuda(), ws.cuda(), epilogue=SWIGLU)
    assert torch.equal(out, out[:1].expand_as(out))
    _check_swiglu(out[0], gate, torch.full_like(gate, up))


@pytest.mark.parametrize("N,K", [(512, 128), (512, 4096), (40000, 128)])
@pytest.mark.parametrize("up", [1.0, 1e30])
def test_gemv_w4_swiglu_over_the_range_of_gates(N, K, up):
    """One weight of a row is its scale, the others zero: gate and up are bf16 scales."""
    gate = _gates().bfloat16().repeat(N // 512 + 1)[: N // 2]
    codes = torch.full((N, K // 2), 0x88, dtype=torch.uint8)
    codes[:, 0] = 0x89
    scales = torch.ones(N, K // 32, dtype=torch.bfloat16)
    scales[:, 0] = torch.stack([gate, torch.full_like(gate, up)], dim=1).flatten()
    x = torch.ones(3, K, dtype=torch.bfloat16)
    out = binding.gemv_w4(x.cuda(), codes.cuda(), scales.cuda(), 32, epilogue=SWIGLU)
    for row in out:
        _check_swiglu(row, gate, torch.full_like(gate, up).bfloat16())


@pytest.mark.parametrize("M,N,K", FORMS)
@pytest.mark.parametrize("epi", [F32, RESID])
def test_gemm_q8_scales_whose_product_leaves_fp32(M, N, K, epi):
    """Rows and weights far from 1: what counts is that the output is in range, not the scales' product."""
    g = torch.Generator().manual_seed(M)
    xq = torch.randint(0x70, 0x7F, (M, K), generator=g, dtype=torch.uint8).view(E4M3).cuda()  # 128 to 448
    wq = torch.randint(0x70, 0x7F, (N, K), generator=g, dtype=torch.uint8).view(E4M3).cuda()
    rows = [1.7 * 2.0 ** -80, 1.3 * 2.0 ** 90, 1.9, 1.1 * 2.0 ** -61, 1.5 * 2.0 ** -120, 1.2 * 2.0 ** 118, 2.0 ** -149, 0.0]
    cols = [1.1 * 2.0 ** -62, 1.9 * 2.0 ** -100, 1.3, 1.7 * 2.0 ** -80, 1.2 * 2.0 ** 40, 1.5 * 2.0 ** -20, 1.6 * 2.0 ** 100]
    xs = torch.tensor(rows).repeat(M // 8 + 1)[:M].cuda()
    ws = torch.tensor(cols).repeat(N // 7 + 1)[:N].cuda()
    a, b = xq.double(), wq.double()
    y = (a @ b.T) * xs.double()[:, None] * ws.double()[None, :]  # the terms are of one sign
    base = torch.randn(M, N, generator=g).cuda() if epi == RESID else None
    out = binding.gemm_q8(xq, xs, wq, ws, epilogue=epi, out=None if base is None else base.clone())
    ref = y if base is None else base.double() + y
    tol = (K / 16 + 10) * 2 ** -23 * y.abs() + 2 ** -23 * ref.abs() + 2.0 ** -148
    most = torch.finfo(torch.float32).max
    past = y.abs() > 1.01 * most  # none is nearer to it
    assert not bool(((y.abs() > 0.99 * most) ^ past).any())
    assert torch.equal(torch.isinf(out), past) and not bool(torch.isnan(out).any())
    err = (out.double() - ref).abs()
    assert bool((err <= tol)[~past].all()), f"error / tolerance {float((err / tol)[~past].max()):.3g}"


@pytest.mark.parametrize("M,N,K", FORMS)
def test_gemm_q8_a_zero_sum_stays_zero(M, N, K):
    """Scales whose product is past fp32's largest number, on rows whose products cancel or are zero."""
    xq, wq = torch.zeros(M, K), torch.zeros(N, K)
    xq[:, :2] = 1
    wq[:, 0], wq[:, 1] = 1, -1
    out = binding.gemm_q8(xq.to(E4M3).cuda(), torch.full((M,), 2.0 ** 90, device="cuda"), wq.to(E4M3).cuda(),
                          torch.full((N,), 2.0 ** 90, device="cuda"))
    assert not out.any()


@pytest.mark.parametrize("M,C", [(5, 16), (3, 1024), (700, 1040), (310, 4112), (2, 16384)])
@pytest.mark.parametrize("delta", [None, torch.bfloat16])
@pytest.mark.parametrize("eps", [0.0, 1e-38])
def test_add_rmsnorm_q8_rows_whose_squares_underflow(M, C, delta, eps):
    """Without an eps that carries them, the mean squares of tiny rows are below fp32's numbers."""
    g = torch.Generator().manual_seed(M + C)
    size = 10.0 ** -torch.linspace(0, 37, M)[torch.randperm(M, generator=g)]
    h = (torch.randn(M, C, generator=g) * size[:, None]).cuda()
    d = None if delta is None else (torch.randn(M, C, generator=g) * size[:, None]).to(delta).cuda()
    gain = (1 + 0.05 * torch.randn(C, generator=g)).cuda()
    h[M // 2] = 0
    if d is not None:
        d[M // 2] = 0
    want = h.clone() if d is None else h + d.float()
    q, s = binding.add_rmsnorm_q8(h, gain, eps, delta=d)
    assert torch.equal(h, want)
    hd = want.double()
    eps32 = float(torch.tensor(eps, dtype=torch.float32))
    y = hd / torch.sqrt(hd.pow(2).mean(dim=1, keepdim=True) + eps32) * gain.double()
    y[M // 2] = 0
    top = y.abs().amax(dim=1)
    assert bool(torch.isfinite(s).all())
    # as for ordinary rows, and h * gain may be a subnormal number: C terms of 2^-149 against the row's top
    lost = 2.0 ** -149 / (hd * gain.double()).abs().amax(dim=1).clamp(min=2.0 ** -149)
    live = top > 0
    assert float(((s.double() * 448 / top.where(live, torch.ones_like(top)) - 1).abs() - lost)[live].max()) <= 42 * 2 ** -24
    assert float(s[M // 2]) == 0.0 and not q[M // 2].float().any()


def _w4_reference(w, group, zeros):
    """The definition on the CPU: fp32 operations that IEEE rounds alike everywhere, the range of a group
    taken at a sixteenth of its size where it is past fp32."""
    N, K = w.shape
    g = w.cpu().float().view(N, K // group, group)
    lo, hi = g.amin(dim=2).clamp(max=0), g.amax(dim=2).clamp(min=0)
    if zeros:
        wide = torch.isinf(hi - lo)
        s = ((hi - lo) / torch.full_like(hi, 15)).where(~wide, (hi / 16 - lo / 16) / torch.full_like(hi, 15) * 16)
    else:
        s = g.abs().amax(dim=2) / torch.full_like(hi, 7)
    s = s.to(torch.bfloat16)
    div = torch.where(s.float() > 0, s.float(), torch.ones(()))
    z = torch.round(-lo / div).clamp(0, 15) if zeros else torch.full_like(div, 8)
    code = (torch.round(g / div[:, :, None]) + z[:, :, None]).clamp(0, 15).view(N, K).to(torch.uint8)
    return code, s, z.to(torch.uint8)


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("zeros", [False, True])
def test_quant_w4_groups_far_from_one(group, zeros):
    """Groups of every size a bf16 number has, subnormal ones and ranges past fp32's largest among them."""
    g = torch.Generator().manual_seed(group)
    N, K = 300, 4 * group
    power = torch.cat([torch.arange(-139, 129), torch.full((N - 268,), 128)]).double()
    w = (torch.rand(N, K, generator=g, dtype=torch.float64) * 2 - 1) * (2.0 ** power)[:, None] * 0.996
    w[:, 0], w[:, 1] = 0.99 * 2.0 ** power, -0.99 * 2.0 ** power
    w[:, group:2 * group] = w[:, group:2 * group].abs()
    w = w.to(torch.bfloat16)
    assert bool(torch.isfinite(w).all())
    codes, scales, zp = binding.quant_w4(w.cuda(), group, with_zeros=zeros)
    code, s, z = _w4_reference(w, group, zeros)
    c = codes.cpu()
    assert torch.equal(scales.cpu(), s)
    assert torch.equal(torch.stack([c & 15, c >> 4], dim=2).view(N, K), code)
    if zeros:
        assert torch.equal(zp.cpu(), z)


def test_tensors_written_in_place_are_marked_as_changed():
    """A tensor that autograd has saved and a call writes: the backward pass refuses it, as after torch's own calls.
    One that requires a gradient itself is refused at the call, and is left as it was."""
    h, gain, d = torch.ones(4, 64, device="cuda"), torch.ones(64, device="cuda"), torch.ones(4, 64, device="cuda")
    xq, xs = binding.quant_q8(h)
    wq, ws = binding.quant_q8(torch.ones(32, 64, device="cuda"))
    codes, scales, _ = binding.quant_w4(torch.ones(32, 64, device="cuda").bfloat16(), 32)
    x, out = h.bfloat16(), torch.zeros(4, 32, device="cuda")
    calls = {
        "h": (h, lambda t: binding.add_rmsnorm_q8(t, gain, 1e-6, delta=d)),
        "gemm out": (out, lambda t: binding.gemm_q8(xq, xs, wq, ws, epilogue=RESID, out=t)),
        "gemv out": (out, lambda t: binding.gemv_w4(x, codes, scales, 32, out=t)),
    }
    for name, (t, call) in calls.items():
        t = t.clone()
        leaf = torch.ones_like(t, requires_grad=True)
        y = (leaf * t).sum()  # saves t
        call(t)
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            y.backward()
        own = t.clone().requires_grad_()
        before = own.detach().clone()
        with pytest.raises(binding.Qwen3Error) as e:
            call(own)
        assert e.value.code == binding.QWEN3_E_INVALID and torch.equal(own.detach(), before), name
        with torch.no_grad():
            call(own)
        with torch.inference_mode():
            call(t.clone())
    version = h._version  # without an addend h is only read
    binding.add_rmsnorm_q8(h, gain, 1e-6)
    assert h._version == version
