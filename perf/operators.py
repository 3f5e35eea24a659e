"""Cases of the projections on 8-bit and 4-bit operands: the residual add with RMSNorm into 8-bit
rows, the row quantiser, the 8-bit GEMM, the 4-bit weight quantiser and the decode projection
on 4-bit weights.

Formats: 8-bit rows are e4m3 codes with one fp32 scale per row, value = code * scale.  4-bit
weights [N, K] are two codes to a byte (the even column in the low nibble), bf16 scales [N, K / G]
and zero points [N, K / G] (8 where there are none), value = scale * (code - zero).  Epilogues:
"f32" out = x W^T, "resid" out += x W^T, "swiglu" bf16 silu(gate) * up of rows 2j (gate), 2j + 1 (up).
"""

import math

import torch

own = False

EPS = 1e-6
Q8_MAX = 448.0  # the largest e4m3 value


def listed():
    return [
        # decode, one sequence: the QKV projection at hidden 1024 -- the smallest call, latency alone
        dict(name="gemv_w4 qkv 1 row", op="gemv_w4", M=1, K=1024, N=4096, G=128, zeros=False, x="bf16", epi="f32"),
        # batched decode of 32 sequences: gate_up + SwiGLU on rows that the norm left in 8 bits
        dict(name="gemv_w4 gate_up 32 rows", op="gemv_w4", M=32, K=1024, N=6144, G=64, zeros=True, x="e4m3", epi="swiglu"),
        # decode of a wide model: a down projection added into the residual, 13 rows
        dict(name="gemv_w4 down 13 rows", op="gemv_w4", M=13, K=10240, N=8192, G=128, zeros=False, x="bf16", epi="resid"),
        # a short prompt or a large decode batch: o_proj into the residual
        dict(name="gemm_q8 o_proj 33 rows", op="gemm_q8", M=33, K=2048, N=1024, epi="resid"),
        # the packed ragged prefill (8 sequences, 23,460 tokens): gate_up + SwiGLU
        dict(name="gemm_q8 gate_up 23460 rows", op="gemm_q8", M=23460, K=1024, N=6144, epi="swiglu"),
        # the largest: a projection of a wide model over 8,191 tokens
        dict(name="gemm_q8 wide 8191 rows", op="gemm_q8", M=8191, K=8192, N=7168, epi="f32"),
        # decode of 5 sequences: the norm between attention and MLP
        dict(name="add_rmsnorm_q8 5 rows", op="add_rmsnorm_q8", M=5, C=1024, d="f32"),
        # the same over the packed prefill
        dict(name="add_rmsnorm_q8 23460 rows", op="add_rmsnorm_q8", M=23460, C=1024, d="bf16"),
        # a chunk of rows of a wide MLP's activation
        dict(name="quant_q8 77 rows", op="quant_q8", M=77, K=14336, x="f32"),
        # the packed prefill's attention output before o_proj
        dict(name="quant_q8 23460 rows", op="quant_q8", M=23460, K=2048, x="bf16"),
        # one layer's gate_up weights
        dict(name="quant_w4 gate_up", op="quant_w4", N=6144, K=1024, G=128, zeros=False),
        # the head: vocabulary x hidden, fine groups with zero points
        dict(name="quant_w4 head", op="quant_w4", N=151936, K=1024, G=32, zeros=True),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["gemv_w4", "gemv_w4", "gemm_q8", "gemm_q8", "add_rmsnorm_q8", "quant_q8", "quant_w4"])
    weights = 151936 * 1024
    if op == "gemv_w4":
        G, epi = rng.choice([32, 64, 128]), rng.choice(["f32", "resid", "swiglu"])
        K = G * _log_int(rng, 1, 16384 // G)
        N = _log_int(rng, 2, min(151936, weights // K))
        N -= N % 2 if epi == "swiglu" else 0
        return dict(op=op, M=_log_int(rng, 1, 32), K=K, N=N, G=G, zeros=rng.random() < 0.5,
                    x=rng.choice(["bf16", "e4m3"]), epi=epi)
    if op == "gemm_q8":
        return dict(op=op, M=_log_int(rng, 1, 8191), K=16 * _log_int(rng, 1, 512), N=16 * _log_int(rng, 1, 448),
                    epi=rng.choice(["f32", "resid", "swiglu"]))
    if op == "add_rmsnorm_q8":
        C = 16 * _log_int(rng, 2, 1024)
        return dict(op=op, M=_log_int(rng, 1, min(65536, 23460 * 1024 // C)), C=C, d=rng.choice(["f32", "bf16", "none"]))
    if op == "quant_q8":
        K = 16 * _log_int(rng, 1, 1024)
        return dict(op=op, M=_log_int(rng, 1, min(65536, 23460 * 2048 // K)), K=K, x=rng.choice(["f32", "bf16"]))
    G = rng.choice([32, 64, 128])
    K = G * _log_int(rng, 1, 16384 // G)
    return dict(op=op, N=_log_int(rng, 1, weights // K), K=K, G=G, zeros=rng.random() < 0.5)


# ---- inputs ---------------------------------------------------------------------------------


def _q8(y):
    """Rows of y (fp32) in 8 bits: e4m3 codes and the scale of each row."""
    amax = y.abs().amax(dim=1, keepdim=True)
    scale = amax / Q8_MAX
    q = torch.where(amax > 0, y / scale, torch.zeros_like(y))
    return q.to(torch.float8_e4m3fn), scale[:, 0]


def _w4(w, G, zeros):
    """Codes, scales and zero points (None: 8) of w [N, K] in groups of G columns."""
    N, K = w.shape
    g = w.float().view(N, K // G, G)
    if zeros:
        lo, hi = g.amin(dim=2).clamp(max=0.0), g.amax(dim=2).clamp(min=0.0)
        scale = ((hi - lo) / 15.0).to(torch.bfloat16)
    else:
        scale = (g.abs().amax(dim=2) / 7.0).to(torch.bfloat16)
    s = scale.float()
    one = torch.where(s > 0, s, torch.ones_like(s))
    zp = torch.round(-lo / one).clamp(0, 15) if zeros else torch.full_like(s, 8.0)
    code = (torch.round(g / one[:, :, None]) + zp[:, :, None]).clamp(0, 15).to(torch.uint8).view(N, K)
    return code[:, 0::2] | (code[:, 1::2] << 4), scale, zp.to(torch.uint8) if zeros else None


def _normal(gen, shape, dtype=torch.float32, scale=1.0):
    return (torch.randn(shape, generator=gen, device="cuda") * scale).to(dtype)


_F = {"f32": torch.float32, "bf16": torch.bfloat16}


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op = case["op"]
    s = dict(case)
    if op in ("gemv_w4", "gemm_q8"):
        M, K, N = case["M"], case["K"], case["N"]
        x = _normal(gen, (M, K), torch.bfloat16)
        # weights with the spread over output rows that trained projections have
        w = _normal(gen, (N, K), torch.bfloat16, 0.02) * _normal(gen, (N, 1)).exp().sqrt().to(torch.bfloat16)
        if op == "gemv_w4":
            s["codes"], s["scales"], s["zp"] = _w4(w, case["G"], case["zeros"])
            s["xs"] = None
            s["xq"] = x
            if case["x"] == "e4m3":
                s["xq"], s["xs"] = _q8(x.float())
        else:
            s["xq"], s["xs"] = _q8(x.float())
            s["wq"], s["ws"] = _q8(w.float())
        s["out"] = _normal(gen, (M, N)) if case["epi"] == "resid" else None
    elif op == "add_rmsnorm_q8":
        M, C = case["M"], case["C"]
        # a residual stream: a few channels are an order of magnitude larger than the rest
        s["h"] = _normal(gen, (M, C)) * (1.0 + 9.0 * (torch.rand(C, generator=gen, device="cuda") < 0.01))
        s["delta"] = None if case["d"] == "none" else _normal(gen, (M, C), _F[case["d"]])
        s["gain"] = 1.0 + _normal(gen, (C,), scale=0.05)
    elif op == "quant_q8":
        s["xin"] = _normal(gen, (case["M"], case["K"]), _F[case["x"]])
    else:
        s["w"] = _normal(gen, (case["N"], case["K"]), torch.bfloat16, 0.02)
    return s


# ---- the operators, plain and the framework's -----------------------------------------------


def _unpack_w4(codes, scales, zp, G):
    N, K = codes.shape[0], codes.shape[1] * 2
    q = torch.stack([codes & 15, codes >> 4], dim=2).view(N, K // G, G).float()
    q = q - (8.0 if zp is None else zp.float()[:, :, None])
    return (q * scales.float()[:, :, None]).view(N, K)


def _finish(y, epi, out):
    if epi == "resid":
        out += y
        return out
    if epi == "swiglu":
        g, u = y[:, 0::2], y[:, 1::2]
        return (g / (1.0 + torch.exp(-g)) * u).to(torch.bfloat16)
    return y


def _plain(s):
    op = s["op"]
    if op == "gemv_w4":
        x = s["xq"].float()
        if s["xs"] is not None:
            x = x * s["xs"][:, None]
        return _finish(x @ _unpack_w4(s["codes"], s["scales"], s["zp"], s["G"]).T, s["epi"], s["out"])
    if op == "gemm_q8":
        x, w = s["xq"].float() * s["xs"][:, None], s["wq"].float() * s["ws"][:, None]
        return _finish(x @ w.T, s["epi"], s["out"])
    if op == "add_rmsnorm_q8":
        h = s["h"]
        if s["delta"] is not None:
            h += s["delta"].float()
        y = h * torch.rsqrt((h * h).mean(dim=1, keepdim=True) + EPS) * s["gain"]
        return (h, *_q8(y))
    if op == "quant_q8":
        return _q8(s["xin"].float())
    return _w4(s["w"], s["G"], s["zeros"])


_lib = None


def _binding():
    global _lib
    if _lib is None:
        from qwen3_decoder_forward_gb300 import binding as _lib
    return _lib


_EPI = {"f32": 0, "resid": 1, "swiglu": 2}  # QWEN3_EPI_*


def _framework(s):
    b = _lib or _binding()
    op = s["op"]
    if op == "gemv_w4":
        return b.gemv_w4(s["xq"], s["codes"], s["scales"], s["G"], zeros=s["zp"], x_scale=s["xs"],
                         epilogue=_EPI[s["epi"]], out=s["out"])
    if op == "gemm_q8":
        return b.gemm_q8(s["xq"], s["xs"], s["wq"], s["ws"], epilogue=_EPI[s["epi"]], out=s["out"])
    if op == "add_rmsnorm_q8":
        return (s["h"], *b.add_rmsnorm_q8(s["h"], s["gain"], EPS, delta=s["delta"]))
    if op == "quant_q8":
        return b.quant_q8(s["xin"])
    return b.quant_w4(s["w"], s["G"], with_zeros=s["zeros"])


def run(state):
    if own:
        return _framework(state)
    return _plain(state)


def work(case):
    op = case["op"]
    if op in ("gemv_w4", "gemm_q8"):
        M, K, N = case["M"], case["K"], case["N"]
        out = {"f32": 4, "resid": 8, "swiglu": 1}[case["epi"]] * M * N
        if op == "gemv_w4":
            G = case["G"]
            w = N * K // 2 + N * (K // G) * (3 if case["zeros"] else 2)
            x = M * K * 2 if case["x"] == "bf16" else M * K + 4 * M
        else:
            w, x = N * K + 4 * N, M * K + 4 * M
        return {"bytes": w + x + out, "flops": 2 * M * N * K}
    if op == "add_rmsnorm_q8":
        M, C = case["M"], case["C"]
        d = {"f32": 4 + 4, "bf16": 4 + 2, "none": 0}[case["d"]]  # the sum written back, the addend read
        return {"bytes": M * C * (4 + d + 1) + 4 * M + 4 * C, "flops": 6 * M * C}
    if op == "quant_q8":
        M, K = case["M"], case["K"]
        return {"bytes": M * K * ((4 if case["x"] == "f32" else 2) + 1) + 4 * M, "flops": 3 * M * K}
    N, K, G = case["N"], case["K"], case["G"]
    return {"bytes": N * K * 2 + N * K // 2 + N * (K // G) * (3 if case["zeros"] else 2), "flops": 4 * N * K}


# ---- the definitions in 64 bits -------------------------------------------------------------


def _nearest_e4m3(v):
    """v (float64) rounded to the nearest e4m3 value, ties to even, saturating at 448."""
    _, e = torch.frexp(v)  # |v| in [2^(e-1), 2^e)
    step = torch.ldexp(torch.ones_like(v), (e - 1).clamp(min=-6) - 3)
    return (torch.round(v / step) * step).clamp(-Q8_MAX, Q8_MAX)


def _rows_e4m3(y):
    top = y.abs().max(dim=1).values
    share = Q8_MAX / torch.where(top > 0, top, torch.ones_like(top))
    return _nearest_e4m3(y * share.unsqueeze(1)), top / Q8_MAX


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "quant_w4":  # whole numbers but for the scales
        g = s["w"].double().unflatten(1, (-1, case["G"]))
        if case["zeros"]:
            span = torch.relu(g.max(dim=2).values) + torch.relu(-g.min(dim=2).values)
            return None, span / 15, None
        return None, g.abs().max(dim=2).values / 7, None
    if op == "quant_q8":
        return _rows_e4m3(s["xin"].double())
    if op == "add_rmsnorm_q8":
        h = s["h"].double()
        if s["delta"] is not None:
            h = h + s["delta"].double()
        norm = torch.sqrt(h.pow(2).sum(dim=1) / h.shape[1] + EPS)
        return (h, *_rows_e4m3(h / norm.unsqueeze(1) * s["gain"].double()))
    x = s["xq"].to(torch.float32).double()
    if s["xs"] is not None:
        x = torch.einsum("mk,m->mk", x, s["xs"].double())
    if op == "gemm_q8":
        w = torch.einsum("nk,n->nk", s["wq"].to(torch.float32).double(), s["ws"].double())
    else:
        N, K, G = case["N"], case["K"], case["G"]
        w = torch.empty(N, K, dtype=torch.float64, device=x.device)
        w[:, 0::2] = (s["codes"] % 16).double()
        w[:, 1::2] = torch.div(s["codes"], 16, rounding_mode="floor").double()
        zero = torch.full((N, K // G), 8.0, dtype=torch.float64, device=x.device) if s["zp"] is None else s["zp"].double()
        w = (w.unflatten(1, (-1, G)) - zero.unsqueeze(2)).mul_(s["scales"].double().unsqueeze(2)).flatten(1)
    y = torch.einsum("mk,nk->mn", x, w)
    if case["epi"] == "resid":
        return s["out"].double() + y
    if case["epi"] == "swiglu":
        gate, up = y.unflatten(1, (-1, 2)).unbind(2)
        return gate * torch.sigmoid(gate) * up
    return y
