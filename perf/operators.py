"""Workloads of the microscaled (MX) operators: the root-mean-square norm with an 8-bit output, the
quantization of activations and weights, and the product on quantized operands.

``run`` makes one pass.  With ``own`` false it computes the operator's formula with elementary
torch operations; with ``own`` true it calls the library.  Both read the same inputs in the same
layouts, so their outputs can be compared value by value.

Formats.  A block is 32 consecutive input channels.  Its scale is a power of two, stored as the
byte E that stands for 2^(E - 127), with E = max(biased exponent of max|p| - e_max, 0); its
elements are p / 2^(E - 127) rounded to nearest even and saturated, as e4m3 (8 bits, e_max = 8) or
as e2m1 (4 bits, e_max = 2).  E = 255 marks a block that holds an infinity or a NaN.

Layouts (Kb = K / 32 rounded up to a multiple of 4, Nt = ceil(N / 64)):
  activations  codes e4m3 [M, K], or uint8 [M, K/2] with channel 2i in the low half of byte i;
               scales [M, K/32]
  weights      codes uint8 [Nt, Kb, 64, 16] (16 bytes: the 32 channels of one block of one column,
               low half first); scales [Nt, Kb, 64], where byte 4i + j belongs to column 16j + i of
               the tile; blocks past K and columns past N are zero
"""
import math

import torch

own = False

BLOCK = 32
EMAX = {8: 8, 4: 2}
LARGEST = {8: 448.0, 4: 6.0}


# ---------------------------------------------------------------- cases
def listed():
    return [
        # one decoded token through the norm in front of q|k|v
        dict(name="norm_decode", op="norm", M=1, K=8192, residual=True, scaled=False, y=False, codes=True),
        # a prefill chunk, with the input scales of an AWQ search folded into the output
        dict(name="norm_prefill", op="norm", M=4096, K=8192, residual=True, scaled=True, y=False, codes=True),
        # a ragged batch whose norm feeds a 4-bit integer layer (bf16) and an MX one (8 bits)
        dict(name="norm_ragged", op="norm", M=333, K=5120, residual=False, scaled=True, y=True, codes=True),
        # offline: the square layer packed and read back to score its error
        dict(name="pack_square", op="pack", K=4096, N=4096, scaled=False),
        # offline: the widest layer of the 70B-shaped block, with its input scales
        dict(name="pack_wide", op="pack", K=8192, N=28672, scaled=True),
        # a small decode batch in front of down: silu(gate) * up into 8 bits
        dict(name="quantize_decode", op="quantize", M=16, K=28672, gate=True, scaled=True),
        # the same on a prefill chunk of the 11008-channel layer
        dict(name="quantize_prefill", op="quantize", M=8192, K=11008, gate=True, scaled=False),
        # one token through the fused q|k|v projection: latency and weight traffic
        dict(name="product_decode", op="product", M=1, K=8192, N=10240, bits=8),
        # an odd decode batch through down: weight traffic
        dict(name="product_batch", op="product", M=13, K=28672, N=8192, bits=8),
        # a short ragged prompt from bf16 activations, quantized to 4 bits on the way
        dict(name="linear_short", op="linear", M=257, K=5120, N=13824, bits=4),
        # prefill through gate or up with 8-bit activations, through down with 4-bit ones
        dict(name="product_prefill8", op="product", M=4096, K=8192, N=28672, bits=8),
        dict(name="product_prefill4", op="product", M=4096, K=28672, N=8192, bits=4),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "pack", "quantize", "product", "product", "linear"])
    K = BLOCK * _log(rng, 16, 896)
    if op == "pack":
        N = _log(rng, 200, 28672)
        return dict(op=op, K=K, N=min(N, 8192 * 28672 // K), scaled=rng.random() < 0.5)
    if op in ("norm", "quantize"):
        M = min(_log(rng, 1, 8192), 4096 * 8192 // K)
        if op == "quantize":
            return dict(op=op, M=M, K=K, gate=rng.random() < 0.5, scaled=rng.random() < 0.5)
        form = rng.choice(["codes", "y", "both"])
        return dict(op=op, M=M, K=K, residual=rng.random() < 0.5, scaled=form != "y" and rng.random() < 0.5,
                    y=form != "codes", codes=form != "y")
    M, N = _log(rng, 1, 4096), 8 * _log(rng, 16, 3584)
    N = max(8, min(N, 8192 * 28672 // K // 8 * 8))
    return dict(op=op, M=M, K=K, N=N, bits=rng.choice([4, 8]))


def _kb(K):
    return -(-K // (4 * BLOCK)) * 4


def work(case):
    K = case["K"]
    if case["op"] == "pack":
        n = K * case["N"]
        packed = n // 2 + n // BLOCK
        return {"bytes": 2 * (2 * n + packed) + (8 * K if case["scaled"] else 0), "flops": 4 * n}
    M = case["M"]
    n = M * K
    if case["op"] == "norm":
        b = 2 * n + 2 * K + (4 * K if case["scaled"] else 0) + (4 * n if case["residual"] else 0)
        b += (2 * n if case["y"] else 0) + (n + n // BLOCK if case["codes"] else 0)
        return {"bytes": b, "flops": 8 * n}
    if case["op"] == "quantize":
        b = 2 * n * (2 if case["gate"] else 1) + (4 * K if case["scaled"] else 0) + n + n // BLOCK
        return {"bytes": b, "flops": (10 if case["gate"] else 4) * n}
    N = case["N"]
    weights = K * N // 2 + K * N // BLOCK
    acts = 2 * n if case["op"] == "linear" else n * case["bits"] // 8 + n // BLOCK
    return {"bytes": acts + weights + 2 * M * N, "flops": 2 * M * N * K}


# ---------------------------------------------------------------- the formats, in 32 bits
def _scale_and_codes(p, bits):
    """p float32 [..., K] -> (E uint8 [..., K/32], p / 2^(E-127) float32 [..., K/32, 32], zero in a
    block that holds an infinity or a NaN)."""
    blocks = p.unflatten(-1, (-1, BLOCK))
    e = (blocks.abs().amax(-1).view(torch.int32) >> 23) & 255
    E = torch.where(e == 255, e, (e - EMAX[bits]).clamp_min(0))
    step = ((254 - E).clamp(1, 254) << 23).view(torch.float32)      # 2^(127 - E)
    q = torch.where((e == 255)[..., None], torch.zeros_like(blocks), blocks * step[..., None])
    return E.to(torch.uint8), q


def _e4m3(q):
    return q.clamp(-448.0, 448.0).to(torch.float8_e4m3fn).flatten(-2)


def _e2m1(q):
    """4-bit codes (uint8, not yet paired): sign, then the index among 0, .5, 1, 1.5, 2, 3, 4, 6."""
    a = q.abs()
    c = torch.signbit(q).to(torch.uint8) * 8
    for half, inclusive in ((0.25, 0), (0.75, 1), (1.25, 0), (1.75, 1), (2.5, 0), (3.5, 1), (5.0, 0)):
        c += (a >= half) if inclusive else (a > half)
    return c.flatten(-2)


def _pair(c):
    return c[..., 0::2] | (c[..., 1::2] << 4)


def _values4(b):
    """uint8 pairs [..., n] -> float32 [..., 2n]."""
    c = torch.stack((b & 15, b >> 4), -1).flatten(-2).to(torch.int32)
    exponent, mantissa = (c >> 1) & 3, (c & 1).float()
    a = torch.where(exponent == 0, 0.5 * mantissa, (1.0 + 0.5 * mantissa) * torch.exp2((exponent - 1).float()))
    return torch.where(c >= 8, -a, a)


def _steps(E):
    """2^(E - 127) as float32; NaN where E = 255."""
    v = torch.ldexp(torch.ones((), device=E.device), E.to(torch.int32) - 127)
    return torch.where(E == 255, torch.full_like(v, math.nan), v)


def _pack_weights(W, s):
    """W bf16 [K, N] -> codes, scales in the layout of the weights."""
    K, N = W.shape
    p = W.float() if s is None else W.float() * s[:, None]
    E, q = _scale_and_codes(p.t().contiguous(), 4)
    c = _pair(_e2m1(q)).unflatten(-1, (-1, 16))                         # [N, K/32, 16]
    Nt, Kb = -(-N // 64), _kb(K)
    codes = torch.zeros((Nt * 64, Kb, 16), dtype=torch.uint8, device=W.device)
    scales = torch.zeros((Nt * 64, Kb), dtype=torch.uint8, device=W.device)
    codes[:N, :K // BLOCK], scales[:N, :K // BLOCK] = c, E
    codes = codes.view(Nt, 64, Kb, 16).transpose(1, 2).contiguous()
    scales = scales.view(Nt, 4, 16, Kb).permute(0, 3, 2, 1).reshape(Nt, Kb, 64).contiguous()
    return codes, scales


def _weights(codes, scales, K, N):
    """The values that packed weights stand for, float32 [K, N]."""
    Nt, Kb = scales.shape[:2]
    v = _values4(codes) * _steps(scales).view(Nt, Kb, 16, 4).transpose(2, 3).reshape(Nt, Kb, 64, 1)
    return v.permute(1, 3, 0, 2).reshape(Kb * BLOCK, Nt * 64)[:K, :N]


def _acts(codes, scales):
    v = codes.float() if codes.dtype == torch.float8_e4m3fn else _values4(codes)
    return (v.unflatten(-1, (-1, BLOCK)) * _steps(scales.view(torch.uint8))[..., None]).flatten(-2)


# ---------------------------------------------------------------- inputs
def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    def acts(M, K):
        """Activations with one channel in a hundred 50 times larger."""
        gain = torch.where(torch.rand(K, generator=g, device="cuda") < 0.01, 50.0, 1.0)
        return (normal(M, K) * gain).to(torch.bfloat16)

    def buffer(*shape, dtype=torch.uint8):
        return torch.zeros(shape, dtype=dtype, device="cuda")

    K, op = case["K"], case["op"]
    st = dict(case=dict(case), s=torch.exp(normal(K)) if case.get("scaled") else None)
    if op == "pack":
        N = case["N"]
        st["W"] = (normal(K, N) / math.sqrt(K)).to(torch.bfloat16)
        st["codes"], st["scales"] = buffer(-(-N // 64), _kb(K), 64, 16), buffer(-(-N // 64), _kb(K), 64)
        st["back"] = buffer(K, N, dtype=torch.bfloat16)
        return st
    M = case["M"]
    if op in ("norm", "quantize", "linear"):
        st["X"] = acts(M, K)
        bits = case.get("bits", 8)
        if op != "norm" or case["codes"]:
            st["codes"] = buffer(M, K, dtype=torch.float8_e4m3fn) if bits == 8 else buffer(M, K // 2)
            st["scales"] = buffer(M, K // BLOCK, dtype=torch.float8_e8m0fnu)
    if op == "norm":
        st["weight"] = (1 + 0.1 * normal(K)).to(torch.bfloat16)
        st["residual"] = acts(M, K) if case["residual"] else None
        st["residual_out"] = buffer(M, K, dtype=torch.bfloat16) if case["residual"] else None
        st["Y"] = buffer(M, K, dtype=torch.bfloat16) if case["y"] else None
    if op == "quantize":
        st["gate"] = normal(M, K).to(torch.bfloat16) if case["gate"] else None
    if op in ("product", "linear"):
        N, bits = case["N"], case["bits"]
        st["wcodes"], st["wscales"] = _pack_weights((normal(K, N) / math.sqrt(K)).to(torch.bfloat16), None)
        st["Y"] = buffer(M, N, dtype=torch.bfloat16)
        if op == "product":
            E, q = _scale_and_codes(acts(M, K).float(), bits)
            st["codes"] = _e4m3(q) if bits == 8 else _pair(_e2m1(q)).contiguous()
            st["scales"] = E.view(torch.float8_e8m0fnu)
        if own:
            from weight_only_int4_act_amd import awq
            st["ws"] = awq.workspace(awq.awq_mx_gemm_workspace_size(M, K, N, bits), "cuda")
    return st


EPS = 1e-5


# ---------------------------------------------------------------- one pass
def run(st):
    return _run_own(st) if own else _run_plain(st)


def _run_own(st):
    from weight_only_int4_act_amd import awq
    op = st["case"]["op"]
    if op == "pack":
        awq.awq_mx_pack(st["W"], st["s"], st["codes"], st["scales"])
        awq.awq_mx_unpack(st["codes"], st["scales"], st["s"], st["back"])
        return st["back"]
    if op == "norm":
        awq.awq_rms_norm(st["X"], st["residual"], st["weight"], EPS, st["residual_out"], st["Y"], st["s"],
                         st.get("codes"), st.get("scales"))
        return {k: st[k] for k in ("residual_out", "Y", "codes", "scales") if st.get(k) is not None}
    if op in ("quantize", "linear"):
        awq.awq_mx_quantize(st["X"], st.get("gate"), st["s"], st["codes"], st["scales"])
        if op == "quantize":
            return {"codes": st["codes"], "scales": st["scales"]}
    awq.awq_mx_gemm(st["codes"], st["scales"], st["wcodes"], st["wscales"], st["Y"], st["ws"])
    return st["Y"]


def _run_plain(st):
    case = st["case"]
    op, s = case["op"], st["s"]
    if op == "pack":
        v = _weights(*_pack_weights(st["W"], s), case["K"], case["N"])
        return (v if s is None else v / s[:, None]).to(torch.bfloat16)
    if op == "norm":
        h, out = st["X"].float(), {}
        if case["residual"]:
            h = h + st["residual"].float()
            out["residual_out"] = h.to(torch.bfloat16)
        mean = h.double().square().mean(-1, keepdim=True)
        y = h * torch.rsqrt(mean + EPS).float() * st["weight"].float()
        if case["y"]:
            out["Y"] = y.to(torch.bfloat16)
        if case["codes"]:
            E, q = _scale_and_codes(y if s is None else y / s, 8)
            out["codes"], out["scales"] = _e4m3(q), E.view(torch.float8_e8m0fnu)
        return out
    if op == "product":
        x = _acts(st["codes"], st["scales"])
    else:
        p = st["X"].float()
        if case.get("gate"):
            gate = st["gate"].float()
            p = gate / (1 + torch.exp(-gate)) * p
        E, q = _scale_and_codes(p if s is None else p / s, case.get("bits", 8))
        if op == "quantize":
            return {"codes": _e4m3(q), "scales": E.view(torch.float8_e8m0fnu)}
        x = _acts(_pair(_e2m1(q)) if case["bits"] == 4 else _e4m3(q), E)
    return (x @ _weights(st["wcodes"], st["wscales"], case["K"], case["N"])).to(torch.bfloat16)


# ---------------------------------------------------------------- the definition, in 64 bits
def _exact_round(p, bits, rounded=True):
    """float64 [R, K] -> the scaled elements (float64 [R, K]) and the blocks' power-of-two scales
    [R, K/32, 1].  Not rounded: the number that a code stands for before its rounding, which does not jump
    where a value lies next to the border of two codes."""
    b = p.reshape(p.shape[0], -1, BLOCK)
    top = torch.linalg.vector_norm(b, ord=math.inf, dim=-1, keepdim=True)
    exponent = torch.frexp(top).exponent.double() - 1 - EMAX[bits]
    scale = torch.exp2(torch.where(top > 0, exponent, torch.full_like(exponent, -127.0)).clamp_min(-127))
    v = (b / scale).clamp(-LARGEST[bits], LARGEST[bits])
    if rounded:
        mantissa, least = (3, -6) if bits == 8 else (1, 0)
        grid = torch.exp2((torch.frexp(v).exponent.double() - 1).clamp_min(least) - mantissa)
        v = torch.round(v / grid) * grid
    return v.reshape(p.shape), scale


def _exact_values4(b):
    table = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6], dtype=torch.float64,
                         device=b.device)
    i = b.long()
    out = torch.empty(b.shape[:-1] + (2 * b.shape[-1],), dtype=torch.float64, device=b.device)
    out[..., 0::2], out[..., 1::2] = table[i % 16], table[i // 16]
    return out


def _exact_weights(st):
    K, N = st["case"]["K"], st["case"]["N"]
    W = torch.empty((K, N), dtype=torch.float64, device="cuda")
    for t in range(st["wcodes"].shape[0]):
        v = _exact_values4(st["wcodes"][t].transpose(0, 1).reshape(64, -1))[:, :K]         # [64, K]
        E = st["wscales"][t].double()                                                      # [Kb, 64]
        column = torch.arange(64, device="cuda")
        E = E[:, 4 * (column % 16) + column // 16].t()                                     # [64, Kb]
        v = v * torch.exp2(E - 127).repeat_interleave(BLOCK, 1)[:, :K]
        n = min(64, N - 64 * t)
        W[:, 64 * t:64 * t + n] = v[:n].t()
    return W


def exact(case, seed):
    st = prepare(case, seed)
    op, s = case["op"], st["s"]
    s = None if s is None else s.double()
    if op == "pack":
        W = st["W"].double()
        out = torch.empty_like(W)
        for c in range(0, case["N"], 1024):
            p = W[:, c:c + 1024] if s is None else W[:, c:c + 1024] * s[:, None]
            v, scale = _exact_round(p.t().contiguous(), 4)
            v = (v.reshape(v.shape[0], -1, BLOCK) * scale).reshape(v.shape).t()
            out[:, c:c + 1024] = v if s is None else v / s[:, None]
        return out
    if op == "norm":
        h = st["X"].double() + (st["residual"].double() if case["residual"] else 0.0)
        y = h / torch.sqrt((h * h).sum(-1, keepdim=True) / case["K"] + EPS) * st["weight"].double()
        out = {"residual_out": h} if case["residual"] else {}
        if case["y"]:
            out["Y"] = y
        if case["codes"]:
            out["codes"], out["scales"] = _exact_round(y if s is None else y / s, 8, rounded=False)[0], None
        return out
    if op == "product":
        E = torch.exp2(st["scales"].view(torch.uint8).double() - 127).repeat_interleave(BLOCK, 1)
        x = (st["codes"].double() if case["bits"] == 8 else _exact_values4(st["codes"])) * E
        return x @ _exact_weights(st)
    p = st["X"].double()
    if case.get("gate"):
        p = p * st["gate"].double() * torch.sigmoid(st["gate"].double())
    p = p if s is None else p / s
    if op == "quantize":
        return {"codes": _exact_round(p, 8, rounded=False)[0], "scales": None}
    v, scale = _exact_round(p, case["bits"])
    return (v.reshape(case["M"], -1, BLOCK) * scale).reshape(p.shape) @ _exact_weights(st)
