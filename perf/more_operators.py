"""Workloads of the 8-bit operators of a block's attention half: the product in 8-bit floating point with
float32 scales for blocks of 128, with the packing of its weights and the quantization of its activations;
the norms of queries and keys with the rotation and the append to an 8-bit cache; and the attention that
reads that cache.

``run`` makes one pass.  With ``own`` false it computes the operator's formula with elementary torch
operations; with ``own`` true it calls the library.  Both read the same inputs in the same layouts, so their
outputs can be compared value by value.

Formats.  Elements are e4m3 (largest 448).
  product   a group is 128 consecutive channels of one row of activations, or 128 channels x 128 columns of
            weights: s = max(max|p|, 448 * 2^-120) / 448 (float32), element = p / s.
  cache     a block is T tokens of one sequence and one key/value head; K and V have a scale byte E each, which
            stands for 2^(E - 127): the least E >= 0 under which the largest number is at most 448.

Layouts (Kc = ceil(K / 128), Nt = ceil(N / 64)):
  activations  codes [M, K], scales float32 [M, Kc]
  weights      codes [Nt, Kc, 8, 64, 16]: byte b of (t, c, 2f + h, 16g + i) is channel 128c + 64h + 16g + b of
               column 64t + 16f + i, zero past K and N; scales float32 [ceil(N / 128), Kc]
  cache        K codes [blocks, Hk, T, D]; V codes [blocks, Hk, T / 16, D, 16], the 16 tokens of a group side by
               side; scale bytes [blocks, Hk, 2], K's and V's
  sequences    the new tokens of sequence b are rows cu[b] .. cu[b + 1] of q|k|v and of q; they are the last of
               its length[b] tokens; its i-th block of tokens is block table[b, i] of the cache
"""
import math

import torch

own = False

GROUP = 128
LARGEST = 448.0
LEAST = 2.0 ** -120
EPS = 1e-6
BASE = 10000.0


# ---------------------------------------------------------------- cases
def listed():
    return [
        # offline: the square layer
        dict(name="pack_square", op="pack", K=4096, N=4096),
        # offline: the widest layer of the 70B-shaped block
        dict(name="pack_wide", op="pack", K=8192, N=28672),
        # a small decode batch in front of down: silu(gate) * up
        dict(name="quantize_decode", op="quantize", M=16, K=28672, gate=True),
        # a prefill chunk in front of q|k|v
        dict(name="quantize_prefill", op="quantize", M=4096, K=8192, gate=False),
        # one token through the fused q|k|v projection: latency and weight traffic
        dict(name="product_decode", op="product", M=1, K=8192, N=10240),
        # a short ragged prompt
        dict(name="product_short", op="product", M=257, K=5120, N=13824),
        # a prefill chunk through gate or up
        dict(name="product_prefill", op="product", M=4096, K=8192, N=28672),
        # one token of each of 64 sequences, with norms, into blocks of 64 tokens
        dict(name="append_decode", op="append", B=64, n=1, L=700, Hq=64, Hk=8, D=128, T=64, R=128, norm=True,
             interleaved=False),
        # four ragged prompts of a 40-head model without norms, blocks of 16 tokens that they share with nothing older
        dict(name="append_prefill", op="append", B=4, n=2047, L=2047, Hq=40, Hk=40, D=128, T=16, R=128, norm=False,
             interleaved=False),
        # one sequence, one token: latency
        dict(name="attention_one", op="attention", B=1, n=1, L=4097, Hq=64, Hk=8, D=128, T=64),
        # a ragged decode batch of long sequences: cache traffic
        dict(name="attention_decode", op="attention", B=64, n=1, L=8192, Hq=64, Hk=8, D=128, T=64),
        # a prefill chunk behind as many cached tokens
        dict(name="attention_prefill", op="attention", B=1, n=4096, L=8192, Hq=64, Hk=8, D=128, T=64),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["pack", "quantize", "product", "product", "append", "attention", "attention"])
    if op in ("pack", "quantize", "product"):
        K = 16 * _log(rng, 16, 1792)
        if op == "quantize":
            return dict(op=op, M=min(_log(rng, 1, 8192), 4096 * 8192 // K), K=K, gate=rng.random() < 0.5)
        N = max(8, min(8 * _log(rng, 16, 3584), 8192 * 28672 // K // 8 * 8))
        return dict(op=op, K=K, N=N) if op == "pack" else dict(op=op, M=_log(rng, 1, 4096), K=K, N=N)
    Hq, Hk = rng.choice([(64, 8), (32, 8), (40, 8), (32, 32), (40, 40), (16, 1), (12, 4)])
    D, T, B = rng.choice([64, 128, 128]), rng.choice([16, 32, 64, 128]), _log(rng, 1, 64)
    n = 1 if rng.random() < 0.5 else _log(rng, 2, 2048)
    if op == "append":
        n = min(n, max(1, 8188 * 120 // (B * (Hq + 2 * Hk))))
        L = n + (0 if rng.random() < 0.3 else _log(rng, 1, 1500))
        return dict(op=op, B=B, n=n, L=L, Hq=Hq, Hk=Hk, D=D, T=T, R=rng.choice([D, D, D // 2]),
                    norm=rng.random() < 0.5, interleaved=rng.random() < 0.3)
    L = n + _log(rng, 1, 16384)
    L = max(n, min(L, 64 * 8192 * 8 // (B * Hk)))
    n = max(1, min(n, 4096 * 8192 * 32 // (B * L * Hq)))
    return dict(op=op, B=B, n=n, L=L, Hq=Hq, Hk=Hk, D=D, T=T)


def _lengths(case):
    """(tokens, new tokens) of each sequence: the first has L and n, the others up to as many, spread evenly."""
    out = []
    for b in range(case["B"]):
        u = 1.0 if b == 0 else (b * 0.6180339887498949) % 1.0
        n = max(1, int(case["n"] * (0.5 + 0.5 * u)))
        out.append((max(n, int(case["L"] * u)), n))
    return out


def work(case):
    if case["op"] in ("pack", "quantize", "product"):
        K = case["K"]
        c = -(-K // GROUP)
        if case["op"] == "pack":
            N = case["N"]
            return {"bytes": 3 * K * N + 4 * c * -(-N // GROUP), "flops": 3 * K * N}
        M = case["M"]
        acts = M * K + 4 * M * c
        if case["op"] == "quantize":
            return {"bytes": 2 * M * K * (2 if case["gate"] else 1) + acts, "flops": (8 if case["gate"] else 3) * M * K}
        N = case["N"]
        return {"bytes": acts + K * N + 4 * c * -(-N // GROUP) + 2 * M * N, "flops": 2 * M * N * K}
    Hq, Hk, D = case["Hq"], case["Hk"], case["D"]
    lengths = _lengths(case)
    M = sum(n for _, n in lengths)
    if case["op"] == "append":
        return {"bytes": M * D * (2 * (Hq + 2 * Hk) + 2 * Hq + 2 * Hk), "flops": M * D * (8 * (Hq + Hk) + 4 * Hk)}
    seen = sum(n * L - n * (n - 1) // 2 for L, n in lengths)
    return {"bytes": 4 * M * Hq * D + 2 * sum(L for L, _ in lengths) * Hk * D, "flops": 4 * seen * Hq * D}


# ---------------------------------------------------------------- formats and layouts, in 32 bits
def _pad(x, rows, cols):
    return torch.nn.functional.pad(x, (0, cols - x.shape[1], 0, rows - x.shape[0]))


def _quantize_rows(p):
    """p float32 [M, K] -> codes e4m3 [M, K], scales [M, Kc]."""
    M, K = p.shape
    c = -(-K // GROUP)
    g = _pad(p, M, c * GROUP).view(M, c, GROUP)
    s = g.abs().amax(-1).clamp_min(LARGEST * LEAST) / LARGEST
    return (g / s[..., None]).view(M, c * GROUP)[:, :K].to(torch.float8_e4m3fn), s


def _weights_layout(v):
    """[Kc * 128, Nt * 64] -> [Nt, Kc, 8, 64, 16]."""
    c, t = v.shape[0] // GROUP, v.shape[1] // 64
    return v.view(c, 2, 4, 16, t, 4, 16).permute(4, 0, 5, 1, 2, 6, 3).reshape(t, c, 8, 64, 16)


def _weights_back(codes):
    """[Nt, Kc, 8, 64, 16] -> [Kc * 128, Nt * 64]."""
    t, c = codes.shape[:2]
    return codes.view(t, c, 4, 2, 4, 16, 16).permute(1, 3, 4, 6, 0, 2, 5).reshape(c * GROUP, t * 64)


def _pack_weights(W):
    K, N = W.shape
    c, nb, nt = -(-K // GROUP), -(-N // GROUP), -(-N // 64)
    v = _pad(W.float(), c * GROUP, nb * GROUP).view(c, GROUP, nb, GROUP)
    s = v.abs().amax((1, 3)).clamp_min(LARGEST * LEAST) / LARGEST                # [Kc, Nb]
    q = (v / s[:, None, :, None]).view(c * GROUP, nb * GROUP)[:, :nt * 64]
    return _weights_layout(q).to(torch.float8_e4m3fn), s.t().contiguous()


def _spread(s, K, N):
    """[Nb, Kc] -> [K, N]."""
    return s.t().repeat_interleave(GROUP, 0)[:K].repeat_interleave(GROUP, 1)[:, :N]


def _scale_byte(top):
    """The least E >= 0 with top <= 448 * 2^(E - 127), for float32 numbers; int32."""
    bits = top.view(torch.int32)
    return ((bits >> 23) - 8 + ((bits & 0x7fffff) > 0x600000).int()).clamp_min(0)


def _step(E):
    return torch.ldexp(torch.ones((), device=E.device), E.int() - 127)


def _v_layout(v):
    """[.., T, D] -> [.., T / 16, D, 16]."""
    return v.unflatten(-2, (-1, 16)).transpose(-1, -2)


def _v_back(v):
    return v.transpose(-1, -2).flatten(-3, -2)


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

    def buffer(*shape, dtype):
        return torch.zeros(shape, dtype=dtype, device="cuda")

    f8, e8, f32, bf16 = torch.float8_e4m3fn, torch.float8_e8m0fnu, torch.float32, torch.bfloat16
    st = dict(case=dict(case))
    op = case["op"]
    if op in ("pack", "quantize", "product"):
        K = case["K"]
        c = -(-K // GROUP)
        if op in ("pack", "product"):
            N = case["N"]
            W = (normal(K, N) / math.sqrt(K)).to(bf16)
        if op == "pack":
            st["W"] = W
            st["codes"] = buffer(-(-N // 64), c, 8, 64, 16, dtype=f8)
            st["scales"] = buffer(-(-N // GROUP), c, dtype=f32)
            return st
        M = case["M"]
        if op == "quantize":
            st["X"], st["gate"] = acts(M, K), normal(M, K).to(bf16) if case["gate"] else None
            st["codes"], st["scales"] = buffer(M, K, dtype=f8), buffer(M, c, dtype=f32)
            return st
        st["codes"], st["scales"] = _quantize_rows(acts(M, K).float())
        st["wcodes"], st["wscales"] = _pack_weights(W)
        st["Y"] = buffer(M, N, dtype=bf16)
        if own:
            from weight_only_int4_act_amd import awq
            st["ws"] = awq.workspace(awq.awq_fp8_gemm_workspace_size(M, K, N), "cuda")
        return st
    B, Hq, Hk, D, T = (case[k] for k in ("B", "Hq", "Hk", "D", "T"))
    lengths = _lengths(case)
    width = -(-max(L for L, _ in lengths) // T)
    used = [-(-L // T) for L, _ in lengths]
    blocks = sum(used) + 3                                      # a pool with a few blocks that no sequence has
    order = torch.randperm(blocks, generator=g, device="cuda").to(torch.int32)
    table = torch.full((B, width), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, u in enumerate(used):
        table[b, :u] = order[at:at + u]
        at += u
    cu = [0]
    for _, n in lengths:
        cu.append(cu[-1] + n)
    M = cu[-1]
    st |= dict(table=table, cu=torch.tensor(cu, dtype=torch.int32, device="cuda"),
               length=torch.tensor([L for L, _ in lengths], dtype=torch.int32, device="cuda"), max_q=case["n"])
    # what is cached: heads of their own sizes, and some channels of K much larger than the rest
    k, v = buffer(blocks, Hk, T, D, dtype=f8), buffer(blocks, Hk, T // 16, D, 16, dtype=f8)
    E = buffer(blocks, Hk, 2, dtype=torch.uint8)
    gain = torch.where(torch.rand(Hk, 1, D, generator=g, device="cuda") < 0.03, 4.0, 0.7)
    size = torch.exp(0.5 * normal(Hk, 1, 1))
    for lo in range(0, blocks, 4096):
        m = min(4096, blocks - lo)
        for i, x in enumerate((normal(m, Hk, T, D) * gain, normal(m, Hk, T, D) * size)):
            e = _scale_byte(x.abs().amax((2, 3)))
            c = (x / _step(e)[..., None, None])
            (k if i == 0 else v)[lo:lo + m] = (c if i == 0 else _v_layout(c)).to(f8)
            E[lo:lo + m, :, i] = e.to(torch.uint8)
    st |= dict(k=k, v=v, scales=E.view(e8))
    if op == "append":
        st["qkv"] = (normal(M, Hq + 2 * Hk, D) * torch.exp(0.3 * normal(M, 1, 1))).to(bf16).view(M, -1)
        R, P = case["R"], case["L"]
        angle = torch.arange(P, dtype=torch.float64, device="cuda")[:, None] * \
            BASE ** (-torch.arange(R // 2, dtype=torch.float64, device="cuda") * 2 / R)
        st["rope"] = torch.cat((angle.cos(), angle.sin()), 1).float()
        for name in ("q_weight", "k_weight"):
            st[name] = (1 + 0.1 * normal(D)).to(bf16) if case["norm"] else None
        st["q"] = buffer(M, Hq, D, dtype=bf16)
        return st
    st["q"], st["out"] = normal(M, Hq, D).to(bf16), buffer(M, Hq, D, dtype=bf16)
    if own:
        from weight_only_int4_act_amd import awq
        st["ws"] = awq.workspace(awq.awq_attention_workspace_size(M, B, case["n"], Hq, Hk, D), "cuda")
    return st


# ---------------------------------------------------------------- one pass
def run(st):
    return _run_own(st) if own else _run_plain(st)


def _run_own(st):
    from weight_only_int4_act_amd import awq
    case = st["case"]
    op = case["op"]
    if op == "pack":
        awq.awq_fp8_pack(st["W"], st["codes"], st["scales"])
        return {"codes": st["codes"], "scales": st["scales"]}
    if op == "quantize":
        awq.awq_fp8_quantize(st["X"], st["gate"], st["codes"], st["scales"])
        return {"codes": st["codes"], "scales": st["scales"]}
    if op == "product":
        awq.awq_fp8_gemm(st["codes"], st["scales"], st["wcodes"], st["wscales"], st["Y"], st["ws"])
        return st["Y"]
    if op == "append":
        awq.awq_qkv_append(st["qkv"], st["q_weight"], st["k_weight"], EPS, st["rope"], case["interleaved"], st["cu"],
                           st["length"], st["table"], st["max_q"], st["q"], st["k"], st["v"], st["scales"])
        return {name: st[name] for name in ("q", "k", "v", "scales")}
    awq.awq_attention(st["q"], st["cu"], st["length"], st["table"], st["max_q"], st["k"], st["v"], st["scales"],
                      1 / math.sqrt(case["D"]), True, st["out"], st["ws"])
    return st["out"]


def _tokens(st):
    """Of each new token: its sequence, its position and whether its block began before the new tokens did."""
    cu, length, M = st["cu"].long(), st["length"].long(), st["q"].shape[0]
    row = torch.arange(M, device=cu.device)
    b = torch.searchsorted(cu[1:].contiguous(), row, right=True)
    first = length - (cu[1:] - cu[:-1])
    return b, first[b] + row - cu[b], first


def _rotate(x, rope, pos, R, interleaved):
    """x float32 [M, H, D]; the first R numbers of each head in pairs."""
    cos, sin = rope[pos][:, None, :].chunk(2, -1)
    a, c = (x[..., 0:R:2], x[..., 1:R:2]) if interleaved else (x[..., :R // 2], x[..., R // 2:R])
    a, c = a * cos - c * sin, c * cos + a * sin
    turned = torch.stack((a, c), -1).flatten(-2) if interleaved else torch.cat((a, c), -1)
    return torch.cat((turned, x[..., R:]), -1)


def _heads(st, dtype):
    """q, k, v [M, H, D] of the new tokens, normed and rotated."""
    case = st["case"]
    Hq, Hk, D, R = case["Hq"], case["Hk"], case["D"], case["R"]
    x = st["qkv"].to(dtype).view(-1, Hq + 2 * Hk, D)
    q, k, v = x.split((Hq, Hk, Hk), 1)
    if case["norm"]:
        q, k = (h * torch.rsqrt(h.square().mean(-1, keepdim=True) + EPS) * st[w].to(dtype)
                for h, w in ((q, "q_weight"), (k, "k_weight")))
    pos = _tokens(st)[1]
    q, k = (_rotate(h, st["rope"].to(dtype), pos, R, case["interleaved"]) for h in (q, k))
    return q, k, v


def _run_plain(st):
    case = st["case"]
    op = case["op"]
    if op == "pack":
        codes, scales = _pack_weights(st["W"])
        return {"codes": codes, "scales": scales}
    if op == "quantize":
        p = st["X"].float()
        if case["gate"]:
            gate = st["gate"].float()
            p = gate / (1 + torch.exp(-gate)) * p
        codes, scales = _quantize_rows(p)
        return {"codes": codes, "scales": scales}
    if op == "product":
        K, N = case["K"], case["N"]
        x = st["codes"].float() * st["scales"].repeat_interleave(GROUP, 1)[:, :K]
        w = _weights_back(st["wcodes"]).float()[:K, :N] * _spread(st["wscales"], K, N)
        return (x @ w).to(torch.bfloat16)
    return _plain_append(st) if op == "append" else _plain_attention(st)


def _plain_append(st):
    T = st["case"]["T"]
    q, k, v = _heads(st, torch.float32)
    b, pos, first = _tokens(st)
    block, slot = st["table"][b, pos // T].long(), pos % T
    E = st["scales"].view(torch.uint8).int()
    # sequences whose first new token joins older ones in its block
    seq = torch.arange(len(first), device=q.device)
    joins = (first % T > 0) & (first < st["length"])
    old = st["table"][seq, (first // T).clamp_max(st["table"].shape[1] - 1)].long()
    kept = torch.zeros_like(E)
    kept[old[joins]] = E[old[joins]]
    mine = joins[:, None, None] & (torch.arange(T, device=q.device) < (first % T)[:, None])[:, None, :]   # [B, 1, T]
    out = {"q": q.to(torch.bfloat16)}
    codes = []
    for i, x in enumerate((k, v)):
        top = torch.zeros(E.shape[:2], device=q.device).scatter_reduce_(
            0, block[:, None].expand(-1, x.shape[1]), x.abs().amax(-1), "amax")
        touched = torch.zeros(E.shape[0], dtype=torch.bool, device=q.device)
        touched[block] = True
        e = torch.where(touched[:, None], torch.maximum(_scale_byte(top), kept[:, :, i]), E[:, :, i])
        c = st["k"] if i == 0 else _v_back(st["v"].view(torch.uint8)).view(torch.float8_e4m3fn)
        c = c.view(torch.uint8).clone()
        again = (c[old].view(torch.float8_e4m3fn).float() * _step(E[old, :, i] - e[old] + 127)[..., None, None])
        again = again.to(torch.float8_e4m3fn).view(torch.uint8)
        # (a sequence that joins nothing writes back what its block holds)
        c[old] = torch.where(mine[..., None], again, c[old])
        c[block, :, slot] = (x / _step(e)[block][..., None]).to(torch.float8_e4m3fn).view(torch.uint8)
        codes.append(c)
        E[:, :, i] = e
    st["k"].view(torch.uint8).copy_(codes[0])
    st["v"].view(torch.uint8).copy_(_v_layout(codes[1]))
    st["scales"].view(torch.uint8).copy_(E)
    return out | {name: st[name] for name in ("k", "v", "scales")}


def _cached(st, dtype, block):
    """K and V of the blocks `block` [..], as numbers [.., Hk, T, D]."""
    step = torch.exp2(st["scales"].view(torch.uint8).to(dtype) - 127)[block]
    k = st["k"].view(torch.uint8)[block].view(torch.float8_e4m3fn).to(dtype)
    v = _v_back(st["v"].view(torch.uint8)[block]).view(torch.float8_e4m3fn).to(dtype)
    return k * step[..., 0, None, None], v * step[..., 1, None, None]


def _plain_attention(st):
    case = st["case"]
    B, Hq, Hk, D, n = (case[k] for k in ("B", "Hq", "Hk", "D", "n"))
    G = Hq // Hk
    k, v = _cached(st, torch.float32, st["table"].clamp_min(0).long())         # [B, width, Hk, T, D]
    k, v = (x.transpose(1, 2).flatten(2, 3) for x in (k, v))                   # [B, Hk, L, D]
    b, pos, first = _tokens(st)
    i = pos - first[b]
    q = torch.zeros((B, n, Hq, D), device=k.device)
    q[b, i] = st["q"].float()
    q = q.view(B, n, Hk, G, D).permute(0, 2, 1, 3, 4).reshape(B, Hk, n * G, D)
    s = torch.matmul(q, k.transpose(2, 3).contiguous()) * (1 / math.sqrt(D))   # [B, Hk, n G, L]
    at = (first[:, None] + torch.arange(n, device=k.device)).repeat_interleave(G, 1)          # [B, n G]
    seen = torch.arange(k.shape[2], device=k.device) <= at[..., None]
    s.masked_fill_(~seen[:, None], -math.inf)
    s -= s.amax(-1, keepdim=True)
    s.exp_()
    o = torch.matmul(s, v.contiguous()) / s.sum(-1, keepdim=True)
    o = o.view(B, Hk, n, G, D).permute(0, 2, 1, 3, 4).reshape(B, n, Hq, D)
    return o[b, i].to(torch.bfloat16)


# ---------------------------------------------------------------- the definition, in 64 bits
def _exact_groups(p, axes):
    """Scales of groups: the largest magnitude over `axes`, over 448."""
    return torch.linalg.vector_norm(p, ord=math.inf, dim=axes, keepdim=True).clamp_min(LARGEST * LEAST) / LARGEST


def _exact_weights(st):
    K, N = st["case"]["K"], st["case"]["N"]
    W = torch.empty((K, N), dtype=torch.float64, device="cuda")
    for t in range(st["wcodes"].shape[0]):
        tile = st["wcodes"][t].double().reshape(-1, 4, 2, 4, 16, 16)                    # c, f, h, g, i, b
        tile = tile.permute(1, 4, 0, 2, 3, 5).reshape(64, -1)[:, :K]                    # column, channel
        s = st["wscales"][t // 2].double().repeat_interleave(GROUP)[:K]
        n = min(64, N - 64 * t)
        W[:, 64 * t:64 * t + n] = (tile * s)[:n].t()
    return W


def _exact_byte(top):
    """The least E >= 0 with top <= 448 * 2^(E - 127), as float64."""
    return torch.where(top > 0, torch.ceil(torch.log2(top / LARGEST)) + 127, torch.zeros_like(top)).clamp_min(0)


def _exact_append(st):
    """Every code as the number that it is the rounding of: value over its block's scale."""
    T = st["case"]["T"]
    q, k, v = _heads_exact(st)
    cu, length, table = st["cu"].tolist(), st["length"].tolist(), st["table"].tolist()
    E = st["scales"].view(torch.uint8).double()
    now = [st["k"].double(), st["v"].double().transpose(-1, -2).reshape(st["k"].shape)]
    for b in range(len(length)):
        n = cu[b + 1] - cu[b]
        start = length[b] - n
        for j in range(start // T, -(-length[b] // T)):
            lo, hi = max(start, j * T), min(length[b], (j + 1) * T)
            blk, s0, s1 = table[b][j], lo - j * T, hi - j * T
            for i, x in enumerate((k, v)):
                new = x[cu[b] + lo - start:cu[b] + hi - start].transpose(0, 1)          # [Hk, m, D]
                e = _exact_byte(torch.linalg.vector_norm(new, ord=math.inf, dim=(1, 2)))
                if s0:
                    e = torch.maximum(e, E[blk, :, i])
                    now[i][blk, :, :s0] *= torch.exp2(E[blk, :, i] - e)[:, None, None]
                now[i][blk, :, s0:s1] = new / torch.exp2(e - 127)[:, None, None]
    k, v = now
    return {"q": q, "k": k, "v": v.unflatten(2, (-1, 16)).transpose(-1, -2), "scales": None}


def _heads_exact(st):
    case = st["case"]
    Hq, Hk, D, R = case["Hq"], case["Hk"], case["D"], case["R"]
    x = st["qkv"].double().view(-1, Hq + 2 * Hk, D)
    cu, length = st["cu"].tolist(), st["length"].tolist()
    pos = torch.cat([torch.arange(length[b] - (cu[b + 1] - cu[b]), length[b]) for b in range(len(length))]).cuda()
    rope = st["rope"].double()[pos]
    turn = torch.complex(rope[:, :R // 2].contiguous(), rope[:, R // 2:].contiguous())[:, None]
    out = []
    for h, w in ((x[:, :Hq], "q_weight"), (x[:, Hq:Hq + Hk], "k_weight")):
        if case["norm"]:
            h = h / torch.sqrt((h * h).sum(-1, keepdim=True) / D + EPS) * st[w].double()
        h = h.clone()
        even = slice(0, R, 2) if case["interleaved"] else slice(0, R // 2)
        odd = slice(1, R, 2) if case["interleaved"] else slice(R // 2, R)
        z = torch.complex(h[..., even].contiguous(), h[..., odd].contiguous()) * turn
        h[..., even], h[..., odd] = z.real, z.imag
        out.append(h)
    return out[0], out[1], x[:, Hq + Hk:]


def _exact_attention(st):
    case = st["case"]
    Hq, Hk, D, T = (case[k] for k in ("Hq", "Hk", "D", "T"))
    G = Hq // Hk
    cu, length = st["cu"].tolist(), st["length"].tolist()
    E = st["scales"].view(torch.uint8).double()
    out = torch.empty(st["q"].shape, dtype=torch.float64, device="cuda")
    for b, L in enumerate(length):
        blk = st["table"][b, :-(-L // T)].long()
        step = torch.exp2(E[blk] - 127)                                                 # [nb, Hk, 2]
        k = st["k"].view(torch.uint8)[blk].view(torch.float8_e4m3fn).double()
        v = st["v"].view(torch.uint8)[blk].view(torch.float8_e4m3fn).double().transpose(-1, -2).reshape(k.shape)
        n = cu[b + 1] - cu[b]
        late = torch.arange(L, device="cuda")[None, :] > torch.arange(L - n, L, device="cuda")[:, None]
        for h in range(Hk):
            kh = (k[:, h] * step[:, h, 0, None, None]).reshape(-1, D)[:L]
            vh = (v[:, h] * step[:, h, 1, None, None]).reshape(-1, D)[:L]
            for j in range(h * G, h * G + G):
                s = st["q"][cu[b]:cu[b + 1], j].double() @ kh.t() / math.sqrt(D)
                out[cu[b]:cu[b + 1], j] = torch.softmax(s.masked_fill_(late, -math.inf), -1) @ vh
    return out


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "append":
        return _exact_append(st)
    if op == "attention":
        return _exact_attention(st)
    K = case["K"]
    c = -(-K // GROUP)
    if op == "pack":
        N = case["N"]
        nb, nt = -(-N // GROUP), -(-N // 64)
        W = _pad(st["W"].double(), c * GROUP, nb * GROUP).view(c, GROUP, nb, GROUP)
        s = _exact_groups(W, (1, 3))
        q = (W / s).view(c, 2, 4, 16, 2 * nb, 4, 16)[:, :, :, :, :nt]
        return {"codes": q.permute(4, 0, 5, 1, 2, 6, 3).reshape(nt, c, 8, 64, 16), "scales": s.view(c, nb).t()}
    M = case["M"]
    if op == "quantize":
        p = st["X"].double()
        if case["gate"]:
            p = p * st["gate"].double() * torch.sigmoid(st["gate"].double())
        p = _pad(p, M, c * GROUP).view(M, c, GROUP)
        s = _exact_groups(p, (2,))
        return {"codes": (p / s).view(M, -1)[:, :K], "scales": s.view(M, c)}
    x = st["codes"].double() * st["scales"].double().repeat_interleave(GROUP, 1)[:, :K]
    return x @ _exact_weights(st)
