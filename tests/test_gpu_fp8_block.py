"""The 8-bit operators together, as the attention half of a block uses them, prompt and then token by token: norm, quantizer,
q|k|v product, append, attention, quantizer, o product.  Also on other streams and in captured graphs."""
import numpy as np
import pytest
import torch

from tests.fp8_util import A, DEV, bf16, dev, f32

pytestmark = pytest.mark.gpu

K, HQ, HK, D, T, BLOCKS = 512, 8, 2, 64, 16, 40


@pytest.fixture(scope="module")
def layers():
    rng = np.random.default_rng(0)
    w = lambda k, n: dev(bf16(rng.standard_normal((k, n)) / np.sqrt(k)))   # noqa: E731
    W = {"qkv": w(K, (HQ + 2 * HK) * D), "o": w(HQ * D, K)}
    a = np.arange(300)[:, None] * 10000.0 ** (-np.arange(D // 2) * 2 / D)
    return dict(W=W, packed={n: A.fp8_pack(v) for n, v in W.items()}, norm=dev(bf16(1 + 0.1 * rng.standard_normal(K))),
                qw=dev(bf16(1 + 0.1 * rng.standard_normal(D))), kw=dev(bf16(1 + 0.1 * rng.standard_normal(D))),
                rope=torch.from_numpy(np.concatenate((np.cos(a), np.sin(a)), 1).astype(np.float32)).to(DEV))


def sequences(lengths, table):
    cu = np.concatenate(([0], np.cumsum([n for _, n in lengths]))).astype(np.int32)
    return A.Sequences(torch.from_numpy(cu).to(DEV), torch.tensor([L for L, _ in lengths], dtype=torch.int32, device=DEV),
                       table, max(n for _, n in lengths))


def half(x, L, seqs, cache, stream=None):
    """x [M, K] -> x + attention half."""
    y = torch.empty_like(x)
    A.awq_rms_norm(x, None, L["norm"], 1e-5, None, y, stream=stream)
    qkv = A.fp8_gemm(A.fp8_quantize(y, stream=stream), L["packed"]["qkv"], stream)
    q = A.qkv_append(qkv, seqs, cache, L["rope"], L["qw"], L["kw"], stream=stream)
    att = A.attention(q, seqs, cache, stream=stream)
    return A.fp8_gemm(A.fp8_quantize(att.view(x.shape[0], -1), stream=stream), L["packed"]["o"], stream)


def plain(x, L, mask_len):
    """The same half without any quantization, float64, one sequence from its beginning."""
    x = f32(x).astype(np.float64)
    g = {n: f32(v).astype(np.float64) for n, v in (("norm", L["norm"]), ("qw", L["qw"]), ("kw", L["kw"]),
                                                   ("qkv", L["W"]["qkv"]), ("o", L["W"]["o"]))}
    n = x.shape[0]
    y = x / np.sqrt((x * x).mean(-1, keepdims=True) + 1e-5) * g["norm"]
    h = (y @ g["qkv"]).reshape(n, -1, D)
    q, k, v = h[:, :HQ], h[:, HQ:HQ + HK], h[:, HQ + HK:]
    nrm = lambda t, w: t / np.sqrt((t * t).mean(-1, keepdims=True) + 1e-6) * w   # noqa: E731
    r = L["rope"].double().cpu().numpy()[:n, None]
    c, s = r[..., :D // 2], r[..., D // 2:]
    rot = lambda t: np.concatenate((t[..., :D // 2] * c - t[..., D // 2:] * s,   # noqa: E731
                                    t[..., D // 2:] * c + t[..., :D // 2] * s), -1)
    q, k = rot(nrm(q, g["qw"])), rot(nrm(k, g["kw"]))
    out = np.empty((n, HQ, D))
    for j in range(HQ):
        t = q[:, j] @ k[:, j // (HQ // HK)].T / np.sqrt(D)
        t[np.triu_indices(n, 1)] = -np.inf
        p = np.exp(t - t.max(1, keepdims=True))
        out[:, j] = p @ v[:, j // (HQ // HK)] / p.sum(1, keepdims=True)
    return out.reshape(n, -1) @ g["o"]


def test_prompt_and_tokens_against_unquantized_float64(layers):
    """Three prompts in one call, then token by token: each step's output near that of unquantized arithmetic.  e4m3 rounds by
    2^-4 at most, random in sign, at four places (activations and weights of the products, K and V): their rms, about
    0.026 each, stay well under 0.15; a wrong token, head or scale shows as an error of order one."""
    rng = np.random.default_rng(1)
    cache = A.KVCache(BLOCKS, HK, D, T)
    table = torch.from_numpy(rng.permutation(BLOCKS)[:36].reshape(3, 12).astype(np.int32)).to(DEV)
    tokens = [33, 7, 100]
    xs = [rng.standard_normal((n + 20, K)) for n in tokens]
    got = [[] for _ in tokens]
    state = [0] * 3
    for step in range(21):
        take = [n if step == 0 else 1 for n in tokens]
        x = dev(bf16(np.concatenate([v[s:s + n] for v, s, n in zip(xs, state, take)])))
        state = [s + n for s, n in zip(state, take)]
        y = half(x, layers, sequences(list(zip(state, take)), table), cache)
        for i, part in enumerate(torch.split(y, take)):
            got[i].append(f32(part))
    for v, s, g in zip(xs, state, got):
        want = plain(bf16(v[:s]), layers, s)
        have = np.concatenate(g)
        err = np.linalg.norm(have - want) / np.linalg.norm(want)
        assert err < 0.15, err
        assert (np.linalg.norm(have - want, axis=1) / np.linalg.norm(want, axis=1)).max() < 0.3


def test_on_another_stream(layers):
    x = dev(bf16(np.random.default_rng(2).standard_normal((40, K))))
    table = torch.arange(12, dtype=torch.int32, device=DEV).view(2, 6)
    seqs = sequences([(33, 33), (7, 7)], table)
    ref = half(x, layers, seqs, A.KVCache(BLOCKS, HK, D, T))
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    cache = A.KVCache(BLOCKS, HK, D, T)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        got = half(x, layers, seqs, cache)
    side.synchronize()
    assert torch.equal(ref, got)
    cache = A.KVCache(BLOCKS, HK, D, T)
    torch.cuda.synchronize()
    y = torch.empty_like(x)
    A.awq_rms_norm(x, None, layers["norm"], 1e-5, None, y, stream=side)
    qkv = A.fp8_gemm(A.fp8_quantize(y, stream=side), layers["packed"]["qkv"], side)
    q = A.qkv_append(qkv, seqs, cache, layers["rope"], layers["qw"], layers["kw"], stream=side)
    att = A.attention(q, seqs, cache, stream=side)
    out = A.fp8_gemm(A.fp8_quantize(att.view(40, -1), stream=side), layers["packed"]["o"], side)
    side.synchronize()
    assert torch.equal(ref, out)


def test_captured_decode_replayed_with_growing_lengths(layers):
    """One decode step in two graphs that share workspaces; lengths and tables change on the device between replays.  Every
    replay equals the eager step from the same state, output and cache."""
    n_seq, M = 3, 3
    rng = np.random.default_rng(4)
    cache = A.KVCache(BLOCKS, HK, D, T)
    table = torch.from_numpy(rng.permutation(BLOCKS)[:36].reshape(3, 12).astype(np.int32)).to(DEV)
    tokens = [33, 7, 100]
    half(dev(bf16(rng.standard_normal((140, K)))), layers, sequences(list(zip(tokens, tokens)), table), cache)
    seqs = sequences([(n, 1) for n in tokens], table)
    p = layers["packed"]
    size = max(A.awq_fp8_gemm_workspace_size(M, w.K, w.N) for w in p.values())
    ws = A.workspace(max(size, A.awq_attention_workspace_size(M, n_seq, 1, HQ, HK, D)), DEV)
    x = dev(bf16(rng.standard_normal((M, K))))
    y, qkv, out = torch.empty_like(x), torch.empty(M, p["qkv"].N, dtype=torch.bfloat16, device=DEV), torch.empty_like(x)
    q = torch.empty(M, HQ, D, dtype=torch.bfloat16, device=DEV)
    att = torch.empty_like(q)
    codes = {k: (torch.empty(M, k, dtype=torch.float8_e4m3fn, device=DEV), torch.empty(M, -(-k // 128), device=DEV))
             for k in {K, HQ * D}}

    def step():
        A.awq_rms_norm(x, None, layers["norm"], 1e-5, None, y)
        A.awq_fp8_quantize(y, None, *codes[K])
        A.awq_fp8_gemm(*codes[K], p["qkv"].codes, p["qkv"].scales, qkv, ws)
        A.awq_qkv_append(qkv, layers["qw"], layers["kw"], 1e-6, layers["rope"], False, seqs.cu, seqs.length, seqs.table, 1, q,
                         cache.k, cache.v, cache.scales)
        A.awq_attention(q, seqs.cu, seqs.length, seqs.table, 1, cache.k, cache.v, cache.scales, D ** -0.5, True, att, ws)
        A.awq_fp8_quantize(att.view(M, -1), None, *codes[HQ * D])
        A.awq_fp8_gemm(*codes[HQ * D], p["o"].codes, p["o"].scales, out, ws)

    bufs = [cache.k, cache.v, cache.scales]
    take = lambda: [t.view(torch.uint8).clone() for t in bufs]   # noqa: E731
    start = take()
    step()
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step()
        graphs.append(g)
    for t, s in zip(bufs, start):
        t.view(torch.uint8).copy_(s)
    for i in range(6):
        x.copy_(bf16(rng.standard_normal((M, K))))
        seqs.length += 1
        before = take()
        step()
        want, cached = out.clone(), take()
        torch.cuda.synchronize()
        for g in graphs:
            for t, s in zip(bufs, before):
                t.view(torch.uint8).copy_(s)
            out.fill_(float("nan"))
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, want) and all(torch.equal(a, b) for a, b in zip(take(), cached)), i


def test_two_streams_at_once(layers):
    """Calls on two streams with their own caches, outputs and workspaces."""
    ins = [dev(bf16(np.random.default_rng(30 + i).standard_normal((50, K)))) for i in range(2)]
    table = torch.arange(12, dtype=torch.int32, device=DEV).view(2, 6)
    seqs = sequences([(43, 43), (7, 7)], table)
    want = [half(x, layers, seqs, A.KVCache(BLOCKS, HK, D, T)) for x in ins]
    caches = [A.KVCache(BLOCKS, HK, D, T) for _ in ins]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in ins]
    for _ in range(4):
        got = []
        for st, x, c in zip(streams, ins, caches):
            with torch.cuda.stream(st):
                got.append(half(x, layers, seqs, c))
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, got))
