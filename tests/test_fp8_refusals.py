"""Refusals of the 8-bit operators, on the host: the C entry points reject bad arguments before anything is enqueued and
write nothing, and the binding refuses what the C ABI cannot see."""
import ctypes

import pytest
import torch

from weight_only_int4_act_amd import awq as A

P = lambda v: ctypes.c_void_p(v)   # noqa: E731  never dereferenced: every call below is rejected first
BIG = ctypes.c_size_t(1 << 40)
INV, UNS, WS = A.AWQ_ERR_INVALID_ARG, A.AWQ_ERR_UNSUPPORTED, A.AWQ_ERR_WORKSPACE
L = A.library()
X, G, W, C, S, Y, R, V, F, CU, LEN, TAB, QW, KW = (P(0x100000000 * (i + 1)) for i in range(14))   # far apart
ODD = P(0x10008)


def test_packed_sizes():
    assert A.awq_fp8_codes_bytes(4096, 4096) == 4096 * 4096 and A.awq_fp8_scales_count(4096, 4096) == 32 * 32
    assert A.awq_fp8_codes_bytes(144, 65) == 2 * 2 * 8192 and A.awq_fp8_scales_count(144, 129) == 2 * 2
    for K, N in ((0, 8), (16, 0), (24, 8), (-16, 8), (1 << 40, 8), (16, 1 << 40), (1 << 23, 1 << 20), (65536 * 128, 8)):
        assert A.awq_fp8_codes_bytes(K, N) == 0 and A.awq_fp8_scales_count(K, N) == 0, (K, N)


def test_workspace_sizes_of_bad_sizes():
    for M, K, N in ((0, 64, 8), (1, 40, 8), (1, 64, 0), (65535 * 16 + 1, 64, 8), (1 << 62, 64, 8), (1, 1 << 62, 8),
                    (1, 64, 1 << 62)):
        assert A.awq_fp8_gemm_workspace_size(M, K, N) == 0, (M, K, N)
    for a in ((0, 1, 1, 8, 2, 64), (1, 0, 1, 8, 2, 64), (1, 1, 0, 8, 2, 64), (1, 1, 1, 8, 3, 64), (1, 1, 1, 8, 2, 80),
              (1, 1, 1, 0, 2, 64), (1, 1, 1, 8, 0, 64), (1 << 40, 1, 1, 8, 2, 64), (1, 1, 1, 2048, 2, 64)):
        assert A.awq_attention_workspace_size(*a) == 0, a


def test_pack():
    for W_, K, N, C_, S_ in ((None, 64, 8, C, S), (W, 64, 8, None, S), (W, 64, 8, C, None), (W, 0, 8, C, S), (W, 40, 8, C, S),
                             (W, 64, 0, C, S), (W, 64, -1, C, S), (P(0x10001), 64, 8, C, S), (W, 64, 8, ODD, S),
                             (W, 64, 8, C, P(0x10002)), (W, 1 << 40, 8, C, S), (W, 64, 8, W, S), (W, 64, 8, C, W),
                             (W, 64, 8, C, C)):
        assert L.awq_fp8_pack(W_, K, N, C_, S_, None) == INV, (W_, K, N, C_, S_)


def test_quantize():
    ok = dict(X=X, g=None, M=3, K=64, C=C, S=S)
    for bad in (dict(X=None), dict(C=None), dict(S=None), dict(M=0), dict(K=40), dict(M=1 << 40), dict(K=1 << 40),
                dict(X=ODD), dict(g=ODD), dict(C=ODD), dict(S=P(0x10002)), dict(C=X), dict(S=X), dict(g=C), dict(S=C)):
        a = {**ok, **bad}
        assert L.awq_fp8_quantize(a["X"], a["g"], a["M"], a["K"], a["C"], a["S"], None) == INV, bad


def test_gemm():
    ok = dict(C=C, S=S, M=3, w=W, F=F, K=4096, N=4096, Y=Y, ws=V, n=BIG)
    for bad in (dict(C=None), dict(S=None), dict(w=None), dict(F=None), dict(Y=None), dict(M=0), dict(M=65535 * 16 + 1),
                dict(K=40), dict(N=12), dict(N=0), dict(N=4194312), dict(C=ODD), dict(w=ODD), dict(F=P(0x10002)),
                dict(S=P(0x10002)), dict(Y=ODD), dict(Y=C), dict(Y=W), dict(Y=F), dict(Y=S)):
        a = {**ok, **bad}
        got = L.awq_fp8_gemm(a["C"], a["S"], a["M"], a["w"], a["F"], a["K"], a["N"], a["Y"], a["ws"], a["n"], None)
        assert got == INV, (bad, got)
    for M in (1, 3, 100, 1000):
        need = A.awq_fp8_gemm_workspace_size(M, 4096, 512)
        if need:
            call = lambda ws, n: L.awq_fp8_gemm(C, S, M, W, F, 4096, 512, Y, ws, n, None)   # noqa: B023, E731
            assert call(V, need - 1) == WS and call(None, need) == WS
            assert call(P(V.value + 16), need) == INV and call(Y, need) == INV and call(W, need) == INV
    assert A.awq_fp8_gemm_workspace_size(1, 4096, 512) > 65536


APPEND = dict(x=X, M=5, Hq=8, Hk=2, D=64, qw=QW, kw=KW, eps=1e-5, rope=R, P=100, R=64, il=0, cu=CU, le=LEN, tab=TAB, n=2,
              width=4, mq=3, q=Y, k=C, v=V, e=S, blocks=9, T=16)


def append(**bad):
    a = {**APPEND, **bad}
    return L.awq_qkv_append(a["x"], a["M"], a["Hq"], a["Hk"], a["D"], a["qw"], a["kw"], a["eps"], a["rope"], a["P"], a["R"],
                            a["il"], a["cu"], a["le"], a["tab"], a["n"], a["width"], a["mq"], a["q"], a["k"], a["v"], a["e"],
                            a["blocks"], a["T"], None)


def test_append():
    for bad, st in ((dict(x=None), INV), (dict(q=None), INV), (dict(k=None), INV), (dict(v=None), INV), (dict(e=None), INV),
                    (dict(cu=None), INV), (dict(le=None), INV), (dict(tab=None), INV), (dict(M=0), INV), (dict(M=-1), INV),
                    (dict(M=1 << 40), INV), (dict(Hq=0), INV), (dict(Hk=0), INV), (dict(Hq=9), INV), (dict(Hq=2048), INV),
                    (dict(D=0), INV), (dict(D=96), UNS), (dict(D=256), UNS), (dict(T=8), UNS), (dict(T=48), UNS),
                    (dict(T=256), UNS), (dict(T=0), UNS), (dict(T=-16), UNS), (dict(n=0), INV), (dict(width=0), INV),
                    (dict(mq=0), INV), (dict(blocks=0), INV), (dict(blocks=1 << 40), INV), (dict(width=1 << 27), INV),
                    (dict(n=1 << 30, mq=1 << 20), INV), (dict(eps=0.0), INV), (dict(eps=float("nan")), INV),
                    (dict(eps=2.0), INV), (dict(P=0), INV), (dict(R=0), INV), (dict(R=24), INV), (dict(R=80), INV),
                    (dict(il=2), INV), (dict(x=ODD), INV), (dict(qw=ODD), INV), (dict(kw=ODD), INV), (dict(rope=ODD), INV),
                    (dict(q=ODD), INV), (dict(k=ODD), INV), (dict(v=ODD), INV), (dict(e=P(0x10001)), INV),
                    (dict(cu=P(0x10002)), INV), (dict(le=P(0x10002)), INV), (dict(tab=P(0x10002)), INV), (dict(q=X), INV),
                    (dict(k=X), INV), (dict(v=C), INV), (dict(e=C), INV), (dict(q=V), INV), (dict(q=QW), INV), (dict(k=R), INV),
                    (dict(e=TAB), INV), (dict(v=LEN), INV), (dict(q=CU), INV)):
        assert append(**bad) == st, bad


ATT = dict(q=X, M=5, Hq=8, Hk=2, D=64, cu=CU, le=LEN, tab=TAB, n=2, width=4, mq=3, k=C, v=V, e=S, blocks=9, T=16, scale=0.1,
           causal=1, out=Y, ws=F, size=BIG)


def attend(**bad):
    a = {**ATT, **bad}
    return L.awq_attention(a["q"], a["M"], a["Hq"], a["Hk"], a["D"], a["cu"], a["le"], a["tab"], a["n"], a["width"], a["mq"],
                           a["k"], a["v"], a["e"], a["blocks"], a["T"], a["scale"], a["causal"], a["out"], a["ws"],
                           a["size"], None)


def test_attention():
    for bad, st in ((dict(q=None), INV), (dict(out=None), INV), (dict(k=None), INV), (dict(v=None), INV), (dict(e=None), INV),
                    (dict(cu=None), INV), (dict(le=None), INV), (dict(tab=None), INV), (dict(M=0), INV), (dict(M=1 << 40), INV),
                    (dict(Hq=0), INV), (dict(Hk=0), INV), (dict(Hq=9), INV), (dict(D=0), INV), (dict(D=96), UNS),
                    (dict(T=8), UNS), (dict(T=256), UNS), (dict(n=0), INV), (dict(width=0), INV), (dict(mq=0), INV),
                    (dict(blocks=0), INV), (dict(width=1 << 27), INV), (dict(scale=float("nan")), INV),
                    (dict(scale=float("inf")), INV), (dict(causal=2), INV), (dict(q=ODD), INV), (dict(out=ODD), INV),
                    (dict(k=ODD), INV), (dict(e=P(0x10001)), INV), (dict(cu=P(0x10002)), INV), (dict(out=X), INV),
                    (dict(out=C), INV), (dict(out=V), INV), (dict(out=S), INV), (dict(out=TAB), INV), (dict(ws=X), INV),
                    (dict(ws=Y), INV), (dict(ws=C), INV), (dict(ws=P(F.value + 16)), INV), (dict(ws=None), WS)):
        assert attend(**bad) == st, bad
    need = A.awq_attention_workspace_size(5, 2, 3, 8, 2, 64)
    assert need > 65536 and attend(size=need - 1) == WS


def test_rejected_calls_write_nothing():
    outs = [(ctypes.c_uint8 * 4096)() for _ in range(4)]
    for b in outs:
        ctypes.memset(b, 0xA5, 4096)
    before = [bytes(b) for b in outs]
    q = [ctypes.cast(b, ctypes.c_void_p) for b in outs]
    st = [L.awq_fp8_pack(X, 40, 8, q[0], q[1], None), L.awq_fp8_quantize(X, None, 2, 40, q[0], q[1], None),
          L.awq_fp8_gemm(C, S, 2, W, F, 64, 12, q[0], q[1], BIG, None), append(q=q[0], k=q[1], v=q[2], e=q[3], T=8),
          attend(out=q[0], ws=q[1], causal=3)]
    assert all(v < 0 for v in st), st
    assert [bytes(b) for b in outs] == before


def test_binding_checks():
    bf, u8, f8, f32, i32 = torch.bfloat16, torch.uint8, torch.float8_e4m3fn, torch.float32, torch.int32
    K, N, M = 144, 72, 4
    Wt = torch.zeros(K, N, dtype=bf)
    codes, scales = torch.zeros(2, 2, 8, 64, 16, dtype=u8), torch.zeros(1, 2)
    Xt, xc, xs = torch.zeros(M, K, dtype=bf), torch.zeros(M, K, dtype=f8), torch.zeros(M, 2)
    Yt = torch.zeros(M, N, dtype=bf)

    def no(match, fn, *a):
        with pytest.raises(ValueError, match=match):
            fn(*a)

    no("device tensors", A.awq_fp8_pack, Wt, codes, scales)
    no("W must be", A.awq_fp8_pack, Wt.float(), codes, scales)
    no("multiple of 16", A.awq_fp8_pack, torch.zeros(40, N, dtype=bf), codes, scales)
    no("codes must", A.awq_fp8_pack, Wt, codes[:1], scales)
    no("codes must", A.awq_fp8_pack, Wt, codes.int(), scales)
    no("scales must", A.awq_fp8_pack, Wt, codes, scales.double())
    no("scales must", A.awq_fp8_pack, Wt, codes, scales[:, :1])
    no("device tensors", A.awq_fp8_quantize, Xt, None, xc, xs)
    no("gate must", A.awq_fp8_quantize, Xt, Xt[:2], xc, xs)
    no("codes must", A.awq_fp8_quantize, Xt, None, xc[:, :128], xs)
    no("scales must", A.awq_fp8_quantize, Xt, None, xc, xs[:, :1])
    no("device tensors", A.awq_fp8_gemm, xc, xs, codes, scales, Yt, None)
    no("xcodes must", A.awq_fp8_gemm, xc.float(), xs, codes, scales, Yt, None)
    no("codes must have shape", A.awq_fp8_gemm, xc[:2], xs, codes, scales, Yt, None)
    no("codes must have shape", A.awq_fp8_gemm, xc, xs, codes, scales, torch.zeros(M, 136, dtype=bf), None)
    no("Y must be", A.awq_fp8_gemm, xc, xs, codes, scales, Yt.float(), None)
    no("channels", A.fp8_gemm, A.Fp8Acts(xc[:, :128], xs), A.Fp8Weights(codes, scales, K, N))

    D, T, Hk, Hq = 64, 16, 2, 4
    k, v, e = torch.zeros(5, Hk, T, D, dtype=f8), torch.zeros(5, Hk, 1, D, 16, dtype=f8), torch.zeros(5, Hk, 2, dtype=u8)
    qkv, q = torch.zeros(M, (Hq + 2 * Hk) * D, dtype=bf), torch.zeros(M, Hq, D, dtype=bf)
    cu, ln, tab, rope, w = (torch.zeros(3, dtype=i32), torch.zeros(2, dtype=i32), torch.zeros(2, 3, dtype=i32),
                            torch.zeros(9, D), torch.ones(D, dtype=bf))
    ok = [qkv, w, w, 1e-5, rope, False, cu, ln, tab, 2, q, k, v, e]

    def swap(i, t):
        return [t if j == i else a for j, a in enumerate(ok)]

    no("device tensors", A.awq_qkv_append, *ok)
    for i, t, match in ((0, qkv[:, :-D], "qkv must"), (0, qkv.float(), "qkv must"), (1, w[:32], "q_weight must"),
                        (2, w.float(), "k_weight must"), (4, rope.double(), "rope must"), (4, rope[0], "rope must"),
                        (6, cu[:2], "cu must"), (6, cu.long(), "cu must"), (7, ln.long(), "length must"),
                        (8, tab.long(), "table must"), (8, tab[0], "table must"), (10, q[..., :32], "q must"),
                        (10, q.float(), "q must"), (11, k[0], "k_codes must"), (11, k.float(), "k_codes must"),
                        (12, v[:, :, :, :32], "v_codes must"), (13, e[:2], "scales must"), (13, e.int(), "scales must")):
        no(match, A.awq_qkv_append, *swap(i, t))
    no("device tensors", A.awq_attention, q, cu, ln, tab, 2, k, v, e, 0.1, True, q.clone(), None)
    no("out must", A.awq_attention, q, cu, ln, tab, 2, k, v, e, 0.1, True, q[:2], None)
    no("q must", A.awq_attention, q[..., :32], cu, ln, tab, 2, k, v, e, 0.1, True, q, None)
    no("no head", A.qkv_append, qkv[:, :4 * D], A.Sequences(cu, ln, tab, 2), type("C", (), dict(k=k, v=v, scales=e)))


def test_max_q_past_32_bits():
    """The foreign call would take 2^32 + 1 as 1 and leave rows out."""
    bf, i32 = torch.bfloat16, torch.int32
    k, v, e = (torch.zeros(5, 2, *s, dtype=torch.uint8) for s in ((16, 64), (1, 64, 16), (2,)))
    q, qkv = torch.zeros(4, 4, 64, dtype=bf), torch.zeros(4, 8 * 64, dtype=bf)
    seqs = torch.zeros(3, dtype=i32), torch.zeros(2, dtype=i32), torch.zeros(2, 3, dtype=i32), (1 << 32) + 1
    with pytest.raises(ValueError, match="max_q"):
        A.awq_qkv_append(qkv, None, None, 1e-5, None, False, *seqs, q, k, v, e)
    with pytest.raises(ValueError, match="max_q"):
        A.awq_attention(q, *seqs, k, v, e, 0.1, True, q.clone(), None)
