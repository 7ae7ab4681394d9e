"""Refusals of the microscaled operators, on the host: the C entry points reject bad arguments
before anything is enqueued and write nothing, and the binding refuses what the C ABI cannot see."""
import ctypes

import pytest
import torch

from weight_only_int4_act_amd import awq as A

P = lambda v: ctypes.c_void_p(v)   # noqa: E731  never dereferenced: every call below is rejected first
BIG = ctypes.c_size_t(1 << 40)
INV, UNS, WS = A.AWQ_ERR_INVALID_ARG, A.AWQ_ERR_UNSUPPORTED, A.AWQ_ERR_WORKSPACE
L = A.library()
X, G, W, C, S, Y, R, V, F = (P(0x100000000 * (i + 1)) for i in range(9))   # far apart


def test_packed_sizes():
    assert A.awq_mx_codes_bytes(4096, 4096) == 4096 * 4096 // 2
    assert A.awq_mx_scales_bytes(4096, 4096) == 4096 * 4096 // 32
    assert A.awq_mx_codes_bytes(96, 65) == 2 * 4 * 64 * 16 and A.awq_mx_scales_bytes(96, 65) == 2 * 4 * 64
    for K, N in ((0, 8), (32, 0), (33, 8), (-32, 8), (1 << 40, 8), (32, 1 << 40), (1 << 23, 1 << 20)):
        assert A.awq_mx_codes_bytes(K, N) == 0 and A.awq_mx_scales_bytes(K, N) == 0, (K, N)


def test_gemm_workspace_size():
    for M, K, N, bits in ((0, 64, 8, 8), (1, 48, 8, 8), (1, 64, 0, 8), (1, 64, 8, 16), (65535 * 16 + 1, 64, 8, 8),
                          (1 << 62, 64, 8, 8), (1, 1 << 62, 8, 8), (1, 64, 1 << 62, 8)):
        assert A.awq_mx_gemm_workspace_size(M, K, N, bits) == 0, (M, K, N, bits)


def test_pack_and_unpack():
    for W_, K, N, C_, S_ in ((None, 64, 8, C, S), (W, 64, 8, None, S), (W, 64, 8, C, None), (W, 0, 8, C, S),
                             (W, 48, 8, C, S), (W, 64, 0, C, S), (W, 64, -1, C, S), (P(0x10001), 64, 8, C, S),
                             (W, 64, 8, P(0x10008), S), (W, 64, 8, C, P(0x10004)), (W, 1 << 40, 8, C, S),
                             (W, 64, 8, W, S), (W, 64, 8, C, W), (W, 64, 8, C, C)):
        assert L.awq_mx_pack(W_, K, N, None, C_, S_, None) == INV, (W_, K, N, C_, S_)
        if not (C_ is S_):
            assert L.awq_mx_unpack(C_, S_, K, N, None, W_, None) == INV, (W_, K, N, C_, S_)
    assert L.awq_mx_pack(W, 64, 8, P(0x10002), C, S, None) == INV           # s misaligned
    assert L.awq_mx_pack(W, 64, 8, C, C, S, None) == INV                    # s overlaps the codes


def test_quantize():
    ok = dict(X=X, g=None, M=3, K=64, s=None, bits=8, C=C, S=S)
    for bad, st in ((dict(X=None), INV), (dict(C=None), INV), (dict(S=None), INV), (dict(M=0), INV), (dict(K=40), INV),
                    (dict(M=1 << 40), INV), (dict(K=1 << 40), INV), (dict(bits=16), UNS), (dict(bits=0), UNS),
                    (dict(X=P(0x10008)), INV), (dict(g=P(0x10008)), INV), (dict(s=P(0x10004)), INV),
                    (dict(C=P(0x10008)), INV), (dict(C=X), INV), (dict(S=X), INV), (dict(g=C), INV), (dict(S=C), INV),
                    (dict(s=C), INV)):
        a = {**ok, **bad}
        assert L.awq_mx_quantize(a["X"], a["g"], a["M"], a["K"], a["s"], a["bits"], a["C"], a["S"], None) == st, bad


def test_rms_norm():
    ok = dict(X=X, r=R, w=W, M=3, K=64, eps=1e-5, ro=V, Y=Y, s=F, bits=8, C=C, S=S)
    for bad, st in ((dict(X=None), INV), (dict(w=None), INV), (dict(Y=None, C=None, S=None, s=None), INV),
                    (dict(C=None), INV), (dict(S=None), INV), (dict(r=None), INV), (dict(C=None, S=None), INV),
                    (dict(M=0), INV), (dict(K=0), INV), (dict(K=40), INV), (dict(K=36, C=None, S=None, s=None), INV),
                    (dict(eps=0.0), INV), (dict(eps=-1.0), INV), (dict(eps=float("nan")), INV),
                    (dict(eps=float("inf")), INV), (dict(bits=5), UNS), (dict(X=P(0x10008)), INV),
                    (dict(r=P(0x10008)), INV), (dict(w=P(0x10008)), INV), (dict(ro=P(0x10008)), INV),
                    (dict(Y=P(0x10008)), INV), (dict(s=P(0x10004)), INV), (dict(C=P(0x10008)), INV),
                    (dict(ro=Y), INV), (dict(Y=P(X.value + 64)), INV), (dict(ro=P(R.value + 64)), INV),
                    (dict(Y=W), INV), (dict(C=X), INV), (dict(S=R), INV), (dict(C=Y), INV), (dict(S=C), INV),
                    (dict(ro=X, Y=X), INV)):
        a = {**ok, **bad}
        got = L.awq_rms_norm(a["X"], a["r"], a["w"], a["M"], a["K"], a["eps"], a["ro"], a["Y"], a["s"], a["bits"],
                             a["C"], a["S"], None)
        assert got == st, (bad, got)


def test_gemm():
    ok = dict(C=C, S=S, bits=8, M=3, w=W, F=F, K=4096, N=4096, Y=Y, ws=V, n=BIG)
    for bad, st in ((dict(C=None), INV), (dict(S=None), INV), (dict(w=None), INV), (dict(F=None), INV),
                    (dict(Y=None), INV), (dict(M=0), INV), (dict(M=65535 * 16 + 1), INV), (dict(K=40), INV),
                    (dict(N=12), INV), (dict(N=0), INV), (dict(bits=6), UNS), (dict(C=P(0x10008)), INV),
                    (dict(w=P(0x10008)), INV), (dict(F=P(0x10008)), INV), (dict(Y=P(0x10008)), INV), (dict(Y=C), INV),
                    (dict(Y=W), INV), (dict(Y=F), INV), (dict(Y=S), INV)):
        a = {**ok, **bad}
        got = L.awq_mx_gemm(a["C"], a["S"], a["bits"], a["M"], a["w"], a["F"], a["K"], a["N"], a["Y"], a["ws"], a["n"],
                            None)
        assert got == st, (bad, got)
    for M in (1, 3, 100, 1000):
        need = A.awq_mx_gemm_workspace_size(M, 4096, 4096, 8)
        if need:
            a = ok
            call = lambda ws, n: L.awq_mx_gemm(C, S, 8, M, W, F, 4096, 4096, Y, ws, n, None)   # noqa: E731
            assert call(V, need - 1) == WS and call(None, need) == WS
            assert call(P(V.value + 16), need) == INV and call(Y, need) == INV and call(W, need) == INV


def test_rejected_calls_write_nothing():
    outs = [(ctypes.c_uint8 * 4096)() for _ in range(4)]
    for b in outs:
        ctypes.memset(b, 0xA5, 4096)
    before = [bytes(b) for b in outs]
    q = [ctypes.cast(b, ctypes.c_void_p) for b in outs]
    st = [L.awq_mx_pack(X, 48, 8, None, q[0], q[1], None), L.awq_mx_unpack(C, S, 48, 8, None, q[0], None),
          L.awq_mx_quantize(X, None, 2, 64, None, 6, q[0], q[1], None),
          L.awq_rms_norm(X, R, W, 2, 64, 0.0, q[0], q[1], None, 8, q[2], q[3], None),
          L.awq_mx_gemm(C, S, 8, 2, W, F, 64, 12, q[0], q[1], BIG, None)]
    assert all(v < 0 for v in st), st
    assert [bytes(b) for b in outs] == before


def test_binding_checks():
    bf, u8, f32 = torch.bfloat16, torch.uint8, torch.float32
    K, N, M = 96, 72, 4
    Wt = torch.zeros(K, N, dtype=bf)
    codes, scales = torch.zeros(2, 4, 64, 16, dtype=u8), torch.zeros(2, 4, 64, dtype=u8)
    Xt, x8, xs = torch.zeros(M, K, dtype=bf), torch.zeros(M, K, dtype=torch.float8_e4m3fn), torch.zeros(M, 3, dtype=u8)
    x4 = torch.zeros(M, K // 2, dtype=u8)
    w, Yt = torch.ones(K, dtype=bf), torch.zeros(M, N, dtype=bf)

    def no(match, fn, *a):
        with pytest.raises(ValueError, match=match):
            fn(*a)

    no("device tensors", A.awq_mx_pack, Wt, None, codes, scales)
    no("device tensors", A.awq_mx_pack, Wt, None, codes, scales.view(torch.float8_e8m0fnu))
    no("W must be", A.awq_mx_pack, Wt.float(), None, codes, scales)
    no("multiple of 32", A.awq_mx_pack, torch.zeros(40, N, dtype=bf), None, codes, scales)
    no("s must", A.awq_mx_pack, Wt, torch.ones(K + 1), codes, scales)
    no("s must", A.awq_mx_pack, Wt, torch.ones(K, dtype=torch.float64), codes, scales)
    no("codes must", A.awq_mx_pack, Wt, None, codes[:1], scales)
    no("scales must", A.awq_mx_unpack, codes, scales.float(), None, Wt)
    no("device tensors", A.awq_mx_quantize, Xt, None, None, x8, xs)
    no("device tensors", A.awq_mx_quantize, Xt, None, None, x4, xs)
    no("activation codes", A.awq_mx_quantize, Xt, None, None, x8.float(), xs)
    no("codes must have shape", A.awq_mx_quantize, Xt, None, None, x8[:, :64], xs)
    no("codes must have shape", A.awq_mx_quantize, Xt, None, None, x8.view(u8), xs)   # 8 bits are float8_e4m3fn
    no("scales must have shape", A.awq_mx_quantize, Xt, None, None, x8, xs[:, :2])
    no("gate must", A.awq_mx_quantize, Xt, Xt[:2], None, x8, xs)
    no("device tensors", A.awq_rms_norm, Xt, None, w, 1e-5, None, Xt)
    no("weight must", A.awq_rms_norm, Xt, None, w.float(), 1e-5, None, Xt)
    no("residual must", A.awq_rms_norm, Xt, Xt[:, :64], w, 1e-5, None, Xt)
    no("given together", A.awq_rms_norm, Xt, None, w, 1e-5, None, None, None, x8, None)
    no("multiple of 8", A.awq_rms_norm, torch.zeros(2, 36, dtype=bf), None, w, 1e-5, None, None)
    no("device tensors", A.awq_mx_gemm, x8, xs, codes, scales, Yt, None)
    no("device tensors", A.awq_mx_gemm, x4, xs, codes, scales, Yt, None)
    no("codes must have shape", A.awq_mx_gemm, x8, xs, codes, scales, torch.zeros(M, 136, dtype=bf), None)
    no("codes must have shape", A.awq_mx_gemm, x8[:2], xs, codes, scales, Yt, None)
    no("Y must be", A.awq_mx_gemm, x8, xs, codes, scales, Yt.float(), None)
    no("8 or 4 bits", A.mx_quantize, Xt, None, 16)
    meta = torch.zeros(M, K, dtype=bf)[:, ::2]
    no("multiple of 32|contiguous|device", A.awq_mx_quantize, meta, None, None, x4, xs)
