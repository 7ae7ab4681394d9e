"""The microscaled operators together, as a decoder block uses them: an AWQ search gives the input
scales, weights are packed with them, the norm (with the residual) writes quantized activations divided
by them, and the product reads both; the gated quantizer feeds the last layer.  Also on other streams
and in captured graphs."""
import numpy as np
import pytest
import torch

from oracle import mx_oracle as O
from tests.mx_util import A, DEV, bf16, check_product, dev, f32, host_acts, rows
from weight_only_int4_act_amd import inputs as I

pytestmark = pytest.mark.gpu

K, F, T = 512, 1024, 256


def layers(seed=0):
    rng = np.random.default_rng(seed)
    w = lambda k, n: dev(bf16(rng.standard_normal((k, n)) / np.sqrt(k)))   # noqa: E731
    return {"qkv": w(K, 3 * K), "gate_up": w(K, 2 * F), "down": w(F, K), "norm1": dev(bf16(1 + 0.1 * rng.standard_normal(K))),
            "norm2": dev(bf16(1 + 0.1 * rng.standard_normal(K)))}


def pack_with_search(X, W):
    """The input scales of the framework's search over the layer, and its MX weights under them."""
    cfg = A.qconfig(128, True, 21)
    s = A.run_layer(X, W, cfg)["q"].s
    return A.mx_pack(W, s)


def block(h, r, L, q, bits):
    """norm -> q|k|v; norm -> gate|up -> gated -> down.  Returns every intermediate."""
    out = {}
    out["a1"], out["r1"] = A.rms_norm(h, L["norm1"], residual=r, s=q["qkv"].s, bits=bits)
    out["y1"] = A.mx_gemm(out["a1"], q["qkv"])
    att = out["y1"][:, :K].contiguous()                    # stands in for attention's output
    out["att"] = att
    out["a2"], out["r2"] = A.rms_norm(att, L["norm2"], residual=out["r1"], s=q["gate_up"].s, bits=bits)
    out["y2"] = A.mx_gemm(out["a2"], q["gate_up"])
    out["g"], out["u"] = out["y2"][:, :F].contiguous(), out["y2"][:, F:].contiguous()
    out["a3"] = A.mx_quantize(out["u"], q["down"].s, bits, gate=out["g"])
    out["y3"] = A.mx_gemm(out["a3"], q["down"])
    return out


@pytest.fixture(scope="module")
def packed():
    L = layers()
    X = dev(rows(T, K, 1))
    XF = dev(rows(T, F, 2))
    return L, {"qkv": pack_with_search(X, L["qkv"]), "gate_up": pack_with_search(X, L["gate_up"]),
               "down": pack_with_search(XF, L["down"])}


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("M", [1, 5, 130])
def test_block_against_float64(packed, M, bits):
    L, q = packed
    out = block(dev(rows(M, K, 3)), dev(rows(M, K, 4)), L, q, bits)
    torch.cuda.synchronize()
    for a, y, name in (("a1", "y1", "qkv"), ("a2", "y2", "gate_up"), ("a3", "y3", "down")):
        c, E, b = host_acts(out[a].codes, out[a].scales)
        w = O.weights_values(q[name].codes.cpu().numpy(), q[name].scales.view(torch.uint8).cpu().numpy(), q[name].K,
                             q[name].N)
        check_product(out[y], O.values(c, E, b), w, bits, (name, M, bits))
    # the chain's own error against unquantized float64: the formats' rounding, at most 2^-4 (e4m3) or
    # 2^-2 (e2m1) per element, random in sign; a wrong scale or layer would show as an error of order one
    x = f32(out["u"]).astype(np.float64)
    p = O.gated(x, f32(out["g"]).astype(np.float64))
    y = p @ f32(L["down"]).astype(np.float64)
    err = np.linalg.norm(f32(out["y3"]) - y) / np.linalg.norm(y)
    assert err < 0.5, err


def test_on_another_stream(packed):
    L, q = packed
    h, r = dev(rows(9, K, 3)), dev(rows(9, K, 4))
    ref = block(h, r, L, q, 8)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = block(h, r, L, q, 8)
    side.synchronize()
    assert torch.equal(ref["y3"], got["y3"]) and torch.equal(ref["r2"], got["r2"])
    # the helpers' own stream argument: their outputs and workspaces belong to that stream
    a, _ = A.rms_norm(h, L["norm1"], residual=r, s=q["qkv"].s, stream=side)
    y = A.mx_gemm(a, q["qkv"], stream=side)
    side.synchronize()
    assert torch.equal(y, ref["y1"])


@pytest.mark.parametrize("M", [1, 13, 130])
def test_captured_and_replayed(packed, M):
    """The block in one graph, replayed with new inputs between eager calls: every replay equals the
    eager result.  Two graphs share the workspaces, as calls on one stream may."""
    L, q = packed
    h, r = dev(rows(M, K, 3)), dev(rows(M, K, 4))
    n = max(A.awq_mx_gemm_workspace_size(M, w.K, w.N, 8) for w in q.values())
    ws = A.workspace(n, DEV)
    ac = {k: (torch.empty((M, k), dtype=torch.float8_e4m3fn, device=DEV),
              torch.empty((M, k // 32), dtype=torch.uint8, device=DEV)) for k in (K, F)}
    Y = {w: torch.empty((M, q[w].N), dtype=torch.bfloat16, device=DEV) for w in q}
    ro = torch.empty_like(h)

    def step():
        A.awq_rms_norm(h, r, L["norm1"], 1e-5, ro, None, q["qkv"].s, *ac[K])
        A.awq_mx_gemm(*ac[K], q["qkv"].codes, q["qkv"].scales, Y["qkv"], ws)
        A.awq_mx_gemm(*ac[K], q["gate_up"].codes, q["gate_up"].scales, Y["gate_up"], ws)
        up, gate = Y["gate_up"][:, :F].contiguous(), Y["gate_up"][:, F:].contiguous()
        A.awq_mx_quantize(up, gate, q["down"].s, *ac[F])
        A.awq_mx_gemm(*ac[F], q["down"].codes, q["down"].scales, Y["down"], ws)

    step()
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step()
        graphs.append(g)
    for i in range(4):
        h.copy_(rows(M, K, 10 + i))
        r.copy_(rows(M, K, 20 + i))
        step()
        want = {k: v.clone() for k, v in Y.items()} | {"ro": ro.clone()}
        torch.cuda.synchronize()
        for g in graphs:
            for t in (*Y.values(), ro):
                t.fill_(float("nan"))
            g.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(want[k], v) for k, v in {**Y, "ro": ro}.items()), i


def test_two_streams_at_once(packed):
    """Calls on two streams with their own outputs and workspaces."""
    L, q = packed
    ins = [(dev(rows(33, K, 30 + i)), dev(rows(33, K, 40 + i))) for i in range(2)]
    want = [block(h, r, L, q, 8)["y3"] for h, r in ins]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in ins]
    got = []
    for _ in range(5):
        got = []
        for st, (h, r) in zip(streams, ins):
            with torch.cuda.stream(st):
                got.append(block(h, r, L, q, 8)["y3"])
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, got))
