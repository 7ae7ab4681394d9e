"""The 8-bit operators where a buffer passes 4 GiB: what lies behind is computed as it would be at the front."""
import numpy as np
import pytest
import torch

from oracle import fp8_oracle as O
from tests.fp8_util import A, DEV, F8, Batch, attend, bf16, check_product, dev, product, u8

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def give_back():
    yield
    torch.cuda.empty_cache()


@pytest.mark.parametrize("lengths", [[(300, 1), (77, 2)], [(300, 60), (40, 40)], [(300, 300)]])
def test_cache(lengths):
    """Blocks from the 33000th on, 128 KiB each, against the same blocks from the first on."""
    Hq, Hk, D, T, off = 32, 8, 128, 128, 33000
    B = Batch(lengths, Hq, Hk, D, T, 1)
    B.upload()
    small = dict(B.d)
    large = {k: torch.empty((off + B.blocks, *small[k].shape[1:]), dtype=torch.uint8, device=DEV) for k in "kvE"}
    for k in "kvE":
        large[k][off:] = small[k].view(torch.uint8)
    assert large["k"].numel() > 1 << 32
    large = dict(small, table=torch.where(small["table"] < 0, -1, small["table"] + off), k=large["k"].view(F8),
                 v=large["v"].view(F8), E=large["E"])
    qkv = dev(bf16(B.rng.standard_normal((B.M, (Hq + 2 * Hk) * D)).astype(np.float32)))
    rope = torch.from_numpy(B.rng.standard_normal((400, D)).astype(np.float32)).to(DEV)
    outs = []
    for d in (small, large):
        q = torch.full((B.M, Hq, D), 3.0, dtype=torch.bfloat16, device=DEV)
        A.awq_qkv_append(qkv, None, None, 1e-6, rope, False, d["cu"], d["length"], d["table"], B.max_q, q, d["k"], d["v"],
                         d["E"])
        B.d = d
        outs.append((q, attend(B, q)))
    assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])
    for k in "kvE":
        assert np.array_equal(u8(small[k]), u8(large[k][off:])), k


def test_activations():
    M, K = 66000, 65552                                      # codes of 4.03 GiB
    x = torch.zeros((M, K), dtype=torch.bfloat16, device=DEV)
    tail = dev(bf16(np.random.default_rng(2).standard_normal((9, K)).astype(np.float32)))
    x[-9:] = tail
    a, b = A.fp8_quantize(x), A.fp8_quantize(tail)
    assert torch.equal(a.codes[-9:].view(torch.uint8), b.codes.view(torch.uint8)) and torch.equal(a.scales[-9:], b.scales)
    assert not a.codes[:-9].view(torch.uint8).any()
    del x
    # and their product with a few columns
    wc, ws_, w = (lambda q: (q.codes, q.scales, q))(A.fp8_pack(dev(bf16(np.random.default_rng(3).standard_normal((K, 8)).astype(np.float32) / 256))))
    Y = product(a.codes, a.scales, wc, ws_, 8)
    assert not Y[:-9].any()
    xs = O.code_value(u8(b.codes)) * O.spread_rows(b.scales.cpu().numpy(), K)
    wv = O.code_value(O.weights_codes(u8(wc), K, 8)) * O.spread_weights(ws_.cpu().numpy(), K, 8)
    check_product(Y[-9:], xs, wv, "activations")


@pytest.mark.parametrize("M", [1, 33, 300])
def test_weights_and_results(M):
    K, N = 8192, 528008                                      # codes of 4.03 GiB
    tail = dev(bf16(np.random.default_rng(4).standard_normal((K, 72)).astype(np.float32) / 64))
    W = torch.zeros((K, N), dtype=torch.bfloat16, device=DEV)
    first = N // 128 * 128 - 64                              # in the last 128 columns but one and the last
    W[:, first:] = tail
    q = A.fp8_pack(W)
    del W
    a = A.fp8_quantize(dev(bf16(np.random.default_rng(5).standard_normal((M, K)).astype(np.float32))))
    Y = product(a.codes, a.scales, q.codes, q.scales, N)
    assert not Y[:, :first].any()
    part = A.Fp8Weights(q.codes[first // 64:], q.scales[first // 128:], K, 72)
    xs = O.code_value(u8(a.codes)) * O.spread_rows(a.scales.cpu().numpy(), K)
    s = np.stack([part.scales[0].cpu().numpy(), part.scales[1].cpu().numpy()])
    codes = O.weights_codes(u8(part.codes), K, 72)
    scale = np.repeat(np.repeat(s, [64, 8], axis=0).T, 128, axis=0)
    check_product(Y[:, first:], xs, O.code_value(codes) * scale, "weights")
    # what was packed there is what packing the columns of each group alone gives
    for lo, hi, at in ((0, 64, first), (64, 72, first + 64)):
        alone = torch.zeros((K, 128), dtype=torch.bfloat16, device=DEV)
        alone[:, at % 128:at % 128 + hi - lo] = tail[:, lo:hi]
        p = A.fp8_pack(alone)
        assert torch.equal(p.scales[0], q.scales[at // 128])
        assert torch.equal(p.codes[at % 128 // 64].view(torch.uint8), q.codes[at // 64].view(torch.uint8))


def test_result_rows():
    M, K, N = 70000, 128, 32768                              # Y of 4.3 GiB
    rng = np.random.default_rng(6)
    x, w = (dev(bf16(rng.standard_normal(s).astype(np.float32))) for s in ((M, K), (K, N)))
    a, q = A.fp8_quantize(x), A.fp8_pack(w)
    Y = product(a.codes, a.scales, q.codes, q.scales, N)
    xs = O.code_value(u8(a.codes[-200:])) * O.spread_rows(a.scales[-200:].cpu().numpy(), K)
    ws_ = O.code_value(O.weights_codes(u8(q.codes), K, N)) * O.spread_weights(q.scales.cpu().numpy(), K, N)
    check_product(Y[-200:], xs, ws_, "rows")
