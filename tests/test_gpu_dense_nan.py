"""NaN and infinities of one row through block quantisation, the 8-bit product and the
shared expert: the row is NaN where the formulas are, other rows keep their bits."""
import numpy as np
import pytest

from dense_util import dev, random_problem
from oracle import dense, numerics as nx

pytestmark = pytest.mark.gpu
NAN, INF = float("nan"), float("inf")


@pytest.mark.parametrize("wide", [False, True])
def test_blocks_without_a_number(wide):
    """NaN alone or among zeros: the scale is 1, a NaN's code NaN, a zero's a zero."""
    import torch

    import routed_expert_prefill_amd as rep

    x = torch.randn(23, 256, generator=torch.Generator().manual_seed(3))
    x[0] = NAN
    x[1, :128] = NAN
    x[2, :128] = 0.0
    x[2, 5] = NAN
    x[3, 128:] = -0.0
    x[3, 255] = -NAN
    x[5, 128:] = 0.0
    x[5, 128:136] = NAN  # one lane's elements
    x[7] = 0.0
    x[22, 1::2] = NAN
    x[22, ::2] = 0.0
    x = x if wide else x.to(torch.bfloat16)
    q, s = (t.cpu().numpy() for t in rep.quant_blocks_fp8(x.cuda()))
    v = x.float().numpy().reshape(-1, 128)
    q, s = q.reshape(-1, 128), s.reshape(-1)
    nan = np.isnan(v)
    assert np.array_equal(q & 0x7F == 0x7F, nan)
    none = nan.any(1)
    assert (s[none] == 1).all() and not (q[none] & 0x7F)[~nan[none]].any()
    rq, rs = dense.quant_blocks(v[~none])
    assert np.array_equal(q[~none], rq) and np.array_equal(s[~none], rs[:, 0])


@pytest.mark.parametrize("M", [1, 3, 16, 40, 300])
@pytest.mark.parametrize("N,K", [(140, 256), (512, 1152)])
def test_a_row_of_a_product(M, N, K):
    import torch

    import routed_expert_prefill_amd as rep

    _, _, w, ws = random_problem(N, 1, N, K)
    dw, dws = dev(w, ws)
    x = torch.randn(M, K, generator=torch.Generator().manual_seed(M)).to(torch.bfloat16)
    for dtype in (torch.float32, torch.bfloat16):
        want = rep.matmul_fp8(x.cuda(), dw, dws, out_dtype=dtype)
        assert torch.isfinite(want).all()
        keep = torch.arange(M) != M // 2
        for bad in (lambda r: r.fill_(NAN), lambda r: r[128:].fill_(NAN), lambda r: r[3:4].fill_(NAN),
                    lambda r: r[K - 1:].fill_(INF)):
            y = x.clone()
            bad(y[M // 2])
            got = rep.matmul_fp8(y.cuda(), dw, dws, out_dtype=dtype)
            assert torch.isnan(got[M // 2]).all()
            assert torch.equal(got[keep], want[keep])


# few rows with codes of h made on the way; h in fp32 in tiles of 32 x 64, 64 x 64 and
# 64 x 128; codes of h from tiles of 64 x 256 and 128 x 256
SHARED = [(1, 256, 384), (5, 1024, 256), (16, 2048, 128), (40, 2048, 128), (256, 512, 1152),
          (401, 640, 1280), (33, 256, 256), (300, 128, 256), (2049, 256, 1152)]


@pytest.mark.parametrize("T,d,f", SHARED)
def test_a_row_of_the_shared_expert(T, d, f):
    """One NaN (or infinity) of x makes g and u NaN in all features, and so out."""
    import torch

    import routed_expert_prefill_amd as rep

    parts = [random_problem(i, 1, n, k)[2:] for i, (n, k) in enumerate(((f, d), (f, d), (d, f)))]
    W = [w for w, _ in parts] + [s for _, s in parts]
    x = torch.randn(T, d, generator=torch.Generator().manual_seed(T)).to(torch.bfloat16)
    q, xs = dense.quant_blocks(x.float().numpy())
    at, keep = T // 2, torch.arange(T) != T // 2
    dW = dev(*W)
    for dtype in (torch.float32, torch.bfloat16):
        want = rep.shared_ffn(x.cuda(), *dW, out_dtype=dtype)
        want_codes = rep.shared_ffn(tuple(dev(q, xs)), *dW, out_dtype=dtype)
        assert torch.isfinite(want).all()
        for value in (NAN, INF):
            y = x.clone()
            y[at, d - 1] = value
            got = rep.shared_ffn(y.cuda(), *dW, out_dtype=dtype)
            assert torch.isnan(got[at]).all() and torch.equal(got[keep], want[keep])
        for code, scale in ((0x7F, None), (0xFF, None), (None, np.nan)):
            q2, xs2 = q.copy(), xs.copy()
            if code is not None:
                q2[at, 1] = code
            else:
                xs2[at, 0] = scale
            got = rep.shared_ffn(tuple(dev(q2, xs2)), *dW, out_dtype=dtype)
            assert torch.isnan(got[at]).all() and torch.equal(got[keep], want_codes[keep])


def test_a_block_of_h_without_a_number():
    """A NaN scale of one block of gate rows: h's block is NaN in every row, out too."""
    import torch

    import routed_expert_prefill_amd as rep

    for T, d, f in ((1, 256, 256), (40, 2048, 256), (33, 256, 256), (2049, 256, 1152)):
        parts = [random_problem(i, 1, n, k)[2:] for i, (n, k) in enumerate(((f, d), (f, d), (d, f)))]
        W = [w for w, _ in parts] + [s.copy() for _, s in parts]
        W[3][1, 0] = np.nan
        x = torch.randn(T, d, generator=torch.Generator().manual_seed(T)).to(torch.bfloat16).cuda()
        assert torch.isnan(rep.shared_ffn(x, *dev(*W))).all(), T
    assert nx.e4m3_decode(np.uint8([0x7F]))[0] != 0
