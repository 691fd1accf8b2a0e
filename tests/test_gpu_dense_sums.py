"""Sums of the 8-bit products are fp32's whatever the result's type, unless the caller
asks for short ones.

Two columns, or features of h, of the largest products there are (448 * 448, 2^17.6)
cancel in every result; what is left is the sum of the others, small whole numbers.
All partial sums are whole numbers, in quarters, below 2^22: exact in fp32 in any
order, so that bf16 results are the exact ones rounded once."""
import numpy as np
import pytest

from dense_util import U, bf16_room, dev, exact_problem, host, product_room, random_problem
from oracle import dense, numerics as nx

pytestmark = pytest.mark.gpu


def _cancelling(seed, M, N, K):
    q, xs, w, ws = exact_problem(seed, M, N, K)
    top = nx.e4m3_encode(np.array([448.0, -448.0]))
    at = K // 2
    q[:, at] = q[:, at + 40] = top[0]
    w[:, at], w[:, at + 40] = top
    return q, xs, w, ws


SIZES = [(1, 64, 512), (16, 200, 512), (17, 200, 512), (40, 2048, 256), (129, 1416, 384),
         (300, 516, 896), (777, 1416, 1152), (2049, 2500, 256)]


@pytest.mark.parametrize("M,N,K", SIZES)
def test_small_products_beside_large_ones(M, N, K):
    import torch

    import routed_expert_prefill_amd as rep

    p = _cancelling(M + N, M, N, K)
    want = dense.matmul(*p)
    q, xs, w, ws = dev(*p)
    assert np.array_equal(host(rep.matmul_fp8((q, xs), w, ws)), want)
    assert np.array_equal(host(rep.matmul_fp8((q, xs), w, ws, out_dtype=torch.bfloat16)), nx.bf16_round(want))


@pytest.mark.parametrize("M,N,K", [(7, 1000, 2048), (40, 2048, 4096), (777, 1416, 1152), (2500, 1030, 384)])
def test_bf16_results_are_the_sums_rounded_once(M, N, K):
    import torch

    import routed_expert_prefill_amd as rep

    p = random_problem(M + N, M, N, K)
    want, total = dense.matmul(*p), dense.matmul_abs(*p)
    q, xs, w, ws = dev(*p)
    low = host(rep.matmul_fp8((q, xs), w, ws, out_dtype=torch.bfloat16))
    room = product_room(K, total)
    assert (np.abs(low - want) <= room + 2.0 ** -8 * (np.abs(want) + room)).all()


@pytest.mark.parametrize("T,d,f", [(3, 256, 256), (40, 2048, 128), (300, 256, 256), (777, 512, 256)])
def test_the_shared_experts_down_product(T, d, f):
    """Two features of h are equal and the largest; down's weights of them cancel."""
    import torch

    import routed_expert_prefill_amd as rep

    wg, wu, wd = (random_problem(i, 1, n, k)[2] for i, (n, k) in enumerate(((f, d), (f, d), (d, f))))
    sg, su, sd = (np.full((-(-n // 128), k // 128), 2.0 ** -11, np.float32) for n, k in ((f, d), (f, d), (d, f)))
    wu[60] = nx.e4m3_encode(nx.e4m3_decode(wu[60]) * 0 + 448)
    wg[60] = wu[60]
    wg[100], wu[100] = wg[60], wu[60]
    wd[:, 60], wd[:, 100] = nx.e4m3_encode(np.array([448.0, -448.0]))
    x = np.abs(np.random.default_rng(T).standard_normal((T, d))).astype(np.float32)
    q, xs = dense.quant_blocks(x)
    args = [tuple(dev(q, xs)), *dev(wg, wu, wd, sg, su, sd)]
    wide = host(rep.shared_ffn(*args))
    low = host(rep.shared_ffn(*args, out_dtype=torch.bfloat16))
    h = np.abs(dense.shared_hidden(q, xs, wg, wu, sg, su))
    total = h * (1 + 2.0 ** -3) @ np.abs(dense.weight_values(wd, sd)).T  # a code is half a step off, 2^-4
    room = 2 * product_room(f, total)
    assert (np.abs(low - wide) <= room + 2.0 ** -8 * (np.abs(wide) + room)).all()


@pytest.mark.parametrize("M,N,K", [(5, 300, 512), (40, 2048, 256), (300, 516, 896), (777, 1416, 1152), (2049, 2500, 256)])
def test_short_sums(M, N, K):
    """Exact where the products of eight columns lie near each other, within the bound
    of 13 bits elsewhere; refused for fp32 results."""
    import torch

    import routed_expert_prefill_amd as rep

    p = exact_problem(M, M, N, K)
    q, xs, w, ws = dev(*p)
    kw = dict(out_dtype=torch.bfloat16, short_sums=True)
    out = torch.full((M + 2, N), 7.0, dtype=torch.bfloat16, device="cuda")
    assert rep.matmul_fp8((q, xs), w, ws, out=out[:M], short_sums=True).data_ptr() == out.data_ptr()
    assert np.array_equal(host(out[:M]), nx.bf16_round(dense.matmul(*p))) and (out[M:] == 7).all()
    p = random_problem(M + N, M, N, K)
    want, total = dense.matmul(*p), dense.matmul_abs(*p)
    q, xs, w, ws = dev(*p)
    low = host(rep.matmul_fp8((q, xs), w, ws, **kw))
    assert (np.abs(low - want) <= bf16_room(K, total, want)).all()
    # rows in bf16
    x = torch.randn(M, K, generator=torch.Generator().manual_seed(M)).to(torch.bfloat16).cuda()
    a, b = rep.matmul_fp8(x, w, ws, **kw), rep.matmul_fp8(rep.quant_blocks_fp8(x), w, ws, **kw)
    cq, cs = (t.cpu().numpy() for t in rep.quant_blocks_fp8(x))
    want, total = dense.matmul(cq, cs, *p[2:]), dense.matmul_abs(cq, cs, *p[2:])
    for got in (a, b):
        assert (np.abs(host(got) - want) <= bf16_room(K, total, want)).all()
    for bad in (dict(), dict(out_dtype=torch.float32), dict(out=torch.empty(M, N, device="cuda"))):
        with pytest.raises(ValueError, match="short_sums"):
            rep.matmul_fp8((q, xs), w, ws, **{**bad, "short_sums": True})


@pytest.mark.parametrize("T,d,f", [(3, 256, 256), (300, 256, 256), (1030, 640, 256)])
def test_short_sums_of_the_shared_expert(T, d, f):
    import torch

    import routed_expert_prefill_amd as rep

    wg, wu, wd = (random_problem(i, 1, n, k)[2] for i, (n, k) in enumerate(((f, d), (f, d), (d, f))))
    sg, su, sd = (np.full((n // 128, k // 128), 2.0 ** -9, np.float32) for n, k in ((f, d), (f, d), (d, f)))
    x = torch.randn(T, d, generator=torch.Generator().manual_seed(T)).to(torch.bfloat16).cuda()
    W = dev(wg, wu, wd, sg, su, sd)
    wide = host(rep.shared_ffn(x, *W))
    low = host(rep.shared_ffn(x, *W, out_dtype=torch.bfloat16, short_sums=True))
    q, xs = (t.cpu().numpy() for t in rep.quant_blocks_fp8(x))
    h = np.abs(dense.shared_hidden(q, xs, wg, wu, sg, su))
    total = h * (1 + 2.0 ** -3) @ np.abs(dense.weight_values(wd, sd)).T
    assert (np.abs(low - wide) <= product_room(f, total) + bf16_room(f, total, np.abs(wide) + U * total)).all()
    with pytest.raises(ValueError, match="short_sums"):
        rep.shared_ffn(x, *W, short_sums=True)


def test_no_rows_and_the_entry_points():
    import ctypes

    import torch

    import routed_expert_prefill_amd as rep
    from routed_expert_prefill_amd import _lib

    q, xs, w, ws = dev(*exact_problem(1, 3, 140, 256))
    got = rep.matmul_fp8((q[:0], xs[:0]), w, ws, out_dtype=torch.bfloat16, short_sums=True)
    assert got.shape == (0, 140) and got.dtype == torch.bfloat16
    y = torch.zeros(3, 140, device="cuda")
    lib = _lib.load()
    for kind in (_lib.MOE_DT_F32 | _lib.MOE_SHORT_SUMS, _lib.MOE_SHORT_SUMS << 1, 2):
        rc = lib.moe_matmul_fp8(q.data_ptr(), xs.data_ptr(), 3, 140, 256, w.data_ptr(), ws.data_ptr(),
                                y.data_ptr(), kind, None, 0, ctypes.c_void_p(0))
        assert rc == _lib.MOE_EUNSUPPORTED
    torch.cuda.synchronize()
    assert not y.any()
