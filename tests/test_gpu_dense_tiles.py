"""Every kernel of the 8-bit products and the shared expert, at sizes that fill no tile:
one block of columns, a few, and more than 64 stages (whose weight scales are loaded a
second time).  Products are exact (dense_util.exact_problem: whole numbers in quarters
below 2^24 up to the most columns here, 65,664), in fp32, bf16 and with short sums; the
shared expert is held to the bounds of test_gpu_dense.py."""
import numpy as np
import pytest

from dense_tiles import PRODUCTS, SHARED, SHORT, columns
from dense_util import bf16_room, dev, exact_problem, host, two_powers, whole_codes
from oracle import dense, numerics as nx
from test_gpu_dense import _shared_bounds

pytestmark = pytest.mark.gpu

ROWS = 67  # different rows of x; the others repeat them


@pytest.mark.parametrize("mode", ["f32", "bf16", "short"])
@pytest.mark.parametrize("tile", list(SHORT))
def test_product(mode, tile):
    import torch

    import routed_expert_prefill_amd as rep

    if mode != "short" and tile not in PRODUCTS:
        return  # these tiles are for short sums alone
    M, N = SHORT[tile]
    kw = {"f32": dict(out_dtype=torch.float32), "bf16": dict(out_dtype=torch.bfloat16),
          "short": dict(out_dtype=torch.bfloat16, short_sums=True)}[mode]
    for K in columns(tile):
        print(mode, tile, K, flush=True)
        q, xs, w, ws = exact_problem(M + K, min(M, ROWS), N, K)
        assert 9 * K * 4 * 4 < 1 << 24
        dq, dxs, dw, dws = dev(q, xs, w, ws)
        want = torch.from_numpy(dense.matmul(q, xs, w, ws)).cuda().to(kw["out_dtype"])
        at = torch.arange(M, device="cuda") % ROWS
        out = torch.full((M + 1, N), 7.0, dtype=kw["out_dtype"], device="cuda")
        rep.matmul_fp8((dq[at], dxs[at]), dw, dws, out=out[:M], short_sums=mode == "short")
        assert torch.equal(out[:M], want[at]), K
        assert (out[M:] == 7).all()


@pytest.mark.parametrize("T,d,f", [s for sizes in SHARED.values() for s in sizes])
def test_shared(T, d, f):
    import torch

    import routed_expert_prefill_amd as rep

    rng = np.random.default_rng(T + d)
    u = min(T, ROWS)
    q, xs = whole_codes(rng, (u, d)), two_powers(rng, (u, d // 128))
    wg, wu, wd = whole_codes(rng, (f, d)), whole_codes(rng, (f, d)), whole_codes(rng, (d, f))
    small = np.float32(2.0 ** -round(np.log2(8 * d ** 0.5)))  # |g| up to about 16
    sg, su = (two_powers(rng, (f // 128, d // 128)) * small for _ in range(2))
    sd = (rng.random((d // 128, f // 128)) + 0.5).astype(np.float32)
    p = (q, xs, wg, wu, wd, sg, su, sd)
    want, room, either, total = _shared_bounds(*p)
    assert either.mean() < 0.05  # few codes lie next to a midpoint: the test tells
    dq, dxs, *W = dev(*p)
    at = torch.arange(T, device="cuda") % ROWS
    rows = (dq[at], dxs[at])
    out = torch.full((T + 2, d), 7.0, device="cuda")
    rep.shared_ffn(rows, *W, out=out[:T])
    assert (out[T:] == 7).all()
    assert torch.equal(out[:T], out[:u][at])  # a row's result depends on no other
    off = np.abs(host(out[:u]) - want)
    assert (off <= room).all(), (off / room).max()
    for short in (False, True):
        low = rep.shared_ffn(rows, *W, out_dtype=torch.bfloat16, short_sums=short)
        assert torch.equal(low, low[:u][at])
        slack = bf16_room(f, total, want) if short else 2.0 ** -8 * (np.abs(want) + room)
        assert (np.abs(host(low[:u]) - want) <= room + slack).all()
    assert nx.e4m3_decode(np.uint8([0x38]))[0] == 1
