"""Sizes whose offsets pass 32 bits, and grids that pass one line of workgroups."""
import numpy as np
import pytest

from dense_util import dev, exact_problem, host
from oracle import dense
from oracle.select import route_select as select_ref

pytestmark = pytest.mark.gpu


def _many(t, n):
    """n rows that repeat t's."""
    import torch

    return t[torch.arange(n, device="cuda") % t.shape[0]]


@pytest.mark.parametrize("M,N", [(70003, 24), (3, 66003), (40, 66003)])
def test_codes_beyond_32_bits(M, N):
    import torch

    import routed_expert_prefill_amd as rep

    K, p = 65536, 5  # sums up to 9 * K * 4 quarters: exact
    q, xs, w, ws = exact_problem(1, min(M, 37), min(N, 128 * p), K)
    want = dense.matmul(q, xs, w, ws)
    dq, dxs, dw, dws = dev(q, xs, w, ws)
    big_q, big_s = (_many(dq, M), _many(dxs, M)) if M > 37 else (dq, dxs)
    big_w, big_ws = (_many(dw, N), _many(dws, -(-N // 128))) if N > 128 * p else (dw, dws)
    assert max(big_q.numel(), big_w.numel()) > 1 << 32
    got = rep.matmul_fp8((big_q, big_s), big_w, big_ws)
    ref = torch.from_numpy(want).float().cuda()
    ref = ref[torch.arange(M, device="cuda") % ref.shape[0]][:, torch.arange(N, device="cuda") % ref.shape[1]]
    assert torch.equal(got, ref)


def test_rows_beyond_32_bits_are_quantised():
    import torch

    import routed_expert_prefill_amd as rep

    x = torch.randn(53, 65536, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).cuda()
    big = _many(x, 66001)
    q, s = rep.quant_blocks_fp8(big)
    assert q.numel() > 1 << 32
    want = rep.quant_blocks_fp8(x)
    for at in (0, 32768, 65536, 66001 - 53):
        rows = torch.arange(at, at + 53, device="cuda")
        assert torch.equal(q[at:at + 53], want[0][rows % 53]) and torch.equal(s[at:at + 53], want[1][rows % 53])


def test_more_tiles_than_a_line():
    import torch

    import routed_expert_prefill_amd as rep

    M = (1 << 27) + 70  # of 32 rows, 2^22 and a few
    q, xs, w, ws = exact_problem(2, 96, 1, 128)
    want = torch.from_numpy(dense.matmul(q, xs, w, ws)).to(torch.bfloat16).cuda()
    dq, dxs, dw, dws = dev(q, xs, w, ws)
    got = rep.matmul_fp8((_many(dq, M), _many(dxs, M)), dw, dws, out_dtype=torch.bfloat16)
    for at in (0, (1 << 27) - 96, M - 96):
        assert torch.equal(got[at:at + 96], want[torch.arange(at, at + 96, device="cuda") % 96]), at
    assert not torch.isnan(got.float().sum())


def test_more_tokens_than_a_line():
    import torch

    import routed_expert_prefill_amd as rep

    T = (1 << 24) + 9  # four tokens to a workgroup
    z = np.random.default_rng(3).standard_normal((50, 8)).astype(np.float32)
    ids, w = rep.route_select(_many(dev(z)[0], T), 2, groups=2, top_groups=1)
    ri, rw = select_ref(z, 2, groups=2, top_groups=1)
    for at in (0, (1 << 24) - 45, T - 50):
        rows = np.arange(at, at + 50) % 50
        assert np.array_equal(ids[at:at + 50].cpu().numpy(), ri[rows])
        assert np.allclose(host(w[at:at + 50]), rw[rows], rtol=2.0 ** -23, atol=0)
