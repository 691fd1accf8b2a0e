"""Zeros of both signs, and numbers whose codes are zeros, in blocks that are not all
zeros: a code keeps its element's sign, as the rule and the row quantisation have it."""
import numpy as np
import pytest

from oracle import dense, numerics as nx

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("scale", [1.0, 1e-4, 3e7, 2.0 ** -100])
def test_signs_of_zeros(wide, scale):
    import torch

    import routed_expert_prefill_amd as rep

    x = torch.randn(9, 384, generator=torch.Generator().manual_seed(5)) * scale
    x[:, ::3] = -0.0
    x[:, 1::9] = 0.0
    x[1:, 4::7] = -1e-9 * scale
    x[2:, 7::11] = 2.0 ** -126
    x[2:, 8::13] = -2.0 ** -126
    if wide:
        x[3:, 10::17] = -1e-45
    x[8, :128] = -0.0
    x = x if wide else x.to(torch.bfloat16)
    q, s = rep.quant_blocks_fp8(x.cuda())
    rq, rs = dense.quant_blocks(x.float().numpy())
    assert np.array_equal(s.cpu().numpy(), rs) and np.array_equal(q.cpu().numpy(), rq)
    assert (rq == 0x80).any() and (rq == 0).any()
    if not wide:
        q2, s2 = rep.quant_rows_fp8(x.cuda().view(-1, 128))
        assert torch.equal(q2.view(q.shape), q) and torch.equal(s2.view(s.shape), s)
    assert nx.e4m3_decode(np.uint8([0x80]))[0] == 0
