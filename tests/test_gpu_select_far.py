"""Logits so far below that a sigmoid score is subnormal in fp64: the order and the
gates are still those of the formulas.  A subnormal score of d = 2^-1074 n is off by a
step of 2^-1074 at most, the sum of k of them by k, so a renormalised gate by
(k + 1) / n of itself, and by fp32's rounding."""
import numpy as np
import pytest

from oracle.select import route_select as ref
from gpu_util import np_dev

pytestmark = pytest.mark.gpu


def _both(z, k, **kw):
    import torch

    import routed_expert_prefill_amd as rep

    bias = kw.pop("bias", None)
    ids, w = rep.route_select(np_dev(z), k, bias=None if bias is None else np_dev(bias), **kw)
    torch.cuda.synchronize()
    return (ids.cpu().numpy(), w.cpu().numpy()), ref(z, k, bias=bias, **kw)


@pytest.mark.parametrize("E,groups,top", [(32, 1, 1), (64, 8, 3), (60, 5, 2), (256, 8, 4)])
@pytest.mark.parametrize("low,high", [(-743.0, -700.0), (-735.0, -709.0), (-712.0, -690.0)])
def test_subnormal_scores(E, groups, top, low, high):
    rng = np.random.default_rng(E)
    z = rng.uniform(low, high, (50, E)).astype(np.float32)
    z[1, ::2] = -np.inf
    z[2, 3:] = -800.0  # 0 in fp64 too
    z[3] = -800.0
    z[4, 5] = np.nan  # the rules for NaN as well
    k = 4
    (ids, w), (ri, rw) = _both(z, k, groups=groups, top_groups=top)
    assert np.array_equal(ids, ri)
    # z -743 .. -700: the chosen score n of 2^-1074
    chosen = np.take_along_axis(z.astype(np.float64), ri.astype(np.int64), 1)
    with np.errstate(over="ignore", divide="ignore"):
        room = 2.0 ** -23 + (k + 1) / np.maximum(np.exp(chosen + 1074 * np.log(2)), 1e-3)
    nan = np.isnan(rw)
    assert np.array_equal(nan, np.isnan(w)) and nan[4].any()
    assert (np.abs(w - rw)[~nan] <= (room * np.abs(rw))[~nan] + 2.0 ** -149).all()
    ok = np.delete(np.arange(50), [3, 4])
    assert np.allclose(w[ok].sum(1), 1, rtol=1e-6, atol=0) and (w[3] == 0).all()


def test_a_far_score_under_a_bias():
    """The bias chooses, the score weighs."""
    z = np.full((3, 16), -720.0, np.float32)
    z[0, 7], z[1, 9], z[2, 11] = -711.0, -715.0, -702.0
    bias = np.linspace(0, 1, 16).astype(np.float32)
    (ids, w), (ri, rw) = _both(z, 6, bias=bias)
    assert np.array_equal(ids, ri) and np.allclose(w, rw, rtol=1e-5, atol=0) and (w > 0).all()
    (ids, w), (ri, rw) = _both(z, 6, bias=bias, renormalise=False)
    assert np.array_equal(ids, ri) and (w == 0).all()  # below fp32
