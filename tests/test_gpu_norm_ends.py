"""GPU residual addition and RMS norm where numbers end: no numbers, values and
products at both ends of fp32, and the most rows.  Tolerances as in
test_gpu_norm.py."""
import numpy as np
import pytest

from oracle import numerics as nx
from gpu_util import torch_dev
from test_gpu_norm import _check, _ref

pytestmark = pytest.mark.gpu

WIDTHS = [384, 640, 4096, 8200]  # a wave to a row; one, two and eight chunks a thread


def _rows(d, n, seed):
    import torch

    return torch.randn(n, d, generator=torch.Generator().manual_seed(seed)), torch.ones(d)


def _norm(x, w, **kw):
    import torch

    import routed_expert_prefill_amd as rep

    dev = torch_dev()
    if kw.get("residual") is not None:
        kw["residual"] = kw["residual"].to(dev)
    got = rep.add_rmsnorm(x.to(dev), w.to(dev), want_fp8=True, **kw)
    torch.cuda.synchronize()
    return got


def _no_numbers(got, x, w):
    """y, s and the codes are NaN exactly where the formulas are."""
    y, _, q, s = got
    _, n = _ref(x, None, w, 1e-6)
    y, s = y.cpu().double().numpy(), s.cpu().double().numpy()
    assert np.array_equal(np.isnan(y), np.isnan(n))
    top = np.abs(n).max(-1)  # NaN where one element is
    assert np.array_equal(np.isnan(s), np.isnan(top))
    with np.errstate(invalid="ignore", divide="ignore"):
        t = n / np.where(top == 0, 1.0, top / 448)[:, None]
    assert np.array_equal(np.isnan(nx.e4m3_decode(q.cpu().numpy())), np.isnan(t))


@pytest.mark.parametrize("d", WIDTHS)
def test_no_number_in_the_weight(d):
    x, w = _rows(d, 5, d)
    clean = _norm(x, w)
    w[d - 3] = float("nan")
    got = _norm(x, w)
    _no_numbers(got, x, w)
    keep = np.arange(d) != d - 3
    assert np.array_equal(got[0].cpu().double().numpy()[:, keep],
                          clean[0].cpu().double().numpy()[:, keep])


@pytest.mark.parametrize("d", WIDTHS)
def test_no_numbers_from_infinities(d):
    """An infinity times a weight of zero, and an infinite weight times zero."""
    x, w = _rows(d, 6, d + 1)
    w[7] = 0
    x[1, 7] = float("inf")
    x[2, 9] = float("-inf")
    x[3, d - 1] = float("nan")
    got = _norm(x, w)
    _no_numbers(got, x, w)
    fine = [0, 4, 5]
    _check([None if t is None else t[fine] for t in got], x[fine], None, w, float(np.float32(1e-6)))
    w[11] = float("inf")
    x[4, 11] = 0
    got = _norm(x, w)
    _no_numbers(got, x, w)
    s, q = got[3].cpu().numpy(), got[2].cpu().numpy()
    assert np.isnan(s[4]) and s[5] == float("inf") and s[0] == float("inf")
    assert not np.delete(nx.e4m3_decode(q[[0, 5]]), 11, 1).any()
