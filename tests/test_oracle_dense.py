"""Pins of oracle/select.py and oracle/dense.py against definitions they do not
share code with."""
import numpy as np
import pytest
import torch
from scipy.special import expit, softmax

from oracle import dense, numerics as nx, select


@pytest.mark.parametrize("scores", ["sigmoid", "softmax"])
def test_plain_selection_is_a_sort_of_the_scores(scores):
    rng = np.random.default_rng(0)
    z = rng.standard_normal((40, 24)).astype(np.float32)
    bias = rng.standard_normal(24).astype(np.float32) * 0.3
    ids, w = select.route_select(z, 5, scores, bias, renormalise=False, scale=2.5)
    s = expit(z.astype(np.float64)) if scores == "sigmoid" else softmax(z.astype(np.float64), axis=1)
    order = np.argsort(-(s + bias.astype(np.float64)), axis=1, kind="stable")[:, :5]
    assert np.array_equal(ids, order)
    assert np.allclose(w, 2.5 * np.take_along_axis(s, order, 1), rtol=1e-7, atol=0)
    _, w = select.route_select(z, 5, scores, bias, scale=2.5)
    assert np.allclose(w.sum(1), 2.5, rtol=1e-6)


@pytest.mark.parametrize("group_top", [1, 2])
def test_groups_against_torch(group_top):
    rng = np.random.default_rng(1)
    z = rng.standard_normal((60, 32)).astype(np.float32)
    ids, _ = select.route_select(z, 4, "sigmoid", None, 8, 3, group_top)
    s = torch.from_numpy(expit(z.astype(np.float64)))
    value = s.view(60, 8, 4).topk(group_top, -1).values.sum(-1)
    keep = torch.zeros(60, 8, dtype=torch.bool).scatter_(1, value.topk(3, -1).indices, True)
    want = s.masked_fill(~keep.repeat_interleave(4, 1), -1.0).topk(4, -1).indices
    assert np.array_equal(ids, want.numpy())


def test_ends_of_the_selection():
    inf, nan = np.inf, np.nan
    f = select.route_select
    # ties to the lower index; closed-form gates
    ids, w = f(np.zeros((2, 8)), 3, "softmax")
    assert (ids == [0, 1, 2]).all() and np.allclose(w, 1 / 3)
    # all out of service: the lowest indices, gates of zero
    ids, w = f(np.full((1, 6), -inf), 2, "softmax")
    assert ids.tolist() == [[0, 1]] and (w == 0).all()
    # one left: the others weigh nothing, whatever their bias
    z = np.full((1, 6), -inf)
    z[0, 4] = 1.0
    ids, w = f(z, 3, "sigmoid", np.array([5.0, 0, 0, 0, 0, 9.0]))
    assert ids.tolist() == [[4, 0, 1]] and w.tolist() == [[1, 0, 0]]
    # a group with one in service counts with that one alone; an empty one is last
    z = np.array([[2.0, -inf, -inf, -inf, 1.0, 1.0]])
    assert f(z, 2, "sigmoid", None, 3, 1)[0].tolist() == [[4, 5]]
    assert f(z, 2, "sigmoid", None, 3, 2)[0].tolist() == [[0, 4]]
    # NaN first
    ids, w = f(np.array([[3.0, nan, 1.0]]), 2, "sigmoid")
    assert ids.tolist() == [[1, 0]] and np.isnan(w).all()
    ids, w = f(np.array([[3.0, -inf, inf]]), 3, "softmax", renormalise=False)
    assert ids.tolist() == [[0, 2, 1]] and np.isnan(w[0, :2]).all() and w[0, 2] == 0


def test_products_against_torch():
    rng = np.random.default_rng(2)
    x = torch.from_numpy(rng.standard_normal((7, 384)).astype(np.float32))
    q, s = dense.quant_blocks(x.numpy())
    blocks = x.view(7, 3, 128)
    want = (blocks / torch.from_numpy(s)[..., None]).to(torch.float8_e4m3fn)
    assert np.array_equal(q.reshape(7, 3, 128), want.view(torch.uint8).numpy())
    assert np.abs(dense.row_values(q, s) - x.numpy()).max() <= 2.0 ** -4 * np.abs(x.numpy()).max()
    w = torch.from_numpy(rng.standard_normal((200, 384)).astype(np.float32)).to(torch.float8_e4m3fn)
    ws = (rng.random((2, 3)) + 0.5).astype(np.float32)
    wv = w.double()
    for i in range(2):
        for j in range(3):
            wv[128 * i:128 * (i + 1), 128 * j:128 * (j + 1)] *= float(ws[i, j])
    xv = want.double() * torch.from_numpy(s).double()[..., None]
    ref = (xv.view(7, 384) @ wv.T).numpy()
    wc = w.view(torch.uint8).numpy()
    assert np.allclose(dense.matmul(q, s, wc, ws), ref, rtol=0, atol=1e-11)
    assert (np.abs(ref) <= dense.matmul_abs(q, s, wc, ws)).all()
    h = dense.shared_hidden(q, s, wc, wc, ws, ws)
    g = torch.from_numpy(ref)
    assert np.allclose(h, (torch.nn.functional.silu(g) * g).numpy(), rtol=1e-12)
    assert nx.e4m3_decode(wc).shape == (200, 384)
