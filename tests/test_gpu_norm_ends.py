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
    x[2, d - 4] = 3e38  # beside a NaN of the same thread: still the formula's number
    w[d - 4] = 4
    far = _norm(x, w)
    _no_numbers(far, x, w)
    n = _ref(x, None, w, 1e-6)[1][2, d - 4]
    assert abs(far[0][2, d - 4].item() - n) <= (2.0 ** -8 + 2.0 ** -21) * n
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


@pytest.mark.parametrize("d", WIDTHS)
@pytest.mark.parametrize("xt,rt,wt", [("bf16", None, "bf16"), ("f32", None, "f32"),
                                      ("bf16", "bf16", "f32"), ("f32", "f32", "bf16")])
def test_products_beyond_fp32(d, xt, rt, wt):
    """|v weight| above 3.4e38 where n is an ordinary number; the sum itself stays
    below it."""
    import torch

    T = {"bf16": torch.bfloat16, "f32": torch.float32, None: None}
    x, w = _rows(d, 6, d + 2)
    x = x.clamp(-3, 3)
    x[1] *= 1e38 / (3 if rt else 1)
    x[2] = x[2].sign() * 2e38 / (2 if rt else 1)
    x[3, 5] = 1.5e38  # one element alone
    x[4] *= 1e30
    w = (w + torch.rand(d, generator=torch.Generator().manual_seed(1))) * 2
    w[:4] = torch.tensor([1e-3, 1e5, -7, 0])
    x, w = x.to(T[xt]), w.to(T[wt])
    r = None if rt is None else (x.float() * 0.4).to(T[rt])
    got = _norm(x, w, residual=r, eps=1e-5)
    assert torch.isfinite(got[0]).all() and torch.isfinite(got[3]).all()
    _check(got, x, r, w, float(np.float32(1e-5)))
    one = _norm(x, w, residual=r, eps=1e-5, want_bf16=False)
    import routed_expert_prefill_amd as rep

    dev = torch_dev()
    y = rep.add_rmsnorm(x.to(dev), w.to(dev), eps=1e-5,
                        residual=None if r is None else r.to(dev))[0]
    assert torch.equal(y.view(torch.int16), got[0].view(torch.int16))
    assert torch.equal(one[2], got[2]) and torch.equal(one[3], got[3])


@pytest.mark.parametrize("d", WIDTHS)
def test_products_below_fp32(d):
    """|v weight| below fp32's numbers where a small eps lets r bring n back."""
    import torch

    x, w = _rows(d, 6, d + 3)
    eps = float(np.float32(2e-38))
    x[0] *= 1e-22
    x[1] *= 1e-24
    x[2] *= 1e-30
    x[3] = 0
    x[4, 1:] *= 1e-18
    w = w * 1e-21
    w[-8:] = 1
    got = _norm(x, w, eps=eps)
    _check(got, x, None, w, eps)
    assert got[3][3] == 1 and not got[2][3].any() and (got[0][:3] != 0).any()


def test_a_sum_beyond_fp32_is_no_number():
    """v is formed in fp32: what overflows there is an infinity."""
    import torch

    x, w = _rows(640, 3, 9)
    x[1, 20] = 3e38
    r = x.clone()
    y, ro, q, s = (t.cpu() for t in _norm(x, w, residual=r))
    assert torch.isinf(ro[1, 20]) and torch.isnan(y[1, 20]) and torch.isnan(s[1])
    assert not y[1, :20].any() and np.isnan(nx.e4m3_decode(q[1].numpy())).all()
    fine = [0, 2]
    _check((y[fine], ro[fine], q[fine], s[fine]), x[fine], r[fine], w, float(np.float32(1e-6)))


@pytest.mark.parametrize("rows,d", [((1 << 26) + 5, 8), ((1 << 24) + 3, 520)])
def test_more_rows_than_one_dimension_of_a_grid(rows, d):
    """One workgroup of 256 threads to four rows or to one: 2^32 threads and more."""
    import torch

    import routed_expert_prefill_amd as rep

    g = torch.Generator("cuda").manual_seed(rows)
    x = torch.randn(rows, d, generator=g, device="cuda", dtype=torch.bfloat16)
    w = (1 + 0.1 * torch.randn(d, generator=g, device="cuda")).to(torch.bfloat16)
    y = torch.full((rows + 2, d), 7.0, dtype=torch.bfloat16, device="cuda")
    rep.add_rmsnorm(x, w, y=y[:rows])
    torch.cuda.synchronize()
    assert (y[rows:] == 7).all()
    step = 1 << 22
    for a in range(0, rows, step):
        part = rep.add_rmsnorm(x[a:a + step], w)[0]
        assert torch.equal(part.view(torch.int16), y[a:min(a + step, rows)].view(torch.int16)), a
    _check((y[rows - 9:rows], None, None, None), x[-9:].cpu(), None, w.cpu(),
           float(np.float32(1e-6)))
