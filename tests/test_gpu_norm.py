"""GPU residual addition and RMS norm against the formulas in 64 bits.

Tolerances, from the arithmetic: fp32 n = (v * weight) * r carries the
roundings of v (2^-24), of two products (2 x 2^-24) and of r (the mean's
conversion counts half, the root and the quotient one each: 2.5 x 2^-24), so
|n - n64| <= 6 x 2^-24 |n64|; bf16 adds half a step, at most 2^-8 of the
value.  residual_out is one fp32 addition rounded once more, and compared bit
for bit.  A scale adds one division.  A code is the nearest to n / s: within
half a step of it, and 2^-18 of the value for n's own error; and exactly the
nearest to the quotient that 64 bits give (test_codes_are_the_nearest)."""
import numpy as np
import pytest

from oracle import numerics as nx
from gpu_util import torch_dev

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


def _inputs(rows, d, xt, rt, wt, seed, scale=1.0):
    import torch

    g = torch.Generator().manual_seed(seed)
    x = (torch.randn(rows, d, generator=g) * scale).to(xt)
    r = None if rt is None else (torch.randn(rows, d, generator=g) * 3 * scale).to(rt)
    w = (1 + 0.2 * torch.randn(d, generator=g)).to(wt)
    return x, r, w


def _ref(x, r, w, eps):
    v = x.double().numpy() + (0 if r is None else r.double().numpy())
    with np.errstate(invalid="ignore", over="ignore"):
        n = v * w.double().numpy() / np.sqrt((v * v).mean(-1, keepdims=True) + eps)
    return v, n


def _check(got, x, r, w, eps):
    import torch

    y, ro, q, s = got
    v, n = _ref(x, r, w, eps)
    if ro is not None:
        want = (x.float() if r is None else r.float() + x.float()).to(ro.dtype)
        assert torch.equal(ro.cpu().view(torch.uint8), want.view(torch.uint8))
    if y is not None:
        off = np.abs(y.cpu().double().numpy() - n)
        assert (off <= (2.0 ** -8 + 7 * U) * np.abs(n) + 2.0 ** -134).all(), off.max()
    if q is not None:
        sc = s.cpu().double().numpy()
        top = np.abs(n).max(-1)
        want = np.where(top == 0, 1.0, top / 448)
        assert (np.abs(sc - want) <= 8 * U * want).all()
        val = nx.e4m3_decode(q.cpu().numpy())
        t = n / sc[:, None]
        step = np.exp2(np.floor(np.log2(np.maximum(np.abs(t), 2.0 ** -6))) - 3)
        assert (np.abs(val - t) <= step / 2 + 2.0 ** -18 * np.abs(t)).all()


CASES = [
    # every width class and its edges, odd row counts, one row
    (1, 8), (3, 64), (5, 504), (7, 512), (9, 520), (2, 2048), (3, 2056), (1, 4096), (37, 4096),
    (5, 4104), (3, 8192), (2, 8200), (1, 16384), (4, 16376), (1031, 1416), (4099, 128),
]


@pytest.mark.parametrize("rows,d", CASES)
@pytest.mark.parametrize("xt,rt,wt", [("bf16", "bf16", "bf16"), ("bf16", "f32", "f32"),
                                      ("f32", "bf16", "bf16"), ("f32", "f32", "bf16"),
                                      ("bf16", None, "bf16"), ("f32", None, "f32")])
def test_matches_the_formulas(rows, d, xt, rt, wt):
    import torch

    import routed_expert_prefill_amd as rep

    T = {"bf16": torch.bfloat16, "f32": torch.float32, None: None}
    x, r, w = _inputs(rows, d, T[xt], T[rt], T[wt], seed=rows * 7 + d)
    dev = torch_dev()
    dx, dw, dr = x.to(dev), w.to(dev), None if r is None else r.to(dev)
    got = rep.add_rmsnorm(dx, dw, eps=1e-5, residual=dr, want_fp8=True)
    torch.cuda.synchronize()
    _check(got, x, r, w, 1e-5)
    assert (got[1] is None) == (r is None)
    # inputs are left as they were, and one output alone is the same
    assert torch.equal(dx.cpu().view(torch.uint8), x.view(torch.uint8))
    y2 = rep.add_rmsnorm(dx, dw, eps=1e-5, residual=dr)[0]
    _, _, q3, s3 = rep.add_rmsnorm(dx, dw, eps=1e-5, residual=dr, want_bf16=False, want_fp8=True)
    assert torch.equal(y2.view(torch.int16), got[0].view(torch.int16))
    assert torch.equal(q3, got[2]) and torch.equal(s3, got[3])


@pytest.mark.parametrize("rows,d,xt,rt,wt", [
    (1500, 1416, "bf16", "f32", "bf16"), (401, 4096, "bf16", "bf16", "bf16"),
    (300, 8200, "f32", "f32", "f32"), (2000, 384, "f32", None, "bf16"),
])
def test_codes_are_the_nearest(rows, d, xt, rt, wt):
    """Every code is that of the quotient in 64 bits: v weight is exact there
    but for the residual's addition, and so is its product with 448."""
    import torch

    import routed_expert_prefill_amd as rep

    types = {"bf16": torch.bfloat16, "f32": torch.float32, None: None}
    x, r, w = _inputs(rows, d, types[xt], types[rt], types[wt], seed=rows)
    if r is not None:
        r[:, :: d // 4] *= 50  # the rest lies in the low codes, subnormal ones among them
    dev = torch_dev()
    _, _, q, _ = rep.add_rmsnorm(x.to(dev), w.to(dev), want_fp8=True,
                                 residual=None if r is None else r.to(dev))
    p = _ref(x, r, w, 1e-6)[0] * w.double().numpy()
    t = p * 448 / np.abs(p).max(-1, keepdims=True)
    assert np.array_equal(q.cpu().numpy(), nx.e4m3_encode(t))


@pytest.mark.parametrize("d", [384, 4096])
def test_in_place_and_given_outputs(d):
    import torch

    import routed_expert_prefill_amd as rep

    dev = torch_dev()
    rows = 19
    x, r, w = _inputs(rows, d, torch.bfloat16, torch.bfloat16, torch.bfloat16, seed=3)
    ref = rep.add_rmsnorm(x.to(dev), w.to(dev), residual=r.to(dev), want_fp8=True)
    res = torch.full((rows + 2, d), 7.0, dtype=torch.bfloat16, device=dev)
    y = torch.full((rows + 2, d), 7.0, dtype=torch.bfloat16, device=dev)
    q = torch.full((rows + 2, d), 9, dtype=torch.uint8, device=dev)
    s = torch.full((rows + 4,), 9.0, device=dev)
    res[:rows] = r.to(dev)
    got = rep.add_rmsnorm(x.to(dev), w.to(dev), residual=res[:rows], residual_out=res[:rows],
                          y=y[:rows], q=q[:rows], s=s[:rows])
    torch.cuda.synchronize()
    for a, b in zip(got, ref):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    # rows behind the last one stay as they were
    assert (res[rows:] == 7).all() and (y[rows:] == 7).all() and (q[rows:] == 9).all()
    assert (s[rows:] == 9).all()
    # without a residual the sum is x itself, written where asked
    out = torch.empty_like(x, device=dev)
    _, ro, _, _ = rep.add_rmsnorm(x.to(dev), w.to(dev), residual_out=out)
    assert ro is out and torch.equal(out.cpu().view(torch.int16), x.view(torch.int16))


def test_rows_of_extreme_values():
    import torch

    import routed_expert_prefill_amd as rep

    dev = torch_dev()
    d = 640
    x = torch.randn(9, d, generator=torch.Generator().manual_seed(1))
    x[0] = 0  # an all-zero row
    x[1] *= 1e25  # squares beyond fp32
    x[2] *= 1e-25  # squares below fp32; eps decides
    x[3, 5] = 3e4  # one outlier pushes the rest to the low codes
    x[4, 100] = float("nan")
    x[5, 101] = float("inf")
    x[6] = 1e-30
    x[7] = -0.0
    w = torch.ones(d)
    y, _, q, s = rep.add_rmsnorm(x.to(dev), w.to(dev), eps=1e-6, want_fp8=True)
    torch.cuda.synchronize()
    fine = [0, 1, 2, 3, 6, 7, 8]
    _check((y[fine], None, q[fine], s[fine]), x[fine], None, w, float(np.float32(1e-6)))
    assert s[0] == 1 and not q[0].any() and s[7] == 1 and not q[7].any()
    assert torch.isnan(y[4]).all() and torch.isnan(s[4])
    assert torch.isnan(y[5, 101]) and torch.isnan(s[5]) and (y[5, :101] == 0).all()
    assert np.isnan(nx.e4m3_decode(q[4:6].cpu().numpy())).all()


def test_no_rows_and_refusals():
    import torch

    import routed_expert_prefill_amd as rep

    dev = torch_dev()
    x = torch.zeros(4, 256, dtype=torch.bfloat16, device=dev)
    w = torch.ones(256, dtype=torch.bfloat16, device=dev)
    y, ro, q, s = rep.add_rmsnorm(x[:0], w, residual=x[:0], want_fp8=True)
    assert y.shape == (0, 256) and ro.shape == (0, 256) and q.shape == (0, 256) and s.shape == (0,)
    for bad in (dict(x=x.cpu()), dict(x=x[0]), dict(weight=w[:128]), dict(weight=w.half()),
                dict(x=x.half()), dict(residual=x[:2]), dict(residual=x.half()),
                dict(residual=x, residual_out=x.float()), dict(y=x.float()), dict(q=x),
                dict(s=torch.ones(3, device=dev)), dict(x=x[:, ::2], weight=w[::2]),
                dict(residual=x.cpu())):
        with pytest.raises((TypeError, ValueError)):
            rep.add_rmsnorm(**{"x": x, "weight": w, **bad})
    with pytest.raises(RuntimeError, match="MOE_EINVAL"):
        rep.add_rmsnorm(x, w, want_bf16=False)
    with pytest.raises(RuntimeError, match="MOE_EINVAL"):
        rep.add_rmsnorm(x, w, eps=0.0)
    with pytest.raises(RuntimeError, match="MOE_EUNSUPPORTED"):
        rep.add_rmsnorm(x[:, :4].contiguous(), w[:4])
    with pytest.raises(RuntimeError, match="MOE_EALIGN"):
        rep.add_rmsnorm(x.view(-1)[4:4 + 512].view(2, 256), w)


def test_own_stream_and_graph_replays():
    import torch

    import routed_expert_prefill_amd as rep

    dev = torch_dev()
    x, r, w = (t.to(dev) for t in _inputs(33, 4096, torch.bfloat16, torch.bfloat16,
                                          torch.bfloat16, seed=5))
    eager = [t.clone() for t in rep.add_rmsnorm(x, w, residual=r, want_fp8=True)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = rep.add_rmsnorm(x, w, residual=r, want_fp8=True)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    for a, b in zip(other, eager):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        cap = rep.add_rmsnorm(x, w, residual=r, want_fp8=True)
    for _ in range(3):
        for t in cap:
            t.view(torch.uint8).fill_(255)
        g.replay()
        torch.cuda.synchronize()
        for a, b in zip(cap, eager):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
        (x.float() * 2).sum().item()


def _call_both_ways(monkeypatch, call):
    """call() through the extension module and without it."""
    import routed_expert_prefill_amd as rep

    native = rep._native()
    assert native is not None
    used = []

    class Spy:
        def __getattr__(self, name):
            def run(*args):
                used.append(getattr(native, name)(*args))
                return used[-1]
            return run

    monkeypatch.setattr(rep, "_native", lambda: Spy())
    first = call()
    monkeypatch.setattr(rep, "_native", lambda: None)
    second = call()
    monkeypatch.undo()
    return first, second, used[0]


@pytest.mark.parametrize("xt,rt", [("bf16", "f32"), ("f32", "bf16"), ("f32", None)])
@pytest.mark.parametrize("want", [dict(), dict(want_fp8=True), dict(want_fp8=True, want_bf16=False),
                                  "outputs"])
def test_with_and_without_the_extension(monkeypatch, xt, rt, want):
    import torch

    import routed_expert_prefill_amd as rep

    types = {"bf16": torch.bfloat16, "f32": torch.float32, None: None}
    x, r, w = (None if t is None else t.to(torch_dev())
               for t in _inputs(33, 640, types[xt], types[rt], torch.bfloat16, seed=2))

    def call():
        kw = want
        if want == "outputs":
            kw = dict(y=torch.empty_like(x, dtype=torch.bfloat16), s=torch.empty(33, device=x.device),
                      residual_out=torch.empty_like(x if r is None else r))
        got = rep.add_rmsnorm(x, w, residual=r, **kw)
        if want == "outputs":
            assert got[0] is kw["y"] and got[3] is kw["s"] and got[1] is kw["residual_out"]
        return got

    a, b, used = _call_both_ways(monkeypatch, call)
    assert used is not None
    for p, q in zip(a, b):
        assert (p is None) == (q is None)
        if p is not None:
            assert p.dtype == q.dtype and torch.equal(p.view(torch.uint8), q.view(torch.uint8))


def test_the_extension_leaves_refusals_to_python(monkeypatch):
    import torch

    import routed_expert_prefill_amd as rep

    x, r, w = (t.to(torch_dev()) for t in _inputs(4, 64, torch.bfloat16, torch.float32,
                                                  torch.bfloat16, seed=3))
    for kw in (dict(x=x.t()), dict(x=x[:, ::2]), dict(weight=w[:8]), dict(weight=w.double()),
               dict(residual=r[:2]), dict(residual=r.cpu()), dict(y=torch.empty_like(r)),
               dict(q=torch.empty_like(x)), dict(s=torch.empty(3, device=x.device)),
               dict(residual_out=torch.empty_like(x)), dict(eps=-1.0), dict(want_bf16=False)):
        args = dict(x=x, weight=w, residual=r, **{k: v for k, v in kw.items()
                                                  if k not in ("x", "weight", "residual")})
        args.update({k: v for k, v in kw.items() if k in ("x", "weight", "residual")})

        def call():
            with pytest.raises((TypeError, ValueError, RuntimeError)) as e:
                rep.add_rmsnorm(**args)
            return str(e.value)

        a, b, used = _call_both_ways(monkeypatch, call)
        assert a == b and used is None
