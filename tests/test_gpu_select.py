"""GPU expert selection against the fp64 oracle: ids equal, gates within one fp32
step (both are formed in fp64 and rounded once; the exponentials differ in the
last bits of the double)."""
import numpy as np
import pytest

from oracle.select import route_select as ref
from gpu_util import np_dev

pytestmark = pytest.mark.gpu


def _gpu(z, k, bias=None, **kw):
    import torch

    import routed_expert_prefill_amd as rep

    zd = z if isinstance(z, torch.Tensor) else np_dev(z)
    ids, w = rep.route_select(zd, k, bias=None if bias is None else np_dev(bias), **kw)
    torch.cuda.synchronize()
    return ids.cpu().numpy(), w.cpu().numpy()


def _check(z, k, bias=None, **kw):
    ids, w = _gpu(z, k, bias, **kw)
    ri, rw = ref(z.float().cpu().numpy() if hasattr(z, "cpu") else z, k, bias=bias, **kw)
    assert np.array_equal(ids, ri)
    assert np.array_equal(np.isnan(w), np.isnan(rw))
    fine = ~np.isnan(rw)
    assert (np.abs(w - rw)[fine] <= np.spacing(np.abs(rw))[fine]).all()
    return ids, w


SHAPES = [  # T, E, k, groups, top_groups
    (1, 1, 1, 1, 1), (5, 7, 7, 1, 1), (33, 64, 6, 1, 1), (100, 256, 6, 8, 4), (17, 256, 16, 4, 2),
    (64, 100, 3, 10, 3), (257, 255, 8, 5, 5), (31, 24, 3, 1, 1), (3, 128, 2, 64, 1), (9, 60, 4, 20, 7),
    (40, 65, 1, 13, 1), (1, 256, 8, 8, 4), (2, 256, 6, 32, 3), (7, 192, 8, 3, 1), (1031, 160, 6, 8, 3),
]


@pytest.mark.parametrize("scores", ["sigmoid", "softmax"])
@pytest.mark.parametrize("T,E,k,groups,top", SHAPES)
def test_random_logits(scores, T, E, k, groups, top):
    import torch

    rng = np.random.default_rng(T * 1000 + E)
    z = rng.standard_normal((T, E)).astype(np.float32) * 1.5
    bias = (rng.standard_normal(E) * 0.1).astype(np.float32)
    for b in (None, bias):
        for group_top in (1, 2):
            _check(z, k, b, scores=scores, groups=groups, top_groups=top, group_top=group_top,
                   scale=2.5)
    _check(z, k, bias, scores=scores, groups=groups, top_groups=top, renormalise=False)
    _check(torch.from_numpy(z).to(torch.bfloat16).cuda(), k, bias, scores=scores, groups=groups,
           top_groups=top)


@pytest.mark.parametrize("scores", ["sigmoid", "softmax"])
def test_ties_and_neighbours(scores):
    rng = np.random.default_rng(7)
    z = rng.integers(-2, 3, (200, 256)).astype(np.float32)  # heavy ties
    for groups, top in ((1, 1), (8, 3), (64, 20)):
        _check(z, 6, scores=scores, groups=groups, top_groups=top)
        _check(z, 16, scores=scores, groups=groups, top_groups=top, group_top=1)
    _check(np.full((4, 32), -3.5, np.float32), 5, scores=scores, groups=4, top_groups=2)
    # neighbouring fp32 logits, whose scores are equal in fp32 and not in fp64
    base = rng.standard_normal((300, 1)).astype(np.float32) + 3
    steps = rng.integers(-3, 4, (300, 96))
    z = base.copy().repeat(96, 1)
    for _ in range(3):
        z = np.where(steps > 0, np.nextafter(z, np.float32(9)), np.where(steps < 0, np.nextafter(z, np.float32(-9)), z))
        steps = np.sign(steps) * (np.abs(steps) - 1).clip(0)
    for groups, top in ((1, 1), (6, 2)):
        _check(z, 8, scores=scores, groups=groups, top_groups=top)
    # and a bias that brings choices within less than an fp32 step
    bias = (0.5 + rng.integers(-2, 3, 96) * 2.0 ** -25).astype(np.float32)
    _check(np.round(z * 4) / 4, 8, bias, scores=scores, groups=6, top_groups=3)


@pytest.mark.parametrize("scores", ["sigmoid", "softmax"])
def test_large_and_small_logits(scores):
    rng = np.random.default_rng(8)
    z = (rng.standard_normal((64, 48)) * 60).astype(np.float32)  # scores that end at 0 and 1
    _check(z, 6, scores=scores)
    _check(z, 6, scores=scores, groups=6, top_groups=2)
    # far below: scores under fp32's range still weigh
    ids, w = _check((-200 - rng.random((8, 16))).astype(np.float32), 4, scores=scores)
    assert np.allclose(w.sum(1), 1, rtol=1e-6)
    _check((-200 - rng.random((8, 16))).astype(np.float32), 4, scores=scores, renormalise=False)
    _check(np.full((2, 16), 3e38, np.float32), 4, scores=scores)
    _check(np.full((2, 16), -3e38, np.float32), 4, scores=scores)


@pytest.mark.parametrize("scores", ["sigmoid", "softmax"])
@pytest.mark.parametrize("groups,top", [(1, 1), (6, 2)])
def test_experts_out_of_service(scores, groups, top):
    rng = np.random.default_rng(9)
    z = rng.standard_normal((90, 48)).astype(np.float32)
    z[rng.random(z.shape) < 0.5] = -np.inf
    z[10:14] = -np.inf  # none in service
    z[20:30, 8:] = -np.inf  # one group
    z[30:40, :] = np.where(np.arange(48) == 17, z[30:40, :], -np.inf)
    bias = rng.standard_normal(48).astype(np.float32)
    for b in (None, bias):
        ids, w = _check(z, 7, b, scores=scores, groups=groups, top_groups=top)
        assert (w[10:14] == 0).all()
        assert all(len(set(r)) == 7 for r in ids.tolist()) and ids.min() >= 0 and ids.max() < 48


@pytest.mark.parametrize("groups,top", [(1, 1), (4, 2)])
def test_nan_and_infinities(groups, top):
    rng = np.random.default_rng(10)
    z = rng.standard_normal((40, 32)).astype(np.float32)
    z[3, 9] = np.nan
    z[5, [1, 30]] = np.nan
    z[7, 4] = np.inf
    z[8, [4, 20]] = np.inf
    z[9, :] = np.nan
    z[11, 3] = np.nan
    z[11, 4:] = -np.inf
    for scores in ("sigmoid", "softmax"):
        ids, w = _check(z, 5, scores=scores, groups=groups, top_groups=top)
        assert ids.min() >= 0 and ids.max() < 32
        keep = [0, 1, 2, 4, 6, 10] + list(range(12, 40))  # rows beside those
        assert np.isfinite(w[keep]).all()
        bias = np.zeros(32, np.float32)
        bias[2], bias[8], bias[13] = np.nan, np.inf, -np.inf
        _check(z[12:], 5, bias, scores=scores, groups=groups, top_groups=top)


def test_given_outputs_rows_behind_and_refusals():
    import torch

    import routed_expert_prefill_amd as rep

    z = torch.randn(9, 64, generator=torch.Generator().manual_seed(1)).cuda()
    ids, w = rep.route_select(z, 4, groups=8, top_groups=2)
    gi = torch.full((12, 4), -7, dtype=torch.int32, device="cuda")
    gw = torch.full((12, 4), -7.0, device="cuda")
    got = rep.route_select(z, 4, groups=8, top_groups=2, topk_ids=gi[:9], topk_w=gw[:9])
    assert torch.equal(gi[:9], ids) and torch.equal(gw[:9], w) and (gi[9:] == -7).all() and (gw[9:] == -7).all()
    assert got[0].data_ptr() == gi.data_ptr()
    e = rep.route_select(z[:0], 4)
    assert e[0].shape == (0, 4) and e[1].shape == (0, 4)
    # the numbers' own types: int() of numpy and a whole scale
    a = rep.route_select(z, np.int64(4), groups=np.int32(8), top_groups=2, scale=1)
    assert torch.equal(a[0], ids) and torch.equal(a[1], w)
    for bad in (dict(logits=z.cpu()), dict(logits=z[0]), dict(logits=z.half()), dict(logits=z[:, ::2]),
                dict(bias=z[0].half()), dict(bias=z[0, :10].contiguous()), dict(bias=z[0].cpu()),
                dict(scores="linear"), dict(topk_ids=gi), dict(topk_w=gw[:9].double()),
                dict(topk_ids=gw[:9]), dict(k=2.5), dict(k=1 << 32), dict(k=0), dict(groups=None)):
        with pytest.raises((TypeError, ValueError)):
            rep.route_select(**{"logits": z, "k": 4, **bad})
    for bad in (dict(k=17), dict(groups=7), dict(groups=8, top_groups=9), dict(groups=32, top_groups=1, k=3),
                dict(group_top=3)):
        with pytest.raises(RuntimeError, match="MOE_EUNSUPPORTED"):
            rep.route_select(**{"logits": z, "k": 4, **bad})
    for bad in (dict(groups=0), dict(top_groups=-1), dict(scale=float("nan"))):
        with pytest.raises(RuntimeError, match="MOE_EINVAL"):
            rep.route_select(**{"logits": z, "k": 4, **bad})
    with pytest.raises(RuntimeError, match="MOE_EALIGN"):
        rep.route_select(z.view(-1)[1:65].view(1, 64), 4)


def test_own_stream_graph_replays_and_no_module(monkeypatch):
    import torch

    import routed_expert_prefill_amd as rep

    g = torch.Generator().manual_seed(2)
    zs = [torch.randn(77, 256, generator=g).cuda() for _ in range(3)]
    call = lambda z: rep.route_select(z, 6, groups=8, top_groups=4, scores="softmax")  # noqa: E731
    want = [[t.clone() for t in call(z)] for z in zs]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = call(zs[0])
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(other, want[0]))
    z = zs[0].clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cap = call(z)
    for i in (1, 2, 0, 1):
        z.copy_(zs[i])
        for t in cap:
            t.fill_(-1)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(cap, want[i]))
    monkeypatch.setattr(rep, "_native", lambda: None)
    assert all(torch.equal(a, b) for a, b in zip(call(zs[2]), want[2]))


def test_groups_whose_sums_round_apart():
    """Two groups of nearly one value under a bias of 128: choices half a step (2^-17)
    from fp32 numbers, of one group just above and of the other below, whose sums are
    halfway between fp32 numbers too.  Four roundings, all of the largest size, move the
    groups' fp32 values 2^-14 apart; scores of the last place decide."""
    rng = np.random.default_rng(128)
    T, u = 20000, 2.0 ** -16
    m1 = rng.integers(int(0.55 / u), int(0.6 / u), T)
    m2 = rng.integers(int(0.8 / u), int(0.85 / u), T)
    m2 += (1 - m1 - m2) % 4
    shift = rng.integers(0, 20, T)
    m = np.stack([m1, m2, m1 + shift, m2 - shift], 1)
    near = rng.integers(-3, 4, (T, 4)) * 2.0 ** -24
    s = (m + 0.5) * u + near
    z = np.log(s / (1 - s)).astype(np.float32)
    turned = rng.random(T) < 0.5
    z[turned] = z[turned][:, [2, 3, 0, 1]]
    _check(z, 2, np.full(4, 128.0, np.float32), groups=2, top_groups=1)
