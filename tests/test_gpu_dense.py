"""GPU block quantisation, 8-bit products and the shared expert against 64 bits.

Codes and scales of the quantisation are compared bit for bit.  Products are
checked twice: on whole numbers and powers of two, whose sums are exact in fp32
in any order, so that results have to be equal; and on random codes within the
rounding of fp32 sums (dense_util.product_room).

The shared expert's codes of h may fall either way where the quotient lies next to
a midpoint.  On whole-number products g and u are exact, and h = silu(g) * u is
off by at most (|g| + 8) 2^-23 |h|: the exponential's argument, a product, by a
step of |g|, its value, the sum, the quotient and the product by a step or two
each.  h's scale is off by as much as its block's largest |h|, and by the
quotient's rounding.  Each code then lies between those of the two ends, and so
does each sum of the down product (plus its own rounding)."""
import numpy as np
import pytest

from dense_util import (U, bf16_room, dev, exact_problem, host, product_room, random_problem,
                        two_powers, whole_codes)
from oracle import dense, numerics as nx

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ quantisation


@pytest.mark.parametrize("rows,cols", [(1, 128), (3, 256), (1, 4096), (17, 384), (5, 8320),
                                       (401, 1152), (1031, 128), (2, 1 << 17)])
@pytest.mark.parametrize("wide", [False, True])
def test_blocks_match_the_rule(rows, cols, wide):
    import torch

    import routed_expert_prefill_amd as rep

    g = torch.Generator().manual_seed(rows + cols)
    x = torch.randn(rows, cols, generator=g) * torch.exp(3 * torch.randn(rows, 1, generator=g))
    x[:, ::17] *= 30
    x[0, :128] = 0
    x = x if wide else x.to(torch.bfloat16)
    q, s = rep.quant_blocks_fp8(x.cuda())
    rq, rs = dense.quant_blocks(x.float().numpy())
    assert np.array_equal(s.cpu().numpy(), rs) and np.array_equal(q.cpu().numpy(), rq)
    if not wide:  # the row quantisation with a block to a row
        q2, s2 = rep.quant_rows_fp8(x.cuda().view(-1, 128))
        assert torch.equal(q2.view(q.shape), q) and torch.equal(s2.view(s.shape), s)


def test_blocks_of_extreme_values():
    import torch

    import routed_expert_prefill_amd as rep

    x = torch.randn(16, 128, generator=torch.Generator().manual_seed(1))
    x[0] = -0.0
    x[1] *= 1e37
    x[2] *= 1e-38
    x[3] = 1e-45  # a quotient below the smallest number
    x[4] = x[4].sign() * 3e-43
    x[5, 7] = float("nan")
    x[6, 9] = float("inf")
    x[7, 3] = 3e4
    x[8] = float("nan")
    q, s = rep.quant_blocks_fp8(x.cuda())
    q, s = q.cpu().numpy(), s.cpu().numpy()[:, 0]
    fine = [1, 2, 7] + list(range(9, 16))
    rq, rs = dense.quant_blocks(x.numpy()[fine])
    assert np.array_equal(q[fine], rq) and np.array_equal(s[fine], rs[:, 0])
    assert s[0] == 1 and not q[0].any()
    tiny = np.float32(2.0 ** -149)
    assert s[3] == tiny and (nx.e4m3_decode(q[3]) == 1).all()
    assert s[4] == tiny and np.array_equal(nx.e4m3_decode(q[4]), nx.e4m3_decode(nx.e4m3_encode(x[4].double().numpy() / 2.0 ** -149)))
    rest = np.delete(x[5].numpy(), 7)
    rq, rs = dense.quant_blocks(np.append(rest, 0)[None].astype(np.float32))
    assert s[5] == rs[0, 0] and np.array_equal(np.delete(q[5], 7), rq[0, :127]) and q[5, 7] & 0x7F == 0x7F
    assert np.isinf(s[6]) and q[6, 9] & 0x7F == 0x7F and not (np.delete(q[6], 9) & 0x7F).any()
    assert s[8] == 1 or np.isnan(s[8])


def test_blocks_given_outputs_and_refusals():
    import torch

    import routed_expert_prefill_amd as rep

    x = torch.randn(5, 256, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).cuda()
    q = torch.full((7, 256), 9, dtype=torch.uint8, device="cuda")
    s = torch.full((8, 2), 9.0, device="cuda")
    want = rep.quant_blocks_fp8(x)
    got = rep.quant_blocks_fp8(x, q=q[:5], s=s[:5])
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert (q[5:] == 9).all() and (s[5:] == 9).all()
    e = rep.quant_blocks_fp8(x[:0])
    assert e[0].shape == (0, 256) and e[1].shape == (0, 2)
    for bad in (dict(x=x.cpu()), dict(x=x[0]), dict(x=x.half()), dict(x=x[:, :192].contiguous()),
                dict(x=x[:, ::2]), dict(q=q), dict(q=x), dict(s=s[:4]), dict(s=s[:5].double())):
        with pytest.raises((TypeError, ValueError)):
            rep.quant_blocks_fp8(**{"x": x, **bad})
    with pytest.raises(RuntimeError, match="MOE_EALIGN"):
        rep.quant_blocks_fp8(x.view(-1)[4:4 + 256].view(1, 256))


# ------------------------------------------------------------------ products


ROWS = [1, 2, 3, 4, 5, 8, 9, 15, 16, 17, 31, 32, 33, 48, 63, 64, 65, 96, 127, 128, 129, 192, 255, 256, 257, 300, 513]
COLS = [(1, 128), (5, 256), (16, 128), (100, 384), (127, 1152), (128, 128), (130, 512), (256, 640),
        (384, 256), (516, 896), (1416, 128), (2049, 256), (72, 8320), (264, 4096)]


@pytest.mark.parametrize("N,K", COLS)
def test_whole_numbers_are_exact(N, K):
    """Every number of rows about the tiles' edges, both outputs, rows behind the last left alone."""
    import torch

    import routed_expert_prefill_amd as rep

    q, xs, w, ws = exact_problem(N + K, max(ROWS), N, K)
    want = dense.matmul(q, xs, w, ws)
    dq, dxs, dw, dws = dev(q, xs, w, ws)
    for M in ROWS:
        for dtype in (torch.float32, torch.bfloat16):
            out = torch.full((M + 3, N), 7.0, dtype=dtype, device="cuda")
            rep.matmul_fp8((dq[:M].contiguous(), dxs[:M].contiguous()), dw, dws, out=out[:M])
            got = host(out)
            ref = want[:M] if dtype == torch.float32 else nx.bf16_round(want[:M])
            assert np.array_equal(got[:M], ref), (M, dtype)
            assert (got[M:] == 7).all(), (M, dtype)


@pytest.mark.parametrize("M,N,K", [(1, 4096, 4096), (7, 1000, 2048), (24, 516, 1152), (40, 2048, 4096),
                                   (100, 640, 640), (777, 1416, 1152), (1500, 2048, 1024), (2500, 1030, 384)])
def test_random_codes(M, N, K):
    import torch

    import routed_expert_prefill_amd as rep

    p = random_problem(M + N, M, N, K)
    want, total = dense.matmul(*p), dense.matmul_abs(*p)
    q, xs, w, ws = dev(*p)
    got = host(rep.matmul_fp8((q, xs), w, ws))
    off = np.abs(got - want)
    assert (off <= product_room(K, total)).all(), (off / product_room(K, total)).max()
    low = host(rep.matmul_fp8((q, xs), w, ws, out_dtype=torch.bfloat16))
    assert (np.abs(low - want) <= bf16_room(K, total, want)).all()
    # all in all: half a step of bf16 is 2^-8 of a value at most, spread evenly
    assert np.linalg.norm(low - want) <= 2.0 ** -8 / np.sqrt(3) * np.linalg.norm(want) * 1.1
    # the same bits from call to call
    assert torch.equal(rep.matmul_fp8((q, xs), w, ws).cpu(), torch.from_numpy(got).float())


@pytest.mark.parametrize("M", [1, 3, 6, 16, 20, 50, 130, 700])
@pytest.mark.parametrize("N,K", [(200, 384), (2048, 4096)])
def test_rows_in_bf16(M, N, K):
    """Quantised by the call as by quant_blocks_fp8."""
    import torch

    import routed_expert_prefill_amd as rep

    rng = np.random.default_rng(M)
    x = torch.from_numpy(rng.standard_normal((M, K))).to(torch.bfloat16)
    x[:, ::100] *= 40
    x[0, :128] = 0
    q, xs = dense.quant_blocks(x.float().numpy())
    _, _, w, ws = random_problem(N, 1, N, K)
    want, total = dense.matmul(q, xs, w, ws), dense.matmul_abs(q, xs, w, ws)
    dw, dws = dev(w, ws)
    got = host(rep.matmul_fp8(x.cuda(), dw, dws))
    off = np.abs(got - want)
    assert (off <= product_room(K, total)).all(), (off / product_room(K, total)).max()


@pytest.mark.parametrize("M", [1, 9, 33, 300])
def test_nan_and_zero_blocks(M):
    """A NaN row or weight stays with its row or column; zero codes give +0 or -0."""
    import torch

    import routed_expert_prefill_amd as rep

    q, xs, w, ws = exact_problem(5, M, 140, 512)
    q[M // 2, 200] = 0x7F
    w[131, 300] = 0xFF
    if M > 1:
        q[0] = 0
    got = host(rep.matmul_fp8(tuple(dev(q, xs)), *dev(w, ws)))
    assert np.isnan(got[M // 2]).all() and np.isnan(got[:, 131]).all()
    keep = np.delete(np.arange(M), M // 2)
    cols = np.delete(np.arange(140), 131)
    ref = dense.matmul(q[keep], xs[keep], w[cols[:128]], ws[:1])
    assert np.array_equal(got[np.ix_(keep, cols[:128])], ref)
    if M > 1:
        assert (got[0, cols] == 0).all()


def test_matmul_refusals():
    import torch

    import routed_expert_prefill_amd as rep

    q, xs, w, ws = dev(*exact_problem(1, 6, 130, 256))
    x = torch.zeros(6, 256, dtype=torch.bfloat16, device="cuda")
    out = torch.empty(6, 130, device="cuda")
    assert rep.matmul_fp8(x[:0], w, ws).shape == (0, 130)
    assert rep.matmul_fp8((q[:0], xs[:0]), w, ws, out_dtype=torch.bfloat16).dtype == torch.bfloat16
    for bad in (dict(x=x.cpu()), dict(x=x.float()), dict(x=x[0]), dict(x=(q,)), dict(x=(q, xs[:5])),
                dict(x=(x, xs)), dict(x=(q, xs.double())), dict(x=q), dict(x=x[:, :128].contiguous()),
                dict(x=x[:, :192].contiguous()), dict(w=w[0]), dict(w=w.view(torch.int8)), dict(w=None),
                dict(w=w[:, ::2]), dict(s=ws[:1]), dict(s=ws.half()), dict(s=ws.cpu()), dict(out=out[:5]),
                dict(out=out.double()), dict(out=out.T.contiguous().T), dict(out_dtype=torch.float16),
                dict(workspace=out), dict(x=[q, xs])):
        with pytest.raises((TypeError, ValueError)):
            rep.matmul_fp8(**{"x": x, "w": w, "s": ws, **bad})
    with pytest.raises(RuntimeError, match="MOE_EWORKSPACE"):
        rep.matmul_fp8(x, w, ws, workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
    # codes need none
    rep.matmul_fp8((q, xs), w, ws, workspace=torch.empty(0, dtype=torch.uint8, device="cuda"))
    with pytest.raises(RuntimeError, match="MOE_EALIGN"):
        rep.matmul_fp8(x.view(-1)[4:4 + 512].view(2, 256), w, ws)


# ------------------------------------------------------------------ the shared expert


def _shared_problem(seed, T, d, f):
    """g and u exact in fp32, |g| up to about 16."""
    rng = np.random.default_rng(seed)
    q, xs = whole_codes(rng, (T, d)), two_powers(rng, (T, d // 128))
    wg, wu, wd = whole_codes(rng, (f, d)), whole_codes(rng, (f, d)), whole_codes(rng, (d, f))
    sg, su = (two_powers(rng, (f // 128, d // 128)) * np.float32(2.0 ** -6) for _ in range(2))
    sd = (rng.random((d // 128, f // 128)) + 0.5).astype(np.float32)
    return q, xs, wg, wu, wd, sg, su, sd


def _shared_bounds(q, xs, wg, wu, wd, sg, su, sd):
    """The middle and the half width of what out may be, which codes of h may fall
    either way, and the sums of the terms' magnitudes."""
    g = dense.matmul(q, xs, wg, sg)
    h = nx.silu(g) * dense.matmul(q, xs, wu, su)
    T, f = h.shape
    off = (np.abs(g) + 8) * 2 * U * np.abs(h)
    hb, ob = h.reshape(T, -1, 128), off.reshape(T, -1, 128)
    at = np.abs(hb).argmax(-1)[..., None]
    top = np.take_along_axis(np.abs(hb), at, -1)
    # |h| that may be the largest: by how much the largest may be off
    slack = (np.abs(hb) + ob).max(-1, keepdims=True) - top
    s = np.where(top == 0, 1.0, top / 448)
    rel = np.where(top == 0, 0.0, slack / np.where(top == 0, 1, top) + U)
    t = hb / s
    room = ob / s + np.abs(t) * (rel + U)
    lo, hi = nx.e4m3_decode(nx.e4m3_encode(t - room)), nx.e4m3_decode(nx.e4m3_encode(t + room))
    lo, hi = np.minimum(lo, hi), np.maximum(lo, hi)
    mid, half = (lo + hi) / 2 * s, (hi - lo) / 2 * s + np.abs(hi) * s * rel
    wv = dense.weight_values(wd, sd)
    out = mid.reshape(T, f) @ wv.T
    total = (np.abs(mid) + half).reshape(T, f) @ np.abs(wv).T
    return out, half.reshape(T, f) @ np.abs(wv).T + product_room(f, total), lo != hi, total


SHARED = [(1, 128, 128), (1, 512, 256), (2, 256, 384), (5, 640, 128), (13, 1152, 640), (16, 384, 256),
          (17, 512, 512), (33, 256, 256), (64, 256, 128), (100, 128, 640), (129, 384, 384),
          (300, 512, 256), (777, 256, 384)]


@pytest.mark.parametrize("T,d,f", SHARED)
def test_shared_matches_the_formulas(T, d, f):
    import torch

    import routed_expert_prefill_amd as rep

    p = _shared_problem(T + d, T, d, f)
    want, room, either, total = _shared_bounds(*p)
    assert either.mean() < 0.05  # few codes lie next to a midpoint: the test tells
    q, xs, *W = dev(*p)
    out = torch.full((T + 2, d), 7.0, device="cuda")
    rep.shared_ffn((q, xs), *W, out=out[:T])
    got = host(out)
    off = np.abs(got[:T] - want)
    assert (off <= room).all(), (off / room).max()
    assert (got[T:] == 7).all()
    low = host(rep.shared_ffn((q, xs), *W, out_dtype=torch.bfloat16))
    assert (np.abs(low - want) <= room + bf16_room(f, total, want)).all()
    # rows in bf16: whole numbers whose blocks quantise to themselves
    v = dense.row_values(p[0], np.ones_like(p[1]))
    v[:, ::128] = 448
    x = torch.from_numpy(v).to(torch.bfloat16).cuda()
    a = rep.shared_ffn(x, *W)
    b = rep.shared_ffn(rep.quant_blocks_fp8(x), *W)
    room = _shared_bounds(*dense.quant_blocks(v.astype(np.float32)), *p[2:])[1]
    assert (np.abs(host(a) - host(b)) <= 2 * room).all()


def test_shared_refusals():
    import torch

    import routed_expert_prefill_amd as rep

    q, xs, *W = dev(*_shared_problem(1, 4, 256, 384))
    names = ("w_gate", "w_up", "w_down", "s_gate", "s_up", "s_down")
    good = {"x": (q, xs), **dict(zip(names, W))}
    assert rep.shared_ffn(**{**good, "x": (q[:0], xs[:0])}).shape == (0, 256)
    for n in names:
        for bad in (None, good[n].cpu(), good[n].half(), good[n][:1], good[n].T):
            with pytest.raises((TypeError, ValueError)):
                rep.shared_ffn(**{**good, n: bad})
    for bad in (dict(x=q), dict(x=(q, xs, xs)), dict(out=torch.empty(4, 384, device="cuda")),
                dict(out_dtype=torch.float16), dict(workspace=torch.empty(9, device="cuda")),
                dict(w_gate=W[0][:100].contiguous())):
        with pytest.raises((TypeError, ValueError)):
            rep.shared_ffn(**{**good, **bad})
    with pytest.raises(RuntimeError, match="MOE_EWORKSPACE"):
        rep.shared_ffn(**good, workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))


# ------------------------------------------------------------------ streams, graphs, without the module


@pytest.mark.parametrize("T", [1, 5, 40, 300])
def test_streams_graphs_and_no_module(T, monkeypatch):
    import torch

    import routed_expert_prefill_amd as rep

    d, f = 512, 384
    _, _, *W = dev(*_shared_problem(3, 1, d, f))
    g = torch.Generator().manual_seed(T)
    xs = [torch.randn(T, d, generator=g).to(torch.bfloat16).cuda() for _ in range(3)]

    def calls(x):
        codes = rep.quant_blocks_fp8(x)
        return [*codes, rep.matmul_fp8(x, W[0], W[3]), rep.matmul_fp8(codes, W[0], W[3], out_dtype=torch.bfloat16),
                rep.shared_ffn(x, *W), rep.shared_ffn(codes, *W, out_dtype=torch.bfloat16)]

    same = lambda a, b: all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(a, b))  # noqa: E731
    want = [[t.clone() for t in calls(x)] for x in xs]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = calls(xs[0])
    torch.cuda.current_stream().wait_stream(side)
    assert same(other, want[0])
    # two graphs that replay in turn, with eager calls between
    graphs = []
    for _ in range(2):
        x = xs[0].clone()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            cap = calls(x)
        graphs.append((x, graph, cap))
    for i, j in ((1, 0), (2, 1), (0, 0), (1, 1), (2, 0)):
        x, graph, cap = graphs[j]
        x.copy_(xs[i])
        for t in cap:
            t.view(torch.uint8).fill_(255)
        graph.replay()
        eager = calls(xs[(i + 1) % 3])
        torch.cuda.synchronize()
        assert same(cap, want[i]) and same(eager, want[(i + 1) % 3])
    monkeypatch.setattr(rep, "_native", lambda: None)
    assert same(calls(xs[1]), want[1])


def test_two_streams_at_once():
    """Calls that overlap on two streams, each with its own workspace."""
    import torch

    import routed_expert_prefill_amd as rep

    _, _, *W = dev(*_shared_problem(3, 1, 1024, 512))
    g = torch.Generator().manual_seed(1)
    xs = [torch.randn(200, 1024, generator=g).to(torch.bfloat16).cuda() for _ in range(2)]
    want = [rep.shared_ffn(x, *W) for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in xs]
    got = [[], []]
    for _ in range(4):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                got[i].append(rep.shared_ffn(xs[i], *W))
    torch.cuda.synchronize()
    assert all(torch.equal(o, want[i]) for i in range(2) for o in got[i])


def test_made_outputs_are_as_torch_makes_them():
    import torch

    import routed_expert_prefill_amd as rep

    z = torch.randn(3, 64, device="cuda")
    x = torch.randn(3, 256, device="cuda", dtype=torch.bfloat16)
    w = torch.zeros(256, 256, dtype=torch.uint8, device="cuda")
    s = torch.ones(2, 2, device="cuda")

    def calls():
        return (*rep.route_select(z, 4), *rep.quant_blocks_fp8(x), rep.matmul_fp8(x, w, s),
                rep.shared_ffn(x, w, w, w, s, s, s, out_dtype=torch.bfloat16))

    def look(outs):
        kinds = (torch.int32, torch.float32, torch.uint8, torch.float32, torch.float32,
                 torch.bfloat16)
        for o, kind in zip(outs, kinds, strict=True):
            like = torch.empty(o.shape, dtype=kind, device="cuda")
            assert type(o) is type(like) and o.dtype == kind and o.device == like.device
            assert o.is_contiguous() and not o.requires_grad
            assert o.is_inference() == like.is_inference()
            assert o.untyped_storage().nbytes() == like.untyped_storage().nbytes()
            assert o.untyped_storage().device == like.device
        return [o.clone() for o in outs]

    kept = look(calls())
    with torch.inference_mode():
        again = look(calls())
    z.requires_grad_()
    for a, b, c in zip(kept, again, look(calls()), strict=True):
        assert torch.equal(a, b) and torch.equal(a, c)
    before = torch.cuda.memory_allocated()
    outs = calls()
    assert torch.cuda.memory_allocated() > before  # the allocator's own blocks
    del outs
    assert torch.cuda.memory_allocated() == before
    with torch.cuda.stream(torch.cuda.Stream()):
        other = calls()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(kept, other, strict=True))
