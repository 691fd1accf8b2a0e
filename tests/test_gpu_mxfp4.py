"""GPU grouped FFN with MXFP4 weights vs the fp64 oracle.

The weights' values are bf16 numbers, so the oracle takes them as bf16.
Tolerances: both sides round h to bf16, so what is left is the order of fp32
sums (about 1e-6 of a row's norm) and the h values that it pushes over a
rounding border: a share of about 2e-6 / 2^-8 = 5e-4 of them, each off by a
step of at most 2^-7, hence sqrt(5e-4) x 2^-7 = 2e-4 of the outputs' norm:
relative Frobenius 1e-3.  One such step moves an output by at most
2^-7 |h| |w|, with |h| < 16 rms(h) and |w| < 4 rms(w) against a sum of f >= 128
terms: 2^-7 x 64 / 11 = 0.045 of the outputs' rms."""
import ctypes

import numpy as np
import pytest

from oracle import moe as omoe
from oracle.route import route_table
from gpu_util import bf16_dev, np_dev, rel_frob, routing_with_counts
from mxfp4_util import bf16_source, mx_weights
from test_gpu_ffn import CLASS_COUNTS, QUEUE_COUNTS, _x

pytestmark = pytest.mark.gpu


def _close(got, ref):
    rel = rel_frob(got, ref)
    big = np.abs(got - ref).max() / np.sqrt(np.mean(ref * ref))
    assert rel <= 1e-3 and big <= 0.05, (rel, big)


def _dev(W):
    return [np_dev(W[n]) for n in ("wg", "wu", "wd", "sg", "su", "sd")]


def _problem(counts, k, d, f, seed, masked=13, invalid=0):
    E = len(counts)
    ids, mask = routing_with_counts(counts, k, seed=seed, masked_extra=masked,
                                    invalid_extra=invalid)
    w = np.random.default_rng(seed + 1).random(ids.shape).astype(np.float32)
    return E, ids, w, mask, _x(ids.shape[0], d, seed + 2), mx_weights(E, d, f, seed + 3)


def _run(p, y_fill=float("nan"), **kw):
    import torch

    import routed_expert_prefill_amd as rep

    E, ids, w, mask, x, W = p
    run = rep.MoEPrefill(*ids.shape, E, x.shape[1], W["wg"].shape[1], weights="mxfp4")
    run.decode = False  # the grouped path for few routes too
    if y_fill is not None:
        run.y.fill_(y_fill)
    out = run(bf16_dev(x), np_dev(ids), np_dev(w), np_dev(mask), *_dev(W), **kw)
    torch.cuda.synchronize()
    return run, out.cpu().numpy().astype(np.float64)


@pytest.mark.parametrize("counts,k,d,f", [
    (CLASS_COUNTS, 6, 384, 256),  # every tile class; half a stage left over
    (CLASS_COUNTS, 6, 256, 640),  # the same for the down projection
    (QUEUE_COUNTS, 6, 256, 256),  # several tiles to an expert, both queues
    ([1] * 30 + [0] * 9, 3, 1152, 128),
    ([65, 3], 2, 128, 128),  # one half stage is all there is
    ([513], 1, 512, 384),
    ([31, 33, 300], 2, 128, 1024),
])
def test_matches_oracle(counts, k, d, f):
    p = _problem(counts, k, d, f, seed=d + f + k)
    E, ids, w, mask, x, W = p
    run, out = _run(p)
    rt = route_table(ids, mask, E)
    n = int(rt.offsets[E])
    y = run.y.cpu().numpy()
    assert np.isnan(y[n:]).all() and not np.isnan(y[:n]).any()
    src = bf16_source(W)
    sample = [int(rt.sorted_routes[i]) for i in range(0, n, 5)]
    _close(y[rt.route_rows[sample]], omoe.route_outputs_ref(x, ids, src, sample))
    _close(out, omoe.moe_ref_blocked(x, ids, w, mask, src, E)[0])


def test_full_width():
    """Stages, rings and items at the widths of the real layer."""
    p = _problem([300, 257, 190, 120, 64, 33, 9, 1, 0, 16], 6, 4096, 2048, seed=77)
    E, ids, w, mask, x, W = p
    _, out = _run(p)
    _close(out, omoe.moe_ref_blocked(x, ids, w, mask, bf16_source(W), E)[0])


@pytest.mark.parametrize("rows", [13, 60, 90, 100, 128, 150, 180, 220, 256])
def test_many_tiles_of_one_height(rows):
    """Enough items of one tile height, at a reduction of 4096 columns, to keep
    every workgroup at it for several rounds: a stage that started ahead of
    its loads would show here."""
    E, d, f = 40, 4096, 1024
    p = _problem([rows - e % 3 for e in range(E)], 4, d, f, seed=rows)
    _, ids, w, mask, x, W = p
    _, out = _run(p)
    sub = [0, 1, 7, 20, 39]  # the reference of every expert would take minutes: these experts' share
    only = np.where(np.isin(ids, sub), mask, 0).astype(np.uint8)
    _, part = _run((E, ids, w, only, x, W))
    _close(part, omoe.moe_ref_blocked(x, ids, w, only, bf16_source(W), E)[0])
    # and the whole as the sum of eight shares, each run by itself.  A share has
    # fewer items, so its tiles may be shorter and their sums in another order:
    # the tolerance above
    total = np.zeros_like(out)
    for g in range(8):
        share = np.where(ids % 8 == g, mask, 0).astype(np.uint8)
        total += _run((E, ids, w, share, x, W))[1]
    _close(out, total)


@pytest.mark.parametrize("E,d,f", [
    (96, 1536, 1536),  # both projections by slices of 512 columns
    (160, 1024, 640),  # gate/up only, its last item half full
    (200, 640, 1024),  # down only, the same
    (130, 5120, 512),  # rows too long for LDS: the smallest tiles too
])
def test_tiles_of_up_to_64_rows(E, d, f):
    """Enough items that tiles of up to 64 rows stream their weights: every
    number of 16-row tiles, beside shorter and taller tiles."""
    sizes = [17, 24, 32, 33, 40, 48, 49, 60, 64, 9, 16, 70, 0, 1]
    p = _problem([sizes[e % len(sizes)] for e in range(E)], 4, d, f, seed=E)
    _, ids, w, mask, x, W = p
    run, out = _run(p)
    rt = route_table(ids, mask, E)
    n = int(rt.offsets[E])
    y = run.y.cpu().numpy()
    assert np.isnan(y[n:]).all() and not np.isnan(y[:n]).any()
    sample = [int(rt.sorted_routes[i]) for i in range(0, n, 41)]
    _close(y[rt.route_rows[sample]], omoe.route_outputs_ref(x, ids, bf16_source(W), sample))
    # every row, by another path: a call of few experts' routes takes other tiles
    for g in range(0, 24, 8):
        some = np.where((ids >= g) & (ids < g + 8), mask, 0).astype(np.uint8)
        part, _ = _run((E, ids, w, some, x, W))
        rows = [r for r in range(ids.size) if some.flat[r]]
        there = route_table(ids, some, E).route_rows[rows]
        _close(y[rt.route_rows[rows]].astype(np.float64),
               part.y.cpu().numpy()[there].astype(np.float64))


def test_masked_and_out_of_range_routes_add_exact_zeros():
    p = _problem([5, 0, 40, 3], 3, 256, 128, seed=5, masked=20, invalid=6)
    E, ids, w, mask, x, W = p
    mask[3] = 0  # a token with no route left
    _, out = _run(p)
    ok = (mask != 0) & (ids >= 0) & (ids < E)
    assert (ok.sum(1) == 0).any()
    none = out[ok.sum(1) == 0]
    assert not none.any() and not np.signbit(none).any()
    _close(out, omoe.moe_ref_blocked(x, ids, w, mask, bf16_source(W), E)[0])


def test_all_routes_masked():
    p = _problem([0, 0, 0], 2, 256, 128, seed=6, masked=8)
    _, out = _run(p)
    assert not out.any() and not np.signbit(out).any()


def test_scales_over_their_whole_range():
    """Row n of the down projection has scale byte n everywhere: outputs from
    2^-127 up, through overflow to infinity, and NaN for 255."""
    d, f = 256, 256
    p = _problem([40, 2], 2, d, f, seed=8)
    E, ids, w, mask, x, W = p
    W["sd"][:] = np.arange(256, dtype=np.uint8)[None, :, None]
    run, _ = _run(p)
    plain = {n: a.copy() for n, a in W.items()}
    plain["sd"][:] = 127
    rt = route_table(ids, mask, E)
    n = int(rt.offsets[E])
    y = run.y.cpu().numpy()[:n].astype(np.float64)
    unit = omoe.route_outputs_ref(x, ids, bf16_source(plain), [int(r) for r in rt.sorted_routes[:n]])
    assert np.isnan(y[:, 255]).all()
    s = np.arange(255)
    for lo, hi in ((20, 100), (100, 180), (180, 235)):
        _close(y[:, lo:hi] * np.exp2(127.0 - s[lo:hi]), unit[:, lo:hi])
    # down to the smallest scale: subnormal weights and sums, to 2^-126 of the products
    low = y[:, :20]
    assert (np.abs(low - unit[:, :20] * np.exp2(s[:20] - 127.0)) <=
            np.abs(unit[:, :20]).max() * np.exp2(s[:20] - 127.0) * 0.05 + 64 * 2.0 ** -126).all()


def test_bf16_output_and_shared_rows():
    import torch

    import routed_expert_prefill_amd as rep

    p = _problem([30, 70, 0, 5], 2, 384, 256, seed=9)
    E, ids, w, mask, x, W = p
    T, k = ids.shape
    shared = np.random.default_rng(1).standard_normal((T, 384)).astype(np.float32)
    _, plain = _run(p)
    _, f32 = _run(p, shared=np_dev(shared))
    assert np.array_equal(f32, (plain.astype(np.float32) + shared).astype(np.float64))
    run = rep.MoEPrefill(T, k, E, 384, 256, weights="mxfp4", out_dtype=torch.bfloat16)
    run.decode = False
    out = run(bf16_dev(x), np_dev(ids), np_dev(w), np_dev(mask), *_dev(W), shared=np_dev(shared))
    want = torch.from_numpy(f32.astype(np.float32)).to(torch.bfloat16)
    assert torch.equal(out.cpu().view(torch.int16), want.view(torch.int16))


def test_runs_again_bit_for_bit_and_in_graph_replays():
    import torch

    import routed_expert_prefill_amd as rep

    p = _problem([0, 31, 64, 65, 130, 200, 300, 700, 5, 0, 1], 6, 512, 256, seed=10)
    E, ids, w, mask, x, W = p
    args = (bf16_dev(x), np_dev(ids), np_dev(w), np_dev(mask), *_dev(W))
    run = rep.MoEPrefill(*ids.shape, E, 512, 256, weights="mxfp4")
    eager = run(*args).clone()
    run.ffn_ws.fill_(255)
    assert torch.equal(run(*args).view(torch.int32), eager.view(torch.int32))
    # the stages again on one plan
    desc, rt = run.desc, run.rt
    rep.ffn_plan(desc, args[0], rt.offsets, run.ffn_ws)
    for _ in range(2):
        run.y.fill_(float("nan"))
        rep.ffn_gate_up(desc, args[0], rt.sorted_routes, args[4], args[5], args[7], args[8],
                        run.ffn_ws)
        rep.ffn_down(desc, rt.offsets, args[6], args[9], run.y, run.ffn_ws)
        out = rep.combine(run.y, rt.route_rows, args[2], args[3], row_limit=run.row_limit)
        assert torch.equal(out.view(torch.int32), eager.view(torch.int32))
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        run(*args)
    for _ in range(3):
        run.out.fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(run.out.view(torch.int32), eager.view(torch.int32))
        assert torch.equal(run(*args).view(torch.int32), eager.view(torch.int32))


@pytest.mark.parametrize("d,f", [(4864, 256), (128, 4736)])
def test_few_rows_of_a_long_reduction(d, f):
    """Rows too long for LDS: tiles of at most 16 rows then go through the
    ring, here with a last group of codes that is half there."""
    p = _problem([1, 16, 5, 17, 0, 9], 2, d, f, seed=d)
    E, ids, w, mask, x, W = p
    _, out = _run(p)
    _close(out, omoe.moe_ref_blocked(x, ids, w, mask, bf16_source(W), E)[0])


def test_not_a_number_stays_in_its_token():
    """Tiles of every height with a NaN and an infinity in one row each."""
    p = _problem(CLASS_COUNTS, 6, 384, 256, seed=12)
    E, ids, w, mask, x, W = p
    _, clean = _run(p)
    x = x.copy()
    x[3, 7], x[50, 300] = 0x7FC0, 0x7F80
    _, out = _run((E, ids, w, mask, x, W))
    read = (mask != 0).any(1)
    assert read[3] and read[50] and np.isnan(out[3]).all()
    rest = np.delete(np.arange(ids.shape[0]), [3, 50])
    assert np.array_equal(out[rest], clean[rest])


def test_an_expert_named_twice_by_a_token():
    p = _problem([20, 3, 0, 0], 4, 256, 128, seed=13, masked=0)
    E, ids, w, mask, x, W = p
    ids[:] = np.array([0, 1, 0, 0], np.int32)
    _, out = _run(p)
    _close(out, omoe.moe_ref_blocked(x, ids, w, mask, bf16_source(W), E)[0])


def test_two_streams_and_the_workspaces_end():
    """Two layers at once, each on a stream and in a workspace of its own, that
    write nothing behind the bytes they asked for."""
    import ctypes

    import torch

    import routed_expert_prefill_amd as rep

    lib = rep.load_library()
    runs = []
    for seed in (14, 15):
        p = _problem([70, 0, 300, 9, 130], 3, 512, 256, seed=seed)
        E, ids, w, mask, x, W = p
        layer = rep.MoEPrefill(*ids.shape, E, 512, 256, weights="mxfp4")
        layer.decode = False
        n = lib.moe_grouped_ffn_workspace(ctypes.byref(layer.desc))
        layer.ffn_ws = torch.full((n + 4096,), 0xA5, dtype=torch.uint8, device="cuda")
        runs.append((layer, n, (bf16_dev(x), np_dev(ids), np_dev(w), np_dev(mask), *_dev(W)),
                     _run(p)[1]))
    streams = [torch.cuda.Stream() for _ in runs]
    torch.cuda.synchronize()
    for _ in range(5):
        for s, (layer, _, args, _) in zip(streams, runs):
            with torch.cuda.stream(s):
                layer(*args)
    torch.cuda.synchronize()
    for layer, n, _, want in runs:
        assert np.array_equal(layer.out.cpu().numpy().astype(np.float64), want)
        assert (layer.ffn_ws[n:] == 0xA5).all()


@pytest.mark.parametrize("decode", [False, True])
def test_two_graphs_share_a_layer(decode):
    """Two captures of one layer, one workspace and one output, on other inputs
    each, replayed in turn between eager calls."""
    import torch

    import routed_expert_prefill_amd as rep

    counts = ([3, 0, 9, 8], [20, 0, 0, 0]) if decode else ([70, 0, 300, 9], [9, 200, 0, 170])
    problems = [_problem(c, 2, 512, 256, seed=30 + i, masked=379 - sum(c) if not decode else 0)
                for i, c in enumerate(counts)]
    layer = rep.MoEPrefill(*problems[0][1].shape, 4, 512, 256, weights="mxfp4")
    assert layer.decode == decode
    runs = []
    for E, ids, w, mask, x, W in problems:
        assert ids.shape == problems[0][1].shape
        args = (bf16_dev(x), np_dev(ids), np_dev(w), np_dev(mask), *_dev(W))
        eager = layer(*args).clone()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            layer(*args)
        runs.append((g, args, eager))
    for _ in range(3):
        for g, args, eager in runs:
            layer.out.fill_(float("nan"))
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(layer.out.view(torch.int32), eager.view(torch.int32))
            assert torch.equal(layer(*args).view(torch.int32), eager.view(torch.int32))


def test_refusals():
    import torch

    import routed_expert_prefill_amd as rep

    p = _problem([3, 4], 1, 256, 128, seed=11, masked=0)
    E, ids, w, mask, x, W = p
    rt = rep.route_build(np_dev(ids), np_dev(mask), E)
    names = ("w_gate", "w_up", "w_down", "s_gate", "s_up", "s_down")
    good = dict(zip(names, _dev(W)))

    def call(**kw):
        g = {**good, **kw}
        return rep.grouped_ffn(bf16_dev(x), rt.offsets, rt.sorted_routes, g["w_gate"], g["w_up"],
                               g["w_down"], 1, g["s_gate"], g["s_up"], g["s_down"])

    call()
    for bad in (dict(w_gate=good["w_gate"][:, :64].contiguous()), dict(w_down=good["w_up"]),
                dict(s_up=good["s_up"].float()), dict(s_up=None),
                dict(s_down=good["s_down"][:, :, :2].contiguous()),
                dict(w_up=good["w_up"].transpose(1, 2)), dict(s_up=good["s_up"].cpu())):
        with pytest.raises((TypeError, ValueError)):
            call(**bad)
    base = (bf16_dev(x), rt.offsets, rt.sorted_routes, *(good[n] for n in names[:3]), 1,
            *(good[n] for n in names[3:]))
    for bad in (dict(y=torch.empty(6, 256, device="cuda")), dict(y=torch.empty(7, 128, device="cuda")),
                dict(workspace=torch.empty(1 << 20, dtype=torch.uint8))):
        with pytest.raises(ValueError):
            rep.grouped_ffn(*base, **bad)
    with pytest.raises(RuntimeError, match="MOE_EWORKSPACE"):
        rep.grouped_ffn(*base, workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        rep.MoEPrefill(7, 1, 2, 256, 128, weights="int4")
    with pytest.raises(ValueError):
        rep.MoEPrefill(7, 1, 2, 256, 128, fp8=True, weights="mxfp4")
    with pytest.raises(TypeError):
        rep.MoEPrefill(7, 1, 2, 256, 128, weights="mxfp4", out_dtype=torch.float16)
