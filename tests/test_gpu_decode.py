"""GPU routed experts for single tokens (MXFP4) vs the formulas in 64 bits and
vs the grouped path.

Tolerances.  Against 64 bits: h is kept as two bf16 numbers, which leaves at
most 2^-8 of a rest of at most 2^-8 of it: 2^-16; fp32 sums of up to 8448
terms add sqrt(8448) x 2^-25 = 3e-6 of a row's norm, twice.  Relative Frobenius
1e-4, and one output, a sum of f >= 128 terms with |h| < 16 rms(h) and
|w| < 4 rms(w), moves by less than 2^-16 x 64 x sqrt(f) / sqrt(f) of the
outputs' rms: 2e-3.  Against the grouped path, which rounds h to bf16: at most
2^-8 of each h, so at most 2^-8 of the outputs' norm where the errors add at
random, and for one output 4.5 standard deviations of the rounding's rms
(2^-8 / sqrt(3)): 0.0102, taken as 0.012 of the outputs' rms."""
import numpy as np
import pytest

from oracle import numerics as nx
from gpu_util import bf16_dev, np_dev, rel_frob
from mxfp4_util import mx_weights, unrounded_ref
from test_gpu_ffn import _x
from test_gpu_mxfp4 import _dev
from test_gpu_norm import _call_both_ways

pytestmark = pytest.mark.gpu


def _close(got, ref, rel=1e-4, big=2e-3):
    r = rel_frob(got, ref)
    b = np.abs(got - ref).max() / np.sqrt(np.mean(ref * ref))
    assert r <= rel and b <= big, (r, b)


def _problem(T, k, E, d, f, seed, mask_p=0.0, same=False):
    rng = np.random.default_rng(seed)
    if same:  # every route names one expert
        ids = np.full((T, k), E - 1, np.int32)
    else:
        ids = np.stack([rng.permutation(E)[:k] for _ in range(T)]).astype(np.int32)
    w = rng.random((T, k)).astype(np.float32)
    mask = (rng.random((T, k)) >= mask_p).astype(np.uint8)
    return ids, w, mask, _x(T, d, seed + 1), mx_weights(E, d, f, seed + 2)


def _decode(p, **kw):
    import torch

    import routed_expert_prefill_amd as rep

    ids, w, mask, x, W = p
    out = rep.decode_ffn(bf16_dev(x), np_dev(ids), np_dev(w),
                         None if mask is None else np_dev(mask), *_dev(W), **kw)
    torch.cuda.synchronize()
    return out


def _ref(p):
    ids, w, mask, x, W = p
    return unrounded_ref(nx.bf16_bits_to_f64(x), ids, w, mask, W)


@pytest.mark.parametrize("T,k,E,d,f,mask_p,same", [
    (1, 1, 1, 128, 128, 0, False),  # one step, one half of the reduction empty
    (1, 6, 16, 512, 256, 0, False),
    (1, 6, 16, 4096, 2048, 0, False),  # the widths of the real layer
    (4, 6, 24, 4096, 2048, 0.05, False),
    (3, 5, 7, 1152, 640, 0.4, False),  # ragged shares of steps, shared experts
    (2, 16, 16, 384, 1152, 0, False),
    (64, 1, 3, 256, 384, 0, False),  # many rows to an expert
    (10, 6, 8, 640, 128, 0.3, False),
    (13, 4, 4, 256, 256, 0, True),  # 52 routes of one expert
    (1, 2, 5, 8448, 4352, 0, False),  # several rounds of loads per wave
    (64, 1, 64, 128, 128, 0, False),
])
def test_matches_oracle(T, k, E, d, f, mask_p, same):
    p = _problem(T, k, E, d, f, seed=T + k + d + f, mask_p=mask_p, same=same)
    out = _decode(p)
    _close(out.cpu().numpy().astype(np.float64), _ref(p))
    # the same bits on every call, and from a workspace that held something else
    assert (_decode(p).view(out.dtype) == out).all()


def test_matches_the_grouped_path():
    import torch

    import routed_expert_prefill_amd as rep

    p = _problem(8, 6, 32, 1024, 512, seed=3, mask_p=0.1)
    ids, w, mask, x, W = p
    args = (bf16_dev(x), np_dev(ids), np_dev(w), np_dev(mask), *_dev(W))
    layer = rep.MoEPrefill(8, 6, 32, 1024, 512, weights="mxfp4")
    assert layer.decode
    a = layer(*args).cpu().numpy().astype(np.float64)
    layer.decode = False
    b = layer(*args).cpu().numpy().astype(np.float64)
    _close(a, b, 2.0 ** -8, 0.012)
    ev = [torch.cuda.Event(enable_timing=True) for _ in range(6)]
    layer.decode = True
    c = layer(*args, stage_events=ev).cpu().numpy().astype(np.float64)  # by stages
    assert np.array_equal(b, c)
    assert not rep.MoEPrefill(11, 6, 32, 1024, 512, weights="mxfp4").decode
    assert not rep.MoEPrefill(1, 6, 32, 1024, 512).decode


def test_masked_and_out_of_range_routes():
    """Such routes add exact zeros and their gates are not read."""
    p = _problem(5, 4, 9, 256, 128, seed=4)
    ids, w, mask, x, W = p
    ids[0, 1], ids[1, 0], ids[2, 3] = 9, -1, 2 ** 31 - 1
    mask[3], mask[4, 0], mask[4, 2] = 0, 0, 0
    off = (mask == 0) | (ids < 0) | (ids >= 9)
    want = _ref((ids, np.where(off, 0, w).astype(np.float32), mask, x, W))
    w[off] = np.nan
    out = _decode(p).cpu().numpy().astype(np.float64)
    assert not out[3].any() and not np.signbit(out[3]).any()
    _close(out, want)
    # without a mask only the ids decide
    w = np.where((ids < 0) | (ids >= 9), np.nan, 0.5).astype(np.float32)
    _close(_decode((ids, w, None, x, W)).cpu().numpy().astype(np.float64),
           _ref((ids, np.nan_to_num(w), None, x, W)))


def test_outputs_and_shared_rows():
    import torch

    import routed_expert_prefill_amd as rep

    p = _problem(3, 2, 4, 384, 256, seed=5, mask_p=0.3)
    shared = np.random.default_rng(1).standard_normal((3, 384)).astype(np.float32)
    plain = _decode(p)
    both = _decode(p, shared=np_dev(shared))
    assert torch.equal(both, plain + np_dev(shared))
    rows = torch.full((5, 384), 7.0, dtype=torch.bfloat16, device="cuda:0")
    out = _decode(p, shared=np_dev(shared), out=rows[:3])
    assert torch.equal(out.view(torch.int16), both.to(torch.bfloat16).view(torch.int16))
    assert (rows[3:] == 7).all()
    assert _decode(p, out_dtype=torch.bfloat16).dtype == torch.bfloat16


def test_not_a_number_stays_in_its_token():
    p = _problem(4, 2, 4, 256, 128, seed=6)
    clean = _decode(p).cpu().numpy()
    ids, w, mask, x, W = p
    x = x.copy()
    x[1, 7] = 0x7FC0
    out = _decode((ids, w, mask, x, W)).cpu().numpy()
    assert np.isnan(out[1]).all()
    assert np.array_equal(np.delete(out, 1, 0), np.delete(clean, 1, 0))


def test_graph_replays():
    import torch

    import routed_expert_prefill_amd as rep

    p = _problem(2, 6, 16, 512, 256, seed=7)
    ids, w, mask, x, W = p
    args = (bf16_dev(x), np_dev(ids), np_dev(w), np_dev(mask), *_dev(W))
    layer = rep.MoEPrefill(2, 6, 16, 512, 256, weights="mxfp4", out_dtype=torch.bfloat16)
    eager = layer(*args).clone()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        layer(*args)
    for i in range(4):
        layer.out.fill_(float("nan"))
        layer.ffn_ws.fill_(255)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(layer.out.view(torch.int16), eager.view(torch.int16))
        # other ids through the same graph, and back
        args[1].copy_(np_dev((ids + 1 + i) % 16))
        g.replay()
        torch.cuda.synchronize()
        assert not torch.equal(layer.out.view(torch.int16), eager.view(torch.int16))
        args[1].copy_(np_dev(ids))


def test_two_streams_and_the_workspaces_end():
    import torch

    import routed_expert_prefill_amd as rep

    lib = rep.load_library()
    runs = []
    for seed in (17, 18):
        p = _problem(5, 4, 12, 640, 384, seed=seed, mask_p=0.2)
        ids, w, mask, x, W = p
        n = lib.moe_decode_ffn_workspace(rep.ffn_desc(5, 4, 12, 640, 384, weights="mxfp4"))
        ws = torch.full((n + 4096,), 0xA5, dtype=torch.uint8, device="cuda")
        out = torch.full((7, 640), 7.0, device="cuda")
        runs.append(((bf16_dev(x), np_dev(ids), np_dev(w), np_dev(mask), *_dev(W)), n, ws, out,
                     _decode(p)))
    streams = [torch.cuda.Stream() for _ in runs]
    torch.cuda.synchronize()
    for _ in range(5):
        for s, (args, _, ws, out, _) in zip(streams, runs):
            with torch.cuda.stream(s):
                rep.decode_ffn(*args, out=out[:5], workspace=ws)
    torch.cuda.synchronize()
    for _, n, ws, out, want in runs:
        assert torch.equal(out[:5].view(torch.int32), want.view(torch.int32))
        assert (out[5:] == 7).all() and (ws[n:] == 0xA5).all()


def test_with_and_without_the_extension(monkeypatch):
    import torch

    import routed_expert_prefill_amd as rep

    p = _problem(5, 4, 12, 640, 384, seed=21, mask_p=0.2)
    ids, w, mask, x, W = p
    shared = torch.randn(5, 640, device="cuda")
    args = (bf16_dev(x), np_dev(ids), np_dev(w), np_dev(mask), *_dev(W))
    for mask_too in (True, False):
        for dtype in (torch.float32, torch.bfloat16):
            layer = rep.MoEPrefill(5, 4, 12, 640, 384, weights="mxfp4", out_dtype=dtype)
            call = args if mask_too else (*args[:3], None, *args[4:])

            def run():
                layer.out.fill_(float("nan"))
                return layer(*call, shared=shared).clone()

            a, b, used = _call_both_ways(monkeypatch, run)
            assert used is True and torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    # what the module leaves to the Python code
    layer = rep.MoEPrefill(5, 4, 12, 640, 384, weights="mxfp4")
    for i, bad in ((0, args[0][:3]), (1, args[1].long()), (2, args[2].cpu()), (3, args[3].bool()),
                   (4, args[4].transpose(0, 1)), (6, args[4]), (9, args[9].float())):
        call = (*args[:i], bad, *args[i + 1:])

        def run():
            with pytest.raises((TypeError, ValueError)) as e:
                layer(*call)
            return str(e.value)

        a, b, used = _call_both_ways(monkeypatch, run)
        assert a == b and used is None


def test_refusals():
    import torch

    import routed_expert_prefill_amd as rep

    ids, w, mask, x, W = _problem(3, 2, 4, 256, 128, seed=8)
    names = ("x", "topk_ids", "topk_w", "route_mask", "w_gate", "w_up", "w_down", "s_gate", "s_up",
             "s_down")
    good = dict(zip(names, (bf16_dev(x), np_dev(ids), np_dev(w), np_dev(mask), *_dev(W))))
    rep.decode_ffn(**good)
    for bad in (dict(x=good["x"].float()), dict(x=good["x"][:2]), dict(x=good["x"][:0]),
                dict(x=good["x"].cpu()), dict(topk_ids=good["topk_ids"].long()),
                dict(topk_w=good["topk_w"][:, :1]), dict(route_mask=good["route_mask"][:2]),
                dict(w_gate=good["w_down"]), dict(s_up=good["s_up"].float()),
                dict(s_down=good["s_gate"]), dict(w_up=good["w_up"].cpu()),
                dict(shared=torch.zeros(3, 128, device="cuda")),
                dict(out=torch.zeros(3, 256, device="cuda", dtype=torch.float16)),
                dict(w_down=good["w_down"].transpose(0, 1)),
                dict(workspace=torch.empty(4096, dtype=torch.uint8)),
                dict(out=torch.zeros(2, 256, device="cuda"))):
        with pytest.raises((TypeError, ValueError)):
            rep.decode_ffn(**{**good, **bad})
    with pytest.raises(RuntimeError, match="MOE_EWORKSPACE"):
        rep.decode_ffn(**good, workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
    many = _problem(33, 2, 4, 128, 128, seed=9)
    with pytest.raises(RuntimeError, match="MOE_EUNSUPPORTED"):
        _decode(many)
