"""The operators as a served layer runs them one after another: the residual's
addition and norm, the router, the routed experts (fp8 rows fed with the norm's
codes; MXFP4 for a prompt and for single tokens), and the next layer's norm
taking their output.  Each step is held to its own reference on the inputs that
it really got, with the tolerances of its own tests."""
import numpy as np
import pytest

from oracle import moe as omoe
from oracle import numerics as nx
from oracle.router import route_topk as topk_ref
from gpu_util import np_dev, rel_frob, routing_with_counts
from mxfp4_util import bf16_source, mx_weights, unrounded_ref
from test_gpu_ffn import FP8_TOL, _dev_weights, _weights, _x
from test_gpu_mxfp4 import _close, _dev
from test_gpu_norm import _check

pytestmark = pytest.mark.gpu


def _bits(t):
    import torch

    return t.cpu().view(torch.int16).numpy().view(np.uint16)


def _stream(T, d, seed):
    import torch

    g = torch.Generator().manual_seed(seed)
    return [torch.randn(T, d, generator=g).to(torch.bfloat16) for _ in range(2)] + [
        (1 + 0.1 * torch.randn(d, generator=g)).to(torch.bfloat16) for _ in range(2)]


@pytest.mark.parametrize("T,k,E,d,f", [(1, 6, 16, 512, 256), (9, 4, 12, 384, 128),
                                       (150, 3, 10, 640, 384)])
def test_mxfp4_layer(T, k, E, d, f):
    import torch

    import routed_expert_prefill_amd as rep

    x, res, w1, w2 = _stream(T, d, seed=T + d)
    W = mx_weights(E, d, f, seed=5)
    wr = np.random.default_rng(3).standard_normal((d, E)).astype(np.float32) * 0.05
    layer = rep.MoEPrefill(T, k, E, d, f, weights="mxfp4", out_dtype=torch.bfloat16)
    assert layer.decode == (T * k <= 64)
    dx, dres, dw1, dw2 = (t.cuda() for t in (x, res, w1, w2))
    y, res1, _, _ = rep.add_rmsnorm(dx, dw1, residual=dres)
    logits = y.float() @ np_dev(wr)
    ids, gates = rep.route_topk(logits, k)
    out = layer(y, ids, gates, None, *_dev(W))
    y2, res2, _, _ = rep.add_rmsnorm(out, dw2, residual=res1, residual_out=res1)
    torch.cuda.synchronize()
    _check((y, None, None, None), x, res, w1, 1e-6)
    ids_ref, _ = topk_ref(logits.cpu().numpy(), None, k)
    assert np.array_equal(ids.cpu().numpy(), ids_ref)
    if layer.decode:  # h not rounded to bf16
        ref = unrounded_ref(nx.bf16_bits_to_f64(_bits(y)), ids.cpu().numpy(), gates.cpu().numpy(),
                            None, W)
    else:
        ref = omoe.moe_ref_blocked(_bits(y), ids.cpu().numpy(), gates.cpu().numpy(), None,
                                   bf16_source(W), E)[0]
    got = nx.bf16_bits_to_f64(_bits(out))
    # bf16 rounding of the output on top: at most 2^-8, 2^-9 in the mean
    assert rel_frob(got, ref) <= 1e-3 + 2.0 ** -9
    first = (res.float() + x.float()).to(torch.bfloat16)
    _check((y2, res2, None, None), out.cpu(), first, w2, 1e-6)


def _fp8_problem(seed):
    counts, k, d, f = [31, 0, 70, 200, 300, 5], 3, 512, 256
    ids, mask = routing_with_counts(counts, k, seed=seed, masked_extra=7)
    w = np.random.default_rng(seed).random(ids.shape).astype(np.float32)
    return len(counts), k, d, f, ids, mask, w, _weights(len(counts), d, f, True, seed + 1)


def test_fp8_on_given_codes_is_the_fp8_path():
    import torch

    import routed_expert_prefill_amd as rep

    E, k, d, f, ids, mask, w, W = _fp8_problem(1)
    T = ids.shape[0]
    x = torch.from_numpy(_x(T, d, 4).view(np.int16)).view(torch.bfloat16).cuda()
    Wd = _dev_weights(W, True)
    weights = [Wd[n] for n in ("wg", "wu", "wd", "sg", "su", "sd")]
    args = (np_dev(ids), np_dev(w), np_dev(mask), *weights)
    layer = rep.MoEPrefill(T, k, E, d, f, fp8=True)
    want = layer(x, *args).clone()
    q, s = rep.quant_rows_fp8(x)
    q0, s0 = q.clone(), s.clone()
    for _ in range(2):
        layer.ffn_ws.fill_(255)
        layer.y.fill_(float("nan"))
        got = layer((q, s), *args)
        assert torch.equal(got.view(torch.int32), want.view(torch.int32))
    assert torch.equal(q, q0) and torch.equal(s, s0)
    with pytest.raises(ValueError):
        layer((q, s), *args, stage_events=[None] * 6)
    with pytest.raises(ValueError):
        rep.MoEPrefill(T, k, E, d, f)((q, s), *args)
    # on a stream of its own, and replayed
    with torch.cuda.stream(torch.cuda.Stream()):
        got = layer((q, s), *args)
        torch.cuda.synchronize()
        assert torch.equal(got.view(torch.int32), want.view(torch.int32))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        layer((q, s), *args)
    for _ in range(3):
        layer.out.fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(layer.out.view(torch.int32), want.view(torch.int32))
        assert torch.equal(layer(x, *args).view(torch.int32), want.view(torch.int32))
    rt = layer.rt
    for bad in (dict(y=layer.y[1:]), dict(y=layer.y[:, :256].contiguous()),
                dict(workspace=layer.ffn_ws.cpu()), dict(xq=q[:, :256].contiguous()), dict(xs=s[:5]), dict(xq=x), dict(xs=s.cpu()),
                dict(w_down=Wd["wg"]), dict(s_up=Wd["sd"]), dict(offsets=rt.counts)):
        a = dict(xq=q, xs=s, offsets=rt.offsets, sorted_routes=rt.sorted_routes, k=k,
                 **dict(zip(("w_gate", "w_up", "w_down", "s_gate", "s_up", "s_down"), weights)))
        with pytest.raises((TypeError, ValueError)):
            rep.grouped_ffn_codes(**{**a, **bad})


def test_fp8_layer_takes_the_norms_codes():
    import torch

    import routed_expert_prefill_amd as rep

    E, k, d, f, ids, mask, w, W = _fp8_problem(2)
    T = ids.shape[0]
    x, res, w1, _ = _stream(T, d, seed=7)
    y, _, q, s = rep.add_rmsnorm(x.cuda(), w1.cuda(), residual=res.cuda(), want_fp8=True)
    Wd = _dev_weights(W, True)
    layer = rep.MoEPrefill(T, k, E, d, f, fp8=True)
    out = layer((q, s), np_dev(ids), np_dev(w), np_dev(mask),
                *[Wd[n] for n in ("wg", "wu", "wd", "sg", "su", "sd")])
    torch.cuda.synchronize()
    _check((y, None, q, s), x, res, w1, 1e-6)
    # the same codes through the definitions
    xr = nx.e4m3_decode(q.cpu().numpy()) * s.cpu().numpy().astype(np.float64)[:, None]
    ref = np.zeros((T, d))
    for e in range(E):
        We = omoe.dequant_expert({n: W[n][e] for n in W}, True)
        for t, j in zip(*np.nonzero((ids == e) & (mask != 0))):
            h = omoe.h_operand(We["wg"] @ xr[t], We["wu"] @ xr[t], True)
            ref[t] += float(w[t, j]) * (We["wd"] @ h)
    got = out.cpu().numpy().astype(np.float64)
    assert np.abs(got - ref).max() <= FP8_TOL[0] and rel_frob(got, ref) <= FP8_TOL[1]
