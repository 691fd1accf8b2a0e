"""The status of a call is that of its own launches: an error that an earlier
HIP call left on the thread is neither reported nor cleared."""

import pytest

from gpu_util import bf16_dev, np_dev
from test_gpu_decode import _problem
from test_gpu_mxfp4 import _dev

pytestmark = pytest.mark.gpu


@pytest.fixture
def stale():
    """Returns a function that leaves an error on this thread and returns its
    number, and one that reads the number that is there."""
    import torch

    import routed_expert_prefill_amd as rep

    torch.cuda.synchronize()
    hip = rep.load_library()  # whose handle finds the HIP runtime it is linked to

    def leave():
        hip.hipGetLastError()
        bad = hip.hipSetDevice(1 << 20)
        assert bad != 0 and hip.hipPeekAtLastError() == bad
        return bad

    yield leave, hip.hipPeekAtLastError
    hip.hipGetLastError()
    assert hip.hipPeekAtLastError() == 0


@pytest.mark.parametrize("native", [True, False])
def test_norm_in_place(stale, monkeypatch, native):
    import torch

    import routed_expert_prefill_amd as rep

    leave, last = stale
    g = torch.Generator().manual_seed(1)
    x, r = (torch.randn(5, 640, generator=g).to(torch.bfloat16).cuda() for _ in range(2))
    w = torch.ones(640, dtype=torch.bfloat16, device="cuda")
    want = rep.add_rmsnorm(x, w, residual=r)
    got, y = r.clone(), torch.empty_like(x)
    if native:
        assert rep._native() is not None
    else:
        monkeypatch.setattr(rep, "_native", lambda: None)
    torch.cuda.synchronize()
    bad = leave()
    rep.add_rmsnorm(x, w, residual=got, residual_out=got, y=y)
    assert last() == bad
    rep.load_library().hipGetLastError()
    torch.cuda.synchronize()
    assert torch.equal(got.view(torch.int16), want[1].view(torch.int16))
    assert torch.equal(y.view(torch.int16), want[0].view(torch.int16))


def test_experts(stale):
    import torch

    import routed_expert_prefill_amd as rep

    leave, last = stale
    ids, w, mask, x, W = _problem(5, 4, 12, 640, 384, seed=2)
    args = (bf16_dev(x), np_dev(ids), np_dev(w), np_dev(mask), *_dev(W))
    layer = rep.MoEPrefill(5, 4, 12, 640, 384, weights="mxfp4")
    want = layer(*args).clone()
    rt = rep.route_build(args[1], args[3], 12)
    y, ws = torch.empty(20, 640, device="cuda"), layer.ffn_ws
    rows = rep.grouped_ffn(args[0], rt.offsets, rt.sorted_routes, *args[4:7], 4, *args[7:], y=y,
                           workspace=ws).clone()
    layer.out.fill_(float("nan"))
    y.fill_(float("nan"))
    n = int(rt.offsets[12])
    torch.cuda.synchronize()
    bad = leave()
    layer(*args)
    rep.grouped_ffn(args[0], rt.offsets, rt.sorted_routes, *args[4:7], 4, *args[7:], y=y,
                    workspace=ws)
    assert last() == bad
    rep.load_library().hipGetLastError()
    torch.cuda.synchronize()
    assert torch.equal(layer.out.view(torch.int32), want.view(torch.int32))
    assert torch.equal(y[:n].view(torch.int32), rows[:n].view(torch.int32))


@pytest.mark.parametrize("weights", ["bf16", "fp8"])
def test_the_path(stale, weights):
    """Router, route builds, row codes, FFN (fp8: on codes too) and combines."""
    import torch

    import routed_expert_prefill_amd as rep

    leave, last = stale
    T, k, E, d, f = 900, 6, 16, 256, 128  # more routes than one workgroup builds
    g = torch.Generator("cuda").manual_seed(3)
    x = torch.randn(T, d, generator=g, device="cuda", dtype=torch.bfloat16)
    logits = torch.randn(T, E, generator=g, device="cuda")
    shared = torch.randn(T, d, generator=g, device="cuda")
    shapes = ((E, f, d), (E, f, d), (E, d, f))
    if weights == "bf16":
        W = [torch.randn(s, generator=g, device="cuda", dtype=torch.bfloat16) * 0.05 for s in shapes]
        S = [None] * 3
    else:
        W = [torch.randint(0, 120, s, generator=g, device="cuda", dtype=torch.uint8) for s in shapes]
        S = [torch.rand(E, s[1] // 128, s[2] // 128, generator=g, device="cuda") for s in shapes]
    ids, w = rep.route_topk(logits, k)
    rt, few = rep.route_build(ids, None, E), rep.route_build(ids[:4].contiguous(), None, E)
    rbw = torch.empty(1 << 20, dtype=torch.uint8, device="cuda")
    desc = rep.ffn_desc(T, k, E, d, f, weights=weights)
    ws = torch.empty(rep.load_library().moe_grouped_ffn_workspace(desc), dtype=torch.uint8,
                     device="cuda")
    y, out, both = (torch.zeros(n, d, device="cuda") for n in (T * k, T, T))
    q, s = rep.quant_rows_fp8(x)
    yq, ids4 = torch.zeros_like(y), ids[:4].contiguous()

    def calls():
        rep.route_topk(logits, k, topk_ids=ids, topk_w=w)
        rep.route_build(ids, None, E, out=rt, workspace=rbw)
        rep.route_build(ids4, None, E, out=few, workspace=rbw)
        rep.route_build_noalloc(ids4, None, E, out=few)
        rep.quant_rows_fp8(x, q=q, s=s)
        rep.grouped_ffn(x, rt.offsets, rt.sorted_routes, *W, k, *S, y=y, workspace=ws)
        if weights == "fp8":
            rep.grouped_ffn_codes(q, s, rt.offsets, rt.sorted_routes, *W, k, *S, y=yq, workspace=ws)
        rep.combine(y, rt.route_rows, w, None, out=out)
        rep.combine_shared(y, rt.route_rows, w, None, shared=shared, out=both)

    outputs = [ids, w, *rt, *few, q, s, y, yq, out, both]
    calls()
    want = [t.clone() for t in outputs]
    for t in outputs:
        t.zero_()
    torch.cuda.synchronize()
    bad = leave()
    calls()
    assert last() == bad
    rep.load_library().hipGetLastError()
    torch.cuda.synchronize()
    for t, u in zip(outputs, want):
        assert torch.equal(t.view(torch.uint8), u.view(torch.uint8))
