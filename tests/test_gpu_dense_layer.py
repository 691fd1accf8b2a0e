"""The operators as a served layer runs them: residual and norm, router, expert
selection by groups, routed experts, shared expert."""
import numpy as np
import pytest

from dense_util import dev, host
from helpers import small_problem
from oracle import dense, moe as omoe, numerics as nx
from oracle.select import route_select as select_ref
from gpu_util import bf16_dev

pytestmark = pytest.mark.gpu
E, K, D, F, FS = 16, 4, 512, 256, 384


def _weights(seed):
    import torch

    _, _, _, _, W = small_problem(seed, 1, E, K, D, F)
    rng = np.random.default_rng(seed)
    S = []
    for rows, cols in ((FS, D), (FS, D), (D, FS)):
        S.append(nx.e4m3_encode(np.clip(rng.standard_normal((rows, cols)) * 112, -448, 448)))
    S += [(rng.uniform(0.5, 2.0, (w.shape[0] // 128, w.shape[1] // 128)) * 0.05 / 112).astype(np.float32) for w in S]
    router = torch.from_numpy(rng.standard_normal((D, E)).astype(np.float32) * 0.05)
    return W, S, router


@pytest.mark.parametrize("T", [1, 5, 70, 300])
def test_a_layer(T):
    import torch

    import routed_expert_prefill_amd as rep

    W, S, router = _weights(T)
    g = torch.Generator().manual_seed(T)
    x, res = (torch.randn(T, D, generator=g).to(torch.bfloat16).cuda() for _ in range(2))
    norm_w = torch.ones(D, dtype=torch.bfloat16, device="cuda")
    bias = (0.1 * torch.randn(E, generator=g)).cuda()
    dW, dS, dr = [bf16_dev(W[n]) for n in ("wg", "wu", "wd")], dev(*S), router.cuda()
    layer = rep.MoEPrefill(T, K, E, D, F)
    keep = {}

    def run(x, res):
        y, res, _, _ = rep.add_rmsnorm(x, norm_w, residual=res)
        logits = y.float() @ dr
        ids, w = rep.route_select(logits, K, bias=bias, groups=4, top_groups=2, scale=2.5)
        shared = rep.shared_ffn(y, *dS)
        out = layer(y, ids, w, None, *dW, shared=shared)
        keep.update(y=y, logits=logits, ids=ids, w=w, shared=shared)
        return out

    out = run(x, res).clone()
    y, logits = keep["y"], keep["logits"]
    ids, w = keep["ids"].cpu().numpy(), keep["w"].cpu().numpy()
    ri, rw = select_ref(logits.cpu().numpy(), K, bias=bias.cpu().numpy(), groups=4, top_groups=2, scale=2.5)
    assert np.array_equal(ids, ri) and (np.abs(w - rw) <= np.spacing(rw)).all()
    yb = y.view(torch.int16).cpu().numpy().view(np.uint16)
    routed = omoe.moe_ref_per_token(yb, ids, w, np.ones((T, K), np.uint8), omoe.dict_source(W), E)
    # the shared rows have tests of their own; here that they are those of the formulas at all:
    # a code of h is half a step off its value, 2^-4 of it, x's codes likewise
    q, xs = dense.quant_blocks(y.float().cpu().numpy())
    want = dense.shared_hidden(q, xs, S[0], S[1], S[3], S[4]) @ dense.weight_values(S[2], S[5]).T
    shared = host(keep["shared"])
    assert np.linalg.norm(shared - want) <= 2.0 ** -4 * np.linalg.norm(want)
    got = host(out)
    ref = routed + shared
    assert np.abs(got - ref).max() <= 2e-2 and np.linalg.norm(got - ref) <= 1e-3 * np.linalg.norm(ref)

    # the same in a graph, with other inputs between the replays
    gx, gr = x.clone(), res.clone()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cap = run(gx, gr)
    for i in range(4):
        nx_, nr = (torch.randn(T, D, generator=g).to(torch.bfloat16).cuda() for _ in range(2))
        if i == 2:
            nx_, nr = x, res
        eager = run(nx_, nr).clone()
        gx.copy_(nx_)
        gr.copy_(nr)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(cap, eager)
        if i == 2:
            assert torch.equal(cap, out)


def test_an_earlier_error_is_neither_reported_nor_cleared():
    import torch

    import routed_expert_prefill_amd as rep

    _, S, _ = _weights(1)
    dS = dev(*S)
    x = torch.randn(70, D, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).cuda()
    z = torch.randn(70, E, generator=torch.Generator().manual_seed(2)).cuda()
    calls = (lambda: rep.route_select(z, K), lambda: rep.quant_blocks_fp8(x),
             lambda: [rep.matmul_fp8(x, dS[0], dS[3])], lambda: [rep.shared_ffn(x, *dS)],
             lambda: [rep.shared_ffn(x[:1], *dS)])
    want = [[t.clone() for t in c()] for c in calls]
    hip = rep.load_library()
    torch.cuda.synchronize()
    try:
        hip.hipGetLastError()
        bad = hip.hipSetDevice(1 << 20)
        assert bad != 0
        got = []
        for c in calls:
            got.append(c())
            assert hip.hipPeekAtLastError() == bad
    finally:
        hip.hipGetLastError()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for x, y in zip(got, want) for a, b in zip(x, y))
