"""Calls of the dense operators that pair kernels otherwise not seen together, or share
buffers between calls as a serving loop does."""
import numpy as np
import pytest

from dense_util import bf16_room, dev, exact_problem, host, random_problem, two_powers, whole_codes
from oracle import dense
from test_gpu_dense import _shared_bounds

pytestmark = pytest.mark.gpu


# tiles for gate and up with h in fp32, or in codes, in front of few rows' down product;
# the few rows' kernel in front of tiles
@pytest.mark.parametrize("T,d,f", [(16, 4096, 4096), (16, 256, 8192), (16, 16384, 640), (17, 16384, 128)])
def test_kernels_of_both_kinds_in_one_call(T, d, f):
    import torch

    import routed_expert_prefill_amd as rep

    rng = np.random.default_rng(T + d)
    q, xs = whole_codes(rng, (T, d)), two_powers(rng, (T, d // 128))
    wg, wu, wd = whole_codes(rng, (f, d)), whole_codes(rng, (f, d)), whole_codes(rng, (d, f))
    small = np.float32(2.0 ** -round(np.log2(8 * d ** 0.5)))
    sg, su = (two_powers(rng, (f // 128, d // 128)) * small for _ in range(2))
    sd = (rng.random((d // 128, f // 128)) + 0.5).astype(np.float32)
    want, room, either, _ = _shared_bounds(q, xs, wg, wu, wd, sg, su, sd)
    assert either.mean() < 0.05
    rows, W = tuple(dev(q, xs)), dev(wg, wu, wd, sg, su, sd)
    off = np.abs(host(rep.shared_ffn(rows, *W)) - want)
    assert (off <= room).all(), (off / room).max()
    low = host(rep.shared_ffn(rows, *W, out_dtype=torch.bfloat16))
    assert (np.abs(low - want) <= room + 2.0 ** -8 * (np.abs(want) + room)).all()
    x = torch.randn(T, d, generator=torch.Generator().manual_seed(T)).to(torch.bfloat16).cuda()
    a, b = rep.shared_ffn(x, *W), rep.shared_ffn(rep.quant_blocks_fp8(x), *W)
    room = _shared_bounds(*(t.cpu().numpy() for t in rep.quant_blocks_fp8(x)), wg, wu, wd, sg, su, sd)[1]
    assert (np.abs(host(a) - host(b)) <= 2 * room).all()


def test_one_workspace_for_every_number_of_rows():
    """A workspace for the most rows serves fewer, whatever kernels they take and
    whatever the call before left in it."""
    import torch

    import routed_expert_prefill_amd as rep

    d, f, most = 640, 1280, 2100
    lib = rep.load_library()
    W = dev(*(t for i, (n, k) in enumerate(((f, d), (f, d), (d, f))) for t in random_problem(i, 1, n, k)[2:3]),
            *(np.full((n // 128, k // 128), 2.0 ** -9, np.float32) for n, k in ((f, d), (f, d), (d, f))))
    room = torch.full((lib.moe_shared_ffn_workspace(most, d, f),), 0x7F, dtype=torch.uint8, device="cuda")
    keep = torch.full((lib.moe_matmul_fp8_workspace(most, f, d) + 512,), 0x7F, dtype=torch.uint8, device="cuda")
    x = torch.randn(most, d, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).cuda()
    for T in (most, 1, 401, 16, 33, 1030, 17, 5, 300, most):
        y = x[:T].contiguous()
        for kw in (dict(), dict(out_dtype=torch.bfloat16), dict(out_dtype=torch.bfloat16, short_sums=True)):
            assert torch.equal(rep.shared_ffn(y, *W, workspace=room, **kw), rep.shared_ffn(y, *W, **kw)), T
            assert torch.equal(rep.matmul_fp8(y, W[0], W[3], workspace=keep, **kw),
                               rep.matmul_fp8(y, W[0], W[3], **kw)), T
    assert (keep[-512:] == 0x7F).all()


def test_two_graphs_with_one_workspace_replayed_in_turn():
    import torch

    import routed_expert_prefill_amd as rep

    d, f = 512, 384
    W = dev(*(random_problem(i, 1, n, k)[2] for i, (n, k) in enumerate(((f, d), (f, d), (d, f)))),
            *(np.full((n // 128, k // 128), 2.0 ** -9, np.float32) for n, k in ((f, d), (f, d), (d, f))))
    room = torch.empty(rep.load_library().moe_shared_ffn_workspace(300, d, f), dtype=torch.uint8, device="cuda")
    xs = [torch.randn(T, d, generator=torch.Generator().manual_seed(T)).to(torch.bfloat16).cuda() for T in (300, 7)]
    want = [rep.shared_ffn(x, *W) for x in xs]
    graphs = []
    for x in xs:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = rep.shared_ffn(x, *W, workspace=room)
        graphs.append((graph, out))
    for i in (0, 1, 1, 0, 1, 0):
        graph, out = graphs[i]
        out.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[i])
        room.fill_(0x7F)


@pytest.mark.parametrize("M", [1, 40, 300])
def test_scales_of_zero_and_one_buffer_for_both_weights(M):
    """Blocks whose scale is 0 count nothing; gate and up may be one matrix."""
    import torch

    import routed_expert_prefill_amd as rep

    q, xs, w, ws = exact_problem(M, M, 256, 512)
    xs[:, 1] = 0
    ws[1, 2] = 0
    got = host(rep.matmul_fp8(tuple(dev(q, xs)), *dev(w, ws)))
    assert np.array_equal(got, dense.matmul(q, xs, w, ws))
    wd = whole_codes(np.random.default_rng(M), (512, 256))
    sd = np.ones((4, 2), np.float32)
    ws *= np.float32(2.0 ** -6)
    p = (q, xs, w, w, wd, ws, ws, sd)
    want, room, _, total = _shared_bounds(*p)
    dw, dws = dev(w, ws)
    rows = tuple(dev(q, xs))
    dwd, dsd = dev(wd, sd)
    off = np.abs(host(rep.shared_ffn(rows, dw, dw, dwd, dws, dws, dsd)) - want)
    assert (off <= room).all()
    low = host(rep.shared_ffn(rows, dw, dw, dwd, dws, dws, dsd, out_dtype=torch.bfloat16, short_sums=True))
    assert (np.abs(low - want) <= room + bf16_room(256, total, want)).all()
