"""GPU MXFP4 paths at the ends of their ranges: the longest rows of the direct
way and the first past them, and the smallest scales."""
import numpy as np
import pytest

from oracle import moe as omoe
from oracle import numerics as nx
from gpu_util import bf16_dev, np_dev
from mxfp4_util import bf16_source
from test_gpu_mxfp4 import _close, _dev, _problem, _run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d,f", [
    (4736, 128), (128, 4736),  # the longest reduction whose rows fit LDS
    (4864, 128), (128, 4864),  # the ring, whole groups of codes
    (4992, 128), (128, 4992),  # the ring, a last group that is half there
])
def test_few_rows_about_the_longest_row_in_lds(d, f):
    """Tiles of at most 16 rows in either projection, beside one of 17."""
    p = _problem([1, 16, 5, 17, 0, 9], 2, d, f, seed=d + f)
    E, ids, w, mask, x, W = p
    _, out = _run(p)
    _close(out, omoe.moe_ref_blocked(x, ids, w, mask, bf16_source(W), E)[0])


def _one_hot(sel, d, f):
    """Tokens whose x has one element, and expert weights such that u is one
    weight times that element, exactly: token i reads column c of scale group
    sel[i], whose up scale is the byte sel[i], all codes among the rows."""
    n = len(sel)
    e = np.clip(140 - sel, None, 127)  # x = 2^e
    x = np.zeros((n, d), np.uint16)
    col = 32 * np.arange(n) + (5 * np.arange(n)) % 32
    x[np.arange(n), col] = (e + 127) << 7  # bf16 2^e
    wg = np.zeros((f, d), np.uint8)
    wu = np.zeros((f, d), np.uint8)
    sg = np.full((f, d // 32), 127, np.uint8)
    su = np.full((f, d // 32), 127, np.uint8)
    rows = np.arange(f)
    for i, c in enumerate(col):
        wg[:, c] = 2  # 1.0, scaled so that g = 32
        sg[:, i] = 132 - e[i]
        wu[:, c] = (rows + c) % 16
        su[:, i] = sel[i]
    wd = np.zeros((d, f), np.uint8)
    wd[rows, rows] = 2
    pack = lambda a: a[None, :, 0::2] | a[None, :, 1::2] << 4  # noqa: E731
    W = {"wg": pack(wg), "wu": pack(wu), "wd": pack(wd), "sg": sg[None], "su": su[None],
         "sd": np.full((1, d, f // 32), 127, np.uint8)}
    val = nx.mxfp4_decode(W["wu"][0], W["su"][0])[:, col].T  # [n, f], exact
    return x, W, 32 * val * np.exp2(e.astype(np.float64))[:, None]


@pytest.mark.parametrize("way,sel", [
    ("item", np.arange(0, 128)), ("item", np.arange(125, 253)),
    ("direct", np.arange(0, 16)), ("direct", np.arange(237, 253)),
    ("ring", np.arange(0, 16)), ("stream", np.arange(0, 64)), ("tall", np.arange(0, 128)),
    ("decode", np.arange(0, 32)), ("decode", np.arange(221, 253)),
])
def test_every_code_under_every_scale_is_exact(way, sel):
    """The weights of scale byte 0 and up, subnormal ones among them, come out
    whole: u = w x, h = silu(32) u = 32 u to less than fp32's half step (it has
    two significant bits, so no rounding touches it), and y = h."""
    import torch

    import routed_expert_prefill_amd as rep

    d, f = {"item": (4096, 128), "tall": (4096, 256), "direct": (1024, 128), "ring": (4864, 128),
            "stream": (2048, 256), "decode": (1024, 128)}[way]
    x, W, want = _one_hot(sel, d, f)
    n, E = len(sel), 1
    if way in ("stream", "tall"):  # as many such experts as give the workgroups a second round
        E = 200
        W = {k: np.repeat(v, E, 0) for k, v in W.items()}
        x, want = np.tile(x, (E, 1)), np.tile(want, (E, 1))
    T = len(x)
    ids = (np.arange(T) // n).astype(np.int32)[:, None]
    args = (bf16_dev(x), np_dev(ids), np_dev(np.ones((T, 1), np.float32)), None, *_dev(W))
    if way == "decode":
        out = rep.decode_ffn(*args)
    else:
        layer = rep.MoEPrefill(T, 1, E, d, f, weights="mxfp4")
        layer.decode = False
        out = layer(*args)
    torch.cuda.synchronize()
    assert (want != 0).any(1).all() and np.isfinite(want).all()
    got = out[:, :f].cpu().numpy().astype(np.float64)
    assert np.array_equal(got, want)
    assert not out[:, f:].any()


@pytest.mark.parametrize("d,f", [(1 << 24, 128), (128, 1 << 24)])
def test_the_widest_rows(d, f):
    """Offsets up to 2^31 in either projection, 20 tokens grouped and one by itself.
    h is rounded to bf16 (2^-8 at most) on the grouped path; fp32 sums of 2^24
    terms in steps of 16 add less than 2^-12."""
    import torch

    import routed_expert_prefill_amd as rep

    gen = torch.Generator("cuda").manual_seed(f)
    table = torch.tensor([v if c < 8 else -v for c in range(16)
                          for v in ([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0][c % 8],)],
                         dtype=torch.float64, device="cuda")
    T, low = 20, 114 if d > f else 124

    def weights(rows, cols, byte):
        codes = torch.randint(0, 256, (1, rows, cols // 2), generator=gen, dtype=torch.uint8,
                              device="cuda")
        scales = torch.randint(byte, byte + 2, (1, rows, cols // 32), generator=gen,
                               dtype=torch.uint8, device="cuda")
        return codes, scales

    def times(a, codes, scales):
        """a [T, cols] @ w.T in 64 bits, 2^24 weights at a time."""
        _, rows, half = codes.shape
        out = torch.zeros(T, rows, dtype=torch.float64, device="cuda")
        step_c = min(half, 1 << 16)
        step_r = min(rows, (1 << 23) // step_c)
        for r in range(0, rows, step_r):
            for c in range(0, half, step_c):
                b = codes[0, r:r + step_r, c:c + step_c].long()
                w = table[torch.stack([b & 15, b >> 4], -1).flatten(1)]
                s = scales[0, r:r + step_r, c // 16:(c + step_c) // 16].double()
                w = w * torch.exp2(s - 127).repeat_interleave(32, 1)
                out[:, r:r + step_r] += a[:, 2 * c:2 * (c + step_c)] @ w.T.contiguous()
        return out

    x = torch.randn(T, d, generator=gen, device="cuda").to(torch.bfloat16)
    (wg, sg), (wu, su), (wd, sd) = weights(f, d, low), weights(f, d, low), weights(d, f, 238 - low)
    g, u = times(x.double(), wg, sg), times(x.double(), wu, su)
    want = times(g / (1 + torch.exp(-g)) * u, wd, sd)
    ids = torch.zeros(T, 1, dtype=torch.int32, device="cuda")
    ones = torch.ones(T, 1, device="cuda")
    layer = rep.MoEPrefill(T, 1, 1, d, f, weights="mxfp4")
    layer.decode = False
    out = layer(x, ids, ones, None, wg, wu, wd, sg, su, sd).double()
    one = rep.decode_ffn(x[7:8], ids[:1], ones[:1], None, wg, wu, wd, sg, su, sd).double()
    norm = torch.linalg.vector_norm
    for got, ref, tol in ((out, want, 2.0 ** -8 + 2.0 ** -12), (one, want[7:8], 2.0 ** -12)):
        assert torch.isfinite(got).all()
        assert norm(got - ref) <= tol * norm(ref), (norm(got - ref) / norm(ref)).item()
