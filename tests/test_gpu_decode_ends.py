"""GPU routed experts for single tokens where numbers end."""
import numpy as np
import pytest

from gpu_util import bf16_dev, np_dev
from test_gpu_decode import _decode, _problem, _ref
from test_gpu_mxfp4 import _dev

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,k,E,same", [(1, 1, 4, False), (9, 1, 4, False), (7, 1, 3, True)])
def test_infinite_weights_of_the_down_projection(T, k, E, same):
    """A product of 2^128 and more is an infinity with the sign of h, as in the
    grouped path, though h comes in two parts, of which the second may be zero
    or have the other sign."""
    import torch

    import routed_expert_prefill_amd as rep

    d, f = 384, 256
    p = _problem(T, k, E, d, f, seed=T + E, same=same)
    ids, w, mask, x, W = p
    w += 0.5
    rng = np.random.default_rng(7)
    rows, codes = rng.permutation(d)[:90], (0x07, 0x0F, 0x70, 0xF0)
    for i, n in enumerate(rows):  # one weight of 6 * 2^127 in a group of zeros
        c = int(rng.integers(0, f // 2))
        W["wd"][:, n, c // 16 * 16:c // 16 * 16 + 16] = 0
        W["wd"][:, n, c] = codes[i % 4]
        W["sd"][:, n, c // 16] = 254
    # 6 * 2^127 h where an infinity is meant; the other terms are below 10^5, so
    # past 10^6 h is above 10^-33, a bf16 number with its sign
    want = _ref(p)
    out = _decode(p).cpu().numpy().astype(np.float64)
    big = np.zeros(d, bool)
    big[rows] = True
    assert (np.abs(want[:, big]) > 1e6).all() and np.isfinite(out[:, ~big]).all()
    assert np.array_equal(out[:, big], np.sign(want[:, big]) * np.inf)
    layer = rep.MoEPrefill(T, k, E, d, f, weights="mxfp4")
    layer.decode = False
    grouped = layer(bf16_dev(x), np_dev(ids), np_dev(w), np_dev(mask), *_dev(W))
    assert np.array_equal(grouped.cpu().numpy()[:, big], out[:, big].astype(np.float32))
    torch.cuda.synchronize()
