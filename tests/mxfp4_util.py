"""Random MXFP4 expert weights for the tests, and the same weights as bf16
bits (exact: every MXFP4 value is a bf16 number) for the oracle."""
import numpy as np

from oracle import numerics as nx


def mx_weights(E, d, f, seed, lo=118, hi=122):
    """Codes drawn uniformly (zeros, both signs) and scales from lo..hi."""
    rng = np.random.default_rng(seed)
    W = {}
    for n, rows, cols in (("g", f, d), ("u", f, d), ("d", d, f)):
        W["w" + n] = rng.integers(0, 256, (E, rows, cols // 2), dtype=np.uint8)
        W["s" + n] = rng.integers(lo, hi + 1, (E, rows, cols // 32), dtype=np.uint8)
    return W


def as_bf16_bits(codes, scales):
    v = nx.mxfp4_decode(codes, scales).astype(np.float32)
    bits = v.view(np.uint32)
    assert not (bits & 0xFFFF).any()
    return (bits >> 16).astype(np.uint16)


def bf16_source(W):
    """The oracle's expert source over the same weights."""
    return lambda e: {n: as_bf16_bits(W[n][e], W["s" + n[1]][e]) for n in ("wg", "wu", "wd")}


def unrounded_ref(x, ids, w, mask, W):
    """The layer in 64 bits, h not rounded; x fp64 [T, d]."""
    out = np.zeros_like(x)
    E = W["wg"].shape[0]
    on = (ids >= 0) & (ids < E) & (True if mask is None else mask != 0)
    for e in np.unique(ids[on]):
        t, j = np.nonzero(on & (ids == e))
        g, u, d = (nx.mxfp4_decode(W["w" + n][e], W["s" + n][e]) for n in "gud")
        y = (nx.silu(x[t] @ g.T) * (x[t] @ u.T)) @ d.T
        np.add.at(out, t, w[t, j].astype(np.float64)[:, None] * y)
    return out
