"""8-bit products with block scales, and the shared expert (fp64 numpy).

TEST INFRASTRUCTURE ONLY (see the package docstring).

Rows are E4M3 codes with one fp32 scale for each block of 128 columns, weights
E4M3 codes with one for each block of 128 x 128; a matrix with an odd number of
rows has a last block of fewer.  Values are exact, products and sums in 64 bits.
"""
from __future__ import annotations

import numpy as np

from . import numerics as nx


def quant_blocks(x: np.ndarray):
    """Codes [M, K] and scales [M, K / 128] of fp32 rows: ``quant_rows_fp8`` on blocks."""
    x = np.asarray(x, np.float32)
    q, s = nx.quant_rows_fp8(x.reshape(-1, 128))
    return q.reshape(x.shape), s.reshape(x.shape[0], -1)


def row_values(q: np.ndarray, s: np.ndarray) -> np.ndarray:
    return nx.e4m3_decode(q) * np.repeat(np.asarray(s, np.float64), 128, axis=1)


def weight_values(w: np.ndarray, s: np.ndarray) -> np.ndarray:
    wide = np.repeat(np.repeat(np.asarray(s, np.float64), 128, axis=0)[:w.shape[0]], 128, axis=1)
    return nx.e4m3_decode(w) * wide


def matmul(q, xs, w, ws) -> np.ndarray:
    return row_values(q, xs) @ weight_values(w, ws).T


def matmul_abs(q, xs, w, ws) -> np.ndarray:
    """The sums of the terms' magnitudes: what rounding errors are relative to."""
    return np.abs(row_values(q, xs)) @ np.abs(weight_values(w, ws)).T


def shared_hidden(q, xs, wg, wu, sg, su) -> np.ndarray:
    """silu(g) * u."""
    return nx.silu(matmul(q, xs, wg, sg)) * matmul(q, xs, wu, su)
