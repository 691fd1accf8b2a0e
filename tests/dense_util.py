"""Inputs and comparisons of the tests of 8-bit products (no arithmetic of the path)."""
import numpy as np

from oracle import dense, numerics as nx

U = 2.0 ** -24


def whole_codes(rng, shape):
    """Codes of whole numbers -3 .. 3."""
    return nx.e4m3_encode(rng.integers(-3, 4, shape).astype(np.float64))


def two_powers(rng, shape):
    return np.exp2(rng.integers(-1, 2, shape)).astype(np.float32)


def exact_problem(seed, M, N, K):
    """Codes and scales whose product is exact in fp32 whatever the order of sums:
    whole numbers up to 9 * K * 4, in quarters (K up to 2^16)."""
    rng = np.random.default_rng(seed)
    return (whole_codes(rng, (M, K)), two_powers(rng, (M, K // 128)), whole_codes(rng, (N, K)),
            two_powers(rng, (-(-N // 128), K // 128)))


def random_problem(seed, M, N, K):
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((M, K)) * np.exp(rng.standard_normal((M, K // 128)).repeat(128, 1))
    w = rng.standard_normal((N, K))
    q, s = dense.quant_blocks(x.astype(np.float32))
    return (q, s, nx.e4m3_encode(w * 100),
            (rng.random((-(-N // 128), K // 128)) + 0.2).astype(np.float32) * np.float32(1e-3))


def product_room(K, total):
    """How far a product may be off, given the sums of its terms' magnitudes: a
    block's 128 products are exact, its 127 sums, the scales' product and the
    K / 128 additions of blocks round once each.  Twice that: the matrix unit's own
    additions may round toward zero, a whole step."""
    return (127 + 1 + K // 128) * 2 * U * total


def bf16_room(K, total, v):
    """The same of bf16 results: the 8-bit matrix instruction keeps of eight
    products what lies within 13 bits of the largest, so that seven may lose up to
    2^-13 of it; then the result's rounding."""
    return product_room(K, total) + 7 * 2.0 ** -13 * total + 2.0 ** -8 * np.abs(v) + 2.0 ** -134


def dev(*arrays):
    import torch

    return [torch.from_numpy(np.ascontiguousarray(a)).cuda() for a in arrays]


def host(t):
    return t.double().cpu().numpy()
