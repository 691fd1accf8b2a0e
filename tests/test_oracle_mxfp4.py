"""The oracle's MXFP4 decoding against the format's definition, written out."""
import numpy as np

from oracle import numerics as nx
from mxfp4_util import as_bf16_bits, mx_weights


def test_every_code_and_scale():
    # all sixteen codes in one group of 32, each twice, under every scale
    codes = np.arange(32, dtype=np.uint8) % 16
    packed = (codes[0::2] | codes[1::2] << 4).astype(np.uint8)
    by_hand = [0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6] * 2
    for s in range(255):
        got = nx.mxfp4_decode(packed, np.array([s], np.uint8))
        want = np.array(by_hand) * 2.0 ** (s - 127)
        assert np.array_equal(got, want) and np.array_equal(np.signbit(got), np.signbit(want))
    assert np.isnan(nx.mxfp4_decode(packed, np.array([255], np.uint8))).all()


def test_layout_low_half_first_and_groups_of_32():
    packed = np.zeros((2, 32), np.uint8)  # two rows of 64 columns
    packed[0, 0] = 0x52  # columns 0, 1 = codes 2, 5
    packed[1, 16] = 0x0B  # column 32 of row 1 = code 11
    scales = np.array([[127, 128], [126, 130]], np.uint8)
    v = nx.mxfp4_decode(packed, scales)
    want = np.zeros((2, 64))
    want[0, 0], want[0, 1], want[1, 32] = 1.0, 3.0, -1.5 * 8
    assert np.array_equal(v, want)


def test_values_are_bf16_numbers():
    W = mx_weights(2, 64, 32, seed=0, lo=1, hi=250)
    bits = as_bf16_bits(W["wg"], W["sg"])
    assert np.array_equal(nx.bf16_bits_to_f64(bits), nx.mxfp4_decode(W["wg"], W["sg"]))
