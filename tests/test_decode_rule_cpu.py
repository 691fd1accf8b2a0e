"""Which layers MoEPrefill sends to decode_ffn, by the shapes whose times the
rule's comment gives: the measured faster way, or grouped where the ids decide."""
import pytest

from routed_expert_prefill_amd import MoEPrefill

WIDE, NARROW = (4096, 2048), (1024, 512)


@pytest.mark.parametrize("T,k,E,size,decode", [
    (1, 6, 256, WIDE, True), (4, 6, 256, WIDE, True), (10, 6, 256, WIDE, True),
    (8, 8, 256, WIDE, True), (11, 6, 256, WIDE, False),  # 66 routes
    (16, 2, 8, WIDE, True), (8, 4, 4, WIDE, True), (4, 8, 8, WIDE, True), (2, 16, 16, WIDE, True),
    (24, 1, 1, WIDE, True), (32, 1, 1, WIDE, False), (32, 1, 2, WIDE, False),
    (32, 1, 4, WIDE, True), (32, 1, 8, WIDE, True),
    (20, 2, 32, WIDE, True), (20, 2, 16, WIDE, False), (16, 4, 16, WIDE, False),
    (16, 4, 8, WIDE, False), (10, 4, 8, WIDE, False), (32, 2, 32, WIDE, False),
    (64, 1, 256, WIDE, False), (32, 1, 256, WIDE, True),
    (32, 2, 16, NARROW, True), (16, 4, 16, NARROW, True), (32, 1, 1, NARROW, True),
    (64, 1, 16, NARROW, False),
])
def test_rule(T, k, E, size, decode):
    assert MoEPrefill._decodes(T, k, E, *size) is decode
