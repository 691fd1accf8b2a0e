"""Every kernel that the rule of the 8-bit products can choose is reached by a size of
the GPU tests (dense_tiles.py), in one stage and in more than 64 of them."""
import pytest

from dense_tiles import PRODUCTS, SHARED, SHORT, Rule, columns


@pytest.fixture(scope="module")
def rule(tmp_path_factory):
    return Rule(str(tmp_path_factory.mktemp("rule")))


def test_each_tile_has_sizes(rule):
    reached = set()
    for mode, sizes in (("bf16", PRODUCTS), ("f32", PRODUCTS), ("short", SHORT)):
        for tile, (M, N) in sizes.items():
            for K, got in zip(columns(tile), rule.ask([(mode, M, N, K) for K in columns(tile)])):
                assert got[:2] == (False, False) and got[3] == tile, (mode, M, N, K, got)
                reached.add((mode, tile))
    for name, sizes in SHARED.items():
        for (T, d, f), got in zip(sizes, rule.ask([("swiglu", T, f, d) for T, d, f in sizes])):
            mode = "swiglu codes" if got[2] else "swiglu"
            want = "few" if got[0] else mode + " " + got[3]
            assert want == name and got[0] == got[1], (T, d, f, got)
            if not got[0]:
                reached.add((mode, got[3]))
    assert reached == rule.has


def test_more_workgroups_than_a_line(rule):
    """What test_gpu_dense_large.py runs for the second line of workgroups of the product."""
    M = (1 << 27) + 70
    (few, few_bf16, _, tile, workgroups), = rule.ask([("bf16", M, 1, 128)])
    assert not few and not few_bf16 and tile == "32x32" and workgroups > 1 << 22
