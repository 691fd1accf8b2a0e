"""Every kernel that the rule of the 8-bit products can choose is reached by a size of
the GPU tests (dense_tiles.py), in one stage and in more than 64 of them."""
import random

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


def test_few_rows_stay_within_a_line_of_workgroups(rule):
    rng = random.Random(1)
    asked = [(rng.choice(["bf16", "swiglu"]), rng.randint(1, 16), 128 * rng.randint(1, 1 << 14), 128 * rng.randint(1, 64))
             for _ in range(4000)]
    asked += [("bf16", M, N, 128) for M in (1, 16) for N in ((1 << 18) - 5, (1 << 20) + 1, 1 << 26, (1 << 31) - 257)]
    got = rule.ask(asked)
    few = [a for a, g in zip(asked, got) if g[0] or g[1]]
    assert few and max(a[2] for a in few) < 1 << 18
    assert not any(g[0] or g[1] for g in rule.ask([("bf16", 17, 128, 128), ("swiglu", 17, 128, 4096)]))


def test_more_workgroups_than_a_line(rule):
    """What test_gpu_dense_large.py runs for the second line of workgroups of the product."""
    M = (1 << 27) + 70
    (few, few_bf16, _, tile, workgroups), = rule.ask([("bf16", M, 1, 128)])
    assert not few and not few_bf16 and tile == "32x32" and workgroups > 1 << 22
