"""CPU tests of the rule that chooses a product's variant and its cut
(csrc/linear_plan.h): every tile is computed whole or in parts, never twice, the
parts' sums fit the workspace that is asked for, and each variant's conditions
hold wherever the rule chooses it."""
import random

import pytest

import linear_plan

PAIRS = [("f32", "f32"), ("bf16", "bf16"), ("bf16", "f32"), ("f8", "bf16"), ("f8", "f32")]
SIZE = {"f32": 4, "bf16": 2, "f8": 1}


def sizes(n, seed):
    g = random.Random(seed)
    for _ in range(n):
        yield tuple(int(2 ** g.uniform(0, top)) for top in (18, 15, 17))


@pytest.mark.parametrize("dtype,out", PAIRS)
def test_plans_are_whole(dtype, out):
    seen = set()
    for M, K, N in list(sizes(4000, 1)) + [(2 ** 31 - 1, 1, 1), (1, 1, 2 ** 31 - 1), (2 ** 28, 16, 128), (2 ** 28 - 1, 16, 128), (175, 3912, 12740)]:
        for cus in (256, 104):
            path, full, rest, splits, ws = linear_plan.plan(M, K, N, dtype, out, cus)
            at = (M, K, N, cus, path)
            seen.add((path, splits > 1))
            if path in ("rows", "columns"):
                assert (full, rest, splits, ws) == (0, 0, 1, 0), at
                if path == "rows":
                    assert -(-M // 64) < 65536 and -(-N // 16) * 512 < 2 ** 32, at
                else:
                    assert N <= 128 and K * SIZE[dtype] % 16 == 0 and -(-M // 64) * 512 < 2 ** 32, at
                continue
            tile = int(path.removeprefix("tile"))
            assert full + rest == -(-M // tile) * -(-N // tile), at
            steps = -(-K * SIZE[dtype] // 128)
            assert (rest == 0 and splits == 1) or (splits > 1 and rest * splits <= cus * (2 if tile == 128 else 1)), at
            assert splits <= steps and ws == (splits * rest * tile * tile * 4 if splits > 1 else 0), at
            if tile == 256:
                assert K * SIZE[dtype] % 16 == 0 and (dtype, out) != ("f8", "f32"), at
    want = {("rows", False), ("columns", False), ("tile128", False), ("tile128", True), ("tile256", False), ("tile256", True)}
    if dtype == "f32":  # the large tile saves float32 no time but by its cut: few sizes take it
        want -= {("tile256", False)}
        seen -= {("tile256", False)}
    if (dtype, out) == ("f8", "f32"):
        want -= {("tile256", False), ("tile256", True)}
    assert seen == want


def test_tile_grids_stay_within_a_launch():
    # up to 512 threads a workgroup, fewer than 2^32 threads in a dimension, 65,535 rows
    largest = linear_plan.plan(2 ** 31 - 1, 1, 1, "bf16", "bf16")[1]
    assert largest * 256 >= 2 ** 32  # one row of workgroups would not do
    for n in (1, 2, 255, 256, 2 ** 22 - 1, 2 ** 22, 2 ** 22 + 1, 3 * 2 ** 22, largest, 2 ** 31):
        x, y = linear_plan.grid(n)
        assert x * 512 < 2 ** 32 and y < 65536 and n <= x * y < n + x
        assert y == 1 or n > 2 ** 22
