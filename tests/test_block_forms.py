"""The choice of a form for products in 8-bit blocks, on the CPU."""
import random

import pytest

from block_forms import NAMES, form


@pytest.mark.parametrize("n,m,k,groups", [
    (109, 4096, 256, 1), (218, 4096, 128, 1), (437, 4096, 64, 1), (1750, 4096, 16, 1),
    (3500, 4096, 8, 1), (28000, 4096, 1, 1), (64, 12288, 16, 1),
    (96, 4096, 16, 1), (512, 256, 256, 64), (1750, 256, 256, 64), (512, 512, 128, 32), (32, 1408, 2048, 16)])
def test_many_passes_over_few_workgroups_are_not_taken(n, m, k, groups):
    """Narrow matrices, and experts whose rows may all be one's: 16-bit rows are written as blocks
    by a launch of their own."""
    assert form(n, m, k, groups, x16=True) != "own rows"


@pytest.mark.parametrize("n,m,k,groups", [
    (1, 12288, 4096, 1), (2, 12288, 4096, 1), (4, 4096, 4096, 1), (64, 4096, 64, 1),
    (32, 12288, 64, 1), (16, 256, 256, 64), (64, 256, 256, 64), (8, 1408, 2048, 16)])
def test_few_rows_are_one_launch(n, m, k, groups):
    assert form(n, m, k, groups, x16=True) == "own rows"


def test_rows_written_by_the_workgroups_are_bounded():
    """Whatever the sizes, wherever the rows go: four passes of 16 rows at most, and no more elements
    than some 33,000 a compute unit, in whole blocks."""
    rng = random.Random(3)
    own = 0
    for _ in range(20000):
        n, m, k = (int(2 ** rng.uniform(0, top)) for top in (16, 16, 16))
        groups = int(2 ** rng.uniform(0, 9)) if rng.random() < 0.5 else 1
        if form(n, m, k, groups, x16=True) != "own rows":
            continue
        own += 1
        assert n <= 64 and n * -(-k // 128) * 128 <= 33000
    assert own > 500


def test_every_form_is_taken_and_none_is_missing():
    rng = random.Random(4)
    seen = set()
    for _ in range(20000):
        n, m, k = (int(2 ** rng.uniform(0, top)) for top in (13, 14, 14))
        groups = rng.choice([1, 1, 4, 64])
        seen.add(form(n, m, k, groups, transposed=rng.random() < 0.3, x16=rng.random() < 0.5))
    assert seen == set(NAMES) - {"none"}
    # 2^24 rows of 2^20 columns are 2^28 tiles of 256 x 256
    assert form(1 << 24, 1 << 20, 128) == "none"
    assert form(1 << 24, 1 << 20, 128, transposed=True) == "none"
