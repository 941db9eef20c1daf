"""The cases of test_gpu_few_shared.py are what they say: the second product's
columns are shared, which shows in the workspace, and there are more of them than
workgroups (no GPU needed)."""
import pytest

import bit_grouped_gemm_amd as moe
from test_gpu_few_shared import CASES

CUS = 256  # the workgroups that share columns


def up256(n):
    return (n + 255) // 256 * 256


def unshared(T, H, I, E, k):
    """Bytes of the routing notes and of h, without the shared columns' sums."""
    rows = 8 if T <= 8 else 16 if T <= 16 else 32
    tiles = min(min(E, T * k) + T * k // rows, T * k)
    return 256 + up256(8 * tiles) + up256(4 * tiles * rows) + 2 * up256(2 * T * k * I)


@pytest.mark.parametrize("T,k,E,H,I,columns", CASES)
def test_columns_are_shared(T, k, E, H, I, columns):
    wide = 16 if T <= 8 else 32
    assert moe.moe_layer_mm_workspace_size(T, H, I, E, k) == unshared(T, H, I, E, k) + CUS * 2 * T * wide * 4
    tiles = -(-H // wide)
    assert tiles // CUS == columns and tiles % CUS


def test_the_cases_have_every_row_tile():
    assert {8 if c[0] <= 8 else 16 if c[0] <= 16 else 32 for c in CASES} == {8, 16, 32}
    assert {c[-1] for c in CASES} == {1, 2, 3}


def test_where_they_are_not():
    """Columns that fill the CUs, and a product too short for another launch."""
    for T, k, E, H, I in ((19, 8, 8, 8192, 2048), (19, 8, 8, 12296, 264), (1, 1, 1, 64, 64)):
        assert moe.moe_layer_mm_workspace_size(T, H, I, E, k) == unshared(T, H, I, E, k)
