"""Loss and gradient in one call at every number of tiles that a row's cluster may have, 9 to 16
(more blocks than are portable) and rows whose last tile is empty among them: a few rows, whose own
blocks weigh the lists, and more, with the lists' kernel beside. Tolerances as in
test_gpu_distill.py."""
from __future__ import annotations

import pytest
import torch

from tests.test_gpu_distill import check, teacher
from tests.test_gpu_sample import make

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


def tiles(V, dtype):
    """Tiles of 2,048 16-byte vectors, the row off the 16-byte grid or not."""
    per = 16 // dtype.itemsize
    return -(-((V + 2 * per - 2) // per) // 2048)


# (the last two of each type fill their tiles and have an empty one behind them)
ROWS = [(60001, BF16, 4), (70000, BF16, 5), (90003, BF16, 6), (110000, BF16, 7), (140000, BF16, 9),
        (151936, BF16, 10), (180001, BF16, 11), (190000, BF16, 12), (200003, BF16, 13),
        (225000, BF16, 14), (240000, BF16, 15), (260001, BF16, 16), (16384, BF16, 2),
        (131072, BF16, 9), (245760, BF16, 16),
        (40000, F32, 5), (57001, F32, 7), (90000, F32, 11), (65536, F32, 9), (122880, F32, 16)]


@pytest.mark.parametrize("V,dtype,n", ROWS)
def test_every_cluster(V, dtype, n):
    assert tiles(V, dtype) == n
    few, many = min(3, 148 // n), 148 // n + 2
    for rows, kind in ((few, "zipf"), (many, "normal")):
        x = make(rows, V, dtype, kind, seed=n)
        ids, val, lse = teacher(x, 40, seed=n)
        ids[0], ids[0, 0], ids[0, 1] = -1, 0, V - 1     # a row whose ends are listed
        g = torch.linspace(0.5, 2.0, rows).cuda()
        check(x, ids, val, lse, 1.0, g)
        if rows == few:
            check(x, ids, val, None, 0.7)


@pytest.mark.parametrize("V,dtype,n", [(151936, BF16, 10), (245760, BF16, 16), (90000, F32, 11)])
def test_rows_apart_in_larger_clusters(V, dtype, n):
    """Rows off the 16-byte grid, their gradients elsewhere on it, and rows in error among them."""
    rows = 148 // n + 3
    x = make(rows, V, dtype, "zipf", pad=3, shift=1)
    ids, val, lse = teacher(x, 17)
    x[1, V - 1] = float("nan")
    x[2, 0] = float("inf")
    ids[3] = -1
    check(x, ids, val, lse, 1.0, grad_pad=5)
