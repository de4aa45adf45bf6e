"""What the grid of the layer norm tests holds."""
import itertools

import pytest
import torch

import test_gpu_layer_norm_grid as grid


@pytest.mark.parametrize("widths", [grid.NARROW, grid.HELD, grid.LONG], ids=["narrow", "held", "long"])
def test_every_combination_occurs(widths):
    """Type, rows on 16 bytes or not, residual and probability, in every form of the kernels."""
    have = {(dtype, order == "odd", residual, p) for _, cols, dtype, order, residual, p in grid.CASES if cols in widths}
    every = set(itertools.product((torch.bfloat16, torch.float32), (False, True), (False, True), (0.0, 0.1, 0.5)))
    assert have == every


def test_many_rows_with_and_without_dropout():
    """Beside staged weights, of which 504 and 4096 columns are whole columns of a warp or not."""
    many = {(cols, dtype, residual, p) for rows, cols, dtype, order, residual, p in grid.CASES if rows > 16 * 152 and order != "odd"}
    for cols, dtype, (residual, p) in itertools.product((504, 1000, 1024, 3000, 4096), (torch.bfloat16, torch.float32),
                                                        itertools.product((False, True), (0.0, 0.1))):
        assert (cols, dtype, residual, p) in many


def test_cases_are_unlike():
    assert len(set(grid.CASES)) == len(grid.CASES)
