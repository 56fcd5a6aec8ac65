"""What the Python layer of the post-training losses does with its arguments (no GPU)."""

import pytest
import torch

from cross_entropy_gb300.losses import _per_row


@pytest.mark.parametrize("x", [[1.0, 2.0, 3.0], (1.0, 2.0, 3.0), torch.ones(3), torch.ones(2, 3)])
def test_values_that_fit_no_row_are_refused_by_name(x):
    with pytest.raises(ValueError, match="advantages must have one value per row"):
        _per_row(x, (4, 2), "advantages", torch.device("cpu"))


def test_values_per_row_broadcast():
    cpu = torch.device("cpu")
    assert _per_row([1.0, 2.0], (2,), "advantages", cpu).tolist() == [1.0, 2.0]
    assert _per_row(3.0, (2, 2), "advantages", cpu).tolist() == [3.0] * 4
    assert _per_row([[1.0], [2.0]], (2, 2), "advantages", cpu).tolist() == [1.0, 1.0, 2.0, 2.0]
    assert _per_row([1.0, 2.0, 3.0, 4.0], (2, 2), "advantages", cpu).tolist() == [1.0, 2.0, 3.0, 4.0]
