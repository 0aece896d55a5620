"""A weight without columns is refused by every entry point (CPU: no call reaches the
library)."""
import pytest
import torch

import mxfp4_block_amax_amd as fp4
from tests.test_layers_arguments import library  # noqa: F401  (a fixture)


@pytest.mark.parametrize("rows", [0, 3])
@pytest.mark.parametrize("fmt", [fp4.MXFP4, fp4.NVFP4])
def test_refused(library, fmt, rows):  # noqa: F811
    x = torch.zeros(rows, 0)
    nothing = torch.zeros(5, 0, dtype=torch.uint8)
    out = torch.full((rows, 5), 7.0)
    for how in ({}, {"out": out}, {"out_dtype": torch.bfloat16}):
        with pytest.raises(ValueError):
            fp4.linear_w4(fmt, x, nothing, nothing, torch.ones(1), **how)
    with pytest.raises(ValueError):
        fp4.linear_w4_packed(fmt, x, torch.zeros(64, dtype=torch.uint8), 5, torch.ones(1))
    assert not library.calls


def test_no_rows(library):  # noqa: F811
    y = fp4.linear_w4(fp4.MXFP4, torch.zeros(0, 64), torch.zeros(5, 32, dtype=torch.uint8),
                      torch.zeros(5, 2, dtype=torch.uint8))
    assert y.shape == (0, 5) and not library.calls
