"""Host-side tests of the binding's arguments by position."""
import torch

import pytest

from tp_reduce_residual_gb300 import build as nbuild
from tp_reduce_residual_gb300 import experts


@pytest.fixture(scope="module", autouse=True)
def _library():
    nbuild.build()


def test_product_takes_its_stream_by_position():
    """(a, w, scale, out, stream), of 4-bit and of 8-bit rows; what came later comes after it."""
    q = torch.zeros(4, 16, dtype=torch.uint8)
    four = experts.FP4(q, torch.zeros(experts.fp4_scales_shape(4, 32, "nvfp4"), dtype=torch.uint8), "nvfp4")
    eight = experts.Int8(torch.zeros(4, 32, dtype=torch.int8), torch.ones(4))
    for rows in (four, eight):
        with pytest.raises(ValueError, match="CUDA tensor"):  # all that is wrong with the call
            experts.expert_product(rows, rows, 1.0, None, 0)
    with pytest.raises(ValueError, match="no workspace"):
        experts.expert_product(four, four, workspace=torch.zeros(16, dtype=torch.uint8))
    with pytest.raises(ValueError, match="no workspace"):
        experts.expert_product(four, four, 1.0, None, None, torch.zeros(16, dtype=torch.uint8))
