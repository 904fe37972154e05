"""The 8-bit products at the edges of what their header allows.  Operands and tolerances as in test_gpu_e4m3.py."""
import pytest
import torch

import chunked_gated_delta_bwd_gb300 as gdr
from tests.test_gpu_e4m3 import _built, _check_linear, _operands  # noqa: F401  (the fixture builds the library)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M", [3, 16, 29, 64])
@pytest.mark.parametrize("K,N,blocks", [(4096, 152 * 128, True), (4112, 153 * 128, True), (2048 + 16, 20000, False)])
def test_few_rows_through_many_turns_of_the_scales(M, K, N, blocks):
    """More tiles than multiprocessors, so that one block walks the whole inner dimension and its two halves of the
    scales' buffer are each filled again and again; the same bits every time."""
    ops = _operands(M, K, N, 21, blocks=blocks)
    _check_linear(ops)
    first = gdr.linear_e4m3(*ops)
    assert all(torch.equal(first, gdr.linear_e4m3(*ops)) for _ in range(20))
