"""Refusals of the 8-bit products at the ends of their ranges, on the host (the pointers are never dereferenced:
every call has to be refused before any launch)."""
import pytest

from chunked_gated_delta_bwd_gb300 import build, e4m3
from tests.test_dla_abi import INVALID, at


@pytest.fixture(scope="module")
def E():
    build.build()
    return e4m3._lib()


@pytest.mark.parametrize("rows", [(1 << 31) - 127, (1 << 31) - 2, (1 << 31) - 1, 1 << 31, 1 << 62])
def test_linear_rows_past_the_last_tile_refused(E, rows):
    assert E.gdr_linear_e4m3(rows, 16, 8, at(0), at(1), 1, at(2), at(3), at(4), at(5), None) == INVALID
    assert b"rows" in E.gdr_last_error()
