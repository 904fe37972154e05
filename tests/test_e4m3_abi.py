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


def test_quant_shared_memory_refused(E):
    R, C = 130, 256  # x: 66560 bytes of bf16; codes: 33280; scales: 1040 of rows, 16 of tiles
    ok = [R, C, at(0), 0, 0, 0, at(1), at(2), None, None, None]
    for i, bad in ((6, at(0)), (6, at(0) + 66544), (6, at(0) - 33264), (7, at(0) + 16), (7, at(1) + 33264), (7, at(1) - 1024)):
        assert E.gdr_quant_e4m3(*ok[:i], bad, *ok[i + 1:]) == INVALID, (i, bad)
        assert b"share" in E.gdr_last_error()
    ok = [R, C, at(0), 1024, 1, 1, at(1), at(2), at(3), at(4), None]  # (rows of a wider float32 tensor; the last ends the extent)
    for i, bad in ((6, at(0) + 4 * (129 * 1024 + 256) - 16), (8, at(1)), (8, at(0)), (9, at(2)), (9, at(3) + 33264), (8, at(2) - 16)):
        assert E.gdr_quant_e4m3(*ok[:i], bad, *ok[i + 1:]) == INVALID, (i, bad)
        assert b"share" in E.gdr_last_error()


def test_linear_shared_memory_refused(E):
    ok = [100, 256, 136, at(0), at(1), 2, at(2), at(3), at(4), at(5), None]  # y: 27200 bytes
    for bad in (at(0), at(0) + 25584, at(0) - 27184, at(1) + 784, at(2) + 34800, at(3), at(3) - 16, at(4) + 528):
        assert E.gdr_linear_e4m3(*ok[:9], bad, None) == INVALID, bad
        assert b"share" in E.gdr_last_error()
