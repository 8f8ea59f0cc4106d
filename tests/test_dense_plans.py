"""The tables of tilings that the GPU tests run through are the library's, on the CPU."""
import os

import pytest

import dense_plans as dp
from activation_sparse_decode_gemv_b200 import binding as pb


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not os.environ.get("PI_FFN_LIB"):  # another build given: use it as is
        from activation_sparse_decode_gemv_b200 import build
        build.build()
    yield pb.lib()
    pb.pi_debug_dense_plan(-1)


def test_tables_are_the_librarys(lib):
    for product in range(5):
        split = set() if product == dp.WEIGHT else {(1, nt, s) for nt, s in dp.SPLIT}
        want = {(mb, nt, 0) for mb, nt in dp.PAIR[product]} | split
        got = {(mb, nt, s) for mb in range(-1, 4) for nt in range(-16, 321) for s in range(-1, 10)
               if lib.pi_debug_dense_plan(product, mb, nt, s) == pb.PI_OK}
        assert got == want, product


def test_refusals(lib):
    for a in ((-2, 0, 0, 0), (5, 1, 256, 0), (-1, 1, 256, 0), (-1, 0, 0, 1), (0, 0, 0, 0)):
        assert lib.pi_debug_dense_plan(*a) == pb.PI_ERR_INVALID_ARG
    assert lib.pi_debug_dense_plan(-1, 0, 0, 0) == pb.PI_OK
