"""What sum_out of the norm may share memory with, decided before anything is
enqueued (the pointers are never read)."""
import pytest

import weight_rnn_gb300 as wr
from weight_rnn_gb300 import build as wbuild

BASE, OTHER, W, Y, R = (i << 40 for i in (1, 2, 3, 4, 5))


@pytest.fixture(scope="module")
def lib():
    wbuild.build()
    return wr.load_library()


@pytest.mark.parametrize("x,ldx,residual,ldr,rows,fine", [
    (BASE, 64, OTHER, 64, 4, True), (OTHER, 64, BASE, 64, 4, True), (BASE, 64, BASE, 64, 4, True),
    (OTHER, 128, BASE, 64, 4, True), (BASE, 128, OTHER, 64, 1, True),
    (BASE, 128, OTHER, 64, 4, False), (OTHER, 64, BASE, 128, 4, False),
    # both start where the sum does, one of them with rows that lie elsewhere
    (BASE, 128, BASE, 64, 4, False), (BASE, 64, BASE, 128, 4, False), (BASE, 128, BASE, 64, 1, True),
])
def test_sum_in_place(lib, x, ldx, residual, ldr, rows, fine):
    for quant in (False, True):
        wr.delta_inject_failure(1)  # arguments that pass end here
        try:
            if quant:
                st = lib.delta_add_rmsnorm_quant(x, residual, W, Y, R, BASE, rows, 64, ldx, ldr, 1e-6, 1, 0, None)
            else:
                st = lib.delta_add_rmsnorm_fwd(x, residual, W, Y, BASE, R, rows, 64, ldx, ldr, 1e-6, 1, 0, None)
        finally:
            wr.delta_inject_failure(0)
        assert st == (wr.DELTA_ERR_CUDA if fine else wr.DELTA_ERR_INVALID), wr.delta_last_error()
