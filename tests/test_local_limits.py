"""How long the window kernels' waits may last."""
import ctypes

import pytest

from block_sparse_attention_qp_gb300 import binding as msa
from block_sparse_attention_qp_gb300 import build

BOTH = (msa.OP_WINDOW_FORWARD, msa.OP_WINDOW_BACKWARD)


@pytest.fixture(scope="module")
def lib():
    return msa.load_library(build.build())


@pytest.mark.parametrize("op", BOTH)
@pytest.mark.parametrize("S,W,sinks", [(2 ** 23, 2 ** 23, 0), (2 ** 23, 2 ** 22, 2 ** 22), (2 ** 23, 2 ** 21, 4),
                                       (2 ** 20, 2 ** 20, 0), (65536, 512, 4), (128, 1, 0), (1, 1, 0)])
def test_a_unit_fits_its_wait(lib, op, S, W, sinks):
    """A unit walks its window in 128-key tiles, 2.2 us each at 1,507 MHz; the warps that store its rows wait for the
    walk's end.  Five times that leaves room for lower clocks; short windows give up after little more than 200 ms."""
    tiles = min(S, W + sinks) / 128
    ms = msa.msa_window_wait_limit_ms(msa.WindowShape(1, S, 8, 1, 128, W, sinks, 0.1), op)
    assert ms >= 200 + 5 * 2.2e-3 * tiles
    assert ms <= 201 + 0.05 * (tiles + 4)


def test_limits_refused(lib):
    s = msa.WindowShape(1, 1000, 8, 1, 128, 100, 0, 0.1)
    assert msa.msa_window_wait_limit_ms(s, msa.OP_WINDOW_DECODE) == 200  # waits of single tiles
    assert lib.msa_window_wait_limit_ms(None, msa.OP_WINDOW_FORWARD) == 0
    with pytest.raises(msa.MSAError, match="not a window op"):
        msa.msa_window_wait_limit_ms(s, msa.OP_FORWARD)
    s.window = 0
    with pytest.raises(msa.MSAError, match="window"):
        msa.msa_window_wait_limit_ms(s, msa.OP_WINDOW_FORWARD)
    assert lib.msa_window_wait_limit_ms(ctypes.byref(s), msa.OP_WINDOW_BACKWARD) == 0
