"""Layer norm at the ends of its range: rows that are not finite."""
import numpy as np
import pytest

from tests import _block_ref as ref
from tests.test_fp4_gpu import as_np, on_gpu
from tests.test_norm_gpu import EPS, qg, rows, torch, _no_device_timeouts  # noqa: F401 (fixtures)

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------- codes behind the row

def scale_rows(s, rows_, fmt):
    """Scale bytes of the packed layout as (row, block), with the blocks behind the last one."""
    s = as_np(s)
    tr, tc, _ = s.shape
    return s.reshape(tr, tc, 32, 4, 4).transpose(0, 3, 2, 1, 4).reshape(tr * 128, tc * 4)[:rows_]


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("fmt", ["nv", "mx"])
@pytest.mark.parametrize("M,D", [(3, 100), (200, 100), (200, 33), (300, 515), (200, 1064), (200, 4100), (160, 8200)])
def test_codes_behind_rows_that_are_not_finite(torch, qg, M, D, fmt, dtype):
    """A NaN or an infinity makes all of its row NaN, but what lies behind the row stays 0."""
    X = on_gpu(torch, rows(M, D, 5 + D), dtype)
    X[1, D // 2] = float("nan")
    X[M - 1, 0] = float("inf")
    q, s, _, _ = qg.layer_norm_fp4(X, None, None, EPS, fmt)
    blocks = -(-D // ref.BLOCK[fmt])
    byte = scale_rows(s, M, fmt)
    assert not byte[:, blocks:].any()
    nan_scale = 0x7F if fmt == "nv" else 0xFF
    assert ((byte[:, :blocks] == nan_scale).all(axis=1) == np.isin(np.arange(M), (1, M - 1))).all()
    codes = as_np(q)
    codes = np.stack((codes & 15, codes >> 4), axis=2).reshape(M, -1)
    assert not codes[:, D:].any()
