"""What the cache's calls promise about lengths, sizes, windows, buffers and streams."""
import pytest
import torch

from test_gpu_kv import FP32, Case, ec, i32  # noqa: F401 (ec is a fixture)
from test_gpu_kv_rows import check, normal

pytestmark = pytest.mark.gpu
INT_MAX = 2 ** 31 - 1


@pytest.mark.parametrize("window,sinks", [(20, INT_MAX), (20, INT_MAX - 14), (20, 350), (INT_MAX, 0), (INT_MAX, INT_MAX), (349, INT_MAX)])
@pytest.mark.parametrize("qh", [4, 80])
def test_sinks_and_windows_past_every_token(ec, window, sinks, qh):
    """Sinks and windows of any size, also where rows lie before the first token."""
    lens, new = [350, 3, 40], [6, 5, 1]
    c = Case(ec, lens, 1, 128, 16)
    k, v = normal(30, sum(lens), 1, 128), normal(31, sum(lens), 1, 128)
    c.fill(k, v)
    check(ec, c, k, v, new, normal(32, sum(new), qh, 128), FP32, window=window, sinks=sinks)
