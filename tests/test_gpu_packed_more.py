"""More of packed attention and rotary positions on the GPU."""
import pytest

import packed_ref as ref
from test_gpu_packed import backward_checked, forward_checked, fp32_default  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D", [64, 128])
def test_the_least_scale(D):
    """All keys weigh the same; LSE, the log of their number, is divided by 2^-120 on the way."""
    q, k, v, do, cu = ref.inputs([300, 1, 77], 4, 2, D, seed=2)
    forward_checked(q, k, v, cu, True, 2.0 ** -120)
    backward_checked(q, k, v, do, cu, True, 2.0 ** -120)
