"""The order in which ftd_cache_evict keeps rows, on the inputs where it can go wrong: zeros of both signs."""
import numpy as np
import pytest

import decode_step_masked_gb300 as ftd
from tests.test_evict_gpu import check

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    import torch
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a CUDA device")
    ftd.build_library()
    ftd.load_library()


@pytest.mark.parametrize("L,budget", [(640, 400), (640, 1), (500, 499), (9000, 4000)])
@pytest.mark.parametrize("values", [(0.0, -0.0), (0.0, -0.0, 1.0, -1.0), (0.0, -0.0, 1e-45, -1e-45, np.nan, -np.inf)])
def test_zeros_of_both_signs_are_equal(L, budget, values):
    """Equal weights stay by the lower row, and 0.0 == -0.0."""
    rng = np.random.default_rng(L + budget)
    acc = rng.choice(np.array(values, np.float32), (2, 2, 16 * (-(-L // 16))))
    check("f16", 2, 2, 64, acc.shape[2], [L, L], budget, acc=acc)
