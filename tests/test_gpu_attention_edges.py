"""Arguments of the attention calls at the edge of what their header allows; tolerances as in test_gpu_attention.py."""
import numpy as np
import pytest
import torch

from tests.test_gpu_attention import _lib, case, check, run  # noqa: F401 (the fixture builds the library)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("S,n,g,Hkv,top", [(40, 1, 4, 2, 3000), (150, 1, 1, 2, 700), (9, 16, 8, 3, 2500)])
def test_tree_attention_runs_of_head_size_64(S, n, g, Hkv, top):
    """Caches cut into runs, whose lengths every block works out in space that its first tiles then take; call after call
    the same."""
    rng = np.random.default_rng([S, top])
    lens = [0, top, 1, 64, 63] + [int(v) for v in np.exp(rng.uniform(0, np.log(top), S - 5))]
    c = case(12, S, n, g, Hkv, 64, lens, 16)
    o, status = run(c)
    assert status == 0
    for s in range(S):
        check(c, o, s)
    for _ in range(5):
        np.testing.assert_array_equal(run(c)[0], o)
