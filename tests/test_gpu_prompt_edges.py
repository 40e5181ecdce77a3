"""Arguments of the prompt calls at the edge of what their header allows; tolerances as in test_gpu_prompt.py."""
import numpy as np
import pytest
import torch

from tests.test_gpu_prompt import U, _lib, reference, run_scan, scan_case  # noqa: F401 (the fixture builds the library)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("H,G", [(4, 1), (3, 3)])
@pytest.mark.parametrize("cu,bad", [([200, 400, 0, 200], {1}), ([330, 500, 130, 330, 0, 130], {1, 3}), ([70, 450, 64, 70, 0, 64], {1, 3})], ids=str)
def test_prompt_scan_sequences_in_any_order(H, G, cu, bad):
    """A sequence that is skipped because its rows run backwards, and behind it one whose rows lie before the others'."""
    from speculative_decoding_mamba2_gb300 import SSM_STATUS_SEQ_RANGE
    S, T = len(cu) - 1, max(cu)
    c = scan_case(51, H, G, [T] + [0] * (S - 1))
    c["cu"] = np.array(cu, np.int32)
    y, h, status = run_scan(c)
    assert status == SSM_STATUS_SEQ_RANGE
    for s in range(S):
        if s in bad:
            assert (h[c["slots"][s]] == 7.0).all()
            continue
        ry, rh = reference(c, s)
        my, mh = reference(c, s, magnitude=True)
        assert (np.abs(y[cu[s]:cu[s + 1]] - ry) <= U * np.abs(ry) + (U + 2.0 ** -12) * my + 1e-30).all(), s
        chunks = -(-(cu[s + 1] - cu[s]) // 64)
        assert (np.abs(h[c["slots"][s], 0] - rh) <= 4e-6 * (1 + chunks) * mh + 1e-30).all(), s
