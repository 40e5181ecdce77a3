"""The oracle of the 8-bit cache, rotary positions and token scores on values worked out by hand, and against torch's own e4m3."""
import numpy as np
import pytest
import torch

import oracle


def test_e4m3_by_hand():
    # the largest, halfway between 1 and 1.125 (to even), 1.1875 between 1.125 and 1.25, the least normal, a half of the least subnormal
    x = [448.0, 460.0, 1e9, -1e9, 1.0625, 1.1875, 2.0 ** -6, 2.0 ** -10, 1.5 * 2.0 ** -9, -0.0]
    np.testing.assert_array_equal(oracle.e4m3(x), [448, 448, 448, -448, 1.0, 1.25, 2.0 ** -6, 0.0, 2.0 ** -8, 0.0])
    assert np.isnan(oracle.e4m3([np.inf, -np.inf, np.nan])).all()


def test_e4m3_as_torch_rounds():
    v = torch.arange(0x8000, dtype=torch.int32).to(torch.int16).view(torch.bfloat16)
    v = v[torch.isfinite(v.float()) & (v.float() <= 448)].float()
    v = torch.cat([v, v * 1.003, torch.linspace(0, 448, 10001)]).clamp(max=448)
    v = torch.cat([v, -v])
    np.testing.assert_array_equal(oracle.e4m3(v.double().numpy()), v.to(torch.float8_e4m3fn).double().numpy())


@pytest.mark.parametrize("most,scale", [(0.0, 2.0 ** -100), (448.0, 1.0), (448.5, 2.0), (224.0, 0.5), (1.0, 2.0 ** -8), (1.75, 2.0 ** -8),
                                        (1.76, 2.0 ** -7), (1e-40, 2.0 ** -100), (3.38953e38, 2.0 ** 120)])
def test_least_scale_by_hand(most, scale):
    assert oracle.least_scale([0.0, -most, most / 3, np.inf, np.nan]) == scale


def test_commit_grows_a_block():
    """One head, blocks of 8, two rows held: a row 16 times as large doubles the scale four times; a value of 2^-6 of the new scale's
    unit is kept, one that falls between its steps is rounded to even."""
    pages, scales = np.zeros((2, 1, 16, 1)), np.ones((2, 1, 2))
    pages[1, 0, 8:10, 0] = [448.0, 2.0 ** -5 + 2.0 ** -8]  # (28 * 16, and 2^-9 * (16 + 2) before the step down)
    n = oracle.kv_commit_fp8(pages, scales, np.array([[[1.0]], [[7168.0]]]), [1, 0], [1], 10)
    assert n == 12 and scales[1, 0, 1] == 16.0 and scales[1, 0, 0] == 1.0
    np.testing.assert_array_equal(pages[1, 0, 8:12, 0], [28.0, 2.0 ** -9, 448.0, 2.0 ** -4])


def test_rope_by_hand():
    x = np.arange(1.0, 7.0).reshape(1, 1, 6)
    quarter = np.array([np.pi / 2, 0.0])
    y, _ = oracle.rope(x, np.array([1]), quarter)
    np.testing.assert_allclose(y[0, 0], [-3, 2, 1, 4, 5, 6], atol=1e-12)
    y, _ = oracle.rope(x, np.array([1]), quarter, interleaved=True, amplitude=2.0)
    np.testing.assert_allclose(y[0, 0], [-4, 2, 6, 8, 5, 6], atol=1e-12)


def test_rope_frequencies_by_hand():
    np.testing.assert_allclose(oracle.rope_frequencies(4, 100.0), [1.0, 0.1])
    np.testing.assert_allclose(oracle.rope_frequencies(4, 100.0, "linear", 4.0), [0.25, 0.025])
    f = oracle.rope_frequencies(8, 100.0, "base", 4.0)
    np.testing.assert_allclose(f[[0, 3]], [1.0, 100.0 ** -0.75 / 4.0])  # the fastest kept, the slowest divided
    f = oracle.rope_frequencies(4, 100.0, "by_parts", 4.0, 100 * 2 * np.pi, 10.0, 190.0)  # 100 and 10 turns
    np.testing.assert_allclose(f, [0.5 + 0.5 / 4, 0.025])


def test_token_scores_by_hand():
    x = np.log([[1.0, 2.0, 1.0, 4.0]])
    lp, h, top, tlp = oracle.token_scores(x, np.array([[3, 0, -1, 7]]), 4)
    np.testing.assert_allclose(lp[0, :3], [-np.log(2), -np.log(8), 0.0])
    assert np.isnan(lp[0, 3])
    np.testing.assert_allclose(h, [1.75 * np.log(2)])
    assert top.tolist() == [[3, 1, 0, 2]]
    np.testing.assert_allclose(tlp[0], np.log([0.5, 0.25, 0.125, 0.125]))
    assert oracle.token_scores(np.array([[np.nan, 1.0, -np.inf, 2.0]]), np.zeros((1, 0), int), 4)[2].tolist() == [[3, 1, 2, 0]]
