"""Arguments of the prompt calls at the edge of what their header allows; tolerances as in test_gpu_prompt.py."""
import numpy as np
import pytest
import torch

from tests.test_gpu_prompt import N, P, U, _lib, bf, host, ints, params, reference, run_scan, scan_case  # noqa: F401 (the fixture builds the library)

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


@pytest.mark.parametrize("cu,slots,T,max_len,bad", [([0, 9, 9], [0, 1], 9, 0, True), ([0, 0, 0], [0, 5], 0, 7, True), ([0, 4, 4], [0, 1], 0, 7, True),
                                                    ([0, 0, 0], [1, 0], 0, 0, False), ([3, 3, 3], [1, 0], 9, 0, False)], ids=str)
def test_prompt_conv_checks_sequences_without_rows_to_write(cu, slots, T, max_len, bad):
    """No rows, or a bound of 0: sequences that are out of range are still reported; nothing is written."""
    from speculative_decoding_mamba2_gb300 import SSM_STATUS_SEQ_RANGE, Dims, ssm_prompt_conv
    rng = np.random.default_rng(52)
    cd = P + 2 * N
    prm, _ = params(rng, 1, 1)
    x, _ = bf(rng.standard_normal((T, cd)))
    ring, ring64 = bf(rng.standard_normal((2, 4, cd)))
    head, out = ints([3, 8]), torch.full((T, cd), 9.0, dtype=torch.bfloat16, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    ssm_prompt_conv(Dims(n_heads=1, ring_cap=4), prm, 0, ints(cu), max_len, x, ring, head, out, slots=ints(slots), status=status)
    assert int(status) == (SSM_STATUS_SEQ_RANGE if bad else 0)
    assert head.tolist() == [3, 8] and (host(ring) == ring64).all() and (host(out) == 9.0).all()


def test_one_token_of_a_buffer_of_any_width():
    """The row stride of a single row says nothing: a token in a buffer whose rows are not multiples of 8 long, by every call."""
    from speculative_decoding_mamba2_gb300 import (Dims, ssm_prompt_conv, ssm_prompt_scan, ssm_prompt_scan_workspace_size,
                                                   ssm_scan_step)
    c = scan_case(53, 2, 1, [1])
    y0, h0, _ = run_scan(c)
    d, prm = Dims(n_heads=2), c["prm"]
    row = torch.full((1, c["x"].size(1) + 2 * N + 5), 9.0, dtype=torch.bfloat16, device="cuda")
    x, B, C = row[:, :2 * P], row[:, 2 * P:2 * P + N], row[:, 2 * P + N:2 * P + 2 * N]
    for to, k in ((x, "x"), (B, "B"), (C, "C")):
        to.copy_(c[k])
    ws = torch.empty(ssm_prompt_scan_workspace_size(d, 1, 1, 1), dtype=torch.uint8, device="cuda")
    for call in ("scan", "step"):
        h, y = torch.from_numpy(c["h0"]).cuda(), torch.zeros(1, 2 * P + 3, dtype=torch.bfloat16, device="cuda")
        if call == "scan":
            ssm_prompt_scan(d, prm, 0, ints([0, 1]), 1, x, B, C, c["dt"], h, h, y[:, :2 * P], ws, slots=ints(c["slots"]))
            np.testing.assert_array_equal(host(y[:, :2 * P]).reshape(1, 2, P), y0)
        else:
            ssm_scan_step(d, prm, 0, x, B, C, c["dt"], h, h, y[:, :2 * P], slots=ints(c["slots"]))
            assert (np.abs(host(y[:, :2 * P]).reshape(2, P) - y0[0]) <= 4 * U * reference(c, 0, magnitude=True)[0][0]).all()
        assert (host(y[:, 2 * P:]) == 0).all()
    outs = []
    for wide in (row[:, :d.conv_dim], row[:, :d.conv_dim].contiguous()):
        ring, head = torch.zeros(1, 20, d.conv_dim, dtype=torch.bfloat16, device="cuda"), ints([3])
        out = torch.zeros_like(wide)
        ssm_prompt_conv(d, prm, 0, ints([0, 1]), 1, wide, ring, head, out)
        outs.append((host(out), host(ring)))
    for a, b in zip(*outs):
        np.testing.assert_array_equal(a, b)


@pytest.mark.parametrize("H,G,S", [(24, 1, 5), (6, 3, 130)])
def test_scan_step_y_in_the_place_of_x(H, G, S):
    """The single token's y written over x: as into a tensor of its own."""
    from speculative_decoding_mamba2_gb300 import Dims, ssm_scan_step
    c = scan_case(54, H, G, [1] * S)
    outs = []
    for y in (torch.empty(S, H * P, dtype=torch.bfloat16, device="cuda"), c["x"]):
        h = torch.from_numpy(c["h0"]).cuda()
        ssm_scan_step(Dims(n_heads=H), c["prm"], 0, c["x"], c["B"], c["C"], c["dt"], h, h, y, slots=ints(c["slots"]))
        outs.append((host(y), host(h)))
    for a, b in zip(*outs):
        np.testing.assert_array_equal(a, b)
