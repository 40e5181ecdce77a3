"""Values of x that are not finite, in the prompt scan: what they reach, and that nothing else changes.

A value of x in column p of a head makes that column of y, from its token on, and that row of the state something that is
not finite.  Every other output is the same products and sums of the same values as without it: equal to the last bit."""
import numpy as np
import pytest
import torch

from tests.test_gpu_prompt import P, _lib, run_scan, scan_case  # noqa: F401 (the fixture builds the library)

pytestmark = pytest.mark.gpu
VALUES = [float("inf"), -float("inf"), float("nan")]


def put(c, where, rng):
    """Such values at (token row, head, column): (x as it was, first token of each (sequence, head, column) reached)."""
    was, reach = c["x"].clone(), {}
    for row, head, p in where:
        c["x"][row, head * P + p] = VALUES[int(rng.integers(3))]
        s = int(np.searchsorted(c["cu"], row, side="right")) - 1
        reach[s, head, p] = min(row, reach.get((s, head, p), row))
    return was, reach


def check_reach(c, reach, y0, h0, y, h):
    want_y, want_h = np.zeros(y.shape, bool), np.zeros(h.shape[:1] + h.shape[2:4], bool)
    for (s, head, p), row in reach.items():
        want_y[row:c["cu"][s + 1], head, p] = True
        want_h[c["slots"][s], head, p] = True
    np.testing.assert_array_equal(~np.isfinite(y), want_y)
    np.testing.assert_array_equal(y[~want_y], y0[~want_y])
    np.testing.assert_array_equal(~np.isfinite(h[:, 0]), np.broadcast_to(want_h[..., None], h[:, 0].shape))
    np.testing.assert_array_equal(h[:, 0][~want_h], h0[:, 0][~want_h])


@pytest.mark.parametrize("H,G,lens", [(4, 1, [1200, 130]), (3, 3, [100, 30]), (3, 3, [1200, 130]), (4, 2, [70])], ids=str)
@pytest.mark.parametrize("at", [0, 17, 64])
def test_one_value_reaches_one_column(H, G, lens, at):
    c = scan_case(41, H, G, lens)
    y0, h0, _ = run_scan(c)
    _, reach = put(c, [(at, 1, 5)], np.random.default_rng(at))
    y, h, status = run_scan(c)
    assert status == 0
    check_reach(c, reach, y0, h0, y, h)


@pytest.mark.parametrize("lens", [[330, 201, 129, 251] * 4, [240] * 9], ids=str)
def test_values_in_one_chunk_of_many_walks(lens):
    """Every sequence and pair of heads has a value in its chunk 3 (the last one and a short one among them), each at
    another token and column.  More walks than SMs: one follows the other in the same shared memory; call after call."""
    H = 80
    c = scan_case(42, H, 1, lens)
    y0, h0, _ = run_scan(c)
    rng = np.random.default_rng(43)
    for _ in range(3):
        where = []
        for s, n in enumerate(lens):
            chunk = min(3, (n - 1) // 64)
            for pair in range(H // 2):
                if rng.random() < 0.8:
                    row = int(rng.integers(chunk * 64, min(n, chunk * 64 + 64)))
                    where.append((int(c["cu"][s]) + row, 2 * pair + int(rng.integers(2)), int(rng.integers(P))))
        was, reach = put(c, where, rng)
        y, h, status = run_scan(c)
        assert status == 0
        check_reach(c, reach, y0, h0, y, h)
        c["x"].copy_(was)


@pytest.mark.parametrize("H,G,lens", [(80, 1, [700, 640, 333]), (24, 1, [2000, 130]), (3, 3, [330, 65])], ids=str)
def test_values_in_many_chunks(H, G, lens):
    """Several in each chunk, or in every second one, at random tokens and columns: what one chunk's outputs still need is
    not what a later chunk marks."""
    c = scan_case(44, H, G, lens)
    y0, h0, _ = run_scan(c)
    rng = np.random.default_rng(45)
    for step, each in ((1, 2), (2, 3), (2, 1)):
        where = [(int(c["cu"][s]) + int(rng.integers(k * 64, min(n, k * 64 + 64))), int(rng.integers(H)), int(rng.integers(P)))
                 for s, n in enumerate(lens) for k in range(0, -(-n // 64), step) for _ in range(each * H // 2)]
        was, reach = put(c, where, rng)
        y, h, status = run_scan(c)
        assert status == 0
        check_reach(c, reach, y0, h0, y, h)
        c["x"].copy_(was)


@pytest.mark.parametrize("H,G,lens", [(24, 1, [2000, 130, 700]), (3, 3, [330, 65]), (3, 3, [2000])], ids=str)
@pytest.mark.parametrize("odd", [False, True])
def test_y_in_the_place_of_x(H, G, lens, odd):
    """y written over x: as into a tensor of its own, also where x has values that are not finite."""
    from speculative_decoding_mamba2_gb300 import Dims, ssm_prompt_scan, ssm_prompt_scan_workspace_size
    c = scan_case(46, H, G, lens)
    rng = np.random.default_rng(47)
    if odd:
        put(c, [(int(rng.integers(c["T"])), int(rng.integers(H)), int(rng.integers(P))) for _ in range(200)], rng)
    y0, h0, _ = run_scan(c)
    d, h = Dims(n_heads=H), torch.from_numpy(c["h0"]).cuda()
    ws = torch.empty(ssm_prompt_scan_workspace_size(d, c["S"], c["T"], max(lens), G), dtype=torch.uint8, device="cuda")
    ssm_prompt_scan(d, c["prm"], 0, torch.from_numpy(c["cu"]).cuda(), max(lens), c["x"], c["B"], c["C"], c["dt"], h, h, c["x"], ws,
                    slots=torch.from_numpy(c["slots"]).cuda())
    np.testing.assert_array_equal(c["x"].double().cpu().numpy().reshape(c["T"], H, P), y0)
    np.testing.assert_array_equal(h.double().cpu().numpy()[c["slots"]], h0[c["slots"]])
