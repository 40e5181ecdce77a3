"""Arguments of the attention calls at the edge of what their header allows; tolerances as in test_gpu_attention.py."""
import numpy as np
import pytest
import torch

from tests.test_gpu_attention import _lib, bf, case, check, host, ints, run  # noqa: F401 (the fixture builds the library)

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


@pytest.mark.parametrize("room", [0, 1, 2, 5])
def test_kv_commit_lengths_up_to_an_int32(room):
    """A cache `room` rows below the longest length that an int32 holds, under a page table that goes on behind it."""
    from speculative_decoding_mamba2_gb300 import SSM_STATUS_SEQ_RANGE, ssm_kv_commit
    rng = np.random.default_rng(61)
    n, Hkv, D, page, pool = 4, 2, 64, 1024, 3
    (kp, kp64), (vp, vp64) = (bf(rng.standard_normal((1, pool, Hkv, page, D))) for _ in range(2))
    (k, k64), (v, v64) = (bf(rng.standard_normal((1, n, Hkv * D))) for _ in range(2))
    table = torch.zeros(1, (1 << 21) + 2, dtype=torch.int32, device="cuda")
    table[0, (1 << 21) - 1], table[0, 1 << 21] = 2, 1
    length, want = (1 << 31) - 1 - room, min(room, 4)
    out, status = ints([0]), torch.zeros(1, dtype=torch.int32, device="cuda")
    ssm_kv_commit(1, n, ints([[0, 1, 2, 3]]), ints([4]), k, v, kp, vp, table, ints([length]), out, status=status)
    assert int(status) == (SSM_STATUS_SEQ_RANGE if want < 4 else 0) and int(out[0]) == length + want
    for pages, rows in ((kp64, k64), (vp64, v64)):
        for i in range(want):
            pages[0, 2, :, (length + i) % page] = rows[0, i].reshape(Hkv, D)
    np.testing.assert_array_equal(host(kp), kp64)
    np.testing.assert_array_equal(host(vp), vp64)


@pytest.mark.parametrize("n,g,D", [(8, 4, 128), (40, 2, 64), (6, 2, 128)])
def test_tree_attention_rows_do_not_depend_on_each_other(n, g, D):
    """Children of one root, whose own rows score 4 (in powers of two) above the cache: whether one of them has a far larger k, and
    its rows' maximum grows, changes no bit of the others."""
    c = case(62, 1, n, g, 1, D, [100], 64)
    u = np.random.default_rng([62, D]).choice([-1.0, 1.0], D)
    c["q"], _ = bf(np.tile(u, (n, g)))
    c["k"], _ = bf(np.tile(u * 2.8 / np.sqrt(D), (n, 1)))
    c["par"][0] = [-1] + [0] * (n - 1)
    c["kp"], _ = bf(c["kp64"] * 0.3)
    o0, _ = run(c)
    c["k"][-1] = torch.from_numpy(u * 8.0)
    o, status = run(c)
    assert status == 0 and not np.array_equal(o[0][-1], o0[0][-1])
    np.testing.assert_array_equal(o[0][:-1], o0[0][:-1])
