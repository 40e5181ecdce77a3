"""Rotary positions on the GPU against the fp64 oracle.

Tolerance, before any run (u = 2^-8): the output's rounding u|ref|; beside it, relative to amplitude (|a| + |b|): the angle as an fp32
number of half turns (2^-24 of pi: 2^-22), sine and cosine to 2^-22, two products and a sum (2^-22); the table's and the
oracle's angles in 64 bits, each off by at most 3 * 2^-53 of an angle of up to 2^31 (2^-20).  Together below 2^-18."""
import numpy as np
import pytest
import torch

import oracle
from tests.test_gpu_attention import _lib, bf, host, ints, tree  # noqa: F401 (the fixture builds the library)

pytestmark = pytest.mark.gpu
U, MORE = 2.0 ** -8, 2.0 ** -18


def rows(rng, T, heads, D, pad=8):
    """(a view of T rows with other columns beside them, its values)"""
    t, v = bf(rng.standard_normal((T, heads * D + pad)))
    return t[:, :heads * D], v[:, :heads * D].reshape(T, heads, D)


def near(got, x, pos, freq, inter, amp, D):
    ref, mag = oracle.rope(x, pos, freq, inter, amp)
    got = host(got).reshape(x.shape)
    assert (np.abs(got - ref) <= U * np.abs(ref) + MORE * mag).all()
    np.testing.assert_array_equal(got[:, :, 2 * len(freq):], x[:, :, 2 * len(freq):])


SHAPES = [  # T, Hq, Hkv, D, rot
    (1, 1, 1, 64, 64), (1, 32, 8, 128, 128), (7, 5, 1, 128, 32), (3, 4, 0, 64, 2), (5, 0, 3, 64, 62), (333, 8, 2, 128, 64),
    (2, 3, 3, 72, 24), (17, 2, 1, 8, 8), (9, 1, 2, 512, 512), (40, 8, 8, 128, 20), (1, 1, 1, 64, 16), (6000, 12, 4, 128, 128),
    (70001, 2, 1, 64, 48)]


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_rope(shape, inter):
    import speculative_decoding_mamba2_gb300 as L
    T, Hq, Hkv, D, rot = shape
    rng = np.random.default_rng([1, *shape])
    freq = L.ssm_rope_frequencies(rot)
    pos = rng.integers(0, 1 << 17, T)
    pos[0], pos[-1] = 0, 131071
    amp = 1.0 if T % 2 else 1.25
    turns, p = L.ssm_rope_turns(freq).cuda(), ints(pos)
    given = [rows(rng, T, h, D) if h else (None, None) for h in (Hq, Hkv)]
    out = [None if x is None else torch.full((T, x.shape[1] + 16), 7.0, dtype=torch.bfloat16, device="cuda") for x, _ in given]
    view = [None if o is None else o[:, 8:-8] for o in out]
    L.ssm_rope(D, p, turns, given[0][0], view[0], given[1][0], view[1], interleaved=inter, amplitude=amp)
    some = np.unique(np.concatenate([[0, T - 1], rng.integers(0, T, 300)]))
    for (x, v), o, w in zip(given, out, view):
        if x is not None:
            near(w[torch.from_numpy(some).cuda()], v[some], pos[some], freq, inter, amp, D)
            assert (host(o[:, :8]) == 7).all() and (host(o[:, -8:]) == 7).all()
            np.testing.assert_array_equal(host(x).reshape(v.shape), v)
    # in their places: the same bits
    L.ssm_rope(D, p, turns, given[0][0], given[0][0], given[1][0], given[1][0], interleaved=inter, amplitude=amp)
    for (x, _), w in zip(given, view):
        assert x is None or torch.equal(x, w)


@pytest.mark.parametrize("pos", [[0, 1, -1, 5, -77], [2 ** 31 - 1, -2 ** 31, 2 ** 30 + 1, 12345678, 10 ** 9]])
def test_rope_far_and_backward_positions(pos):
    import speculative_decoding_mamba2_gb300 as L
    rng = np.random.default_rng(2)
    freq = L.ssm_rope_frequencies(64, 500000.0)
    x, v = rows(rng, 5, 3, 64)
    out = torch.empty_like(x).contiguous()
    L.ssm_rope(64, ints(pos), L.ssm_rope_turns(freq).cuda(), x, out)
    near(out, v, np.array(pos, float), freq, False, 1.0, 64)


def test_rope_turned_back():
    """At the opposite position the rows come back but for two roundings."""
    import speculative_decoding_mamba2_gb300 as L
    rng = np.random.default_rng(3)
    turns, pos = L.ssm_rope_turns(L.ssm_rope_frequencies(128)).cuda(), rng.integers(0, 10 ** 6, 50)
    x, v = rows(rng, 50, 4, 128)
    out, back = torch.empty_like(x).contiguous(), torch.empty_like(x).contiguous()
    L.ssm_rope(128, ints(pos), turns, x, out)
    L.ssm_rope(128, ints(-pos), turns, out, back)
    a, b = np.abs(v[:, :, :64]), np.abs(v[:, :, 64:])
    mag = np.concatenate([a + b, a + b], 2)
    assert (np.abs(host(back).reshape(v.shape) - v) <= U * np.abs(v) + (2 * U + MORE) * mag).all()


def test_rope_values_that_are_not_finite():
    """They reach their pair's two columns and no others."""
    import speculative_decoding_mamba2_gb300 as L
    rng = np.random.default_rng(4)
    turns = L.ssm_rope_turns(L.ssm_rope_frequencies(64)).cuda()
    x, _ = rows(rng, 4, 2, 128)
    want = torch.empty_like(x).contiguous()
    L.ssm_rope(128, ints([3, 5, 7, 9]), turns, x, want)
    x[1, 5], x[2, 128 + 100] = float("inf"), float("nan")
    out = torch.empty_like(want)
    L.ssm_rope(128, ints([3, 5, 7, 9]), turns, x, out)
    same = torch.ones_like(out, dtype=torch.bool)
    same[1, 5] = same[1, 37] = same[2, 228] = False
    assert torch.equal(out[same], want[same]) and not torch.isfinite(out[~same]).any()


@pytest.mark.parametrize("S,n,inter", [(1, 1, False), (3, 16, True), (5, 64, False)])
def test_tree_rope(S, n, inter):
    import speculative_decoding_mamba2_gb300 as L
    rng = np.random.default_rng([5, S, n])
    par = np.stack([tree(40 + s, n) for s in range(S)])
    lay = L.ssm_tree_layout_build(par)[0]
    lens = rng.integers(0, 70000, S)
    lens[0] = 0
    pos = (lens[:, None] + lay[:, :, 1]).reshape(-1)
    freq = L.ssm_rope_frequencies(96, scaling="linear", factor=4.0)
    (q, qv), (k, kv) = rows(rng, S * n, 4, 128), rows(rng, S * n, 2, 128)
    qo, ko = torch.empty_like(q), torch.empty_like(k)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    L.ssm_tree_rope(S, n, 128, torch.from_numpy(lay).cuda(), ints(lens), L.ssm_rope_turns(freq).cuda(), q, qo, k, ko, interleaved=inter,
                    status=status)
    assert int(status) == 0
    near(qo, qv, pos, freq, inter, 1.0, 128)
    near(ko, kv, pos, freq, inter, 1.0, 128)


def test_tree_rope_bad_device_data():
    import speculative_decoding_mamba2_gb300 as L
    rng = np.random.default_rng(6)
    lay = L.ssm_tree_layout_build(np.stack([tree(1, 9)] * 2))[0]
    pos = np.concatenate([lay[0, :, 1], 50 + lay[1, :, 1]])
    lay[1, 4, 1], lay[1, 5, 1] = 9, -1
    pos[[13, 14]] = 50
    freq = L.ssm_rope_frequencies(64)
    q, qv = rows(rng, 18, 1, 64)
    out, status = torch.empty_like(q), torch.zeros(1, dtype=torch.int32, device="cuda")
    L.ssm_tree_rope(2, 9, 64, torch.from_numpy(lay).cuda(), ints([-3, 50]), L.ssm_rope_turns(freq).cuda(), q, out, status=status)
    assert int(status) == L.SSM_STATUS_BAD_LAYOUT | L.SSM_STATUS_SEQ_RANGE
    near(out, qv, pos, freq, False, 1.0, 64)


def test_rope_of_as_many_rows_as_an_int32_counts():
    """2^31 - 1 rows of one head of 8: the first and the last ones turned, and those between as they were where the position is 0."""
    import speculative_decoding_mamba2_gb300 as L
    T = 2 ** 31 - 1
    freq = L.ssm_rope_frequencies(8)
    x = torch.zeros(T, 8, dtype=torch.bfloat16, device="cuda")
    pos = torch.zeros(T, dtype=torch.int32, device="cuda")
    some = torch.tensor([0, 1, 2 ** 30, 2 ** 30 + 1, T - 258, T - 2, T - 1], device="cuda")
    put, v = bf(np.random.default_rng(4).standard_normal((7, 8)))
    x[some] = put
    at = [3, 0, 70, 0, 12, 5, 9]
    pos[some] = ints(at)
    L.ssm_rope(8, pos, L.ssm_rope_turns(freq).cuda(), x, x)
    near(x[some], v.reshape(7, 1, 8), np.array(at, float), freq, False, 1.0, 8)
    np.testing.assert_array_equal(host(x[some[[1, 3]]]), v[[1, 3]])
