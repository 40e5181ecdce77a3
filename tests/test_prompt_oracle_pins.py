"""The fp64 oracle of the prompt and attention calls, pinned on the CPU by independent means: the
tree oracle on a chain, splitting a sequence, closed forms."""
import numpy as np

import oracle
from synth import Shape, Workload, batch
from tests.helpers import f64, params_at


def test_prompt_conv_and_scan_equal_a_chain_tree():
    """A prompt of n tokens is a chain tree: conv, scan and commit agree with the tree oracle."""
    w = Workload(96, "prompt pin", Shape(H=3), 1, 1, trees=(("chain", 11),))
    b = batch(w)
    prm = params_at(b["params"], 0)
    xbc, dt, ring, head = f64(b["xBC"][0, 0]), f64(b["dt"][0, 0]), f64(b["ring"][0, 0]), int(b["ring_head"][0, 0])
    h0 = b["h0"][0, 0].astype(np.float64)
    y_ref = oracle.verify(prm, b["parent"][0], xbc, dt, h0, ring, head)
    h_ref, ring_ref, head_ref = oracle.commit(prm, b["parent"][0], list(range(11)), xbc, dt, h0, ring, head)
    R = ring.shape[0]
    post, last, _ = oracle.prompt_conv(prm["conv_w"], prm["conv_b"], xbc, np.stack([ring[(head - j) % R] for j in (3, 2, 1)]))
    d = 3 * 64
    y, h = oracle.prompt_scan(post[:, :d].reshape(11, 3, 64), post[:, None, d:d + 128], post[:, None, d + 128:], dt,
                              prm["dt_bias"], prm["A_log"], prm["D"], h0)
    np.testing.assert_allclose(y.reshape(y_ref.shape), y_ref, rtol=1e-12, atol=1e-12)
    np.testing.assert_allclose(h, h_ref, rtol=1e-12, atol=1e-12)
    np.testing.assert_array_equal(last, np.stack([ring_ref[(head_ref - j) % R] for j in (3, 2, 1)]))


def test_prompt_scan_splits_anywhere():
    rng = np.random.default_rng(5)
    T, H, G, P, N = 9, 4, 2, 3, 5
    x, B, C, dt = (rng.standard_normal(s) for s in ((T, H, P), (T, G, N), (T, G, N), (T, H)))
    prm = rng.standard_normal(H), rng.standard_normal(H), rng.standard_normal(H)
    h0 = rng.standard_normal((H, P, N))
    y, h = oracle.prompt_scan(x, B, C, dt, *prm, h0)
    for k in (0, 1, 4, 9):
        y1, h1 = oracle.prompt_scan(x[:k], B[:k], C[:k], dt[:k], *prm, h0)
        y2, h2 = oracle.prompt_scan(x[k:], B[k:], C[k:], dt[k:], *prm, h1)
        np.testing.assert_allclose(np.concatenate([y1, y2]), y, rtol=1e-13)
        np.testing.assert_allclose(h2, h, rtol=1e-13)


def test_prompt_scan_closed_form():
    # one head, one value, one state: softplus(dt) = log 2 at dt = 0, A = -1: a = 1/2
    l2 = np.log(2.0)
    one = np.ones((3, 1, 1))
    y, h = oracle.prompt_scan(one, one, one, np.zeros((3, 1)), np.zeros(1), np.zeros(1), np.zeros(1), np.zeros((1, 1, 1)))
    np.testing.assert_allclose(y[:, 0, 0], [l2, 1.5 * l2, 1.75 * l2])
    np.testing.assert_allclose(h[0, 0, 0], 1.75 * l2)


def test_tree_attention_closed_forms():
    rng = np.random.default_rng(6)
    n, Hq, Hkv, D, m = 5, 4, 2, 3, 7
    q, k, v = rng.standard_normal((n, Hq, D)), rng.standard_normal((n, Hkv, D)), rng.standard_normal((n, Hkv, D))
    kc, vc = rng.standard_normal((m, Hkv, D)), rng.standard_normal((m, Hkv, D))
    par = np.array([-1, 0, 0, 1, 2])
    # equal scores: the mean of what a node sees
    o, _ = oracle.tree_attention(q, 0 * k, v, par, 0 * kc, vc, 1.0)
    np.testing.assert_allclose(o[3, 1], np.concatenate([vc[:, 0], v[[0, 1, 3], 0]]).mean(0))
    # a node equals a one-node tree over the cache with its ancestors appended
    o, _ = oracle.tree_attention(q, k, v, par, kc, vc, 0.7)
    o1, _ = oracle.tree_attention(q[4:], k[4:], v[4:], [-1], np.concatenate([kc, k[[0, 2]]]), np.concatenate([vc, v[[0, 2]]]), 0.7)
    np.testing.assert_allclose(o[4], o1[0])
    # other nodes' rows do not matter
    k2, v2 = k.copy(), v.copy()
    k2[[1, 3]], v2[[1, 3]] = np.nan, np.inf
    np.testing.assert_array_equal(oracle.tree_attention(q, k2, v2, par, kc, vc, 0.7)[0][[0, 2, 4]], o[[0, 2, 4]])


def test_kv_commit_crosses_pages():
    pages = np.zeros((4, 1, 2, 1))
    rows = np.arange(1.0, 6.0).reshape(5, 1, 1)
    assert oracle.kv_commit(pages, rows, [0, 2, 4], [3, 0, 1], 1) == 4
    np.testing.assert_array_equal(pages[:, 0, :, 0], [[3, 5], [0, 0], [0, 0], [0, 1]])
