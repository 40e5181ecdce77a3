"""Tree attention over an 8-bit cache and the commit into it, on the GPU against the fp64 oracle.

Tolerance, before any run (u = 2^-8), as for the 16-bit cache, over the values that the cache stands for (which the tensor cores take
without a rounding): the output's rounding u|ref|; the weights are rounded to 16 bits for their product with v, each summand off by at
most u: u·mag with mag = sum of weight·|v|; fp32 scores, sums and exponentials: below 2^-11·mag for scores whose products add up to
at most 100 in absolute value (8 accumulations of 2^-23·100, the exponential 2^-22).  A commit's bits are the oracle's."""
import numpy as np
import pytest
import torch

import oracle
from tests.test_gpu_attention import U, _chain, _lib, bf, host, ints, tree  # noqa: F401 (the fixture builds the library)

pytestmark = pytest.mark.gpu
F8 = torch.float8_e4m3fn


def pages(rng, L, pool, Hkv, page, D, block, spread=0.5):
    """(e4m3 pages, scales on the GPU; what the pages hold, the scales, in fp64): blocks of different sizes, as a commit scales them."""
    x = rng.standard_normal((L, pool, Hkv, page // block, block * D)) * np.exp(spread * rng.standard_normal((L, pool, Hkv, page // block, 1)))
    most = np.abs(x).max(-1)
    scale = np.exp2(np.ceil(np.log2(most / 448.0)))
    held = torch.from_numpy((x / scale[..., None]).reshape(L, pool, Hkv, page, D)).to(F8)
    return held.cuda(), torch.from_numpy(scale).float().cuda(), held.double().numpy(), scale


def case(seed, S, n, g, Hkv, D, lens, page, block, qscale=1.0, fused=False, spread=0.5):
    rng = np.random.default_rng([seed, S, n, g, Hkv, D, page, block])
    Hq = g * Hkv
    per = max(1, max(-(-(l + n) // page) for l in lens))
    pool = S * per + 2
    c = dict(S=S, n=n, g=g, Hq=Hq, Hkv=Hkv, D=D, lens=list(lens), page=page, block=block, pool=pool, scale=D ** -0.5)
    c["par"] = np.stack([tree(seed + s, n) for s in range(S)])
    w = (Hq + 2 * Hkv) * D
    row, row64 = bf(rng.standard_normal((S * n, w + 8)) * np.concatenate([np.full(Hq * D, qscale), np.ones(2 * Hkv * D + 8)]))
    cut = [slice(0, Hq * D), slice(Hq * D, (Hq + Hkv) * D), slice((Hq + Hkv) * D, w)]
    (c["q"], c["k"], c["v"]), (q64, k64, v64) = (row[:, s] for s in cut), (row64[:, s] for s in cut)
    if not fused:
        c["q"], c["k"], c["v"] = c["q"].contiguous(), c["k"].contiguous(), c["v"].contiguous()
    c["q64"], c["k64"], c["v64"] = q64.reshape(S, n, Hq, D), k64.reshape(S, n, Hkv, D), v64.reshape(S, n, Hkv, D)
    for x in "kv":
        c[x + "p"], c[x + "s"], held, scale = (t[0] for t in pages(rng, 1, pool, Hkv, page, D, block, spread))
        c[x + "p64"] = held * np.repeat(scale, block, -1)[..., None]
    c["table"] = rng.permutation(pool)[:S * per].astype(np.int32).reshape(S, per)
    return c


def run(c, max_len=None, table=None, lens=None, layout=None, stream=None):
    from speculative_decoding_mamba2_gb300 import (ssm_tree_attention_fp8, ssm_tree_attention_fp8_workspace_size,
                                                   ssm_tree_layout_build)
    S, n, Hq, Hkv, D = (c[k] for k in ("S", "n", "Hq", "Hkv", "D"))
    max_len = max(c["lens"]) if max_len is None else max_len
    lay = ssm_tree_layout_build(c["par"])[0] if layout is None else layout
    ws = torch.full((ssm_tree_attention_fp8_workspace_size(S, n, Hq, Hkv, D, max_len),), 255, dtype=torch.uint8, device="cuda")
    o = torch.full((S * n, Hq * D + 8), 9.0, dtype=torch.bfloat16, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    ssm_tree_attention_fp8(S, n, Hq, Hkv, D, torch.from_numpy(lay).cuda(), c["q"], c["k"], c["v"], c["kp"], c["vp"], c["ks"], c["vs"],
                           ints(c["table"] if table is None else table), ints(c["lens"] if lens is None else lens), max_len, c["scale"],
                           o[:, :Hq * D], ws, status=status, stream=stream)
    torch.cuda.synchronize()
    assert (host(o[:, Hq * D:]) == 9.0).all()
    return host(o[:, :Hq * D]).reshape(S, n, Hq, D), int(status)


def cache(c, s, length):
    at = np.arange(length)
    pg, row = c["table"][s, at // c["page"]], at % c["page"]
    return c["kp64"][pg, :, row], c["vp64"][pg, :, row]


def near(c, o, s, kc, vc, par=None, scores=1.0):
    ref, mag = oracle.tree_attention(c["q64"][s], c["k64"][s], c["v64"][s], c["par"][s] if par is None else par, kc, vc, c["scale"])
    assert (np.abs(o[s] - ref) <= U * np.abs(ref) + (U + scores * 2.0 ** -11) * mag).all(), (s, np.max(np.abs(o[s] - ref) / mag))


def check(c, o, s, length=None, par=None):
    near(c, o, s, *cache(c, s, c["lens"][s] if length is None else length), par=par)


SHAPES = [  # S, n, g, Hkv, D, lens, page, block
    (1, 1, 1, 1, 64, [0], 8, 8), (1, 1, 1, 2, 128, [1], 16, 8), (3, 1, 8, 2, 128, [63, 64, 65], 32, 32), (2, 7, 1, 3, 64, [0, 200], 8, 8),
    (2, 16, 4, 2, 128, [129, 31], 64, 16), (1, 5, 5, 1, 128, [1000], 16, 16), (3, 16, 2, 2, 64, [17, 0, 300], 128, 8),
    (1, 64, 1, 1, 128, [70], 64, 64), (1, 40, 8, 1, 128, [333], 64, 8), (2, 64, 4, 1, 64, [64, 5], 32, 16), (1, 9, 12, 1, 64, [2000], 256, 128),
    (1, 33, 2, 2, 64, [100], 8, 8), (1, 23, 32, 1, 128, [90], 1024, 1024), (2, 3, 2, 1, 128, [1500, 1024], 1024, 256)]


@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_tree_attention_fp8(shape):
    S, n, g, Hkv, D, lens, page, block = shape
    c = case(1, S, n, g, Hkv, D, lens, page, block, fused=n % 2 == 1)
    o, status = run(c)
    assert status == 0
    for s in range(S):
        check(c, o, s)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n,g", [(1, 4), (16, 4), (40, 8)])
def test_tree_attention_fp8_long_cache_is_split(n, g, D):
    c = case(2, 3, n, g, 2, D, [4099, 130, 0], 64, 32)
    o, status = run(c)
    assert status == 0
    for s in range(3):
        check(c, o, s)


def test_tree_attention_fp8_large_scores():
    """Scores far apart (the maximum moves by hundreds between tiles): the weights of all but a few rows are 0."""
    c = case(3, 2, 16, 4, 1, 64, [700, 90], 16, 8, qscale=60.0)
    o, status = run(c)
    assert status == 0
    for s in range(2):  # products of a score add up to 60 times the ones above
        near(c, o, s, *cache(c, s, c["lens"][s]), scores=60)


@pytest.mark.parametrize("lo,hi", [(-20, 20), (-100, -60), (-8, 100)])
def test_tree_attention_fp8_scales_far_apart(lo, hi):
    """Blocks of v whose scales differ by many powers of two: what they add up to is right relative to the largest."""
    c = case(4, 2, 9, 2, 2, 128, [500, 77], 32, 8)
    rng = np.random.default_rng([4, hi + 200])
    by = np.exp2(rng.integers(lo, hi + 1, c["vs"].shape))
    held = c["vp64"] / np.repeat(c["vs"].double().cpu().numpy(), c["block"], -1)[..., None]
    c["vs"] = torch.from_numpy(by).float().cuda()
    c["vp64"] = held * np.repeat(by, c["block"], -1)[..., None]
    o, status = run(c)
    assert status == 0
    for s in range(2):
        check(c, o, s)


@pytest.mark.parametrize("to", [2.0 ** -100, 3e-20, 1.0, 7.0])
def test_tree_attention_fp8_scales_that_are_no_powers_of_two(to):
    """Any scale in the range is taken, for k and for v."""
    c = case(5, 1, 6, 3, 1, 64, [200], 16, 16)
    rng = np.random.default_rng(5)
    for x in "kv":
        held = c[x + "p64"] / np.repeat(c[x + "s"].double().cpu().numpy(), c["block"], -1)[..., None]
        s = torch.from_numpy((rng.uniform(1.0, 2.0, c[x + "s"].shape) * (to if x == "v" else 0.003))).float()
        s = s.clamp(min=2.0 ** -100)
        c[x + "s"], c[x + "p64"] = s.cuda(), held * np.repeat(s.double().numpy(), c["block"], -1)[..., None]
    o, status = run(c)
    assert status == 0
    check(c, o, 0)


def test_tree_attention_fp8_a_flat_tail():
    """One row of the cache that stands out over thousands of equal rows, whose small weights add up to more than its own."""
    c = case(6, 1, 2, 4, 1, 128, [20000], 64, 64)
    rng = np.random.default_rng(6)
    at = np.arange(20000)
    pg, row = c["table"][0, at // 64], at % 64
    for x in "kv":
        held = oracle.e4m3(rng.standard_normal(128))
        full = np.broadcast_to(held, c[x + "p64"].shape).copy()
        full[pg[777], :, row[777]] = oracle.e4m3(rng.standard_normal(128))
        c[x + "p"], c[x + "p64"] = torch.from_numpy(full).to(F8).cuda(), full
        c[x + "s"].fill_(1.0)
    near_, far = c["kp64"][pg[777], 0, row[777]], c["kp64"][pg[0], 0, row[0]]
    q = (near_ - far) / np.sum((near_ - far) ** 2) * 8.0 / c["scale"]  # scores 8 apart: weights of e^-8, 20000 of them
    c["q"], q64 = bf(np.broadcast_to(np.tile(q, 4), (2, 512)))
    c["q64"] = q64.reshape(1, 2, 4, 128)
    o, status = run(c)
    assert status == 0
    check(c, o, 0)


@pytest.mark.parametrize("value", [float("inf"), float("nan"), -float("inf")])
@pytest.mark.parametrize("n,g", [(7, 1), (16, 4), (40, 8)])
def test_tree_attention_fp8_masked_rows_do_not_matter(n, g, value):
    """Rows of nodes that are not finite change nothing in the nodes that do not descend from them; nor does what stands behind the
    cache's last row (NaN, under scales that are none), nor in pages of no sequence."""
    c = case(7, 2, n, g, 1, 128, [75, 130], 64, 16)
    o0, _ = run(c)
    bad = 2
    c["k"][bad].fill_(value)
    c["v"][bad].fill_(value)
    used = np.zeros((c["pool"], c["page"]), bool)
    for s in range(2):
        at = np.arange(c["lens"][s])
        used[c["table"][s, at // c["page"]], at % c["page"]] = True
    hole = torch.from_numpy(~used).cuda()[:, None, :, None].expand(-1, c["Hkv"], -1, c["D"])
    none = torch.from_numpy(~used.reshape(c["pool"], -1, c["block"]).any(-1)).cuda()[:, None].expand(-1, c["Hkv"], -1)
    for x in "kv":
        c[x + "p"].view(torch.uint8)[hole] = 0x7F
        c[x + "s"][none] = value
    o, status = run(c)
    assert status == 0
    below = {v for v in range(n) if bad in _chain(c["par"][0], v)}
    clean = [v for v in range(n) if v not in below]
    np.testing.assert_array_equal(o[0][clean], o0[0][clean])
    np.testing.assert_array_equal(o[1], o0[1])
    assert not np.isfinite(o[0][sorted(below)]).any(axis=-1).all()


def test_tree_attention_fp8_one_value_reaches_one_column():
    """An infinite value of v in a row that a node sees: that column alone, in the nodes that see it.  A NaN that the cache holds in
    v: that column of all nodes."""
    c = case(8, 1, 16, 2, 1, 64, [40], 16, 8)
    o0, _ = run(c)
    c["v"][3, 11] = float("inf")
    o, _ = run(c)
    below = [v for v in range(16) if 3 in _chain(c["par"][0], v)]
    rest = [v for v in range(16) if v not in below]
    assert np.isposinf(o[0][below][:, :, 11]).all()
    cols = np.arange(64) != 11
    np.testing.assert_array_equal(o[0][rest], o0[0][rest])
    # the row's other values are added by themselves: the same sums in another order
    assert (np.abs(o[0][below][:, :, cols] - o0[0][below][:, :, cols]) <= 2 * U * np.abs(o0[0][below][:, :, cols]) + 1e-5).all()
    c = case(8, 1, 16, 2, 1, 64, [40], 16, 8)
    c["vp"].view(torch.uint8)[c["table"][0, 1], 0, 5, 20] = 0x7F
    o, _ = run(c)
    assert np.isnan(o[0][:, :, 20]).all()
    cols = np.arange(64) != 20
    np.testing.assert_array_equal(o[0][:, :, cols], o0[0][:, :, cols])


def test_tree_attention_fp8_bad_device_data():
    from speculative_decoding_mamba2_gb300 import (SSM_STATUS_BAD_LAYOUT, SSM_STATUS_SCALE, SSM_STATUS_SEQ_RANGE,
                                                   ssm_tree_layout_build)
    c = case(9, 2, 9, 2, 2, 64, [100, 60], 16, 8)
    o, status = run(c, lens=[100, -1])
    assert status == SSM_STATUS_SEQ_RANGE
    check(c, o, 0)
    check(c, o, 1, length=0)
    o, status = run(c, lens=[101, 60])  # above the bound
    assert status == SSM_STATUS_SEQ_RANGE
    check(c, o, 0, length=0)
    check(c, o, 1)
    t = c["table"].copy()
    t[0, 1], t[1, 0] = -1, c["pool"]  # rows 16..31 of one, rows 0..15 of the other are absent
    o, status = run(c, table=t)
    assert status == SSM_STATUS_SEQ_RANGE
    for s, gone in ((0, range(16, 32)), (1, range(16))):
        kc, vc = cache(c, s, c["lens"][s])
        keep = [i for i in range(c["lens"][s]) if i not in gone]
        near(c, o, s, kc[keep], vc[keep])
    lay = ssm_tree_layout_build(c["par"])[0]
    lay[1, 4, 0], lay[1, 5, 0] = 4, 99  # its own parent; no node
    o, status = run(c, layout=lay)
    assert status == SSM_STATUS_BAD_LAYOUT
    par = c["par"][1].copy()
    par[[4, 5]] = -1
    check(c, o, 0)
    check(c, o, 1, par=par)
    for value in (0.0, -1.0, float("nan"), float("inf"), 2.0 ** -101, 2.0 ** 121):  # rows 8..15 of one, 56..59 of the other, of every head
        c = case(9, 2, 9, 2, 2, 64, [100, 60], 16, 8)
        c["ks"][c["table"][0, 0], :, 1] = value
        c["vs"][c["table"][1, 3], :, 1] = value
        o, status = run(c)
        assert status == SSM_STATUS_SCALE
        for s, gone in ((0, range(8, 16)), (1, range(56, 60))):
            kc, vc = cache(c, s, c["lens"][s])
            keep = [i for i in range(c["lens"][s]) if i not in gone]
            near(c, o, s, kc[keep], vc[keep])


def test_tree_attention_fp8_another_stream():
    c = case(10, 1, 16, 4, 2, 128, [3001], 64, 32)
    o0, _ = run(c)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    np.testing.assert_array_equal(run(c, stream=side)[0], o0)


@pytest.mark.parametrize("S,n,g,Hkv,D,top", [(40, 1, 4, 2, 128, 3001), (9, 16, 8, 3, 128, 2500), (80, 2, 1, 8, 64, 400), (33, 5, 3, 1, 64, 900)])
def test_tree_attention_fp8_ragged_batches(S, n, g, Hkv, D, top):
    """Caches from nothing to `top` rows, under the longest length as the bound and under a loose one; call after call the same."""
    rng = np.random.default_rng([S, top])
    lens = [0, top, 1, 64, 63] + [int(v) for v in np.exp(rng.uniform(0, np.log(top), S - 5))]
    c = case(11, S, n, g, Hkv, D, lens, 32, 16)
    for max_len in (None, 10 ** 6):
        o, status = run(c, max_len=max_len)
        assert status == 0
        for s in range(S):
            check(c, o, s)
        np.testing.assert_array_equal(run(c, max_len=max_len)[0], o)


@pytest.mark.parametrize("S,n,Hkv,D,L,page,block,in_place", [(1, 1, 1, 64, 1, 8, 8, False), (3, 7, 2, 128, 2, 16, 8, True), (5, 40, 3, 64, 3, 16, 16, False),
                                                             (2, 64, 8, 128, 1, 1024, 128, True), (4, 64, 1, 64, 2, 64, 64, False),
                                                             (9, 16, 8, 128, 4, 64, 16, True)])
def test_kv_commit_fp8(S, n, Hkv, D, L, page, block, in_place):
    """Paths that start and end anywhere in blocks, large rows among them so that blocks grow; the bits of the definition."""
    from speculative_decoding_mamba2_gb300 import ssm_kv_commit_fp8
    rng = np.random.default_rng([12, S, n, L])
    mp = n + 3
    lens = rng.integers(0, 3 * page, S)
    lens[0] = page - 1
    pl = np.array([0 if s == 2 else 1 + (5 * s + n - 1) % n for s in range(S)])
    path = np.full((S, mp), -1, np.int32)
    for s in range(S):
        path[s, :pl[s]] = np.sort(rng.permutation(n)[:pl[s]])
    per = int(max(-(-(lens + pl) // page)))
    pool = S * per + 1
    table = rng.permutation(pool)[:S * per].astype(np.int32).reshape(S, per)
    (kp, ks, kp64, ks64), (vp, vs, vp64, vs64) = (pages(rng, L, pool, Hkv, page, D, block) for _ in range(2))
    grow = np.exp2(np.round(3 * rng.standard_normal((L, S * n, 1))))
    (k, k64), (v, v64) = (bf(rng.standard_normal((L, S * n, Hkv * D)) * grow) for _ in range(2))
    ln = ints(lens)
    out = ln if in_place else torch.zeros(S, dtype=torch.int32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    ssm_kv_commit_fp8(S, n, ints(path), ints(pl), k, v, kp, vp, ks, vs, ints(table), ln, out, status=status)
    assert int(status) == 0
    for l in range(L):
        for s in range(S):
            for held, scale, rows in ((kp64, ks64, k64), (vp64, vs64, v64)):
                new = oracle.kv_commit_fp8(held[l], scale[l], rows[l].reshape(S, n, Hkv, D)[s], path[s, :pl[s]], table[s], int(lens[s]))
                assert int(out[s]) == new
    for got, want in ((kp, kp64), (vp, vp64), (ks, ks64), (vs, vs64)):
        np.testing.assert_array_equal(host(got), want)


@pytest.mark.parametrize("D", [64, 128])
def test_kv_commit_fp8_extreme_values(D):
    """Zeros, the least and the largest magnitudes, values that are not finite: the definition's bits; a block of zeros that then
    gets rows; step by step as in one go but for what the older rows lose when a block grows."""
    from speculative_decoding_mamba2_gb300 import ssm_kv_commit_fp8
    rng = np.random.default_rng(13)
    n, page = 8, 8
    base = rng.standard_normal((1, n, D))
    scale = np.array([0.0, 1e-38, 1e-30, 1e-3, 1.0, 448.0, 1e30, 3e38]).reshape(1, n, 1)
    with np.errstate(over="ignore"):
        k, k64 = bf(np.clip(base * scale, -3.3e38, 3.3e38))
    k[0, 4, 3], k[0, 4, 4], k[0, 5, 9] = float("inf"), float("nan"), -float("inf")
    k64[0, 4, 3], k64[0, 4, 4], k64[0, 5, 9] = np.inf, np.nan, -np.inf
    table, z = ints([[1]]), lambda: (torch.zeros(1, 2, 1, page, D, dtype=F8, device="cuda"), torch.full((1, 2, 1, 1), 5.0, device="cuda"))
    (kp, ks), (vp, vs) = z(), z()
    h = dict(k=(np.zeros((2, 1, page, D)), np.full((2, 1, 1), 5.0)))
    ln = ints([0])
    for i in range(n):
        ssm_kv_commit_fp8(1, n, ints([[i]]), ints([1]), k, k, kp, vp, ks, vs, table, ln, ln)
        oracle.kv_commit_fp8(*h["k"], k64[0][:, None], [i], [1], i)
        for got, want in ((kp[0], h["k"][0]), (ks[0], h["k"][1]), (vp[0], h["k"][0]), (vs[0], h["k"][1])):
            np.testing.assert_array_equal(host(got), want)
    assert int(ln) == 8 and torch.isnan(kp.float()).sum() == 3


def test_kv_commit_fp8_bad_device_data():
    from speculative_decoding_mamba2_gb300 import SSM_STATUS_PATH_RANGE, SSM_STATUS_SCALE, SSM_STATUS_SEQ_RANGE, ssm_kv_commit_fp8
    rng = np.random.default_rng(14)
    S, n, Hkv, D, page, pool = 4, 6, 1, 64, 8, 9
    (kp, ks, kp64, ks64), (vp, vs, vp64, vs64) = (pages(rng, 1, pool, Hkv, page, D, 8) for _ in range(2))
    (k, k64), (v, v64) = (bf(rng.standard_normal((1, S * n, Hkv * D))) for _ in range(2))
    table = np.array([[0, 1], [2, 3], [4, -1], [6, 7]], np.int32)
    path = np.array([[0, 1, 6, 2], [0, 1, 2, 3], [0, 2, 3, 4], [0, 1, 2, 5]], np.int32)
    lens, pl = [3, 14, 6, -2], [4, 4, 4, 9]
    out = torch.zeros(S, dtype=torch.int32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def both(status_is, counts):
        status.zero_()
        ssm_kv_commit_fp8(S, n, ints(path), ints(pl), k, v, kp, vp, ks, vs, ints(table), ints(lens), out, status=status)
        assert int(status) == status_is
        for s, m in enumerate(counts):
            for held, scale, rows in ((kp64, ks64, k64), (vp64, vs64, v64)):
                if m:
                    oracle.kv_commit_fp8(held[0], scale[0], rows[0].reshape(S, n, Hkv, D)[s], path[s, :m], table[s], lens[s])
        for got, want in ((kp, kp64), (vp, vp64), (ks, ks64), (vs, vs64)):
            np.testing.assert_array_equal(host(got), want)
        return out.cpu().numpy()

    # an entry that is no node, the end of the page table, a page that is none, a negative length
    np.testing.assert_array_equal(both(SSM_STATUS_PATH_RANGE | SSM_STATUS_SEQ_RANGE, [2, 2, 2, 0]), [5, 16, 8, -2])
    # scales that are none, of blocks that have rows: replaced
    for value in (float("nan"), 0.0, -1.0, float("inf")):
        ks[0, 0], ks64[0, 0], vs[0, 3], vs64[0, 3] = value, value, value, value
        both(SSM_STATUS_PATH_RANGE | SSM_STATUS_SEQ_RANGE | SSM_STATUS_SCALE, [2, 2, 2, 0])
    # ... and of one that has none yet: it does not count
    lens[0], ks[0, 0], ks64[0, 0] = 0, float("nan"), float("nan")
    both(SSM_STATUS_PATH_RANGE | SSM_STATUS_SEQ_RANGE, [2, 2, 2, 0])


@pytest.mark.parametrize("room", [0, 1, 5])
def test_kv_commit_fp8_lengths_up_to_an_int32(room):
    """A cache `room` rows below the longest length that an int32 holds, under a page table that goes on behind it."""
    from speculative_decoding_mamba2_gb300 import SSM_STATUS_SEQ_RANGE, ssm_kv_commit_fp8
    rng = np.random.default_rng(15)
    n, Hkv, D, page, block, pool = 4, 2, 64, 1024, 64, 3
    (kp, ks, kp64, ks64), (vp, vs, vp64, vs64) = (pages(rng, 1, pool, Hkv, page, D, block) for _ in range(2))
    (k, k64), (v, v64) = (bf(rng.standard_normal((1, n, Hkv * D))) for _ in range(2))
    table = torch.zeros(1, (1 << 21) + 2, dtype=torch.int32, device="cuda")
    table[0, (1 << 21) - 1], table[0, 1 << 21] = 2, 1
    length, want = (1 << 31) - 1 - room, min(room, 4)
    out, status = ints([0]), torch.zeros(1, dtype=torch.int32, device="cuda")
    ssm_kv_commit_fp8(1, n, ints([[0, 1, 2, 3]]), ints([4]), k, v, kp, vp, ks, vs, table, ints([length]), out, status=status)
    assert int(status) == (SSM_STATUS_SEQ_RANGE if want < 4 else 0) and int(out[0]) == length + want
    if want:
        at = length % page
        for held, scale, rows in ((kp64, ks64, k64), (vp64, vs64, v64)):
            oracle.kv_commit_fp8(held[0], scale[0], rows[0].reshape(n, Hkv, D), list(range(want)), [2], at)
    for got, ref in ((kp, kp64), (vp, vp64), (ks, ks64), (vs, vs64)):
        np.testing.assert_array_equal(host(got), ref)


def test_fp8_pages_past_32_bit_offsets():
    """Pages whose bytes lie past 2^32: read by the attention, written by the commit, as in a small pool."""
    from speculative_decoding_mamba2_gb300 import ssm_kv_commit_fp8
    c = case(16, 2, 4, 2, 2, 128, [300, 60], 128, 32)
    o0, status = run(c)
    assert status == 0
    total = 140000  # pages of 2 x 128 x 128: 4.6e9 bytes
    far = {x: torch.empty((total,) + c[x].shape[1:], dtype=c[x].dtype, device="cuda") for x in ("kp", "vp", "ks", "vs")}
    base = total - c["pool"]
    for x, t in far.items():
        t.view(torch.uint8)[base:] = c[x].view(torch.uint8)
    near_ = {x: c[x].clone() for x in far}
    big = dict(c, **far, table=c["table"] + base)
    o, status = run(big)
    assert status == 0
    np.testing.assert_array_equal(o, o0)
    path, pl, out = ints([[0, 1], [0, -1]]), ints([2, 1]), torch.zeros(2, dtype=torch.int32, device="cuda")
    k, v = 9.0 * c["k"].contiguous()[None], 9.0 * c["v"].contiguous()[None]
    for t, table in ((near_, c["table"]), (far, big["table"])):
        ssm_kv_commit_fp8(2, 4, path, pl, k, v, t["kp"][None], t["vp"][None], t["ks"][None], t["vs"][None], ints(table), ints(c["lens"]), out)
    torch.cuda.synchronize()
    assert out.tolist() == [302, 61]
    for x in far:
        a, b, was = (t.view(torch.uint8) for t in (far[x][base:].contiguous(), near_[x], c[x]))
        assert torch.equal(a, b) and not torch.equal(b, was)


def test_tree_attention_fp8_a_cache_of_zeros():
    """Keys and values that are all 0, in blocks of the least scale, as a commit of zeros leaves them."""
    c = case(20, 2, 9, 2, 2, 128, [3000, 65], 32, 8)
    for x in "kv":
        c[x + "p"] = torch.zeros_like(c[x + "p"])
        c[x + "s"] = torch.full_like(c[x + "s"], 2.0 ** -100)
        c[x + "p64"] = np.zeros_like(c[x + "p64"])
    o, status = run(c)
    assert status == 0
    for s in range(2):
        check(c, o, s)


@pytest.mark.parametrize("D", [64, 128])
def test_tree_attention_fp8_graphs_that_share_a_workspace(D):
    """Two captured calls over one workspace, replayed in turn after the lengths and q have changed: as called one by one."""
    from speculative_decoding_mamba2_gb300 import (ssm_tree_attention_fp8, ssm_tree_attention_fp8_workspace_size,
                                                   ssm_tree_layout_build)
    cases = [case(21, 1, 16, 4, 2, D, [4000], 64, 16), case(22, 5, 1, 8, 2, D, [700, 0, 64, 1500, 3], 32, 32)]
    sizes = [ssm_tree_attention_fp8_workspace_size(c["S"], c["n"], c["Hq"], c["Hkv"], D, max(c["lens"])) for c in cases]
    ws = torch.empty(max(sizes), dtype=torch.uint8, device="cuda")
    calls = []
    for c in cases:
        lay, table, lens = torch.from_numpy(ssm_tree_layout_build(c["par"])[0]).cuda(), ints(c["table"]), ints(c["lens"])
        o, status = torch.empty(c["S"] * c["n"], c["Hq"] * D, dtype=torch.bfloat16, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")

        def call(c=c, lay=lay, table=table, lens=lens, o=o, status=status):
            ssm_tree_attention_fp8(c["S"], c["n"], c["Hq"], c["Hkv"], D, lay, c["q"], c["k"], c["v"], c["kp"], c["vp"], c["ks"], c["vs"],
                                   table, lens, max(c["lens"]), c["scale"], o, ws, status=status)
        call()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            call()
        calls.append((c, graph, lens, o, status, call))  # (the call holds the layout and the table)
    for turn in range(3):
        for c, graph, lens, o, status, _ in calls:
            less = [max(l - 13 * turn, 0) for l in c["lens"]]
            lens.copy_(ints(less))
            c["q"].mul_(-1.0)
            c["q64"] = -c["q64"]
            o.fill_(9.0)
            graph.replay()
            torch.cuda.synchronize()
            assert int(status) == 0
            for s in range(c["S"]):
                check(c, host(o).reshape(c["S"], c["n"], c["Hq"], D), s, less[s])


FEW = [  # S, n, g, Hkv, lens, page, block: up to 16 query rows of a key/value head
    (1, 1, 8, 1, [0], 8, 8), (2, 8, 1, 2, [7, 8], 8, 8), (1, 2, 4, 3, [1], 64, 64), (3, 1, 1, 2, [15, 16, 17], 16, 8), (2, 9, 1, 2, [333, 0], 32, 16),
    (1, 16, 1, 2, [5000], 64, 32), (2, 1, 16, 1, [4097, 70], 128, 128), (1, 3, 5, 2, [2047], 8, 8), (4, 2, 8, 2, [129, 127, 1, 900], 1024, 512),
    (80, 1, 4, 8, [40 + 3 * i for i in range(80)], 32, 32), (1, 1, 3, 1, [70000], 256, 64)]


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("shape", FEW, ids=lambda s: str(s)[:40])
def test_tree_attention_fp8_few_rows(shape, D):
    S, n, g, Hkv, lens, page, block = shape
    c = case(23, S, n, g, Hkv, D, lens, page, block, fused=n % 2 == 1)
    o, status = run(c)
    assert status == 0
    for s in range(S):
        check(c, o, s)


@pytest.mark.parametrize("n,g", [(1, 8), (6, 2)])
def test_tree_attention_fp8_few_rows_of_large_scores_and_scales_far_apart(n, g):
    c = case(24, 2, n, g, 2, 128, [1700, 90], 16, 8, qscale=60.0)
    o, status = run(c)
    assert status == 0
    for s in range(2):  # products of a score add up to 60 times the ones of the tolerance
        near(c, o, s, *cache(c, s, c["lens"][s]), scores=60)
    c = case(25, 2, n, g, 2, 128, [1700, 90], 16, 8)
    by = np.exp2(np.random.default_rng([25, n]).integers(-60, 40, c["vs"].shape))
    held = c["vp64"] / np.repeat(c["vs"].double().cpu().numpy(), c["block"], -1)[..., None]
    c["vs"] = torch.from_numpy(by).float().cuda()
    c["vp64"] = held * np.repeat(by, c["block"], -1)[..., None]
    o, status = run(c)
    assert status == 0
    for s in range(2):
        check(c, o, s)


@pytest.mark.parametrize("n,g,D", [(1, 4, 128), (4, 2, 64), (12, 1, 128)])
def test_tree_attention_fp8_few_rows_bad_device_data(n, g, D):
    """Lengths, pages and scales that are out of range; a NaN of v in the cache and an infinity in a node's row: their columns alone."""
    from speculative_decoding_mamba2_gb300 import SSM_STATUS_SCALE, SSM_STATUS_SEQ_RANGE
    c = case(26, 2, n, g, 2, D, [100, 600], 16, 8)
    o, status = run(c, lens=[-5, 600])
    assert status == SSM_STATUS_SEQ_RANGE
    check(c, o, 0, length=0)
    check(c, o, 1)
    t = c["table"].copy()
    t[0, 1], t[1, 0] = -1, c["pool"]
    o, status = run(c, table=t)
    assert status == SSM_STATUS_SEQ_RANGE
    for s, gone in ((0, range(16, 32)), (1, range(16))):
        kc, vc = cache(c, s, c["lens"][s])
        keep = [i for i in range(c["lens"][s]) if i not in gone]
        near(c, o, s, kc[keep], vc[keep])
    clean, _ = run(c)
    col = np.arange(D) != 11
    c["vp"].view(torch.uint8)[c["table"][1, 30], 1, 5, 11] = 0x7F
    c["v"][0, 2 * D - 3] = float("inf")  # node 0 of one, its second head
    o, status = run(c)
    assert status == 0
    np.testing.assert_array_equal(o[1][:, :g], clean[1][:, :g])
    np.testing.assert_array_equal(o[1][:, g:][:, :, col], clean[1][:, g:][:, :, col])
    assert np.isnan(o[1][:, g:, 11]).all()
    seen = [v for v in range(n) if 0 in _chain(c["par"][0], v)]
    assert np.isposinf(o[0][seen][:, g:, D - 3]).all()
    rest = [v for v in range(n) if v not in seen]
    np.testing.assert_array_equal(o[0][rest], clean[0][rest])
    c["ks"][c["table"][0, 0], :, 1] = 0.0
    c["vs"][c["table"][1, 3], :, 1] = float("inf")
    c["vp"].view(torch.uint8)[c["table"][1, 3], :, 8:] = 0x7F  # not multiplied
    c["vp"].view(torch.uint8)[c["table"][1, 30], 1, 5, 11] = 0
    c["vp64"][c["table"][1, 30], 1, 5, 11] = 0
    c["v"][0, 2 * D - 3] = 0.0
    c["v64"][0, 0, 1, D - 3] = 0.0
    o, status = run(c)
    assert status == SSM_STATUS_SCALE
    for s, gone in ((0, range(8, 16)), (1, range(56, 64))):
        kc, vc = cache(c, s, c["lens"][s])
        keep = [i for i in range(c["lens"][s]) if i not in gone]
        near(c, o, s, kc[keep], vc[keep])


@pytest.mark.parametrize("n,g,D", [(1, 4, 128), (1, 4, 64), (4, 4, 128), (9, 4, 64)])
def test_tree_attention_fp8_without_a_cache(n, g, D):
    """No cached rows: pages, scales and the table, whatever its width, may be NULL."""
    from speculative_decoding_mamba2_gb300 import binding as B
    from speculative_decoding_mamba2_gb300 import ssm_tree_attention_fp8_workspace_size, ssm_tree_layout_build
    c = case(27, 3, n, g, 2, D, [0, 0, 0], 16, 8)
    Hq = c["Hq"]
    lay = torch.from_numpy(ssm_tree_layout_build(c["par"])[0]).cuda()
    ws = torch.empty(ssm_tree_attention_fp8_workspace_size(3, n, Hq, 2, D, 0), dtype=torch.uint8, device="cuda")
    o = torch.empty(3 * n, Hq * D, dtype=torch.bfloat16, device="cuda")
    lens, status = ints([0, 0, 0]), ints([0])
    rc = B.lib().ssm_tree_attention_fp8(3, n, Hq, 2, D, lay.data_ptr(), c["q"].data_ptr(), Hq * D, c["k"].data_ptr(), 2 * D, c["v"].data_ptr(),
                                        2 * D, None, None, None, None, 5, 16, 8, None, 7, lens.data_ptr(), 0, c["scale"], o.data_ptr(), Hq * D,
                                        ws.data_ptr(), ws.numel(), status.data_ptr(), torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    assert rc == B.SSM_OK and int(status) == 0
    for s in range(3):
        check(c, host(o).reshape(3, n, Hq, D), s, length=0)


def _own_key_over_a_flat_cache(n, g, D, length, nats):
    """A cache of nearly equal scores, `nats` below those of a node's own row and its ancestors'."""
    c = case(28, 1, n, g, 1, D, [length], 64, 32)
    u = np.random.default_rng([28, n, D]).choice([-1.0, 1.0], D)
    c["q"], c["q64"] = bf(np.broadcast_to(np.tile(u, g), (n, g * D)))
    c["k"], c["k64"] = bf(np.broadcast_to(u * nats / np.sqrt(D), (n, D)))
    c["q64"], c["k64"] = c["q64"].reshape(1, n, g, D), c["k64"].reshape(1, n, 1, D)
    c["ks"], c["kp64"] = c["ks"] * 2.0 ** -4, c["kp64"] * 2.0 ** -4
    return c


@pytest.mark.parametrize("length,nats", [(320, 6.0), (16384, 10.0)])  # not cut into runs; cut
@pytest.mark.parametrize("n,g,D", [(1, 4, 128), (1, 8, 64), (12, 1, 128), (16, 4, 128), (40, 2, 64)])
def test_tree_attention_fp8_values_of_any_size(n, g, D, length, nats):
    """Values of the cache and of the nodes' rows, all multiplied by a power of two: o is, and nothing else of it changes.  (The
    cache's weights are half of a root's, however small its values are beside 1.)"""
    c = _own_key_over_a_flat_cache(n, g, D, length, nats)
    o0, status = run(c)
    assert status == 0
    check(c, o0, 0)
    for by in (2.0 ** -10, 2.0 ** -16, 2.0 ** -30, 2.0 ** 20):
        d = dict(c, v=c["v"] * by, v64=c["v64"] * by, vs=c["vs"] * by, vp64=c["vp64"] * by)
        o, status = run(d)
        assert status == 0
        check(d, o, 0)
        np.testing.assert_array_equal(o, o0 * by)


@pytest.mark.parametrize("first,own", [(2.0 ** -100, 1.0), (2.0 ** -100, 2.0 ** 12), (2.0 ** -20, 2.0 ** 40), (2.0 ** 30, 1.0), (2.0 ** 90, 2.0 ** 30),
                                       (2.0 ** -100, 2.0 ** 48), (1.0, 2.0 ** 96)])
@pytest.mark.parametrize("n,g,length", [(1, 4, 700), (16, 4, 700), (3, 4, 300), (40, 2, 300)])
def test_tree_attention_fp8_first_blocks_of_another_size(n, g, length, first, own):
    """The cache's first 64 rows, zeros under the least scale among them, and the nodes' own rows far larger or smaller than the rest."""
    c = _own_key_over_a_flat_cache(n, g, 128, length, 6.0)
    pg = c["table"][0, 0]
    if first == 2.0 ** -100:
        c["vp"].view(torch.uint8)[pg] = 0
    held = c["vp"][pg].double().cpu().numpy()
    c["vs"][pg], c["vp64"][pg] = first, held * first
    c["v"], c["v64"] = c["v"] * own, c["v64"] * own
    o, status = run(c)
    assert status == 0
    check(c, o, 0)


@pytest.mark.parametrize("n,g,D", [(8, 4, 128), (40, 2, 64), (6, 2, 128)])
def test_tree_attention_fp8_rows_do_not_depend_on_each_other(n, g, D):
    """Children of one root, whose scores over the cache are 4 (in powers of two) above those of their own rows, and one whose are 12
    above: whether its k, far larger, hides the cache from it changes no bit of the others."""
    c = case(29, 1, n, g, 1, D, [300], 64, 16)
    u = np.random.default_rng([29, D]).choice([-1.0, 1.0], D)
    q = np.tile(u, (n, g))
    q[-1] *= 3.0
    c["q"], _ = bf(q)
    c["k"].zero_()
    c["par"][0] = [-1] + [0] * (n - 1)
    held = (c["kp64"] * 0.3 + u * 2.8 / np.sqrt(D)) * 64.0
    c["kp"], c["ks"] = torch.from_numpy(held).to(F8).cuda(), torch.full_like(c["ks"], 2.0 ** -6)
    o0, _ = run(c)
    c["k"][-1] = torch.from_numpy(u * 8.0)
    o, status = run(c)
    assert status == 0 and not np.array_equal(o[0][-1], o0[0][-1])
    np.testing.assert_array_equal(o[0][:-1], o0[0][:-1])


@pytest.mark.parametrize("value", [float("inf"), float("nan"), -float("inf")])
@pytest.mark.parametrize("n,g", [(7, 1), (16, 4), (40, 8)])
def test_tree_attention_fp8_a_bad_row_reaches_all_its_descendants(n, g, value):
    """A row of k and v that is not finite: no value of any node that descends from it is."""
    c = case(7, 2, n, g, 1, 128, [75, 130], 64, 16)
    c["k"][2].fill_(value)
    c["v"][2].fill_(value)
    o, _ = run(c)
    below = [v for v in range(n) if 2 in _chain(c["par"][0], v)]
    assert below and not np.isfinite(o[0][below]).any()


@pytest.mark.parametrize("n,g,D,lens", [(1, 4, 128, [3000, 65]), (12, 1, 64, [900, 7]), (16, 4, 128, [3000, 129]), (40, 8, 64, [700, 64])])
def test_tree_attention_fp8_weights_of_cached_rows(n, g, D, lens):
    """Weights of cached rows are held to 11 bits, not 8.  Tolerance: the output's rounding U|ref|, the fp32 part 2^-11 of all (as above),
    U of what the nodes' own rows add, 2^-11 of what the cache adds, and, for weights below fp16's normal numbers, 2^-32 of the largest
    product of a weight and its scale for each cached row, times its value of at most 448 of that scale."""
    c = case(30, 2, n, g, 2, D, lens, 64, 16)
    o, status = run(c)
    assert status == 0
    for s in range(2):
        kc, vc = cache(c, s, lens[s])
        args = c["q64"][s], c["k64"][s]
        ref, mag = oracle.tree_attention(*args, c["v64"][s], c["par"][s], kc, vc, c["scale"])
        own = oracle.tree_attention(*args, c["v64"][s], c["par"][s], kc, np.zeros_like(vc), c["scale"])[1]
        tail = lens[s] * 2.0 ** -32 * 448.0 * float(c["vs"].max())
        assert (np.abs(o[s] - ref) <= U * np.abs(ref) + 2.0 ** -11 * mag + U * own + 2.0 ** -11 * (mag - own) + tail).all()


@pytest.mark.parametrize("by", [2.0 ** -6, 2.0 ** -10, 2.0 ** -13, 2.0 ** -30])
@pytest.mark.parametrize("n,g,D,length,nats", [(1, 4, 128, 16384, 10.0), (1, 8, 64, 320, 6.0), (16, 4, 128, 16384, 10.0), (40, 2, 64, 320, 6.0)])
def test_tree_attention_fp8_small_values_of_one_sign(n, g, D, length, nats, by):
    """The same with values of the cache that are all positive, so that what a flat cache adds to a root's o is half of it and nothing of
    that averages out."""
    c = _own_key_over_a_flat_cache(n, g, D, length, nats)
    c["vp"].view(torch.uint8).bitwise_and_(0x7F)
    d = dict(c, v=c["v"] * by, v64=c["v64"] * by, vs=c["vs"] * by, vp64=np.abs(c["vp64"]) * by)
    o, status = run(d)
    assert status == 0
    check(d, o, 0)
