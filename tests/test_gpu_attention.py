"""Tree attention over a paged cache and the commit of the accepted path, on the GPU against the fp64 oracle.

Tolerance, before any run (u = 2^-8): the output's rounding u|ref|; the weights are rounded to bf16 for their product
with v, each summand off by at most u: u·mag with mag = sum of weight·|v|; fp32 scores, sums and exponentials: below
2^-11·mag for scores whose products add up to at most 100 in absolute value (8 accumulations of 2^-23·100, the
exponential 2^-22).  A commit copies: equal.
"""
import numpy as np
import pytest
import torch

import oracle
from synth import Shape, Workload, tree_parents

pytestmark = pytest.mark.gpu
U = 2.0 ** -8


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from speculative_decoding_mamba2_gb300 import build
    build.build()
    assert torch.cuda.is_available(), "GPU tests need CUDA"


def bf(v):
    t = torch.from_numpy(np.ascontiguousarray(v, np.float32)).bfloat16()
    return t.cuda(), t.double().numpy()


def host(t):
    return t.double().cpu().numpy()


def ints(v):
    return torch.tensor(np.asarray(v), dtype=torch.int32, device="cuda")


def tree(seed, n):
    return np.arange(-1, n - 1, dtype=np.int32) if n < 3 else \
        tree_parents(Workload(300 + seed, "t", Shape(H=1), 1, 1, trees=(("random", n, 3, 12),)), seed)


def case(seed, S, n, g, Hkv, D, lens, page, qscale=1.0, fused=False):
    rng = np.random.default_rng([seed, S, n, g, Hkv, D, page])
    Hq = g * Hkv
    per = max(1, max(-(-(l + n) // page) for l in lens))
    pool = S * per + 2
    c = dict(S=S, n=n, g=g, Hq=Hq, Hkv=Hkv, D=D, lens=list(lens), page=page, pool=pool, scale=D ** -0.5)
    c["par"] = np.stack([tree(seed + s, n) for s in range(S)])
    if fused:  # q, k and v are columns of one projection's output
        w = (Hq + 2 * Hkv) * D
        row, row64 = bf(rng.standard_normal((S * n, w + 8)) * np.concatenate([np.full(Hq * D, qscale), np.ones(2 * Hkv * D + 8)]))
        cut = [slice(0, Hq * D), slice(Hq * D, (Hq + Hkv) * D), slice((Hq + Hkv) * D, w)]
        (c["q"], c["k"], c["v"]), (q64, k64, v64) = (row[:, s] for s in cut), (row64[:, s] for s in cut)
    else:
        (c["q"], q64), (c["k"], k64), (c["v"], v64) = (bf(rng.standard_normal((S * n, h * D)) * f)
                                                       for h, f in ((Hq, qscale), (Hkv, 1.0), (Hkv, 1.0)))
    c["q64"], c["k64"], c["v64"] = q64.reshape(S, n, Hq, D), k64.reshape(S, n, Hkv, D), v64.reshape(S, n, Hkv, D)
    c["kp"], c["kp64"] = bf(rng.standard_normal((pool, Hkv, page, D)))
    c["vp"], c["vp64"] = bf(rng.standard_normal((pool, Hkv, page, D)))
    c["table"] = rng.permutation(pool)[:S * per].astype(np.int32).reshape(S, per)
    return c


def run(c, max_len=None, table=None, lens=None, layout=None, stream=None):
    from speculative_decoding_mamba2_gb300 import (ssm_tree_attention, ssm_tree_attention_workspace_size,
                                                   ssm_tree_layout_build)
    S, n, Hq, Hkv, D = (c[k] for k in ("S", "n", "Hq", "Hkv", "D"))
    max_len = max(c["lens"]) if max_len is None else max_len
    lay = ssm_tree_layout_build(c["par"])[0] if layout is None else layout
    ws = torch.full((ssm_tree_attention_workspace_size(S, n, Hq, Hkv, D, max_len),), 255, dtype=torch.uint8, device="cuda")
    o = torch.full((S * n, Hq * D + 8), 9.0, dtype=torch.bfloat16, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    ssm_tree_attention(S, n, Hq, Hkv, D, torch.from_numpy(lay).cuda(), c["q"], c["k"], c["v"], c["kp"], c["vp"],
                       ints(c["table"] if table is None else table), ints(c["lens"] if lens is None else lens), max_len, c["scale"],
                       o[:, :Hq * D], ws, status=status, stream=stream)
    torch.cuda.synchronize()
    assert (host(o[:, Hq * D:]) == 9.0).all()
    return host(o[:, :Hq * D]).reshape(S, n, Hq, D), int(status)


def cache(c, s, length):
    at = np.arange(length)
    pg, row = c["table"][s, at // c["page"]], at % c["page"]
    return c["kp64"][pg, :, row], c["vp64"][pg, :, row]


def check(c, o, s, length=None, par=None):
    kc, vc = cache(c, s, c["lens"][s] if length is None else length)
    ref, mag = oracle.tree_attention(c["q64"][s], c["k64"][s], c["v64"][s], c["par"][s] if par is None else par, kc, vc, c["scale"])
    assert (np.abs(o[s] - ref) <= U * np.abs(ref) + (U + 2.0 ** -11) * mag).all(), (s, np.max(np.abs(o[s] - ref) / mag))


SHAPES = [  # S, n, g, Hkv, D, lens, page
    (1, 1, 1, 1, 64, [0], 8), (1, 1, 1, 2, 128, [1], 16), (3, 1, 8, 2, 128, [63, 64, 65], 32), (2, 7, 1, 3, 64, [0, 200], 8),
    (2, 16, 4, 2, 128, [129, 31], 64), (1, 5, 5, 1, 128, [1000], 16), (3, 16, 2, 2, 64, [17, 0, 300], 128),
    (1, 64, 1, 1, 128, [70], 64), (1, 40, 8, 1, 128, [333], 64), (2, 64, 4, 1, 64, [64, 5], 32), (1, 9, 12, 1, 64, [2000], 256),
    (1, 33, 2, 2, 64, [100], 8), (1, 23, 32, 1, 128, [90], 1024)]


@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_tree_attention(shape):
    S, n, g, Hkv, D, lens, page = shape
    c = case(1, S, n, g, Hkv, D, lens, page, fused=n % 2 == 1)
    o, status = run(c)
    assert status == 0
    for s in range(S):
        check(c, o, s)


@pytest.mark.parametrize("n,g", [(1, 4), (16, 4), (40, 8)])
def test_tree_attention_long_cache_is_split(n, g):
    """Long caches beside short and empty ones: splits that a short sequence does not reach."""
    c = case(2, 3, n, g, 2, 128, [4099, 130, 0], 64)
    o, status = run(c)
    assert status == 0
    for s in range(3):
        check(c, o, s)


def test_tree_attention_large_scores():
    """Scores far apart (the maximum moves by hundreds between tiles): the weights of all but a few rows are 0."""
    c = case(3, 2, 16, 4, 1, 64, [700, 90], 16, qscale=60.0)
    o, status = run(c)
    assert status == 0
    kc = [cache(c, s, c["lens"][s]) for s in range(2)]
    for s in range(2):
        ref, mag = oracle.tree_attention(c["q64"][s], c["k64"][s], c["v64"][s], c["par"][s], *kc[s], c["scale"])
        # products of a score add up to 60 times the ones above: 60 * 2^-11 of mag
        assert (np.abs(o[s] - ref) <= U * np.abs(ref) + (U + 60 * 2.0 ** -11) * mag).all()


@pytest.mark.parametrize("value", [float("inf"), float("nan"), -float("inf")])
@pytest.mark.parametrize("n,g", [(7, 1), (16, 4), (40, 8)])
def test_tree_attention_masked_rows_do_not_matter(n, g, value):
    """K and V rows of nodes that are not finite change nothing in the nodes that do not descend from them; nor does
    what stands behind the cache's last row, nor in pages of no sequence."""
    c = case(4, 2, n, g, 1, 128, [75, 130], 64)
    o0, _ = run(c)
    bad = 2
    c["k"][bad].fill_(value)
    c["v"][bad].fill_(value)
    used = np.zeros((c["pool"], c["page"]), bool)
    for s in range(2):
        at = np.arange(c["lens"][s])
        used[c["table"][s, at // c["page"]], at % c["page"]] = True
    hole = torch.from_numpy(~used).cuda()[:, None, :, None].expand(-1, c["Hkv"], -1, c["D"])
    c["kp"][hole] = value
    c["vp"][hole] = value
    o, status = run(c)
    assert status == 0
    below = set()
    for v in range(n):
        u = v
        while u >= 0:
            if u == bad:
                below.add(v)
            u = int(c["par"][0][u])
    clean = [v for v in range(n) if v not in below]
    np.testing.assert_array_equal(o[0][clean], o0[0][clean])
    np.testing.assert_array_equal(o[1], o0[1])
    assert not np.isfinite(o[0][sorted(below)]).any(axis=-1).all()


def test_tree_attention_one_value_reaches_one_column():
    """An infinite value of v in a row that a node sees: that column alone, in the nodes that see it."""
    c = case(5, 1, 16, 2, 1, 64, [40], 16)
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


def _chain(par, v):
    out = []
    while v >= 0:
        out.append(v)
        v = int(par[v])
    return out


def test_tree_attention_bad_device_data():
    from speculative_decoding_mamba2_gb300 import SSM_STATUS_BAD_LAYOUT, SSM_STATUS_SEQ_RANGE, ssm_tree_layout_build
    c = case(6, 2, 9, 2, 2, 64, [100, 60], 16)
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
        ref, mag = oracle.tree_attention(c["q64"][s], c["k64"][s], c["v64"][s], c["par"][s], kc[keep], vc[keep], c["scale"])
        assert (np.abs(o[s] - ref) <= U * np.abs(ref) + (U + 2.0 ** -11) * mag).all()
    lay = ssm_tree_layout_build(c["par"])[0]
    lay[1, 4, 0], lay[1, 5, 0] = 4, 99  # its own parent; no node
    o, status = run(c, layout=lay)
    assert status == SSM_STATUS_BAD_LAYOUT
    par = c["par"][1].copy()
    par[[4, 5]] = -1
    check(c, o, 0)
    check(c, o, 1, par=par)


def test_tree_attention_another_stream():
    c = case(7, 1, 16, 4, 2, 128, [3000], 64)
    o0, _ = run(c)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    np.testing.assert_array_equal(run(c, stream=side)[0], o0)


def test_tree_attention_equals_chain_over_longer_cache():
    """The last node of a chain equals a single token whose ancestors stand in the cache."""
    c = case(8, 1, 12, 4, 2, 64, [50], 16)
    c["par"] = np.arange(-1, 11, dtype=np.int32)[None]
    o, _ = run(c)
    one = dict(c, n=1, lens=[61], par=np.array([[-1]], np.int32), q=c["q"][11:], k=c["k"][11:], v=c["v"][11:],
               kp=c["kp"].clone(), vp=c["vp"].clone())
    for i in range(11):
        pg, row = c["table"][0, (50 + i) // 16], (50 + i) % 16
        one["kp"][pg, :, row] = c["k"][i].view(2, 64)
        one["vp"][pg, :, row] = c["v"][i].view(2, 64)
    o1, _ = run(one)
    kc, vc = cache(c, 0, 50)
    ref, mag = oracle.tree_attention(c["q64"][0], c["k64"][0], c["v64"][0], c["par"][0], kc, vc, c["scale"])
    assert (np.abs(o1[0, 0] - o[0, 11]) <= 2 * U * np.abs(ref[11]) + 2 * (U + 2.0 ** -11) * mag[11]).all()


@pytest.mark.parametrize("S,n,Hkv,D,L,page,in_place", [(1, 1, 1, 64, 1, 8, False), (3, 7, 2, 128, 2, 8, True), (5, 40, 3, 64, 3, 16, False),
                                                       (2, 64, 8, 128, 1, 1024, True)])
def test_kv_commit(S, n, Hkv, D, L, page, in_place):
    from speculative_decoding_mamba2_gb300 import ssm_kv_commit
    rng = np.random.default_rng([9, S, n, L])
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
    (kp, kp64), (vp, vp64) = (bf(rng.standard_normal((L, pool, Hkv, page, D))) for _ in range(2))
    (k, k64), (v, v64) = (bf(rng.standard_normal((L, S * n, Hkv * D))) for _ in range(2))
    ln = ints(lens)
    out = ln if in_place else torch.zeros(S, dtype=torch.int32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    ssm_kv_commit(S, n, ints(path), ints(pl), k, v, kp, vp, ints(table), ln, out, status=status)
    assert int(status) == 0
    for l in range(L):
        for s in range(S):
            for pages, rows in ((kp64, k64), (vp64, v64)):
                new = oracle.kv_commit(pages[l], rows[l].reshape(S, n, Hkv, D)[s], path[s, :pl[s]], table[s], int(lens[s]))
                assert int(out[s]) == new
    np.testing.assert_array_equal(host(kp), kp64)
    np.testing.assert_array_equal(host(vp), vp64)


def test_kv_commit_bad_device_data():
    from speculative_decoding_mamba2_gb300 import SSM_STATUS_PATH_RANGE, SSM_STATUS_SEQ_RANGE, ssm_kv_commit
    rng = np.random.default_rng(10)
    S, n, Hkv, D, page, pool = 4, 6, 1, 64, 8, 9
    (kp, kp64), (vp, vp64) = (bf(rng.standard_normal((1, pool, Hkv, page, D))) for _ in range(2))
    (k, k64), (v, v64) = (bf(rng.standard_normal((1, S * n, Hkv * D))) for _ in range(2))
    table = np.array([[0, 1], [2, 3], [4, -1], [6, 7]], np.int32)
    path = np.array([[0, 1, 6, 2], [0, 1, 2, 3], [0, 2, 3, 4], [0, 1, 2, 5]], np.int32)
    lens, pl = [3, 14, 6, -2], [4, 4, 4, 9]
    out = torch.zeros(S, dtype=torch.int32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    ssm_kv_commit(S, n, ints(path), ints(pl), k, v, kp, vp, ints(table), ints(lens), out, status=status)
    assert int(status) == SSM_STATUS_PATH_RANGE | SSM_STATUS_SEQ_RANGE
    # an entry that is no node, the end of the page table, a page that is none, a negative length
    for s, m in enumerate([2, 2, 2, 0]):
        for pages, rows in ((kp64, k64), (vp64, v64)):
            oracle.kv_commit(pages[0], rows[0].reshape(S, n, Hkv, D)[s], path[s, :m], table[s], max(lens[s], 0))
    np.testing.assert_array_equal(out.cpu().numpy(), [5, 16, 8, -2])
    np.testing.assert_array_equal(host(kp), kp64)
    np.testing.assert_array_equal(host(vp), vp64)


@pytest.mark.parametrize("S,n,g,Hkv,top", [(40, 1, 4, 2, 3000), (9, 16, 8, 3, 2500), (80, 2, 1, 8, 400), (33, 5, 3, 1, 900)])
def test_tree_attention_ragged_batches(S, n, g, Hkv, top):
    """Caches from nothing to `top` rows, cut into runs of the same length (or not at all: 80 x 8 CTAs are enough), under the
    longest length as the bound and under a loose one."""
    rng = np.random.default_rng([S, top])
    lens = [0, top, 1, 64, 63] + [int(v) for v in np.exp(rng.uniform(0, np.log(top), S - 5))]
    c = case(8, S, n, g, Hkv, 128, lens, 32)
    for max_len in (None, 10 ** 6):
        o, status = run(c, max_len=max_len)
        assert status == 0
        for s in range(S):
            check(c, o, s)


def test_tree_attention_bad_lengths_beside_long_caches():
    """A length below 0 or past its pages counts as an empty cache; the others, cut into runs, are as they were."""
    from speculative_decoding_mamba2_gb300 import SSM_STATUS_SEQ_RANGE
    c = case(9, 4, 5, 2, 2, 64, [2000, 300, 1500, 700], 16)
    o, status = run(c, lens=[2000, -7, 1 << 30, 700], max_len=2000)
    assert status == SSM_STATUS_SEQ_RANGE
    for s, length in enumerate([2000, 0, 0, 700]):
        check(c, o, s, length=length)


def test_pages_past_32_bit_offsets():
    """Pages whose bytes and elements lie past 2^32: read by the attention, written by the commit, as in a small pool."""
    from speculative_decoding_mamba2_gb300 import ssm_kv_commit
    c = case(10, 2, 4, 2, 2, 128, [300, 64], 128)
    o0, status = run(c)
    assert status == 0
    total = 140000  # pages of 2 x 128 x 128 bf16: 4.6e9 elements
    far = {k: torch.empty(total, c["Hkv"], c["page"], c["D"], dtype=torch.bfloat16, device="cuda") for k in ("kp", "vp")}
    base = total - c["pool"]
    for k, pages in far.items():
        pages[base:] = c[k]
    near = {k: c[k].clone() for k in far}
    big = dict(c, **far, table=c["table"] + base)
    o, status = run(big)
    assert status == 0
    np.testing.assert_array_equal(o, o0)
    path, pl, out = ints([[0, 1], [0, -1]]), ints([2, 1]), torch.zeros(2, dtype=torch.int32, device="cuda")
    for kp, vp, table in ((near["kp"], near["vp"], c["table"]), (far["kp"], far["vp"], big["table"])):
        ssm_kv_commit(2, 4, path, pl, c["k"].contiguous()[None], c["v"].contiguous()[None], kp[None], vp[None], ints(table), ints(c["lens"]), out)
    torch.cuda.synchronize()
    assert out.tolist() == [302, 65]
    for k in far:
        assert torch.equal(far[k][base:], near[k]) and not torch.equal(near[k], c[k])
