"""Prompt conv, prompt scan and single-token scan on the GPU against the fp64 oracle.

Tolerances, before any run (u = 2^-8: one rounding to bf16, relative):
* conv: the output's rounding, u|ref|, and fp32 arithmetic of four products and a SiLU, 4e-6 of the summands' size.
* y: the output's rounding u|ref|; the scores and the state that y reads are rounded to bf16 once, so each summand
  may be off by u: u·mag, where mag is the oracle's run over absolute values; fp32 sums and exponentials, below
  2^-12·mag (exponents are sums of at most 64 terms: 64·2^-24·|S|·e^S; products add 128 + 64 terms).
* h: fp32 with products kept to 24 bits: per chunk of 64 tokens at most 4e-6 of mag (exponent sums 1.4e-6, the
  exponential 2.4e-7, 12 accumulations 1.5e-6), carried from chunk to chunk.
* one token: fp32 throughout, 2e-6·mag for h, and u|ref| + 2e-6·mag·N^(1/2) for y.
"""
import numpy as np
import pytest
import torch

import oracle

pytestmark = pytest.mark.gpu
U = 2.0 ** -8
P, N = 64, 128


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from speculative_decoding_mamba2_gb300 import build
    build.build()
    assert torch.cuda.is_available(), "GPU tests need CUDA"


def bf(v):
    """fp32 values rounded to bf16: (the GPU tensor, the values as fp64)."""
    t = torch.from_numpy(np.ascontiguousarray(v, np.float32)).bfloat16()
    return t.cuda(), t.double().numpy()


def f32(v):
    return torch.from_numpy(np.ascontiguousarray(v, np.float32)).cuda()


def host(t):
    return t.double().cpu().numpy()


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def params(rng, H, L):
    cd = H * P + 2 * N
    u = np.exp(rng.uniform(np.log(1e-3), np.log(0.1), (L, H)))
    p = dict(conv_w=rng.uniform(-0.5, 0.5, (L, cd, 4)), conv_b=0.1 * rng.standard_normal((L, cd)),
             dt_bias=np.log(np.expm1(u)), A_log=np.log(rng.uniform(1, 16, (L, H))), D=1 + 0.1 * rng.standard_normal((L, H)))
    p = {k: v.astype(np.float32) for k, v in p.items()}
    return {k: f32(v) for k, v in p.items()}, {k: v.astype(np.float64) for k, v in p.items()}


def scan_case(seed, H, G, lens, L=1, layer=0, extra_slots=1, fresh=False, pad=8, scale=1.0):
    """Tensors of one scan call; x, B, C are column views of one wider buffer."""
    rng = np.random.default_rng([seed, H, G, len(lens)])
    T, S = sum(lens), len(lens)
    prm, prm64 = params(rng, H, L)
    width = H * P + 2 * G * N
    v = rng.standard_normal((T, width + pad)) * scale
    row, row64 = bf(v / (1 + np.exp(-v)))
    dtw, dt64 = bf(0.5 * rng.standard_normal((T, H + 3)))
    n_slots = S + extra_slots
    h0 = (0.1 * rng.standard_normal((n_slots, L, H, P, N))).astype(np.float32)
    c = dict(H=H, G=G, L=L, layer=layer, lens=lens, T=T, S=S, prm=prm, prm64=prm64, n_slots=n_slots, h0=h0, fresh=fresh,
             x=row[:, :H * P], B=row[:, H * P:H * P + G * N], C=row[:, H * P + G * N:width], dt=dtw[:, :H],
             slots=rng.permutation(n_slots)[:S].astype(np.int32), cu=np.concatenate([[0], np.cumsum(lens)]).astype(np.int32))
    c["x64"], c["B64"], c["C64"] = (row64[:, :H * P].reshape(T, H, P), row64[:, H * P:H * P + G * N].reshape(T, G, N),
                                    row64[:, H * P + G * N:width].reshape(T, G, N))
    c["dt64"] = dt64[:, :H]
    return c


def reference(c, s, magnitude=False):
    """Oracle of sequence s."""
    p, l = c["prm64"], c["layer"]
    at = slice(c["cu"][s], c["cu"][s + 1])
    h0 = np.zeros((c["H"], P, N)) if c["fresh"] else c["h0"][c["slots"][s], l]
    return oracle.prompt_scan(c["x64"][at], c["B64"][at], c["C64"][at], c["dt64"][at], p["dt_bias"][l], p["A_log"][l], p["D"][l],
                              h0, magnitude)


def run_scan(c, in_place=False, max_len=None, stream=None):
    from speculative_decoding_mamba2_gb300 import Dims, ssm_prompt_scan, ssm_prompt_scan_workspace_size
    d = Dims(n_heads=c["H"], n_layers=c["L"])
    max_len = max(c["lens"]) if max_len is None else max_len
    h0 = f32(c["h0"])
    h = h0 if in_place else torch.full_like(h0, 7.0)
    y = torch.full((c["T"], c["H"] * P + 8), 9.0, dtype=torch.bfloat16, device="cuda")
    size = ssm_prompt_scan_workspace_size(d, c["S"], c["T"], max_len, c["G"])
    ws = torch.full((size,), 255, dtype=torch.uint8, device="cuda")  # NaN patterns: contents do not matter
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    ssm_prompt_scan(d, c["prm"], c["layer"], ints(c["cu"]), max_len, c["x"], c["B"], c["C"], c["dt"], None if c["fresh"] else h0, h,
                    y[:, :c["H"] * P], ws, slots=ints(c["slots"]), status=status, stream=stream)
    torch.cuda.synchronize()
    assert (host(y[:, c["H"] * P:]) == 9.0).all()  # nothing past a row
    return host(y[:, :c["H"] * P]).reshape(c["T"], c["H"], P), host(h), int(status)


def check_scan(c, y, h, in_place=False):
    touched = np.zeros(h.shape[:2], bool)
    for s in range(c["S"]):
        ry, rh = reference(c, s)
        my, mh = reference(c, s, magnitude=True)
        gy, gh = y[c["cu"][s]:c["cu"][s + 1]], h[c["slots"][s], c["layer"]]
        assert (np.abs(gy - ry) <= U * np.abs(ry) + (U + 2.0 ** -12) * my + 1e-30).all(), (s, "y")
        chunks = -(-c["lens"][s] // 64)
        assert (np.abs(gh - rh) <= 4e-6 * (1 + chunks) * mh + 1e-30).all(), (s, "h", np.max(np.abs(gh - rh) / (mh + 1e-30)))
        touched[c["slots"][s], c["layer"]] = True
    rest = c["h0"] if in_place else np.full_like(c["h0"], 7.0)
    np.testing.assert_array_equal(h[~touched], rest[~touched])


LENS = [[1], [2, 1, 3], [63, 64, 65], [128, 1, 0, 127], [0], [200, 17]]


@pytest.mark.parametrize("lens", LENS, ids=str)
@pytest.mark.parametrize("H,G", [(1, 1), (4, 1), (6, 3)])
def test_prompt_scan(H, G, lens):
    c = scan_case(1, H, G, lens)
    y, h, status = run_scan(c)
    assert status == 0
    check_scan(c, y, h)


@pytest.mark.parametrize("H,G,lens", [(2, 1, [777]), (3, 3, [1025, 300]), (24, 1, [513])])
def test_prompt_scan_long_axis(H, G, lens):
    """Few (sequence, head) pairs: a sequence's chunks are divided over segments; shorter ones use fewer."""
    c = scan_case(2, H, G, lens, fresh=H == 24)
    y, h, status = run_scan(c)
    assert status == 0
    check_scan(c, y, h)


@pytest.mark.parametrize("H,G,lens", [(2, 1, [65 * k + 3 for k in range(1, 9)]), (24, 2, [300 + 17 * k for k in range(13)])])
def test_prompt_scan_many_chunks(H, G, lens):
    """Enough (sequence, head) pairs that a sequence's chunks follow each other in one block."""
    c = scan_case(14, H, G, lens)
    y, h, status = run_scan(c)
    assert status == 0
    check_scan(c, y, h)


def test_prompt_scan_layers_in_place_and_loose_bound():
    c = scan_case(3, 4, 2, [70, 0, 5], L=3, layer=1)
    y, h, status = run_scan(c, in_place=True, max_len=1000)
    assert status == 0
    check_scan(c, y, h, in_place=True)


def test_prompt_scan_continues_itself():
    """A prompt in two calls equals it in one, within the bound of its parts."""
    c = scan_case(4, 4, 1, [150])
    _, h, _ = run_scan(c)
    a, b = dict(c, lens=[90], T=90, cu=np.array([0, 90], np.int32)), dict(c, lens=[60], T=60, cu=np.array([0, 60], np.int32))
    for k in ("x", "B", "C", "dt", "x64", "B64", "C64", "dt64"):
        a[k], b[k] = c[k][:90], c[k][90:]
    _, h1, _ = run_scan(a)
    b["h0"] = h1.astype(np.float32)
    y2, h2, _ = run_scan(b)
    check_scan(b, y2, h2)
    _, mh = reference(c, 0, magnitude=True)
    s = c["slots"][0]
    assert (np.abs(h2[s, 0] - h[s, 0]) <= 4e-6 * 8 * mh).all()


def test_prompt_scan_extreme_decays():
    """Step sizes from 0 to 80 at A = -16: decays of 1, and decays that are 0, next to each other."""
    c = scan_case(5, 4, 1, [140, 65])
    rng = np.random.default_rng(55)
    dt, dt64 = bf(rng.choice([-100.0, -20.0, 0.0, 5.0, 80.0], (c["T"], c["H"])))
    c["dt"], c["dt64"] = dt, dt64
    c["prm"]["A_log"].fill_(np.log(np.float32(16.0)))
    c["prm64"]["A_log"] = c["prm"]["A_log"].double().cpu().numpy()
    y, h, status = run_scan(c)
    assert status == 0 and np.isfinite(y).all() and np.isfinite(h).all()
    check_scan(c, y, h)


@pytest.mark.parametrize("what", ["x", "B", "C", "dt"])
@pytest.mark.parametrize("value", [float("inf"), float("nan")])
def test_prompt_scan_what_comes_later_does_not_matter(what, value):
    """A token that is not finite leaves the tokens before it, and the other sequences and heads, as they were."""
    c = scan_case(6, 4, 1, [100, 30])
    at = 70
    y0, h0, _ = run_scan(c)
    t = c[what] if what == "dt" else c["x"]._base
    if what == "dt":
        t[at, 1] = value
    else:
        col = dict(x=1 * P + 5, B=c["H"] * P + 9, C=c["H"] * P + N + 9)[what]
        t[at, col] = value
    y, h, status = run_scan(c)
    assert status == 0
    np.testing.assert_array_equal(y[:at], y0[:at])
    np.testing.assert_array_equal(y[100:], y0[100:])
    assert not np.isfinite(y[at, 1]).all()
    if what in ("x", "dt"):
        np.testing.assert_array_equal(y[:100, [0, 2, 3]], y0[:100, [0, 2, 3]])
        np.testing.assert_array_equal(h[c["slots"][0], 0][[0, 2, 3]], h0[c["slots"][0], 0][[0, 2, 3]])
    if what == "x":  # one value of x reaches one row of the state
        keep = np.arange(P) != 5
        assert np.isfinite(h[c["slots"][0], 0, 1][keep]).all() and not np.isfinite(h[c["slots"][0], 0, 1, 5]).any()
        assert np.isfinite(y[:100, 1][:, keep]).all()


def test_prompt_scan_skips_what_is_out_of_range():
    from speculative_decoding_mamba2_gb300 import SSM_STATUS_SEQ_RANGE
    for wrong in ("slot", "first", "long", "order"):
        c = scan_case(7, 4, 1, [20, 30, 10])
        slots, cu = c["slots"].copy(), c["cu"].copy()
        bad = {1}
        if wrong == "slot":
            c["slots"][1] = c["n_slots"]
        elif wrong == "first":
            c["cu"][0], bad = -3, {0}
        elif wrong == "order":
            c["cu"][2], bad = 10, {1, 2}  # sequence 2 then has 50 rows: more than the bound
        y, h, status = run_scan(c, max_len=20 if wrong == "long" else 30)
        assert status == SSM_STATUS_SEQ_RANGE
        c["slots"], c["cu"] = slots, cu
        good = [s for s in range(3) if s not in bad]
        for s in good:
            ry, rh = reference(c, s)
            my, _ = reference(c, s, magnitude=True)
            assert (np.abs(y[cu[s]:cu[s + 1]] - ry) <= U * np.abs(ry) + (U + 2.0 ** -12) * my).all(), (wrong, s)
        for s in bad:
            assert (y[cu[s]:cu[s + 1]] == 9.0).all() and (h[slots[s]] == 7.0).all(), (wrong, s)


def test_prompt_scan_another_stream():
    c = scan_case(8, 4, 1, [300])
    y0, h0, _ = run_scan(c)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y, h, _ = run_scan(c, stream=side)
    np.testing.assert_array_equal(y, y0)
    np.testing.assert_array_equal(h, h0)


def test_prompt_scan_empty_calls():
    c = scan_case(9, 4, 1, [0, 0])
    y, h, status = run_scan(c, max_len=0)
    assert status == 0
    for s in range(2):
        np.testing.assert_array_equal(h[c["slots"][s], 0], c["h0"][c["slots"][s], 0])


@pytest.mark.parametrize("H,G,S,fresh", [(1, 1, 1, False), (4, 2, 3, False), (24, 1, 5, True), (6, 3, 17, False)])
def test_scan_step(H, G, S, fresh):
    from speculative_decoding_mamba2_gb300 import Dims, ssm_scan_step
    for in_place in (False, True):
        c = scan_case(11, H, G, [1] * S, L=2, layer=1, fresh=fresh)
        h0 = f32(c["h0"])
        h = h0 if in_place else torch.full_like(h0, 7.0)
        y = torch.empty(S, H * P, dtype=torch.bfloat16, device="cuda")
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        ssm_scan_step(Dims(n_heads=H, n_layers=2), c["prm"], 1, c["x"], c["B"], c["C"], c["dt"], None if fresh else h0, h, y,
                      slots=ints(c["slots"]), status=status)
        y, h = host(y).reshape(S, H, P), host(h)
        assert int(status) == 0
        for s in range(S):
            ry, rh = reference(c, s)
            my, mh = reference(c, s, magnitude=True)
            assert (np.abs(y[s] - ry[0]) <= U * np.abs(ry[0]) + 2e-6 * N ** 0.5 * my[0]).all()
            assert (np.abs(h[c["slots"][s], 1] - rh) <= 2e-6 * mh).all()
        rest = np.ones(c["n_slots"], bool)
        rest[c["slots"]] = False
        keep = c["h0"] if in_place else np.full_like(c["h0"], 7.0)
        np.testing.assert_array_equal(h[rest], keep[rest])
        np.testing.assert_array_equal(h[:, 0], keep[:, 0])


def test_scan_step_bad_slot():
    from speculative_decoding_mamba2_gb300 import SSM_STATUS_SEQ_RANGE, Dims, ssm_scan_step
    c = scan_case(12, 4, 1, [1, 1, 1])
    h = f32(c["h0"])
    y = torch.full((3, 4 * P), 9.0, dtype=torch.bfloat16, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    ssm_scan_step(Dims(n_heads=4), c["prm"], 0, c["x"], c["B"], c["C"], c["dt"], h, h, y, slots=ints([0, -1, 4]), status=status)
    assert int(status) == SSM_STATUS_SEQ_RANGE
    assert (host(y[1:]) == 9.0).all() and not (host(y[0]) == 9.0).all()
    np.testing.assert_array_equal(host(h)[1:], c["h0"][1:])


def test_scan_steps_follow_a_prompt():
    """A prompt, then its next tokens one by one, against the whole sequence."""
    from speculative_decoding_mamba2_gb300 import Dims, ssm_scan_step
    c = scan_case(13, 4, 1, [75])
    ry, rh = reference(c, 0)
    my, mh = reference(c, 0, magnitude=True)
    a = dict(c, lens=[70], T=70, cu=np.array([0, 70], np.int32), **{k: c[k][:70] for k in ("x", "B", "C", "dt")})
    _, h, _ = run_scan(a)
    h, s = f32(h), ints(c["slots"])
    y = torch.empty(1, 4 * P, dtype=torch.bfloat16, device="cuda")
    for t in range(70, 75):
        ssm_scan_step(Dims(n_heads=4), c["prm"], 0, *(c[k][t:t + 1] for k in ("x", "B", "C", "dt")), h, h, y, slots=s)
        assert (np.abs(host(y).reshape(4, P) - ry[t]) <= U * np.abs(ry[t]) + 3e-5 * my[t]).all()
    assert (np.abs(host(h)[c["slots"][0], 0] - rh) <= 2e-5 * mh).all()


@pytest.mark.parametrize("H,lens", [(1, [1]), (3, [1, 2, 3, 4]), (2, [7, 8, 9, 0, 25]), (24, [1, 1, 1]), (80, [19, 2]), (2, [35, 32, 33, 71]), (130, [37, 1])])
def test_prompt_conv(H, lens):
    from speculative_decoding_mamba2_gb300 import Dims, ssm_prompt_conv
    rng = np.random.default_rng([21, H])
    L, layer, R, T, S = 2, 1, 7, sum(lens), len(lens)
    cd = H * P + 2 * N
    prm, prm64 = params(rng, H, L)
    x, x64 = bf(rng.standard_normal((T, cd + 8)) * 2)
    ring, ring64 = bf(rng.standard_normal((S + 1, L, R, cd)))
    head = rng.integers(0, 50, (S + 1, L)).astype(np.int32)
    slots = rng.permutation(S + 1)[:S].astype(np.int32)
    out = torch.full((T, cd + 16), 9.0, dtype=torch.bfloat16, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    hd = ints(head)
    cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    ssm_prompt_conv(Dims(n_heads=H, n_layers=L, ring_cap=R), prm, layer, ints(cu), max(lens), x[:, :cd], ring, hd, out[:, :cd],
                    slots=ints(slots), status=status)
    got, new_ring, new_head = host(out), host(ring), hd.cpu().numpy()
    assert int(status) == 0 and (got[:, cd:] == 9.0).all()
    for s in range(S):
        k, f = slots[s], int(head[slots[s], layer])
        win = np.stack([ring64[k, layer, (f - j) % R] for j in (3, 2, 1)])
        rows = x64[cu[s]:cu[s + 1], :cd]
        ref, last, mag = oracle.prompt_conv(prm64["conv_w"][layer], prm64["conv_b"][layer], rows, win)
        assert (np.abs(got[cu[s]:cu[s + 1], :cd] - ref) <= U * np.abs(ref) + 4e-6 * mag + 1e-33).all()
        assert new_head[k, layer] == f + lens[s]
        np.testing.assert_array_equal(np.stack([new_ring[k, layer, (f + lens[s] - j) % R] for j in (3, 2, 1)]), last)
    rest = [k for k in range(S + 1) if k not in slots]
    np.testing.assert_array_equal(new_ring[rest], ring64[rest])
    np.testing.assert_array_equal(new_ring[:, 0], ring64[:, 0])
    np.testing.assert_array_equal(new_head[:, 0], head[:, 0])
    np.testing.assert_array_equal(new_head[rest], head[rest])


def test_prompt_conv_skips_what_is_out_of_range():
    from speculative_decoding_mamba2_gb300 import SSM_STATUS_SEQ_RANGE, Dims, ssm_prompt_conv
    rng = np.random.default_rng(22)
    cd = 64 + 256
    prm, _ = params(rng, 1, 1)
    x, _ = bf(rng.standard_normal((20, cd)))
    for cu, slots in (([0, 10, 20], [5, 1]), ([-1, 10, 20], [0, 1]), ([0, 15, 20], [0, 1]), ([0, 30, 20], [0, 1])):
        ring, ring64 = bf(rng.standard_normal((2, 4, cd)))
        head = ints([3, 3])
        out = torch.full((20, cd), 9.0, dtype=torch.bfloat16, device="cuda")
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        ssm_prompt_conv(Dims(n_heads=1, ring_cap=4), prm, 0, ints(cu), 12, x, ring, head, out, slots=ints(slots), status=status)
        assert int(status) == SSM_STATUS_SEQ_RANGE
        assert head[0] == 3 and (host(ring)[0] == ring64[0]).all() and (host(out)[:10] == 9.0).all()


@pytest.mark.parametrize("H,G,lens", [(4, 1, [63, 64, 65]), (4, 2, [1, 128, 0, 127, 2]), (2, 1, [190, 0, 3]), (6, 3, [64] * 5),
                                      (24, 1, [1 + (37 * k) % 401 for k in range(40)]), (24, 1, [2000, 30, 700])], ids=str)
def test_prompt_scan_ragged_batches(H, G, lens):
    """Short, whole-chunk and empty sequences beside long ones, under the longest length and under a loose bound."""
    c = scan_case(21, H, G, lens)
    for max_len in (None, 10 ** 6):
        y, h, status = run_scan(c, max_len=max_len)
        assert status == 0
        check_scan(c, y, h)


def test_prompt_scan_extreme_decays_long():
    """Decays of 1 and of 0 next to each other, over chunks and segments."""
    c = scan_case(22, 4, 1, [1000, 65, 140])
    rng = np.random.default_rng(56)
    dt, dt64 = bf(rng.choice([-100.0, -20.0, 0.0, 5.0, 80.0], (c["T"], c["H"])))
    c["dt"], c["dt64"] = dt, dt64
    c["prm"]["A_log"].fill_(np.log(np.float32(16.0)))
    c["prm64"]["A_log"] = c["prm"]["A_log"].double().cpu().numpy()
    y, h, status = run_scan(c)
    assert status == 0 and np.isfinite(y).all() and np.isfinite(h).all()
    check_scan(c, y, h)


@pytest.mark.parametrize("what", ["x", "B", "C", "dt"])
@pytest.mark.parametrize("value", [float("inf"), -float("inf"), float("nan")])
@pytest.mark.parametrize("at", [64, 200, 1100])
def test_prompt_scan_what_comes_later_does_not_matter_long(what, value, at):
    """As above over many chunks: at a chunk's first token, inside one, and in a later segment."""
    c = scan_case(23, 4, 1, [1200, 130])
    y0, h0, _ = run_scan(c)
    t = c[what] if what == "dt" else c["x"]._base
    if what == "dt":
        t[at, 1] = value if value > 0 or value != value else float("nan")  # (softplus of -infinity is 0)
    else:
        t[at, dict(x=1 * P + 5, B=c["H"] * P + 9, C=c["H"] * P + N + 9)[what]] = value
    y, h, status = run_scan(c)
    assert status == 0
    np.testing.assert_array_equal(y[:at], y0[:at])
    np.testing.assert_array_equal(y[1200:], y0[1200:])
    np.testing.assert_array_equal(h[c["slots"][1]], h0[c["slots"][1]])
    assert not np.isfinite(y[at, 1]).all()
    s = c["slots"][0]
    if what in ("x", "dt"):
        np.testing.assert_array_equal(y[:, [0, 2, 3]], y0[:, [0, 2, 3]])
        np.testing.assert_array_equal(h[s, 0][[0, 2, 3]], h0[s, 0][[0, 2, 3]])
    if what == "x":  # one value of x reaches one row of the state
        keep = np.arange(P) != 5
        assert np.isfinite(h[s, 0, 1][keep]).all() and np.isfinite(y[:, 1][:, keep]).all()
    if what == "C":  # an output alone
        np.testing.assert_array_equal(h, h0)
        np.testing.assert_array_equal(y[at + 1:], y0[at + 1:])


def test_prompt_scan_skips_what_is_out_of_range_long():
    from speculative_decoding_mamba2_gb300 import SSM_STATUS_SEQ_RANGE
    for wrong in ("slot", "first", "long", "order"):
        c = scan_case(24, 4, 1, [200, 300, 100])
        slots, cu = c["slots"].copy(), c["cu"].copy()
        bad = {1}
        if wrong == "slot":
            c["slots"][1] = -1
        elif wrong == "first":
            c["cu"][0], bad = -3, {0}
        elif wrong == "order":
            c["cu"][2], bad = 100, {1, 2}  # sequence 2 then has 500 rows: more than the bound
        y, h, status = run_scan(c, max_len=250 if wrong == "long" else 300)
        assert status == SSM_STATUS_SEQ_RANGE
        c["slots"], c["cu"] = slots, cu
        for s in range(3):
            if s in bad:
                assert (y[cu[s]:cu[s + 1]] == 9.0).all() and (h[slots[s]] == 7.0).all(), (wrong, s)
                continue
            ry, rh = reference(c, s)
            my, mh = reference(c, s, magnitude=True)
            assert (np.abs(y[cu[s]:cu[s + 1]] - ry) <= U * np.abs(ry) + (U + 2.0 ** -12) * my).all(), (wrong, s)
            assert (np.abs(h[slots[s], 0] - rh) <= 4e-6 * 6 * mh).all(), (wrong, s)


@pytest.mark.parametrize("H,G", [(3, 3), (4, 1)])
def test_prompt_scan_in_place_over_segments(H, G):
    """A prompt cut into segments (by either kernel), its state written over the one it starts from: as out of place."""
    c = scan_case(25, H, G, [3000, 100, 1300])
    y0, h0, _ = run_scan(c)
    y, h, status = run_scan(c, in_place=True)
    assert status == 0
    np.testing.assert_array_equal(y, y0)
    check_scan(c, y, h, in_place=True)
    for s in range(c["S"]):
        np.testing.assert_array_equal(h[c["slots"][s], 0], h0[c["slots"][s], 0])


@pytest.mark.parametrize("H,G", [(2, 1), (1, 1)])
def test_prompt_scan_and_conv_past_32_bit_offsets(H, G):
    """Rows 2^25 elements apart (the last one starts past 2^32 elements): as rows side by side, by either scan kernel."""
    from speculative_decoding_mamba2_gb300 import Dims, ssm_prompt_conv, ssm_prompt_scan, ssm_prompt_scan_workspace_size
    T, ld = 200, 1 << 25
    c = scan_case(26, H, G, [T])
    y0, h0, _ = run_scan(c)
    d = Dims(n_heads=H)
    wide = torch.empty(T, ld, dtype=torch.bfloat16, device="cuda")
    cols, at = {}, 0
    for k, n in (("x", H * P), ("B", G * N), ("C", G * N), ("dt", H), ("y", H * P), ("pre", d.conv_dim), ("post", d.conv_dim)):
        cols[k], at = wide[:, at:at + n], at + (n + 7) // 8 * 8
    for k in ("x", "B", "C", "dt"):
        cols[k].copy_(c[k])
    h = torch.empty_like(f32(c["h0"]))
    ws = torch.empty(ssm_prompt_scan_workspace_size(d, 1, T, T, G), dtype=torch.uint8, device="cuda")
    ssm_prompt_scan(d, c["prm"], 0, ints(c["cu"]), T, cols["x"], cols["B"], cols["C"], cols["dt"], f32(c["h0"]), h, cols["y"], ws,
                    slots=ints(c["slots"]))
    np.testing.assert_array_equal(host(cols["y"]).reshape(T, H, P), y0)
    np.testing.assert_array_equal(host(h)[c["slots"][0]], h0[c["slots"][0]])

    pre = torch.randn(T, d.conv_dim, device="cuda").bfloat16()
    prm = dict(conv_w=torch.randn(1, d.conv_dim, 4, device="cuda"), conv_b=torch.randn(1, d.conv_dim, device="cuda"))
    cols["pre"].copy_(pre)
    outs = []
    for x, out in ((pre, torch.empty_like(pre)), (cols["pre"], cols["post"])):
        ring, head = torch.zeros(1, 1, 20, d.conv_dim, dtype=torch.bfloat16, device="cuda"), torch.full((1, 1), 3, dtype=torch.int32, device="cuda")
        ssm_prompt_conv(d, prm, 0, ints([0, T]), T, x, ring, head, out)
        outs.append((out.clone(), ring, head))
    for a, b in zip(*outs):
        assert torch.equal(a, b)
