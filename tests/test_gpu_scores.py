"""Log probabilities, entropy and top alternatives on the GPU against the fp64 oracle.

Tolerance, before any run: a thread adds up at most V / 512 terms one after the other and the threads' sums are joined in 30 steps,
each a rounding of 2^-24 of a sum of positive terms; a term's exponential is off by 2^-21 and its argument by 2^-22 of itself, which
adds at most 2^-22 E|argument| (below ln V + 30 here) to the sum; the difference to the maximum and the final sum round by 2^-23 of
themselves.  So a log probability is off by at most  E = (V / 512 + 64) 2^-24 + (ln V + 32) 2^-22 + 2^-20  and 2^-22 of itself,
and the entropy, whose second sum's terms are weighted by arguments, by E (1 + ln V) + 2^-22 of itself.  Indices are equal."""
import numpy as np
import pytest
import torch

import oracle
from tests.test_gpu_attention import _lib, host, ints  # noqa: F401 (the fixture builds the library)

pytestmark = pytest.mark.gpu


def run(x, tokens, k, scale=1.0, entropy=True, stream=None):
    from speculative_decoding_mamba2_gb300 import ssm_token_scores
    T, m = tokens.shape
    f = lambda *shape: torch.full(shape, 7.0, device="cuda")  # noqa: E731
    lp, h, tlp, top = f(T, m), f(T), f(T, k), torch.full((T, k), 7, dtype=torch.int32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    ssm_token_scores(x, ints(tokens).view(T, m), lp, h if entropy else None, top, tlp, scale=scale, status=status, stream=stream)
    torch.cuda.synchronize()
    return host(lp), host(h), top.cpu().numpy(), host(tlp), int(status)


def check(x, tokens, k, scale=1.0, bad=0):
    lp, h, top, tlp, status = run(x, tokens, k, scale)
    assert status == bad
    want = oracle.token_scores(x.double().cpu().numpy(), tokens, k, scale)
    V = x.shape[1]
    E = (V / 512 + 64) * 2.0 ** -24 + (np.log(V) + 32) * 2.0 ** -22 + 2.0 ** -20
    np.testing.assert_array_equal(top, want[2])
    for got, ref, e in ((lp, want[0], E), (tlp, want[3], E), (h, want[1], E * (1 + np.log(V)))):
        np.testing.assert_allclose(got, ref, rtol=2.0 ** -22, atol=e)


def logits(rng, T, V, dtype, spread=2.0, ld=None, at=0):
    """A view of T rows of V logits, `at` elements into rows of ld."""
    x = rng.standard_normal((T, V)) * spread
    x[np.arange(T), rng.integers(0, V, T)] += rng.uniform(0, 12, T)
    ld = V if ld is None else ld
    buf = torch.full((T, ld), float("nan"), dtype=dtype, device="cuda")  # what stands beside the rows is not theirs
    buf[:, at:at + V] = torch.from_numpy(x).to(dtype)
    return buf[:, at:at + V]


SHAPES = [  # T, V, m, k, ld, at
    (1, 1, 1, 1, 1, 0), (3, 2, 2, 2, 2, 0), (2, 31, 0, 31, 40, 3), (5, 100, 3, 32, 100, 0), (1, 511, 1, 1, 520, 8), (4, 4097, 2, 8, 4097, 0),
    (1, 32003, 1, 4, 32003, 0), (2, 50280, 5, 16, 50288, 1), (17, 128259, 3, 8, 128259, 0), (1, 151936, 700, 32, 151936, 0),
    (700, 1000, 1, 4, 1001, 0), (3, 200000, 1, 0, 200000, 0), (2, 262145, 2, 5, 262160, 7)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=str)
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_token_scores(shape, dtype):
    T, V, m, k, ld, at = shape
    rng = np.random.default_rng([1, *shape])
    x = logits(rng, T, V, dtype, ld=ld, at=at)
    tok = rng.integers(0, V, (T, m))
    if m > 1:
        tok[:, 0], tok[0, 1] = int(x[0].argmax()), -1
    check(x, tok, k)


@pytest.mark.parametrize("scale", [0.2, 5.0])
def test_token_scores_temperature(scale):
    rng = np.random.default_rng(2)
    check(logits(rng, 3, 40001, torch.float32), rng.integers(0, 40001, (3, 4)), 6, scale)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=str)
@pytest.mark.parametrize("V", [77, 5000, 131075])
def test_token_scores_ties(V, dtype):
    """Rows of one value, of few values, rising, falling, and with many equal maxima: the lowest indices first."""
    rng = np.random.default_rng([3, V])
    x = torch.zeros(7, V, dtype=dtype, device="cuda")
    x[1] = -3.0
    x[2] = torch.from_numpy(rng.integers(-2, 3, V)).to(dtype)
    x[3] = torch.linspace(-20, 20, V).to(dtype)
    x[4] = torch.linspace(20, -20, V).to(dtype)
    x[5, ::7] = 4.0
    x[6, 1::2] = -0.0  # equal to the zeros beside them
    check(x, rng.integers(0, V, (7, 2)), min(32, V))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=str)
@pytest.mark.parametrize("V,allowed", [(1000, 1), (1000, 5), (50280, 3), (151936, 40)])
def test_token_scores_masked_vocabulary(V, allowed, dtype):
    """Minus infinity for all but a few tokens, fewer than the alternatives asked for in some: probabilities 0 behind them."""
    rng = np.random.default_rng([4, V])
    x = torch.full((3, V), -float("inf"), dtype=dtype, device="cuda")
    for t in range(3):
        at = rng.permutation(V)[:allowed]
        x[t, torch.from_numpy(at).cuda()] = torch.from_numpy(rng.standard_normal(allowed)).to(dtype).cuda()
    x[2, V - 1] = 1.0
    check(x, rng.integers(0, V, (3, 3)), 8)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=str)
def test_token_scores_lowest_value_as_a_mask(dtype):
    rng = np.random.default_rng(5)
    x = torch.full((2, 3001), torch.finfo(dtype).min, dtype=dtype, device="cuda")
    x[0, ::100] = torch.from_numpy(rng.standard_normal(31)).to(dtype).cuda()
    tok = np.array([[0, 100], [0, 3000]])
    lp, h, top, tlp, status = run(x, tok, 4)
    want = oracle.token_scores(x.double().cpu().numpy(), tok, 4)
    assert status == 0
    np.testing.assert_array_equal(top, want[2])
    for got, ref in ((lp, want[0]), (h, want[1]), (tlp, want[3])):
        np.testing.assert_allclose(got, ref, rtol=2.0 ** -20, atol=1e-4)


@pytest.mark.parametrize("V", [40, 9001])
def test_token_scores_values_that_are_not_numbers(V):
    """NaN, plus infinity, nothing but minus infinity: NaN for the row's numbers, its order all the same; other rows as they were."""
    rng = np.random.default_rng([6, V])
    x = logits(rng, 5, V, torch.float32)
    tok = rng.integers(0, V, (5, 2))
    clean = run(x, tok, 6)
    x[1, 3], x[2, V - 2], x[3] = float("nan"), float("inf"), -float("inf")
    lp, h, top, tlp, status = run(x, tok, 6)
    want = oracle.token_scores(x.double().cpu().numpy(), tok, 6)
    assert status == 0
    np.testing.assert_array_equal(top, want[2])
    assert np.isnan(h[1:4]).all() and np.isnan(lp[1]).all() and np.isnan(lp[3]).all() and np.isnan(tlp[[1, 3]]).all()
    for got, was in zip((lp, h, top, tlp), clean):
        np.testing.assert_array_equal(got[[0, 4]], was[[0, 4]])
    x[0] = float("nan")
    x[0, 5] = 1.0
    assert run(x, tok, 6)[2][0].tolist() == [5, 0, 1, 2, 3, 4]


def test_token_scores_far_from_zero():
    """Logits around 3000 (fp32, steps of 2^-12): as exact as around 0."""
    rng = np.random.default_rng(7)
    x = logits(rng, 2, 30011, torch.float32) + 3000.0
    check(x, rng.integers(0, 30011, (2, 3)), 5)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=str)
@pytest.mark.parametrize("scale", [2.0 ** -100, 1.0, 2.0 ** 100])
def test_token_scores_as_far_from_zero_as_there_are(scale, dtype):
    """The largest and the lowest values of fp32 side by side, at any temperature: nothing that is not a number; what a log
    probability is below fp32 becomes minus infinity."""
    rng = np.random.default_rng([12, int(np.log2(scale)) + 200])
    x = torch.from_numpy(rng.choice([-3e38, -1e38, -1.0, 0.0, 2.0, 1e38], (4, 9001))).to(dtype).cuda()
    x[0, ::1000], x[1] = 3e38, -3e38
    x[1, 5], x[2, 7], x[3] = -1e38, 2e38, 1e30
    x[3, 9:] = -1e30
    tok = rng.integers(0, 9001, (4, 3))
    tok[:, 0] = 5
    lp, h, top, tlp, status = run(x, tok, 6, scale)
    want = oracle.token_scores(x.double().cpu().numpy(), tok, 6, scale)
    low = lambda v: np.where(v < -float(np.finfo(np.float32).max), -np.inf, v)  # noqa: E731
    E = (9001 / 512 + 64) * 2.0 ** -24 + (np.log(9001) + 32) * 2.0 ** -22 + 2.0 ** -20
    assert status == 0
    np.testing.assert_array_equal(top, want[2])
    for got, ref, e in ((lp, low(want[0]), E), (tlp, low(want[3]), E), (h, want[1], E * (1 + np.log(9001)))):
        np.testing.assert_allclose(got, ref, rtol=2.0 ** -22, atol=e)


def test_token_scores_bad_tokens():
    from speculative_decoding_mamba2_gb300 import SSM_STATUS_TOKEN_RANGE
    rng = np.random.default_rng(8)
    check(logits(rng, 2, 99, torch.float32), np.array([[0, 99, -1], [-2, 98, 1 << 30]]), 1, bad=SSM_STATUS_TOKEN_RANGE)


def test_token_scores_parts_alone():
    """Tokens, entropy and alternatives asked for one by one: as together, and what is not asked for stays."""
    from speculative_decoding_mamba2_gb300 import ssm_token_scores
    rng = np.random.default_rng(9)
    x, tok = logits(rng, 6, 20001, torch.bfloat16), rng.integers(0, 20001, (6, 2))
    lp, h, top, tlp, _ = run(x, tok, 4)
    lp1, h1 = torch.empty(6, 2, device="cuda"), torch.empty(6, device="cuda")
    top1 = torch.empty(6, 4, dtype=torch.int32, device="cuda")
    ssm_token_scores(x, ints(tok), lp1, None, None)
    ssm_token_scores(x, None, None, h1, None)
    ssm_token_scores(x, None, None, None, top1)
    np.testing.assert_array_equal(host(lp1), lp)
    np.testing.assert_array_equal(host(h1), h)
    np.testing.assert_array_equal(top1.cpu().numpy(), top)


def test_token_scores_another_stream_and_again():
    rng = np.random.default_rng(10)
    x, tok = logits(rng, 9, 60001, torch.float32), rng.integers(0, 60001, (9, 2))
    first = run(x, tok, 12)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for s in (None, side, None):
        for a, b in zip(run(x, tok, 12, stream=s), first):
            np.testing.assert_array_equal(a, b)


def test_token_scores_past_32_bit_offsets():
    rng = np.random.default_rng(11)
    ld = (1 << 31) + 64
    buf = torch.empty(3, ld, dtype=torch.bfloat16, device="cuda")
    buf[:, :5000] = torch.from_numpy(rng.standard_normal((3, 5000))).cuda()
    check(buf[:, :5000], rng.integers(0, 5000, (3, 2)), 3)


def test_token_scores_none():
    assert run(torch.empty(0, 50, device="cuda"), np.zeros((0, 2), int), 3)[4] == 0


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=str)
@pytest.mark.parametrize("scale", [2.0 ** -100, 2.0 ** -60, 0.5, 1.0, 5.0, 2.0 ** 100])
def test_token_scores_largest_logit_near_a_mask(scale, dtype):
    """Rows whose largest logits, far inside the row, are -1e38 over max(1, scale log2 e), with the lower half of its bits cleared, a step
    or a few either side of it, or half of it, beside minus infinity and -3e38: those below count as little as they should."""
    V = 9001
    c = np.float32(scale) * np.float32(1.4426950408889634)
    low = (np.float32(-1e38) / np.maximum(c, np.float32(1))).reshape(1).view(np.uint32) & np.uint32(0xFFFF0000)
    unit = 1 if dtype == torch.float32 else 1 << 16
    steps = [-2 * unit, -unit, 0, unit, 2 * unit, 1 << 16, -(1 << 23), -(1 << 23) - unit, unit - (1 << 23)]  # (2^23: a factor of two)
    x = np.full((2 * len(steps), V), -np.inf, np.float32)
    for i, step in enumerate(steps):
        top = (low.astype(np.int64) + step).astype(np.uint32).view(np.float32)[0]
        x[2 * i:2 * i + 2, 4000:4011] = top
        x[2 * i + 1, ::2] = np.minimum(x[2 * i + 1, ::2], np.float32(-3e38))
        x[2 * i + 1, 1::2] = np.maximum(x[2 * i + 1, 1::2], np.where(top < -3e38, -np.inf, np.float32(-3e38)))
    x = torch.from_numpy(x).to(dtype).cuda()
    tok = np.tile([4000, 1, 4010], (2 * len(steps), 1))
    lp, h, top, tlp, status = run(x, tok, 12, scale)
    want = oracle.token_scores(x.double().cpu().numpy(), tok, 12, scale)
    far = lambda v: np.where(v < -float(np.finfo(np.float32).max), -np.inf, v)  # noqa: E731
    E = (V / 512 + 64) * 2.0 ** -24 + (np.log(V) + 32) * 2.0 ** -22 + 2.0 ** -20
    assert status == 0
    np.testing.assert_array_equal(top, want[2])
    for got, ref, e in ((lp, far(want[0]), E), (tlp, far(want[3]), E), (h, want[1], E * (1 + np.log(V)))):
        np.testing.assert_allclose(got, ref, rtol=2.0 ** -22, atol=e)
