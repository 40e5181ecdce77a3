"""examples/hybrid_round.py with rotary positions and with an 8-bit cache beside them.

Rotary positions alone add a rounding of q and k to a layer, and the bar of 0.1 that the example has without them stands.  With
8 bits the rounds see a draft's own ancestors in bf16 and the single steps in e4m3, and rows that the two compute 0.9 % apart are
rounded apart: by a step (8.8 % of the value, on average over a binade) with the probability 0.9 / 8.8, so 2.8 % rms in rows that
were generated, which are up to 40 of 190.  Over K and V of a layer that is 2.8 % * sqrt(2 * 40 / 190) = 1.8 % of its output, over two
layers and with the 0.9 % of before 2.7 % of the logits' deviation (rms); 4.5 times that over some 10^4 logits is 0.12, and the
bar leaves a factor 2.  A stale scale or a lost row is a difference of order one."""
import pytest

from tests.test_gpu_hybrid import example  # noqa: F401 (a fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kw,bar", [(dict(S=2, prompt_len=150, tokens=20, rope=True), 0.1), (dict(S=1, prompt_len=1, tokens=6, Hkv=4, page=128, rope=True), 0.1),
                                    (dict(S=2, prompt_len=150, tokens=20, rope=True, fp8=True), 0.25),
                                    (dict(S=3, prompt_len=190, tokens=10, nodes=31, page=8, fp8=True), 0.25)], ids=str)
def test_rounds_equal_single_steps(example, kw, bar):  # noqa: F811
    per_round, worst = example.run(seed=5, **kw)
    assert per_round > 1.0
    assert worst < bar
