"""The drafts' operators together, as a step of a hybrid model uses them."""
import pytest

from examples import serve_drafts

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n,largest,seed", [(3, 8, 0), (1, 1, 1), (5, 20, 2)])
def test_drafts_equal_single_decoding(n, largest, seed):
    """The drafted path rounds q, k and v of the GDN layer to fp16 where the one-token path does not, 2^-11 of each: the
    state, a sum of their products, may be off by 2^-9 with the errors of the steps before.  Downstream a number may
    then fall on the other side of a rounding to bf16 (q, k, v and o of the attention): a step of 2^-8 each, 2^-7 of y
    and, at its weight of a half, 2^-8 of x.  The logits have a standard deviation of 3, so the largest of their
    changes (3 deviations), which is the relative change of a probability, is at most 9 * 2^-8."""
    p, state, rate = serve_drafts.serve(n=n, rounds=3, largest=largest, seed=seed)
    assert p <= 9 * 2.0 ** -8 and state <= 2.0 ** -9 and 1 <= rate <= largest
