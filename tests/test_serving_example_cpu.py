"""The serving example's self-check: a difference that is no number is not lost."""
import math

from examples import serve_attention

NAN = float("nan")


def test_the_worst_difference_keeps_what_is_no_number():
    def worst(values):
        w = 0.0
        for v in values:
            w = serve_attention.worse(w, v)
        return w
    assert worst([1e-3, 3e-3, 2e-3]) == 3e-3 and worst([]) == 0.0
    for values in ([NAN], [NAN, 1e-3], [1e-3, NAN], [1e-3, NAN, 5.0], [math.inf, NAN, 1.0]):
        assert math.isnan(worst(values))
    assert worst([1.0, math.inf]) == math.inf
