"""What the serving example and smoke() would notice."""
import math

import pytest

from examples import serve_attention

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("call", [0, 3])
def test_a_tree_that_is_no_number_shows(monkeypatch, call):
    real, calls = serve_attention.difference, []

    def once_nan(a, b):
        calls.append(real(a, b))
        return float("nan") if len(calls) == call + 1 else calls[-1]

    monkeypatch.setattr(serve_attention, "difference", once_nan)
    tree, extension = serve_attention.serve("e4m3", prompts=(150, 33), rounds=1, extension=1, nodes=30)
    assert len(calls) > call + 2             # the extension's is the last
    assert math.isnan(tree) and math.isfinite(extension)
