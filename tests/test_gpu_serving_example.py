"""The serving example: rotary positions, the cache and its attention together, beside the prefill.

Two computations of one value are compared, by the relative L2 difference of a token's heads (of the whole
extension).  Each rounds its probabilities (bf16, or fp16 over 8-bit codes) and its output (bf16) by at most
2^-8 of the value, independently, with a root mean square of a third of that or so: 4e-3 each, 8e-3 together.
The extension's prefill sees an 8-bit cache's keys and values rounded to bf16 once more: the scores (of
deviation 1) move by about 2^-9, and so the probabilities, and the values by as much: 4e-3 more.
"""
import pytest

from examples import serve_attention

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", ["bf16", "i8", "e4m3"])
@pytest.mark.parametrize("sizes", [dict(), dict(prompts=(130, 1), nodes=30, extension=64, hq=8, hkv=2, d=128, rot=128, page=16),
                                   dict(prompts=(65, 64, 63, 200), nodes=3, rounds=4, extension=1, hq=4, hkv=4, d=64, rot=32, page=32)])
def test_serving_one_layer(kind, sizes):
    tree, extension = serve_attention.serve(kind, **sizes)
    assert tree <= 8e-3
    assert extension <= (8e-3 if kind == "bf16" else 1.2e-2)
