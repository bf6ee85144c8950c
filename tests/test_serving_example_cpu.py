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


def test_smoke_takes_both_kernels_of_the_cache_attention(monkeypatch):
    """Its trees have rows enough for the kernel for many (the threshold of the source), its single tokens do not."""
    import os
    import re

    import __graft_entry__ as entry
    calls = []
    monkeypatch.setattr(serve_attention, "serve", lambda *a, **kw: calls.append(kw) or (0.0, 0.0))
    entry._smoke_serving()
    kw = calls[0]
    nodes, least, ratio = kw.get("nodes", 12), kw.get("least", 1), kw.get("hq", 16) // kw.get("hkv", 4)
    src = os.path.join(entry.ROOT if hasattr(entry, "ROOT") else os.path.dirname(entry.__file__),
                       "hybrid_gated_deltanet_q4k_gb300", "csrc", "k_attn_cache.cu")
    many = int(re.search(r"AC_TREE_ROWS = (\d+);", open(src).read()).group(1))
    assert min(nodes, least * len(kw["prompts"])) * ratio >= many > ratio
