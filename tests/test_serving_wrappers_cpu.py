"""What the serving wrappers refuse before a call: memory that is not the device's.

There is no GPU here: the device's tensors are fake ones (shapes, strides and devices without memory), and a call
that gets through is caught before the library.
"""
import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode

from hybrid_gated_deltanet_q4k_gb300 import api
from hybrid_gated_deltanet_q4k_gb300 import lib as gl


class Passed(Exception):
    pass


class NoLib:
    def __getattr__(self, name):
        def call(*args, **kw):
            raise Passed(name)
        return call


@pytest.fixture
def fake(monkeypatch):
    monkeypatch.setattr(gl, "ptr", lambda t: 0)
    monkeypatch.setattr(gl, "stream_handle", lambda stream=None: 0)
    gl.load(build=True)
    with FakeTensorMode(allow_non_fake_inputs=True):
        yield


def _new(shape, dtype=torch.bfloat16, device="cuda"):
    return torch.empty(shape, dtype=dtype, device=device)


def _cache(kind="i8"):
    c = api.KvCache.new(kind, 4, 2, 16, 64)
    c.lib = NoLib()
    return c


def test_a_cache_lies_on_one_device(fake):
    k, s = _new((4, 2, 16, 64), torch.int8), _new((4, 2, 16), torch.float32)
    hk, hs = _new((4, 2, 16, 64), torch.int8, "cpu"), _new((4, 2, 16), torch.float32, "cpu")
    other = _new((4, 2, 16), torch.float32, "cuda:1")
    api.KvCache("i8", k, k, s, s)
    for parts in [(hk, hk, hs, hs), (hk, k, s, s), (k, hk, s, s), (k, k, hs, s), (k, k, s, hs), (k, k, s, other)]:
        with pytest.raises(ValueError, match="device"):
            api.KvCache("i8", *parts)
    with pytest.raises(ValueError, match="device"):
        api.KvCache.new("bf16", 4, 2, 16, 64, device="cpu")


ATTEND = dict(q=((3, 4, 64), torch.bfloat16), lens=((2,), torch.int32), block_table=((2, 5), torch.int32),
              o=((3, 4, 64), torch.bfloat16), workspace=((1 << 20,), torch.uint8), cu_q=((3,), torch.int32),
              tree=((3,), torch.int64))


def test_attend_takes_the_device_s_tensors_alone(fake):
    c = _cache()
    ok = {name: _new(*a) for name, a in ATTEND.items()}
    with pytest.raises(Passed, match="gdn_attn_cache"):
        c.attend(**ok, max_q=2)
    for name, a in ATTEND.items():
        for device in ("cpu", "cuda:1"):
            with pytest.raises(ValueError, match=name):
                c.attend(**{**ok, name: _new(*a, device=device)}, max_q=2)
    with pytest.raises(ValueError, match="workspace"):
        c.attend(**{**ok, "workspace": _new((1,), torch.uint8).expand(1 << 20)}, max_q=2)


@pytest.mark.parametrize("call", ["write", "read"])
def test_store_and_fetch_take_the_device_s_tensors_alone(fake, call):
    c = _cache()
    ok = dict(k=_new((3, 2, 64)), v=_new((3, 2, 64)), slots=_new((3,), torch.int64))
    if call == "write":
        ok["rows"] = _new((3,), torch.int32)
    with pytest.raises(Passed, match="gdn_kv"):
        getattr(c, call)(**ok)
    for name, t in ok.items():
        for device in ("cpu", "cuda:1"):
            with pytest.raises(ValueError, match=name):
                getattr(c, call)(**{**ok, name: _new(tuple(t.shape), t.dtype, device)})


def test_rope_takes_the_device_s_tensors_alone(fake):
    r = api.RopeTable(32)
    r.lib = NoLib()
    ok = dict(positions=_new((3,), torch.int32), q=_new((3, 4, 64)), k=_new((3, 2, 64)), q_out=_new((3, 4, 64)), k_out=_new((3, 2, 64)))
    with pytest.raises(Passed, match="gdn_rope"):
        r.apply(**ok)
    for name, t in ok.items():
        for device in ("cpu", "cuda:1"):
            with pytest.raises(ValueError):
                r.apply(**{**ok, name: _new(tuple(t.shape), t.dtype, device)})


@pytest.mark.parametrize("first,n", [(-1, 1), (-16, 4), (0, 81), (80, 1), (70, 11), (3, -1)])
def test_slots_outside_the_pages_are_refused(fake, first, n):
    """An index past the table would be a failed assertion on the device, and one below zero another token's slot."""
    c = _cache()
    with pytest.raises(ValueError, match="pages"):
        c.slots(_new((5,), torch.int32), first, n)


@pytest.mark.parametrize("first,n", [(0, 0), (80, 0), (0, 80), (15, 18), (79, 1)])
def test_slots_inside_the_pages(first, n):
    c = object.__new__(api.KvCache)
    c.page_tokens = 16
    pages = torch.tensor([7, 2, -1, 0, 9], dtype=torch.int32)
    want = [int(pages[t // 16]) * 16 + t % 16 for t in range(first, first + n)]
    assert c.slots(pages, first, n).tolist() == want and c.slots(pages, first, n).dtype is torch.int64


def test_the_contract_asks_for_distinct_slots():
    """Nothing orders two writers of one slot, so no text may promise that one of them wins."""
    import os
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    header = " ".join(open(os.path.join(root, "include", "gdn.h")).read().replace(" * ", " ").split())
    assert "hold one of the tokens" not in header
    assert "The slots of a call that are not negative must differ" in header
    assert "no slot twice" in " ".join(api.KvCache.write.__doc__.split())
