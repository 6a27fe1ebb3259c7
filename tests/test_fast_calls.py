"""What the binding makes of its extension's answers (no GPU: the extension is a stand-in, or is handed nothing it takes)."""
import os

import pytest

import replayssm_persistent_rssm_amd as rp
import replayssm_persistent_rssm_amd._binding as b

CALLS = {"page_fork": lambda: rp.rssm_page_fork(None, None, None, None, None, None, None, page_size=16, page_bytes=1024),
         "page_compact": lambda: rp.rssm_page_compact(None, None, None, None, None, page_size=16, page_bytes=1024)}


class StandIn:
    def __init__(self, answer):
        self.answer, self.calls = answer, []

    def __getattr__(self, name):
        return lambda *args: self.calls.append(name) or self.answer


@pytest.mark.parametrize("name", CALLS)
def test_a_failed_launch_is_the_library_s_error(monkeypatch, name):
    """With its status, as every other error, and the call is not made again."""
    mod = StandIn(rp.RSSM_ERR_HIP)
    monkeypatch.setattr(b, "_fast", lambda: (mod, lambda: 0, lambda i: 0))
    monkeypatch.setattr(b, "_launch", lambda *a: pytest.fail("made again"))
    monkeypatch.setattr(b, "rssm_last_error", lambda: "launch of it failed")
    with pytest.raises(rp.RssmError, match="launch of it failed") as e:
        CALLS[name]()
    assert e.value.status == rp.RSSM_ERR_HIP and mod.calls == [name]


@pytest.mark.parametrize("name", CALLS)
def test_the_other_answers(monkeypatch, name):
    mod = StandIn(True)
    monkeypatch.setattr(b, "_fast", lambda: (mod, lambda: 0, lambda i: 0))
    CALLS[name]()
    mod.answer = False                       # the binding's own checks name what is wrong
    with pytest.raises((TypeError, ValueError, AttributeError)):
        CALLS[name]()
    assert mod.calls == [name, name]


def test_the_extension_raises_nothing_itself():
    """It takes or leaves a call, or hands on a status."""
    text = open(os.path.join(os.path.dirname(b.__file__), "csrc", "fast_calls.cpp")).read()
    assert "PyErr_Set" not in text and "return nullptr;" not in text
    mod = b._fast()[0]
    for name in ("page_fork", "page_compact", "page_extend", "causal_conv", "selective_scan", "rotary_append"):
        assert getattr(mod, name)(0, 0, *[None] * 13) is False
