"""How the binding finds the stream of a call: the caller's, else torch's current
one, also where torch lacks the undocumented short way to it."""

from types import SimpleNamespace

import pytest
import torch

import combine_moe_gate_gb300 as M


def test_a_given_stream_is_taken(monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_stream", lambda: pytest.fail("not asked for"))
    assert M._stream(SimpleNamespace(cuda_stream=1234)) == 1234


def test_without_the_short_way_the_documented_one_is_used(monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_stream", lambda: SimpleNamespace(cuda_stream=77))
    monkeypatch.setattr(M, "_raw_stream", None)
    assert M._stream(None) == 77


def test_the_short_way_is_asked_for_the_current_device(monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 3)
    monkeypatch.setattr(M, "_raw_stream", lambda device: 100 + device)
    assert M._stream(None) == 103


@pytest.mark.gpu
def test_both_ways_agree():
    for s in (torch.cuda.current_stream(), torch.cuda.Stream()):
        with torch.cuda.stream(s):
            assert M._stream(None) == s.cuda_stream == torch.cuda.current_stream().cuda_stream
