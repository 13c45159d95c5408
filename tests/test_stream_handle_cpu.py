"""The stream that the entry points get, on a PyTorch with and without the private
short way to its handle."""
import types

import torch

import entropy_logits_bf16_gb300 as rlk


def test_stream_with_and_without_the_private_name(monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 3)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda i: types.SimpleNamespace(cuda_stream=100 + i))
    monkeypatch.setattr(rlk, "_raw_stream", lambda i: 200 + i)
    assert (rlk._stream(torch.device("cuda")), rlk._stream(torch.device("cuda:1"))) == (203, 201)
    monkeypatch.setattr(rlk, "_raw_stream", None)
    assert (rlk._stream(torch.device("cuda")), rlk._stream(torch.device("cuda:1"))) == (103, 101)
