"""The current stream comes from torch's public call where its quick private one
is missing."""
import importlib.util
import sys

import pytest
import torch

import optimizer_step_gb300.embedding as embedding

pytestmark = pytest.mark.gpu


def test_the_stream_without_torchs_private_call(monkeypatch):
    monkeypatch.delattr(torch._C, "_cuda_getCurrentRawStream", raising=False)
    name = "optimizer_step_gb300.embedding_without_private_call"
    spec = importlib.util.spec_from_file_location(name, embedding.__file__)
    module = importlib.util.module_from_spec(spec)
    monkeypatch.setitem(sys.modules, name, module)
    spec.loader.exec_module(module)
    table = torch.ones(10, 8, device="cuda")
    ids = torch.arange(4, device="cuda")
    lib, seen = module._lib.load(), []
    enqueue = lib.train_embed
    monkeypatch.setattr(lib, "train_embed", lambda *a: seen.append(a[-1]) or enqueue(*a))
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        out = module.embed(table, ids, scale=2.0)
    side.synchronize()
    assert seen == [side.cuda_stream] and torch.equal(out, 2.0 * table[:4])
