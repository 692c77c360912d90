"""The smoke run goes through every kind of layer once and times none."""
import pytest
import torch

import __graft_entry__
from examples import moe_layer

pytestmark = pytest.mark.gpu


def test_smoke_times_nothing(monkeypatch):
    """Each format's layer is called once: what the run launches is one pass of every operator."""
    calls = []
    plain = moe_layer.MoELayer.__call__

    def counted(self, *args, **kw):
        calls.append(self.format)
        return plain(self, *args, **kw)

    monkeypatch.setattr(moe_layer.MoELayer, "__call__", counted)
    __graft_entry__.smoke()
    torch.cuda.synchronize()
    assert sorted(calls) == ["bf16", "int8", "nvfp4"]


def test_example_times_on_request(capsys):
    small = ["--tokens", "5", "--hidden", "256", "--width", "128", "--shards", "1", "--format", "bf16"]
    moe_layer.main([*small, "--timed", "2"])
    assert "us a layer" in capsys.readouterr().out
    moe_layer.main([*small, "--timed", "0"])
    assert "us a layer" not in capsys.readouterr().out
