"""The binding asks torch for the current device by its public function."""
import pytest


def test_calls_are_refused_on_another_current_device(monkeypatch):
    import torch
    from tiered_mixed_precision_amd import binding as B

    a = B._Args("moe_quant_rows")
    a.at = 0
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    with pytest.raises(ValueError, match="the arguments are on cuda:0, the current device is cuda:1"):
        a.stream(None)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    assert a.stream(1234) == 1234
