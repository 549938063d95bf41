"""Checks of the target-step calls' Python binding that need no GPU."""
import os

import pytest
import torch


@pytest.fixture(scope="module")
def dsv():
    from serving_draft_verify_gb300 import build as b
    if not os.path.exists(b.LIB):
        b.build()
    import serving_draft_verify_gb300 as m
    return m


class _Elsewhere:
    """A stand-in for a tensor on the second GPU; anything but its device is out of bounds."""

    shape = (4, 2, 16, 64)
    device = torch.device("cuda", 1)
    dtype = torch.float32

    def get_device(self):
        return 1


def test_tensors_of_another_device_are_refused(dsv, monkeypatch):
    """The library launches on the current device: tensors of another one would be read from there."""
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch.cuda, "device_count", lambda: 2)
    monkeypatch.setattr(dsv._binding, "_several", None)
    x = _Elsewhere()
    for call in (lambda: dsv.dspark_plan_rows(x, x, x, x, x, x, 16, 8), lambda: dsv.dspark_write_kv(x, x, x, x, x),
                 lambda: dsv.dspark_paged_attention(x, x, x, x, x, x, 4), lambda: dsv.dspark_adjust_logits(x)):
        with pytest.raises(ValueError, match="cuda:1, the current device is cuda:0"):
            call()
