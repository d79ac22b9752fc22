"""What is run where a device is present."""
from __future__ import annotations

import pathlib

import pytest
import torch

from . import conftest


class Item:
    def __init__(self, name, fixtures=(), keywords=()):
        self.path, self.fixturenames, self.keywords, self.marks = pathlib.Path(name), fixtures, set(keywords), []

    def add_marker(self, mark):
        self.marks.append(mark.name)


def skipped(monkeypatch, device: bool, *items):
    monkeypatch.setattr(torch.cuda, "is_available", lambda: device)
    conftest.pytest_collection_modifyitems(None, list(items))
    return [i.marks == ["skip"] for i in items]


@pytest.mark.parametrize("device", [False, True])
def test_addresses_of_nothing_never_meet_a_device(monkeypatch, device):
    # a call that passes the checks is launched where there is a device
    assert skipped(monkeypatch, device, Item("tests/test_q8_host.py", ("lib", "kw")),
                   Item("tests/test_q8_host.py", ("monkeypatch",)), Item("tests/test_abi_host.py", ("lib",)),
                   Item("tests/test_rope_gpu.py", (), ("gpu",))) == [device, False, False, not device]
