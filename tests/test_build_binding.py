"""The compiled Python calls are rebuilt for another torch, and a module that could
not be rebuilt is not left for the new library."""
import os

import pytest

from weight_rnn_gb300 import build as wbuild


@pytest.fixture
def module(tmp_path, monkeypatch):
    """a module that was built before, newer than its sources"""
    wbuild.build()
    path = tmp_path / "_fast.so"
    path.write_bytes(b"old")
    made = []
    monkeypatch.setattr(wbuild, "BINDING", str(path))
    monkeypatch.setattr(wbuild, "_binding_note", lambda: str(tmp_path / "note"), raising=False)
    monkeypatch.setattr(wbuild, "binding_command", lambda obj: made.append(obj) or ["true"])
    monkeypatch.setattr(wbuild, "link_binding", lambda obj: path.write_bytes(b"new"))
    return path, made, monkeypatch


def note(text):
    with open(wbuild._binding_note(), "w") as f:
        f.write(text)


def test_kept_while_nothing_changed(module):
    path, made, _ = module
    note(wbuild.binding_made_with())
    wbuild.build()
    assert not made and path.read_bytes() == b"old"


def test_rebuilt_for_another_torch(module):
    path, made, monkeypatch = module
    note(wbuild.binding_made_with())
    monkeypatch.setattr(wbuild, "binding_made_with", lambda: "torch 0.0")
    wbuild.build()
    assert made and path.read_bytes() == b"new"


@pytest.mark.parametrize("how", ["compile", "link", "nothing to compile with"])
def test_not_left_behind(module, how, capfd):
    path, _, monkeypatch = module
    os.utime(path, (1, 1))  # older than its sources
    if how == "compile":
        monkeypatch.setattr(wbuild, "binding_command", lambda obj: ["false"])
    elif how == "link":
        def fails(obj):
            raise RuntimeError("link")
        monkeypatch.setattr(wbuild, "link_binding", fails)
    else:
        monkeypatch.setattr(wbuild, "binding_command", lambda obj: None)
    wbuild.build()
    assert not path.exists()
