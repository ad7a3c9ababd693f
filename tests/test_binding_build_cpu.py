"""CPU checks of the compiled part of the binding: one that does not fit is not
used.  A build that fails leaves none behind, another version of PyTorch asks
for a new one, and a module that was built for other argument structures or
another PyTorch is left alone."""

import os
import struct
import subprocess
import sys
import types

import pytest
import torch

import linear_attention_speculative_kda_gb300 as package
from linear_attention_speculative_kda_gb300 import api
from linear_attention_speculative_kda_gb300 import build as kbuild


@pytest.fixture()
def place(monkeypatch, tmp_path):
    """A build whose library is there and whose binding goes to tmp_path."""
    library, binding = tmp_path / "libkda.so", tmp_path / "_binding.so"
    library.write_bytes(b"library")
    monkeypatch.setattr(kbuild, "LIBRARY", str(library))
    monkeypatch.setattr(kbuild, "BINDING", str(binding))
    monkeypatch.setattr(kbuild, "_stale", lambda: False)
    monkeypatch.setattr(kbuild, "_build_library", lambda verbose: None)
    return binding


def _writes(text):
    return lambda output: [sys.executable, "-c", f"open({output!r}, 'w').write({text!r})"]


def test_a_failed_build_leaves_no_old_module(monkeypatch, place, capsys):
    monkeypatch.setattr(kbuild, "binding_command", _writes("new"))
    kbuild.build()
    assert place.read_text() == "new"
    monkeypatch.setattr(kbuild, "binding_command",
                        lambda output: [sys.executable, "-c", "raise SystemExit('no headers')"])
    kbuild.build(force=False)
    assert place.read_text() == "new"              # it is not older than its sources
    os.utime(place, (0, 0))
    kbuild.build()
    assert not place.exists() and "no headers" in capsys.readouterr().err


@pytest.mark.parametrize("error", [ImportError("no torch"), FileNotFoundError("no g++"),
                                   subprocess.SubprocessError("killed")])
def test_what_is_not_installed_is_no_error(monkeypatch, place, capsys, error):
    place.write_text("old")
    os.utime(place, (0, 0))

    def command(output):
        raise error
    monkeypatch.setattr(kbuild, "binding_command", command)
    assert kbuild.build() == kbuild.LIBRARY
    assert not place.exists() and str(error) in capsys.readouterr().err


def test_a_compiler_that_is_not_there(monkeypatch, place, capsys):
    monkeypatch.setattr(kbuild, "binding_command", lambda output: ["/nonexistent/g++", output])
    assert kbuild.build() == kbuild.LIBRARY
    assert not place.exists() and "nonexistent" in capsys.readouterr().err


def test_another_pytorch_asks_for_a_new_module(monkeypatch, place):
    monkeypatch.setattr(kbuild, "binding_command", _writes("first"))
    kbuild.build()
    monkeypatch.setattr(kbuild, "binding_command", _writes("second"))
    kbuild.build()
    assert place.read_text() == "first"
    monkeypatch.setattr(torch, "__version__", torch.__version__ + ".other")
    kbuild.build()
    assert place.read_text() == "second"
    monkeypatch.setattr(kbuild, "binding_command", _writes("third"))
    kbuild.build(force=True)
    assert place.read_text() == "third"


def _module(version=None, sizes=None):
    m = types.ModuleType("_binding")
    m.torch_version = torch.__version__ if version is None else version
    m.argument_sizes = tuple(struct.calcsize(f) for f in (
        "=9if6qQqiiiiQQ8Q2i2Q", "=9if6qQqiiiiQQ4Q2i6Q", "=Qq4i8Q")) if sizes is None else sizes
    return m


@pytest.mark.parametrize("module,fits", [
    (_module(), True),
    (_module(version="1.0"), False),
    (_module(sizes=(1, 2, 3)), False),
    (types.ModuleType("_binding"), False)])          # one from before they were recorded
def test_only_a_module_that_fits_is_used(monkeypatch, module, fits):
    monkeypatch.setitem(sys.modules, package.__name__ + "._binding", module)
    monkeypatch.setattr(package, "_binding", module, raising=False)
    monkeypatch.setattr(api, "_quick", None)
    api._load_quick()
    assert api._quick is (module if fits else None)


def test_the_built_module_says_what_it_was_built_for():
    kbuild.build()
    binding = pytest.importorskip(package.__name__ + "._binding")
    assert binding.torch_version == torch.__version__
    assert binding.argument_sizes == _module().argument_sizes
