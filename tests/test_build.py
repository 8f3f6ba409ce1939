"""The quick binding is optional: what becomes of a build without it, or with one for another torch."""

import subprocess
import sys
from types import SimpleNamespace

import pytest

import paged_kv_cache_386_b200 as pkv
from paged_kv_cache_386_b200 import build


@pytest.fixture
def elsewhere(monkeypatch, tmp_path):
    """The binding's place, empty; the library counts as built."""
    build.build()
    monkeypatch.setattr(build, "BINDING", tmp_path / "_binding.so")
    return tmp_path / "_binding.so"


@pytest.mark.parametrize("command", [["false"], ["/nonexistent/compiler"]])
@pytest.mark.parametrize("force", [False, True])
def test_a_binding_that_cannot_be_built_is_a_warning(elsewhere, monkeypatch, command, force):
    monkeypatch.setattr(build, "binding_command", lambda *a: command)
    monkeypatch.setattr(build, "command", lambda **kw: ["true"])
    elsewhere.write_bytes(b"of another time")
    with pytest.warns(UserWarning, match="_binding.so was not built"):
        assert build.build(force=force) == build.LIB
    assert not elsewhere.exists()  # rather none than one that does not fit


def test_a_library_that_cannot_be_built_is_an_error(elsewhere, monkeypatch):
    monkeypatch.setattr(build, "command", lambda **kw: ["false"])
    with pytest.raises(subprocess.CalledProcessError):
        build.build(force=True)


def test_a_binding_for_another_torch_is_built_again(elsewhere, monkeypatch):
    built = []

    def command(out):
        built.append(out)
        return ["true"]

    monkeypatch.setattr(build, "binding_command", command)
    elsewhere.write_bytes(b"torch 1.0, python 2.7")
    build.build()
    assert built == [elsewhere]
    elsewhere.write_bytes(b"..." + build.binding_tag().encode() + b"\0...")
    build.build()
    assert built == [elsewhere]


@pytest.mark.parametrize("there", [None, SimpleNamespace(), SimpleNamespace(built_for="torch 1.0, python 2.7")])
def test_a_binding_for_another_torch_is_not_used(monkeypatch, there):
    build.build()
    monkeypatch.setattr(pkv, "_ext", None)
    monkeypatch.setitem(sys.modules, "paged_kv_cache_386_b200._binding", there)
    if hasattr(pkv, "_binding"):
        monkeypatch.setattr(pkv, "_binding", there)
    assert pkv._quick() is False


def test_the_built_binding_is_used(monkeypatch):
    build.build()
    monkeypatch.setattr(pkv, "_ext", None)
    assert pkv._quick() and pkv._binding.built_for == build.binding_tag()
