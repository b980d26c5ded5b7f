"""When build() compiles again: the library and the binding are each as new as what they are made
of, also where an earlier build replaced the one and failed at the other."""
import os

import pytest

from chunked_gated_delta_gdr_gb300 import build as b


@pytest.fixture
def tree(tmp_path, monkeypatch):
    """A source tree and its two products; at(name, t) sets a file's time."""
    for d in ("csrc", "include"):
        (tmp_path / d).mkdir()
    names = {"header": "include/gdr.h", "binding source": f"csrc/{b.BINDING_SOURCE}",
             "library": "libgdr.so", "binding": "_mixer.so"}
    names.update({s: f"csrc/{s}" for s in b.SOURCES})
    monkeypatch.setattr(b, "CSRC", str(tmp_path / "csrc"))
    monkeypatch.setattr(b, "INCLUDE", str(tmp_path / "include"))
    monkeypatch.setattr(b, "LIB", str(tmp_path / names["library"]))
    monkeypatch.setattr(b, "BINDING", str(tmp_path / names["binding"]))
    late = os.path.getmtime(b.__file__) + 1000  # the build script is a dependency, too

    def at(name, t):
        f = tmp_path / names[name]
        f.touch()
        os.utime(f, (late + t, late + t))

    for n in names:
        at(n, 0)
    at("library", 10)
    at("binding", 11)
    return at


def test_products_newer_than_all_sources_are_kept(tree):
    assert not b._stale()


@pytest.mark.parametrize("changed", ["header", "binding source", b.SOURCES[0], b.SOURCES[-1]])
def test_a_changed_source_is_compiled(tree, changed):
    tree(changed, 20)
    assert b._stale()


def test_a_binding_older_than_the_header_is_compiled(tree):
    """The header changed, the library was built anew, the binding's compiler failed."""
    tree("header", 20)
    tree("library", 30)
    assert b._stale()


def test_a_missing_product_is_built(tree):
    os.remove(b.BINDING)
    assert b._stale()
