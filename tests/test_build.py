"""The build, on sources of its own: the C library does not wait for the
binding, and each is rebuilt when what it is made of changes."""
import ctypes
import os

import pytest

from mla_paged_kv_concat_gb300 import build


@pytest.fixture
def tree(tmp_path, monkeypatch):
    """A library of one function; the binding's steps only write files."""
    src = tmp_path / "csrc"
    src.mkdir()
    (src / "one.cu").write_text('extern "C" int one() { return 1; }\n')
    (src / "bind.cpp").write_text("// binding\n")
    (tmp_path / "include").mkdir()
    names = dict(ROOT=tmp_path, CSRC=src, BUILD=tmp_path / "_build", LIB=tmp_path / "libone.so",
                 BIND=tmp_path / "_calls.so", BIND_SRC=src / "bind.cpp")
    for k, v in names.items():
        monkeypatch.setattr(build, k, str(v))
    made = []

    def compile_bind():
        made.append("bind")
        return str(tmp_path / "bind.o")

    def link_bind(obj):
        (tmp_path / "_calls.so").write_text("binding\n")

    compile_lib = build._compile
    monkeypatch.setattr(build, "_compile", lambda s: made.append("lib") or compile_lib(s))
    monkeypatch.setattr(build, "_compile_bind", compile_bind)
    monkeypatch.setattr(build, "_link_bind", link_bind)
    return tmp_path, made


def change(path):
    """Newer than everything that is there."""
    t = path.stat().st_mtime + 10
    for p in path.parent.parent.rglob("*"):
        t = max(t, p.stat().st_mtime + 10)
    os.utime(path, (t, t))


def test_library_is_linked_before_the_binding_fails(tree, monkeypatch):
    root, _ = tree

    def no_headers():
        raise RuntimeError("g++ failed: no torch headers")

    monkeypatch.setattr(build, "_compile_bind", no_headers)
    with pytest.raises(RuntimeError, match="no torch headers"):
        build.build()
    assert ctypes.CDLL(str(root / "libone.so")).one() == 1
    assert not build.up_to_date()


def test_only_what_changed_is_built(tree):
    root, made = tree
    assert build.build() == str(root / "libone.so")
    # build.py itself is older than what was just made
    assert sorted(made) == ["bind", "lib"] and build.up_to_date()
    build.build()
    assert len(made) == 2
    change(root / "csrc" / "bind.cpp")
    assert not build.up_to_date()
    build.build()
    assert made[2:] == ["bind"]


@pytest.mark.parametrize("what", ["torch", "python", "stamp"])
def test_binding_is_made_anew_for_another_torch_or_python(tree, monkeypatch, what):
    """Its file times say nothing about the versions it was compiled for."""
    root, made = tree
    build.build()
    assert build.up_to_date()
    if what == "torch":
        import importlib.metadata as md
        old = md.version
        monkeypatch.setattr(md, "version", lambda n: old(n) + ".post1")
    elif what == "python":
        monkeypatch.setattr(build.sys.implementation, "cache_tag", "cpython-999")
    else:
        for p in (root / "_build").glob("*.versions"):
            p.unlink()
    assert not build.up_to_date()
    build.build()
    assert made[2:] == ["bind"] and build.up_to_date()
