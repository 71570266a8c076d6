"""What a build makes, and when it makes it again, with stand-ins for the sources."""
import os
import shutil

import pytest


@pytest.fixture
def tree(tmp_path, monkeypatch):
    """The build module on a source tree of its own: one unit, a binding, a header folder."""
    from memory_hierarchy_reuse_gb300 import build as b

    csrc, include = tmp_path / "csrc", tmp_path / "include"
    csrc.mkdir()
    include.mkdir()
    (csrc / "unit.cu").write_text('extern "C" int unit() { return 7; }\n')
    (csrc / "torch_binding.cpp").write_text("// a binding\n")
    for name, value in [("CSRC", csrc), ("INCLUDE", include), ("BUILD_DIR", tmp_path / "objects"),
                        ("LIB", tmp_path / "lib.so"), ("BINDING", tmp_path / "binding.so"),
                        ("BINDING_SOURCE", csrc / "torch_binding.cpp")]:
        monkeypatch.setattr(b, name, str(value))
    monkeypatch.setattr(b, "SOURCES", ["unit.cu"])
    return b


def fake_binding(b, monkeypatch, made):
    def make():
        made.append(1)
        with open(b.BINDING, "w") as f:
            f.write("binding")

    monkeypatch.setattr(b, "_build_binding", make)


def test_library_does_not_need_torch(tree, monkeypatch):
    """The C library is whole without torch; only the binding is left out."""
    monkeypatch.setattr(tree, "_torch_root", lambda: None)
    assert tree.build() == tree.LIB and os.path.exists(tree.LIB) and not os.path.exists(tree.BINDING)
    built = os.path.getmtime(tree.LIB)
    assert tree.build() == tree.LIB and os.path.getmtime(tree.LIB) == built  # nothing is stale


def test_library_is_there_when_the_binding_does_not_compile(tree):
    """A binding that fails is an error, after the library has been linked."""
    with open(tree.BINDING_SOURCE, "w") as f:
        f.write("#error no binding\n")
    with pytest.raises(RuntimeError, match="torch_binding"):
        tree.build()
    assert os.path.exists(tree.LIB) and not os.path.exists(tree.BINDING)


def test_each_part_is_made_again_for_its_own_reasons(tree, monkeypatch):
    made = []
    fake_binding(tree, monkeypatch, made)
    tree.build()
    assert len(made) == 1
    tree.build()
    assert len(made) == 1
    library = os.stat(tree.LIB).st_mtime_ns
    later = os.stat(tree.BINDING).st_mtime + 10
    os.utime(tree.BINDING_SOURCE, (later, later))  # the binding's source
    tree.build()
    assert len(made) == 2 and os.stat(tree.LIB).st_mtime_ns == library


def test_another_torch_makes_the_binding_again(tree, monkeypatch, tmp_path):
    """An upgraded torch, or another installation of it, leaves no binding of the old one."""
    made = []
    fake_binding(tree, monkeypatch, made)
    root = tmp_path / "torch"
    root.mkdir()
    (root / "version.py").write_text('__version__ = "1"\n')
    monkeypatch.setattr(tree, "_torch_root", lambda: str(root))
    tree.build()
    tree.build()
    assert len(made) == 1
    library = os.stat(tree.LIB).st_mtime_ns
    (root / "version.py").write_text('__version__ = "2"\n')
    tree.build()
    tree.build()
    assert len(made) == 2
    shutil.copytree(root, tmp_path / "other")
    monkeypatch.setattr(tree, "_torch_root", lambda: str(tmp_path / "other"))
    tree.build()
    assert len(made) == 3 and os.stat(tree.LIB).st_mtime_ns == library
