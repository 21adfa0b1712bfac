"""What build() does where a part cannot be compiled, with the compilers replaced."""
import os

import pytest

from attention_relation_kl_b200 import build as b


@pytest.fixture
def compilers(monkeypatch, tmp_path):
    """The outputs in a folder of their own; commands are recorded and write their output."""
    ran, broken = [], set()

    def run(cmd, verbose):
        name = os.path.basename(cmd[0])
        if name in broken:
            raise RuntimeError(f"{name} failed")
        ran.append(name)
        with open(cmd[cmd.index("-o") + 1], "w") as f:
            f.write(name)

    monkeypatch.setattr(b, "_run", run)
    monkeypatch.setattr(b, "nvcc_path", lambda: "nvcc")
    monkeypatch.setattr(b, "LIB", str(tmp_path / "librelkl.so"))
    monkeypatch.setattr(b, "MARSHAL", str(tmp_path / "_marshal.so"))
    monkeypatch.delenv("RELKL_CHECKS", raising=False)
    return ran, broken


def test_the_library_is_built_where_the_module_cannot_be(compilers):
    ran, broken = compilers
    broken.add("g++")
    with pytest.warns(UserWarning, match="marshalling module"):
        assert b.build() == b.LIB
    assert ran == ["nvcc"] and os.path.exists(b.LIB) and not os.path.exists(b.MARSHAL)
    broken.clear()
    b.build()
    assert ran == ["nvcc", "g++"] and os.path.exists(b.MARSHAL)
    # a module that a failed build would have replaced does not stay
    broken.add("g++")
    with pytest.warns(UserWarning):
        b.build(force=True)
    assert not os.path.exists(b.MARSHAL)


def test_a_library_that_cannot_be_built_is_an_error(compilers):
    ran, broken = compilers
    broken.add("nvcc")
    with pytest.raises(RuntimeError, match="nvcc"):
        b.build()
    assert ran == []


def test_the_module_is_built_again_for_another_torch(compilers, monkeypatch):
    ran, _ = compilers
    b.build()
    b.build()
    assert ran == ["nvcc", "g++"]
    real = b.importlib.metadata.version
    monkeypatch.setattr(b.importlib.metadata, "version", lambda name: real(name) + ".other")
    b.build()
    assert ran == ["nvcc", "g++", "g++"]
    b.build()
    assert ran == ["nvcc", "g++", "g++"]
    os.remove(b.MARSHAL + ".torch")          # one that says nothing of it
    b.build()
    assert ran == ["nvcc", "g++", "g++", "g++"]
