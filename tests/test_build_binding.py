"""When the torch binding is built: not without torch, and again for another torch or Python."""
import os

import pytest

from auto_regressive_decode_b200 import build


@pytest.fixture
def fake(tmp_path, monkeypatch):
    """A binding and its note in a folder of their own; the compiler's calls are written down."""
    calls = []

    def run_into(target, cmd):
        calls.append(target)
        with open(target, "w"):
            pass
    monkeypatch.setattr(build, "BIND", str(tmp_path / "_mk_torch.so"))
    monkeypatch.setattr(build, "BIND_FOR", str(tmp_path / "_mk_torch.so.for"))
    monkeypatch.setattr(build, "_run_into", run_into)
    return calls


def test_built_once(fake):
    assert build.build_binding() == build.BIND and fake == [build.BIND]
    assert build.build_binding() == build.BIND and len(fake) == 1
    build.build_binding(force=True)
    assert len(fake) == 2


@pytest.mark.parametrize("note", ["torch 1.0, Python 3.12.3\n", "", None])
def test_built_again_for_another_torch(fake, note):
    build.build_binding()
    if note is None:
        os.remove(build.BIND_FOR)
    else:
        with open(build.BIND_FOR, "w") as f:
            f.write(note)
    assert build.binding_stale()
    build.build_binding()
    assert len(fake) == 2 and not build.binding_stale()


def test_the_c_abi_is_built_without_torch(fake, monkeypatch):
    find = build.importlib.util.find_spec
    monkeypatch.setattr(build.importlib.util, "find_spec", lambda name, *a: None if name == "torch" else find(name, *a))
    monkeypatch.setattr(build, "stale", lambda: False)
    assert build.build() == build.LIB and fake == []
    assert build.build_binding() is None and not os.path.exists(build.BIND)
