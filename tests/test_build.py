"""What the build makes where torch is missing or another one, with compilers
that only write their output files."""
import os
import types

import pytest

from bitonic_networks_gb300 import build as b


@pytest.fixture
def tree(tmp_path, monkeypatch):
    """Outputs below tmp_path, no compiler; `torch(n)` installs the n-th torch, or none."""
    for name, file in (("PKG", ""), ("BUILD_DIR", "_build"), ("LIB_PATH", "libgsort.so"), ("OPS_PATH", "_ops.so"),
                       ("OPS_STAMP", "_build/ops.stamp")):
        monkeypatch.setattr(b, name, str(tmp_path / file), raising=False)

    def run(cmd, what):
        with open(cmd[cmd.index("-o") + 1], "w"):
            return types.SimpleNamespace(stdout="", stderr="")

    def torch(n):
        spec = None
        if n is not None:
            home = tmp_path / f"torch{n}"
            home.mkdir(exist_ok=True)
            (home / "version.py").write_text(f"__version__ = '2.{n}'\n")
            spec = types.SimpleNamespace(submodule_search_locations=[str(home)])
        monkeypatch.setattr(b.importlib.util, "find_spec", lambda name: spec)

    monkeypatch.setattr(b, "_run", run)
    monkeypatch.setattr(b, "nvcc", lambda: os.path.join("cuda", "bin", "nvcc"))
    torch(9)
    return torch


def test_both_are_built_and_then_up_to_date(tree):
    assert not b.up_to_date()
    assert b.build() == b.LIB_PATH and os.path.exists(b.LIB_PATH) and os.path.exists(b.OPS_PATH)
    assert b.up_to_date()


def test_the_library_is_linked_without_torch(tree):
    tree(None)
    with pytest.raises(RuntimeError, match="torch"):
        b.build()
    assert os.path.exists(b.LIB_PATH) and not os.path.exists(b.OPS_PATH)


def test_the_library_is_linked_without_a_host_compiler(tree, monkeypatch):
    run = b._run

    def no_gxx(cmd, what):
        if cmd[0] == "g++":
            raise FileNotFoundError("g++")
        return run(cmd, what)

    monkeypatch.setattr(b, "_run", no_gxx)
    with pytest.raises(FileNotFoundError):
        b.build()
    assert os.path.exists(b.LIB_PATH)


def test_a_stale_library_is_linked_after_torch_has_gone(tree):
    b.build()
    os.utime(b.LIB_PATH, (0, 0))
    tree(None)
    with pytest.raises(RuntimeError, match="torch"):
        b.build()
    assert os.path.getmtime(b.LIB_PATH) > 0


def test_a_module_for_another_torch_is_not_up_to_date(tree):
    b.build()
    assert b.up_to_date()
    tree(11)
    assert not b.up_to_date()
    b.build()
    assert b.up_to_date()
