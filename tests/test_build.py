"""What the in-tree build makes, with the compilers replaced by a recorder (no GPU, nothing is compiled)."""
import importlib.util
import os
import subprocess

import pytest


@pytest.fixture
def build(tmp_path, monkeypatch):
    import __graft_entry__
    mod = __graft_entry__._load_build_module()
    for name in ("LIB", "OPS", "BUILD"):
        monkeypatch.setattr(mod, name, str(tmp_path / os.path.basename(getattr(mod, name))))
    commands = []

    def record(cmd, **_):
        commands.append(cmd)
        with open(cmd[cmd.index("-o") + 1], "w"):
            pass
        return subprocess.CompletedProcess(cmd, 0, "", "")

    monkeypatch.setattr(mod.subprocess, "run", record)
    monkeypatch.setattr(mod, "_nvcc", lambda: "/usr/local/cuda/bin/nvcc")
    return mod, commands


def test_the_library_builds_without_torch(build, monkeypatch):
    mod, commands = build
    find = importlib.util.find_spec
    monkeypatch.setattr(importlib.util, "find_spec", lambda name, *a: None if name == "torch" else find(name, *a))
    assert mod.build() == mod.LIB and os.path.exists(mod.LIB) and not os.path.exists(mod.OPS)
    sources = [os.path.basename(c[c.index("-c") + 1]) for c in commands if "-c" in c]
    assert sorted(sources) == sorted(mod.CUDA_SOURCES + mod.CXX_SOURCES)
    n = len(commands)
    mod.build()
    assert len(commands) == n                     # up to date without the module


def test_a_torch_without_cuda_counts_as_none(build, monkeypatch, tmp_path):
    mod, _ = build
    spec = importlib.util.spec_from_file_location("torch", tmp_path / "torch" / "__init__.py", submodule_search_locations=[str(tmp_path / "torch")])
    monkeypatch.setattr(importlib.util, "find_spec", lambda name, *a: spec)
    mod.build()
    assert os.path.exists(mod.LIB) and not os.path.exists(mod.OPS)


def test_the_module_is_built_beside_the_library_where_torch_is(build):
    mod, commands = build
    mod.build()
    assert os.path.exists(mod.LIB) and os.path.exists(mod.OPS)
    made = [c[c.index("-o") + 1] for c in commands]
    assert made.index(next(p for p in made if p.startswith(mod.LIB))) < made.index(next(p for p in made if p.startswith(mod.OPS)))
