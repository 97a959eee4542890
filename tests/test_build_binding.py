"""Building the quick binding beside another process that does the same (CPU)."""
import multiprocessing
import os
import subprocess
import types

import pytest

from paged_kv_cache_164_gb300 import build as pkv_build


@pytest.fixture
def folder(tmp_path, monkeypatch):
    monkeypatch.setattr(pkv_build, "OUT_DIR", str(tmp_path))
    monkeypatch.setattr(pkv_build, "BINDING", str(tmp_path / "pkv_binding.so"))
    monkeypatch.setattr(pkv_build, "_binding_command", lambda: ["compiler"])
    return tmp_path


def _compiler(monkeypatch, meanwhile=lambda: None, rc=0):
    def run(cmd, **kw):
        meanwhile()
        if rc == 0:
            with open(cmd[cmd.index("-o") + 1], "w") as f:
                f.write("built")
        return types.SimpleNamespace(returncode=rc, stderr="no header")
    monkeypatch.setattr(subprocess, "run", run)


def test_a_binding_that_another_process_takes_away_does_not_stop_the_build(folder, monkeypatch):
    old = folder / "pkv_binding.so"
    exists = os.path.exists
    _compiler(monkeypatch)
    # there when this process looks, gone when it acts
    monkeypatch.setattr(os.path, "exists", lambda p: p == str(old) or exists(p))
    assert pkv_build.build_binding(force=True)
    assert old.read_text() == "built"


def test_the_last_build_stays_in_place_until_the_next_is_there(folder, monkeypatch):
    old = folder / "pkv_binding.so"
    old.write_text("before")
    seen = []
    _compiler(monkeypatch, lambda: seen.append(old.exists() and old.read_text()))
    assert pkv_build.build_binding(force=True)
    assert seen == ["before"] and old.read_text() == "built"
    assert pkv_build.build_binding() and len(seen) == 1  # up to date
    assert sorted(os.listdir(folder)) == ["pkv_binding.so", "pkv_binding.so.stamp"]


def test_a_build_that_fails_leaves_none_of_other_headers(folder, monkeypatch, capsys):
    (folder / "pkv_binding.so").write_text("before")
    _compiler(monkeypatch, rc=1)
    assert not pkv_build.build_binding(force=True)
    assert "no header" in capsys.readouterr().err
    assert "pkv_binding.so" not in os.listdir(folder)


def _build(folder, start, out):
    pkv_build.OUT_DIR = folder
    pkv_build.BINDING = os.path.join(folder, "pkv_binding.so")

    def run(cmd, **kw):
        with open(cmd[cmd.index("-o") + 1], "w") as f:
            f.write("built")
        return types.SimpleNamespace(returncode=0, stderr="")
    pkv_build._binding_command = lambda: ["compiler"]
    pkv_build.subprocess = types.SimpleNamespace(run=run)
    start.wait()
    out.put([pkv_build.build_binding(force=True) for _ in range(200)])


def test_many_builds_at_once(tmp_path):
    ctx = multiprocessing.get_context("spawn")
    start, out = ctx.Barrier(4), ctx.Queue()
    jobs = [ctx.Process(target=_build, args=(str(tmp_path), start, out)) for _ in range(4)]
    for j in jobs:
        j.start()
    results = [out.get(timeout=120) for _ in jobs]
    for j in jobs:
        j.join()
    assert all(all(r) for r in results)
    assert sorted(os.listdir(tmp_path)) == ["pkv_binding.so", "pkv_binding.so.stamp"]
