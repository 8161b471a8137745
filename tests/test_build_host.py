"""CPU tests of the build step's order: both libraries are made before either
takes its place, and the one that needs torch is left out where there is none.
The compilers are stand-ins."""
import importlib.util
import os
import subprocess

import pytest

import zero_sharded_optimizer_sm_b200 as z


@pytest.fixture
def step(tmp_path, monkeypatch):
    """The build step over a folder of its own, with old libraries in place."""
    path = os.path.join(os.path.dirname(z.__file__), "build.py")
    spec = importlib.util.spec_from_file_location("build_step", path)
    step = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(step)
    for name, value in dict(HERE=str(tmp_path), LIB=str(tmp_path / "libzero_sm.so"), CALLS=str(tmp_path / "_calls.so"),
                            SOURCES=["csrc/a.cu", "csrc/b.cpp"]).items():
        monkeypatch.setattr(step, name, value)
    for name in ("libzero_sm.so", "_calls.so"):
        (tmp_path / name).write_text("old")
    step.failing, step.folder, step.ran = None, tmp_path, []

    def run(cmd, **kw):
        tool = os.path.basename(cmd[0]) + (" link" if "-shared" in cmd else "")
        step.ran.append(tool)
        if tool == step.failing:
            if kw.get("check"):
                raise subprocess.CalledProcessError(1, cmd)
            return subprocess.CompletedProcess(cmd, 1, "", "")
        with open(cmd[cmd.index("-o") + 1], "w") as f:
            f.write("new")
        return subprocess.CompletedProcess(cmd, 0, "", "")

    monkeypatch.setattr(step.subprocess, "run", run)
    return step


def _held(step):
    return {n: (step.folder / n).read_text() for n in ("libzero_sm.so", "_calls.so") if (step.folder / n).exists()}


def test_both_are_replaced(step):
    assert step.build() == step.LIB
    assert _held(step) == {"libzero_sm.so": "new", "_calls.so": "new"}
    assert step.ran[-2:] == ["nvcc link", "g++ link"]


@pytest.mark.parametrize("failing", ["nvcc", "nvcc link", "g++ link"])
def test_a_step_that_fails_leaves_both_as_they_were(step, failing):
    step.failing = failing
    with pytest.raises(subprocess.CalledProcessError):
        step.build()
    assert _held(step) == {"libzero_sm.so": "old", "_calls.so": "old"}


def test_without_torch_there_is_the_library_alone(step, monkeypatch, capsys):
    """Calls that were made for an older library do not stay beside the new one."""
    find = importlib.util.find_spec
    monkeypatch.setattr(importlib.util, "find_spec", lambda name, *a: None if name == "torch" else find(name, *a))
    assert step.build() == step.LIB
    assert _held(step) == {"libzero_sm.so": "new"}
    assert "torch" in capsys.readouterr().out
    step.build()  # nor are they missed
    assert _held(step) == {"libzero_sm.so": "new"}
