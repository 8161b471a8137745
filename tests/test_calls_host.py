"""CPU tests of the compiled Python calls as the shortcut that they are: the
package works without them, and with ones that do not load or were built for
another torch, by the long way."""
import os
import shutil
import subprocess
import sys

import pytest

import zero_sharded_optimizer_sm_b200 as z

NAME = "zero_sharded_optimizer_sm_b200"
SCRIPT = """
import sys, warnings
sys.path.insert(0, sys.argv[1])
import zero_sharded_optimizer_sm_b200 as z
assert z.__file__.startswith(sys.argv[1]) and z.zero_version() == 3
import torch
if sys.argv[2] == "another torch":
    torch.__version__ = "1.99.0+cu1"
x, w = torch.zeros(4, 64, dtype=torch.bfloat16), torch.ones(64, dtype=torch.bfloat16)
calls = (lambda: z.mx8_quantize(x), lambda: z.rms_norm(x, w), lambda: z.rms_norm_backward(x, x, w, w),
         lambda: z.embedding(torch.zeros(3, dtype=torch.int64), x),
         lambda: z.embedding_backward(x, torch.zeros(4, dtype=torch.int64), 9))
with warnings.catch_warnings(record=True) as said:
    warnings.simplefilter("always")
    for call in calls:  # the long way's refusals
        try:
            call()
        except ValueError:
            continue
        raise SystemExit("not refused")
    assert z._calls().mx8_dequantize(None, None) is None
said = [str(s.message) for s in said if "_calls.so" in str(s.message)]
if sys.argv[2] == "whole":
    assert not said and type(z._calls()).__name__ == "module", said
else:
    assert len(said) == 1 and "build" in said[0], said
print("fine")
"""


@pytest.mark.parametrize("kind", ["whole", "missing", "garbage", "another torch"])
def test_the_package_without_its_compiled_calls(tmp_path, kind):
    package = tmp_path / NAME
    package.mkdir()
    shutil.copy(os.path.join(os.path.dirname(z.__file__), "__init__.py"), package)
    shutil.copy(z.LIB_PATH, package)
    if kind == "garbage":
        (package / "_calls.so").write_bytes(b"\x7fELF of something else")
    elif kind != "missing":
        shutil.copy(z.CALLS_PATH, package)
    run = subprocess.run([sys.executable, "-c", SCRIPT, str(tmp_path), kind], capture_output=True, text=True, cwd=tmp_path)
    assert run.returncode == 0 and run.stdout.strip() == "fine", run.stderr


def test_the_package_needs_its_library(tmp_path):
    package = tmp_path / NAME
    package.mkdir()
    shutil.copy(os.path.join(os.path.dirname(z.__file__), "__init__.py"), package)
    run = subprocess.run([sys.executable, "-c", f"import {NAME}"], capture_output=True, text=True, cwd=tmp_path)
    assert run.returncode != 0 and "libzero_sm.so is missing" in run.stderr
