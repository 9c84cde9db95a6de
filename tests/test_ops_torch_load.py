"""The package without a usable _cp_torch.so: the coded table's part imports and
works, a dense operator on tensors says why it does not."""
from __future__ import annotations

import os
import shutil
import subprocess
import sys

import pytest
import torch

from trellis_coded_row_amd import build as cpbuild

NAME = os.path.basename(cpbuild.PKG)
PROGRAM = f"""
import torch
import {NAME} as cp
print("table", cp.cp_record_bytes(64, 4), cp.cp_supported(64, 4), hasattr(cp, "Table"), cp.cp_gemm_fp8_workspace_bytes(0, 1, 1, 0))
try:
    cp.rms_norm(torch.ones(4, 8), torch.ones(8))
except (ImportError, ValueError) as e:
    print(type(e).__name__, e)
"""


@pytest.fixture
def copy(tmp_path):
    """A copy of the package, its libraries and headers."""
    shutil.copytree(cpbuild.PKG, tmp_path / NAME, ignore=shutil.ignore_patterns("__pycache__", "*.hip", "*.tmp*"))
    shutil.copytree(os.path.join(cpbuild.ROOT, "include"), tmp_path / "include")
    return tmp_path


def run(folder, compiler="/nonexistent/c++"):
    r = subprocess.run([sys.executable, "-W", "always", "-c", PROGRAM], cwd=folder, capture_output=True, text=True,
                       timeout=300, env=dict(os.environ, PYTHONPATH=str(folder), CXX=compiler))
    assert r.returncode == 0, r.stderr[-600:]
    first, second = r.stdout.splitlines()[:2]
    assert first.startswith("table ") and first.endswith(" True 0")
    return second, r.stderr


def test_as_built(copy):
    result, errors = run(copy)
    assert result.startswith("ValueError") and "older than its sources" not in errors


def test_missing_and_without_a_compiler(copy):
    os.remove(copy / NAME / "_cp_torch.so")
    result, _ = run(copy)
    assert result.startswith("ImportError") and "rms_norm" in result and "/nonexistent/c++" in result


def test_built_for_another_torch(copy):
    path = copy / NAME / "_cp_torch.so"
    held, mark = path.read_bytes(), b"[built for torch " + torch.__version__.encode()
    assert mark in held
    path.write_bytes(held.replace(mark, b"[built for torch " + b"x" * len(torch.__version__)))
    result, _ = run(copy)
    assert result.startswith("ImportError") and "/nonexistent/c++" in result


def test_not_a_library(copy):
    path = copy / NAME / "_cp_torch.so"
    path.write_bytes(f"{cpbuild._torch_mark()} {cpbuild._source_mark()}".encode())
    result, _ = run(copy)
    assert result.startswith("ImportError")


def test_older_than_its_sources(copy):
    with open(copy / NAME / "csrc" / "cp_torch.cpp", "a") as f:
        f.write("// changed\n")
    result, errors = run(copy)
    assert result.startswith("ValueError") and "older than its sources" in errors


def test_without_its_sources(copy):
    shutil.rmtree(copy / NAME / "csrc")
    shutil.rmtree(copy / "include")
    result, errors = run(copy)
    assert result.startswith("ValueError") and "older than its sources" not in errors


def test_built_again_where_it_is_missing(copy):
    os.remove(copy / NAME / "_cp_torch.so")
    result, _ = run(copy, os.environ.get("CXX", "g++"))
    assert result.startswith("ValueError") and (copy / NAME / "_cp_torch.so").exists()
