"""The build on the CPU, with stand-ins for the compilers: what is built where the binding's part is missing, and when it is
built again."""
import os
import stat

import pytest
import torch

from gemm_dequant_gemv_q8_b200 import build as qbuild

# writes what -o names and one line to the log
COMPILER = """#!/bin/sh
echo "$@" >> "{log}"
while [ $# -gt 0 ]; do
  if [ "$1" = -o ]; then echo made > "$2"; fi
  shift
done
"""


@pytest.fixture
def sandbox(tmp_path, monkeypatch):
    """Outputs in a folder of their own, both compilers replaced.  Returns (folder, lines of the log)."""
    log, cc = tmp_path / "log", tmp_path / "cc"
    cc.write_text(COMPILER.format(log=log))
    cc.chmod(cc.stat().st_mode | stat.S_IXUSR)
    monkeypatch.setattr(qbuild, "HERE", str(tmp_path))
    monkeypatch.setattr(qbuild, "LIB", str(tmp_path / "libqlin.so"))
    monkeypatch.setattr(qbuild, "BINDING", str(tmp_path / "_qlin_torch.so"))
    monkeypatch.setattr(qbuild, "NVCC", str(cc))
    monkeypatch.setenv("CXX", str(cc))
    return tmp_path, lambda: log.read_text().splitlines() if log.exists() else []


def test_the_library_does_not_wait_for_the_binding(sandbox, monkeypatch):
    folder, _ = sandbox
    monkeypatch.setenv("CXX", str(folder / "no_such_compiler"))
    with pytest.raises(Exception):
        qbuild.build()
    assert os.path.exists(qbuild.LIB) and not os.path.exists(qbuild.BINDING)


def test_the_binding_is_built_again_for_another_torch(sandbox, monkeypatch):
    _, lines = sandbox
    qbuild.build_binding()
    qbuild.build_binding()
    assert len(lines()) == 1
    monkeypatch.setattr(torch, "__version__", torch.__version__ + ".other")
    qbuild.build_binding()
    qbuild.build_binding()
    assert len(lines()) == 2
    os.remove(qbuild.BINDING)
    qbuild.build_binding()
    assert len(lines()) == 3 and os.path.exists(qbuild.BINDING)


def test_everything_is_built_once(sandbox):
    _, lines = sandbox
    qbuild.build()
    n = len(lines())
    assert n == len(qbuild.sources()) + 2 and os.path.exists(qbuild.LIB) and os.path.exists(qbuild.BINDING)
    qbuild.build()
    assert len(lines()) == n
    qbuild.build(force=True)
    assert len(lines()) == 2 * n
