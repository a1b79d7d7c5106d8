"""What works without a GPU build of torch and without a host compiler."""
import os
import subprocess
import sys

import pytest

from bit_weight_gemm_amd import build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_host_queries_without_torchs_gpu_functions():
    code = ("import torch\n"
            "for n in ('_cuda_getCurrentRawStream', '_cuda_getDevice'):\n"
            "    if hasattr(torch._C, n): delattr(torch._C, n)\n"
            "from bit_weight_gemm_amd import binding as B\n"
            "print(B.biloco_gemm_workspace_bytes(1, 256, 256, 16), B.biloco_attn_workspace_bytes(1, 1, 4, 2, 64, 1, 10))\n")
    p = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True)
    assert p.returncode == 0, p.stderr
    assert len(p.stdout.split()) == 2


@pytest.fixture
def places(tmp_path, monkeypatch):
    """build() with its products in tmp_path and its compilers' runs noted."""
    for n in ("BUILD", "LIB", "BINDING", "RESOURCES"):
        monkeypatch.setattr(build, n, str(tmp_path / os.path.basename(getattr(build, n))))
    monkeypatch.setattr(build, "_compile", lambda src, *a: src + ".o")
    runs = []

    def run(cmd, **kw):
        runs.append(cmd[0])
        with open(cmd[cmd.index("-o") + 1], "w") as f:
            f.write("built")
        return subprocess.CompletedProcess(cmd, 0, "", "")
    monkeypatch.setattr(build.subprocess, "run", run)
    return runs


def test_library_is_built_without_a_host_compiler(places, monkeypatch, capsys):
    with open(build.BINDING, "w") as f:
        f.write("of an earlier build")
    which = build.shutil.which
    monkeypatch.setattr(build.shutil, "which", lambda n, *a, **kw: None if n == "g++" else which(n, *a, **kw))
    assert build.build() == build.LIB and os.path.exists(build.LIB)
    assert "g++" not in places and not os.path.exists(build.BINDING)      # nor a stale one
    assert "g++" in capsys.readouterr().out


def test_both_are_built_with_one(places):
    build.build()
    assert "g++" in places and os.path.exists(build.LIB) and os.path.exists(build.BINDING)


def test_a_binding_that_does_not_compile_fails_the_build(places, monkeypatch):
    run = build.subprocess.run

    def fails(cmd, **kw):
        return subprocess.CompletedProcess(cmd, 1, "", "no") if cmd[0] == "g++" else run(cmd, **kw)
    monkeypatch.setattr(build.subprocess, "run", fails)
    with pytest.raises(RuntimeError, match="g\\+\\+"):
        build.build()
