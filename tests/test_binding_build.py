"""When the paged cache's binding is compiled again, and that one compiled for another torch is refused (CPU)."""
import os
import subprocess

import pytest
import torch

from io_aware_exact_19_b200 import build as fa_build


def test_binding_is_rebuilt_for_another_torch(tmp_path, monkeypatch):
    outputs = []

    def compiler(cmd, **kw):
        outputs.append(cmd[cmd.index("-o") + 1])
        open(outputs[-1], "w").close()
        return subprocess.CompletedProcess(cmd, 0, "", "")

    monkeypatch.setattr(fa_build, "BINDING", str(tmp_path / "_paged.so"))
    monkeypatch.setattr(fa_build, "BUILD", str(tmp_path))
    monkeypatch.setattr(fa_build, "_nvcc", lambda: "/usr/local/cuda/bin/nvcc")
    monkeypatch.setattr(fa_build.subprocess, "run", compiler)
    fa_build._build_binding()
    fa_build._build_binding()
    assert len(outputs) == 1 and os.path.exists(fa_build.BINDING)
    monkeypatch.setattr(torch, "__version__", "0.0.0+other")  # the files are newer than every source
    fa_build._build_binding()
    fa_build._build_binding()
    assert len(outputs) == 2
    assert all(str(os.getpid()) in out for out in outputs)  # builds at the same time do not share a file


def test_binding_for_another_torch_is_refused(monkeypatch):
    fa_build.build()
    from io_aware_exact_19_b200 import paged
    assert paged._load_binding() is paged._binding
    monkeypatch.setattr(paged, "binding_stamp", lambda: "another torch")
    with pytest.raises(FileNotFoundError, match="built for another torch"):
        paged._load_binding()
