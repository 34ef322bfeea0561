"""CPU: what the build does on machines that lack some of what the marshalling
extension takes. Compilers are replaced by a function that notes the command and
writes the output file; PyTorch's folder by one made for the test."""
import importlib.util
import os
import subprocess
import sysconfig
from types import SimpleNamespace

import pytest

from dense_gemm_gb300 import build as b


@pytest.fixture
def machine(tmp_path, monkeypatch):
    """A machine on which nothing is built yet, with a PyTorch that has CUDA parts."""
    torch = tmp_path / "torch"
    for f in ("include/c10/cuda/CUDAStream.h", "lib/libc10_cuda.so", "__init__.py"):
        p = torch / f
        p.parent.mkdir(parents=True, exist_ok=True)
        p.write_text("")
    (torch / "version.py").write_text("__version__ = '9.9.0+cu130'\n")
    find = importlib.util.find_spec
    monkeypatch.setattr(importlib.util, "find_spec",
                        lambda name, *a: SimpleNamespace(origin=str(torch / "__init__.py")) if name == "torch" else find(name, *a))
    monkeypatch.setattr(b, "HERE", str(tmp_path))
    monkeypatch.setattr(b, "LIB", str(tmp_path / "libgemm_f16.so"))
    monkeypatch.setattr(b, "NATIVE", str(tmp_path / "_native.so"), raising=False)  # a fixed name, where there is one
    monkeypatch.setattr(b, "nvcc", lambda: "/usr/local/cuda/bin/nvcc")
    monkeypatch.delenv("CXX", raising=False)
    commands = []

    def run(cmd, check=True, **kw):
        commands.append(cmd[0])
        if not cmd[0].endswith("nvcc"):
            headers = [i[2:] for i in cmd if i.startswith("-I")]
            if not any(os.path.exists(os.path.join(i, "c10", "cuda", "CUDAStream.h")) for i in headers):
                raise subprocess.CalledProcessError(1, cmd)
            if cmd[0] != "g++":
                raise FileNotFoundError(cmd[0])
        with open(cmd[cmd.index("-o") + 1], "w") as f:
            f.write("built")

    monkeypatch.setattr(subprocess, "run", run)
    return SimpleNamespace(torch=torch, commands=commands, dir=tmp_path)


def test_both_are_built_where_both_can_be(machine):
    assert b.build() == b.LIB and os.path.exists(b.LIB)
    assert sorted(machine.commands) == ["/usr/local/cuda/bin/nvcc", "g++"]
    b.build()
    assert len(machine.commands) == 2  # both are up to date


@pytest.mark.parametrize("lacks", ["headers", "library", "compiler"])
def test_the_library_needs_neither_pytorchs_cuda_parts_nor_a_compiler_for_it(machine, lacks, monkeypatch, capfd):
    if lacks == "headers":
        (machine.torch / "include/c10/cuda/CUDAStream.h").unlink()
    elif lacks == "library":
        (machine.torch / "lib/libc10_cuda.so").unlink()
    else:
        monkeypatch.setenv("CXX", str(machine.dir / "no-such-compiler"))
    assert b.build() == b.LIB and os.path.exists(b.LIB)
    assert machine.commands == ["/usr/local/cuda/bin/nvcc"]
    said = capfd.readouterr().err
    assert "_native" in said and {"headers": "CUDAStream.h", "library": "libc10_cuda.so", "compiler": "no-such-compiler"}[lacks] in said


def test_an_error_in_the_extension_is_not_passed_over(machine, monkeypatch):
    run = subprocess.run

    def fails(cmd, **kw):
        if cmd[0] == "g++":
            raise subprocess.CalledProcessError(1, cmd)
        run(cmd, **kw)

    monkeypatch.setattr(subprocess, "run", fails)
    with pytest.raises(subprocess.CalledProcessError):
        b.build()
    assert os.path.exists(b.LIB)


def test_another_pytorch_gets_an_extension_of_its_own(machine, monkeypatch):
    """The same sources and file times, another PyTorch or Python: what is there is
    neither taken for up to date nor found by the operators."""
    b.build()
    (machine.torch / "version.py").write_text("__version__ = '9.10.0+cu130'\n")
    b.build()
    assert machine.commands.count("g++") == 2
    config = sysconfig.get_config_var
    monkeypatch.setattr(sysconfig, "get_config_var", lambda name: "cpython-399-other" if name == "SOABI" else config(name))
    b.build()
    assert machine.commands.count("g++") == 3
    b.build()
    assert machine.commands.count("g++") == 3
    assert len(list(machine.dir.glob("_native*.so"))) == 3


def test_the_operators_name_what_is_missing(machine, monkeypatch):
    import torch
    from dense_gemm_gb300 import GemmError, ops
    monkeypatch.setattr(ops, "_module", None)
    monkeypatch.setattr(ops, "load_library", lambda: None)
    x = torch.zeros(2, 8)
    with pytest.raises(GemmError, match="_native.*build it with"):
        ops.rms_norm(x, x[0])
    (machine.torch / "lib/libc10_cuda.so").unlink()
    with pytest.raises(GemmError, match="_native.*libc10_cuda.so is missing"):
        ops.rms_norm(x, x[0])
