"""Building the Python binding of the small calls (host only)."""
import os
import subprocess

import pytest


@pytest.mark.parametrize("change", ["version", "python"])
def test_another_torch_or_python_rebuilds_the_binding(monkeypatch, tmp_path, change):
    """... also where its files are older than the binding."""
    from invariant_verify_gb300 import build
    torch_dir = tmp_path / "torch"
    torch_dir.mkdir()
    (torch_dir / "version.py").write_text("__version__ = '2.9.1+cu130'\n")
    os.utime(torch_dir / "version.py", (1, 1))
    ran = []

    def compiler(cmd, **kw):
        out = cmd[cmd.index("-o") + 1]
        with open(out, "w") as f:
            f.write("built")
        ran.append(cmd)
        return subprocess.CompletedProcess(cmd, 0, "", "")

    class Spec:
        submodule_search_locations = [str(torch_dir)]

    soabi = ["cpython-312"]
    monkeypatch.setattr(build, "TORCH_LIB", str(tmp_path / "_biv_torch.so"))
    monkeypatch.setattr(build, "nvcc", lambda: "/usr/local/cuda/bin/nvcc")
    monkeypatch.setattr(build.subprocess, "run", compiler)
    monkeypatch.setattr(build.importlib.util, "find_spec", lambda name: Spec)
    monkeypatch.setattr(build.sysconfig, "get_config_var", lambda name: soabi[0])
    build._compile_torch()
    build._compile_torch()
    assert len(ran) == 1                           # nothing has changed
    if change == "version":
        (torch_dir / "version.py").write_text("__version__ = '2.11.0+cu130'\n")
        os.utime(torch_dir / "version.py", (1, 1))
    else:
        soabi[0] = "cpython-313"
    build._compile_torch()
    assert len(ran) == 2


def test_the_library_builds_without_torch(monkeypatch, tmp_path):
    from invariant_verify_gb300 import build
    monkeypatch.setattr(build, "TORCH_LIB", str(tmp_path / "_biv_torch.so"))
    monkeypatch.setattr(build.importlib.util, "find_spec", lambda name: None)
    monkeypatch.setattr(build.subprocess, "run", lambda *a, **kw: pytest.fail("nothing is compiled"))
    build._compile_torch()
    assert not os.listdir(tmp_path)
