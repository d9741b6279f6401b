"""What build() makes anew, and what an import says of a part that is not there."""

import importlib.util
import os
import shutil
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PKG = os.path.join(ROOT, "sparse_mla_decode_csr_gb300")


@pytest.fixture
def build(tmp_path, monkeypatch):
    """build.py with objects in a folder of their own, and the commands that it ran."""
    spec = importlib.util.spec_from_file_location("build_under_test", os.path.join(PKG, "build.py"))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    module.ran = []

    def run(cmd, what, verbose):
        module.ran.append(os.path.basename(cmd[cmd.index("-c") + 1]))
        open(cmd[cmd.index("-o") + 1], "w").close()

    monkeypatch.setattr(module, "_run", run)
    monkeypatch.setattr(module, "BUILD", str(tmp_path))
    return module


def test_the_binding_is_made_anew_for_another_pytorch(build, tmp_path, monkeypatch):
    binding, kernel = (os.path.join(build.CSRC, f) for f in ("smla_binding.cpp", "smla_pack.cu"))
    for _ in range(2):
        build._compile(binding, False), build._compile(kernel, False)
    assert build.ran == ["smla_binding.cpp", "smla_pack.cu"]
    other = tmp_path / "torch"
    other.mkdir()
    for version in ("7.0.0", "7.0.1"):
        (other / "version.py").write_text(f"__version__ = '{version}'\n")
        monkeypatch.setattr(build, "_torch", lambda *path: os.path.join(str(other), *path))
        build.ran.clear()
        for _ in range(2):
            build._compile(binding, False), build._compile(kernel, False)
        assert build.ran == ["smla_binding.cpp"]


def test_the_binding_is_made_anew_for_another_python(build, monkeypatch):
    binding = os.path.join(build.CSRC, "smla_binding.cpp")
    build._compile(binding, False)
    ask = build.sysconfig.get_config_var
    monkeypatch.setattr(build.sysconfig, "get_config_var", lambda name: "cpython-99" if name == "SOABI" else ask(name))
    build._compile(binding, False)
    assert build.ran == ["smla_binding.cpp"] * 2


@pytest.mark.parametrize("kept", [[], ["libsmla.so"]])
def test_an_import_without_a_library_says_how_to_build_it(kept, tmp_path):
    pkg = tmp_path / "partial_smla"
    pkg.mkdir()
    for f in ["__init__.py", *kept]:
        shutil.copy(os.path.join(PKG, f), pkg)
    r = subprocess.run([sys.executable, "-c", "import partial_smla"], cwd=tmp_path, capture_output=True, text=True)
    assert r.returncode != 0 and "ImportError" in r.stderr and "is not built" in r.stderr and "g.build()" in r.stderr
