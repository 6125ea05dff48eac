"""libprune24.so and the calls that ctypes marshals do not depend on the marshalling of torch tensors in C++: neither
on its build nor on its loading. No GPU is needed."""
import importlib.util
import os
import shutil
import subprocess
import sys

import pytest

from tests.conftest import ROOT

PACKAGE = "semi_structured_sparse_prune24_gb300"


@pytest.fixture
def build(tmp_path, monkeypatch):
    """build.py with folders of its own, and in the place of every compiler's run a note and an empty output."""
    spec = importlib.util.spec_from_file_location("_build_under_test", os.path.join(ROOT, PACKAGE, "build.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    for name, path in (("BUILD", "o"), ("LIBDIR", "lib"), ("LIB", "lib/libprune24.so"), ("MARSHAL", "lib/_p24_torch.so")):
        monkeypatch.setattr(mod, name, str(tmp_path / path))
    mod.fails, mod.ran = "nothing", []

    def run(cmd, what):
        mod.ran.append(cmd)
        if any(str(a).endswith(mod.fails) for a in cmd):
            raise RuntimeError(what)
        open(cmd[cmd.index("-o") + 1], "w").write(str(len(mod.ran)))
    monkeypatch.setattr(mod, "_run", run)
    return mod


@pytest.mark.parametrize("fails", ["p24_torch.cpp", "p24_torch.o"])
def test_the_library_is_linked_where_the_marshalling_fails(build, fails):
    build.build()
    assert os.path.exists(build.LIB) and os.path.exists(build.MARSHAL)
    os.remove(build.LIB)
    build.fails = fails
    with pytest.raises(RuntimeError, match="p24_torch"):
        build.build()
    assert os.path.exists(build.LIB)
    assert not os.path.exists(build.MARSHAL)        # nothing of an earlier build is left to be loaded


def test_the_marshalling_is_built_for_this_torch(build):
    import torch
    build.build()
    cmd = next(c for c in build.ran if any(str(a).endswith("p24_torch.cpp") for a in c))
    assert f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}" in cmd


SCRIPT = """
import torch
{before}
import {package} as P
assert P.ld_vals(8200) == 4104 and P.lib.p24_strerror(0)
try:
    P.p24_rmsnorm(torch.zeros(2, 8))
except {error} as e:
    assert {says!r} in str(e), str(e)
else:
    raise SystemExit("no error")
"""


@pytest.mark.parametrize("before,marshal,error,says", [
    ("", "missing", "ImportError", "not built"),
    ("", "broken", "ImportError", "not available"),
    ("torch.__version__ = '9.9.9'", "whole", "ImportError", "this is 9.9.9"),
    ("", "whole", "ValueError", "CUDA tensor"),
])
def test_the_package_without_its_marshalling(tmp_path, before, marshal, error, says):
    to = tmp_path / PACKAGE
    shutil.copytree(os.path.join(ROOT, PACKAGE), to, ignore=shutil.ignore_patterns("csrc", "__pycache__", "*.tmp"))
    so = to / "_lib" / "_p24_torch.so"
    if marshal != "whole":
        so.unlink()
    if marshal == "broken":
        so.write_bytes(b"no library")
    script = SCRIPT.format(before=before, package=PACKAGE, error=error, says=says)
    r = subprocess.run([sys.executable, "-c", script], cwd=tmp_path, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
