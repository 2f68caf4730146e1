"""The binding's compiled quick path is optional, and never one of another torch or Python: the
package imports without it, and calls then take the ctypes path.  CPU only, in child processes
that import a copy of the package."""
import os
import shutil
import subprocess
import sys

import pytest

import mla_latent_kv_22_b200 as M
from mla_latent_kv_22_b200 import build

PKG = os.path.dirname(M.__file__)
PROGRAM = """
import warnings
with warnings.catch_warnings(record=True) as w:
    warnings.simplefilter("always")
    import copied as M
print("warned", sum(issubclass(x.category, RuntimeWarning) and "build it with" in str(x.message) for x in w))
import torch
print("quick", M._binding.__class__.__name__ == "module", M._binding.append() is NotImplemented)
try:
    M.mla_append(*[torch.zeros(2)] * 6)
except ValueError as e:
    print("refused:", e)
"""


def run(tmp_path, *binding):
    """A copy of the package with those extensions; what PROGRAM says of it."""
    pkg = tmp_path / "copied"
    pkg.mkdir()
    for f in ("__init__.py", "build.py"):
        shutil.copy(os.path.join(PKG, f), pkg)
    os.symlink(os.path.join(PKG, "libmla.so"), pkg / "libmla.so")
    for source, name in binding:
        if source is None:
            (pkg / name).write_bytes(b"no extension")
        else:
            os.symlink(source, pkg / name)
    r = subprocess.run([sys.executable, "-c", PROGRAM], cwd=tmp_path, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr
    return r.stdout.splitlines()


REFUSED = "refused: c_kv must be [N, 512]"


def test_with_the_extension(tmp_path):
    path = build.binding_path()
    assert os.path.exists(path), "built with the library"
    assert run(tmp_path, (path, os.path.basename(path))) == ["warned 0", "quick True True", REFUSED]


@pytest.mark.parametrize("other", ["missing", "unversioned", "other torch", "broken"])
def test_without_it_the_package_imports_and_warns(tmp_path, other):
    path = build.binding_path()
    name = os.path.basename(path)
    binding = {"missing": [], "unversioned": [(path, "_binding.so")], "broken": [(None, name)],
               "other torch": [(path, name.replace("torch-", "torch-9."))]}[other]
    assert run(tmp_path, *binding) == ["warned 1", "quick False True", REFUSED]


def test_the_file_follows_torch_and_python(monkeypatch):
    import torch
    path = build.binding_path()
    assert torch.__version__ in path and path.endswith(build.sysconfig.get_config_var("EXT_SUFFIX"))
    monkeypatch.setattr(torch, "__version__", "9.9.9")
    assert build.binding_path() != path and not build.up_to_date()
