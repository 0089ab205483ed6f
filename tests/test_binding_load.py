"""CPU: the package without, and with another torch's, module for the paged calls."""
import importlib.util
import os
import shutil
import subprocess
import sys

import pytest

qdk = pytest.importorskip("query_driven_key_b200")
PKG = os.path.dirname(qdk.__file__)

CODE = """
import query_driven_key_b200 as qdk, torch
assert qdk.__file__.startswith({root!r}), qdk.__file__
assert qdk.think_t_from_lambda(128, 0.4) > 0 and qdk.think_extend_pages_workspace_size() == 256
{before}
t = torch.zeros(4, 2, 128)
try:
    qdk.think_gather_pages(t, t, t, t)
except {error} as e:
    print("raised", e)
"""


def package(tmp_path, binding: bool):
    root = os.path.join(tmp_path, "query_driven_key_b200")
    os.makedirs(root)
    for f in ["__init__.py", "libthink.so"] + (["_binding.so"] if binding else []):
        shutil.copy(os.path.join(PKG, f), root)
    return str(tmp_path)


def run(root, before, error):
    r = subprocess.run([sys.executable, "-c", CODE.format(root=root, before=before, error=error)], cwd=root, capture_output=True,
                       text=True, env=dict(os.environ, PYTHONPATH=root), timeout=300)
    assert r.returncode == 0, r.stderr
    return r.stdout


def test_import_and_other_calls_without_the_binding(tmp_path):
    assert "raised _binding.so not found" in run(package(tmp_path, False), "", "ImportError")


def test_another_torch_is_refused(tmp_path):
    root = package(tmp_path, True)
    assert "raised _binding.so was built with torch" in run(root, "torch.__version__ = '0.0.1'", "ImportError")
    assert "raised" in run(root, "", "qdk.ThinkError")


def test_build_sees_another_torch():
    spec = importlib.util.spec_from_file_location("_think_build_under_test", os.path.join(PKG, "build.py"))
    build = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(build)
    import torch
    with open(build.BINDING, "rb") as f:
        assert f"torch_version={torch.__version__}\0".encode() in f.read()
    assert not build._binding_is_current("0.0.1")
