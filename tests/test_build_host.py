"""The compiled module (_marshal.so) against the torch and Python it was made for: a copy of the package without
it, with one made for another torch, or with one that does not load keeps every call that does not need it, and the
others say what to do; the build replaces it."""
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PKG = os.path.join(ROOT, "sparse_attention_09_b200")
PROBE = """
import torch, sparse_attention_09_b200 as dsa
assert dsa.__file__.startswith({where!r}), dsa.__file__
assert dsa.dsa_status_string(0) == "ok" and dsa.dsa_rope_frequencies(64, 1e4)[1] == 1.0
x = torch.zeros(4, 8)
try:
    dsa.dsa_rmsnorm(x, x[0], 1e-6, y=x)
except ImportError as e:
    assert "build.py" in str(e) and "_marshal.so" in str(e), e
    print("unbuilt")
except ValueError:
    print("built")
"""


def package_copy(tmp_path, marshal):
    pkg = tmp_path / "sparse_attention_09_b200"
    pkg.mkdir()
    for name in ("__init__.py", "build.py", "sharding.py", "libdsa.so"):
        os.symlink(os.path.join(PKG, name), pkg / name)
    if marshal is not None:
        (pkg / "_marshal.so").write_bytes(marshal)
    return str(tmp_path)


def probe(where):
    env = dict(os.environ, PYTHONPATH=where)
    res = subprocess.run([sys.executable, "-c", PROBE.format(where=where)], cwd=where, env=env, capture_output=True, text=True, timeout=300)
    assert res.returncode == 0, res.stderr
    return res.stdout.split()[-1]


def built():
    with open(os.path.join(PKG, "_marshal.so"), "rb") as f:
        return f.read()


def _build_module():
    from sparse_attention_09_b200 import build
    return build


@pytest.mark.parametrize("state", ["present", "absent", "of another torch", "of another Python", "broken"])
def test_package_with_and_without_its_module(tmp_path, state):
    target = _build_module().marshal_target().encode()
    data = built()
    assert data.count(target) == 1
    if state == "of another torch":
        import torch
        data = data.replace(b"for torch " + torch.__version__.encode()[:3], b"for torch 1.0")
    elif state == "of another Python":
        data = data.replace(b"cpython-3", b"cpython-2")
    elif state == "broken":
        data = target + b" and no module"
    where = package_copy(tmp_path, None if state == "absent" else data)
    assert probe(where) == ("built" if state == "present" else "unbuilt")


def test_build_replaces_a_module_of_another_torch(tmp_path, monkeypatch):
    build = _build_module()
    path = str(tmp_path / "_marshal.so")
    monkeypatch.setattr(build, "MARSHAL_PATH", path)
    calls = []

    def compiled(cmd, **kw):
        calls.append(cmd)
        with open(cmd[cmd.index("-o") + 1], "wb") as f:
            f.write(built())
        return subprocess.CompletedProcess(cmd, 0, "", "")

    monkeypatch.setattr(build.subprocess, "run", compiled)
    assert not build.marshal_current()
    build._build_marshal(False)                       # absent
    assert len(calls) == 1 and build.marshal_current()
    build._build_marshal(False)                       # current
    assert len(calls) == 1
    monkeypatch.setattr("torch.__version__", "99.0")  # the torch beside it has changed
    assert not build.marshal_current()
    build._build_marshal(False)
    assert len(calls) == 2 and any("torch 99.0" in c for c in calls[1])
