"""The build and the import where the native binding cannot be had: the library and the
products do not depend on it, and the calls that do say so."""
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture()
def build():
    import __graft_entry__

    mod = __graft_entry__._load_build_module()
    mod.build()
    return __graft_entry__._load_build_module()              # a copy of its own to change


@pytest.mark.parametrize("compiler", ["false", "/nonexistent/g++"])
def test_library_is_linked_although_the_binding_is_not_compiled(build, monkeypatch, tmp_path, compiler):
    before = os.stat(build.BINDING).st_mtime_ns
    monkeypatch.setenv("CXX", compiler)
    monkeypatch.setattr(build, "LIB", str(tmp_path / "libq4nx.so"))
    monkeypatch.setattr(build, "_stale", lambda target, deps: "serving" in os.path.basename(target))
    with pytest.raises(RuntimeError, match="serving_binding.cpp"):
        build.build()
    assert os.path.getsize(build.LIB) > 0 and os.stat(build.BINDING).st_mtime_ns == before


def test_no_binding_without_torch(build, monkeypatch, tmp_path):
    real = build.importlib.util.find_spec
    monkeypatch.setattr(build.importlib.util, "find_spec", lambda name, *a: None if name == "torch" else real(name, *a))
    monkeypatch.setattr(build, "LIB", str(tmp_path / "libq4nx.so"))
    monkeypatch.setattr(build, "BINDING", str(tmp_path / "_serving.so"))
    assert build.build() == build.LIB
    assert os.path.getsize(build.LIB) > 0 and not os.path.exists(build.BINDING)


def test_binding_is_linked_again_for_another_torch(build, monkeypatch, tmp_path):
    # two torches whose objects are both there, the later one's link newer than either
    objs = {}
    for version in ("1.0", "2.0"):
        objs[version] = tmp_path / f"serving_binding-torch{version}.o"
        objs[version].write_bytes(b"")
        os.utime(objs[version], (1, 1))
    linked, binding = [], tmp_path / "_serving.so"

    def jobs(version):
        link = [sys.executable, "-c", "import sys; open(sys.argv[-1], 'w').write(sys.argv[1])", str(objs[version])]
        return ["true", "-o", str(objs[version])], link

    monkeypatch.setattr(build, "BINDING", str(binding))
    monkeypatch.setattr(build, "OBJS", str(tmp_path))
    monkeypatch.setattr(build, "LIB", os.devnull)
    monkeypatch.setattr(build, "_stale", lambda target, deps: target == str(binding) and not binding.exists())
    for version in ("1.0", "2.0", "2.0", "1.0"):
        monkeypatch.setattr(build, "_binding_jobs", lambda nvcc: jobs(version))
        before = os.stat(binding).st_ino if binding.exists() else 0
        build.build()
        assert binding.read_text() == str(objs[version])
        linked.append(os.stat(binding).st_ino != before)
    assert linked == [True, True, False, True]


def test_products_without_the_binding(build):
    code = """
import sys
sys.modules["dequant_gemv_gb300._serving"] = None            # as if there were no such file
import dequant_gemv_gb300 as q
import torch
assert q.q4nx_chunk_bytes(q.Q4NX_Q4_1) == 5120 and q.lib.q4nx_decode(None, 16, 16, None) == q.Q4NX_E_NULL
assert q.q4nx_kv_page_bytes(64, 1, 16) == 16 * 80
try:
    q.q4nx_logprobs(torch.zeros(1, 2))
except ImportError as e:
    assert "_build.py" in str(e) and "logprobs" in str(e)
else:
    raise AssertionError("q4nx_logprobs did not refuse")
"""
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
