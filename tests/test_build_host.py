"""What the build script compiles and links, with a compiler that only writes
its output file: after a change of torch or Python, and without torch."""

import importlib.util
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture
def B(tmp_path, monkeypatch):
    """The build script with its outputs in a folder of its own; `B.ran` lists
    the files that a build wrote."""
    path = os.path.join(ROOT, "kv_cache_vector_turboquant_b200", "build.py")
    spec = importlib.util.spec_from_file_location("_build_under_test", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    mod.ran = []

    def run(cmd, **_):
        out = cmd[cmd.index("-o") + 1]
        with open(out, "w") as f:
            f.write(" ".join(cmd))
        mod.ran.append(os.path.basename(out).removesuffix(".tmp"))
        return subprocess.CompletedProcess(cmd, 0, "", "")

    monkeypatch.setattr(mod.subprocess, "run", run)
    monkeypatch.setattr(mod, "_nvcc", lambda: "nvcc")
    monkeypatch.setattr(mod, "BUILD", str(tmp_path / "objects"))
    for name in ("LIB", "TEST_LIB", "OPS_LIB"):
        monkeypatch.setattr(mod, name, str(tmp_path / os.path.basename(getattr(mod, name))))
    return mod


def _built(B):
    B.ran.clear()
    B.build()
    return sorted(B.ran)


def test_everything_once(B):
    objects = [s + ".o" for s in B.SOURCES + B.TEST_SOURCES + B.OPS_SOURCES]
    assert _built(B) == sorted(objects + ["libtq.so", "libtq_test.so", "_ops.so"])
    assert _built(B) == []


def test_another_torch_or_python_compiles_the_extension_again(B, monkeypatch):
    _built(B)
    abi = B._abi(B._torch())
    monkeypatch.setattr(B, "_abi", lambda torch: abi + "+other")
    ran = _built(B)
    assert "tq_torch.cpp.o" in ran and "_ops.so" in ran
    assert not any(s + ".o" in ran for s in B.SOURCES + B.TEST_SOURCES)
    assert _built(B) == []


def test_the_library_builds_without_torch(B, monkeypatch, capsys):
    with monkeypatch.context() as m:
        m.setattr(B.importlib.util, "find_spec", lambda name: None)
        ran = _built(B)
        assert "libtq.so" in ran and "libtq_test.so" in ran and not {"_ops.so", "tq_torch.cpp.o"} & set(ran)
        assert "_ops.so is not built" in capsys.readouterr().err
        assert _built(B) == []
    ran = _built(B)  # torch is there: the extension alone is compiled
    assert "tq_torch.cpp.o" in ran and "_ops.so" in ran
    assert not any(s + ".o" in ran for s in B.SOURCES + B.TEST_SOURCES)
