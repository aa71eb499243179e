"""What build() makes, and when (no GPU needed; the compilers are stood in for)."""
import os

import pytest

from attention_fa2_forward_02_gb300 import build as B


@pytest.fixture
def tree(tmp_path, monkeypatch):
    """A built tree in a folder of its own; the compilers write their file and are recorded."""
    csrc, include = tmp_path / "csrc", tmp_path / "include"
    csrc.mkdir()
    include.mkdir()
    for name in ("api.cu", "common.cuh", "internal.h", "torch_args.cpp"):
        (csrc / name).write_text("")
    (include / "fa2.h").write_text("")
    torch = tmp_path / "torch"
    torch.mkdir()
    (torch / "version.py").write_text("__version__ = '1'\n")
    for name, path in {"CSRC": csrc, "INCLUDE": include, "BUILD_DIR": tmp_path / "_build", "LIB": tmp_path / "lib.so",
                       "TORCH_LIB": tmp_path / "ext.so", "TORCH_SRC": csrc / "torch_args.cpp",
                       "TORCH_STAMP": tmp_path / "_build" / "stamp"}.items():
        monkeypatch.setattr(B, name, str(path))
    calls = []

    class Done:
        returncode, stdout, stderr = 0, "", ""

    def compiler(cmd, **kw):
        out = cmd[cmd.index("-o") + 1]
        open(out, "w").close()
        calls.append(os.path.basename(out))
        return Done()

    monkeypatch.setattr(B.subprocess, "run", compiler)
    monkeypatch.setattr(B, "_nvcc", lambda: "/usr/local/cuda/bin/nvcc")
    monkeypatch.setattr(B, "_torch_dir", lambda: str(torch))
    B.build()
    assert sorted(calls) == ["api.o", "ext.so.tmp", "lib.so.tmp"]
    # everything written before the libraries, so that a touched file is newer
    for root, _, files in os.walk(tmp_path):
        for f in files:
            os.utime(os.path.join(root, f), (1e9, 1e9))
    for f in ("LIB", "TORCH_LIB"):
        os.utime(getattr(B, f), (2e9, 2e9))
    monkeypatch.setattr(B, "__file__", str(csrc / "api.cu"))
    calls.clear()
    return tmp_path, calls


def touch(path):
    os.utime(path, (3e9, 3e9))


def test_nothing_to_do(tree):
    assert B.build() == B.LIB and tree[1] == []


def test_without_torch_the_library_is_built(tree, monkeypatch, capsys):
    path, calls = tree
    monkeypatch.setattr(B, "_torch_dir", lambda: None)
    touch(path / "csrc" / "api.cu")
    assert B.build() == B.LIB
    assert calls == ["api.o", "lib.so.tmp"] and "torch is not installed" in capsys.readouterr().err


def test_torch_is_looked_for_without_importing_it(monkeypatch):
    monkeypatch.setattr(B.importlib.util, "find_spec", lambda name: None)
    assert B._torch_dir() is None


def test_each_part_for_its_own_sources(tree):
    path, calls = tree
    touch(path / "csrc" / "torch_args.cpp")
    B.build()
    assert calls == ["ext.so.tmp"]
    calls.clear()
    os.utime(path / "csrc" / "torch_args.cpp", (1e9, 1e9))
    touch(path / "csrc" / "common.cuh")
    B.build()
    assert calls == ["api.o", "lib.so.tmp"]


def test_another_torch_has_its_own_extension(tree):
    path, calls = tree
    (path / "torch" / "version.py").write_text("__version__ = '2'\n")
    B.build()
    assert calls == ["ext.so.tmp"]
    calls.clear()
    os.utime(B.TORCH_LIB, (2e9, 2e9))
    B.build()
    assert calls == []


def test_a_failing_extension_leaves_a_library(tree, monkeypatch):
    path, calls = tree
    ok = B.subprocess.run

    def compiler(cmd, **kw):
        r = ok(cmd, **kw)
        if "ext.so" in cmd[cmd.index("-o") + 1]:
            r.returncode = 1
        return r

    monkeypatch.setattr(B.subprocess, "run", compiler)
    os.remove(B.LIB)
    with pytest.raises(RuntimeError, match="g\\+\\+ failed"):
        B.build(force=True)
    assert os.path.exists(B.LIB)
