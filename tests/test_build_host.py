"""What build() makes with, without and against another torch (CPU only: the
compilers are stood in for)."""
import os
import subprocess
import sys

import pytest
import torch

from attention_fa2_forward_03_gb300 import build, fa2


@pytest.fixture
def made(tmp_path, monkeypatch):
    """build() into an empty folder; the compilers only write their output
    (those in `broken` fail). Returns (outputs so far, broken)."""
    done, broken = [], set()
    for name in ("LIB", "DEBUG_LIB", "TORCH_LIB", "TORCH_STAMP"):
        monkeypatch.setattr(build, name, str(tmp_path / os.path.basename(getattr(build, name))))

    class Compiler:
        def __init__(self, cmd):
            out = cmd[cmd.index("-o") + 1]
            self.returncode = int(cmd[0] in broken)
            if not self.returncode:
                done.append(os.path.basename(out).split(".tmp")[0])
                open(out, "w").close()

        def wait(self):
            return self.returncode

    monkeypatch.setattr(build.subprocess, "Popen", Compiler)
    return done, broken


def test_everything_is_made_once(made):
    done, _ = made
    assert build.build() == build.LIB and sorted(done) == ["_kv4_torch.so", "libfa2.so", "libfa2_debug.so"]
    assert build.built_for() == torch.__version__
    build.build()
    assert len(done) == 3


def test_the_c_library_is_made_without_torch(made, monkeypatch):
    done, _ = made
    monkeypatch.setattr(build, "installed_torch", lambda: None)
    assert build.build() == build.LIB and sorted(done) == ["libfa2.so", "libfa2_debug.so"]
    build.build(force=True)
    assert len(done) == 4 and not os.path.exists(build.TORCH_LIB)


def test_no_torch_is_found_where_there_is_none():
    code = "import sys; sys.modules['torch'] = None\nfrom attention_fa2_forward_03_gb300 import build\nassert build.installed_torch() is None"
    subprocess.run([sys.executable, "-c", code], check=True, cwd=build.ROOT)
    assert build.installed_torch() == (torch.__version__, os.path.dirname(torch.__file__))


def test_an_extension_that_does_not_compile_leaves_the_libraries(made):
    done, broken = made
    broken.add("g++")
    with pytest.raises(subprocess.CalledProcessError):
        build.build()
    assert sorted(done) == ["libfa2.so", "libfa2_debug.so"] and os.path.exists(build.LIB) and os.path.exists(build.DEBUG_LIB)


def test_an_extension_of_another_torch_is_made_again(made, monkeypatch):
    done, _ = made
    build.build()
    monkeypatch.setattr(build, "installed_torch", lambda: ("0.1", "/torch"))
    assert build.needs_build(build.TORCH_LIB)
    build.build()
    assert done[3:] == ["_kv4_torch.so"] and build.built_for() == "0.1"
    # and is not loaded as it is
    monkeypatch.setattr(fa2, "_kv4_mod", None)
    monkeypatch.setattr(fa2, "KV4_TORCH_LIB", build.TORCH_LIB)
    monkeypatch.setattr(fa2, "load", lambda: None)
    with pytest.raises(ImportError, match="built for torch 0.1"):
        fa2._kv4()
    os.remove(build.TORCH_LIB)
    with pytest.raises(ImportError, match="missing"):
        fa2._kv4()
