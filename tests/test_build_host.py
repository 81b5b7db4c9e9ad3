"""What the build needs, without compiling: the C libraries need no torch; the Python module is built where
there is a torch with CUDA, after them."""
import importlib.metadata
import os

import pytest

from io_aware_exact_fa2_gb300 import build as fa2_build


class Box:
    """A tree of its own, compilers that only write down what they are asked for, and any torch or none."""

    def __init__(self, tmp, monkeypatch):
        self.tmp, self.made, self.fail = tmp, [], False
        for name in ("LIB_PATH", "CACHE_LIB_PATH", "PAGED_LIB_PATH", "PY_MODULE_PATH"):
            monkeypatch.setattr(fa2_build, name, str(tmp / os.path.basename(getattr(fa2_build, name))))
        monkeypatch.setattr(fa2_build, "BUILD", str(tmp / "_build"))
        monkeypatch.setattr(fa2_build, "_compile", lambda src, *a: src)
        monkeypatch.setattr(fa2_build, "_link", self.link)
        monkeypatch.setattr(fa2_build, "nvcc", lambda: "/usr/local/cuda/bin/nvcc")
        monkeypatch.setattr(fa2_build.subprocess, "run", self.run)
        monkeypatch.setattr(fa2_build.importlib.util, "find_spec", lambda name: self.spec)
        monkeypatch.setattr(fa2_build.importlib.metadata, "version", self.version)
        self.torch(None)

    def torch(self, version, cuda=True):
        self.number, self.spec = version, None
        if version:
            root = self.tmp / "torch"
            (root / "lib").mkdir(parents=True, exist_ok=True)
            for name in ("libc10.so", "libc10_cuda.so"):
                (root / "lib" / name).unlink(missing_ok=True)
                if cuda or name == "libc10.so":
                    (root / "lib" / name).touch()
            self.spec = type("Spec", (), {"origin": str(root / "__init__.py")})

    def version(self, name):
        if self.number is None:
            raise importlib.metadata.PackageNotFoundError(name)
        return self.number

    def link(self, objs, out, bdir):
        self.made.append(os.path.basename(out))
        open(out, "w").close()

    def run(self, cmd, **kw):
        assert any(str(x).endswith(fa2_build.PY_SOURCE) for x in cmd)
        if not self.fail:
            open(cmd[cmd.index("-o") + 1], "w").close()
            self.made.append("module")
        return type("Done", (), {"returncode": int(self.fail), "stdout": "", "stderr": "no such header"})

    def build(self):
        self.made = []
        fa2_build.build()
        return self.made


LIBS = ["libfa2_gb300.so", "libfa2_cache_gb300.so", "libfa2_paged_gb300.so"]


@pytest.fixture
def box(tmp_path, monkeypatch):
    return Box(tmp_path, monkeypatch)


@pytest.mark.parametrize("version", [None, "2.11.0+cpu"])
def test_the_libraries_are_built_without_a_cuda_torch(box, capsys, version):
    box.torch(version, cuda=False)
    assert not fa2_build.is_fresh()
    assert box.build() == LIBS
    assert "torch" in capsys.readouterr().err
    assert fa2_build.is_fresh() and box.build() == []
    box.torch("2.11.0+cu130")             # one with CUDA is installed
    assert not fa2_build.is_fresh()
    assert box.build() == ["module"]


def test_the_module_follows_torch_and_the_libraries_do_not(box):
    box.torch("2.11.0+cu130")
    assert sorted(box.build()) == sorted(LIBS + ["module"])
    assert fa2_build.is_fresh() and box.build() == []
    box.torch("2.9.1+cu130")
    assert not fa2_build.is_fresh()
    assert box.build() == ["module"]


def test_a_module_that_does_not_compile_fails_behind_the_libraries(box):
    box.torch("2.11.0+cu130")
    box.fail = True
    with pytest.raises(RuntimeError, match="no such header"):
        box.build()
    assert box.made == LIBS
    box.fail = False
    assert box.build() == ["module"]
