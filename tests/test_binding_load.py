"""The compiled short way to the calls around the linear is optional: where its module was
not built, was built for another torch or Python, or is damaged, every call goes through
ctypes and the library works as without it."""
import os
import shutil
import subprocess
import sys

import pytest

import w4a4_mxfp4_quantize_b200 as mq

PACKAGE = os.path.dirname(os.path.abspath(mq.__file__))


@pytest.fixture
def copy(tmp_path):
    """The package with its library, without the compiled module; runs code on it."""
    mq.build()
    root = tmp_path / "w4a4_mxfp4_quantize_b200"
    root.mkdir()
    shutil.copy(os.path.join(PACKAGE, "__init__.py"), root)
    os.symlink(os.path.join(PACKAGE, "csrc"), root / "csrc")
    os.symlink(os.path.join(os.path.dirname(PACKAGE), "include"), tmp_path / "include")
    shutil.copy(os.path.join(PACKAGE, "libmacaq.so"), root)  # newer than the sources: not built again

    def run(code, **env):
        r = subprocess.run([sys.executable, "-c", "import w4a4_mxfp4_quantize_b200 as mq\n" + code], cwd=tmp_path,
                           env={**os.environ, "PYTHONPATH": str(tmp_path), **env}, capture_output=True, text=True,
                           timeout=300)
        assert r.returncode == 0, r.stdout[-1000:] + r.stderr[-3000:]
        return r.stdout + r.stderr

    run.root = root
    return run


def name():
    return os.path.basename(mq._BINDING_PATH)


WORKS = "assert mq.weight_bytes(1, 1024, 1024) == (1024 * 512, 1024 * 32) and mq._fast is None"


def test_absent_module(copy):
    copy(WORKS)


@pytest.mark.parametrize("content", [b"", b"not a library", b"\x7fELF" + bytes(60)])
def test_damaged_module_is_reported_and_left_out(copy, content):
    (copy.root / name()).write_bytes(content)
    assert "RuntimeWarning" in copy(WORKS)


def test_module_of_another_torch_is_not_loaded(copy):
    # a file for another torch or Python has another name: not ours, neither loaded nor reported
    other = "_binding.so"
    assert other != name()
    (copy.root / other).write_bytes(b"not a library")
    assert "Warning" not in copy(WORKS)


def test_the_name_says_what_the_module_was_built_for():
    import sysconfig

    import torch

    assert torch.__version__ in name() and sysconfig.get_config_var("SOABI") in name() and name().endswith(".so")


def test_module_that_cannot_be_compiled_leaves_the_library(copy):
    # no compiler on the path: the library is there, and build() says that the short way is not
    out = copy("mq.build()\n" + WORKS, PATH="/nonexistent")
    assert "RuntimeWarning" in out


def test_built_module_is_loaded():
    mq.build()
    mq.lib()
    assert mq._fast is not None
