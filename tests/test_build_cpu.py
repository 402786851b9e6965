"""What the build needs: the library nvcc alone, the serving calls' marshalling module Python's and torch's headers too."""
import os
import subprocess
import sys

import pytest

from rank_weight_reconstruction_gb300 import build_lib


@pytest.fixture(scope="module", autouse=True)
def built():
    build_lib.build()


@pytest.mark.parametrize("lacking", ["Python.h", "torch", "compiler"])
def test_the_library_is_built_without_what_the_module_needs(monkeypatch, tmp_path, capsys, lacking):
    monkeypatch.setattr(build_lib, "MARSHAL_PATH", str(tmp_path / "_marshal.so"))
    if lacking == "Python.h":
        monkeypatch.setattr(build_lib.sysconfig, "get_paths", lambda: {"include": str(tmp_path)})
    elif lacking == "torch":
        monkeypatch.setattr(build_lib.importlib.util, "find_spec", lambda name: None)
    else:
        monkeypatch.delenv("CXX", raising=False)
        which = build_lib.shutil.which
        monkeypatch.setattr(build_lib.shutil, "which", lambda name: None if name in ("g++", "c++") else which(name))
    assert build_lib.build() == build_lib.LIB_PATH
    assert not os.path.exists(build_lib.MARSHAL_PATH) and "not built" in capsys.readouterr().err
    with pytest.raises(RuntimeError, match="not found"):
        build_lib.build_marshal()


def test_a_module_built_against_another_torch_is_not_up_to_date(monkeypatch):
    assert build_lib.marshal_up_to_date()
    monkeypatch.setattr(build_lib.importlib.metadata, "version", lambda name: "0.0")
    assert not build_lib.marshal_up_to_date()


def test_the_binding_says_that_the_module_is_missing():
    code = ("from rank_weight_reconstruction_gb300 import binding, build_lib\n"
            "build_lib.MARSHAL_PATH += '.gone'\n"
            "try:\n    binding.aq_kv_read(None, None)\n"
            "except RuntimeError as e:\n    print(e)\n")
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, cwd=build_lib.ROOT, timeout=300)
    assert "is missing: build it" in r.stdout, r.stdout + r.stderr
