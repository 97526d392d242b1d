"""What the build leaves behind where a part of it cannot be built."""
import os
import sysconfig

import pytest

from context_long_attention_ulysses_gb300 import build


@pytest.fixture
def small(tmp_path, monkeypatch):
    """A build of one translation unit into a folder of its own, with Python's headers taken from `include`."""
    include = tmp_path / "include"
    include.mkdir()
    monkeypatch.setattr(build, "BUILD", str(tmp_path))
    monkeypatch.setattr(build, "LIB", str(tmp_path / "libusp.so"))
    monkeypatch.setattr(build, "BINDING", str(tmp_path / os.path.basename(build.BINDING)))
    monkeypatch.setattr(build, "SOURCES", ["diag.cu"])
    paths = {**sysconfig.get_paths(), "include": str(include)}
    monkeypatch.setattr(build.sysconfig, "get_paths", lambda: paths)
    return include


def test_the_library_is_built_without_pythons_headers(small, capsys):
    assert build.build() == build.LIB and os.path.exists(build.LIB) and not os.path.exists(build.BINDING)
    assert "Python.h" in capsys.readouterr().err


def test_the_library_is_linked_before_a_binding_that_fails_is_reported(small):
    (small / "Python.h").write_text("#error not these\n")
    with pytest.raises(RuntimeError, match="not these"):
        build.build()
    assert os.path.exists(build.LIB) and not os.path.exists(build.BINDING)


def test_a_unit_that_fails_leaves_no_library(small, monkeypatch):
    monkeypatch.setattr(build, "FLAGS", [*build.FLAGS, "--no-such-flag"])
    with pytest.raises(RuntimeError, match="diag.cu"):
        build.build()
    assert not os.path.exists(build.LIB)


def test_a_module_is_for_the_python_that_it_was_built_for():
    """Another version builds its own, and does not load this one's."""
    assert os.path.basename(build.BINDING) == "uspbinding" + sysconfig.get_config_var("EXT_SUFFIX")
    assert sysconfig.get_config_var("EXT_SUFFIX") != ".so"
