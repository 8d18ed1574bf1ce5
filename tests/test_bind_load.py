"""The marshalling extension is an extra: built for this Python and torch or not
used at all, and no call of the library depends on it."""
import os
import platform
import sys
import warnings

import pytest
import torch

import speculative_decoding_verification_81_gb300 as sv
from speculative_decoding_verification_81_gb300 import api
from speculative_decoding_verification_81_gb300 import build as svbuild


@pytest.fixture
def fresh(monkeypatch):
    """The binding as a new process finds it, with the library built."""
    svbuild.build()
    for name in ("_lib", "_bind", "_bound"):
        monkeypatch.setattr(api, name, None)


def test_built_for_this_python_and_torch(fresh, monkeypatch):
    here = svbuild.bind_path()
    assert os.path.exists(here)
    api.lib()
    assert api._native() is not None
    monkeypatch.setattr(torch, "__version__", "1.2.3+cu999")
    other = svbuild.bind_path()
    assert other != here and not svbuild.bind_up_to_date(other)
    for name in ("_lib", "_bind", "_bound"):
        monkeypatch.setattr(api, name, None)
    api.lib()
    assert api._native() is None  # another torch's file is not taken


@pytest.mark.parametrize("content", [b"", b"not a library", None])
def test_an_extension_that_does_not_import_is_left_aside(fresh, monkeypatch, tmp_path, content):
    path = tmp_path / "_sv_bind.so"
    if content is None:  # a library without the module in it
        path = svbuild.LIB_PATH
    else:
        path.write_bytes(content)
    monkeypatch.setattr(svbuild, "bind_path", lambda: str(path))
    with pytest.warns(UserWarning, match="without their extension"):
        api.lib()
    assert api._native() is None
    assert sv.status_string(sv.SV_OK).startswith("SV_OK")  # calls that never needed it
    with warnings.catch_warnings():
        warnings.simplefilter("error")
        api.lib()                                           # and no second surprise
    with pytest.raises(ValueError):                         # the interpreted checks take the paged-cache calls
        sv.sv_release_pages(*[torch.zeros(2, dtype=torch.int32)] * 2, torch.zeros((2, 3), dtype=torch.int32),
                            torch.zeros(9, dtype=torch.int32), torch.zeros(1, dtype=torch.int32), 16)


def test_a_build_that_fails_leaves_the_library_and_no_stale_extension(monkeypatch, tmp_path):
    svbuild.build()
    path, source = tmp_path / "_sv_bind.so", tmp_path / "broken.cpp"
    path.write_bytes(b"of an older source")
    os.utime(path, (1, 1))
    source.write_text("#error not today\n")
    monkeypatch.setattr(svbuild, "bind_path", lambda: str(path))
    monkeypatch.setattr(svbuild, "BIND_SOURCE", str(source))
    with pytest.warns(UserWarning, match="not today"):
        assert svbuild.build() == svbuild.LIB_PATH
    assert not path.exists()


def test_a_build_without_a_compiler_leaves_the_library(monkeypatch, tmp_path):
    svbuild.build()
    monkeypatch.setattr(svbuild, "bind_path", lambda: str(tmp_path / "_sv_bind.so"))
    monkeypatch.setenv("PATH", str(tmp_path))
    with pytest.warns(UserWarning, match="left out"):
        assert svbuild.build() == svbuild.LIB_PATH


def test_a_build_without_torch_leaves_the_library(monkeypatch):
    svbuild.build()
    monkeypatch.setitem(sys.modules, "torch", None)
    with pytest.warns(UserWarning, match="left out"):
        assert svbuild.build() == svbuild.LIB_PATH


def test_the_file_name_says_what_it_was_built_for():
    name = os.path.basename(svbuild.bind_path())
    assert "".join(c if c.isalnum() else "_" for c in torch.__version__) in name
    assert f"{sys.version_info[0]}{sys.version_info[1]}" in name and platform.machine() in name
