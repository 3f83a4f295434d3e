"""The build: the C library does not depend on what only the calls from Python need."""

import os
import sysconfig

import pytest

from paged_kv_gqa_14_gb300 import _lib
from paged_kv_gqa_14_gb300 import build as B


def test_the_extension_is_named_for_this_interpreter():
    # another Python version looks for another file, and builds its own
    assert B.CALL.endswith(sysconfig.get_config_var("EXT_SUFFIX")) and len(os.path.basename(B.CALL)) > len("_q8call.so")
    assert _lib.CALL == B.CALL


@pytest.mark.parametrize("compiler", ("/bin/false", "/no/such/compiler"))
def test_the_library_is_built_without_the_extension(tmp_path, monkeypatch, capfd, compiler):
    B.build()
    call = str(tmp_path / os.path.basename(B.CALL))
    monkeypatch.setattr(B, "CALL", call)
    monkeypatch.setattr(_lib, "CALL", call)
    monkeypatch.setattr(_lib, "_q8call", None)
    monkeypatch.setattr(B, "c_compiler", lambda: compiler)
    assert B.build() == B.LIB and os.path.exists(B.LIB) and not os.path.exists(call)
    assert "not built" in capfd.readouterr().out
    with pytest.raises(RuntimeError, match="extension not built"):
        _lib.q8call()
    monkeypatch.undo()
    assert _lib.load().pkv_version() >= 100 and _lib.q8call() is not None
