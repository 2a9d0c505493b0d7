"""A library that does not fit the binding is refused with a message when it is loaded."""
import subprocess

import pytest

import paged_gqa_decode_05_gb300 as pda


@pytest.mark.parametrize("source", ["int pda_abi_version(void) { return 5; }", ""])
def test_a_library_without_an_entry_point(tmp_path, monkeypatch, source):
    src, so = tmp_path / "old.c", tmp_path / "libpda.so"
    src.write_text(source)
    subprocess.run(["gcc", "-shared", "-fPIC", "-o", str(so), str(src)], check=True)
    monkeypatch.setattr(pda, "_LIB", None)
    monkeypatch.setattr(pda, "_LIBPATH", str(so))
    for _ in range(2):  # and again: nothing of it is kept
        with pytest.raises(RuntimeError, match="libpda.so is older .*rebuild"):
            pda.lib()


def test_a_missing_library(tmp_path, monkeypatch):
    monkeypatch.setattr(pda, "_LIB", None)
    monkeypatch.setattr(pda, "_LIBPATH", str(tmp_path / "libpda.so"))
    with pytest.raises(RuntimeError, match="missing"):
        pda.lib()
