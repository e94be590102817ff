"""A library built from other sources is told from this one by the entry points
that it lacks, and by the version where both have them (CPU only)."""

import subprocess

import pytest

from activation_sparsity_fp4_amd import _lib


def _library(tmp_path, monkeypatch, names, version):
    """A shared object with the entry points given, each returning the version, as the library to load."""
    source = tmp_path / "stale.c"
    source.write_text("".join(f"int {n}(void) {{ return {version}; }}\n" for n in names))
    path = tmp_path / "libstale.so"
    subprocess.run(["gcc", "-shared", "-fPIC", str(source), "-o", str(path)], check=True)
    monkeypatch.setattr(_lib, "LIB_PATH", str(path))
    monkeypatch.setattr(_lib, "_lib", None)
    return str(path)


def test_an_older_library_is_named(tmp_path, monkeypatch):
    path = _library(tmp_path, monkeypatch, [n for n in _lib.SIGNATURES if "int8" not in n], 10)
    with pytest.raises(RuntimeError, match="sharq_quantize_int8") as e:
        _lib.lib()
    assert path in str(e.value) and "activation_sparsity_fp4_amd.build" in str(e.value)
    assert not isinstance(e.value, _lib.SharqError) and _lib._lib is None


def test_a_library_of_another_version_is_named(tmp_path, monkeypatch):
    path = _library(tmp_path, monkeypatch, list(_lib.SIGNATURES), 9)
    with pytest.raises(RuntimeError, match="version 9") as e:
        _lib.lib()
    assert path in str(e.value) and _lib._lib is None


def test_this_library_loads():
    assert _lib.lib().sharq_abi_version() == _lib.ABI_VERSION
