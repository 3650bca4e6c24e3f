"""What the binding says about a library that it cannot use (CPU only)."""
import subprocess

import pytest

import block_sparse_video_int8_b200 as bsva


@pytest.mark.parametrize("source,message", [
    ("int bsva_abi_version(void) { return 4; }", "has ABI version 4, this binding expects 5"),
    ("int other(void) { return 0; }", "has ABI version None"),
    ("int bsva_abi_version(void) { return 5; } int bsva_device_checks(void) { return 0; }",
     "older sources: it has no .*bsva_paged_kv_write")])
def test_load_says_what_is_wrong_with_an_older_library(tmp_path, monkeypatch, source, message):
    # the version is compared before any other entry is looked up, and an entry that is missing is named
    src, lib = tmp_path / "old.c", tmp_path / "libold.so"
    src.write_text(source)
    subprocess.run(["gcc", "-shared", "-fPIC", "-o", str(lib), str(src)], check=True)
    monkeypatch.setattr(bsva, "_LIB", None)
    with pytest.raises(RuntimeError, match=message):
        bsva.load(str(lib))
    assert bsva._LIB is None
