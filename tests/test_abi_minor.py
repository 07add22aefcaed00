"""How a program tells a library that has the added entry points from an older one (CPU only)."""
import os
import re
import subprocess

import pytest

from quantized_expert_grouped_amd import abi

HEADER = os.path.join(os.path.dirname(__file__), "..", "include", "moe_prefill.h")


def test_minor_version():
    minor = int(re.search(r"#define MOE_ABI_MINOR (\d+)", open(HEADER).read()).group(1))
    assert abi.abi_minor() == minor >= 1


def test_an_older_library_is_named_as_such(tmp_path, monkeypatch):
    """One that exports version 7's first entry points only: the binding says what is missing."""
    src = tmp_path / "old.c"
    late = {n for n in abi.SIGNATURES if "mxfp4" in n or "balance" in n or n in ("moe_combine_bf16", "moe_abi_minor")}
    src.write_text("".join(f"int {n}(void) {{ return 7; }}\n" for n in abi.SIGNATURES if n not in late))
    path = str(tmp_path / "libold.so")
    subprocess.run(["gcc", "-shared", "-fPIC", str(src), "-o", path], check=True)
    monkeypatch.setattr(abi, "LIB_PATH", path)
    monkeypatch.setattr(abi, "_lib", None)
    with pytest.raises(RuntimeError, match="older than this binding.*moe_mxfp4_quantize.*build"):
        abi.lib()
