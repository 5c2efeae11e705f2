"""CPU: what build() needs and when it compiles again."""
import os
import shutil
import subprocess
import sys

import sparse_mla_attention_fp8_gb300 as smla

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_the_library_needs_no_torch(tmp_path):
    """Without torch there is no Python binding of the paged operators, and everything else."""
    smla.build()
    code = f"""
import sys
sys.modules["torch"] = None  # as if it were not installed
sys.path.insert(0, {ROOT!r})
import sparse_mla_attention_fp8_gb300 as smla
smla.BINDING_PATH = {str(tmp_path / "_binding.so")!r}
smla.LIB_PATH = {str(tmp_path / "libsmla.so")!r}
smla.build()
assert smla.lib().smla_version() == 100
"""
    subprocess.run([sys.executable, "-c", code], check=True)
    assert (tmp_path / "libsmla.so").exists() and not (tmp_path / "_binding.so").exists()


def test_a_binding_that_does_not_compile_leaves_the_library(tmp_path, monkeypatch):
    smla.build()
    monkeypatch.setattr(smla, "BINDING_PATH", str(tmp_path / "_binding.so"))
    monkeypatch.setattr(smla, "LIB_PATH", str(tmp_path / "libsmla.so"))
    monkeypatch.setattr(smla, "_binding_command", lambda out: ["false"])
    try:
        smla.build()
        raise AssertionError("no error")
    except smla.SmlaError as e:
        assert "false failed" in str(e)
    assert (tmp_path / "libsmla.so").exists()


def test_the_binding_follows_the_installed_torch(tmp_path, monkeypatch):
    """Compiled against another torch, it is compiled again."""
    smla.build()
    binding = tmp_path / "_binding.so"
    shutil.copy(smla.BINDING_PATH, binding)
    calls = []
    monkeypatch.setattr(smla, "BINDING_PATH", str(binding))
    monkeypatch.setattr(smla, "_BINDING_STAMP", str(tmp_path / "binding.txt"), raising=False)
    monkeypatch.setattr(smla, "_binding_command", lambda out: calls.append(out) or ["cp", str(binding), out])
    (tmp_path / "binding.txt").write_text("torch 0.1, python 3")
    smla.build()
    assert len(calls) == 1
    smla.build()
    assert len(calls) == 1
