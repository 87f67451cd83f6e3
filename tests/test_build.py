"""The library builds without what only the Python binding needs."""
import os
import subprocess
import sys

import pytest

from linear_attention_fwd_gb300 import build as kbuild

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_library_builds_without_pytorch():
    kbuild.build()
    code = ("import sys, warnings; sys.modules['torch'] = None; warnings.simplefilter('always')\n"
            "from linear_attention_fwd_gb300 import build; print(build.build())")
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True)
    assert r.returncode == 0 and r.stdout.strip() == kbuild.LIB, r.stderr
    assert "_binding.so is not" in r.stderr
    assert os.path.exists(kbuild.BINDING)          # that of another interpreter's PyTorch is left alone


def test_library_builds_where_the_binding_does_not_compile(monkeypatch, tmp_path):
    """build() warns and returns the library, build_binding() raises, and a binding of other sources is gone."""
    kbuild.build()
    monkeypatch.setattr(kbuild, "BINDING", str(tmp_path / "_binding.so"))
    monkeypatch.setattr(kbuild, "BINDING_STAMP", str(tmp_path / "stamp_binding"), raising=False)
    monkeypatch.setenv("CXX", "/bin/false")
    (tmp_path / "_binding.so").write_text("of other sources")
    with pytest.warns(RuntimeWarning, match="_binding.so is not"):
        assert kbuild.build() == kbuild.LIB
    assert not os.path.exists(kbuild.BINDING)
    with pytest.raises(RuntimeError, match="false failed"):
        kbuild.build_binding()
    monkeypatch.setenv("CXX", str(tmp_path / "no_such_compiler"))
    with pytest.warns(RuntimeWarning, match="_binding.so is not"):
        assert kbuild.build() == kbuild.LIB
