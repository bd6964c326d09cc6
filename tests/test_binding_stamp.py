"""CPU tests of the tensor binding's stamp: _bind.so reads torch's objects as the
torch that it was built with lays them out, so a file built for another torch or
Python is not loaded, and is built again."""
import os
import subprocess
import sys

import selective_state_space_selscan_b200 as ss
from selective_state_space_selscan_b200 import build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _python(code):
    r = subprocess.run([sys.executable, "-c", f"import sys; sys.path.insert(0, {ROOT!r})\n" + code],
                       capture_output=True, text=True, timeout=300)
    return r.stdout + r.stderr


def test_the_built_file_carries_the_stamp():
    import torch
    assert torch.__version__ in ss.bind_stamp()
    assert ss.bind_fits() and ss._binding()


def test_a_file_for_another_torch_is_not_loaded():
    out = _python(
        "import torch, warnings\n"
        "torch.__version__ = '1.0.0'\n"
        "import selective_state_space_selscan_b200 as ss\n"
        "with warnings.catch_warnings(record=True) as w:\n"
        "    warnings.simplefilter('always')\n"
        "    print('binding:', ss._binding(), [str(x.message) for x in w])\n"
        "print('loaded:', any(m.endswith('._bind') for m in sys.modules))\n"
        "print('mapped:', '_bind.so' in open('/proc/self/maps').read())\n")
    assert "binding: False" in out and "built for another torch" in out, out
    assert "loaded: False" in out and "mapped: False" in out, out


def test_a_missing_file_is_no_warning(tmp_path):
    assert not ss.bind_fits(str(tmp_path / "_bind.so"))


def test_a_file_for_another_torch_is_built_again(monkeypatch):
    ran = []

    def compiler(cmd, **kw):
        ran.append(cmd)
        raise subprocess.CalledProcessError(1, cmd)

    monkeypatch.setattr(build.subprocess, "check_call", compiler)
    assert build.build_bind() == build.BIND and not ran  # up to date
    monkeypatch.setattr(build, "bind_fits", lambda path: False)
    try:
        build.build_bind()
    except subprocess.CalledProcessError:
        pass
    assert len(ran) == 1 and any(ss.bind_stamp() in a for a in ran[0])


def test_build_without_headers_leaves_the_binding_out(monkeypatch, capsys):
    """The library itself needs no headers of torch's: the build goes on."""
    assert all(os.path.isdir(d) for d in build.bind_headers()) and build.bind_headers()
    real = os.path.exists
    for missing in ("python_variable.h", "Python.h"):
        monkeypatch.setattr(build.os.path, "exists",
                            lambda p, m=missing: not str(p).endswith(m) and real(p))
        assert build.bind_headers() == []
        assert build.build_bind(force=True) is None
        assert "ctypes" in capsys.readouterr().err
