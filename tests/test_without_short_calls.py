"""The extension _calls only saves host time: without it, or with one that does not
load (built for another torch), the library and every operator still work (CPU)."""
import os
import subprocess
import sys

import pytest

from precision_linear_amd import binding, build

HERE = os.path.dirname(os.path.abspath(binding.__file__))


@pytest.fixture(scope="module", autouse=True)
def built():
    if not os.path.exists(binding.library_path):
        build.build()


@pytest.mark.parametrize("extension", [None, b"not a shared library"])
def test_the_library_loads(tmp_path, extension):
    package = tmp_path / "precision_linear_amd"
    package.mkdir()
    for name in ("__init__.py", "binding.py", "libfp8_scaled_mm.so"):
        os.symlink(os.path.join(HERE, name), package / name)
    if extension:
        (package / "_calls.so").write_bytes(extension)
    code = ("import sys, warnings; sys.path.insert(0, sys.argv[1])\n"
            "with warnings.catch_warnings(record=True) as shown:\n"
            "    warnings.simplefilter('always')\n"
            "    from precision_linear_amd import binding\n"
            "assert binding.__file__.startswith(sys.argv[1]) and binding._calls is None\n"
            "print(len([w for w in shown if '_calls' in str(w.message)]), len(binding.config_names()))\n")
    r = subprocess.run([sys.executable, "-c", code, str(tmp_path)], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
    warned, configs = map(int, r.stdout.split())
    assert warned == (extension is not None) and configs == len(binding.config_names())


def test_lib_without_the_extension(monkeypatch):
    monkeypatch.setattr(binding, "_calls", None)
    monkeypatch.setattr(binding, "_lib", None)
    assert binding.lib().fp8_scaled_mm_num_configs() > 0


def test_a_build_whose_extension_fails_says_so_and_leaves_no_old_one(tmp_path, monkeypatch, capsys):
    old = tmp_path / "_calls.so"
    old.write_bytes(b"of an earlier build")
    monkeypatch.setattr(build, "CALLS", str(old))
    monkeypatch.setattr(build, "_calls_command", lambda out: [sys.executable, "-c", "raise SystemExit('no headers')"])
    build._build_calls(str(tmp_path / "new.so"), False)
    assert not old.exists()
    shown = capsys.readouterr().err
    assert "_calls" in shown and "no headers" in shown
