"""The build with stand-ins for its compilers: the library needs hipcc alone, the compiled calls are left out where they
cannot be built, and a failure leaves no compiler running."""
import os
import stat
import sys
import time
import warnings

import pytest

from rotated_w4a8_group_amd import build as b

# writes what it was asked for; fails for a source whose name stands in FAIL, and takes a second for one in SLOW
COMPILER = r'''#!/bin/sh
for a in "$@"; do
  [ "$last" = -o ] && out=$a
  case "$a" in *"$FAIL") [ -n "$FAIL" ] && exit 3;; *"$SLOW") [ -n "$SLOW" ] && sleep 1;; esac
  last=$a
done
echo "$0" > "$out"
'''


@pytest.fixture
def tree(tmp_path, monkeypatch):
    for name in ("hipcc", "g++"):
        f = tmp_path / name
        f.write_text(COMPILER)
        f.chmod(f.stat().st_mode | stat.S_IXUSR)
    monkeypatch.setenv("HIPCC", str(tmp_path / "hipcc"))
    monkeypatch.setenv("CXX", str(tmp_path / "g++"))
    for name in ("FAIL", "SLOW"):
        monkeypatch.setenv(name, "")
    monkeypatch.setattr(b, "BUILD_DIR", str(tmp_path / "objects"))
    monkeypatch.setattr(b, "OUT", str(tmp_path / "libpq.so"))
    monkeypatch.setattr(b, "BINDING", str(tmp_path / "_binding.so"))
    (tmp_path / "_binding.so").write_text("an older one")
    return tmp_path


def test_both(tree):
    with warnings.catch_warnings():
        warnings.simplefilter("error")
        assert b.build() == str(tree / "libpq.so")
    assert (tree / "libpq.so").read_text().strip().endswith("hipcc") and (tree / "_binding.so").read_text().strip().endswith("g++")


@pytest.mark.parametrize("missing", ["g++", "torch", "headers"])
def test_without_what_the_compiled_calls_need(tree, monkeypatch, missing):
    if missing == "g++":
        monkeypatch.setenv("CXX", str(tree / "none"))
    elif missing == "torch":
        monkeypatch.setitem(sys.modules, "torch", None)
    else:
        monkeypatch.setenv("FAIL", "pq_binding.cpp")
    with pytest.warns(UserWarning, match="_binding.so is not built"):
        assert b.build() == str(tree / "libpq.so")
    assert (tree / "libpq.so").exists() and not (tree / "_binding.so").exists()


@pytest.mark.parametrize("source", ["pq_host.cpp", "pq_gemm.hip"])
def test_a_source_that_does_not_compile(tree, monkeypatch, source):
    """Raises after the others have ended, and leaves what was built before."""
    (tree / "libpq.so").write_text("an older one")
    monkeypatch.setenv("FAIL", source)
    monkeypatch.setenv("SLOW", "pq_matvec.hip")
    with pytest.raises(b.subprocess.CalledProcessError) as e:
        b.build()
    assert e.value.returncode == 3 and (tree / "libpq.so").read_text() == "an older one"
    assert (tree / "objects" / "pq_matvec.o").exists()


def test_no_compiler_outlives_an_exception(tree, monkeypatch):
    """An interrupt while the compilers run: they are ended before it goes on."""
    monkeypatch.setenv("SLOW", ".hip")
    started = []

    class Popen(b.subprocess.Popen):
        def __init__(self, *a, **kw):
            super().__init__(*a, **kw)
            started.append(self)

        def wait(self, *a, **kw):
            if not getattr(b, "interrupted", False):
                b.interrupted = True
                raise KeyboardInterrupt
            return super().wait(*a, **kw)
    monkeypatch.setattr(b, "interrupted", False, raising=False)
    monkeypatch.setattr(b.subprocess, "Popen", Popen)
    with pytest.raises(KeyboardInterrupt):
        b.build()
    assert len(started) >= len(b.SOURCES) and all(p.returncode is not None for p in started)
    for p in started:
        for _ in range(50):   # what a compiler had started ends with it
            try:
                os.killpg(p.pid, 0)
            except ProcessLookupError:
                break
            time.sleep(0.01)
        else:
            pytest.fail(f"{p.args[-1]} still has processes")
    assert not os.path.exists(b.OUT)


def test_the_compiled_calls_are_bound_to_a_library_of_their_version_only(monkeypatch):
    """Built for another version of the library, they are left out with a warning, whatever its entry points' addresses."""
    import rotated_w4a8_group_amd as pq
    assert pq._native()
    real = pq.lib()

    class Other:
        pq_abi_version = staticmethod(lambda: real.pq_abi_version() + 1)

        def __getattr__(self, name):
            return getattr(real, name)
    monkeypatch.setattr(pq, "lib", Other)
    monkeypatch.setattr(pq, "_fast", None)
    with pytest.warns(UserWarning, match="ABI version"):
        assert pq._native() is False
    with pytest.raises(TypeError):       # without a version they are not bound at all
        pq._binding.bind(pq._check, *[0] * 6)
