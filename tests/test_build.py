"""The build's order and where it looks for headers, without compiling."""
import os

import pytest

from fp8_scaled_matmul_amd import build


def test_library_is_linked_where_the_binding_does_not_compile(monkeypatch):
    """A user of the C ABI needs neither torch nor g++."""
    linked = []

    def no_compiler():
        raise FileNotFoundError("g++")

    monkeypatch.setattr(build, "_compile", lambda src: src + ".o")
    monkeypatch.setattr(build, "_compile_binding", no_compiler)
    monkeypatch.setattr(build, "_link", lambda cmd, out: linked.append(out))
    with pytest.raises(RuntimeError, match="is built, but not its extension module: g"):
        build.build()
    assert linked == [build.LIB]


def test_a_failing_source_is_named(monkeypatch):
    def fail(src):
        raise RuntimeError("hipcc failed for " + src)

    monkeypatch.setattr(build, "_compile", fail)
    monkeypatch.setattr(build, "_compile_binding", lambda: "binding.o")
    monkeypatch.setattr(build, "_link", lambda cmd, out: pytest.fail("nothing to link"))
    with pytest.raises(RuntimeError, match="hipcc failed"):
        build.build()


def test_hipcc_may_be_a_name_on_path(monkeypatch, tmp_path):
    """Headers are beside the compiler's folder, wherever a link to it lies."""
    rocm, elsewhere = tmp_path / "rocm", tmp_path / "elsewhere"
    (rocm / "bin").mkdir(parents=True)
    elsewhere.mkdir()
    (rocm / "bin" / "hipcc").write_text("#!/bin/sh\n")
    (rocm / "bin" / "hipcc").chmod(0o755)
    (elsewhere / "hipcc").symlink_to(rocm / "bin" / "hipcc")
    want = os.path.realpath(rocm / "include")
    for folder in (rocm / "bin", elsewhere):
        monkeypatch.setenv("PATH", str(folder))
        monkeypatch.setattr(build, "HIPCC", "hipcc")
        assert build._hip_include() == want
    monkeypatch.setattr(build, "HIPCC", str(rocm / "bin" / "hipcc"))
    assert build._hip_include() == want
