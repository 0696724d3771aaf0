"""The C library's build and load stand on nvcc alone; the holders' extension is built apart from it."""

import os
import subprocess
import sys

import pytest

from mixture_experts_decode_router_gb300 import binding as B
from mixture_experts_decode_router_gb300 import build as build_module

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture
def elsewhere(tmp_path, monkeypatch):
    """A build folder of the test's own, an nvcc that makes empty files, and no way to make the extension."""
    nvcc = tmp_path / "nvcc"
    nvcc.write_text('#!/bin/sh\nwhile [ $# -gt 0 ]; do [ "$1" = -o ] && : > "$2"; shift; done\n')
    nvcc.chmod(0o755)
    gxx = tmp_path / "bin" / "g++"
    gxx.parent.mkdir()
    gxx.write_text("#!/bin/sh\necho no headers >&2\nexit 1\n")
    gxx.chmod(0o755)
    monkeypatch.setenv("NVCC", str(nvcc))
    monkeypatch.setenv("PATH", f"{gxx.parent}:{os.environ['PATH']}")
    out = tmp_path / "out"
    monkeypatch.setattr(build_module, "BUILD", str(out))
    monkeypatch.setattr(build_module, "LIB", str(out / "libmoe_gb300.so"))
    monkeypatch.setattr(build_module, "EXT", str(out / "_moe_torch.so"))
    return out


def test_the_library_is_linked_without_the_extension(elsewhere):
    assert build_module.build() == str(elsewhere / "libmoe_gb300.so")
    assert (elsewhere / "libmoe_gb300.so").exists() and not (elsewhere / "_moe_torch.so").exists()
    assert not build_module._stale()               # nothing is left to do for it


def test_a_failed_extension_is_raised_where_it_is_wanted(elsewhere):
    with pytest.raises(RuntimeError, match="g\\+\\+ failed"):
        build_module.build_ext()
    with pytest.raises(RuntimeError, match="g\\+\\+ failed"):
        build_module.build_all()
    assert (elsewhere / "libmoe_gb300.so").exists()


def test_the_library_loads_without_torch(tmp_path):
    """In a process that has no torch, and with no extension built."""
    B.load()
    code = ("import sys; sys.modules['torch'] = None\n"
            "from mixture_experts_decode_router_gb300 import binding as B, build\n"
            f"build.EXT = {str(tmp_path / 'none.so')!r}\n"
            "B.load()\n"
            "assert B.moe_abi_version() == 2 and 'success' in B.moe_status_string(0)\n")
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr


@pytest.mark.parametrize("lang,std", [("c", "c99"), ("c", "c11"), ("c", "gnu99"), ("c++", "c++11"), ("c++", "c++17")])
def test_the_header_in_strict_compilers(lang, std, tmp_path):
    """Strict C99 and C++ take the header, with its matrices' second array under both names."""
    src = tmp_path / "use.c"
    src.write_text('#include "moe.h"\n'
                   "int main(void) {\n"
                   "    moe_qmat_t q = {0};\n"
                   "    const uint8_t z = 0;\n"
                   "    q.zero = &z;\n"
                   "    return (const void*)q.scale2 != (const void*)q.zero || sizeof(q) != 3 * sizeof(void*);\n"
                   "}\n")
    exe = tmp_path / "use"
    flags = ["-Wall", "-Wextra", "-Werror", "-pedantic-errors"] + (["-Wno-missing-field-initializers"] if lang == "c++" else [])
    subprocess.run(["gcc", "-x", lang, f"-std={std}", *flags, "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)],
                   check=True, capture_output=True)
    assert subprocess.run([str(exe)]).returncode == 0
