"""The C library builds where torch is not installed: nvcc alone is enough, and
the compiled calls of the torch layer are left out.  No GPU."""

import os
import stat
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SCRIPT = os.path.join(ROOT, "combine_get_layout_gb300", "build_lib.py")

# A compiler that makes an empty file of what it is asked for.
NVCC = """#!/bin/sh
echo "$@" >> "$CALLED"
while [ $# -gt 0 ]; do
  if [ "$1" = -o ]; then : > "$2"; fi
  shift
done
"""

BUILD = """
import importlib.util, os, sys
spec = importlib.util.spec_from_file_location("build_lib", sys.argv[1])
m = importlib.util.module_from_spec(spec)
spec.loader.exec_module(m)
m.OUT_DIR, m.BUILD_DIR = (os.path.join(sys.argv[2], d) for d in ("lib", "obj"))
m.LIB = os.path.join(m.OUT_DIR, "libep_gb300.so")
assert m.build() == m.LIB and m.up_to_date()
assert m.build() == m.LIB
print(sorted(os.listdir(m.OUT_DIR)), len(m.sources()))
"""


def tool(path, text):
    path.write_text(text)
    path.chmod(path.stat().st_mode | stat.S_IXUSR)
    return str(path)


def without_torch(args, env):
    """A Python that sees the standard library alone."""
    r = subprocess.run([sys.executable, "-S", "-E", *args], capture_output=True, text=True,
                       env=env, cwd=ROOT, timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr
    return r.stdout


def test_build_needs_nvcc_alone(tmp_path):
    env = dict(os.environ, NVCC=tool(tmp_path / "nvcc", NVCC), CALLED=str(tmp_path / "called"))
    bin_dir = tmp_path / "bin"
    bin_dir.mkdir()
    tool(bin_dir / "g++", "#!/bin/sh\nexit 1\n")
    env["PATH"] = str(bin_dir) + os.pathsep + env["PATH"]
    said = without_torch(["-c", BUILD, SCRIPT, str(tmp_path)], env)
    files, sources = said.rsplit(" ", 1)
    assert files == "['libep_gb300.so']"
    lines = (tmp_path / "called").read_text().splitlines()
    # one call a source and one to link, none of them on the second build
    assert len(lines) == int(sources) + 1


def test_script_runs_without_torch():
    from conftest import load_build_module

    lib = load_build_module().build()
    assert without_torch([SCRIPT], dict(os.environ)).strip() == lib


def test_torch_calls_are_built_where_torch_is():
    from conftest import load_build_module

    m = load_build_module()
    m.build()
    path = m.calls_path()
    assert os.path.exists(path) and os.path.dirname(path) == m.OUT_DIR
