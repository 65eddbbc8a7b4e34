"""CPU tests of build.py with stand-ins for the compilers (and for torch), in a copy of the package:
what is built, and when, on machines that lack one of them."""
import os
import shutil
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PKG = "block_swizzle_tile_amd"
COMPILER = """#!/bin/sh
echo "$0" >> "%s/calls"
while [ "$#" -gt 0 ]; do
  if [ "$1" = -o ]; then : > "$2"; fi
  shift
done
"""


@pytest.fixture
def tree(tmp_path):
    """A copy of the package's sources; bin/ has a hipcc and a g++ that only make their output files."""
    for d in (PKG, "include"):
        shutil.copytree(os.path.join(ROOT, d), tmp_path / d,
                        ignore=shutil.ignore_patterns("*.so*", "_build*", "__pycache__"))
    for d in ("bin", "empty", "lib"):
        (tmp_path / d).mkdir()
    for c in ("hipcc", "g++"):
        (tmp_path / "bin" / c).write_text(COMPILER % tmp_path)
        (tmp_path / "bin" / c).chmod(0o755)
    return tmp_path


def fake_torch(tree, version):
    """A torch of that version (None: one that cannot be imported)."""
    t = tree / "lib" / "torch"
    shutil.rmtree(t, ignore_errors=True)
    (t / "utils").mkdir(parents=True)
    (t / "utils" / "__init__.py").write_text("")
    (t / "utils" / "cpp_extension.py").write_text("def include_paths():\n    return []\n")
    (t / "__init__.py").write_text(
        "raise ImportError('no torch here')\n" if version is None else
        "__version__ = %r\nclass _C:\n    _GLIBCXX_USE_CXX11_ABI = True\n" % version)


def run(tree, code="build.build()", path="bin"):
    env = dict(os.environ, HIPCC=str(tree / "bin" / "hipcc"), PYTHONPATH=str(tree / "lib"),
               PYTHONDONTWRITEBYTECODE="1", PATH="%s:/usr/bin:/bin" % (tree / path))
    if path == "empty":
        env["PATH"] = str(tree / path)
    (tree / "calls").write_text("")
    r = subprocess.run([sys.executable, "-c", "from %s import build; %s" % (PKG, code)], cwd=tree,
                       env=env, capture_output=True, text=True, timeout=60)
    calls = [os.path.basename(c) for c in (tree / "calls").read_text().split()]
    return r, calls, sorted(f for f in os.listdir(tree / PKG) if f.endswith(".so"))


def test_library_without_torch(tree):
    """libbst.so takes hipcc alone."""
    fake_torch(tree, None)
    r, calls, libs = run(tree)
    assert r.returncode == 0, r.stderr
    assert libs == ["libbst.so"] and "g++" not in calls and "no torch here" in r.stderr


def test_library_without_host_compiler(tree):
    """With torch but no g++ libbst.so is made all the same, and the rest is an error."""
    fake_torch(tree, "9.8")
    r, calls, libs = run(tree, path="empty")
    assert libs == ["libbst.so"]
    assert r.returncode != 0 and "RuntimeError: _block_fast was not built" in r.stderr


def test_extension_goes_by_torch(tree):
    """Another torch gets an extension of its own; the same one is not built again."""
    tag = sys.implementation.cache_tag
    fake_torch(tree, "9.8+rocm")
    r, calls, libs = run(tree)
    assert r.returncode == 0 and calls.count("g++") == 1, r.stderr
    assert libs == ["_block_fast-%s-torch9.8+rocm.so" % tag, "libbst.so"]
    again = "build.build(force=False)"
    r, calls, libs = run(tree, again)
    assert r.returncode == 0 and calls == [], (calls, r.stderr)
    fake_torch(tree, "9.9")
    r, calls, libs = run(tree, again)
    assert r.returncode == 0 and calls == ["g++"], (calls, r.stderr)
    assert "_block_fast-%s-torch9.9.so" % tag in libs


def test_the_loader_wants_its_own_torch():
    import torch
    from block_swizzle_tile_amd import block
    name = os.path.basename(block.FAST_PATH)
    assert torch.__version__ in name and sys.implementation.cache_tag in name
