"""What importing the package needs: no torch until a call does."""
import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def python(code, *options):
    return subprocess.run([sys.executable, *options, "-c", code], cwd=ROOT, capture_output=True, text=True,
                          timeout=300, env=dict(os.environ, PYTHONDONTWRITEBYTECODE="1"))


def test_star_import_without_torch():
    """-S leaves the installed packages, torch among them, out."""
    r = python("from block_swizzle_tile_amd import *\n"
               "s = make_sched(tile=(64, 64)); assert s.tile_m == 64 and LIB_PATH\n"
               "import sys; assert 'torch' not in sys.modules", "-S")
    assert r.returncode == 0, r.stderr


def test_star_import_with_torch():
    r = python("from block_swizzle_tile_amd import *\n"
               "import block_swizzle_tile_amd as b\n"
               "assert quant_block is b.block.quant_block and callable(grouped_weight_grad)\n"
               "assert 'weight_grad' in b.__all__ and 'gemm' in b.__all__")
    assert r.returncode == 0, r.stderr
