"""CPU check of the block-scaled kernels' global and LDS addressing: builds
tests/native/check_block_bounds.hip host-only, plainly and with the host sanitizers, and requires it
to find every access inside its matrix and every stage covered once."""
import os
import subprocess

import pytest

from test_sanitizers import SAN_OPTS, _env, _reports

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("options", [["-O2"], ["-O1", "-g"] + SAN_OPTS], ids=["plain", "sanitized"])
def test_block_addressing_in_bounds(options, tmp_path):
    exe, tmp = str(tmp_path / "check_block_bounds"), str(tmp_path)
    subprocess.check_call(["/opt/rocm/bin/hipcc", "--cuda-host-only", "-std=c++17"] + options +
                          ["-I", os.path.join(ROOT, "include"),
                           "-I", os.path.join(ROOT, "block_swizzle_tile_amd", "csrc"),
                           os.path.join(ROOT, "tests", "native", "check_block_bounds.hip"),
                           "-o", exe], stderr=subprocess.DEVNULL)
    env = _env(tmp, "")
    env.pop("LD_PRELOAD")
    out = subprocess.run([exe], capture_output=True, text=True, timeout=300, env=env)
    assert out.returncode == 0 and "ALL OK" in out.stdout, (out.stdout[-2000:], _reports(tmp))
    assert not _reports(tmp), _reports(tmp)
