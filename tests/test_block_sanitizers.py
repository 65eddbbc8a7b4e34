"""The host code of the block-scaled operators (block.hip: checks, plans, workspace sizes) under
AddressSanitizer and UndefinedBehaviorSanitizer, as tests/test_sanitizers.py does it for bst.hip:
both are built with the host sanitizers, linked with the other objects of the normal build, and
driven by the C-ABI tests, which need no GPU."""
import os
import subprocess
import sys

import pytest

from test_sanitizers import CSRC, HIPCC, OBJ, ROOT, SAN_OPTS, _clang_asan_runtime, _env, _reports


def test_block_abi_under_sanitizers(tmp_path):
    from block_swizzle_tile_amd import build
    checked = ["bst.hip", "block.hip"]
    objs = [os.path.join(OBJ, s.replace(".hip", ".o")) for s in build.SOURCES if s not in checked]
    if not all(os.path.exists(o) for o in objs):
        pytest.skip("the objects of the normal build are missing (python -m block_swizzle_tile_amd.build)")
    tmp = str(tmp_path)
    lib = os.path.join(tmp, "libbst_san.so")
    mine = [os.path.join(tmp, s.replace(".hip", ".o")) for s in checked]
    # the sanitizers go to the host half only
    running = [subprocess.Popen([HIPCC, "--offload-arch=gfx950", "-O1", "-g", "-std=c++17", "-fPIC",
                                 "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
                                 "-Wno-pass-failed"] + SAN_OPTS +
                                ["-I", os.path.join(ROOT, "include"), "-c", os.path.join(CSRC, s),
                                 "-o", o], stderr=subprocess.DEVNULL) for s, o in zip(checked, mine)]
    assert all([p.wait() == 0 for p in running])
    subprocess.check_call([HIPCC, "--offload-arch=gfx950", "-shared", "-fPIC"] + mine + objs + ["-o", lib])
    r = subprocess.run([sys.executable, "-m", "pytest", "-x", "-q", "-p", "no:cacheprovider", "-k", "not hazards",
                        os.path.join(ROOT, "tests", "test_block_abi.py"),
                        os.path.join(ROOT, "tests", "test_abi.py")], cwd=ROOT,
                       env=_env(tmp, _clang_asan_runtime(), BST_LIB=lib), capture_output=True, text=True,
                       timeout=600)
    assert r.returncode == 0 and " passed" in r.stdout, (r.stdout[-2000:], _reports(tmp))
    assert not _reports(tmp), _reports(tmp)
