"""CPU tests of include/bst_block.h: every declared function is exported, and host-side validation
rejects bad arguments with the documented status before touching the GPU (all pointers are fake or
NULL; no call reaches a launch).  Also the scalar-operand hazard check of the LDS-DMA instructions
in the generated code of the block-scaled products (tests/test_dma_hazards.py states the rule)."""
import ctypes
import os
import re
import subprocess

import pytest

import block_swizzle_tile_amd as bst
from block_swizzle_tile_amd import _lib, block

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "block_swizzle_tile_amd", "csrc")
P = 0x10000        # 16-byte aligned, never dereferenced
BF, HF, FF, E8 = _lib.BF16, _lib.F16, _lib.F32, block.E8M0


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(_lib.LIB_PATH):
        from block_swizzle_tile_amd import build
        build.build()
    return block._bound()


def test_exports_every_declared_symbol(L):
    src = open(os.path.join(ROOT, "include", "bst_block.h")).read()
    src = re.sub(r"/\*.*?\*/", "", src, flags=re.S)
    names = sorted(set(re.findall(r"\b(bst_[a-z_]+)\s*\(", src)))
    assert names == sorted(block.BLOCK_EXPORTS)
    for n in names:
        assert hasattr(L, n), n


def S(**kw):
    return ctypes.byref(bst.make_sched(**kw))


def quant(L, x=BF, M=8, K=256, br=1, X=P, ldx=None, Q=P, ldq=None, Sc=P, lds=None):
    return L.bst_quant_block(x, M, K, br, X, K if ldx is None else ldx, Q, K if ldq is None else ldq,
                             Sc, -(-K // 128) if lds is None else lds, None)


def dequant(L, x=BF, M=8, K=256, br=1, Q=P, ldq=None, s=E8, Sc=P, lds=None, X=P, ldx=None):
    return L.bst_dequant_block(x, M, K, br, Q, K if ldq is None else ldq, s, Sc,
                               -(-K // 128) if lds is None else lds, X, K if ldx is None else ldx, None)


def gemm(L, c=BF, tb=0, M=64, N=256, K=256, A=P, lda=None, sa=E8, SA=P, ldsa=2, B=P, ldb=None,
         sb=FF, SB=P, ldsb=2, C=P, ldc=None, sched=None, ws=None, wsb=0):
    return L.bst_gemm_block_scaled(c, tb, M, N, K, A, K if lda is None else lda, sa, SA, ldsa, B,
                                   (K if tb else N) if ldb is None else ldb, sb, SB, ldsb, C,
                                   N if ldc is None else ldc, sched, ws, wsb, None)


def grouped(L, G=4, gm=P, M=64, N=256, K=256, strideB=65536, strideSB=4, sched=None, **kw):
    a = dict(c=BF, tb=0, A=P, sa=E8, SA=P, B=P, sb=E8, SB=P, C=P, ldsa=2, ldsb=2)
    a.update(kw)
    return L.bst_grouped_gemm_block_scaled(a["c"], a["tb"], G, gm, M, N, K, a["A"], K, a["sa"],
                                           a["SA"], a["ldsa"], a["B"], N, strideB, a["sb"], a["SB"],
                                           a["ldsb"], strideSB, a["C"], N, sched, None)


def grad(L, dy=BF, dw=FF, M=64, N=128, K=256, Q=P, ldq=None, Sc=P, lds=2, dY=P, lddy=None, add=None,
         ldadd=0, dW=P, lddw=None, sched=None, ws=None, wsb=0):
    return L.bst_weight_grad(dy, dw, M, N, K, Q, K if ldq is None else ldq, Sc, lds, dY,
                             N if lddy is None else lddy, add, ldadd, dW, N if lddw is None else lddw,
                             sched, ws, wsb, None)


def ggrad(L, G=4, gm=P, M=64, N=128, K=256, add=None, ldadd=0, strideadd=0, dW=P, lddw=128,
          stridedw=32768, sched=None, ws=None, wsb=0):
    return L.bst_grouped_weight_grad(BF, FF, G, gm, M, N, K, P, K, P, 2, P, N, add, ldadd, strideadd,
                                     dW, lddw, stridedw, sched, ws, wsb, None)


def test_quant_refusals(L):
    assert quant(L, x=_lib.I8) == _lib.E_UNSUPPORTED
    assert quant(L, br=2) == _lib.E_UNSUPPORTED
    assert quant(L, M=-1) == _lib.E_INVAL
    assert quant(L, K=1 << 31) == _lib.E_INVAL
    assert quant(L, M=1 << 30, K=1024) == _lib.E_INVAL              # more than 2^31 - 1 blocks
    assert quant(L, ldx=255) == _lib.E_INVAL
    assert quant(L, ldq=255) == _lib.E_INVAL
    assert quant(L, lds=1) == _lib.E_INVAL
    assert quant(L, ldx=1 << 32) == _lib.E_INVAL
    for k in ("X", "Q", "Sc"):
        assert quant(L, **{k: None}) == _lib.E_INVAL
        assert dequant(L, **{k: None}) == _lib.E_INVAL
    assert quant(L, X=P + 1) == _lib.E_ALIGN
    assert quant(L, x=FF, X=P + 2) == _lib.E_ALIGN
    assert dequant(L, s=BF) == _lib.E_UNSUPPORTED
    assert dequant(L, s=FF, Sc=P + 2) == _lib.E_ALIGN
    assert dequant(L, X=P + 1) == _lib.E_ALIGN
    assert quant(L, M=0, X=None, Q=None, Sc=None) == _lib.OK        # nothing to do
    assert dequant(L, K=0, X=None, Q=None, Sc=None) == _lib.OK
    assert b"block_rows" in (quant(L, br=3), L.bst_last_error())[1]


def test_gemm_refusals(L):
    assert gemm(L, c=_lib.I32) == _lib.E_UNSUPPORTED
    assert gemm(L, tb=2) == _lib.E_INVAL
    assert gemm(L, N=-1) == _lib.E_INVAL
    assert gemm(L, sa=BF) == _lib.E_UNSUPPORTED
    assert gemm(L, sb=_lib.I8) == _lib.E_UNSUPPORTED
    for k in ("A", "B", "C", "SA", "SB"):
        assert gemm(L, **{k: None}) == _lib.E_INVAL
    assert gemm(L, lda=240) == _lib.E_INVAL
    assert gemm(L, lda=257) == _lib.E_ALIGN
    assert gemm(L, A=P + 8) == _lib.E_ALIGN
    assert gemm(L, B=P + 4) == _lib.E_ALIGN
    assert gemm(L, ldb=264) == _lib.E_ALIGN
    assert gemm(L, C=P + 1) == _lib.E_ALIGN
    assert gemm(L, SB=P + 1) == _lib.E_ALIGN                        # fp32 scales
    assert gemm(L, ldsa=1) == _lib.E_INVAL
    assert gemm(L, tb=1, ldsb=1) == _lib.E_INVAL
    assert gemm(L, lda=8 << 20) == _lib.E_UNSUPPORTED               # 256 rows span 2 GiB
    assert gemm(L, ldb=16 << 20) == _lib.E_UNSUPPORTED
    assert gemm(L, ldsa=8 << 20) == _lib.E_UNSUPPORTED
    assert gemm(L, ldc=255) == _lib.E_INVAL
    assert gemm(L, ldc=1 << 40) == _lib.E_INVAL
    assert gemm(L, sched=S(tile=(96, 96))) == _lib.E_UNSUPPORTED
    assert gemm(L, c=FF, sched=S(tile=(256, 256))) == _lib.E_UNSUPPORTED    # 16-bit outputs only
    assert gemm(L, sched=S(offset=0)) == _lib.E_INVAL
    assert gemm(L, sched=S(direction=3)) == _lib.E_INVAL
    assert gemm(L, sched=S(split_k=65)) == _lib.E_INVAL
    assert gemm(L, sched=S(tile_k=64)) == _lib.E_UNSUPPORTED
    for k in ("grid", "path", "shuffle_k", "dynamic", "preload"):
        assert gemm(L, sched=S(**{k: 1})) == _lib.E_UNSUPPORTED
    assert gemm(L, M=0, A=None, B=None, C=None) == _lib.OK
    assert gemm(L, N=0, A=None, B=None, C=None) == _lib.OK


def test_workspace(L):
    s = bst.make_sched(tile=(64, 128), split_k=2)
    need = L.bst_block_workspace_bytes(0, 1, 64, 250, 256, ctypes.byref(s))
    assert need == 2 * 64 * 252 * 4
    assert gemm(L, N=250, ldb=256, sched=ctypes.byref(s)) == _lib.E_WORKSPACE
    assert gemm(L, N=250, ldb=256, sched=ctypes.byref(s), ws=P, wsb=need - 1) == _lib.E_WORKSPACE
    assert gemm(L, N=250, ldb=256, sched=ctypes.byref(s), ws=P + 4, wsb=need) == _lib.E_ALIGN
    g = bst.make_sched(tile=(128, 128), split_k=3)
    need = L.bst_block_workspace_bytes(2, 4, 2048, 128, 256, ctypes.byref(g))
    assert need == 3 * 4 * 256 * 128 * 4
    assert ggrad(L, M=2048, sched=ctypes.byref(g)) == _lib.E_WORKSPACE
    assert L.bst_block_workspace_bytes(4, 1, 1, 1, 1, None) == 0
    assert b"kind" in L.bst_last_error()
    assert L.bst_block_workspace_bytes(2, 0, 1, 1, 1, None) == 0
    assert L.bst_block_workspace_bytes(0, 1, 1, 512, 16384, None) > 0
    assert L.bst_block_workspace_bytes(3, 1, 1, 512, 16384, None) == 0    # few rows: one launch
    assert L.bst_block_workspace_bytes(0, 1, 1, 512, 2048, None) == 0
    # partial sums past what the last addition indexes are refused, not wrapped
    g = bst.make_sched(tile=(128, 128), split_k=2)
    assert L.bst_block_workspace_bytes(2, 1024, 1 << 20, (1 << 31) - 1, (1 << 31) - 1, ctypes.byref(g)) == 0
    assert L.bst_block_workspace_bytes(1, 1, 1 << 20, 1 << 20, 1 << 20, ctypes.byref(g)) == 0
    assert L.bst_block_workspace_bytes(0, 1, 64, 0, 4096, None) == 0
    # a split never has an empty slice: 3 blocks of K cut 8 ways are 3 slices
    s = bst.make_sched(tile=(64, 128), split_k=8)
    assert L.bst_block_workspace_bytes(0, 1, 64, 256, 384, ctypes.byref(s)) == 3 * 64 * 256 * 4


def test_grouped_refusals(L):
    assert grouped(L, G=0) == _lib.E_INVAL
    assert grouped(L, G=1025) == _lib.E_INVAL
    assert grouped(L, gm=None) == _lib.E_INVAL
    assert grouped(L, gm=P + 2) == _lib.E_ALIGN
    assert grouped(L, strideB=8) == _lib.E_ALIGN
    assert grouped(L, strideB=-16) == _lib.E_INVAL
    assert grouped(L, strideSB=-1) == _lib.E_INVAL
    assert grouped(L, sched=S(split_k=2)) == _lib.E_UNSUPPORTED
    assert grouped(L, M=0) == _lib.OK


def test_grad_refusals(L):
    assert grad(L, dy=_lib.E4M3) == _lib.E_UNSUPPORTED
    assert grad(L, dw=_lib.I32) == _lib.E_UNSUPPORTED
    for k in ("Q", "Sc", "dY", "dW"):
        assert grad(L, **{k: None}) == _lib.E_INVAL
    assert grad(L, ldq=264) == _lib.E_ALIGN
    assert grad(L, dY=P + 1) == _lib.E_ALIGN
    assert grad(L, dW=P + 2) == _lib.E_ALIGN
    assert grad(L, lds=1) == _lib.E_INVAL
    assert grad(L, lddy=127) == _lib.E_INVAL
    assert grad(L, lddw=127) == _lib.E_INVAL
    assert grad(L, add=P, ldadd=127) == _lib.E_INVAL
    assert grad(L, add=P + 1, ldadd=128) == _lib.E_ALIGN
    assert grad(L, sched=S(tile=(128, 256))) == _lib.E_UNSUPPORTED
    assert grad(L, sched=S(tile_k=128)) == _lib.E_UNSUPPORTED
    assert grad(L, K=0, Q=None, Sc=None, dW=None) == _lib.OK
    assert ggrad(L, G=0) == _lib.E_INVAL
    assert ggrad(L, gm=None) == _lib.E_INVAL
    assert ggrad(L, stridedw=32767) == _lib.E_INVAL                 # groups of dW overlap
    assert ggrad(L, add=P, ldadd=128, strideadd=-1) == _lib.E_INVAL


def test_python_refuses_cpu_tensors():
    import torch
    x = torch.zeros(4, 128)
    with pytest.raises(ValueError, match="GPU"):
        bst.quant_block(x)
    q = x.to(torch.float8_e4m3fn)
    s = torch.zeros(4, 1, dtype=torch.uint8)
    with pytest.raises(ValueError, match="GPU"):
        bst.dequant_block(q, s)
    with pytest.raises(ValueError, match="GPU"):
        bst.weight_grad(q, s, x)


@pytest.mark.parametrize("tu", ["block_gemm_plain_t", "block_gemm_plain_n", "block_gemm_grouped_t",
                                "block_gemm_grouped_n", "block"])
def test_dma_scalar_operand_hazards(tu, tmp_path):
    """Every `buffer_load ... lds` sits right behind an `s_nop` of at least 4."""
    asm = str(tmp_path / "a.s")
    subprocess.check_call(["/opt/rocm/bin/hipcc", "--offload-arch=gfx950", "-O3", "-std=c++17",
                           "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
                           "-Wno-pass-failed", "-I", os.path.join(ROOT, "include"),
                           "--cuda-device-only", "-S", os.path.join(CSRC, tu + ".hip"), "-o", asm],
                          stderr=subprocess.DEVNULL)
    lines = [re.split(r"\s*;", l)[0].strip() for l in open(asm)]
    lines = [l for l in lines if l and not l.startswith(".") and not l.endswith(":")]
    found = 0
    for prev, cur in zip(lines, lines[1:]):
        if cur.startswith("buffer_load") and cur.endswith("lds"):
            m = re.match(r"s_nop (\d+)", prev)
            assert m and int(m.group(1)) >= 4, (prev, cur)
            found += 1
    assert found >= 32


def test_refuses_more_than_a_launch_holds(L):
    big = (1 << 31) - 1
    # 2^24 + workgroups of 256 or 512 threads
    assert quant(L, M=1, K=big, br=128, ldx=1 << 31, ldq=1 << 31) == _lib.E_UNSUPPORTED
    assert b"one launch" in L.bst_last_error()
    assert gemm(L, M=big, N=16, K=16, lda=16, ldb=16, ldsa=1, ldsb=1) == _lib.E_UNSUPPORTED
    assert gemm(L, tb=1, M=1, N=big, K=16, lda=16, ldb=16, ldsa=1, ldsb=1) == _lib.E_UNSUPPORTED
    assert grouped(L, M=big, N=16, K=16) == _lib.E_UNSUPPORTED
    assert grad(L, M=64, N=1 << 20, K=1 << 20, ldq=1 << 20, lds=1 << 13, lddy=1 << 20,
                lddw=1 << 20, sched=S(tile=(128, 128), split_k=1)) == _lib.E_UNSUPPORTED
    # the last addition counts 16-byte pieces in 31 bits
    wide = dict(M=128, N=1 << 17, K=1 << 17, ldq=1 << 17, lds=1 << 10, sched=S(split_k=2))
    assert grad(L, **wide) == _lib.E_INVAL
    assert b"too large" in L.bst_last_error()
    # 64 rows of Q span 2 GiB
    assert grad(L, ldq=1 << 25) == _lib.E_UNSUPPORTED
    assert grad(L, ldq=(1 << 25) - 16, dY=None) == _lib.E_INVAL     # (accepted, and dY is not)


def test_gradient_tiles_past_64_bits(L):
    """1024 groups of the largest weights in 64 slices, 2^64 workgroups and more, are counted and
    refused (under the undefined-behaviour sanitizer too: test_block_sanitizers.py)."""
    big = (1 << 31) - 1
    for split in (0, 1, 2, 64):
        s = bst.make_sched(split_k=split)
        assert L.bst_block_workspace_bytes(2, 1024, 1 << 30, big, big, ctypes.byref(s)) == 0
    K = 1 << 20
    for split in (0, 1):
        assert L.bst_grouped_weight_grad(BF, FF, 1024, P, 1 << 22, K, K, P, K, P, K // 128, P, K, None, 0, 0,
                                         P, K, K * K, S(split_k=split), None, 0, None) == _lib.E_UNSUPPORTED
        assert b"one launch" in L.bst_last_error()
