"""GPU tests of the block-scaled operators over the whole range of scale bytes, of rows that hold NaN
beside the ones that count, and of sums cut into many slices.  References, tolerances and their
derivation: tests/test_gpu_block.py."""
import math

import pytest
import torch

import block_swizzle_tile_amd as bst
from gpu_util import say
from test_gpu_block import (BF, FF, HF, TILES, check_sum, cut_product, gen, grads, kept, operands,
                            ref_product, same_values, spans, wide)

pytestmark = pytest.mark.gpu

PARTS = {BF: 1, HF: 2, FF: 3}


# ------------------------------------------------------------ scale bytes ---
@pytest.mark.parametrize("tile", [(128, 128), (256, 256)])
@pytest.mark.parametrize("dtype", [BF, HF, FF])
def test_weight_grad_of_every_code_and_scale(dtype, tile):
    """All 256 codes under all 256 scale bytes, one row (and group) for each byte, times a gradient
    of one: the result is the restored bf16 value itself, NaN for byte 255 and for NaN codes."""
    q = torch.arange(256, device="cuda", dtype=torch.uint8).repeat(256, 1).view(torch.float8_e4m3fn)
    s = torch.arange(256, device="cuda", dtype=torch.uint8)[:, None].repeat(1, 2).contiguous()
    one = torch.ones(256, 8, device="cuda", dtype=dtype)
    gm = torch.ones(256, dtype=torch.int32, device="cuda")
    want = bst.dequant_block(q, s).double()
    assert bool(want[255].isnan().all()) and bool(want[:255, 0].isfinite().all())
    got = bst.grouped_weight_grad(q, s, one, gm, sched=bst.make_sched(tile=tile))
    bad = [e for e in range(256) if not all(same_values(got[e, :, n], want[e]) for n in (0, 7))]
    say("every code and scale", dtype, tile, "rows that differ:", bad)
    assert not bad
    for e in (0, 1, 127, 254, 255):      # the same without groups
        got = bst.weight_grad(q[e:e + 1], s[e:e + 1], one[:1], sched=bst.make_sched(tile=tile))
        assert same_values(got[:, 3], want[e]), e


def test_weight_grad_smallest_parts():
    """An fp32 gradient whose last bf16 part is 2^-133, the type's least value, arrives whole."""
    q = torch.ones(1, 16, device="cuda").to(torch.float8_e4m3fn)
    s = torch.full((1, 1), 127, dtype=torch.uint8, device="cuda")
    v = torch.tensor([[2.0 ** -110 * (1 + 2.0 ** -23), -2.0 ** -118 * (1 + 2.0 ** -15), 2.0 ** -133,
                       1.5 * 2.0 ** -126]], device="cuda")
    assert torch.equal(bst.weight_grad(q, s, v), v.expand(16, 4))


@pytest.mark.parametrize("tb", [False, True])
@pytest.mark.parametrize("tile", [(0, 0)] + TILES)
def test_product_nan_scales(tile, tb):
    """A NaN scale byte in one block makes its row (of A) or its block of columns (of B) NaN and
    nothing else, in plain and grouped products, on every kernel."""
    for M in (20, 40, 150):
        N, K = 300, 328
        for kinds in (("e8m0", "e8m0"), ("e8m0", "f32"), ("f32", "e8m0")):
            for out in (BF, FF):
                if out == FF and tile == (256, 256):
                    continue
                A, sa, B, sb = operands(M, N, K, tb, kinds, gen(M), G=2)
                ref, den = ref_product(A, sa, B[1], sb[1], tb)
                cut = cut_product(A, sa, B[1], sb[1], tb)
                nan = torch.zeros(M, N, dtype=torch.bool, device="cuda")
                if kinds[0] == "e8m0":
                    sa[M - 3, 1] = 255
                    nan[M - 3] = True
                if kinds[1] == "e8m0":
                    at = (2, 0) if tb else (0, 2)      # columns 256 ..
                    sb[1][at] = 255
                    nan[:, 256:] = True
                sched = None if tile == (0, 0) else bst.make_sched(tile=tile)
                gm = torch.tensor([0, M], dtype=torch.int32, device="cuda")
                say("nan scales", tile, tb, M, kinds, out)
                for C in (bst.gemm_block_scaled(A, B[1], sa, sb[1], trans_b=tb, out_dtype=out, sched=sched),
                          bst.grouped_gemm_block_scaled(A, B, gm, sa, sb, trans_b=tb, out_dtype=out,
                                                        sched=sched)):
                    assert torch.equal(C.isnan(), nan)
                    check_sum(C[~nan], ref[~nan], den[~nan], K, out, "", cut[~nan])


@pytest.mark.parametrize("tb", [False, True])
@pytest.mark.parametrize("tile", [(0, 0)] + TILES)
def test_product_extreme_scales(tile, tb):
    """Scale bytes at the type's ends whose product is in range: 2^-127 times 2^127, and 2^-127 (as
    a row of zeros has it) beside ordinary ones."""
    for M in (20, 40, 150):
        N, K = 136, 256
        A, sa, B, sb = operands(M, N, K, tb, ("e8m0", "e8m0"), gen(M + 1))
        A = A.clone()
        A.view(torch.uint8)[5] = 0
        for a, b in ((0, 254), (254, 0), (1, 254), (64, 190), (200, 54)):
            sa.fill_(a)
            sb.fill_(b)
            ref, den = ref_product(A, sa, B, sb, tb)
            for out in (BF, FF):
                if out == FF and tile == (256, 256):
                    continue
                say("extreme scales", tile, tb, M, a, b, out)
                sched = None if tile == (0, 0) else bst.make_sched(tile=tile)
                C = bst.gemm_block_scaled(A, B, sa, sb, trans_b=tb, out_dtype=out, sched=sched)
                check_sum(C, ref, den, K, out, str((a, b)), cut_product(A, sa, B, sb, tb))
                assert bool((C[5] == 0).all())


# ------------------------------------------------- what must not be read ---
def test_rows_outside_a_group_do_not_count():
    """NaN codes, scales and gradients behind the last group and in the neighbouring groups."""
    sizes, total, K, N = [70, 33, 200, 1], 400, 136, 72
    g = gen(8)
    q, s = kept(total, K, g)
    dY = grads(total, N, BF, g, True)
    gm = torch.tensor(sizes, dtype=torch.int32, device="cuda")
    W, sw = kept(4 * K, N, g)
    W = W.contiguous().view(torch.uint8)
    W = torch.nn.functional.pad(W, (0, -N % 16)).view(torch.float8_e4m3fn).view(4, K, -1)[..., :N]
    sw = sw[:8].view(4, 2, 1).contiguous()
    for keep, (lo, hi) in enumerate(spans(sizes, total)):
        other = torch.ones(total, dtype=torch.bool, device="cuda")
        other[lo:hi] = False
        q2, s2, d2 = q.clone(), s.clone(), dY.clone()
        q2 = torch.nn.functional.pad(q2.view(torch.uint8), (0, -K % 16)).view(q.dtype)[:, :K]
        q2.view(torch.uint8)[other] = 0x7f
        s2[other] = 255
        d2[other] = math.nan
        x, d = wide(q, s)[lo:hi], dY[lo:hi].double()
        say("neighbours", keep)
        for tile in ((0, 0), (128, 128), (256, 256)):
            dW = bst.grouped_weight_grad(q2, s2, d2, gm, sched=bst.make_sched(tile=tile, split_k=0))
            check_sum(dW[keep], x.t() @ d, x.abs().t() @ d.abs(), hi - lo, FF)
        for tile in [(0, 0)] + TILES:
            C = torch.full((total, N), 7.0, dtype=BF, device="cuda")
            bst.grouped_gemm_block_scaled(q2, W, gm, s2, sw, C, sched=bst.make_sched(tile=tile))
            ref, den = ref_product(q[lo:hi], s[lo:hi], W[keep], sw[keep], False)
            check_sum(C[lo:hi], ref, den, K, BF, "", cut_product(q[lo:hi], s[lo:hi], W[keep], sw[keep], False))
            assert bool((C[sum(sizes):] == 7).all())


# ------------------------------------------------------------ many slices ---
def slices(need, rows, N):
    return need // (rows * -(-N // 4) * 4 * 4)


@pytest.mark.parametrize("dtype", [BF, HF, FF])
def test_weight_grad_many_slices(dtype):
    """More slices than the last addition takes in its first pass over them (1 + 8 + 8)."""
    for M, K, N, split, want in [(8192, 64, 64, 0, 17), (2048, 40, 24, 0, 17), (4096, 72, 33, 17, 17),
                                 (4096, 16, 130, 25, 25), (8192, 136, 40, 33, 33), (4100, 24, 72, 64, 64)]:
        g = gen(M + split)
        q, s = kept(M, K, g)
        dY = grads(M, N, dtype, g, True)
        sched = bst.make_sched(split_k=split, offset=2)
        n = slices(bst.block_workspace_bytes(1, 1, M, N, K, sched), K, N)
        say("many slices", dtype, M, K, N, split, n)
        assert n >= want if split == 0 else n == want
        x, add = wide(q, s), torch.randn(K, N, generator=g, device="cuda")
        ref, den = x.t() @ dY.double() + add.double(), x.abs().t() @ dY.double().abs() + add.double().abs()
        check_sum(bst.weight_grad(q, s, dY, add=add, sched=sched), ref, den, PARTS[dtype] * M + 1, FF)
        if split == 0:
            check_sum(bst.weight_grad(q, s, dY, add=add), ref, den, PARTS[dtype] * M + 1, FF)


@pytest.mark.parametrize("tb", [False, True])
def test_product_many_slices(tb):
    for blocks, K, split in [(64, 8192, 64), (66, 8448, 33), (50, 6390, 25), (34, 4352, 17), (57, 7201, 19)]:
        M, N = 70, 200
        A, sa, B, sb = operands(M, N, K, tb, ("f32", "e8m0"), gen(K))
        ref, den = ref_product(A, sa, B, sb, tb)
        cut = cut_product(A, sa, B, sb, tb)
        for tile in TILES:
            for out in (BF, FF):
                if out == FF and tile == (256, 256):
                    continue
                sched = bst.make_sched(tile=tile, split_k=split)
                n = slices(bst.block_workspace_bytes(3 if tb else 0, 1, M, N, K, sched), M, N)
                say("many slices", tb, blocks, K, split, tile, out, n)
                assert n == split
                C = bst.gemm_block_scaled(A, B, sa, sb, trans_b=tb, out_dtype=out, sched=sched)
                check_sum(C, ref, den, K, out, str((tile, split)), cut)


@pytest.mark.parametrize("dtype", [BF, FF])
@pytest.mark.parametrize("sizes", [[500, 420, 777, 303], [1900, 3, 0, 70, 27], [640] * 3, [4096]])
def test_grouped_weight_grad_many_slices(sizes, dtype):
    """Groups cut into three slices and more; where one group has nearly all rows, the others' later
    slices are empty."""
    total, G, K, N = sum(sizes) + 9, len(sizes), 136, 72
    g = gen(total)
    q, s = kept(total, K, g)
    dY = grads(total, N, dtype, g, True)
    gm = torch.tensor(sizes, dtype=torch.int32, device="cuda")
    x, add = wide(q, s), torch.randn(G, K, N, generator=g, device="cuda")
    stages = -(-(-(-total // G)) // 64)
    for tile in ((128, 128), (256, 256)):
        for split in (3, 5, 19):
            sched = bst.make_sched(tile=tile, split_k=split)
            n = slices(bst.block_workspace_bytes(2, G, total, N, K, sched), G * K, N)
            say("grouped slices", sizes, dtype, tile, split, n)
            assert n == min(split, stages) and n >= 3
            dW = bst.grouped_weight_grad(q, s, dY, gm, add=add, sched=sched)
            for k, (lo, hi) in enumerate(spans(sizes, total)):
                a, b = x[lo:hi], dY[lo:hi].double()
                check_sum(dW[k], a.t() @ b + add[k].double(), a.abs().t() @ b.abs() + add[k].double().abs(),
                          PARTS[dtype] * (hi - lo) + 1, FF, "group %d" % k)


def test_restore_with_32_bit_scales():
    """A code times a 32-bit scale is rounded to fp32, then to the type."""
    g = gen(6)
    q = torch.arange(256, device="cuda", dtype=torch.uint8).repeat(64, 2).view(torch.float8_e4m3fn)
    for block_rows in (1, 128):
        s = torch.exp(3 * torch.randn(64 if block_rows == 1 else 1, 4, generator=g, device="cuda"))
        f = s.repeat_interleave(128, 1).expand(64, 512)
        for out in (BF, HF, FF):
            m = torch.finfo(out).max
            v = q.float() * f
            want = torch.where(v.isnan(), v, v.clamp(-m, m)).to(out)
            assert same_values(bst.dequant_block(q, s, out_dtype=out, block_rows=block_rows), want), out
