"""GPU tests of the block-scaled operators on views: odd bases and pitches of everything but codes,
codes at 16-byte offsets, weights and addends shared by all groups, and outputs of more than 2^31
values.  References, tolerances and their derivation: tests/test_gpu_block.py."""
import pytest
import torch

import block_swizzle_tile_amd as bst
from gpu_util import say
from test_gpu_block import (BF, FF, HF, KINDS, check_sum, cut_product, gen, kept, operands, ref_product,
                            same_values, scales, spans, wide)

pytestmark = pytest.mark.gpu


def inside(t, left, right, fill):
    """A copy of t inside a larger matrix whose other values are fill: (view, check that they still are)."""
    rows, cols = t.shape[-2:]
    big = torch.full((*t.shape[:-2], rows + 2, cols + left + right), fill, device=t.device).to(t.dtype)
    view = big[..., 1:-1, left:left + cols]
    view.copy_(t)

    def kept_():
        b = big.float()
        out = torch.ones_like(b, dtype=torch.bool)
        out[..., 1:-1, left:left + cols] = False
        return bool((b[out] == fill).all())
    return view, kept_


@pytest.mark.parametrize("left,right", [(1, 0), (3, 2), (0, 5), (8, 8)])
def test_views(left, right):
    M, N, K = 70, 200, 264
    for kinds in KINDS:
        for tb in (False, True):
            for tile, split in (((0, 0), 0), ((64, 128), 1), ((64, 128), 2), ((256, 256), 1)):
                for m in (M, 20):
                    g = gen(left * 7 + right)
                    A, sa, B, sb = operands(m, N, K, tb, kinds, g)
                    ref, den = ref_product(A, sa, B, sb, tb)
                    cut = cut_product(A, sa, B, sb, tb)
                    sa2, _ = inside(sa, left, right, 9)
                    sb2, _ = inside(sb, left, right, 9)
                    for out in (BF, FF):
                        if out == FF and tile == (256, 256):
                            continue
                        say("views", left, right, kinds, tb, tile, split, m, out)
                        C, ok = inside(torch.zeros(m, N, device="cuda", dtype=out), left, right, 7)
                        bst.gemm_block_scaled(A, B, sa2, sb2, C, trans_b=tb,
                                              sched=bst.make_sched(tile=tile, split_k=split))
                        check_sum(C, ref, den, K, out, "", cut)
                        assert ok()
    for dtype in (BF, HF, FF):
        for tile, split in (((0, 0), 0), ((128, 128), 1), ((256, 256), 2)):
            for out in (BF, FF):
                g = gen(5)
                q, s = kept(150, K, g)
                s2, _ = inside(s, left, right, 9)
                dY, _ = inside((torch.randn(150, N, generator=g, device="cuda") / 8).to(dtype), left, right, 9)
                add, _ = inside(torch.randn(K, N, generator=g, device="cuda").to(out), right, left, 9)
                W, ok = inside(torch.zeros(K, N, device="cuda", dtype=out), left, right, 7)
                say("gradient views", left, right, dtype, tile, split, out)
                bst.weight_grad(q, s2, dY, W, add=add, sched=bst.make_sched(tile=tile, split_k=split))
                x, d = wide(q, s), dY.double()
                check_sum(W, x.t() @ d + add.double(), x.abs().t() @ d.abs() + add.double().abs(),
                          3 * 150 + 1, out)
                assert ok()


@pytest.mark.parametrize("tb", [False, True])
def test_codes_inside_larger_matrices(tb):
    """A, B and Q as column slices at 16-byte offsets of one larger code matrix."""
    M, N, K, G = 90, 144, 272, 3
    g = gen(3)
    big = torch.randint(0, 0x78, (3 * 300, 800), generator=g, device="cuda", dtype=torch.uint8)
    codes = big.view(torch.float8_e4m3fn)
    A = codes[5:5 + M, 16:16 + K]
    rows, cols = (N, K) if tb else (K, N)
    B = codes.view(G, 300, 800)[:, 1:1 + rows, 352:352 + cols]
    sa, sb = scales((M, 3), "e8m0", g), scales((G, 2, 3) if tb else (G, 3, 2), "f32", g)
    counts = torch.tensor([99, 30, 0, 55, 99], dtype=torch.int32, device="cuda")[1:4]     # a view
    for tile in ((0, 0), (32, 128), (256, 256)):
        sched = bst.make_sched(tile=tile)
        C = bst.grouped_gemm_block_scaled(A, B, counts, sa, sb, trans_b=tb, sched=sched)
        one = B[1:2].expand(G, -1, -1)                       # the same weight for every group
        D = bst.grouped_gemm_block_scaled(A, one, counts, sa, sb[1:2].expand(G, -1, -1), trans_b=tb, sched=sched)
        for k, (lo, hi) in enumerate(spans([30, 0, 55], M)):
            for got, w in ((C, k), (D, 1)):
                if hi > lo:
                    ref, den = ref_product(A[lo:hi], sa[lo:hi], B[w], sb[w], tb)
                    check_sum(got[lo:hi], ref, den, K, BF, "", cut_product(A[lo:hi], sa[lo:hi], B[w], sb[w], tb))
    dY = (torch.randn(M, 40, generator=g, device="cuda") / 8).to(BF)
    add = torch.randn(K, 40, generator=g, device="cuda").expand(G, K, 40)                  # and addend
    W = bst.grouped_weight_grad(A, sa, dY, counts, add=add)
    for k, (lo, hi) in enumerate(spans([30, 0, 55], M)):
        x, d = wide(A, sa)[lo:hi], dY[lo:hi].double()
        check_sum(W[k], x.t() @ d + add[k].double(), x.abs().t() @ d.abs() + add[k].double().abs(), M + 1, FF)


def test_more_than_2_31_values():
    """Codes, products, gradients and restored matrices of 2^31 values and more: their last rows."""
    M, N = 33000, 65552
    g = gen(1)
    x = torch.empty(M, N, dtype=BF, device="cuda")
    x.view(torch.int32).fill_(0x3f803f80)
    x[-40:] = torch.randn(40, N, generator=g, device="cuda").to(BF)
    q, s = bst.quant_block(x)
    q2, s2 = bst.quant_block(x[-40:])
    assert same_values(q[-40:], q2) and torch.equal(s[-40:], s2)
    assert bool((s[0] == 127 - 8).all()) and bool((q[0].float() == 256).all())
    x.zero_()
    bst.dequant_block(q, s, x)
    assert torch.equal(x[-40:], bst.dequant_block(q2, s2)) and bool((x[1] == 1).all())
    del q, s
    say("large quantise and restore")
    K = 144
    A, sa, B, sb = operands(M, N, K, True, ("e8m0", "e8m0"), g)
    for tile in ((256, 256), (128, 128)):
        bst.gemm_block_scaled(A, B, sa, sb, x, trans_b=True, sched=bst.make_sched(tile=tile))
        for rows in (slice(0, 3), slice(M - 3, M)):
            ref, den = ref_product(A[rows], sa[rows], B, sb, True)
            check_sum(x[rows], ref, den, K, BF, "", cut_product(A[rows], sa[rows], B, sb, True))
    say("large product")
    q, s = kept(40, M, g)                 # dW [33000][65552]
    dY = (torch.randn(40, N, generator=g, device="cuda") / 8).to(BF)
    bst.weight_grad(q, s, dY, x)
    for rows in (slice(0, 3), slice(M - 3, M)):
        a, d = wide(q, s)[:, rows], dY.double()
        check_sum(x[rows], a.t() @ d, a.abs().t() @ d.abs(), 40, BF)
