"""GPU test of a mixture of experts' layer in 4 bits, forward and backward, as a user runs it: sort,
quantise, gather of codes and scales, grouped product, weighted sum; then the sum's gradients, the
product with the weights' other quantisation, the gather's gradient, and the experts' weight gradients
from the tokens' 8-bit rows.  Each call's output is compared with its formula in 64 bits from the values
that its inputs stand for, the layer's gradients with those of the unquantised layer in direction; with
and without choices whose expert is elsewhere."""
import pytest
import torch

import block_swizzle_tile_amd as bst
import test_gpu_block as eight
from gpu_util import say
from test_gpu_moe import near
from test_gpu_mx4 import check_sum, gen, grouped_ref, up, wide

pytestmark = pytest.mark.gpu

BF, FF = torch.bfloat16, torch.float32


@pytest.mark.parametrize("T,k,E,first,G,H,N", [(7, 2, 4, 0, 4, 256, 96), (130, 4, 16, 0, 16, 320, 136),
                                               (700, 3, 5, 0, 5, 544, 264), (300, 4, 12, 4, 4, 512, 160)])
def test_layer_forward_and_backward(T, k, E, first, G, H, N):
    say("layer", T, k, E, first, G, H, N)
    g = gen(T)
    x = torch.randn(T, H, generator=g, device="cuda").to(BF)
    w = (torch.randn(G, N, H, generator=g, device="cuda") / 16).to(BF)
    dy = torch.randn(T, N, generator=g, device="cuda").to(BF)
    weights, expert = torch.topk(torch.rand(T, E, generator=g, device="cuda"), k)
    row_of, group_m = bst.moe_sort(expert, G, first=first)
    # ---- forward
    wq, ws = (t.unflatten(0, (G, N)) for t in bst.quant_mx4(w.flatten(0, 1)))
    xq, xs = bst.quant_mx4(x)
    rows, rs = bst.moe_gather(xq, row_of, scale=xs)
    h = bst.grouped_gemm_mx4(rows, wq, group_m, rs, ws)
    y = bst.moe_combine(h, row_of, weights)
    # ---- backward
    dh, dweights = bst.moe_combine_grad(dy, h, row_of, weights)
    vq = torch.empty(G, H, up(N // 2, 16), dtype=torch.float4_e2m1fn_x2, device="cuda")[..., :N // 2]
    vs = torch.empty(G, H, up(-(-N // 32), 4), dtype=torch.uint8, device="cuda")[..., :-(-N // 32)]
    for e in range(G):
        bst.quant_mx4(w[e], vq[e], vs[e], transpose=True)
    dq, ds = bst.quant_mx4(dh)
    drows = bst.grouped_gemm_mx4(dq, vq, group_m, ds, vs)
    dx = bst.moe_combine(drows, row_of)
    kept, kept_s = bst.quant_block(x)
    rows8, rs8 = bst.moe_gather(kept, row_of, scale=kept_s)
    dw = bst.grouped_weight_grad(rows8, rs8, dh, group_m)

    at, sizes = row_of.long(), group_m.tolist()
    live = at >= 0
    assert bool(live.all()) == (G == E) and int(live.sum()) == sum(sizes)
    own = at[live]                                  # rows of the choices that are here
    token = torch.arange(T, device="cuda")[:, None].expand(T, k)[live]
    w64, dy64 = weights.double(), dy.double()
    total = T * k

    def of_choices(r):
        return torch.where(live[..., None], r.double()[at.clamp(min=0)], 0.0)

    assert torch.equal(wide(rows, rs)[own], wide(xq, xs)[token])
    ref, den, n = grouped_ref(rows, rs, wq, ws, sizes, total)
    check_sum(h[:n], ref[:n], den[:n], H, BF)
    terms = w64[..., None] * of_choices(h)
    near(y, terms.sum(1), terms.abs().sum(1), k, BF, "y")
    want = (w64[..., None] * dy64[:, None])[live]
    near(dh[own], want, want.abs(), 1, BF, "dh")
    terms = of_choices(h) * dy64[:, None]
    near(dweights, terms.sum(2), terms.abs().sum(2), N + 8, FF, "dweights")
    ref, den, n = grouped_ref(dq, ds, vq, vs, sizes, total)
    check_sum(drows[:n], ref[:n], den[:n], N, BF)
    terms = of_choices(drows)
    near(dx, terms.sum(1), terms.abs().sum(1), k, BF, "dx")
    assert torch.equal(eight.wide(rows8, rs8)[own], eight.wide(kept, kept_s)[token])
    first_row = 0
    for e, n in enumerate(sizes):
        r, d = eight.wide(rows8, rs8)[first_row:first_row + n], dh[first_row:first_row + n].double()
        eight.check_sum(dw[e], r.t() @ d, r.abs().t() @ d.abs(), n, FF, "dw of %d" % e)
        first_row += n

    # ---- the unquantised layer, by torch's autograd in 64 bits on the CPU
    a, b, c = (t.double().cpu().requires_grad_() for t in (x, w, weights))
    ids, here = expert.cpu() - first, live.cpu()
    out = torch.zeros(T, N, dtype=torch.float64)
    for j in range(k):
        for e in range(G):
            m = (ids[:, j] == e) & here[:, j]
            out = out + torch.where(m[:, None], c[:, j:j + 1] * (a @ b[e].t()), 0.0)
    out.backward(dy.double().cpu())
    for got, want in ((y, out.detach()), (dx, a.grad), (dw, b.grad.transpose(1, 2)), (dweights, c.grad)):
        got = got.double().cpu()
        assert got.shape == want.shape and float((got * want).sum() / (got.norm() * want.norm())) > 0.95
