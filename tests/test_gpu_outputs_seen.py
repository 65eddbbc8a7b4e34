"""GPU test that new outputs and workspaces of the operators reached by the short way come from torch's
dispatcher where something listens to it (a dispatch mode, the profiler), and that calls under it give
the same values."""
import pytest
import torch
from torch.utils._python_dispatch import TorchDispatchMode

import block_swizzle_tile_amd as bst

pytestmark = pytest.mark.gpu

NAMES = ["quant_block", "dequant_block", "gemm_block_scaled", "grouped_gemm_block_scaled", "weight_grad",
         "moe_sort", "moe_sort_many", "moe_gather", "moe_combine", "moe_combine_grad", "quant_mx4",
         "dequant_mx4", "gemm_mx4", "grouped_gemm_mx4"]


class Listener(TorchDispatchMode):
    def __init__(self):
        super().__init__()
        self.made = 0

    def __torch_dispatch__(self, func, types, args=(), kwargs=None):
        out = func(*args, **(kwargs or {}))
        self.made += func is torch.ops.aten.empty.memory_format
        return out


def calls():
    """{name: (call, new tensors that it makes)}"""
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(200, 256, generator=g, device="cuda").to(torch.bfloat16)
    w = torch.randn(128, 256, generator=g, device="cuda").to(torch.bfloat16)
    q, s = bst.quant_block(x)
    wq, ws = bst.quant_block(w, block_rows=128)
    a, sa = bst.quant_mx4(x)
    b, sb = bst.quant_mx4(w)
    one = torch.tensor([200], dtype=torch.int32, device="cuda")
    ids = torch.randint(0, 8, (100, 2), generator=g, device="cuda")
    row_of = bst.moe_sort(ids, 8)[0]
    many = torch.randint(0, 8, (40000, 2), generator=g, device="cuda")
    p = torch.rand(100, 2, generator=g, device="cuda")
    return dict(
        quant_block=(lambda: bst.quant_block(x), 2),
        dequant_block=(lambda: bst.dequant_block(q, s), 1),
        gemm_block_scaled=(lambda: bst.gemm_block_scaled(q, wq, s, ws, trans_b=True), 1),
        grouped_gemm_block_scaled=(lambda: bst.grouped_gemm_block_scaled(q, wq[None], one, s, ws[None],
                                                                          trans_b=True), 1),
        weight_grad=(lambda: bst.weight_grad(q, s, x), 1),
        moe_sort=(lambda: bst.moe_sort(ids, 8), 2),
        moe_sort_many=(lambda: bst.moe_sort(many, 8), 3),
        moe_gather=(lambda: bst.moe_gather(x[:100], row_of), 1),
        moe_combine=(lambda: bst.moe_combine(x, row_of, p), 1),
        moe_combine_grad=(lambda: bst.moe_combine_grad(x[:100], x, row_of, p), 2),
        quant_mx4=(lambda: bst.quant_mx4(x), 2),
        dequant_mx4=(lambda: bst.dequant_mx4(a, sa), 1),
        gemm_mx4=(lambda: bst.gemm_mx4(a, b, sa, sb), 1),
        grouped_gemm_mx4=(lambda: bst.grouped_gemm_mx4(a, b[None], one, sa, sb[None]), 1))


def values(out):
    return [t.view(torch.uint8).cpu() for t in (out if isinstance(out, tuple) else (out,))]


@pytest.mark.parametrize("name", NAMES)
def test_new_outputs_are_seen(name):
    call, new = calls()[name]
    want = values(call())
    with Listener() as seen:
        out = call()
    assert seen.made >= new, (seen.made, new)
    assert all(torch.equal(g, w) for g, w in zip(values(out), want))
    with torch.profiler.profile(activities=[torch.profiler.ProfilerActivity.CPU]) as prof:
        call()
    assert sum(e.count for e in prof.key_averages() if e.key == "aten::empty") >= new
