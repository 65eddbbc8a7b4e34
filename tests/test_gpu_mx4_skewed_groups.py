"""GPU tests of grouped_gemm_mx4 for a few rows a group on average where the groups' loads differ: one
group with all rows, hot ones among many, sizes below zero and past the total, parts of 16 and 32 rows
that end anywhere.  (The loads are not known on the host, so all of these are one kernel's: up to 24 rows
a group on average.)"""
import random

import pytest
import torch

import block_swizzle_tile_amd as bst
from gpu_util import say
from test_gpu_mx4 import check_sum, gen, grouped_ref, operands

pytestmark = pytest.mark.gpu

BF, HF, FF = torch.bfloat16, torch.float16, torch.float32


def check(sizes, total, N, K, out, seed):
    say("skewed", len(sizes), total, N, K, out, max(sizes))
    A, B, sa, sb = operands(total, N, K, gen(seed), len(sizes))
    gm = torch.tensor(sizes, dtype=torch.int32, device="cuda")
    ref, den, live = grouped_ref(A, sa, B, sb, sizes, total)
    C = torch.full((total, N), 7.0, dtype=out, device="cuda")
    bst.grouped_gemm_mx4(A, B, gm, sa, sb, C)
    check_sum(C[:live], ref[:live], den[:live], K, out)
    assert bool((C[live:] == 7).all())


@pytest.mark.parametrize("G,total", [(1, 8), (1, 24), (2, 48), (16, 128), (16, 384), (64, 512), (65, 1560), (200, 1600),
                                     (256, 6144)])
@pytest.mark.parametrize("at", ["first", "middle", "last"])
def test_one_group_has_all_rows(G, total, at):
    sizes = [0] * G
    sizes[dict(first=0, middle=G // 2, last=G - 1)[at]] = total
    check(sizes, total, 16 if G > 128 else 40, 96, BF, G)
    sizes = [1] + sizes[1:]             # a row for the first group, rows behind the last
    sizes[-1] = max(sizes[-1] - 5, 0)
    check(sizes, total, 16 if G > 128 else 25, 70, FF, G + 1)


@pytest.mark.parametrize("out", [BF, HF, FF])
def test_hot_groups_among_many(out):
    rng = random.Random(3)
    for G, per, N, K in ((256, 24, 16, 512), (130, 8, 48, 288), (64, 20, 64, 1024), (8, 24, 500, 1792), (500, 5, 15, 62)):
        total = G * per
        w = [rng.random() ** 8 + 1e-3 for _ in range(G)]
        sizes = [int(total * x / sum(w)) for x in w]
        check(sizes, total, N, K, out, G)


def test_parts_that_end_anywhere():
    """Sizes about the parts of 16 and 32 rows, of none, below zero and past the total."""
    rng = random.Random(5)
    for i in range(20):
        G = rng.choice([3, 20, 64, 70, 129])
        total = rng.choice([8, 24]) * G - rng.randint(0, 7)
        sizes = [rng.choice([0, 0, 0, 0, 1, 15, 16, 17, 31, 32, 33, 48, 65, -4]) for _ in range(G)]
        if i % 5 == 0:
            sizes[rng.randrange(G)] = 2 ** 31 - 1
        check(sizes, total, rng.choice([1, 16, 33]), 2 * rng.randint(1, 300), BF, i)


def test_no_k():
    A, B, sa, sb = operands(20, 16, 0, gen(1), 4)
    gm = torch.tensor([0, 19, 0, 0], dtype=torch.int32, device="cuda")
    C = torch.full((20, 16), 7.0, device="cuda")
    bst.grouped_gemm_mx4(A, B, gm, sa, sb, C)
    assert not bool(C[:19].any()) and bool((C[19] == 7).all())
