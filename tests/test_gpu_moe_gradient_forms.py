"""GPU tests of moe_combine_grad over the product of the choices that the host makes by size: waves a
token (1, 4 or 16), tasks a token (one, or one for every four choices) and stores through the caches
or past them (rows of 16 MB and more); and either side of each limit.  The gradients are compared with
the formula in 64 bits (test_gpu_moe.check_grad)."""
import pytest
import torch

from gpu_util import say
from test_gpu_moe import check_grad

pytestmark = pytest.mark.gpu

BF, HF, FF = torch.bfloat16, torch.float16, torch.float32
NEAR, FAR = "near", "far"


# waves, tasks, stores: tokens, choices, row length, type (for 256 CUs; test_launch_bounds.py checks
# on the CPU that the host chooses so)
FORMS = {
    (1, "one", NEAR): [(1500, 3, 64, BF), (700, 2, 999, HF)],
    (1, "one", FAR): [(40000, 4, 64, BF), (5000, 2, 1013, FF)],
    (1, "more", NEAR): [(600, 5, 1025, BF), (1023, 6, 513, FF)],
    (1, "more", FAR): [(1000, 9, 1000, BF), (1023, 33, 301, FF)],
    (4, "one", NEAR): [(1025, 1, 2051, BF), (300, 3, 1000, FF)],
    (4, "one", FAR): [(1025, 4, 2051, BF), (2100, 2, 2048, HF), (400, 4, 5001, FF)],
    (4, "more", NEAR): [(300, 9, 1000, BF), (100, 13, 2049, HF)],
    (4, "more", FAR): [(300, 9, 4097, BF), (257, 5, 4096, FF)],
    (16, "one", NEAR): [(256, 4, 2056, BF), (3, 4, 4099, FF), (256, 4, 8191, HF)],
    (16, "one", FAR): [(256, 4, 8192, BF), (256, 4, 8193, HF), (255, 3, 11003, BF), (2, 3, 1000001, FF)],
    (16, "more", NEAR): [(20, 6, 7168, HF), (128, 8, 8191, BF), (1, 33, 4097, FF)],
    (16, "more", FAR): [(128, 8, 8192, BF), (128, 8, 8193, HF), (64, 8, 8192, FF), (1, 8, 1048579, FF)],
}


@pytest.mark.parametrize("T,k,H,dtype", [c for cases in FORMS.values() for c in cases])
def test_gradient_of_every_form(T, k, H, dtype):
    say("gradient forms", T, k, H, dtype)
    check_grad(T, k, H, dtype, FF, T + H)
    check_grad(T, k, H, dtype, FF, T + H, drop=4, in_place=True)


@pytest.mark.parametrize("dtype,H", [(BF, 8192), (FF, 4096)])
def test_few_tokens_with_far_rows_of_any_alignment(dtype, H):
    """Sixteen waves a token, rows of 16 MB and more that start anywhere, some choices without a row."""
    check_grad(200, 8, H + 3, dtype, BF, 5, drop=4, pad=5, offset=1)
