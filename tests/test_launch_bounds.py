"""CPU test of the launches of the expert-routing and 4-bit operators: over a sweep of sizes that
crosses every rule by which the host chooses a kernel, each launch has exactly as many threads as
the kernel was compiled for (its launch bound in the code object: the kernels count on it for their
shared memory and for which wave does what), and a launch never holds 2^32 threads.

The calls run in a process of their own on a stand-in for the HIP runtime
(tests/native/record_launches.cpp), which writes launches down instead of running them; pointers are
fake."""
import ctypes
import os
import re
import struct
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIB = os.environ.get("BST_LIB") or os.path.join(ROOT, "block_swizzle_tile_amd", "libbst.so")
READELF = "/opt/rocm/llvm/bin/llvm-readelf"
P = 1 << 20                      # 16-byte aligned, never dereferenced
F16, BF16, F32 = 1, 2, 7
i32, i64 = ctypes.c_int32, ctypes.c_int64
p, sz = ctypes.c_void_p, ctypes.c_size_t


# ---------------------------------------------------- the calls, in a child ---
def gradients(L):
    """Waves a token (1, 4, 16), tasks a token (one, more) and stores (through the caches, past them)
    are chosen by rows, tokens, choices and bytes: all of them crossed."""
    for r, es in ((BF16, 2), (F16, 2), (F32, 4)):
        for H in (1, 8, 256, 512, 516, 1000, 1025, 2048, 2049, 4096, 6144, 8192, 16384, 1 << 20):
            for k in (1, 2, 4, 5, 8, 9, 33):
                for T in (1, 3, 16, 31, 32, 64, 100, 127, 128, 192, 255, 256, 257, 511, 512, 600, 1023, 1024, 1025,
                          4096, 8192, 100000):
                    L.bst_moe_combine_grad(r, i64(T), i32(k), i64(H), p(P), i64(H), p(P), i64(H), i64(T * k), p(P),
                                           F32, p(P), p(P), i64(H), p(P), None)


def sorts(L):
    for n in (0, 1, 64, 100, 2047, 2048, 2049, 8192, 8193, 32768, 32769, 65536, 1 << 20, (1 << 31) - 1):
        for G in (1, 3, 8, 64, 128, 255, 256, 257, 1000, 1024):
            for es in (4, 8):
                L.bst_moe_sort(i32(es), i64(n), p(P), i32(0), i32(G), p(P), p(P), p(P), sz(1 << 40), None)


def moves(L):
    for T in (1, 16, 100, 256, 1024, 8191, 100000):
        for k in (1, 2, 4, 8, 9):
            for nb in (1, 15, 16, 17, 260, 4096, 16384, 65536):
                for sb in (0, 1, 16, 32):
                    L.bst_moe_gather(i64(T), i32(k), i64(nb), p(P), i64(nb), p(P), i64(T * k), p(P), i64(nb), i64(sb),
                                     p(P if sb else 0), i64(sb), p(P if sb else 0), i64(sb), None)
            for r in (BF16, F16, F32):
                for H in (1, 8, 1000, 4096, 8192, 16384):
                    L.bst_moe_combine(r, BF16, i64(T), i32(k), i64(H), p(P), i64(H), i64(T * k), p(P), F32, p(P), None,
                                      i64(0), p(P), i64(H), None)


def quants(L):
    for x in (BF16, F16, F32):
        for M in (1, 31, 32, 33, 200, 2047, 8192, 65536):
            for K in (1, 32, 33, 136, 1001, 4096, 8192):
                q, s = K // 2 + 1, K // 32 + 1
                L.bst_quant_mx4(x, i64(M), i64(K), i32(0), p(P), i64(K), p(P), i64(q), p(P), i64(s), None)
                L.bst_dequant_mx4(x, i64(M), i64(K), p(P), i64(q), p(P), i64(s), p(P), i64(K), None)
                L.bst_quant_mx4(x, i64(M), i64(K), i32(1), p(P), i64(K), p(P), i64(M // 2 + 1), p(P),
                                i64(M // 32 + 1), None)


def products(L):
    for c in (BF16, F32):
        for M in (1, 5, 16, 17, 32, 33, 64, 65, 128, 300, 1024, 2048, 8192):
            for N in (16, 100, 256, 1000, 2048, 4096, 16384):
                for K in (1, 64, 300, 1024, 4096, 7168, 28672):
                    ld, ls = i64((K + 31) // 32 * 16), i64((K + 127) // 128 * 4)
                    a = (p(P), ld, p(P), ls, p(P))
                    L.bst_gemm_mx4(c, i64(M), i64(N), i64(K), *a, ld, p(P), ls, p(P), i64(N), None, p(P), sz(1 << 40),
                                   None)
                    for G in (1, 4, 32, 256):
                        L.bst_grouped_gemm_mx4(c, i32(G), p(P), i64(M), i64(N), i64(K), *a, ld, i64(0), p(P), ls,
                                               i64(0), p(P), i64(N), None, None)


def forms(L):
    """The cases that a GPU test has for each form of the gradient: r, T, k, H as arguments."""
    for a in sys.argv[3:]:
        r, T, k, H = map(int, a.split(","))
        L.bst_moe_combine_grad(r, i64(T), i32(k), i64(H), p(P), i64(H), p(P), i64(H), i64(T * k), p(P), F32, p(P),
                               p(P), i64(H), p(P), None)


def few_rows(L):
    """Grouped products whose first tile count is at most the rows kernel's: N, K, G, M as arguments."""
    for a in sys.argv[3:]:
        N, K, G, M = map(int, a.split(","))
        ld, ls = i64((K + 31) // 32 * 16), i64((K + 127) // 128 * 4)
        L.bst_grouped_gemm_mx4(BF16, i32(G), p(P), i64(M), i64(N), i64(K), p(P), ld, p(P), ls, p(P), ld, i64(0), p(P),
                               ls, i64(0), p(P), i64(N), None, None)


SWEEPS = dict(gradients=gradients, sorts=sorts, moves=moves, quants=quants, products=products)


def child(sweep, path):
    runtime = ctypes.CDLL(None)
    L = ctypes.CDLL(LIB)
    runtime.record_launches(path.encode())
    dict(SWEEPS, forms=forms, few_rows=few_rows)[sweep](L)
    runtime.record_end()


# ------------------------------------------------------------------- tests ---
def kernel_bounds(lib, tmp):
    """{kernel: its launch bound} of all gfx950 code objects in a library."""
    data, bounds, magic = open(lib, "rb").read(), {}, b"__CLANG_OFFLOAD_BUNDLE__"
    at = data.find(magic)
    while at >= 0:
        pos = at + len(magic) + 8
        for _ in range(struct.unpack_from("<Q", data, at + len(magic))[0]):
            off, size, n = struct.unpack_from("<QQQ", data, pos)
            name = data[pos + 24:pos + 24 + n]
            pos += 24 + n
            if b"gfx950" not in name or size == 0:
                continue
            co = os.path.join(tmp, "code")
            with open(co, "wb") as f:
                f.write(data[at + off:at + off + size])
            notes = subprocess.check_output([READELF, "--notes", co], text=True)
            for k in re.split(r"\n  - \.a", notes)[1:]:
                bounds[re.search(r"\.name:\s+(\S+)", k).group(1)] = int(
                    re.search(r"\.max_flat_workgroup_size:\s+(\d+)", k).group(1))
        at = data.find(magic, at + 1)
    return bounds


@pytest.fixture(scope="module")
def recorder(tmp_path_factory):
    if not os.path.exists(LIB):
        from block_swizzle_tile_amd import build
        build.build()
    tmp = tmp_path_factory.mktemp("launches")
    so = str(tmp / "record.so")
    subprocess.check_call(["g++", "-O2", "-std=c++17", "-shared", "-fPIC",
                           os.path.join(ROOT, "tests", "native", "record_launches.cpp"), "-o", so])
    bounds = kernel_bounds(LIB, str(tmp))

    def launches(sweep, *args):
        out = str(tmp / sweep)
        subprocess.run([sys.executable, os.path.abspath(__file__), sweep, out, *args], check=True, timeout=300,
                       env=dict(os.environ, LD_PRELOAD=so, BST_LIB=LIB))
        return [(n, int(g), int(b)) for n, g, b in (line.split() for line in open(out))]

    return bounds, launches


@pytest.mark.parametrize("sweep", list(SWEEPS))
def test_launches_have_the_threads_of_their_kernels(recorder, sweep):
    bounds, launches = recorder
    rows = launches(sweep)
    assert len(rows) > 100
    wrong = {(n, b, bounds.get(n)) for n, g, b in rows if b != bounds.get(n)}
    assert not wrong, sorted(wrong, key=str)
    assert all(0 < g * b < 2 ** 32 for n, g, b in rows)


def test_every_gradient_kernel_is_reached(recorder):
    bounds, launches = recorder
    have = {n for n in bounds if "moe_combine_grad_kernel" in n}
    assert have and {n for n, g, b in launches("gradients")} == have


def test_cases_of_every_gradient_form(recorder):
    """The GPU test's cases are of the forms that it lists them under."""
    import torch
    from test_gpu_moe_gradient_forms import FORMS, NEAR
    kind = {torch.bfloat16: BF16, torch.float16: F16, torch.float32: F32}
    assert len(FORMS) == 12
    want, args = [], []
    for (waves, tasks, stores), cases in FORMS.items():
        for T, k, H, dtype in cases:
            args.append("%d,%d,%d,%d" % (kind[dtype], T, k, H))
            n = T * (1 if tasks == "one" else -(-k // 4))
            want.append(("ILi%dELi%dELb%dEE" % (kind[dtype], waves, stores != NEAR), n if waves > 1 else -(-n // 4)))
            assert tasks == "one" or k > 4
    got = [(re.search(r"I\w+?EE", n).group(0), g) for n, g, b in recorder[1]("forms", *args)]
    assert got == want


def test_rows_of_one_group_find_workgroups(recorder):
    """The kernel for a few rows a group does not know the groups' loads when it is launched: each group
    has workgroups for its first 16 FM rows, and there are as many more as all rows in one group need."""
    sizes = [(16, 7168, 256, 6144), (16, 1024, 256, 2048), (256, 4096, 16, 384), (128, 14336, 64, 512),
             (512, 7168, 8, 192), (2048, 7168, 2, 48), (100, 64, 1, 24), (4096, 4096, 2, 16)]
    got = recorder[1]("few_rows", *("%d,%d,%d,%d" % s for s in sizes))
    assert len(got) == len(sizes)
    for (N, K, G, M), (name, grid, _) in zip(sizes, got):
        fm = int(re.search(r"mx4_rows_kernelILi(\d+)E", name).group(1))
        assert grid >= -(-N // 16) * max(G, -(-M // (16 * fm))), (N, K, G, M, name, grid)
        assert grid >= -(-N // 16) * (G + max(0, -(-M // (16 * fm)) - 1)), (N, K, G, M, name, grid)


if __name__ == "__main__":
    child(sys.argv[1], sys.argv[2])
