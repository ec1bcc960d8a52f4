"""What the product's plan chooses (csrc/product_plan.h, compiled for the host):
for sizes that were measured, a kind and a number of parts that were at most a
tenth slower than the fastest."""

import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
KINDS = ["FEW", "LOW", "STRIP", "DEEP", "PAIR", "HALF", "MID", "TALL", "LONG", "WIDE"]
TILE = {"FEW": (16, 16), "LOW": (32, 32), "STRIP": (32, 64), "DEEP": (64, 64), "PAIR": (64, 64), "HALF": (64, 128), "MID": (128, 128),
        "TALL": (192, 128), "LONG": (128, 128)}
BF16, F32 = 0, 1
SOURCE = """
#include <cstdio>
#include "product_plan.h"
int main() {
    int m, k, n, type;
    while (std::scanf("%d %d %d %d", &m, &k, &n, &type) == 4) {
        const mega_moe::ProductPlan p = mega_moe::product_plan(m, n, k, type);
        std::printf("%d %d\\n", p.kind, p.splits);
    }
}
"""


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    """(m, k, n, type) -> (kind, parts)"""
    cxx = shutil.which("g++") or shutil.which("c++") or shutil.which("clang++")
    if not cxx:
        pytest.skip("no host compiler")
    d = tmp_path_factory.mktemp("plan")
    (d / "plan.cpp").write_text(SOURCE)
    subprocess.run([cxx, "-std=c++17", "-O1", "-I", os.path.join(ROOT, "include"), "-I",
                    os.path.join(ROOT, "fp8_mixture_experts_amd", "csrc"), str(d / "plan.cpp"), "-o", str(d / "plan")], check=True)

    def choose(m, k, n, out_type):
        r = subprocess.run([str(d / "plan")], input=f"{m} {k} {n} {out_type}", capture_output=True, text=True, check=True)
        kind, parts = r.stdout.split()
        return KINDS[int(kind)], int(parts)

    return choose


# (m, k, n, type): what was measured within a tenth of the fastest of all kinds in 1 to 64 parts
MEASURED = {
    (1, 8192, 64, BF16): "FEW:1",
    (8, 8192, 280, BF16): "FEW:1 LOW:4 LOW:8",
    (13, 8192, 560, BF16): "LOW:4 LOW:8 FEW:1 STRIP:8",
    (4, 5632, 472, BF16): "FEW:1",
    (1, 8192, 560, BF16): "FEW:1",
    (16, 8192, 904, BF16): "LOW:4 LOW:8 LOW:2 STRIP:8",
    (32, 5632, 280, BF16): "LOW:4 LOW:8 LOW:1 PAIR:8 LOW:2",
    (64, 8192, 136, BF16): "LOW:8 LOW:4 STRIP:8",
    (128, 8192, 904, BF16): "LOW:2 LOW:1 STRIP:4 PAIR:8",
    (1, 8192, 64, F32): "FEW:1 LOW:8 LOW:4",
    (64, 8192, 64, F32): "LOW:8 LOW:4",
    (128, 8192, 280, F32): "LOW:4",
    (4, 8192, 560, F32): "FEW:1 LOW:4 LOW:8",
    (8, 32768, 136, BF16): "LOW:8 LOW:16 STRIP:16",
    (128, 131072, 128, BF16): "LOW:16",
    (256, 131072, 256, F32): "DEEP:16 PAIR:32",
    (1, 7168, 4096, BF16): "FEW:1",
    (16, 7168, 4096, BF16): "FEW:1",
    (128, 2048, 7168, BF16): "DEEP:1 PAIR:1",
    (576, 2048, 7168, BF16): "TALL:1",
    (1024, 7168, 4096, BF16): "LONG:1",
    (2048, 7168, 4096, BF16): "MID:1 WIDE:2",
    (8192, 7168, 4096, BF16): "WIDE:1",
    (8192, 2048, 7168, BF16): "WIDE:1",
    (1, 7168, 18432, BF16): "FEW:1",
    (1, 7168, 4096, F32): "FEW:1",
    (512, 4096, 4096, F32): "PAIR:1",
    (4096, 4096, 2048, F32): "WIDE:1 MID:1",
}


@pytest.mark.parametrize("size", list(MEASURED), ids=str)
def test_choice_is_near_the_fastest_measured(plan, size):
    kind, parts = plan(*size)
    assert f"{kind}:{parts}" in MEASURED[size].split()


def test_choice_can_be_launched(plan):
    for m in (1, 16, 17, 100, 2 ** 21):
        for k in (0, 128, 8192, 2 ** 21):
            for n in (8, 4096, 2 ** 21):
                for out_type in (BF16, F32):
                    kind, parts = plan(m, k, n, out_type)
                    assert parts == 1 or (parts <= k // 128 and kind != "FEW")
                    assert kind != "FEW" or m <= 16
                    assert out_type == BF16 or kind not in ("STRIP", "HALF", "TALL", "LONG")


def test_sizes_of_the_long_loops_reach_every_kind(plan):
    import torch

    from tests.test_gpu_dense_tiles import CASES
    for dtype, sizes in CASES.items():
        out_type = F32 if dtype == torch.float32 else BF16
        for size, want in sizes.items():
            m, k, n = size
            assert plan(m, k, n, out_type) == want, size
            # (a wave of the few rows' kernel has every 8th or 16th step, and takes three or two at a time)
            steps = k // 128 // want[1]
            assert steps >= 17 and (steps % 8 or size == (1, 7168, 18432)), size
            rows, columns = TILE.get(want[0], (128, 256))
            assert m % rows and (want[0] == "FEW" or n % columns), size
        kinds = {kind for kind, _ in sizes.values()}
        assert kinds == set(KINDS) - (set() if out_type == BF16 else {"STRIP", "HALF", "TALL", "LONG"})
        in_parts = {kind for kind, parts in sizes.values() if parts > 1}
        assert in_parts == ({"LOW", "STRIP", "DEEP", "HALF", "TALL", "LONG", "WIDE"} if out_type == BF16 else {"LOW", "DEEP", "MID", "WIDE"})
    few = [size for size, (kind, _) in CASES[torch.bfloat16].items() if kind == "FEW"]
    # two workgroups to a compute unit: twice and more around their loop of 24 steps
    assert sum(n > 4096 and k // 128 > 24 for m, k, n in few) >= 3 and any(n > 4096 and k // 128 > 48 for m, k, n in few)
