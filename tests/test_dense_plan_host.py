"""The rule that chooses a form of the dense product (csrc/dense_plan.h), as host code:
test_gpu_dense_forms.py's sizes take the forms that they stand for, and no size takes
another one."""

from __future__ import annotations

import math
import os
import random
import subprocess

import pytest

from tests.test_gpu_dense_forms import FORMS, SIZES

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "fp8_block_scaled_moe_amd", "csrc")
NAMES = ["strip 4x4", "strip 16x16", "strip 16x32", "strip 32x32", "strip 32x64", "64x128", "128x128", "128x128, two a CU", "256x256",
         "256x256 and halves"]
PROGRAM = """
#include <cstdio>
#include "dense_plan.h"
static_assert(moe::kDenseStrip4x4 == 0 && moe::kDenseStrip32x64 == 4 && moe::kDense64x128 == 5 && moe::kDenseHalves == 9, "the forms' names");
int main() {
  int T, N, K, split;
  while (std::scanf("%d %d %d %d", &T, &N, &K, &split) == 4) {
    const moe::DensePlan p = moe::dense_plan(T, N, K, split != 0);
    std::printf("%d %d\\n", p.shape, p.splits);
  }
}
"""


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    at = tmp_path_factory.mktemp("plan")
    (at / "plan.cc").write_text(PROGRAM)
    subprocess.run(["g++", "-O1", "-std=c++17", "-Wall", "-Werror", "-I", CSRC, str(at / "plan.cc"), "-o", str(at / "plan")], check=True)

    def forms(sizes, split=1):
        text = "".join(f"{T} {N} {K} {split}\n" for T, N, K in sizes)
        out = subprocess.run([str(at / "plan")], input=text, capture_output=True, text=True, check=True).stdout.split()
        return [(NAMES[int(s)], int(p)) for s, p in zip(out[::2], out[1::2])]

    return forms


def test_sizes_take_the_forms_that_they_stand_for(plan):
    assert plan([s[2:] for s in SIZES]) == [s[:2] for s in SIZES]


def test_no_size_takes_another_form(plan):
    rng = random.Random(1)
    size = lambda hi: round(math.exp(rng.uniform(0, math.log(hi))))  # noqa: E731
    drawn = [(size(16384), size(8192), 8 * size(1024)) for _ in range(60000)] + [(size(1048576), size(1048576), 8 * size(131072)) for _ in range(60000)]
    assert set(plan(drawn)) <= set(FORMS)
    assert {name for name, _ in FORMS} == set(NAMES)


def test_without_a_workspace_k_stays_whole(plan):
    assert {splits for _, splits in plan([s[2:] for s in SIZES], split=0)} == {1}
