"""The variants of the matrix products: that each is taken by a shape that the
GPU tests run, in every split that it has, and that what a call is planned with
is within the limits of the kernel, over the range of shapes."""
import collections
import math
import os
import random
import subprocess

import pytest

import test_gpu_linear as G
from linear_attention_decode_04_gb300 import build as B

Variant = collections.namedtuple("Variant", "rows unit channels pair interleaved threads stage_bytes part_bytes head_bytes")
Plan = collections.namedtuple("Plan", "variant split stages tile_rows")
SMEM, SMS, MAX_STAGES, BLOCK = 227 * 1024, 152, 12, 128


@pytest.fixture(scope="module")
def plans(tmp_path_factory):
    """plans(shapes) -> (the variants, a plan for each (M, N, K, e4m3, gated, whole))"""
    exe = str(tmp_path_factory.mktemp("plan") / "linear_plan")
    here = os.path.dirname(os.path.abspath(__file__))
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", "-I", B.CSRC, os.path.join(here, "linear_plan.cpp"), "-o", exe], check=True)

    def run(shapes):
        text = "\n".join(" ".join(str(int(v)) for v in s) for s in shapes)
        lines = subprocess.run([exe], input=text, capture_output=True, text=True, check=True).stdout.split("\n")
        at = lines.index("-")
        rows = [[int(v) for v in line.split()] for line in lines if line and line != "-"]
        return [Variant(*r) for r in rows[:at]], [Plan(*r) for r in rows[at:]]
    return run


def cases(test, names):
    """The values that a test is parametrised with, of one mark"""
    for mark in test.pytestmark:
        if mark.name == "parametrize" and [n.strip() for n in mark.args[0].split(",")] == names.split():
            return mark.args[1]
    raise AssertionError(f"{test.__name__} is not parametrised with {names}")


def run_on_the_gpu():
    """(M, N, K, e4m3, gated, whole) of GPU tests"""
    for gated, tests in ((False, (G.test_every_tile_and_share_of_k, G.test_tiles_of_128_rows_in_four_parts)),
                         (True, (G.test_every_gated_tile, G.test_gated_tiles_of_two_warpgroups))):
        for test in tests:
            for e4m3, M, N, K in cases(test, "e4m3 M N K"):
                yield M, N, K, e4m3, gated, True       # fp32, or bf16 in whole 16-byte pieces
                yield M, N, K, e4m3, gated, False      # on no boundary


def splits(v, most):
    """Parts of k that a variant can have"""
    return [s for s in (1, 2, 4) if s == 1 or (not v.interleaved and 2 * v.part_bytes <= most * v.stage_bytes)]


def test_gpu_tests_reach_every_variant_and_split(plans):
    shapes = list(run_on_the_gpu())
    variants, taken = plans(shapes)
    assert len(variants) == 13 and len(taken) == len(shapes)
    seen = collections.Counter((p.variant, p.split) for p in taken)
    for i, v in enumerate(variants):
        for s in splits(v, min((SMEM - v.head_bytes) // v.stage_bytes, MAX_STAGES)):
            assert seen[i, s], (i, v, s)


def test_plans_are_within_the_kernels_limits(plans):
    rng = random.Random(0)
    log = lambda lo, hi: int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))  # noqa: E731
    shapes = [(log(1, 60000), 2 * log(1, 100000), log(1, 60000), rng.random() < 0.5, rng.random() < 0.3, rng.random() < 0.5) for _ in range(20000)]
    shapes += [(2 ** 31 - 512, 64, 8, False, False, True), (1, 2 ** 24, 2 ** 24, True, False, True), (1, 2, 1, True, True, False)]
    variants, taken = plans(shapes)
    for (M, N, K, e4m3, gated, whole), p in zip(shapes, taken):
        v, width, blocks = variants[p.variant], N // 2 if gated else N, -(-K * (1 if e4m3 else 2) // BLOCK)
        tiles = -(-M // p.tile_rows) * -(-width // v.channels)
        assert 0 < p.tile_rows <= v.rows and p.tile_rows % v.unit == 0
        assert 1 <= p.stages <= MAX_STAGES and p.stages * v.stage_bytes + v.head_bytes <= SMEM
        assert p.split in (1, 2, 4) and p.split <= blocks
        if p.split > 1:                        # a cluster a tile, at most eight CTAs; its own sums and those sent to it
            part = v.part_bytes // (128 * 8 + 64 * 4) * (128 // p.split * 8 + 64)
            assert tiles * p.split <= (SMS // 2 if v.pair else SMS) and p.split * (2 if v.pair else 1) <= 8
            assert 2 * p.split * part <= p.stages * v.stage_bytes
