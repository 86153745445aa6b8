"""The split of the CTAs between the shared-prefix decode's two lines
(csrc/prefix_split.h) compiled for the host: no line is left much longer than the
work asks for, whatever the number of units."""
import os
import random
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "query_adaptive_chunk_b200", "csrc")
MAIN = r"""
#include <cstdio>
#include "prefix_split.h"
int main() {
  float a, b, lead;
  int ctas, units;
  while (scanf("%f %f %d %d %f", &a, &b, &ctas, &units, &lead) == 5)
    printf("%d\n", csa::pd_line_a_ctas(a, b, ctas, units, lead));
}
"""


@pytest.fixture(scope="module")
def split(tmp_path_factory):
    d = tmp_path_factory.mktemp("split")
    src, exe = str(d / "s.cpp"), str(d / "s")
    with open(src, "w") as f:
        f.write(MAIN)
    subprocess.run(["g++", "-std=c++17", "-O1", "-I", CSRC, src, "-o", exe], check=True)

    def run(cases):
        text = "".join("%r %r %d %d %r\n" % c for c in cases)
        out = subprocess.run([exe], input=text, capture_output=True, text=True, check=True).stdout.split()
        return [int(x) for x in out]
    return run


def _longer(a, b, ctas, n):
    return max(a / n, b / (ctas - n)) if b > 0 else a / n


def batch(B, Hkv, G, prefix, own, ctas=148):
    """One prefix for B sequences (bf16): line a's and line b's work, as prefix_work.cuh counts it."""
    R = 2 * (128 // G * G)
    rows = B * G
    tiles = -(-rows // R)
    cost = 4.0 * (2.0 if rows > R // 2 else 1.25)
    work_a = Hkv * tiles * (2 + -(-prefix // 64)) * cost
    work_b = B * Hkv * (2.0 + -(-own // 16))
    return work_a, work_b, ctas, Hkv * tiles, 2 * cost


@pytest.mark.parametrize("B,Hkv,G,prefix,own", [
    (256, 8, 8, 8192, 240), (256, 8, 8, 8192, 270), (512, 8, 4, 8192, 100), (128, 8, 8, 16384, 300),
    (1024, 8, 1, 4096, 64), (96, 4, 16, 2048, 128), (200, 16, 4, 5000, 77)])
def test_many_units(split, B, Hkv, G, prefix, own):
    c = batch(B, Hkv, G, prefix, own)
    n, = split([c])
    best = min(_longer(c[0], c[1], c[2], m) for m in range(1, c[2]))
    assert _longer(c[0], c[1], c[2], n) <= 1.02 * best + 2 * c[4], (n, c)


def test_whole_ctas_per_unit_where_it_costs_nothing(split):
    assert split([batch(32, 8, 4, 8192, 512)]) == [56]
    assert split([batch(64, 8, 4, 131072, 2048)])[0] % 8 == 0


def test_any_work(split):
    rng = random.Random(3)
    cases = []
    for _ in range(20000):
        lead = rng.choice([10.0, 16.0])
        a, b = (float(int(10 ** rng.uniform(0.5, 7))) for _ in range(2))
        cases.append((a, b if rng.random() < 0.9 else 0.0, rng.choice([148, 148, 132, 2]), rng.choice([0, 1, 4, 8, 31, 64, 100]), lead))
    for c, n in zip(cases, split(cases)):
        a, b, ctas, units, lead = c
        most = ctas - 1 if b > 0 else ctas
        assert 1 <= n <= most, c
        by_work = min(most, max(1, round(ctas * a / (a + b))))
        assert _longer(a, b, ctas, n) <= 1.001 * (_longer(a, b, ctas, by_work) + 2 * lead), (c, n)
