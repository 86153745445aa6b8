"""csrc/rows.h (whether strided sets of rows share memory) compiled for the host
and compared with sets of byte addresses."""
import os
import random
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "query_adaptive_chunk_b200", "csrc")
MAIN = r"""
#include <cstdio>
#include "rows.h"
static bool read(csa::Rows* r) {
  long long p, n[3], st[3], row; int es;
  if (scanf("%lld %lld %lld %lld %lld %lld %lld %lld %d", &p, n, n + 1, n + 2, st, st + 1, st + 2, &row, &es) != 9)
    return false;
  *r = csa::Rows{reinterpret_cast<const void*>(p), 3, {n[0], n[1], n[2]}, {st[0], st[1], st[2]}, row, es};
  return true;
}
int main() {
  csa::Rows a, b;
  while (read(&a) && read(&b))
    printf("%d %d\n", csa::rows_meet(a, b) ? 1 : 0, csa::rows_meet_themselves(a) ? 1 : 0);
}
"""


@pytest.fixture(scope="module")
def ask(tmp_path_factory):
    d = tmp_path_factory.mktemp("rows")
    src, exe = str(d / "rows.cpp"), str(d / "rows")
    with open(src, "w") as f:
        f.write(MAIN)
    subprocess.run(["g++", "-std=c++17", "-O1", "-I", CSRC, src, "-o", exe], check=True)

    def run(pairs):
        text = "".join(" ".join(str(x) for x in (r["p"], *r["n"], *r["st"], r["row"], r["es"])) + "\n"
                       for pair in pairs for r in pair)
        out = subprocess.run([exe], input=text, capture_output=True, text=True, check=True).stdout.split()
        return [(out[2 * i] == "1", out[2 * i + 1] == "1") for i in range(len(pairs))]
    return run


def _rows(r):
    n, st = r["n"], r["st"]
    return [r["p"] + r["es"] * (i * st[0] + j * st[1] + k * st[2])
            for i in range(n[0]) for j in range(n[1]) for k in range(n[2])]


def _bytes(r):
    return {a + x for a in _rows(r) for x in range(r["row"] * r["es"])}


def _truth(a, b):
    cells = [a0 + x * a["es"] for a0 in _rows(a) for x in range(a["row"])]
    return bool(_bytes(a) & _bytes(b)), len(cells) != len(set(cells))


def test_against_sets_of_bytes(ask):
    rng = random.Random(5)
    pairs = []
    for _ in range(4000):
        def one(p):
            return dict(p=p, n=[rng.choice([1, 2, 3, 5]) for _ in range(3)], row=rng.choice([1, 2, 4]),
                        st=[rng.choice([0, 1, 2, 4, 5, 8, 12, 20, 24, 60]) for _ in range(3)], es=rng.choice([2, 4]))
        a, b = one(1000), one(1000 + 2 * rng.randint(-60, 60))
        if rng.random() < 0.5:
            b["st"], b["es"] = list(a["st"]), a["es"]
        if rng.random() < 0.1:
            b["n"][rng.randrange(3)] = 0
        pairs.append((a, b))
    got = ask(pairs)
    wrong = [(p, g, _truth(*p)) for p, g in zip(pairs, got) if g != _truth(*p)]
    assert not wrong, (len(wrong), wrong[0])
    share = sum(g[0] for g in got) / len(got)
    assert 0.2 < share < 0.8  # both answers are met


def test_views_of_one_buffer(ask):
    """Large views: slots of a token-major cache, heads of a packed projection."""
    B, T, H, D = 64, 131072, 8, 128
    cache = dict(p=4096, n=[B, H, T - 1], st=[T * H * D, D, H * D], row=D, es=2)
    last = dict(p=4096 + 2 * (T - 1) * H * D, n=[B, H, 1], st=[T * H * D, D, 1], row=D, es=2)
    q = dict(p=4096, n=[B, 512, 32], st=[512 * 48 * D, 48 * D, D], row=D, es=2)
    k = dict(q, p=4096 + 2 * 32 * D, n=[B, 512, 8])
    off = dict(k, p=k["p"] - 2)
    broadcast = dict(p=4096, n=[B, H, T], st=[0, T * D, D], row=D, es=2)
    swapped = dict(p=4096, n=[B, H, T], st=[D, B * D, B * H * D], row=D, es=2)  # every row once
    got = ask([(cache, last), (last, cache), (cache, dict(last, p=last["p"] - 2)), (q, k), (q, off),
               (broadcast, broadcast), (swapped, last)])
    assert got == [(False, False), (False, False), (True, False), (False, False), (True, False), (True, True),
                   (True, False)]
