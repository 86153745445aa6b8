"""Writes exp2_poly.h: coefficients of the cubic c0 + c1 f + c2 f^2 + c3 f^3
that approximates 2^f on [-1/2, 1/2] with the smallest maximum RELATIVE
error (minimax, found by the Remez exchange algorithm in float64).

Used by the prefill kernel to compute part of its exponentials on the FMA
pipe (Cody-Waite style: 2^x = 2^j * 2^f with j = rint(x), f = x - j), so
that the special-function unit is not the bottleneck.  Run:
    python query_adaptive_chunk_b200/csrc/gen_exp2_poly.py
"""
import os

import numpy as np

DEG = 3
LO, HI = -0.5, 0.5


def remez(deg=DEG, iters=30):
    n = deg + 2
    k = np.arange(n)
    x = 0.5 * (LO + HI) + 0.5 * (HI - LO) * np.cos(np.pi * (n - 1 - k) / (n - 1))  # Chebyshev extrema
    grid = np.linspace(LO, HI, 200001)
    for _ in range(iters):
        # p(x_i) - 2^x_i = (-1)^i E 2^x_i  (equi-oscillating relative error)
        A = np.zeros((n, n))
        for i in range(n):
            A[i, :deg + 1] = x[i] ** np.arange(deg + 1)
            A[i, deg + 1] = -((-1) ** i) * 2.0 ** x[i]
        sol = np.linalg.solve(A, 2.0 ** x)
        c = sol[:deg + 1]
        err = np.polyval(c[::-1], grid) / 2.0 ** grid - 1.0
        # new reference: the extrema of err in each sign run
        s = np.sign(err)
        idx = []
        start = 0
        for i in range(1, len(grid) + 1):
            if i == len(grid) or s[i] != s[start]:
                seg = slice(start, i)
                idx.append(start + int(np.argmax(np.abs(err[seg]))))
                start = i
        if len(idx) < n:
            break
        # keep the n largest alternating extrema
        while len(idx) > n:
            e = np.abs(err[idx])
            drop = 0 if e[0] < e[-1] else len(idx) - 1
            idx.pop(drop)
        x = grid[idx]
    return c, float(np.max(np.abs(err)))


def main():
    c, e = remez()
    path = os.path.join(os.path.dirname(os.path.abspath(__file__)), "exp2_poly.h")
    with open(path, "w") as f:
        f.write("// Generated by gen_exp2_poly.py: minimax (relative error) cubic for 2^f,\n")
        f.write(f"// f in [-1/2, 1/2], Remez exchange in float64; max relative error {e:.3e}.\n")
        f.write("#pragma once\n")
        for i, v in enumerate(c):
            f.write(f"#define CSA_EXP2_C{i} {np.float32(v)!r}f\n".replace("np.float32(", "").replace(")f", "f"))
    print(path, c, e)


if __name__ == "__main__":
    main()
