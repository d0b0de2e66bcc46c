"""Fits the polynomial behind the FMA-pipe tanh of capped attention scores (TanhPoly in
fpx_sm100.cuh) and prints its coefficients and error bound.

Method: tanh(x) = x P(x^2) on [0, 0.85], P of degree 5 with the smallest maximum *absolute* error (an
error in a score is an absolute one), found with the Remez exchange algorithm (equioscillation on 7
alternation points).  The coefficients are then rounded to fp32 and the error of an fp32 evaluation
is measured on a dense grid.

    python dynamic_block_sparse_pooled_b200/csrc/tanh_poly_fit.py
"""
import numpy as np

DEG = 5
HI = 0.85


def remez(deg=DEG, iters=40):
    n = deg + 2
    x = HI * np.cos(np.pi * (np.arange(n) + 0.5) / (2 * n))[::-1]
    grid = np.linspace(1e-9, HI, 400001)
    for _ in range(iters):
        a = np.zeros((n, n))
        for i in range(n):
            a[i, :deg + 1] = x[i] ** (2 * np.arange(deg + 1) + 1)
            a[i, deg + 1] = (-1) ** i
        c = np.linalg.solve(a, np.tanh(x))[:deg + 1]
        err = np.tanh(grid) - grid * np.polyval(c[::-1], grid ** 2)
        turn = np.where(np.diff(np.sign(np.diff(err))) != 0)[0] + 1
        ext = np.append(turn, len(grid) - 1)
        ext = np.sort(ext[np.argsort(-np.abs(err[ext]))[:n]])
        if len(ext) < n or np.allclose(grid[ext], x, rtol=1e-9):
            break
        x = grid[ext]
    return c


if __name__ == "__main__":
    c32 = remez().astype(np.float32)
    g = np.linspace(0, HI, 1000001).astype(np.float32)
    u = g * g
    p = np.full_like(g, c32[DEG])
    for k in range(DEG - 1, -1, -1):
        p = p * u + c32[k]
    err = np.abs((p * g).astype(np.float64) - np.tanh(g.astype(np.float64)))
    for k, v in enumerate(c32):
        print(f"C{k} = {float(v):.15e}f  ({v.view(np.uint32):#010x})")
    print(f"max absolute error on [0, 0.85] with fp32 coefficients: {err.max():.3e}")
