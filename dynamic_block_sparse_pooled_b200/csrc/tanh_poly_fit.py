"""Fits the polynomials behind the FMA-pipe tanh of capped attention scores (TanhPoly in
fpx_sm100.cuh, NearTanh in fpx_softmax.cuh) and prints their coefficients and error bounds.

Method: tanh(x) = x P(x^2) on [0, HI] with the smallest maximum *relative* error, found by Lawson's
iteration: least squares on a dense grid, the weights multiplied by the errors until these
equioscillate.  (The smallest absolute error would leave P(0) 2.3e-6 off for degree 3, and a score
far below its cap with it: its absolute error is that times the score, whatever the cap.)  The
coefficients are then rounded to fp32 and the error of an fp32 evaluation is measured.

    python dynamic_block_sparse_pooled_b200/csrc/tanh_poly_fit.py
"""
import numpy as np


def fit(deg, hi, iters=400):
    x = hi * np.sin(np.linspace(0, np.pi / 2, 4001)[1:])
    basis = np.stack([x ** (2 * j + 1) / np.tanh(x) for j in range(deg + 1)], axis=1)
    w = np.full(len(x), 1.0 / len(x))
    best, best_err = None, np.inf
    for _ in range(iters):
        sw = np.sqrt(w)
        c = np.linalg.lstsq(basis * sw[:, None], sw, rcond=None)[0]
        err = np.abs(basis @ c - 1.0)
        if err.max() < best_err:
            best, best_err = c, err.max()
        w = w * err
        w /= w.sum()
    return best, best_err


if __name__ == "__main__":
    for name, deg, hi in (("TanhPoly", 5, 0.85), ("NearTanh", 3, 0.5)):
        c, e = fit(deg, hi)
        c32 = c.astype(np.float32)
        g = np.linspace(0, hi, 1000001).astype(np.float32)
        u = g * g
        p = np.full_like(g, c32[deg])
        for k in range(deg - 1, -1, -1):
            p = (p.astype(np.float64) * u + c32[k]).astype(np.float32)  # as a fused multiply-add
        exact = np.tanh(g[1:].astype(np.float64))
        err = np.abs((p * g)[1:].astype(np.float64) - exact)
        print(name, ", ".join(f"{float(v):.9e}f" for v in c32))
        print(f"  max relative error on [0, {hi}]: {e:.2e}, evaluated in fp32: "
              f"{(err / exact).max():.2e} (absolute {err.max():.2e})")
