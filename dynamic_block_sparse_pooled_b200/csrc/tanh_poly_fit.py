"""Fits the polynomials behind the FMA-pipe tanh of capped attention scores (TanhPoly in
fpx_sm100.cuh, NearTanh in fpx_attn_sm100.cu) and prints their coefficients and error bounds.

Method: tanh(x) = x P(x^2) on [0, HI] with the smallest maximum *absolute* error (an error in a score
is an absolute one), found by Lawson's iteration: least squares on a dense grid, the weights
multiplied by the errors until these equioscillate.  The coefficients are then rounded to fp32 and
the error of an fp32 evaluation is measured.

    python dynamic_block_sparse_pooled_b200/csrc/tanh_poly_fit.py
"""
import numpy as np


def fit(deg, hi, iters=400):
    x = hi * np.sin(np.linspace(0, np.pi / 2, 4001)[1:])
    basis = np.stack([x ** (2 * j + 1) for j in range(deg + 1)], axis=1)
    w = np.full(len(x), 1.0 / len(x))
    best, best_err = None, np.inf
    for _ in range(iters):
        sw = np.sqrt(w)
        c = np.linalg.lstsq(basis * sw[:, None], np.tanh(x) * sw, rcond=None)[0]
        err = np.abs(basis @ c - np.tanh(x))
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
        err = np.abs((p * g).astype(np.float64) - np.tanh(g.astype(np.float64)))
        print(name, ", ".join(f"{float(v):.9e}f" for v in c32))
        print(f"  max absolute error on [0, {hi}]: {e:.2e}, evaluated in fp32: {err.max():.2e}")
