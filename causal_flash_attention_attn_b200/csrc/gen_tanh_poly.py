"""Coefficients of the polynomial tanh(y) ~ y (c0 + c1 u + ... + cd u^d), u = y^2, on |y| <= 3/4
used by the packed kernels' score cap (csrc/tanh_poly.cuh, tanh_poly2).

Method: minimax in relative error, computed with the Remez exchange algorithm (Remez 1934) for
g(u) = tanh(sqrt u) / sqrt u on [0, 9/16]. Coefficients are rounded to f32 and the error is
measured again in f32 Horner arithmetic. Run: python gen_tanh_poly.py [degree]
"""
import sys

import numpy as np

LIMIT = 0.75


def g(u):
    y = np.sqrt(np.maximum(u, 1e-300))
    return np.where(u < 1e-12, 1.0 - u / 3.0, np.tanh(y) / y)


def remez_rel(deg, hi=LIMIT * LIMIT, iters=30):
    n = deg + 2
    x = 0.5 * hi + 0.5 * hi * np.cos(np.pi * np.arange(n)[::-1] / (n - 1))
    grid = np.linspace(0.0, hi, 200001)
    for _ in range(iters):
        # p(x_i) - g(x_i) = (-1)^i E g(x_i) for c_0 .. c_deg, E
        A = np.zeros((n, n))
        A[:, :deg + 1] = x[:, None] ** np.arange(deg + 1)
        A[:, deg + 1] = -((-1.0) ** np.arange(n)) * g(x)
        c = np.linalg.solve(A, g(x))[:deg + 1]
        err = np.polyval(c[::-1], grid) / g(grid) - 1.0
        # the new reference: the largest error between two sign changes
        segs = np.split(np.arange(len(grid)), np.where(np.diff(np.sign(err)) != 0)[0] + 1)
        ext = [s[np.argmax(np.abs(err[s]))] for s in segs]
        while len(ext) > n:
            k = int(np.argmin(np.abs(err[ext])))
            ext.pop(k if k in (0, len(ext) - 1) else k)
        if len(ext) < n:
            break
        x = grid[ext]
    return c


def f32_error(c):
    """(max relative error of y * Horner in f32 on (0, LIMIT], f32 coefficients)"""
    c32 = np.asarray(c, dtype=np.float32)
    y = np.linspace(1e-4, LIMIT, 1000001).astype(np.float32)
    u = (y * y).astype(np.float32)
    acc = np.full_like(u, c32[-1])
    for k in range(len(c32) - 2, -1, -1):
        acc = (acc.astype(np.float64) * u + c32[k]).astype(np.float32)
    t = (acc * y).astype(np.float32)
    ref = np.tanh(y.astype(np.float64))
    return float(np.max(np.abs(t.astype(np.float64) - ref) / ref)), c32


if __name__ == "__main__":
    deg = int(sys.argv[1]) if len(sys.argv) > 1 else 5
    err, c32 = f32_error(remez_rel(deg))
    print(f"degree {deg}: max relative error {err:.3e} (f32 Horner)")
    for k, v in enumerate(c32):
        print(f"c{k} = {v:.9e}f")
