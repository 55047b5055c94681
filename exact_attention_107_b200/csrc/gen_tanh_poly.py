"""Derives the polynomial of tanh behind quartic2(), tanh_any() and quartic_inverse() in sm100_ptx.cuh.

tanh(z) = z g(z^2) with g(u) = tanh(sqrt u) / sqrt u, smooth in u.  The quartic in u that minimises
the maximum *relative* error of g on [0, LIMIT^2] comes from the Remez exchange algorithm
(E. Ya. Remez, 1934) on the weighted Haar system {u^j} / g(u).

    python exact_attention_107_b200/csrc/gen_tanh_poly.py

prints the coefficients and the inverse's chord (as float32 hex), the maximum relative error of the
float32 evaluation and the inverse's error.
The kernels only need the printed values; this script documents where they come from and is not
part of the build.
"""
from __future__ import annotations

import numpy as np

TERMS = 5
LIMIT = 0.75


def g(u):
    r = np.sqrt(np.maximum(u, 1e-30))
    return np.where(u < 1e-12, 1.0 - u / 3.0, np.tanh(r) / r)


def remez_relative(terms: int = TERMS, limit: float = LIMIT, iters: int = 50):
    end = limit * limit
    k = np.arange(terms + 1)
    ref = end * (1.0 - np.cos(np.pi * k / terms)) / 2.0
    grid = np.linspace(0.0, end, 200001)
    coef = None
    for _ in range(iters):
        A = np.concatenate([np.stack([ref ** j for j in range(terms)], 1) / g(ref)[:, None],
                            -((-1.0) ** k)[:, None]], axis=1)
        coef = np.linalg.solve(A, np.ones(terms + 1))[:terms]
        err = np.polynomial.polynomial.polyval(grid, coef) / g(grid) - 1.0
        runs = np.split(np.arange(len(grid)), np.where(np.diff(np.sign(err)) != 0)[0] + 1)
        ext = [r[np.argmax(np.abs(err[r]))] for r in runs]
        if len(ext) != terms + 1 or np.allclose(grid[ext], ref):
            break
        ref = grid[ext]
    return coef


def eval_f32(z: np.ndarray, c: np.ndarray) -> np.ndarray:
    """The kernels' steps in float32 (each product and sum rounded; the kernels' fused steps round less)."""
    z = z.astype(np.float32)
    c = c.astype(np.float32)
    u = z * z
    p = np.full_like(z, c[-1])
    for a in c[-2::-1]:
        p = p * u + a
    return z * p


def chord(c: np.ndarray):
    """Where quartic_inverse starts: the polynomial's value at LIMIT, and the slope of the chord of its
    inverse from there to 1."""
    z = np.polynomial.Polynomial(np.stack([np.zeros(len(c)), c.astype(np.float64)], 1).ravel())
    at = z(LIMIT)
    one = min(r.real for r in (z - 1.0).roots() if abs(r.imag) < 1e-12 and r.real > LIMIT)
    return np.float32(at), np.float32((one - LIMIT) / (1.0 - at))


def inverse_f32(t: np.ndarray, c: np.ndarray) -> np.ndarray:
    """quartic_inverse's steps in float32: three Newton steps from the chord."""
    t, c = t.astype(np.float32), c.astype(np.float32)
    at, slope = chord(c)
    z = (t - at) * slope + np.float32(LIMIT)
    for _ in range(3):
        u = z * z
        p, d = np.full_like(z, c[-1]), np.full_like(z, np.float32(2 * TERMS - 1) * c[-1])
        for j in range(TERMS - 2, -1, -1):
            p, d = p * u + c[j], d * u + np.float32(2 * j + 1) * c[j]
        z = z - (z * p - t) / d
    return z


if __name__ == "__main__":
    c = remez_relative()
    c32 = c.astype(np.float32)
    for j, v in enumerate(c32):
        print(f"constexpr float kTanhC{j} = {v:.17f}f;   // 0x{v.tobytes()[::-1].hex()}")
    for name, v in zip(("kTanhAtLimit", "kTanhChord"), chord(c32)):
        print(f"constexpr float {name} = {v:.17f}f;   // 0x{v.tobytes()[::-1].hex()}")
    z = np.linspace(1e-6, LIMIT, 1_000_001).astype(np.float32)
    rel = np.abs(eval_f32(z, c32).astype(np.float64) / np.tanh(z.astype(np.float64)) - 1.0)
    print(f"max relative error over (0, {LIMIT}]: {rel.max():.3e}")
    t = np.linspace(float(chord(c32)[0]), 1.0, 1_000_001).astype(np.float32)
    back = inverse_f32(t, c32).astype(np.float64)
    value = back * np.polynomial.polynomial.polyval(back * back, c32.astype(np.float64))
    print(f"max error of the polynomial at its inverse: {np.abs(value - t).max():.3e}")
