"""Derive the polynomial used for 2^f, f in [-1/2, 1/2], by the packed-prompt attention's FMA-pipe exponential
(csrc/prompt.cu, exp2_pair).

2^w = 2^n * 2^f with n = round(w), f = w - n.  The polynomial p of degree 4 has p(0) = 1 exactly, so that w = -127, where
the inputs are clamped, gives exactly 0 when n is added to the exponent field, and the least largest relative error
max |p(f) / 2^f - 1| under that condition: a linear programme in the other four coefficients and the error, on 4,001
points.  Running this script prints the coefficients, rounded to fp32, and the errors of fp32 Horner evaluation; the
kernel's constants must equal the printed ones.
"""
import numpy as np
from scipy.optimize import linprog

DEGREE = 4


def coefficients(degree=DEGREE):
    f = np.linspace(-0.5, 0.5, 4001)
    powers = np.vstack([f ** k / 2.0 ** f for k in range(1, degree + 1)]).T
    rest = 1 - 1 / 2.0 ** f
    one = np.ones((len(f), 1))
    r = linprog(np.eye(degree + 1)[-1], np.vstack([np.hstack([powers, -one]), np.hstack([-powers, -one])]),
                np.hstack([rest, -rest]), bounds=[(None, None)] * degree + [(0, None)], method="highs")
    return np.concatenate([[1.0], r.x[:degree]]).astype(np.float32)


def horner_f32(coef, x):
    x = np.asarray(x, dtype=np.float32)
    p = np.full_like(x, coef[-1])
    for c in coef[-2::-1]:
        p = (p * x + c).astype(np.float32)
    return p


if __name__ == "__main__":
    coef = coefficients()
    f = np.linspace(-0.5, 0.5, 400001).astype(np.float32)
    error = horner_f32(coef, f) / 2.0 ** f.astype(np.float64) - 1
    for k, c in enumerate(coef):
        print(f"c{k} = {float(c).hex()}")
    print(f"relative error: largest {np.abs(error).max():.2e}, mean {error.mean():.2e}")
