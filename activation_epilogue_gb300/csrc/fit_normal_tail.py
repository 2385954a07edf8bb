"""Fit of the standard normal tail that the epilogue of the 4-bit products takes for GELU.

    Phi(-a) = t 2^(P(t) - a^2 / (2 ln 2)),   t = 1 / (1 + 0.4 a),   0 <= a <= 13,

with the variable t of Hastings' approximations ("Approximations for Digital Computers", 1955)
and the polynomial in the exponent, so that the relative error stays small into the tail:
GELU(v) = max(v, 0) - |v| Phi(-|v|).  P has degree 8, fitted by least squares at Chebyshev
nodes with weights that grow where the error is largest (Lawson's iteration).  In fp32 the
relative error is below 6e-7 for a < 2, 1.3e-6 for a < 5 and 8e-6 up to 13 (the rounding of
a^2), and GELU is off by 7e-8 at most.  Past the fitted range, up to 14.4, where the tail leaves
fp32, the fit itself stays within 1.1e-7.

Run it to reprint the constants that w4_unpack.cuh holds (scipy, numpy; a second):

    python activation_epilogue_gb300/csrc/fit_normal_tail.py
"""
import numpy as np
from scipy.special import log_ndtr

C, DEGREE, LARGEST = 0.4, 8, 13.0


def fit(nodes=4000, rounds=60):
    t0 = 1 / (1 + C * LARGEST)
    t = t0 + (1 - t0) * (np.cos((np.arange(nodes) + 0.5) * np.pi / nodes) + 1) / 2
    a = (1 / t - 1) / C
    want = log_ndtr(-a) / np.log(2) + a * a / (2 * np.log(2)) - np.log2(t)
    powers = np.vander(t, DEGREE + 1, increasing=True)
    weights = np.ones(nodes) / nodes
    for _ in range(rounds):
        root = np.sqrt(weights)
        p = np.linalg.lstsq(powers * root[:, None], want * root, rcond=None)[0]
        error = np.abs(powers @ p - want)
        weights *= error / error.max() + 1e-3
        weights /= weights.sum()
    return p, error.max() * np.log(2)


if __name__ == "__main__":
    p, error = fit()
    print(f"largest relative error before rounding {error:.1e}")
    for i, v in enumerate(p.astype(np.float32)):
        print(f"t^{i}: {v:.9g}f")
