"""What the attention over 8-bit caches may be off by, per element and for a row at a time.

With w_j the exact weights (sum 1) and s the gate, the attention's output is

    s sum_j (w_j (1 + d_j) + a_j) e^(x_j) v_j / sum_j w_j e^(x_j) (1 + r)

d_j, a_j: a weight goes to the tensor cores as two e4m3 parts, scaled by powers of two so that the
largest weight among its 32 keys is at most 256. The first part is off by at most half a step, 2^-4
of the weight's power of two 2^e; a remainder below 2^(e-4) has 4 significant bits too, so what is
left is at most 2^(e-9): |d_j| <= 2^-9. Where the second part, 32 times the remainder, falls under
the normal codes, its half step is 2^-10: |a_j| <= 2^-15 / 128 = 2^-22 of the largest of the 32.
r: the output's rounding, |r| <= 2^-8.
x_j: the score's error in natural units, at most the query's (2^-17 of its row's largest magnitude in
each dim) times the key's 1-norm / 16, and fp32 sums of 512 products (2^-15 of their magnitudes'
sum). Both sums see it: 2 x. Exponentials, fp32 sums and the gate: under 2^-10 together.

An element is off by at most (2^-9 + 2 x + 2^-10) mass + 2^-22 rest + 2^-8 |out|, with mass = s sum_j
w_j |v_j| and rest = s sum over blocks of 32 of (largest w_j) (sum of |v_j|).
A row's 256 outputs together, where values are drawn independently of the weights: 2^-8 for the
outputs' rounding, 1.5 x 2^-9 for the weights' (tests/q4_bounds.py), 2^-9 for the rest.
"""
import numpy as np

ROW_BOUND = 1.75 * 2.0 ** -8 + 2.0 ** -9


def score_error(q, k):
    """The largest x_j of queries q [..., 256] against keys k [n, 256]."""
    if len(k) == 0:
        return 0.0
    k1 = float(np.abs(k).sum(-1).max())
    return (2.0 ** -17 + 2.0 ** -15) * float(np.abs(q).max()) * k1 / 16


def allowed(want, mass, x, rest):
    return (2.0 ** -9 + 2 * x + 2.0 ** -10) * mass + 2.0 ** -22 * rest + 2.0 ** -8 * np.abs(want) + 1e-30


def rest_of(q, gate, k, v, length):
    """`rest` of one sequence: q, gate [R, 24, 256]; k, v [>= length + R, 2, 256]; float64."""
    out = np.zeros(q.shape)
    for r in range(q.shape[0]):
        n = length + r + 1
        pad = -n % 32
        for kv in range(2):
            hs = slice(12 * kv, 12 * kv + 12)
            s = q[r, hs] @ k[:n, kv].T / 16
            w = np.exp(s - s.max(-1, keepdims=True))
            w /= w.sum(-1, keepdims=True)
            top = np.pad(w, ((0, 0), (0, pad))).reshape(12, -1, 32).max(-1)
            mags = np.pad(np.abs(v[:n, kv]), ((0, pad), (0, 0))).reshape(-1, 32, 256).sum(1)
            out[r, hs] = top @ mags
    return out / (1 + np.exp(-gate))
