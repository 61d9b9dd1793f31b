"""Newton-Schulz steps in 64 bits, and what their form in fp16 products may be off.

Bounds, over a whole matrix (2-norms relative to the result).  u = 2^-11, half a step of
fp16.  One step X' = a X + P H with H = fp16(X), S = fp16(H H^T), P = fp16(b S + c S S):
each of the three roundings and the operands' own makes an error of relative size u / sqrt(3)
at most (roundings of many entries, evenly spread over their half step, are independent), in
terms whose sizes are |b| s^2 and |c| s^4 for singular values up to s = 1.21.  With the
default coefficients these are below 7 and 4.4 times X, and the sum that they are part of is
X' itself, at least 0.65 X for a direction that has arrived.  Five steps bring most directions
just there.  A later step multiplies what is off by its derivative a + 3 b s^2 + 5 c s^4: -1.1
at s = 0.7, -1.6 at 0.87, -0.7 at 1, 1.7 at 1.13: by 1.5.  In all: (7 (u) + 4.4 (2 u)) / sqrt(3) / 0.65 = 14 u where errors agree in
every direction; over directions that do not agree they add as squares, which leaves less the
wider the matrix is: a third for more than 256 rows, 2.3e-3.  Up to 256 rows S, P and the
products' X have 21 bits: u = 2^-21, without the third.  The result's own rounding to bf16 is
2^-8 of an entry at most; in the norm 2^-8, or over many entries (evenly spread over their
half step) 2^-8 / sqrt(3).
"""
import torch

COEFFICIENTS = (3.4445, -4.7750, 2.0315)


def orth64(G, steps=5, coefficients=COEFFICIENTS):
    X = G.double()
    norm = X.square().sum((-2, -1), keepdim=True).sqrt()
    X = X / torch.where(norm > 0, norm, 1.0)
    a, b, c = coefficients
    for _ in range(steps):
        if X.shape[-2] <= X.shape[-1]:
            S = X @ X.mT
            X = a * X + (b * S + c * S @ S) @ X
        else:
            S = X.mT @ X
            X = a * X + X @ (b * S + c * S @ S)
    return X, norm[..., 0, 0]


def bound(m, n, steps=5):
    steps = 1.5 ** max(0, steps - 5) * (14 * 2.0 ** -21 if min(m, n) <= 256 else 14 * 2.0 ** -11 / 3)
    return (steps ** 2 + (2.0 ** -8) ** 2 / (3 if m * n >= 4096 else 1)) ** 0.5


def hold(got, want, most):
    """2-norms of a matrix, or of each of a batch."""
    off = (got.double() - want).square().sum((-2, -1)).sqrt()
    size = want.square().sum((-2, -1)).sqrt()
    assert torch.isfinite(got).all()
    assert (off <= most * size).all(), (off / size, most)
