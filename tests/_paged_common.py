"""What tells a lost or misweighted part of a long context from rounding, in the output of
paged attention.

Elementwise, with A = sum_j w_j |v_j|: the weights' rounding to bf16 moves an output by at
most 2^-8 A (the normaliser sums the weights before it), the result's own rounding by 2^-8 |out|, and
a score that is off by s by 2 s A (test_gpu_paged.py derives s and the 2^-12). With values of
random sign A is far larger than the output, and a whole visit of 128 keys disappears in that. So

- coded values: those of a block of 128 keys are zero but in one column of D. A column then sums the
  weights of one block in D, A is the output itself, and a block that is lost or counted
  twice changes it by its own size;
- random values by their relative L2 error per row and head: the weights' roundings, at most 2^-8 of each,
  are independent, so the error is some 2^-8 / 2 of the output, which is as random a
  sum, and its own rounding adds as much: 2.3e-3 together. The bar of 1e-2 is four times that, far beyond what
  the norm of 64 columns and more strays, and a visit of 128 of n keys makes sqrt(128 / n): 0.08 at 20,000."""
import numpy as np

RELATIVE = 1e-2


def coded_values(n, Hkv, D):
    """(n, Hkv, D): block b of 128 keys holds 1 to 4 in column (b + 7 h) % D."""
    b = np.arange(n) // 128
    v = np.zeros((n, Hkv, D), np.float32)
    for h in range(Hkv):
        v[np.arange(n), h, (b + 7 * h) % D] = 1 + (b // D) % 4
    return v


def tolerance(want, A, Z):
    score = 10 * 2.0 ** -23 * Z
    return (2.0 ** -8 + 2.0 ** -12 + 2 * score[..., None]) * A + 2.0 ** -8 * np.abs(want)


def relative(got, want):
    """Per row and head."""
    n = np.linalg.norm(want, axis=-1)
    return np.linalg.norm(got - want, axis=-1) / np.where(n > 0, n, 1)
