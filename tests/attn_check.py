"""Shared by the attention tests: the tolerance, from the arithmetic, and the comparison.

A value o = sum p v with the total magnitude S = sum p |v| (p the softmax
weights) is off by at most
  2^-8 |o|        its rounding to bf16,
  2^-8 (S + |o|)  every weight's rounding to bf16 before the second product; the
                  same rounded weights are summed for the division, so a weight
                  off by d_j (at most 2^-8 of it) gives sum p_j d_j (v_j - o),
  2 e S           the scores' error e, in the weights and in their sum: a score
                  is a sum of d products of magnitude at most |q| |k| (Cauchy) in
                  fp32, scaled by one product: e = (d + 4) 2^-24 scale |q| |k|,
                  plus 2^-22 for the exponential,
  (n/8 + 64) 2^-24 S   the fp32 sums over n tokens, in steps of 32 on the matrix
                  core (at most 4 roundings a step) and the joining of parts,
  n 2^-118 max|v| weights too small for fp32: the row's largest weight is kept as
                  1 .. 2^8 (the running reference trails the maximum by at most
                  8 binades), so the sum is at least 1; a weight that fp32 loses
                  is below 2^-126, or, lost when parts are joined, below 2^-126
                  times the 2^8 that its part may hold it scaled by.
"""
from __future__ import annotations

import numpy as np

import workloads as W
from oracle import formats as FM


def tolerance(ref, size, d, n, scale, q_norm, k_norm, v_max):
    e = (d + 4) * 2.0 ** -24 * abs(scale) * q_norm * k_norm + 2.0 ** -22
    return 2.0 ** -7 * np.abs(ref) + (2.0 ** -8 + 2 * e + (n / 8 + 64) * 2.0 ** -24) * size + n * 2.0 ** -118 * v_max


def check(out, ref, size, d, n, scale, q_norm, k_norm, v_max):
    """out: bf16 tensor; ref NaN where nothing is written (not compared)."""
    tol_all = tolerance(ref, size, d, n, scale, q_norm, k_norm, v_max)
    got = FM.bf16_bits_to_f64(W.bf16_bits(out))
    live = ~np.isnan(ref)
    err = np.abs(got - ref)[live]
    tol = tol_all[live]
    bad = ~(err <= tol)
    if bad.any():
        at = np.argwhere(live)[np.argmax(np.where(bad, np.nan_to_num(err / np.maximum(tol, 1e-300), nan=np.inf), 0))]
        raise AssertionError(f"{bad.sum()} of {err.size} values off; worst at {tuple(at)}: got {got[tuple(at)]}, "
                             f"expected {ref[tuple(at)]}, tolerance {tol_all[tuple(at)]}")


def norm(bits):
    """Largest length of a head vector (bf16 bits [..., d])."""
    x = FM.bf16_bits_to_f64(bits)
    return float(np.sqrt((x * x).sum(-1)).max(initial=0.0))
