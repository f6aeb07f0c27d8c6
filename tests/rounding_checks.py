"""Checks of the token mixers' outputs against the roundings that they are allowed.

A term or result x that is rounded once to a type of unit roundoff u is off by less than
u |x|, evenly spread: 0.735 u |x| / sqrt(3) is the root mean square over mantissas spread
as those of products are.  Roundings of different terms are independent, so an output
whose rounded terms have squares that sum to q (``oracle.mixing.linear_squares``,
``attention_squares``) is off by 0.735 sigma, sigma = u sqrt(q / 3).  Sums in fp32 add 2^-20 of the sum of the terms'
magnitudes at most.  Hence, over all outputs of a call:

  root mean square of the errors <= that of sigma, plus 2^-21 of that of the magnitudes;
  every error <= 8 sigma + 2^-19 of the magnitude + half the smallest subnormal.

A decay or a scale that is some percent off, or a term left out, does not pass
(test_mixing_rounding plants them).
"""
import numpy as np


def rms(x):
    return float(np.sqrt(np.mean(np.square(x))))


def check_roundings(u, got, want, squares, magnitudes):
    sigma = u * np.sqrt(squares / 3.0)
    err = np.abs(got - want)
    limit = rms(sigma) + 2.0 ** -21 * rms(magnitudes)
    assert rms(err) <= limit, f"errors of {rms(err):.3e} where {limit:.3e} is the most"
    tol = 8.0 * sigma + 2.0 ** -19 * magnitudes + 2.0 ** -25
    assert np.all(err <= tol), f"worst {np.max(err / tol):.3f} of the bound"
