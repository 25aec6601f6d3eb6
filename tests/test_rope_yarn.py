"""Frequencies scaled by parts ("yarn"), at lengths and borders where no pair turns fast enough, without a GPU."""
from __future__ import annotations

import math

import pytest


@pytest.fixture(scope="module")
def K():
    import verify_kda_decode_gb300 as K
    return K


def radians(r):
    return [t % 2 ** 64 / 2 ** 64 * 2 * math.pi for t in r.turns.tolist()]


@pytest.mark.parametrize("original_len,beta_fast,beta_slow", [(4, 32.0, 1.0), (6, 32.0, 1.0), (7, 32.0, 1.0), (1, 32.0, 1.0), (64, 32.0, 1.0), (512, 200.0, 100.0),
                                                              (4096, 5000.0, 1000.0), (4096, 32.0, 1.0), (4096, 1.0, 1.0), (10 ** 7, 32.0, 1.0), (10 ** 30, 32.0, 1.0)])
@pytest.mark.parametrize("rot", [16, 64, 128])
def test_parts(K, rot, original_len, beta_fast, beta_slow):
    """Divided where a pair turns less than beta_slow times in original_len positions, kept where more than beta_fast times, between
    the two elsewhere, and never closer to kept as pairs get slower."""
    base, factor = 10000.0, 8.0
    r = K.KdaRope.make(rot, base, "yarn", factor, original_len, beta_fast, beta_slow, device="cpu")
    last = 1.0
    for i, f in enumerate(radians(r)):
        plain = base ** (-2.0 * i / rot)
        turns = original_len * plain / (2 * math.pi)
        # turns are fractions of 2^-64: 2^-65 of a turn each, and 64-bit floats on both sides
        tol = 2.0 ** -62 + 1e-13 * plain
        kept = (f - plain / factor) / (plain - plain / factor)
        assert -tol <= f - plain / factor and f - plain <= tol
        if turns < beta_slow * (1 - 1e-9):
            assert abs(f - plain / factor) <= tol, (i, turns, kept)
        if turns > beta_fast * (1 + 1e-9):
            assert abs(f - plain) <= tol, (i, turns, kept)
        assert kept <= last + 1e-9
        last = kept


def test_refusals(K):
    for bad in (dict(beta_fast=0.5), dict(beta_fast=32.0, beta_slow=33.0), dict(original_len=512, beta_slow=100.0), dict(beta_slow=0.0), dict(original_len=math.inf), dict(beta_fast=math.inf),
                dict(original_len=math.nan)):
        with pytest.raises(ValueError):
            K.KdaRope.make(64, scaling="yarn", factor=4.0, device="cpu", **bad)
