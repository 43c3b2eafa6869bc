"""The gated activation in 64 bits and the error bounds of the kernels that
compute it in FP32, shared by the tests of the gated feed-forward operators."""
import math

import numpy as np

ULP = 2.0 ** -24                     # half a step of FP32, relative


def _z(act, g):
    if act == "silu":
        return g, np.ones_like(g)
    c = 2 * math.sqrt(2 / math.pi)
    return c * (g + 0.044715 * g ** 3), c * (1 + 3 * 0.044715 * g * g)


def sigma64(z):
    with np.errstate(over="ignore"):
        return 1 / (1 + np.exp(-z))


def act64(act, g):
    g = np.asarray(g, np.float64)
    return g * sigma64(_z(act, g)[0])


def act_slope64(act, g):
    g = np.asarray(g, np.float64)
    z, dz = _z(act, g)
    s, q = sigma64(z), sigma64(-z)
    return s + g * s * q * dz


# Rounding of the kernels' activation at a given FP32 g.  z is off by at most
# 6 roundings (its constants' included), which moves sigma by sigma (1 - sigma)
# |z| of that; e^-z, 1 + e^-z, the reciprocal and the products are off by at most
# 16 roundings in all.  Below 2^-120 the hardware reciprocal may flush to 0.

def act_error(act, g):
    z, _ = _z(act, g)
    s, q = sigma64(z), sigma64(-z)
    return 16 * ULP * np.abs(g) * s + 6 * ULP * np.abs(g) * s * q * np.abs(z) + np.abs(g) * 2.0 ** -120


def slope_error(act, g):
    z, dz = _z(act, g)
    s, q = sigma64(z), sigma64(-z)
    moved = 6 * ULP * np.abs(z) * s * q * (1 + np.abs(g) * dz)
    return 24 * ULP * (s + np.abs(g) * s * q * dz) + moved + (1 + np.abs(g) * dz) * 2.0 ** -120


def gated_bound(act, g, u, Eg, Eu):
    """|h - act(g) u| when g and u are off by Eg and Eu (the slope of either
    activation lies in [-0.13, 1.13])."""
    a = np.abs(act64(act, g))
    return (np.abs(u) + Eu) * (1.13 * Eg + act_error(act, g)) + a * Eu + 2 * ULP * np.abs(a * u)
