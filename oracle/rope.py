"""Rotary position embedding in float64, one (token, head) row at a time.

TEST INFRASTRUCTURE (oracle): see the package docstring.

Pair p of a row at position t, seen as the complex number a + ib, is multiplied by
m exp(i t f_p); (a, b) = (x[p], x[p + rot/2]) in the half layout, (x[2p], x[2p+1]) in the
interleaved one; the elements from rot on pass through.  The angle is formed from the exact
integer part of t f_p / 2 pi taken out with rational arithmetic, so it is good for any int32
position.
"""

import math
from fractions import Fraction

import numpy as np

# pi to 60 digits
_PI = Fraction("3.14159265358979323846264338327950288419716939937510582097494")


def angle(position, freq):
    """position * freq reduced to [-pi, pi], from exact rational arithmetic."""
    turns = Fraction(int(position)) * Fraction(float(freq)) / (2 * _PI)
    frac = turns - round(turns)
    return float(2 * _PI * frac)


def frequencies(rot, theta, scaling="none", factor=1.0, original=0, low=1.0, high=4.0):
    """Radians per position of each pair and the factor of cosine and sine."""
    out, m = [], 1.0
    if scaling == "yarn":
        m = 0.1 * math.log(factor) + 1.0 if factor > 1 else 1.0
        pair = lambda turns: rot * math.log(original / (2 * math.pi * turns)) / (2 * math.log(theta))
        a, b = max(math.floor(pair(high)), 0), min(math.ceil(pair(low)), rot - 1)
    for p in range(rot // 2):
        f = theta ** (-2.0 * p / rot)
        if scaling == "none":
            g = f
        elif scaling == "linear":
            g = f / factor
        elif scaling == "ntk":
            g = (theta * factor ** (rot / (rot - 2.0))) ** (-2.0 * p / rot)
        elif scaling == "wavelength":
            wave = 2 * math.pi / f
            if wave > original / low:
                g = f / factor
            elif wave < original / high:
                g = f
            else:
                t = (original / wave - low) / (high - low)
                g = (1 - t) * f / factor + t * f
        elif scaling == "yarn":
            t = min(max((p - a) / max(b - a, 0.001), 0.0), 1.0)
            g = t * f / factor + (1 - t) * f
        else:
            raise ValueError(scaling)
        out.append(g)
    return np.array(out, np.float64), m


def rotate(x, positions, freqs, layout="half", m=1.0):
    """x float64 [T, H, D] -> rotated float64 [T, H, D]."""
    x = np.asarray(x, np.float64)
    out = x.copy()
    n = len(freqs)
    for t, pos in enumerate(positions):
        ang = [angle(pos, f) for f in freqs]
        w = m * np.array([complex(math.cos(a), math.sin(a)) for a in ang])
        for h in range(x.shape[1]):
            row = x[t, h]
            z = (row[:n] + 1j * row[n:2 * n] if layout == "half" else row[0:2 * n:2] + 1j * row[1:2 * n:2]) * w
            if layout == "half":
                out[t, h, :n], out[t, h, n:2 * n] = z.real, z.imag
            else:
                out[t, h, 0:2 * n:2], out[t, h, 1:2 * n:2] = z.real, z.imag
    return out
